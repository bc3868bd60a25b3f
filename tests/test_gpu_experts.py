"""GPU parity of the calls that run a mixture of experts' linears: the plan,
the quantizer into expert order, the products by expert and the sum back to
token order.

References: the plan against a stable argsort; codes and scales against the
oracle's quantizer, bit for bit; products against the binary64 product of the
oracle's dequantized operands with the tolerance of gpu_util.gemm_close
(products exact in the tensor core, fp32 sums); the sum against binary64, the
bound counting its fp32 roundings (topk FMAs, each off by at most 2^-24 of the
partial sum, which no term sum of magnitudes is below) and the final one."""
import numpy as np
import pytest
import torch

import workloads
from gpu_util import dev, gemm_close, host_values, mma_offset, nasty_matrix

pytestmark = pytest.mark.gpu

MXFP8, MXFP4, NVFP4, INT8_ROW, FP8_TENSOR = 0, 1, 2, 5, 6
FMTS = (MXFP8, MXFP4, NVFP4, INT8_ROW, FP8_TENSOR)
BLOCK = {MXFP8: 32, MXFP4: 32, NVFP4: 16}


@pytest.fixture(scope="module")
def mxq():
    import microscaling_bit_quantization_b200 as m
    assert torch.cuda.is_available() and m.lib().mxq_device_supported(0) == 1
    m.check()
    return m


# ------------------------------------------------------------------ plan

def ref_plan(ids, n):
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < n)
    key = np.where(ok, flat, n)
    order = np.argsort(key, kind="stable")
    place = np.empty(flat.size, np.int64)
    place[order] = np.arange(flat.size)
    counts = np.bincount(key.astype(np.int64), minlength=n + 1)[:n]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    return offsets.astype(np.int32), np.where(ok, place, -1).astype(np.int32).reshape(ids.shape)


def check_plan(mxq, ids, n, dtype):
    plan = mxq.expert_plan(torch.from_numpy(ids).to(dtype).cuda(), n)
    off, slot = ref_plan(ids, n)
    np.testing.assert_array_equal(plan.offsets.cpu().numpy(), off)
    np.testing.assert_array_equal(plan.slot.cpu().numpy(), slot)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,topk,n", [(0, 4, 8), (1, 1, 1), (1, 8, 64), (5, 3, 512), (31, 1, 2), (33, 2, 33),
                                           (512, 8, 128), (513, 8, 128), (4097, 1, 7), (2049, 3, 512), (40000, 8, 256),
                                           (70001, 1, 3)])
def test_plan(mxq, tokens, topk, n, dtype):
    rng = np.random.default_rng(tokens + n)
    ids = rng.integers(0, n, (tokens, topk))
    check_plan(mxq, ids, n, dtype)
    ids[rng.random((tokens, topk)) < 0.2] = -1
    ids[rng.random((tokens, topk)) < 0.05] = n            # no such expert
    check_plan(mxq, ids, n, dtype)


@pytest.mark.parametrize("rows", [4096, 4098, 5120, 74 * 1024 - 1, 74 * 1024, 74 * 1024 + 1, 74 * 2048 + 1, 300007])
def test_plan_block_boundaries(mxq, rows):
    """Sizes at which the number of blocks, or of a block's rounds, changes."""
    ids = np.random.default_rng(rows).integers(-1, 300, (rows, 1))
    check_plan(mxq, ids, 300, torch.int64 if rows & 1 else torch.int32)


def test_plan_one_expert_none_and_far_ids(mxq):
    check_plan(mxq, np.full((3000, 2), 5), 9, torch.int32)
    check_plan(mxq, np.full((9000, 2), 5), 9, torch.int64)
    check_plan(mxq, np.full((9000, 2), -1), 9, torch.int32)
    far = np.array([[2 ** 32, 1], [2 ** 40 + 3, -2 ** 33], [0, 2 ** 31]])
    check_plan(mxq, far, 4, torch.int64)                  # ids whose low 32 bits name an expert


# ------------------------------------------------------------------ quantize into expert order

def routing(rng, tokens, topk, n, drop=0.1):
    ids = np.stack([rng.permutation(n)[:topk] for _ in range(tokens)]) if tokens else np.zeros((0, topk), np.int64)
    ids[rng.random(ids.shape) < drop] = -1
    return ids


def scale_rows(off, rows):
    """Grouped scale row of every row in expert order, by walking the groups."""
    out, tile = np.zeros(rows, np.int64), 0
    for lo, hi in zip(off[:-1], off[1:]):
        out[lo:hi] = 128 * tile + np.arange(hi - lo)
        tile += (hi - lo + 127) // 128
    return out


def check_grouped(q, oq, fmt, off, src, fill):
    """Rows of q in expert order against rows src of the oracle's oq; everything else still `fill`."""
    used = int(off[-1])
    codes = q.codes.cpu().numpy().reshape(q.rows, -1)
    np.testing.assert_array_equal(codes[:used], oq.codes.view(np.uint8).reshape(oq.rows, -1)[src])
    assert (codes[used:] == fill).all()
    if fmt in BLOCK:
        sp = (q.cols // BLOCK[fmt] + 15) // 16 * 16
        buf = q.scales.cpu().numpy()
        at = mma_offset(scale_rows(off, q.rows)[:used, None], np.arange(q.cols // BLOCK[fmt])[None], sp)
        np.testing.assert_array_equal(buf[at], oq.scales[src])
    elif fmt == INT8_ROW:
        s = q.scales.cpu().view(torch.float32).numpy()
        np.testing.assert_array_equal(s[:used].view(np.uint32), oq.scales[src].view(np.uint32))
        assert (q.scales.cpu().numpy().reshape(-1, 4)[used:] == fill).all()
    if fmt in (NVFP4, FP8_TENSOR):
        np.testing.assert_array_equal(np.float32(q.tensor_scale.item()), np.float32(oq.tensor_scale))


def filled(mxq, fmt, rows, groups, cols, fill=0xFF):
    q = mxq.alloc_grouped(fmt, rows, groups, cols)
    q.codes.fill_(fill)
    if q.scales is not None:
        q.scales.fill_(fill)
    return q


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,topk,n,cols,had,dtype", [
    (37, 3, 5, 64, 0, "bf16"), (1, 8, 64, 1152, 32, "f32"), (150, 1, 2, 576, 0, "f32"), (300, 4, 7, 4608, 0, "bf16"),
    (64, 2, 300, 192, 64, "bf16"), (9, 2, 3, 5120, 256, "bf16"), (33, 32, 40, 64, 16, "f32")])
def test_quantize_grouped(mxq, orc, fmt, tokens, topk, n, cols, had, dtype):
    rng = np.random.default_rng(tokens * 7 + fmt)
    x = nasty_matrix(fmt + tokens, tokens, cols)
    ids = routing(rng, tokens, topk, n)
    ids[0, 0] = 1
    if tokens > 8:
        ids[7] = -1                                       # a padded token: its values reach nothing
    off, slot = ref_plan(ids, n)
    placed = (slot >= 0).any(1)
    vals = host_values(x, dtype)
    xd = dev(x, dtype)
    xd[torch.from_numpy(~placed).cuda()] = float("nan")
    q = filled(mxq, fmt, tokens * topk, n, cols)
    out = mxq.quantize_grouped(xd, fmt, torch.from_numpy(off).cuda(), torch.from_numpy(slot).cuda(), had, out=q)
    assert out is q and mxq.check() == 0
    src = np.zeros(int(off[-1]), np.int64)
    compact = np.cumsum(placed) - 1                       # row among the placed tokens
    for t, i in zip(*np.nonzero(slot >= 0)):
        src[slot[t, i]] = compact[t]
    # every bit as mxq_quantize writes it, for the tokens that have a row
    lib = mxq.quantize(dev(vals[placed], dtype), fmt, had)
    sc = None if lib.scales is None else lib.scales.cpu().numpy()
    oq = orc.quantize(vals[placed], fmt, had)
    same = Bits(lib.codes.cpu().numpy().reshape(oq.rows, -1),
                sc.reshape(oq.rows, -1) if fmt in BLOCK else None if sc is None else sc.view(np.float32),
                None if lib.tensor_scale is None else lib.tensor_scale.item(), oq.rows)
    check_grouped(q, same, fmt, off, src, 0xFF)
    # and as the oracle has them.  The matrix holds blocks of values near 3e38: 32 of them added by a rotation of 64
    # or 256 pass the largest fp32 value (3.4e38), and the definition, fp32 butterflies, then gives infinities and
    # their differences, NaN, whose maximum the definition does not name; such rows have no oracle value
    finite = np.ones(oq.rows, bool)
    if had:
        with np.errstate(over="ignore", invalid="ignore"):
            finite = np.isfinite(orc.hadamard(vals[placed], had)).all(1)
    if finite.all():
        check_grouped(q, oq, fmt, off, src, 0xFF)
    elif fmt not in (NVFP4, FP8_TENSOR):                  # there one such row decides the scale of all
        for a, b in ((same.codes, oq.codes.view(np.uint8).reshape(oq.rows, -1)), (same.scales, oq.scales)):
            np.testing.assert_array_equal(a[finite], b[finite])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("off", [[0, 6, 3, 8], [0, 3, 6, 9], [-1, 3, 6, 8]])
def test_quantize_reports_wrong_offsets(mxq, fmt, off):
    """Offsets out of order or outside the 8 rows: reported by every format, nothing written past the buffers."""
    x = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    q = filled(mxq, fmt, 8, 3, 64)
    guard = torch.full((q.codes.numel() + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    q.codes = guard[:q.codes.numel()]
    mxq.quantize_grouped(x, fmt, torch.tensor(off, dtype=torch.int32, device="cuda"), out=q)
    assert mxq.check() == 1 and mxq.check() == 0
    assert (guard[q.codes.numel():] == 0xAB).all()


class Bits:
    def __init__(self, codes, scales, tensor_scale, rows):
        self.codes, self.scales, self.tensor_scale, self.rows = codes, scales, tensor_scale, rows


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_rows_in_order_and_empty(mxq, orc, fmt):
    rng = np.random.default_rng(fmt)
    off = np.array([0, 0, 130, 131, 131, 200], np.int32)
    x = rng.standard_normal((230, 256)).astype(np.float32)
    xd = dev(x, "bf16")
    xd[200:] = float("nan")                               # rows behind the last group
    q = filled(mxq, fmt, 230, 5, 256)
    mxq.quantize_grouped(xd, fmt, torch.from_numpy(off).cuda(), out=q)
    assert mxq.check() == 0
    check_grouped(q, orc.quantize(host_values(x, "bf16")[:200], fmt), fmt, off, np.arange(200), 0xFF)
    none = filled(mxq, fmt, 6, 3, 64)
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    mxq.quantize_grouped(xd[:3, :64].contiguous(), fmt, zero, torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), out=none)
    assert mxq.check() == 0 and (none.codes == 0xFF).all()
    if fmt in (NVFP4, FP8_TENSOR):
        assert none.tensor_scale.item() == 1.0
    mxq.quantize_grouped(xd[:0], fmt, zero, torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    assert mxq.check() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("had", [0, 32])
def test_quantize_rows_of_no_expert_set_no_scale(mxq, fmt, dtype, had):
    """Tokens without a row, rows behind the last group and tokens of another part's experts, all 1e30 (a maximum drops a
    NaN, not these), among ones near 1: the tensor scale, and everything else, is that of the others alone."""
    rng = np.random.default_rng(fmt)
    tokens, topk, n, cols = 90, 3, 10, 320
    ids = routing(rng, tokens, topk, n, 0.2)
    ids[rng.choice(tokens, 20, replace=False)] = -1
    off, slot = ref_plan(ids, n)
    x = rng.standard_normal((tokens, cols)).astype(np.float32)
    offd, slotd = torch.from_numpy(off).cuda(), torch.from_numpy(slot).cuda()
    for first, last in ((0, n), (3, 7), (9, 10)):
        lo, hi = int(off[first]), int(off[last])
        mine = (slot >= lo) & (slot < hi)
        placed = mine.any(1)
        xd = dev(np.where(placed[:, None], x, np.float32(1e30)), dtype)
        q = filled(mxq, fmt, tokens * topk, last - first, cols)
        mxq.quantize_grouped(xd, fmt, offd[first:last + 1], slotd, had, out=q)
        # the part's rows, each token's choice within it, as rows in order: the library's own quantizer on them
        src = np.zeros(hi - lo, np.int64)
        for t, i in zip(*np.nonzero(mine)):
            src[slot[t, i] - lo] = t
        rows = xd[torch.from_numpy(src).cuda()]
        want = mxq.quantize(rows, fmt, had)
        assert torch.equal(q.codes.view(tokens * topk, -1)[lo:hi].flatten(), want.codes.view(torch.uint8).flatten())
        assert (q.codes.view(tokens * topk, -1)[:lo] == 0xFF).all() and (q.codes.view(tokens * topk, -1)[hi:] == 0xFF).all()
        if fmt in (NVFP4, FP8_TENSOR):
            assert q.tensor_scale.item() == want.tensor_scale.item() < 1
        if fmt in BLOCK:
            sp = (cols // BLOCK[fmt] + 15) // 16 * 16
            at = mma_offset(scale_rows(off[first:last + 1] - lo, hi - lo)[:, None], np.arange(cols // BLOCK[fmt])[None], sp)
            np.testing.assert_array_equal(q.scales.cpu().numpy()[at].reshape(-1), want.scales.cpu().numpy().reshape(-1))
        elif fmt == INT8_ROW:
            s = q.scales.view(torch.float32)
            assert torch.equal(s[lo:hi], want.scales.view(torch.float32))
            assert (q.scales.view(-1, 4)[:lo] == 0xFF).all() and (q.scales.view(-1, 4)[hi:] == 0xFF).all()
        # the same rows in order already (a second linear): 1e30 in the rows before and behind the groups
        y = torch.full((tokens * topk, cols), 1e30, dtype=xd.dtype, device="cuda")
        y[lo:hi] = rows
        z = filled(mxq, fmt, tokens * topk, last - first, cols)
        mxq.quantize_grouped(y, fmt, offd[first:last + 1], None, had, out=z)
        assert torch.equal(z.codes, q.codes)
        assert z.scales is None or torch.equal(z.scales, q.scales)
        assert z.tensor_scale is None or torch.equal(z.tensor_scale, q.tensor_scale)
    assert mxq.check() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("had,cols", [(0, 320), (64, 320), (0, 5120)])
def test_quantize_inputs_that_are_no_numbers(mxq, fmt, dtype, had, cols):
    """NaN, infinities and the largest values: the bits of mxq_quantize, whatever they are, in the right rows; a token that
    names one expert twice, and room for more rows than there are."""
    rng = np.random.default_rng(fmt)
    tokens, topk, n = 40, 3, 6
    x = rng.standard_normal((tokens, cols)).astype(np.float32)
    if fmt not in (NVFP4, FP8_TENSOR):   # (one such value sets the scale of the whole tensor)
        x[3, 7], x[5, 30:70], x[9], x[11, 100], x[12, 0], x[13] = np.nan, np.nan, np.nan, np.inf, -np.inf, np.inf
        x[14, 3], x[14, 4], x[20], x[21, 5] = np.inf, -np.inf, 3e38, -3.3e38
    x[22], x[23, :32] = 0.0, 1e-40
    ids = rng.integers(-1, n, (tokens, topk))
    ids[:, 0] = np.arange(tokens) % n
    ids[7] = 2
    off, slot = ref_plan(ids, n)
    xd = dev(x, dtype)
    q = filled(mxq, fmt, tokens * topk + 33, n, cols)
    mxq.quantize_grouped(xd, fmt, torch.from_numpy(off).cuda(), torch.from_numpy(slot).cuda(), had, out=q)
    assert mxq.check() == 0
    lib = mxq.quantize(xd, fmt, had)
    sc = None if lib.scales is None else lib.scales.cpu().numpy()
    same = Bits(lib.codes.cpu().numpy().reshape(tokens, -1),
                sc.reshape(tokens, -1) if fmt in BLOCK else None if sc is None else sc.view(np.float32),
                None if lib.tensor_scale is None else lib.tensor_scale.item(), tokens)
    src = np.zeros(int(off[-1]), np.int64)
    for t, i in zip(*np.nonzero(slot >= 0)):
        src[slot[t, i]] = t
    check_grouped(q, same, fmt, off, src, 0xFF)


# ------------------------------------------------------------------ products

def deq64(q):
    return np.asarray(q.dequantize(), np.float64)


class Experts:
    """Expert weights and rows in expert order, with the binary64 product."""

    def __init__(self, mxq, orc, fmt, counts, n, k, extra=0, seed=0, had=0):
        rng = np.random.default_rng(seed + fmt)
        self.counts, e = counts, len(counts)
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        rows = int(self.off[-1]) + extra
        x = rng.standard_t(4, (rows, k)).astype(np.float32)
        x[:, rng.choice(k, max(1, k // 64), replace=False)] *= 30
        x = workloads.to_bf16_values(x)
        w = workloads.to_bf16_values((rng.standard_normal((e, n, k)) * 0.02).astype(np.float32))
        self.w = mxq.prepare_experts(dev(w, "bf16"), fmt, had)
        self.offsets = torch.from_numpy(self.off).cuda()
        self.xq = filled(mxq, fmt, rows, e, k)            # scales nobody writes: NaN in every byte format
        xd = dev(x, "bf16")
        xd[int(self.off[-1]):] = float("nan")
        mxq.quantize_grouped(xd, fmt, self.offsets, hadamard_b=had, out=self.xq)
        used = int(self.off[-1])
        self.ref = np.zeros((used, n))
        self.owq = [orc.quantize(w[i], fmt, had) for i in range(e)]
        if used:
            xv = deq64(orc.quantize(x[:used], fmt, had))
            for i in range(e):
                lo, hi = self.off[i], self.off[i + 1]
                self.ref[lo:hi] = xv[lo:hi] @ deq64(self.owq[i]).T

    def run(self, mxq, out_dtype):
        y = torch.full((self.xq.rows, self.w.rows), 7.0, dtype=out_dtype, device="cuda")
        mxq.qlinear_grouped(self.xq, self.w, self.offsets, out=y)
        assert mxq.check() == 0
        return y

    def check(self, mxq, out_dtype):
        y = self.run(mxq, out_dtype)
        used = int(self.off[-1])
        assert (y[used:] == 7.0).all()                    # rows behind the last group stay
        if used:
            gemm_close(y[:used].float().cpu().numpy(), self.ref, bf16_out=out_dtype == torch.bfloat16)
        return y


FEW = [([1], 128, 128), ([0, 3, 0, 1, 0], 264, 512), ([17, 128, 129, 0, 40, 1], 100, 320), ([64, 5], 520, 1152),
       ([2, 0, 1, 1, 0, 4, 1, 1], 2048, 4096), ([33, 31, 32, 16, 15], 1160, 576), ([250, 0, 0, 0], 136, 192),
       ([1] * 70, 72, 64)]
MANY = [([700, 0, 513, 256, 1000], 264, 512), ([600], 100, 320), ([129, 1000, 511, 2000], 520, 1152),
        ([900, 31, 0, 1500], 1160, 64)]


# more items than pairs of SMs, so that a pair goes on to a second one: blocks of 128 rows, and of 256
MIXED = [([100, 5, 64, 128, 33, 1], 2560, 320), ([260, 90, 250, 256, 31, 512], 4608, 256), ([200, 70, 256, 33, 161], 4608, 192)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,n,k", FEW + MANY + MIXED)
def test_product(mxq, orc, fmt, counts, n, k):
    ex = Experts(mxq, orc, fmt, counts, n, k, extra=5)
    ex.check(mxq, torch.float32)
    ex.check(mxq, torch.bfloat16)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_many_rounds_and_k_tiles(mxq, orc, fmt):
    """Several items per pair of SMs with eight k-tiles and more, blocks of 1 to 256 rows."""
    ex = Experts(mxq, orc, fmt, [600, 513, 256, 700, 257], 2816, 2048, extra=3)
    ex.check(mxq, torch.float32)
    ex.check(mxq, torch.bfloat16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[3, 0, 140], [700, 5, 600]])
def test_product_odd_columns_and_8bit_short_k(mxq, orc, fmt, counts):
    """Rows of y that start at no 16-byte boundary, and one k-step of 32 bytes."""
    Experts(mxq, orc, fmt, counts, 131, 64).check(mxq, torch.float32)
    if fmt in (MXFP8, INT8_ROW, FP8_TENSOR):
        Experts(mxq, orc, fmt, counts, 77, 96).check(mxq, torch.bfloat16)
        Experts(mxq, orc, fmt, counts, 8, 32).check(mxq, torch.float32)


def test_product_int8_is_qlinear_bit_for_bit(mxq, orc):
    """Integer sums are exact, so each row has the bits mxq_qlinear gives it, split K or not, few rows or many."""
    for counts, n, k in (([5, 0, 2], 256, 4608), ([1], 128, 4608), ([500, 700], 384, 1152)):
        ex = Experts(mxq, orc, INT8_ROW, counts, n, k)
        y = ex.run(mxq, torch.float32)
        codes, scales = ex.xq.codes.view(-1, k), ex.xq.scales.view(-1, 4)
        wc, ws = ex.w.codes.view(len(counts), n, k), ex.w.scales.view(len(counts), n * 4)
        for e, c in enumerate(counts):
            if not c:
                continue
            lo, hi = int(ex.off[e]), int(ex.off[e + 1])
            a = mxq.QTensor(INT8_ROW, mxq.MMA, c, k, codes[lo:hi].clone(), scales[lo:hi].clone(), None)
            b = mxq.QTensor(INT8_ROW, mxq.MMA, n, k, wc[e].clone(), ws[e].clone(), None)
            assert torch.equal(mxq.qlinear(a, b, out_dtype=torch.float32), y[lo:hi])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[1, 0, 7, 2], [700, 200, 0, 300]])
def test_product_same_bits_twice_and_by_parts(mxq, orc, fmt, counts):
    ex = Experts(mxq, orc, fmt, counts, 256, 2048)
    y = ex.run(mxq, torch.float32)
    assert torch.equal(y, ex.run(mxq, torch.float32))
    # a part of the experts: offsets from the middle, that part's weight, scales laid out from its first group
    first, n, k = 1, 256, 2048
    off = ex.offsets[first:first + 2].clone()
    lo, hi = int(off[0]), int(off[-1])
    part = mxq.ExpertWeight(fmt, 1, n, k, ex.w.codes.view(4, -1)[1].clone(),
                            None if ex.w.scales is None else ex.w.scales.view(4, -1)[1].clone(),
                            None if ex.w.tensor_scales is None else ex.w.tensor_scales[1:2].clone())
    q = mxq.QTensor(fmt, mxq.MMA, ex.xq.rows, k, ex.xq.codes, ex.xq.scales, ex.xq.tensor_scale)
    if fmt in BLOCK:
        sp, tile = (k // BLOCK[fmt] + 15) // 16 * 16, (counts[0] + 127) // 128
        q.scales = torch.zeros(mxq.grouped_scales_bytes(fmt, ex.xq.rows, 1, k), dtype=torch.uint8, device="cuda")
        src = ex.xq.scales[128 * sp * tile:128 * sp * (tile + (hi - lo + 127) // 128)]
        q.scales[:src.numel()] = src
    z = torch.full_like(y, 3.0)
    mxq.qlinear_grouped(q, part, off, out=z)
    assert mxq.check() == 0
    gemm_close(z[lo:hi].cpu().numpy(), ex.ref[lo:hi]) if hi > lo else None
    assert (z[:lo] == 3.0).all() and (z[hi:] == 3.0).all()


@pytest.mark.parametrize("counts,n,k", [([3, 5, 0, 2], 131, 1152), ([200, 130, 5, 301], 78, 96), ([40, 0, 300, 257], 131, 192)])
def test_int8_part_of_the_experts_in_place(mxq, orc, counts, n, k):
    """INT8 scales are fp32, one per channel: the weight of the experts from `first` on is passed as it lies behind the
    others, wherever its scales begin, and the rows' scales may begin at any fp32 as well."""
    ex = Experts(mxq, orc, INT8_ROW, counts, n, k, extra=2)
    y = ex.run(mxq, torch.float32)
    for first, last in ((1, 4), (2, 4), (3, 4), (0, 2)):
        part = mxq.ExpertWeight(INT8_ROW, last - first, n, k, ex.w.codes[first * n * k:last * n * k],
                                ex.w.scales[first * n * 4:last * n * 4], None)
        room = torch.zeros(ex.xq.scales.numel() + 16, dtype=torch.uint8, device="cuda")
        at = 4 * first
        room[at:at + ex.xq.scales.numel()] = ex.xq.scales
        q = mxq.QTensor(INT8_ROW, mxq.MMA, ex.xq.rows, k, ex.xq.codes, room[at:at + ex.xq.scales.numel()], None)
        z = torch.full_like(y, 3.0)
        mxq.qlinear_grouped(q, part, ex.offsets[first:last + 1], out=z)
        assert mxq.check() == 0
        lo, hi = int(ex.off[first]), int(ex.off[last])
        assert torch.equal(z[lo:hi], y[lo:hi])
        assert (z[:lo] == 3.0).all() and (z[hi:] == 3.0).all()


def kernel_of(fmt, rows, groups, n, k):
    """The kernel that launch_fmt (gemm_grouped.cu) picks for these sizes: "split", or a pair's row block and epilogue warps
    per lane quarter.  To be kept in step with it: the tests below name the kernel they are for."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    k_tiles = -(-k // (256 if fmt in (MXFP4, NVFP4) else 128))
    ragged = min(rows, groups)
    items, split = (rows // 128 + ragged) * -(-n // 128), 1
    while split < 4 and items * split * 2 <= sms and k_tiles >= split * 4:
        split *= 2
    if split > 1:
        return "split"
    wide = rows > 80 * groups
    items = (rows // (256 if wide else 128) + ragged) * -(-n // 256)
    if not wide:
        return 128, 1
    rounds_of_two = items <= 2 * min(items, sms // 2)
    return 256, 1 if fmt in BLOCK and not rounds_of_two and k_tiles >= 8 else 2


# counts, n, k (of 8-bit formats; twice that for 4 bits) and the kernel
BY_KERNEL = [([5, 0, 2], 256, 4608, "split"), ([17, 128, 129, 0, 40, 1], 264, 320, (128, 1)),
             ([60, 3, 128, 70, 0, 33], 4608, 1152, (128, 1)), ([500, 700, 3], 384, 320, (256, 2)),
             ([300, 90, 257], 4608, 576, (256, 2)), ([600, 513, 256, 700, 257], 2816, 1024, (256, "many rounds"))]


def kernel_wanted(fmt, kernel):
    if kernel == (256, "many rounds"):   # one epilogue warp per quarter with block scales
        return 256, 1 if fmt in BLOCK else 2
    return kernel


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,n,k,kernel", BY_KERNEL)
def test_every_kernel_same_bits_twice_and_by_parts(mxq, orc, fmt, counts, n, k, kernel):
    """Each kernel: against binary64, the same bits twice, and parts of the experts in place (offsets from the middle, only
    their rows written)."""
    k *= 2 if fmt in (MXFP4, NVFP4) else 1
    ex = Experts(mxq, orc, fmt, counts, n, k, extra=3)
    e, rows = len(counts), ex.xq.rows
    assert kernel_of(fmt, rows, e, n, k) == kernel_wanted(fmt, kernel)
    ex.check(mxq, torch.bfloat16)
    ex.check(mxq, torch.float32)
    y = ex.run(mxq, torch.float32)
    assert torch.equal(y, ex.run(mxq, torch.float32))
    wc = ex.w.codes.view(e, -1)
    ws = None if ex.w.scales is None else ex.w.scales.view(e, -1)
    for first, last in ((1, e), (0, e - 1)):
        part = mxq.ExpertWeight(fmt, last - first, n, k, wc[first:last].flatten(),
                                None if ws is None else ws[first:last].flatten(),
                                None if ex.w.tensor_scales is None else ex.w.tensor_scales[first:last])
        q = mxq.QTensor(fmt, mxq.MMA, rows, k, ex.xq.codes, ex.xq.scales, ex.xq.tensor_scale)
        if fmt in BLOCK:   # scales laid out from the part's first group
            sp, tile = (k // BLOCK[fmt] + 15) // 16 * 16, sum((c + 127) // 128 for c in counts[:first])
            q.scales = torch.full((mxq.grouped_scales_bytes(fmt, rows, last - first, k),), 0xFF, dtype=torch.uint8, device="cuda")
            src = ex.xq.scales[128 * sp * tile:][:q.scales.numel()]
            q.scales[:src.numel()] = src
        z = torch.full_like(y, 3.0)
        mxq.qlinear_grouped(q, part, ex.offsets[first:last + 1], out=z)
        assert mxq.check() == 0
        lo, hi = int(ex.off[first]), int(ex.off[last])
        assert (z[:lo] == 3.0).all() and (z[hi:] == 3.0).all()
        gemm_close(z[lo:hi].cpu().numpy(), ex.ref[lo:hi])
        if fmt == INT8_ROW or kernel_of(fmt, rows, last - first, n, k) != "split" != kernel:
            assert torch.equal(z[lo:hi], y[lo:hi])   # K in one run: an element has its sums' order in any block


@pytest.mark.parametrize("counts,n,k,kernel", BY_KERNEL)
def test_int8_is_qlinear_bit_for_bit_in_every_kernel(mxq, orc, counts, n, k, kernel):
    ex = Experts(mxq, orc, INT8_ROW, counts, n, k)
    assert kernel_of(INT8_ROW, ex.xq.rows, len(counts), n, k) == kernel_wanted(INT8_ROW, kernel)
    codes, scales = ex.xq.codes.view(-1, k), ex.xq.scales.view(-1, 4)
    wc, ws = ex.w.codes.view(len(counts), n, k), ex.w.scales.view(len(counts), n * 4)
    for dt in (torch.float32, torch.bfloat16):
        y = ex.run(mxq, dt)
        for e, c in enumerate(counts):
            if c:
                lo, hi = int(ex.off[e]), int(ex.off[e + 1])
                a = mxq.QTensor(INT8_ROW, mxq.MMA, c, k, codes[lo:hi].clone(), scales[lo:hi].clone(), None)
                b = mxq.QTensor(INT8_ROW, mxq.MMA, n, k, wc[e].clone(), ws[e].clone(), None)
                assert torch.equal(mxq.qlinear(a, b, out_dtype=dt), y[lo:hi])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [131, 100, 7])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_product_split_with_ragged_columns(mxq, orc, fmt, n, out_dtype):
    """K split, N no multiple of 8: the elements of a row's last ones go one by one, and nothing behind y is touched."""
    ex = Experts(mxq, orc, fmt, [5, 0, 2, 129], n, 2048, extra=1)
    rows, used = ex.xq.rows, int(ex.off[-1])
    assert kernel_of(fmt, rows, 4, n, 2048) == "split"
    room = torch.full((rows * n + 1024,), 7.0, dtype=out_dtype, device="cuda")
    y = room[:rows * n].view(rows, n)
    mxq.qlinear_grouped(ex.xq, ex.w, ex.offsets, out=y)
    assert mxq.check() == 0
    assert (y[used:] == 7.0).all() and (room[rows * n:] == 7.0).all()
    gemm_close(y[:used].float().cpu().numpy(), ex.ref, bf16_out=out_dtype == torch.bfloat16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,n,k", [([5, 0, 130], 136, 320), ([3, 2], 100, 2048), ([700, 300], 264, 320)])
def test_product_of_rotated_operands(mxq, orc, fmt, counts, n, k):
    """Both sides quantized behind the Hadamard rotation: the product of what the oracle's rotated codes stand for."""
    ex = Experts(mxq, orc, fmt, counts, n, k, extra=2, had=64)
    ex.check(mxq, torch.float32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,n,k", [([5, 0, 130, 2], 136, 2048), ([70, 3, 128, 90], 264, 320), ([700, 3, 300], 264, 320)])
def test_product_keeps_a_nan_where_it_is(mxq, orc, fmt, counts, n, k):
    """A row of X, and a feature of one expert, that hold a NaN: their row and column of y, and no other element."""
    if fmt in (MXFP4, NVFP4):
        k *= 2
    ex = Experts(mxq, orc, fmt, counts, n, k)
    y = ex.run(mxq, torch.float32)
    row, feature, rows = 4, 37, ex.xq.rows
    if fmt in BLOCK:   # a NaN block scale: 0xFF in E8M0, 0x7F in E4M3
        sp = (k // BLOCK[fmt] + 15) // 16 * 16
        bad = 0x7F if fmt == NVFP4 else 0xFF
        ex.xq.scales[int(mma_offset(row, 3, sp))] = bad
        ex.w.scales.view(len(counts), -1)[2, int(mma_offset(feature, 1, sp))] = bad
    elif fmt == INT8_ROW:
        ex.xq.scales.view(torch.float32)[row] = float("nan")
        ex.w.scales.view(torch.float32).view(len(counts), n)[2, feature] = float("nan")
    else:
        ex.xq.codes.view(rows, k)[row, 3] = 0x7F
        ex.w.codes.view(len(counts), n, k)[2, feature, 40] = 0x7F
    z = ex.run(mxq, torch.float32)
    nan = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
    nan[row] = True
    nan[int(ex.off[2]):int(ex.off[3]), feature] = True
    assert torch.equal(torch.isnan(z), nan) and torch.equal(z[~nan], y[~nan])


@pytest.mark.parametrize("bad", [[0, 5, 3, 20], [-7, 2, 2, 20], [0, 4, 90, 20], [19, 4, 4, 4], [2 ** 31 - 1] * 4])
@pytest.mark.parametrize("fmt", [MXFP8, INT8_ROW])
@pytest.mark.parametrize("scale", [1, 40])
def test_offsets_out_of_order_are_clamped_and_reported(mxq, orc, bad, fmt, scale):
    """No access leaves the buffers (the kernels clamp each offset) and the next check says so, once."""
    ex = Experts(mxq, orc, fmt, [8 * scale, 8 * scale, 4 * scale], 128, 256)
    off = torch.tensor([min(v * scale, 2 ** 31 - 1) for v in bad], dtype=torch.int32, device="cuda")
    mxq.qlinear_grouped(ex.xq, ex.w, off)
    assert mxq.check() == 1 and mxq.check() == 0
    q = mxq.alloc_grouped(fmt, 20 * scale, 3, 256)
    x = torch.randn(20 * scale, 256, device="cuda")
    mxq.quantize_grouped(x, fmt, off, out=q)
    assert mxq.check() == 1 and mxq.check() == 0
    ex.check(mxq, torch.float32)


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("ydt,odt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("tokens,topk,n", [(1, 1, 1), (3, 8, 264), (200, 4, 100), (17, 5, 131), (64, 32, 8), (1000, 2, 1152)])
def test_combine(mxq, ydt, odt, tokens, topk, n):
    rng = np.random.default_rng(tokens + n)
    e = max(topk, 8)
    off, slot = ref_plan(routing(rng, tokens, topk, e, 0.3 if tokens > 1 else 0.0), e)
    y = host_values(rng.standard_normal((tokens * topk, n)).astype(np.float32), ydt)
    w = rng.random((tokens, topk)).astype(np.float32)
    yd = dev(y, ydt)
    yd[int(off[-1]):] = float("nan")                      # rows behind the last group
    for weights in (w, None):
        out = mxq.expert_combine(yd, torch.from_numpy(slot).cuda(), None if weights is None else torch.from_numpy(w).cuda(),
                                 out_dtype=torch.bfloat16 if odt == "bf16" else torch.float32)
        assert mxq.check() == 0
        terms = np.where(slot >= 0, w if weights is not None else 1.0, 0.0)[..., None] * y.astype(np.float64)[np.maximum(slot, 0)]
        ref, mag = terms.sum(1), np.abs(terms).sum(1)
        got = out.float().cpu().numpy().astype(np.float64)
        tol = topk * 2.0 ** -24 * mag * (1 + 1e-6) + (2.0 ** -8 * (np.abs(ref) + 1e-6 * mag) if odt == "bf16" else 0)
        assert (np.abs(got - ref) <= tol).all()
        assert (got[(slot < 0).all(1)] == 0).all()


def test_combine_slots_outside_are_left_out_and_reported(mxq):
    y = torch.ones(4, 16, device="cuda")
    slot = torch.tensor([[0, 4], [2 ** 31 - 1, -2 ** 31], [3, 1]], dtype=torch.int32, device="cuda")
    out = mxq.expert_combine(y, slot)
    assert mxq.check() == 1 and mxq.check() == 0
    assert out[:, 0].tolist() == [1.0, 0.0, 2.0]
    assert (mxq.expert_combine(y[:0], torch.full((2, 3), -1, dtype=torch.int32, device="cuda")) == 0).all()


def test_combine_of_more_outputs_than_31_bits_count(mxq):
    """600,000 tokens of 4096: every token, weights that are powers of two and so exact."""
    t, n = 600000, 4096
    g = torch.Generator("cuda").manual_seed(3)
    y = torch.randn(8, n, device="cuda", generator=g).bfloat16()
    slot = torch.randint(-1, 8, (t, 1), device="cuda", dtype=torch.int32, generator=g)
    weights = 2.0 ** torch.randint(-1, 2, (t, 1), device="cuda", generator=g).float()
    for w in (weights, None):
        out = mxq.expert_combine(y, slot, w)
        assert mxq.check() == 0
        for lo in range(0, t, 100000):
            s = slot[lo:lo + 100000, 0].long()
            want = torch.where(s[:, None] >= 0, y[s.clamp(min=0)], torch.zeros_like(y[:1]))
            assert torch.equal(out[lo:lo + 100000], want if w is None else want * w[lo:lo + 100000].bfloat16())
    for n in (0, 1):
        assert (mxq.expert_combine(torch.ones(3, n, device="cuda"), slot[:4].clamp(0, 2)) == 1).all()
        assert mxq.expert_combine(torch.ones(3, n, device="cuda"), slot[:0]).shape == (0, n)
    assert mxq.check() == 0


# ------------------------------------------------------------------ together

def layer(mxq, x, ids, weights, w, fmt, n):
    """One linear of a mixture of experts, as a user runs it."""
    plan = mxq.expert_plan(ids, n)
    xq = mxq.quantize_grouped(x, fmt, plan.offsets, plan.slot)
    return mxq.expert_combine(mxq.qlinear_grouped(xq, w, plan.offsets), plan.slot, weights)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,topk,e", [(1, 2, 8), (40, 4, 16), (900, 3, 6)])
def test_layer(mxq, orc, fmt, tokens, topk, e):
    rng = np.random.default_rng(tokens + fmt)
    n, k = 264, 320
    x = workloads.to_bf16_values(rng.standard_normal((tokens, k)).astype(np.float32))
    w = workloads.to_bf16_values((rng.standard_normal((e, n, k)) * 0.05).astype(np.float32))
    ids = routing(rng, tokens, topk, e, 0.0)
    gate = rng.random((tokens, topk)).astype(np.float32)
    we = mxq.prepare_experts(dev(w, "bf16"), fmt)
    args = (dev(x, "bf16"), torch.from_numpy(ids).cuda(), torch.from_numpy(gate).cuda(), we, fmt, e)
    y = layer(mxq, *args)
    assert mxq.check() == 0
    xv = deq64(orc.quantize(x, fmt))
    ref, mag = np.zeros((tokens, n)), np.zeros((tokens, n))
    for i in range(e):
        t, j = np.nonzero(ids == i)
        part = gate[t, j, None] * (xv[t] @ deq64(orc.quantize(w[i], fmt)).T)
        np.add.at(ref, t, part)
        np.add.at(mag, t, np.abs(part))
    got = y.float().cpu().numpy()
    # each product rounded to bf16 once (2^-8 of it), the sum once more; fp32 sums as in gemm_close
    assert (np.abs(got - ref) <= 2.0 ** -8 * (mag + np.abs(ref)) + 1e-4 * np.abs(ref).max()).all()
    # captured once, replayed on other inputs; and the same on a stream of its own
    static = [a.clone() for a in args[:3]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = layer(mxq, *static, *args[3:])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
            out = layer(mxq, *static, *args[3:])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(z, y)
    static[1].copy_(static[1].flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, layer(mxq, static[0], static[1], static[2], *args[3:]))
    assert mxq.check() == 0


def test_two_captured_layers_in_flight(mxq):
    """Two captured layers replayed on two streams share nothing."""
    n, k, e = 128, 128, 8
    runs = []
    for seed in (1, 2):
        torch.manual_seed(seed)
        x = torch.randn(64, k, device="cuda", dtype=torch.bfloat16)
        ids = torch.randint(0, e, (64, 2), device="cuda")
        w = mxq.prepare_experts(torch.randn(e, n, k, device="cuda") * 0.05, NVFP4)
        gate = torch.rand(64, 2, device="cuda")
        want = layer(mxq, x, ids, gate, w, NVFP4, e)
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
            out = layer(mxq, x, ids, gate, w, NVFP4, e)
        runs.append((g, s, out, want, (x, ids, w, gate)))
    for _ in range(20):
        for g, s, _, _, _ in runs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, out, want, _ in runs:
        assert torch.equal(out, want)
    assert mxq.check() == 0


def test_stream_argument(mxq):
    s = torch.cuda.Stream()
    ids = torch.randint(0, 4, (50, 2), device="cuda")
    torch.cuda.synchronize()
    a, b = mxq.expert_plan(ids, 4, stream=s), mxq.expert_plan(ids, 4)
    torch.cuda.synchronize()
    assert torch.equal(a.offsets, b.offsets) and torch.equal(a.slot, b.slot)


def test_plan_of_many_choices_captured(mxq):
    """The two-kernel plan, its workspace from the graph's own pool, replayed on other ids."""
    ids = torch.randint(0, 300, (20000, 2), device="cuda", dtype=torch.int32)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        plan = mxq.expert_plan(ids, 300)
    for _ in range(3):
        ids.copy_(torch.randint(-3, 310, (20000, 2), device="cuda", dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        off, slot = ref_plan(ids.cpu().numpy(), 300)
        np.testing.assert_array_equal(plan.offsets.cpu().numpy(), off)
        np.testing.assert_array_equal(plan.slot.cpu().numpy(), slot)
    check_plan(mxq, np.random.default_rng(1).integers(0, 512, (1 << 19, 8)), 512, torch.int64)   # the most choices there can be


@pytest.mark.parametrize("fmt", [MXFP8, INT8_ROW])
def test_rows_past_32_bits(mxq, orc, fmt):
    """Codes of 2.5 GB and products of 4.9 GB: the last rows against the oracle."""
    tokens, topk, e, n, k = 300000, 2, 4, 4096, 4096
    torch.manual_seed(fmt)
    x = torch.empty(tokens, k, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    w = torch.randn(e, n, k, device="cuda") * 0.02
    ids = torch.stack([torch.arange(tokens, device="cuda") % 2, 2 + torch.arange(tokens, device="cuda") % 2], 1)
    plan = mxq.expert_plan(ids, e)
    xq = mxq.quantize_grouped(x, fmt, plan.offsets, plan.slot)
    y = mxq.qlinear_grouped(xq, mxq.prepare_experts(w, fmt), plan.offsets)
    gate = torch.rand(tokens, topk, device="cuda")
    out = mxq.expert_combine(y, plan.slot, gate)
    assert mxq.check() == 0
    pick = np.array([0, 1, 131071, 262144, tokens - 2, tokens - 1])
    xv = deq64(orc.quantize(x[pick].float().cpu().numpy(), fmt))
    wv = [deq64(orc.quantize(w[i].cpu().numpy(), fmt)) for i in range(e)]
    slot = plan.slot[pick].cpu().numpy()
    assert slot.max() >= tokens * topk - 2
    for i, t in enumerate(pick):
        both = [xv[i] @ wv[t % 2].T, xv[i] @ wv[2 + t % 2].T]
        for j in range(2):
            gemm_close(y[slot[i, j]].float().cpu().numpy(), both[j], bf16_out=True)
        wt = gate[t].cpu().numpy().astype(np.float64)
        mag = wt[0] * np.abs(both[0]) + wt[1] * np.abs(both[1])
        ref = wt[0] * both[0] + wt[1] * both[1]
        assert (np.abs(out[t].float().cpu().numpy() - ref) <= 2.0 ** -8 * (mag + np.abs(ref)) + 2e-4 * np.abs(both).max()).all()
