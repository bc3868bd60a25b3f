"""GPU parity of the q/k head step (norm of every head, position rotation,
optional Hadamard rotation and codes) against binary64.

Tolerances, in units u = 2^-24 of the head's values.  Norm: the fp32 sum of
squares of D elements is off by at most (D / 8 + 8) u relative (eight
elements in a lane, a tree over lanes; D <= 256), the root halves that, rsqrtf
adds 4 u, the two products 2 u; the mean of MXQ_NORM_LAYER, taken off each
element, adds (D / 8 + 10) u of the largest |x - mean| + |mean| scale, scaled
by the same norm.  Rotation: 3 u of |a c| + |b s|.  bf16 rounds once more:
2^-8 of the value.  Codes are checked through their fp32 values before coding:
a code may differ from the reference's only where the value lies within the
tolerance of a rounding border, so each dequantized value is within half a
step plus the tolerance of the exact one."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host_values

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
MXFP8, MXFP4, NVFP4, INT8_ROW = 0, 1, 2, 5


@pytest.fixture(scope="module")
def mxq():
    import microscaling_bit_quantization_b200 as m
    assert torch.cuda.is_available() and m.lib().mxq_device_supported(0) == 1
    m.check()
    return m


def tables(n, rot):
    if rot == 0:
        return None, None
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def ref_heads(x, w, cos, sin, pos, norm, eps, interleaved):
    """(values, tolerance without the output's rounding), binary64."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    c = x - x.mean(-1, keepdims=True) if norm == "layer" else x
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    ww = np.ones(d) if w is None else np.asarray(w, np.float64)
    v = c * r * ww
    tol = ((d / 8 + 8) / 2 + 8) * U * np.abs(v)
    if norm == "layer":
        # an error m of the mean moves every element by m and the mean square by at most 2 m mean|c|
        m = (d / 8 + 10) * U * np.abs(x).max(-1, keepdims=True)
        tol = tol + m * r * np.abs(ww) + 2 * m * r * np.abs(v)
    if cos is not None:
        half = cos.shape[1]
        a = np.arange(half) * 2 if interleaved else np.arange(half)
        b = a + 1 if interleaved else a + half
        co, si = cos.astype(np.float64)[pos][:, None], sin.astype(np.float64)[pos][:, None]
        va, vb, ta, tb = v[..., a], v[..., b], tol[..., a], tol[..., b]
        v, tol = v.copy(), tol.copy()
        v[..., a], v[..., b] = va * co - vb * si, vb * co + va * si
        tol[..., a] = ta * np.abs(co) + tb * np.abs(si) + 3 * U * (np.abs(va * co) + np.abs(vb * si))
        tol[..., b] = tb * np.abs(co) + ta * np.abs(si) + 3 * U * (np.abs(vb * co) + np.abs(va * si))
    return v, tol


def inputs(seed, tokens, hq, hk, d, dtype, extra=8):
    rng = np.random.default_rng(seed)
    n = (hq + 2 * hk) * d + extra
    qkv = (rng.standard_normal((tokens, n)) * np.exp(rng.uniform(-2, 2, n)) + 0.3).astype(np.float32)
    t = dev(qkv, dtype)
    vals = host_values(qkv, dtype)
    q, k = t[:, :hq * d].unflatten(1, (hq, d)), t[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)) if hk else None
    return rng, t, q, k, vals[:, :hq * d].reshape(tokens, hq, d), vals[:, hq * d:(hq + hk) * d].reshape(tokens, hk, d)


CASES = [(1, 1, 1, 8, 8), (3, 5, 1, 64, 64), (7, 3, 2, 72, 72), (130, 4, 4, 80, 40), (5, 6, 2, 96, 96), (33, 32, 8, 128, 128),
         (4, 2, 0, 256, 128), (9, 3, 3, 120, 0), (2, 1, 1, 248, 248), (1000, 2, 1, 16, 8), (600, 16, 16, 72, 72)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,d,rot", CASES)
def test_heads(mxq, tokens, hq, hk, d, rot, interleaved, norm, dtype):
    rng, t, q, k, qv, kv = inputs(d + tokens, tokens, hq, hk, d, dtype)
    cos, sin = tables(5000, rot)
    pos = rng.integers(0, 5000, tokens)
    wq, wk = rng.standard_normal((2, d)).astype(np.float32)
    gpu = lambda a, dt=None: None if a is None else torch.from_numpy(a if dt is None else a.astype(dt)).cuda()  # noqa: E731
    before = t.clone()
    for weights, ptype in ((True, np.int32), (False, np.int64)):
        qo, ko = mxq.qk_norm_rope(q, k, gpu(wq) if weights else None, gpu(wk) if weights else None, gpu(cos), gpu(sin),
                                  gpu(pos, ptype), eps=1e-5, norm=norm, interleaved=interleaved)
        assert mxq.check() == 0 and torch.equal(t, before)
        for o, v, w in ((qo, qv, wq), (ko, kv, wk)):
            if o is None:
                continue
            ref, tol = ref_heads(v, w if weights else None, cos, sin, pos, norm, 1e-5, interleaved)
            got = o.float().cpu().numpy().astype(np.float64)
            if dtype == "bf16":
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
            assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / np.maximum(tol, 1e-300)).max()
    # in place, into the parts of the q/k/v row, which keeps everything else
    qi, ki = mxq.qk_norm_rope(q, k, None, None, gpu(cos), gpu(sin), gpu(pos), eps=1e-5, norm=norm, interleaved=interleaved,
                              q_out=q, k_out=k)
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))
    assert torch.equal(t[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


@pytest.mark.parametrize("fmt", [MXFP8, MXFP4, INT8_ROW])
@pytest.mark.parametrize("tokens,hq,hk,d,rot,had", [(1, 1, 1, 32, 32, 32), (5, 3, 2, 64, 64, 0), (33, 8, 2, 128, 128, 128),
                                                   (7, 5, 1, 96, 48, 32), (4, 2, 0, 256, 256, 256), (3, 1, 3, 160, 64, 0),
                                                   (700, 4, 4, 128, 64, 0), (9, 7, 2, 224, 224, 16), (2000, 16, 4, 64, 64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_heads_quantize(mxq, fmt, tokens, hq, hk, d, rot, had, dtype):
    rng, t, q, k, qv, kv = inputs(d + tokens + fmt, tokens, hq, hk, d, dtype, extra=0)
    cos, sin = tables(tokens + 3, rot)
    wq, wk = rng.standard_normal((2, d)).astype(np.float32)
    gpu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    out = mxq.qk_norm_rope_quantize(q, k, gpu(wq), gpu(wk), gpu(cos), gpu(sin), fmt=fmt, hadamard_b=had, interleaved=rot != d)
    assert mxq.check() == 0
    # the library's quantizer on the 32-bit outputs of the same step: same codes wherever the fp32 values are the same
    for o, x, v, w in zip(out, (q, k), (qv, kv), (wq, wk)):
        if o is None:
            continue
        ref, tol = ref_heads(v, w, cos, sin, np.arange(tokens), "rms", 1e-6, rot != d)
        h = v.shape[1]
        ref, tol = ref.reshape(tokens * h, d), tol.reshape(tokens * h, d)
        if had:
            signs = np.array([[(-1.0) ** bin(i & j).count("1") for j in range(had)] for i in range(had)]) / np.sqrt(had)
            blocks, tb = ref.reshape(-1, d // had, had), tol.reshape(-1, d // had, had)
            # log2(had) additions and the factor, each 2^-24 of the largest partial sum; the inputs' tolerance adds up
            grow = np.abs(blocks).sum(-1, keepdims=True) / np.sqrt(had)
            tol = (tb.sum(-1, keepdims=True) / np.sqrt(had) + (np.log2(had) + 2) * U * grow + 0 * blocks).reshape(ref.shape)
            ref = (blocks @ signs).reshape(ref.shape)
        got = mxq.dequantize(o).cpu().numpy().astype(np.float64)
        if fmt == INT8_ROW:
            top = np.abs(ref).max(1, keepdims=True)
            s = o.scales.cpu().view(torch.float32).numpy().astype(np.float64)[:, None]
            assert (np.abs(s - top / 127) <= (tol.max(1, keepdims=True) / 127 + U * top / 127)).all()
            step, clip = s, np.inf
        else:
            e = o.scales.cpu().numpy().reshape(tokens * h, d // 32).astype(np.int64) - 127
            top = np.abs(ref).reshape(tokens * h, d // 32, 32).max(2)
            slack = tol.reshape(tokens * h, d // 32, 32).max(2)
            emax = 8 if fmt == MXFP8 else 2
            lo, hi = np.floor(np.log2(top - slack)) - emax, np.floor(np.log2(top + slack)) - emax
            assert ((e >= lo) & (e <= hi)).all()
            scale = np.repeat(2.0 ** e, 32, 1)
            man, sub, clip = (3, -6, 448.0) if fmt == MXFP8 else (1, 0, 6.0)
            mag = np.minimum(np.maximum(np.abs(ref), 1e-300) / scale, clip)
            step = 2.0 ** (np.maximum(np.floor(np.log2(mag * (1 + 1e-6))), sub) - man) * scale
            clip = clip * scale
        want = np.clip(ref, -clip, clip)
        # half a step; where the value lies just below a power of two the step above it counts
        near = np.abs(got - want) <= step / 2 * (1 + 1e-6) + tol
        assert near.all(), np.abs(got - want)[~near][:5]


@pytest.mark.parametrize("fmt", [MXFP8, MXFP4, INT8_ROW])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scale", [1.0, 1e-30, 1e-38, 1e-42, 1e15])
def test_codes_are_those_of_the_fp32_outputs(mxq, fmt, interleaved, scale):
    """Without the Hadamard rotation the two forms do the same fp32 operations, so the codes have the bits mxq_quantize
    gives the fp32 outputs: for values whose norm is all eps, subnormal ones, and ones near the largest square."""
    g = torch.Generator().manual_seed(5)
    q = (torch.randn(60, 6, 96, generator=g) * scale).cuda()
    k = (torch.randn(60, 2, 96, generator=g) * scale).cuda()
    q[3, 1] = 0
    w = torch.randn(96, generator=g).cuda()
    cos, sin = (torch.from_numpy(a).cuda() for a in tables(60, 64))
    plain = mxq.qk_norm_rope(q, k, w, None, cos, sin, norm="layer", interleaved=interleaved)
    coded = mxq.qk_norm_rope_quantize(q, k, w, None, cos, sin, norm="layer", interleaved=interleaved, fmt=fmt)
    for p, c in zip(plain, coded):
        want = mxq.quantize(p.flatten(0, 1), fmt)
        assert torch.equal(c.codes, want.codes) and torch.equal(c.scales, want.scales)


def test_positions_outside_are_reported_and_nan(mxq):
    q = torch.randn(4, 2, 64, device="cuda")
    cos, sin = (torch.from_numpy(a).cuda() for a in tables(10, 64))
    for bad, dt in ((10, torch.int32), (-1, torch.int32), (2 ** 32 + 1, torch.int64)):
        pos = torch.tensor([0, 9, bad, 3], dtype=dt, device="cuda")
        o, _ = mxq.qk_norm_rope(q, None, None, None, cos, sin, pos)
        assert mxq.check() == 1 and mxq.check() == 0
        nan = torch.isnan(o).flatten(1)
        assert nan[2].all() and not nan[[0, 1, 3]].any()
        for fmt in (MXFP8, MXFP4, INT8_ROW):
            z, _ = mxq.qk_norm_rope_quantize(q, None, None, None, cos, sin, pos, fmt=fmt)
            assert mxq.check() == 1
            v = mxq.dequantize(z).view(4, -1)
            assert torch.isnan(v[2]).all() and not torch.isnan(v[[0, 1, 3]]).any()


def test_empty_zero_rows_and_graph(mxq):
    q = torch.zeros(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    cos, sin = (torch.from_numpy(a).cuda() for a in tables(10, 64))
    o, _ = mxq.qk_norm_rope(q, None, None, None, cos, sin)
    assert (o == 0).all()                                 # a head of zeros: eps keeps it finite
    o, k = mxq.qk_norm_rope(q[:0], q[:0], None, None, cos, sin)
    assert o.shape == (0, 2, 64) and mxq.check() == 0
    x = torch.randn(50, 8, 128, device="cuda", dtype=torch.bfloat16)
    cos, sin = (torch.from_numpy(a).cuda() for a in tables(50, 128))
    want = mxq.qk_norm_rope(x, x, None, None, cos, sin)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        out = mxq.qk_norm_rope(x, x, None, None, cos, sin)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = mxq.qk_norm_rope(x, x, None, None, cos, sin, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(again[0], want[0]) and mxq.check() == 0


@pytest.mark.parametrize("fmt", [None, MXFP8, MXFP4, INT8_ROW])
@pytest.mark.parametrize("tokens,hq,hk,d,interleaved", [(700, 77, 5, 128, True), (700, 77, 5, 128, False), (300, 3, 130, 96, True),
                                                        (2000, 33, 1, 160, False), (1, 300, 300, 32, True), (129, 16, 17, 256, False)])
def test_heads_do_not_depend_on_their_neighbours(mxq, fmt, tokens, hq, hk, d, interleaved):
    """However many heads and tokens share a call, a head gets the bits it gets alone; either side may have no heads."""
    gen = torch.Generator("cuda").manual_seed(tokens + hq)
    q, k = (torch.randn(tokens, h, d, device="cuda", generator=gen).bfloat16() for h in (hq, hk))
    w = torch.rand(d, device="cuda", generator=gen) + 0.5
    cos, sin = (torch.from_numpy(a).cuda() for a in tables(tokens, d))
    had = 0 if fmt is None else d & -d

    def f(q, k, lo, hi):
        pos = torch.arange(lo, hi, device="cuda", dtype=torch.int32)
        if fmt is None:
            return [o for o in mxq.qk_norm_rope(q, k, w, w, cos, sin, pos, interleaved=interleaved)]
        out = mxq.qk_norm_rope_quantize(q, k, w, w, cos, sin, pos, interleaved=interleaved, fmt=fmt, hadamard_b=had)
        return [mxq.dequantize(o).view(hi - lo, -1, d) if o.rows else None for o in out]

    qa, ka = f(q, k, 0, tokens)
    for lo, hi, h0, h1, g0, g1 in ((0, tokens, 0, 1, hk - 1, hk), (tokens // 2, tokens // 2 + 1, hq // 2, hq, 0, hk),
                                   (tokens - 1, tokens, hq - 1, hq, 0, 1), (0, tokens, 0, 0, 0, hk), (0, tokens, 0, hq, 0, 0)):
        qp, kp = f(q[lo:hi, h0:h1].contiguous(), k[lo:hi, g0:g1].contiguous(), lo, hi)
        assert h1 == h0 or torch.equal(qp, qa[lo:hi, h0:h1])
        assert g1 == g0 or torch.equal(kp, ka[lo:hi, g0:g1])
    assert mxq.check() == 0


@pytest.mark.parametrize("fmt", [None, MXFP8])
def test_tokens_past_32_bits(mxq, fmt):
    """2.5 G elements: the last tokens as a call on them alone gives them."""
    t, hq, hk, d = 480000, 32, 8, 128
    x = torch.empty(t, hq + hk, d, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    q, k = x[:, :hq], x[:, hq:]
    cos, sin = (torch.from_numpy(a).cuda() for a in tables(100, d))
    pos = torch.arange(t, device="cuda") % 100
    f = mxq.qk_norm_rope if fmt is None else lambda *a: mxq.qk_norm_rope_quantize(*a, fmt=fmt, hadamard_b=d)
    big = f(q, k, None, None, cos, sin, pos)
    tail = f(q[-5:], k[-5:], None, None, cos, sin, pos[-5:])
    assert mxq.check() == 0
    for b, s, h in zip(big, tail, (hq, hk)):
        if fmt is None:
            assert torch.equal(b[-5:], s)
        else:
            assert torch.equal(b.codes[-5 * h * d:], s.codes) and torch.equal(b.scales[-5 * h * d // 32:], s.scales)


@pytest.mark.parametrize("fmt", [MXFP8, MXFP4, INT8_ROW])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,had", [(64, 64, 0), (96, 64, 0), (96, 64, 32), (128, 96, 0), (128, 128, 128), (256, 256, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_codes_keep_nan(mxq, fmt, interleaved, d, rot, had, dtype, norm):
    """A block (a head in INT8) with a NaN among its fp32 values reads back as NaN, whatever brought it there; every other
    block has the codes it has without it."""
    g = torch.Generator().manual_seed(d + had)
    q, k = torch.randn(40, 5, d, generator=g), torch.randn(40, 3, d, generator=g)
    nan, inf = float("nan"), float("inf")
    clean = [q.clone(), k.clone()]
    for x, z in zip((q, k), clean):
        for (t, h, i), v in {(0, 0, 5): nan, (1, 1, d - 1): nan, (7, 2, 0): inf, (8, 0, d - 3): -inf, (9, 1, 33): inf}.items():
            x[t, h, i] = v
            z[t, h] = 0
        x[20, 1] = nan
        z[20, 1] = 0
        x[21, 2, 3], x[21, 2, 40] = inf, -inf
        z[21, 2] = 0
        x[22, 0], z[22, 0] = x[22, 0] * 1e30, 0           # finite, its squares beyond the largest fp32 value: zeros
    q, k, *clean = (dev(x.numpy(), dtype) for x in (q, k, *clean))
    touched = [~torch.isfinite(x).all(2) | (x.abs().amax(2) > 1e20) for x in (q, k)]
    w = (torch.rand(d, generator=g) + 0.5).cuda()
    cos, sin = (torch.from_numpy(a).cuda() for a in tables(40, rot))

    def coded(q, k, w, eps=1e-6):
        return mxq.qk_norm_rope_quantize(q, k, w, w, cos, sin, fmt=fmt, hadamard_b=had, norm=norm, interleaved=interleaved, eps=eps)

    def nans(q, k, w, eps=1e-6):
        """Blocks of the fp32 outputs, after the rotation, that hold a NaN."""
        out = []
        for p in mxq.qk_norm_rope(q.float(), k.float(), w, w, cos, sin, norm=norm, interleaved=interleaved, eps=eps):
            bad = torch.isnan(p).flatten(0, 1)
            if had:
                bad = bad.unflatten(1, (-1, had)).any(2, keepdim=True).expand(-1, -1, had).flatten(1)
            out.append(bad.unflatten(1, (1 if fmt == INT8_ROW else d // 32, -1)).any(2))
        return out

    def check(got, bad):
        for o, b in zip(got, bad):
            v = mxq.dequantize(o).view(b.shape[0], b.shape[1], -1)
            assert torch.equal(torch.isnan(v).all(2), b) and torch.equal(torch.isnan(v).any(2), b)

    got, base, bad = coded(q, k, w), coded(*clean, w), nans(q, k, w)
    check(got, bad)
    for o, c, b, hit in zip(got, base, bad, touched):
        assert b.any(1).sum() >= 7 and not b[~hit.flatten()].any()
        rows = ~hit.flatten()
        both = lambda z: (z.codes.view(rows.numel(), -1)[rows], z.scales.view(rows.numel(), -1)[rows])  # noqa: E731
        assert all(torch.equal(m, n) for m, n in zip(both(o), both(c)))
    if not had:   # and the blocks beside a NaN in its head: what mxq_quantize gives the fp32 outputs
        for o, p, b in zip(got, mxq.qk_norm_rope(q.float(), k.float(), w, w, cos, sin, norm=norm, interleaved=interleaved), bad):
            want = mxq.quantize(p.flatten(0, 1), fmt)
            v, u = (mxq.dequantize(z).view(b.shape[0], b.shape[1], -1)[~b] for z in (o, want))
            assert torch.equal(v, u)
    # no mean square at all: zeros with eps 0
    q[3, 1] = 0
    bad = nans(q, k, w, 0.0)
    assert bad[0].view(40, 5, -1)[3, 1].all()
    check(coded(q, k, w, 0.0), bad)
    # a weight that is no number
    w[d - 2] = nan
    bad = nans(q, k, w)
    assert all(b.any(1).all() for b in bad)
    check(coded(q, k, w), bad)
    assert mxq.check() == 0


@pytest.mark.parametrize("fmt", [None, MXFP8, MXFP4, INT8_ROW])
def test_heads_captured_strided_and_on_another_stream(mxq, fmt):
    """A captured call replayed on other inputs and positions; every second token of a longer buffer; a stream of its own."""
    t, hq, hk, d = 70, 6, 2, 96
    g = torch.Generator("cuda").manual_seed(9)
    big = torch.randn(2 * t, (hq + hk) * d, device="cuda", generator=g).bfloat16()
    q, k = big[::2, :hq * d].unflatten(1, (hq, d)), big[::2, hq * d:].unflatten(1, (hk, d))
    w = torch.rand(d, device="cuda", generator=g)
    cos, sin = (torch.from_numpy(a).cuda() for a in tables(50, 64))
    pos = torch.randint(0, 50, (t,), device="cuda", generator=g)

    def f(q, k, stream=None):
        if fmt is None:
            return list(mxq.qk_norm_rope(q, k, w, w, cos, sin, pos, norm="layer", stream=stream))
        out = mxq.qk_norm_rope_quantize(q, k, w, w, cos, sin, pos, norm="layer", fmt=fmt, hadamard_b=32, stream=stream)
        return [x for o in out for x in (o.codes, o.scales)]

    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    assert same(f(q, k), f(q.contiguous(), k.contiguous()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = f(q, k, stream=side)
    torch.cuda.synchronize()
    assert same(other, f(q, k))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        out = f(q, k)
    for _ in range(3):
        big.copy_(torch.randn(big.shape, device="cuda", generator=g))
        pos.copy_(torch.randint(0, 50, (t,), device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, f(q, k))
    assert mxq.check() == 0
