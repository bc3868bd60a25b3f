"""Host-side checks of the calls on rows in expert order and of the q/k head
step (no GPU needed): sizes, and arguments refused before any launch."""
import ctypes

import pytest

EINVAL, EUNSUPPORTED, ENOSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def mxq():
    import __graft_entry__
    __graft_entry__.build()
    import microscaling_bit_quantization_b200 as m
    return m


P = ctypes.c_void_p
D = 4096   # an address: nothing is read on the host


def test_sizes(mxq):
    M = mxq
    assert M.grouped_scales_bytes(M.MXFP8, 256, 8, 64) == (2 + 8) * 128 * 16
    assert M.grouped_scales_bytes(M.NVFP4, 3, 64, 4096) == 3 * 128 * 256
    assert M.grouped_scales_bytes(M.INT8_ROW, 10, 4, 64) == 40
    assert M.grouped_scales_bytes(M.FP8_TENSOR, 10, 4, 64) == 0
    assert M.expert_weight_bytes(M.NVFP4, 3, 200, 128) == (3 * 200 * 64, 3 * 256 * 16)
    assert M.expert_weight_bytes(M.INT8_ROW, 2, 10, 64) == (1280, 80)
    assert M.expert_plan_workspace_bytes(4096, 512) == 0
    assert M.expert_plan_workspace_bytes(1 << 22, 512) > 0
    for bad in ((M.NVFP4, 512, 512, 1 << 22), (M.MXFP8, 1, 513, 64), (M.MXFP8, 1, 0, 64), (M.MXFP8, (1 << 22) + 1, 4, 64), (M.MXFP8, -1, 4, 64),
                (M.MXFP8, 4, 4, 48), (9, 4, 4, 64)):
        with pytest.raises(M.MxqError) as e:
            M.grouped_scales_bytes(*bad)
        assert e.value.status == EINVAL
    for f in (M.INT4_G32, M.INT4_G64):
        with pytest.raises(M.MxqError) as e:
            M.grouped_scales_bytes(f, 4, 4, 64)
        assert e.value.status == EUNSUPPORTED
        with pytest.raises(M.MxqError) as e:
            M.expert_weight_bytes(f, 4, 64, 64)
        assert e.value.status == EUNSUPPORTED


def test_plan_refusals(mxq):
    f = mxq.lib().mxq_expert_plan

    def call(ids=D, bits=32, rows=8, n=4, off=D, slot=D, ws=None, wsb=0):
        return f(ids, bits, rows, n, off, slot, ws, wsb, None)

    for bad in (dict(bits=16), dict(rows=-1), dict(rows=(1 << 22) + 1), dict(n=0), dict(n=513), dict(off=None),
                dict(ids=None), dict(slot=None), dict(off=D + 2), dict(slot=D + 1), dict(ids=D + 4, bits=64),
                dict(rows=100000)):
        assert call(**bad) == EINVAL, bad
    assert call(rows=100000, ws=D, wsb=16) == ENOSPACE


def test_quantize_grouped_refusals(mxq):
    M, f = mxq, mxq.lib().mxq_quantize_grouped

    def call(x=D, dt=1, x_rows=4, cols=64, fmt=M.MXFP8, had=0, off=D, n=4, slot=D, topk=2, rows=8, codes=D, scales=D,
             ts=None, ws=None, wsb=0):
        return f(x, dt, x_rows, cols, fmt, had, off, n, slot, topk, rows, codes, scales, ts, ws, wsb, None)

    for bad in (dict(dt=2), dict(cols=48), dict(cols=0), dict(fmt=7), dict(had=48), dict(had=128), dict(off=None), dict(n=0),
                dict(n=513), dict(topk=0), dict(topk=33), dict(slot=None), dict(slot=None, topk=1, x_rows=9),
                dict(rows=-1), dict(rows=(1 << 22) + 1), dict(x=None), dict(x=D + 8), dict(codes=None), dict(codes=D + 8),
                dict(scales=None), dict(scales=D + 2), dict(off=D + 2), dict(slot=D + 2), dict(fmt=M.NVFP4),
                dict(fmt=M.NVFP4, ts=D), dict(fmt=M.NVFP4, ws=D, wsb=4096)):
        assert call(**bad) == EINVAL, bad
    assert call(fmt=M.FP8_TENSOR, ts=D, ws=D, wsb=64) == ENOSPACE
    for fmt in (M.INT4_G32, M.INT4_G64):
        assert call(fmt=fmt) == EUNSUPPORTED


def weight(M, fmt=0, e=4, rows=64, cols=64, codes=D, scales=D, ts=D):
    return M._ExpertWeightC(fmt, e, rows, cols, codes, scales, ts)


def test_product_refusals(mxq):
    M, f = mxq, mxq.lib().mxq_qlinear_grouped

    def call(fmt=M.MXFP8, layout=M.MMA, rows=8, cols=64, codes=D, scales=D, ts=D, off=D, y=D, yd=1, **w):
        q = M._QTensorC(fmt, layout, rows, cols, codes, scales, ts)
        w = weight(M, **{"fmt": fmt, "cols": cols, **w})
        return f(ctypes.byref(q), off, ctypes.byref(w), y, yd, None)

    for bad in (dict(layout=0), dict(rows=-1), dict(rows=(1 << 22) + 1), dict(off=None), dict(off=D + 2), dict(y=None),
                dict(y=D + 8), dict(yd=5), dict(e=0), dict(e=513), dict(cols=48), dict(cols=0), dict(fmt=M.NVFP4, cols=96),
                dict(fmt=8), dict(fmt=M.NVFP4, ts=None), dict(codes=None), dict(scales=None)):
        assert call(**bad) == EINVAL, bad
    q = M._QTensorC(M.MXFP8, M.MMA, 8, 64, D, D, D)
    for w in (weight(M, codes=None), weight(M, scales=None), weight(M, codes=D + 8), weight(M, cols=128),
              weight(M, e=512, rows=1 << 23), weight(M, e=512, rows=1 << 17, cols=1 << 13)):
        assert f(ctypes.byref(q), D, ctypes.byref(w), D, 1, None) == EINVAL
    assert f(ctypes.byref(q), D, ctypes.byref(weight(M, fmt=M.INT8_ROW)), D, 1, None) == EUNSUPPORTED
    assert call(fmt=M.INT4_G32) == EUNSUPPORTED
    assert f(None, D, ctypes.byref(weight(M)), D, 1, None) == EINVAL
    assert f(ctypes.byref(q), D, None, D, 1, None) == EINVAL
    assert call(rows=0, codes=None, scales=None, y=None) == 0     # nothing to do
    g = mxq.lib().mxq_expert_weight_prepare
    assert g(D, 1, 0, ctypes.byref(weight(M, fmt=M.NVFP4)), None, 0, None) == EINVAL      # no workspace
    assert g(D, 1, 0, ctypes.byref(weight(M, fmt=M.NVFP4)), D, 64, None) == ENOSPACE
    assert g(None, 1, 0, ctypes.byref(weight(M)), None, 0, None) == EINVAL
    assert g(D, 1, 48, ctypes.byref(weight(M)), None, 0, None) == EINVAL


def test_combine_refusals(mxq):
    f = mxq.lib().mxq_expert_combine

    def call(y=D, yd=1, rows=8, n=64, slot=D, w=D, tokens=4, topk=2, out=D, od=1):
        return f(y, yd, rows, n, slot, w, tokens, topk, out, od, None)

    for bad in (dict(yd=3), dict(od=-1), dict(rows=-1), dict(n=-1), dict(tokens=-1), dict(topk=0), dict(topk=33),
                dict(slot=None), dict(out=None), dict(y=None), dict(y=D + 1), dict(out=D + 2, od=0), dict(w=D + 2),
                dict(tokens=1 << 20, n=1 << 11), dict(rows=(1 << 22) + 1)):
        assert call(**bad) == EINVAL, bad
    assert call(tokens=0, slot=None, out=None) == 0


class Heads(ctypes.Structure):   # mxq_heads
    _fields_ = [("q", P), ("k", P), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("q_heads", ctypes.c_int32),
                ("k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("tokens", ctypes.c_int64), ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("q_weight", P),
                ("k_weight", P), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("cos_table", P),
                ("sin_table", P), ("n_positions", ctypes.c_int64), ("positions", P), ("position_bits", ctypes.c_int32)]


def test_packed_descriptors_have_the_c_layout(mxq):
    """What the binding packs is what a C structure of the header's fields holds."""
    vals = [11, 22, 256, 128, 4, 2, 64, 1, 3, 1, 0.5, 33, 44, 64, 1, 55, 66, 10, 77, 64]
    assert mxq._HEADS.pack(*vals) == bytes(Heads(*vals))[:mxq._HEADS.size]
    vals = [2, 1, 5, 64, 11, 22, 33]
    assert mxq._QTENSOR.pack(*vals) == bytes(mxq._QTensorC(*vals))
    assert mxq._EXPERT_WEIGHT.pack(*vals) == bytes(mxq._ExpertWeightC(*vals))


def test_heads_refusals(mxq):
    M, L = mxq, mxq.lib()
    good = dict(q=D, k=D, q_stride=256, k_stride=256, q_heads=4, k_heads=2, head_dim=64, dtype=1, tokens=3, norm=0, eps=1e-6,
                q_weight=D, k_weight=None, rot_dim=64, interleaved=0, cos_table=D, sin_table=D, n_positions=10,
                positions=None, position_bits=32)

    def plain(qo=D, qs=256, ko=D, ks=128, **more):
        h = Heads(**{**good, **more})
        return L.mxq_qk_norm_rope(ctypes.byref(h), qo, qs, ko, ks, None)

    def coded(fmt=0, had=0, qc=D, qs=D, kc=D, ks=D, **more):
        h = Heads(**{**good, **more})
        return L.mxq_qk_norm_rope_quantize(ctypes.byref(h), fmt, had, qc, qs, kc, ks, None)

    shared = (dict(q=None), dict(q=D + 8), dict(q_stride=260), dict(q_stride=248), dict(k_stride=120), dict(k=None), dict(head_dim=60),
              dict(head_dim=264), dict(head_dim=0), dict(dtype=2), dict(tokens=-1), dict(norm=2), dict(eps=-1.0),
              dict(eps=float("nan")), dict(rot_dim=72), dict(rot_dim=4), dict(rot_dim=-8), dict(cos_table=None),
              dict(sin_table=D + 4), dict(n_positions=2), dict(n_positions=0), dict(positions=D, position_bits=16),
              dict(positions=D + 4, position_bits=64), dict(q_weight=D + 4), dict(k_weight=D + 8), dict(q_heads=-1))
    for bad in shared:
        assert plain(**bad) == EINVAL, bad
        assert coded(**bad) == EINVAL, bad
    for bad in (dict(qo=None), dict(qo=D + 2), dict(qs=252), dict(qs=128), dict(ko=None), dict(ks=64)):
        assert plain(**bad) == EINVAL, bad
    for bad in (dict(qc=None), dict(qs=None), dict(kc=D + 8), dict(ks=D + 2), dict(had=48), dict(had=128), dict(fmt=-1),
                dict(head_dim=72, rot_dim=0, q_stride=288, k_stride=288)):
        assert coded(**bad) == EINVAL, bad
    for fmt in (M.NVFP4, M.INT4_G32, M.INT4_G64, M.FP8_TENSOR):
        assert coded(fmt=fmt) == EUNSUPPORTED
    for tokens in (1 << 30, (1 << 31) + 1, 1 << 40, (1 << 63) - 1):   # items of tokens and sides are counted in 31 bits
        many = dict(tokens=tokens, rot_dim=0, cos_table=None, sin_table=None)
        assert plain(**many) == EINVAL and coded(**many) == EINVAL, tokens
        assert plain(**many, k_heads=0, k=None) == EINVAL, tokens
    assert plain(tokens=0, q=None, k=None, qo=None, ko=None) == 0
    assert L.mxq_qk_norm_rope(None, D, 256, D, 128, None) == EINVAL


def test_cpu_tensors_are_refused(mxq):
    import torch
    with pytest.raises(ValueError):
        mxq.expert_plan(torch.zeros(2, 2, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        mxq.qk_norm_rope(torch.zeros(2, 2, 64))
    with pytest.raises(ValueError):
        mxq.expert_combine(torch.zeros(2, 64), torch.zeros(1, 2, dtype=torch.int32))


def test_first_argument_by_name(mxq):
    """Every call takes its first tensor by name too, and says what it takes."""
    import inspect
    import torch
    x = torch.zeros(2, 2, 64)
    for f, kw in ((mxq.expert_plan, dict(expert_ids=x, n_experts=4)), (mxq.quantize_grouped, dict(x=x, fmt=0, offsets=x)),
                  (mxq.prepare_experts, dict(w=x, fmt=0)), (mxq.expert_combine, dict(y=x, slot=x)),
                  (mxq.qk_norm_rope, dict(q=x, k=x)), (mxq.qk_norm_rope_quantize, dict(q=x)),
                  (mxq.qlinear_grouped, dict(xq=mxq.QTensor(0, mxq.MMA, 2, 64, x, None, None), w=None, offsets=x))):
        with pytest.raises(ValueError, match="CUDA device"):   # reached the check of the device
            f(**kw)
        assert list(inspect.signature(f).parameters)[0] in kw and "stream" in inspect.signature(f).parameters
        with pytest.raises(TypeError, match="missing"):
            f()


def test_alloc_refuses_no_groups(mxq):
    for n in (0, -1, 513):
        with pytest.raises(mxq.MxqError):
            mxq.alloc_grouped(mxq.MXFP8, 4, n, 64, device="cpu")


def test_int8_sums_that_could_leave_int32_are_refused(mxq):
    """127 * 127 * K < 2^31 up to K = 133,144: the product of two codes' rows cannot wrap in a call that is accepted."""
    M, L = mxq, mxq.lib()
    most = (2 ** 31 - 1) // 127 ** 2
    assert most == 133144
    good, bad = most // 32 * 32, most // 32 * 32 + 32

    def dense(fmt, k, m=0):
        a, b = M._QTensorC(fmt, M.MMA, m, k, D, D, D), M._QTensorC(fmt, M.MMA, 4, k, D, D, D)
        return L.mxq_qlinear(ctypes.byref(a), ctypes.byref(b), None, None, D, 1, None)

    def grouped(fmt, k, m=0):
        q = M._QTensorC(fmt, M.MMA, m, k, D, D, D)
        return L.mxq_qlinear_grouped(ctypes.byref(q), D, ctypes.byref(weight(M, fmt=fmt, cols=k)), D, 1, None)

    for f in (dense, grouped):
        assert f(M.INT8_ROW, good) == 0               # (no rows: nothing to do)
        assert f(M.INT8_ROW, bad) == EINVAL and f(M.INT8_ROW, bad, 8) == EINVAL
        assert f(M.FP8_TENSOR, bad) == 0
    assert L.mxq_expert_weight_prepare(D, 1, 0, ctypes.byref(weight(M, fmt=M.INT8_ROW, cols=bad)), None, 0, None) == EINVAL


def test_limits_the_header_states(mxq):
    """Each index limit of the grouped product, one step on either side (no rows, or no columns, where accepted)."""
    M, f = mxq, mxq.lib().mxq_qlinear_grouped

    def call(fmt, rows, e, n, k):
        q = M._QTensorC(fmt, M.MMA, rows, k, D, D, D)
        return f(ctypes.byref(q), D, ctypes.byref(weight(M, fmt=fmt, e=e, rows=n, cols=k)), D, 1, None)

    # experts' padded rows: 512 * (n + 1) * 128 < 2^31
    assert call(M.MXFP8, 0, 512, 32766 * 128, 64) == 0 and call(M.MXFP8, 0, 512, 32766 * 128 + 1, 64) == EINVAL
    # experts' scale atoms: 512 * n * (k / 4) < 2^31 with k = 2^14
    assert call(M.MXFP8, 0, 512, 1023 * 128, 1 << 18) == 0 and call(M.MXFP8, 0, 512, 1024 * 128, 1 << 18) == EINVAL
    # items and their K stages: T * n * k < 2^31 with T = 2^15 + 1
    assert call(M.MXFP8, 1 << 22, 1, 512 * 128, 2048) == EINVAL
    assert call(M.MXFP8, 1 << 22, 1, 0, 2048) == 0
    L, more = mxq.lib(), dict(q=D, k=D, head_dim=8, dtype=1, tokens=1, norm=0, eps=1e-6, k_heads=1, k_stride=8)
    h = Heads(**{**more, "q_heads": 65537, "q_stride": 1 << 20})
    assert L.mxq_qk_norm_rope(ctypes.byref(h), D, 1 << 20, D, 8, None) == EINVAL
