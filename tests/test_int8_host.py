"""CPU checks of the 8-bit rows: the oracle's pins, and every refusal of the
C entries for INT8 weights, 8-bit tokens and gradient clipping (all caught on
the host before anything is enqueued, so the addresses are never touched)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from oracle import int8_oracle as I8
from oracle import lbq_oracle as O

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def L():
    import group_wise_minmax_amd as L
    return L


def status(L, rc):
    return L._lib.STATUS[rc]


# ------------------------------------------------------------------ oracle pins

def test_codes_are_the_nearest_multiples_of_the_scale():
    x = np.random.default_rng(1).standard_normal((5, 192)).astype(np.float32)
    q, s = I8.quantize_rows(x)
    for i in range(5):
        assert s[i] == np.float32(np.abs(x[i]).max()) / np.float32(127)
        assert np.abs(q[i]).max() == 127
        for v, c in zip(x[i], q[i]):
            t = Fraction(float(v)) / Fraction(float(s[i]))
            # nearest whole number, up to the one rounding of the fp32 quotient
            assert abs(t - int(c)) <= Fraction(1, 2) + abs(t) / 2 ** 24


def test_codes_at_exact_ties_go_to_the_even_number():
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :6] = [127, 0.5, 1.5, 2.5, -0.5, -1.5]  # scale exactly 1
    q, s = I8.quantize_rows(x)
    assert s[0] == 1 and q[0, :6].tolist() == [127, 0, 2, 2, 0, -2]


def test_rows_of_zeros_subnormals_and_nonfinite_values():
    x = np.zeros((5, 64), dtype=np.float32)
    x[1, 3] = 2.0 ** -149
    x[2, 3], x[2, 4] = 2.0 ** -142, -2.0 ** -142
    x[3, 5], x[3, 6] = np.inf, 1
    x[4, 7], x[4, 8] = np.nan, 1
    q, s = I8.quantize_rows(x)
    assert s[0] == 1 and not q[0].any()
    assert s[1] == 1 and not q[1].any()
    assert s[2] == 2.0 ** -149 and q[2, 3] == 127 and q[2, 4] == -127  # 128 steps, held at 127
    assert np.isnan(s[3]) and np.isnan(s[4]) and not q[3:].any()


def test_product_of_whole_numbers():
    rng = np.random.default_rng(2)
    a, b = rng.integers(-127, 128, (3, 128)), rng.integers(-127, 128, (4, 128))
    y = I8.product(a.astype(np.int8), np.full(3, 0.5, np.float32), b.astype(np.int8), np.full(4, 2.0, np.float32))
    assert np.array_equal(y, (a @ b.T).astype(np.float32))
    assert np.array_equal(I8.product_bf16(a.astype(np.int8), np.ones(3, np.float32), b.astype(np.int8),
                                          np.ones(4, np.float32)), O.bf16_bits((a @ b.T).astype(np.float32)))


def test_norm_and_factor():
    assert I8.grad_norm([np.array([3.0]), np.array([[4.0]])]) == 5.0
    assert I8.grad_norm([np.array([3.0]), np.array([[-4.0]]), np.array([])], "inf") == 4.0
    assert I8.clip_factor(0.5, 1.0) == 1.0 and abs(I8.clip_factor(4.0, 1.0) - 0.25) < 1e-6


# ------------------------------------------------------------------ descriptors

def test_layout_and_blob_size(L):
    d = L.make_desc("int8", 1001, 4160)
    assert (d.format, d.bits, d.group, d.double_quant, d.dq_block, d.meta) == (2, 8, 0, 0, 0, 0)
    s = L.lbq_layout(d)
    assert s["packed"] == 1001 * 4160 and s["scales"] == 4 * 1001
    assert s["zeros"] == s["absmax"] == s["absmax_q"] == s["absmax_scale"] == 0
    assert L.lib.lbq_serialized_bytes(ctypes.byref(d)) == 96 + 1001 * 4160 + 4016


@pytest.mark.parametrize("kw,code", [
    (dict(bits=4), "LBQ_E_FORMAT"), (dict(group=128), "LBQ_E_FORMAT"), (dict(double_quant=1), "LBQ_E_FORMAT"),
    (dict(dq_block=256), "LBQ_E_FORMAT"), (dict(meta=1), "LBQ_E_FORMAT"), (dict(k=96), "LBQ_E_SHAPE"),
    (dict(k=0), "LBQ_E_SHAPE"), (dict(k=(1 << 17) + 64), "LBQ_E_SHAPE"), (dict(n=0), "LBQ_E_SHAPE"),
    (dict(format=3), "LBQ_E_FORMAT"),
])
def test_layout_refusals(L, kw, code):
    d = L.make_desc("int8", 64, 256)
    for k, v in kw.items():
        setattr(d, k, v)
    with pytest.raises(L.LbqError) as e:
        L.lbq_layout(d)
    assert e.value.name == code


def q_of(L, **kw):
    q = L.QTensor()
    q.packed, q.scales = FAKE, FAKE + 0x100000
    for k, v in kw.items():
        setattr(q, k, v)
    return q


# ------------------------------------------------------------------ forward

@pytest.mark.parametrize("kw,code", [
    (dict(X=None), "LBQ_E_NULL"), (dict(Y=None), "LBQ_E_NULL"), (dict(X=FAKE + 8), "LBQ_E_ALIGN"),
    (dict(Y=FAKE + 1), "LBQ_E_ALIGN"), (dict(m=-1), "LBQ_E_SHAPE"), (dict(ldy=63), "LBQ_E_SHAPE"),
    (dict(scales=None), "LBQ_E_NULL"), (dict(scales=FAKE + 2), "LBQ_E_ALIGN"), (dict(packed=FAKE + 4), "LBQ_E_ALIGN"),
    (dict(packed=None), "LBQ_E_NULL"), (dict(ws=None), "LBQ_E_WORKSPACE"), (dict(short=1), "LBQ_E_WORKSPACE"),
    (dict(ws=FAKE + 8), "LBQ_E_ALIGN"), (dict(n=(1 << 23) - 255), "LBQ_E_SHAPE"),
])
@pytest.mark.parametrize("m", [7, 65, 300])
def test_linear_fwd_refusals(L, kw, code, m):
    a = dict(X=FAKE, Y=FAKE, m=m, ldy=64, n=64, ws=FAKE, short=0)
    a.update({k: v for k, v in kw.items() if k in a})
    q = q_of(L, **{k: v for k, v in kw.items() if k in ("packed", "scales")})
    d = L.make_desc("int8", a["n"], 256)
    if "n" in kw:
        a["ldy"] = a["n"]
    need = L.lib.lbq_linear_workspace_bytes(ctypes.byref(d), m)
    assert need >= m * 256 + 4 * m
    rc = L.lib.lbq_linear_fwd(ctypes.byref(d), ctypes.byref(q), a["X"], a["m"], a["Y"], a["ldy"], a["ws"],
                              need - a["short"], None)
    assert status(L, rc) == code, L.lib.lbq_last_error_detail()
    descs, qs = (L.Desc * 1)(d), (L.QTensor * 1)(q)
    need = L.lib.lbq_linear_fwd_grouped_workspace_bytes(1, descs, m)
    rc = L.lib.lbq_linear_fwd_grouped(1, descs, qs, a["X"], a["m"], (ctypes.c_void_p * 1)(a["Y"]),
                                      (ctypes.c_int64 * 1)(a["ldy"]), a["ws"], need - a["short"], None)
    assert status(L, rc) == code


def test_grouped_workspace_covers_the_8_bit_weights_of_a_mixed_set(L):
    i8, i4 = L.make_desc("int8", 256, 4096), L.make_desc("minmax", 256, 4096)
    for m in (1, 3, 16, 100, 1000):
        one = L.lib.lbq_linear_workspace_bytes(ctypes.byref(i8), m)
        both = L.lib.lbq_linear_fwd_grouped_workspace_bytes(2, (L.Desc * 2)(i4, i8), m)
        assert both >= one
        q = q_of(L, zeros=FAKE)
        rc = L.lib.lbq_linear_fwd_grouped(2, (L.Desc * 2)(i4, i8), (L.QTensor * 2)(q, q), FAKE, m,
                                          (ctypes.c_void_p * 2)(FAKE, FAKE), (ctypes.c_int64 * 2)(256, 256), None, 0, None)
        if one:
            assert status(L, rc) == "LBQ_E_WORKSPACE"
    assert L.lib.lbq_linear_fwd_grouped_workspace_bytes(1, (L.Desc * 1)(i8), 0) == 0
    assert L.lib.lbq_linear_workspace_bytes(ctypes.byref(i8), 0) == 0


def test_noalloc_refuses_more_than_its_scratch(L):
    d = L.make_desc("int8", 64, 8192)
    q = q_of(L)
    rc = L.lib.lbq_linear_fwd_noalloc(ctypes.byref(d), ctypes.byref(q), FAKE, -1, FAKE, 64, None)
    assert status(L, rc) == "LBQ_E_SHAPE"


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), "LBQ_E_SHAPE"), (dict(k=32), "LBQ_E_SHAPE"), (dict(k=100), "LBQ_E_SHAPE"),
    (dict(k=(1 << 17) + 64, ldx=1 << 18), "LBQ_E_SHAPE"), (dict(ldx=248), "LBQ_E_SHAPE"), (dict(ldx=260), "LBQ_E_ALIGN"),
    (dict(X=None), "LBQ_E_NULL"), (dict(Q=None), "LBQ_E_NULL"), (dict(s=None), "LBQ_E_NULL"),
    (dict(X=FAKE + 8), "LBQ_E_ALIGN"), (dict(Q=FAKE + 8), "LBQ_E_ALIGN"), (dict(s=FAKE + 2), "LBQ_E_ALIGN"),
])
def test_quantize_tokens_refusals(L, kw, code):
    a = dict(X=FAKE, m=3, k=256, ldx=256, Q=FAKE, s=FAKE)
    a.update(kw)
    rc = L.lib.lbq_quantize_tokens(a["X"], a["m"], a["k"], a["ldx"], a["Q"], a["s"], None)
    assert status(L, rc) == code


@pytest.mark.parametrize("kw,code", [
    (dict(fmt="minmax"), "LBQ_E_UNSUPPORTED"), (dict(X=None), "LBQ_E_NULL"), (dict(s=None), "LBQ_E_NULL"),
    (dict(s=FAKE + 1), "LBQ_E_ALIGN"), (dict(X=FAKE + 1), "LBQ_E_ALIGN"), (dict(Y=None), "LBQ_E_NULL"),
    (dict(ldy=10), "LBQ_E_SHAPE"), (dict(m=1 << 31), "LBQ_E_SHAPE"), (dict(m=(1 << 23) - 256), "LBQ_E_SHAPE"),
])
def test_linear_fwd_tokens_refusals(L, kw, code):
    a = dict(fmt="int8", X=FAKE, s=FAKE, Y=FAKE, m=5, ldy=64)
    a.update(kw)
    d = L.make_desc(a["fmt"], 64, 256)
    q = q_of(L, zeros=FAKE)
    rc = L.lib.lbq_linear_fwd_tokens(ctypes.byref(d), ctypes.byref(q), a["X"], a["s"], a["m"], a["Y"], a["ldy"], FAKE,
                                     1 << 40, None)
    assert status(L, rc) == code


def test_empty_batches_pass_without_a_launch(L):
    d, q = L.make_desc("int8", 64, 256), q_of(L)
    assert L.lib.lbq_linear_fwd(ctypes.byref(d), ctypes.byref(q), None, 0, None, 64, None, 0, None) == 0
    assert L.lib.lbq_linear_fwd_tokens(ctypes.byref(d), ctypes.byref(q), None, None, 0, None, 64, None, 0, None) == 0
    assert L.lib.lbq_linear_bwd_dx(ctypes.byref(d), ctypes.byref(q), None, 0, None, None) == 0
    assert L.lib.lbq_quantize_tokens(None, 0, 256, 256, None, None, None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(n=60), "LBQ_E_SHAPE"), (dict(dY=None), "LBQ_E_NULL"), (dict(dX=FAKE + 2), "LBQ_E_ALIGN"),
    (dict(rows=FAKE), "LBQ_E_UNSUPPORTED"), (dict(scales=None), "LBQ_E_NULL"), (dict(n=1 << 23), "LBQ_E_SHAPE"),
])
def test_linear_bwd_dx_refusals(L, kw, code):
    a = dict(n=64, dY=FAKE, dX=FAKE)
    a.update({k: v for k, v in kw.items() if k in a})
    d = L.make_desc("int8", a["n"], 256)
    q = q_of(L, out_rows=kw.get("rows"), **({"scales": None} if "scales" in kw else {}))
    rc = L.lib.lbq_linear_bwd_dx(ctypes.byref(d), ctypes.byref(q), a["dY"], 3, a["dX"], None)
    assert status(L, rc) == code


# ------------------------------------------------------------------ gradients

def grads_of(L, *entries):
    t = (L.Grad * len(entries))()
    for e, (grad, out, numel, dtype) in zip(t, entries):
        e.grad, e.out, e.numel, e.dtype = grad, out, numel, dtype
    return t


A = FAKE
OK = [(A, A, 100, 0), (A + 4096, A + 8192, 100, 1)]


@pytest.mark.parametrize("entries,kw,code", [
    (OK, dict(count=0), "LBQ_E_SHAPE"), (OK, dict(count=-1), "LBQ_E_SHAPE"), (OK, dict(table=None), "LBQ_E_NULL"),
    (OK, dict(kind=2), "LBQ_E_FORMAT"), (OK, dict(norm=None), "LBQ_E_NULL"), (OK, dict(norm=A + 2), "LBQ_E_ALIGN"),
    (OK, dict(ws=None), "LBQ_E_WORKSPACE"), (OK, dict(short=16), "LBQ_E_WORKSPACE"), (OK, dict(ws=A + 8), "LBQ_E_ALIGN"),
    (OK, dict(max_norm=0.0), "LBQ_E_SHAPE"), (OK, dict(max_norm=-1.0), "LBQ_E_SHAPE"),
    (OK, dict(max_norm=float("nan")), "LBQ_E_SHAPE"), (OK, dict(max_norm=float("inf")), "LBQ_E_SHAPE"),
    ([(A, A, -1, 0)], {}, "LBQ_E_SHAPE"), ([(A, A, (1 << 40) + 1, 0)], {}, "LBQ_E_SHAPE"),
    ([(A, A, 8, 3)], {}, "LBQ_E_FORMAT"), ([(None, A, 8, 0)], {}, "LBQ_E_NULL"), ([(A, None, 8, 0)], {}, "LBQ_E_NULL"),
    ([(A + 2, A, 8, 0)], {}, "LBQ_E_ALIGN"), ([(A, A + 1, 8, 1)], {}, "LBQ_E_ALIGN"),
    # the same tensor twice; one output inside another; an output over another's gradient, or shifted over its own
    ([(A, A, 8, 0), (A, A, 8, 0)], {}, "LBQ_E_SHAPE"),
    ([(A, A + 4096, 64, 0), (A + 1024, A + 4100, 8, 0)], {}, "LBQ_E_SHAPE"),
    ([(A, A + 4096, 64, 0), (A + 4096, A + 8192, 64, 0)], {}, "LBQ_E_SHAPE"),
    ([(A, A + 4, 64, 0)], {}, "LBQ_E_SHAPE"),
    ([(A, A, 64, 0), (A + 64, A + 64, 3, 1)], {}, "LBQ_E_SHAPE"),
])
def test_clip_refusals(L, entries, kw, code):
    a = dict(count=len(entries), table=grads_of(L, *entries), kind=0, norm=A, ws=A, short=0, max_norm=1.0)
    a.update(kw)
    need = L.lib.lbq_grad_workspace_bytes(2, grads_of(L, *OK))
    assert need >= 16
    rc = L.lib.lbq_clip_grads(a["count"], a["table"], a["kind"], a["max_norm"], a["norm"], a["ws"], need - a["short"], None)
    assert status(L, rc) == code, L.lib.lbq_last_error_detail()


def test_norm_refusals_and_workspace(L):
    t = grads_of(L, *OK)
    assert status(L, L.lib.lbq_grad_norm(2, t, 5, A, A, 1 << 20, None)) == "LBQ_E_FORMAT"
    assert status(L, L.lib.lbq_grad_norm(2, t, 0, None, A, 1 << 20, None)) == "LBQ_E_NULL"
    assert status(L, L.lib.lbq_grad_norm(2, t, 0, A, None, 0, None)) == "LBQ_E_WORKSPACE"
    # the workspace does not grow with the gradients: one partial sum a workgroup, and a launch takes 120 tensors
    big = grads_of(L, *[(A, A, 1 << 30, 0)] * 300)
    assert 0 < L.lib.lbq_grad_workspace_bytes(300, big) <= 3 * 8 * 2048
    assert L.lib.lbq_grad_workspace_bytes(1, grads_of(L, (None, None, 0, 0))) == 0


def test_sizes_that_are_refused_take_no_workspace(L):
    d = L.make_desc("int8", 64, 256)
    for m in ((1 << 23) - 256, 1 << 31, (1 << 63) - 1):
        assert L.lib.lbq_linear_workspace_bytes(ctypes.byref(d), m) == 0
        assert L.lib.lbq_linear_fwd_tokens_workspace_bytes(ctypes.byref(d), m) == 0
        assert L.lib.lbq_linear_bwd_dx_grouped_workspace_bytes(1, ctypes.byref(d), m) == 0
    assert L.lib.lbq_linear_workspace_bytes(ctypes.byref(d), (1 << 23) - 257) >= ((1 << 23) - 257) * 260


@pytest.mark.parametrize("kw,code", [
    (dict(count=0), "LBQ_E_SHAPE"), (dict(count=9), "LBQ_E_SHAPE"), (dict(other="minmax"), "LBQ_E_UNSUPPORTED"),
    (dict(other_k=512), "LBQ_E_SHAPE"), (dict(ws=FAKE + 8), "LBQ_E_ALIGN"), (dict(dY=None), "LBQ_E_NULL"),
    (dict(m=-1), "LBQ_E_SHAPE"), (dict(m=(1 << 23) - 256), "LBQ_E_SHAPE"), (dict(dX=FAKE + 8), "LBQ_E_ALIGN"),
])
def test_bwd_dx_grouped_ws_refusals(L, kw, code):
    a = dict(count=2, other="int8", other_k=256, ws=FAKE, dY=FAKE, m=40, dX=FAKE)
    a.update(kw)
    descs = (L.Desc * 2)(L.make_desc("int8", 64, 256), L.make_desc(a["other"], 64, a["other_k"]))
    qts = (L.QTensor * 2)(q_of(L), q_of(L, zeros=FAKE))
    dys = (ctypes.c_void_p * 2)(FAKE, a["dY"])
    rc = L.lib.lbq_linear_bwd_dx_grouped_ws(a["count"], descs, qts, dys, a["m"], a["dX"], a["ws"], 1 << 30, None)
    assert status(L, rc) == code


@pytest.mark.parametrize("norm,ws,clip", [
    (A + 8, A + (1 << 20), False), (A + 396, A + (1 << 20), True),  # the norm in a gradient, at its end
    (A + 8192, A + (1 << 20), True),                                # in an output
    (A + (1 << 20), A + 4096, False), (A + (1 << 20), A + 8192 + 192, True),  # the workspace over a gradient, an output
    (A + (1 << 20) + 12, A + (1 << 20), False),                     # one in the other
])
def test_norm_and_workspace_stay_outside_the_tensors(L, norm, ws, clip):
    t = grads_of(L, *OK)
    if clip:
        rc = L.lib.lbq_clip_grads(2, t, 0, 1.0, norm, ws, 1 << 10, None)
    else:
        rc = L.lib.lbq_grad_norm(2, t, 0, norm, ws, 1 << 10, None)
    assert status(L, rc) == "LBQ_E_SHAPE"


def test_python_refusals_without_a_device(L):
    import torch
    with pytest.raises(ValueError):
        L.LbqGradSet([])
    with pytest.raises(ValueError):
        L.LbqGradSet([torch.zeros(4)])
    with pytest.raises(ValueError):
        L.lbq_quantize_tokens(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        L.make_desc("int7", 64, 64)


@pytest.mark.parametrize("numels", [
    (8, (1 << 63) - 1), ((1 << 63) - 1, 8), (1 << 39, 1 << 39, 1), (8, (1 << 63) - 8, 8), ((1 << 40) + 1,), (8, -1),
    ((1 << 40), (1 << 63) - 1, (1 << 63) - 1),
])
def test_sizes_of_gradients_are_bounded_in_all(L, numels):
    """More than 2^40 values over all the tensors, also where their sum passes 64 bits."""
    t = grads_of(L, *[(A, A + (1 << 44) * (i + 1), n, 0) for i, n in enumerate(numels)])
    far = A - (1 << 20)
    assert L.lib.lbq_grad_workspace_bytes(len(numels), t) == 0
    assert status(L, L.lib.lbq_grad_norm(len(numels), t, 0, far, far + 64, 1 << 18, None)) == "LBQ_E_SHAPE"
    assert status(L, L.lib.lbq_clip_grads(len(numels), t, 0, 1.0, far, far + 64, 1 << 18, None)) == "LBQ_E_SHAPE"
    full = grads_of(L, *[(A, A, 1 << 39, 0)] * 2)
    assert L.lib.lbq_grad_workspace_bytes(2, full) == 8 * 2048


def host_set(L, grads, outs=None):
    """A set of CPU tensors, for its table alone (no call takes it)."""
    s = object.__new__(L.LbqGradSet)
    s._grads, s._outs, s.device = grads, grads if outs is None else outs, grads[0].device
    s._tensors, s._table, s._seen = grads + (outs or []), (L.Grad * len(grads))(), None
    s._look()
    return s


def entries(s):
    return [(e.grad, e.out, e.numel, e.dtype) for e in s._table]


@pytest.mark.parametrize("place", ["grads", "outs"])
def test_set_sees_another_type_at_the_same_address(L, place):
    """As many bf16 values at the address of fp32 ones, and fp16 seen as bf16."""
    import torch
    for first, view, code in ((torch.float32, torch.bfloat16, 1), (torch.float16, torch.bfloat16, 1), (torch.float32, torch.float16, 2)):
        g, o = torch.zeros(100, dtype=first), torch.zeros(100, dtype=first)
        s = host_set(L, [g], [o])
        moved = g if place == "grads" else o
        moved.data = moved.data.view(view)[:100]
        with pytest.raises(ValueError):  # the other one is still of the first type
            s._look()
        s = host_set(L, [g := torch.zeros(100, dtype=first)])
        g.data = g.data.view(view)[:100]
        s._look()
        assert entries(s) == [(g.data_ptr(), g.data_ptr(), 100, code)]
        g.data = torch.zeros(100, dtype=torch.float64)
        with pytest.raises(ValueError):
            s._look()


@pytest.mark.parametrize("place", ["grads", "outs"])
def test_set_refuses_a_strided_view_at_the_same_address(L, place):
    import torch
    bufs = [torch.zeros(200), torch.zeros(200)]
    g, o = bufs[0][:100], bufs[1][:100]
    s = host_set(L, [g], [o])
    moved, buf = (g, bufs[0]) if place == "grads" else (o, bufs[1])
    moved.data = buf[::2]
    assert moved.numel() == 100 and moved.data_ptr() == buf.data_ptr()
    with pytest.raises(ValueError):
        s._look()
    m = torch.zeros(10, 10)
    s = host_set(L, [m])
    m.t_()
    with pytest.raises(ValueError):
        s._look()


def test_set_fills_its_table_again_after_a_refusal(L):
    """A first tensor that moved beside a second one that is refused; both back in
    their places the table is that of the first look."""
    import torch
    a, b = torch.zeros(50), torch.zeros(60)
    at, bt = a.data, b.data
    s = host_set(L, [a, b])
    want = entries(s)
    a.data, b.data = torch.zeros(70), torch.zeros(120)[::2]
    with pytest.raises(ValueError):
        s._look()
    a.data, b.data = at, bt
    s._look()
    assert entries(s) == want


def test_serialization_runs_on_the_weights_device(L, monkeypatch):
    """The copies go to a stream of the weight's device: that device is current
    around them (a default stream is the current device's)."""
    import contextlib
    import types

    import torch
    qw = L.QuantizedWeight.empty(L.make_desc("int8", 3, 64), "cpu")
    blob = bytes(96 + 192 + 16)
    inside, calls = [], []

    @contextlib.contextmanager
    def on(device):
        inside.append(device)
        yield
        inside.pop()

    def copies(*args):
        calls.append(list(inside))
        return 0

    def desc_of(_blob, _size, d):
        d._obj.__init__(*[getattr(qw.desc, f) for f, _ in L.Desc._fields_])
        return 0

    fake = types.SimpleNamespace(lbq_serialize=copies, lbq_deserialize=copies, lbq_blob_desc=desc_of,
                                 lbq_serialized_bytes=lambda d: len(blob), lbq_layout=L.lib.lbq_layout)
    monkeypatch.setattr(L, "lib", fake)
    monkeypatch.setattr(L, "_on", on)
    monkeypatch.setattr(L, "_stream", lambda device: None)
    assert len(qw.to_bytes()) == len(blob)
    back = L.QuantizedWeight.from_bytes(blob, "cpu")
    assert (back.n, back.k) == (3, 64)
    assert calls == [[torch.device("cpu")]] * 2
