"""Global gradient norm and clipping on the GPU.

The norm is rounded once from an fp64 sum (2^-24 relative, doubled here for the
square root of the fp64 sum); a scaled value carries the roundings of norm,
norm + 1e-6, the quotient, and the product: five half steps of fp32, and one of
its own type."""
import math

import numpy as np
import pytest
import torch

from oracle import int8_oracle as I8
from gpu_util import DEV

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
HALF = {t: torch.finfo(t).eps / 2 for t in TYPES}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.fixture(scope="module")
def L():
    import group_wise_minmax_amd as L
    assert torch.cuda.is_available()
    return L


def made(sizes, dtypes, seed=0, scale=0.01):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(s, generator=gen, device=DEV) * scale).to(dtypes[i % len(dtypes)]) for i, s in enumerate(sizes)]


def wide(ts):
    return [t.double().cpu().numpy() for t in ts]


def check(L, grads, max_norm, kind="2", outs=None):
    before = wide(grads)
    want = I8.grad_norm(before, kind)
    norm = L.lbq_grad_norm(grads, float(kind))
    assert norm.dtype == torch.float32 and norm.dim() == 0
    assert abs(float(norm) - want) <= 2 * 2 ** -24 * want
    for g, b in zip(grads, before):
        assert np.array_equal(g.double().cpu().numpy(), b)  # the norm alone writes nothing
    again = L.LbqGradSet(grads, outs).clip(max_norm, float(kind))
    assert torch.equal(again, norm)
    c = I8.clip_factor(want, max_norm)
    for g, o, b in zip(grads, outs or grads, before):
        tol = (HALF[g.dtype] + 6 * 2 ** -24) * np.abs(b * c) + TINY[g.dtype]
        assert (np.abs(o.double().cpu().numpy() - b * c) <= tol).all()
        if c == 1.0:
            assert np.array_equal(o.double().cpu().numpy(), b)
        if outs is not None:
            assert np.array_equal(g.double().cpu().numpy(), b)


SIZES = [
    [1], [3], [4095], [4096], [4097], [16384 * 3 + 5], [1, 1, 1], [0, 7, 0, 0, 100], [100003, 1, 5000, 77, 262144],
    [(16, 4096), (4096, 16), (13, 1000), (1000, 13)],
]


@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("dtypes", [TYPES[:1], TYPES[1:2], TYPES[2:], TYPES], ids=["f32", "bf16", "f16", "mixed"])
def test_norm_and_clip(L, sizes, dtypes):
    for kind in ("2", "inf"):
        for max_norm in (1e-3, 1e9):
            grads = made(sizes, dtypes)
            check(L, grads, max_norm, kind)
            grads = made(sizes, dtypes, 1)
            check(L, grads, max_norm, kind, [torch.full_like(g, 9.0) for g in grads])


@pytest.mark.parametrize("count", [119, 120, 121, 700])
def test_more_tensors_than_one_launch_takes(L, count):
    rng = np.random.default_rng(count)
    sizes = [int(v) for v in rng.integers(0, 3000, count)]
    grads = made(sizes, TYPES, count)
    check(L, grads, 0.05)
    grads = made(sizes, TYPES, count)
    check(L, grads, 0.001, "inf", [torch.empty_like(g) for g in grads])


def test_many_values(L):
    """More pieces than workgroups, over several launches."""
    grads = made([(64, 14336), (14336, 64)] * 70, TYPES[:2], 4)
    total = sum(float(g.double().square().sum()) for g in grads)
    outs = [torch.empty_like(g) for g in grads]
    norm = L.LbqGradSet(grads, outs).clip(0.5)
    assert abs(float(norm) - math.sqrt(total)) <= 1e-6 * math.sqrt(total)
    c = 0.5 / (math.sqrt(total) + 1e-6)
    for g, o in zip(grads, outs):
        d = (o.double() - g.double() * c).abs()
        assert bool((d <= (HALF[g.dtype] + 6 * 2 ** -24) * (g.double() * c).abs() + TINY[g.dtype]).all())


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_tensors_at_any_alignment(L, dtype, shift):
    """Views that start and end inside a buffer: the values around them stay."""
    buf = made([20000], [dtype], shift)[0]
    keep = buf.clone()
    views = [buf[shift:shift + 4001], buf[6000 + shift:6000 + shift + 9001], buf[19000:19000 + shift]]
    check(L, views, 0.01)
    mask = torch.ones(20000, dtype=torch.bool, device=DEV)
    for a, n in ((shift, 4001), (6000 + shift, 9001), (19000, shift)):
        mask[a:a + n] = False
    assert torch.equal(buf[mask], keep[mask])
    # outputs aligned differently from the gradients
    out = torch.full((30000,), 3.0, dtype=dtype, device=DEV)
    grads = made([4001, 9001], [dtype], 9)
    check(L, grads, 0.01, outs=[out[shift:shift + 4001], out[10000:10000 + 9001]])
    rest = torch.cat([out[:shift], out[shift + 4001:10000], out[19001:]])
    assert (rest == 3.0).all()


@pytest.mark.parametrize("kind", [2.0, float("inf")])
def test_values_of_every_magnitude(L, kind):
    """Squares beyond fp32 in both directions, zeros, infinities and NaN."""
    big = torch.full((5000,), 1e30, device=DEV)
    want = 1e30 * math.sqrt(5000) if kind == 2.0 else 1e30
    assert abs(float(L.lbq_grad_norm([big], kind)) / want - 1) < 1e-6
    small = torch.full((5000,), 1e-30, device=DEV)
    want = 1e-30 * math.sqrt(5000) if kind == 2.0 else 1e-30
    assert abs(float(L.lbq_grad_norm([small], kind)) / want - 1) < 1e-6
    zero = torch.zeros(777, device=DEV)
    assert float(L.lbq_clip_grad_norm_([zero], 1.0, kind)) == 0.0 and not zero.any()
    if kind == 2.0:  # a norm beyond fp32 is infinite, as is its sum in fp32
        huge = torch.full((5000,), 3e38, device=DEV)
        assert math.isinf(float(L.lbq_grad_norm([huge], kind)))
    for bad, dtype in ((math.inf, torch.float32), (-math.inf, torch.bfloat16), (math.inf, torch.float16)):
        g, h = torch.ones(4100, device=DEV).to(dtype), torch.ones(10, device=DEV)
        g[4099] = bad
        assert math.isinf(float(L.lbq_clip_grad_norm_([g, h], 1.0, kind)))
        assert bool(torch.isnan(g[4099])) and not g[:4099].any() and not h.any()
    for dtype in TYPES:
        g, h = torch.ones(4100, device=DEV).to(dtype), torch.ones(10, device=DEV)
        g[2] = math.nan
        assert math.isnan(float(L.lbq_clip_grad_norm_([h, g], 1.0, kind)))
        assert bool(torch.isnan(g).all()) and bool(torch.isnan(h).all())


def test_repeats_bit_for_bit(L):
    grads = made([100000, 33, 5000000], TYPES[:1], 7)
    outs = [torch.empty_like(g) for g in grads]
    s = L.LbqGradSet(grads, outs)
    first = s.clip(0.1), [o.clone() for o in outs]
    for _ in range(5):
        assert torch.equal(s.clip(0.1), first[0])
        assert all(torch.equal(a, b) for a, b in zip(outs, first[1]))


def test_set_follows_tensors_that_move(L):
    g = torch.nn.Parameter(torch.zeros(50, device=DEV))
    g.grad = torch.ones(50, device=DEV)
    grad = g.grad
    s = L.LbqGradSet([grad])
    assert abs(float(s.norm()) - math.sqrt(50)) < 1e-5
    grad.data = torch.full((50,), 2.0, device=DEV)
    assert abs(float(s.norm()) - 2 * math.sqrt(50)) < 1e-5
    grad.data = torch.full((60,), 2.0, device=DEV)
    assert abs(float(s.norm()) - 2 * math.sqrt(60)) < 1e-5
    grad.data = torch.zeros(60, device=DEV, dtype=torch.float64)
    with pytest.raises(ValueError):
        s.norm()


def test_graph_replays(L):
    """Two captured clippings and an eager one between the replays."""
    a, b = made([9000, 31], TYPES[:2], 1), made([70000], TYPES[:1], 2)
    oa, ob = [torch.empty_like(t) for t in a], [torch.empty_like(t) for t in b]
    sa, sb = L.LbqGradSet(a, oa), L.LbqGradSet(b, ob)
    sa.clip(0.1), sb.clip(0.1)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        na = sa.clip(0.1)
    with torch.cuda.graph(gb):
        nb = sb.clip(0.1)
    for turn in range(4):
        for t in a + b:
            t.copy_(torch.randn(t.shape, device=DEV) * (0.01 + turn))
        ga.replay(), gb.replay()
        torch.cuda.synchronize()
        got = na.clone(), nb.clone(), [o.clone() for o in oa + ob]
        ea, eb = sa.clip(0.1), sb.clip(0.1)
        torch.cuda.synchronize()
        assert torch.equal(got[0], ea) and torch.equal(got[1], eb)
        assert all(torch.equal(x, y) for x, y in zip(got[2], oa + ob))


def test_two_streams_at_once(L):
    sets = [made([400000, 17], TYPES[:1], i) for i in range(2)]
    want = [I8.grad_norm(wide(s)) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    norms = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            norms.append(L.lbq_grad_norm(sets[i % 2]))
    torch.cuda.synchronize()
    for i, n in enumerate(norms):
        assert abs(float(n) - want[i % 2]) <= 2 ** -23 * want[i % 2]


def test_refusals(L):
    g = torch.ones(10, device=DEV)
    for bad in ([g, g], [g, g[5:]]):
        with pytest.raises(L.LbqError) as e:
            L.lbq_clip_grad_norm_(bad, 1.0)
        assert e.value.name == "LBQ_E_SHAPE"
    assert abs(float(L.lbq_grad_norm([g, g])) - math.sqrt(20)) < 1e-5  # a tensor listed twice counts twice
    for kw in (dict(norm_type=1.0), dict(norm_type=0.0)):
        with pytest.raises(ValueError):
            L.lbq_grad_norm([g], **kw)
    for max_norm in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(L.LbqError):
            L.lbq_clip_grad_norm_([g], max_norm)
    for bad in ([g.double()], [torch.ones((4, 4), device=DEV).t()[:, 1:]], [g, torch.ones(3)], []):
        with pytest.raises(ValueError):
            L.lbq_grad_norm(bad)
    with pytest.raises(ValueError):
        L.LbqGradSet([g], [g.half()])
    with pytest.raises(ValueError):
        L.LbqGradSet([g], [g[:5]])
    with pytest.raises(ValueError):
        L.LbqGradSet([g], [])
    assert torch.equal(g, torch.ones(10, device=DEV))


def test_set_follows_tensors_that_change_type_or_layout(L):
    """A view of another type or stride that begins where the tensor did and has as
    many values: scaled as what it is, or refused, and nothing beside it is written."""
    buf = made([200], TYPES[1:2], 3)[0].float()  # finite as bf16 too
    keep = buf.clone()
    g = buf[:100]
    s = L.LbqGradSet([g])
    g.data = buf.view(torch.bfloat16)[:100]
    before = wide([g])
    want = I8.grad_norm(before)
    assert abs(float(s.clip(0.5 * want)) - want) <= 2 ** -23 * want
    c = I8.clip_factor(want, 0.5 * want)
    tol = (HALF[torch.bfloat16] + 6 * 2 ** -24) * np.abs(before[0] * c) + TINY[torch.bfloat16]
    assert (np.abs(wide([g])[0] - before[0] * c) <= tol).all()
    assert torch.equal(buf[50:], keep[50:])
    keep = buf.clone()
    g.data = buf[::2]
    for call in (s.norm, lambda: s.clip(1e-3)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(buf.view(torch.int32), keep.view(torch.int32))
    g.data = buf[100:]
    assert abs(float(s.norm()) - I8.grad_norm(wide([buf[100:]]))) <= 1e-6
