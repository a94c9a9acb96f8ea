"""Every kernel and tile of the 8-bit products and input gradients (the sizes and
the path that each takes: int8_paths, asked of the dispatch rule by the CPU
tests) against the definitions in 64 bits on the GPU.

Products are bit-exact: sums of products of codes are exact in fp64, whatever
their order, and three fp32 roundings and one to bf16 follow.  Gradients and
adapter terms are held to the bounds of their roundings: half a bf16 step, 2^-8
of the value, where something is rounded to bf16, and (n + 2) 2^-24 of the sum of
the magnitudes for an fp32 sum of n terms, doubled for the MFMA's own order.
"""
import ctypes

import numpy as np
import pytest
import torch

import int8_paths as P
from oracle import int8_oracle as I8
from gpu_util import DEV, bf16_bits_host, host

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8   # half a bf16 step, relative
E32 = 2.0 ** -24   # half an fp32 step, relative


@pytest.fixture(scope="module")
def L():
    import group_wise_minmax_amd as L
    assert torch.cuda.is_available()
    return L


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def weights(L, ns, k, seed):
    """Random codes of the whole range and scales of several magnitudes."""
    g = generator(seed)
    out = []
    for n in ns:
        q = torch.randint(-127, 128, (n, k), generator=g, device=DEV, dtype=torch.int8)
        s = (0.5 + torch.rand((n, 1), generator=g, device=DEV)) * 2.0 ** -torch.randint(4, 9, (n, 1), generator=g, device=DEV)
        out.append((L.QuantizedWeight(L.make_desc("int8", n, k), q.view(torch.uint8), s), q, s))
    return out


def tokens(m, k, seed):
    g = generator(seed)
    x = torch.randn((m, k), generator=g, device=DEV)
    x[:, torch.rand(k, generator=g, device=DEV) < 0.01] *= 20
    return x.to(torch.bfloat16)


def product(codes, scales, q, s):
    """fp32 values of the product before the rounding to bf16."""
    acc = torch.mm(codes.double(), q.double().t().contiguous())
    return acc.float() * scales[:, None] * s.t()


def equal(y, want):
    bad = torch.nonzero(y.view(torch.int16) != want.view(torch.int16))
    assert len(bad) == 0, f"{len(bad)} of {want.numel()} differ, first at {bad[0].tolist()}"


@pytest.mark.parametrize("case", P.PRODUCTS, ids=P.named)
def test_products(L, case):
    """Alone and together, from bf16 tokens and from codes, into rows of their own
    and scattered over wider ones."""
    _, m, k, ns = case
    made = weights(L, ns, k, m + k)
    x = tokens(m, k, m)
    codes, scales = L.lbq_quantize_tokens(x)
    rows = np.unique(np.linspace(0, m - 1, 5).astype(int))
    xq, xs = I8.quantize_rows(x[torch.from_numpy(rows).to(DEV)].float().cpu().numpy())
    assert np.array_equal(host(codes)[rows], xq) and np.array_equal(host(scales)[rows], xs)
    wants = [product(codes, scales, q, s).to(torch.bfloat16) for _, q, s in made]
    for (_, q, s), want in zip(made, wants):  # the reference itself, against the oracle
        some = I8.product_bf16(xq, xs, host(q)[:300], host(s).ravel()[:300])
        assert np.array_equal(bf16_bits_host(want)[rows, :300], some)
    for (qw, _, _), want in zip(made, wants):
        equal(L.lbq_linear_fwd_tokens(codes, scales, qw), want)
        equal(L.lbq_linear_fwd(x, qw), want)
    outs = [torch.full((m + 2, n + 3), -7.0, dtype=torch.bfloat16, device=DEV) for n in ns]
    L.lbq_linear_fwd_grouped(x, [qw for qw, _, _ in made], [o[1:m + 1, 1:n + 1] for o, n in zip(outs, ns)])
    for o, n, want in zip(outs, ns, wants):
        equal(o[1:m + 1, 1:n + 1].contiguous(), want)
        o[1:m + 1, 1:n + 1] = -7.0
        assert (o == -7.0).all()
    del outs
    total = sum(ns) + 5
    place = torch.randperm(total, generator=generator(1), device=DEV)[:sum(ns)].split(list(ns))
    wide = torch.full((m, total), -7.0, dtype=torch.bfloat16, device=DEV)
    for (qw, _, _), at in zip(made, place):
        qw.out_rows = at.to(torch.int32).contiguous()
    L.lbq_linear_fwd_grouped(x, [qw for qw, _, _ in made], [wide] * len(ns))
    for at, want in zip(place, wants):
        equal(wide[:, at], want)
    left = torch.ones(total, dtype=torch.bool, device=DEV)
    left[torch.cat(place)] = False
    assert (wide[:, left] == -7.0).all()


@pytest.mark.parametrize("r", [13, 64])
@pytest.mark.parametrize("case", [c for c in P.PRODUCTS if len(c[3]) == 1], ids=P.named)
def test_adapted_products(L, case, r):
    _, m, k, (n,) = case
    sigma = 0.75
    (qw, q, s), = weights(L, (n,), k, m + k)
    x = tokens(m, k, m)
    g = generator(r)
    A = (torch.randn((r, k), generator=g, device=DEV) * 0.05).to(torch.bfloat16)
    B = (torch.randn((n, r), generator=g, device=DEV) * 2.0).to(torch.bfloat16)
    y = L.lbq_lora_fwd(x, qw, A, B, sigma).double()
    base = product(*L.lbq_quantize_tokens(x), q, s).double()
    X, At, Bt = x.double(), A.double().t().contiguous(), B.double().t().contiguous()
    t = sigma * torch.mm(X, At)
    adapter = torch.mm(t, Bt)
    ref = base + adapter
    # T is summed in fp32 and rounded once to bf16, then r fp32 terms and the base, then bf16
    t_err = HALF * t.abs() + (k + 4) * E32 * sigma * torch.mm(X.abs(), At.abs())
    inner = torch.mm(t_err, Bt.abs()) + 2 * (r + 4) * E32 * (base.abs() + torch.mm(t.abs(), Bt.abs()))
    tol = inner + HALF * (ref.abs() + inner) + 1e-38
    assert bool(((y - ref).abs() <= tol).all()), float(((y - ref).abs() / tol).max())
    assert bool((adapter.abs() > 4 * tol).any())  # a missing adapter term would show


@pytest.mark.parametrize("case", [c for c in P.PRODUCTS if len(c[3]) == 1][::2] + [("decode", 3, 1024, (1001,))], ids=P.named)
def test_adapted_products_scattered(L, case):
    """The same bits into scattered channels, and into rows of a wider output."""
    _, m, k, (n,) = case
    (qw, _, _), = weights(L, (n,), k, m + k)
    x = tokens(m, k, m)
    g = generator(2)
    A = (torch.randn((24, k), generator=g, device=DEV) * 0.05).to(torch.bfloat16)
    B = torch.randn((n, 24), generator=g, device=DEV).to(torch.bfloat16)
    want = L.lbq_lora_fwd(x, qw, A, B, 0.5)
    out = torch.full((m, n + 9), -7.0, dtype=torch.bfloat16, device=DEV)
    L.lbq_lora_fwd(x, qw, A, B, 0.5, out=out[:, 3:3 + n])
    equal(out[:, 3:3 + n].contiguous(), want)
    out[:, 3:3 + n] = -7.0
    assert (out == -7.0).all()
    at = torch.randperm(n + 9, generator=g, device=DEV)[:n]
    qw.out_rows = at.to(torch.int32)
    L.lbq_lora_fwd(x, qw, A, B, 0.5, out=out)
    equal(out[:, at], want)
    out[:, at] = -7.0
    assert (out == -7.0).all()


def gradient(dys, made):
    """dX in 64 bits, and what its fp32 sums and its rounding may be off by."""
    whats = [(q.float() * s).to(torch.bfloat16).double() for _, q, s in made]
    ref = sum(torch.mm(d.double(), w) for d, w in zip(dys, whats))
    mag = sum(torch.mm(d.double().abs(), w.abs()) for d, w in zip(dys, whats))
    terms = sum(d.shape[1] for d in dys)
    return ref, mag, 2 * (terms + 2) * E32 * mag


@pytest.mark.parametrize("case", P.GRADIENTS, ids=P.named)
def test_gradients(L, case):
    """Against the formula, bit for bit again, and with an infinity in one token's
    gradients, which spoils that token alone (rows that end inside a step reach
    into the next token's)."""
    _, m, k, ns = case
    made = weights(L, ns, k, m + k)
    qws = [qw for qw, _, _ in made]
    g = generator(m)
    dys = [(torch.randn((m, n), generator=g, device=DEV) * 0.01).to(torch.bfloat16) for n in ns]
    dx = L.lbq_linear_bwd_dx_grouped(dys, qws)
    ref, _, inner = gradient(dys, made)
    tol = HALF * ref.abs() + (1 + HALF) * inner + 1e-38
    assert bool(((dx.double() - ref).abs() <= tol).all()), float(((dx.double() - ref).abs() / tol).max())
    equal(L.lbq_linear_bwd_dx_grouped(dys, qws), dx)
    if len(ns) == 1:
        equal(L.lbq_linear_bwd_dx(dys[0], qws[0]), dx)
    at = m // 2
    for d in dys:
        d[at, :8] = float("inf")
    bad = L.lbq_linear_bwd_dx_grouped(dys, qws)
    keep = torch.arange(m, device=DEV) != at
    equal(bad[keep], dx[keep])
    assert not bool(torch.isfinite(bad[at]).any())


@pytest.mark.parametrize("case", [c for c in P.GRADIENTS if c[0].endswith("ranges") and len(c[3]) == 1], ids=P.named)
def test_unsplit_gradients_are_one(L, case):
    """The C entry without a workspace, and the one whose workspace is a byte short:
    the same kernel and the same bits."""
    _, m, k, (n,) = case
    (qw, q, s), = made = weights(L, (n,), k, m + k)
    dy = (torch.randn((m, n), generator=generator(m), device=DEV) * 0.01).to(torch.bfloat16)
    need = L.lbq_linear_bwd_dx_grouped_workspace_bytes([qw], m)
    assert need > 0
    short = L.lbq_linear_bwd_dx(dy, qw, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    plain, t = torch.empty((m, k), dtype=torch.bfloat16, device=DEV), qw.qtensor()
    assert L.lib.lbq_linear_bwd_dx(ctypes.byref(qw.desc), ctypes.byref(t), dy.data_ptr(), m, plain.data_ptr(),
                                   torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    equal(short, plain)
    ref, _, inner = gradient([dy], made)
    tol = HALF * ref.abs() + (1 + HALF) * inner + 1e-38
    assert bool(((plain.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("r", [13, 64])
@pytest.mark.parametrize("case", P.ADAPTED_GRADIENTS, ids=P.named)
def test_adapted_gradients(L, case, r):
    """(dX, dA, dB) of an adapted layer."""
    _, m, k, (n,) = case
    sigma = 0.75
    (qw, q, s), = made = weights(L, (n,), k, m + k)
    x = tokens(m, k, m)
    g = generator(r)
    dy = (torch.randn((m, n), generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    a = (torch.randn((r, k), generator=g, device=DEV) * 0.5).to(torch.bfloat16)
    b = (torch.randn((n, r), generator=g, device=DEV) * 0.5).to(torch.bfloat16)
    dX, dA, dB = L.lbq_lora_bwd(x, dy, qw, a, b, sigma)
    X, dY, A, B = x.double(), dy.double(), a.double(), b.double()
    At = A.t().contiguous()
    G, T = sigma * torch.mm(dY, B), sigma * torch.mm(X, At)
    g_err = HALF * G.abs() + 2 * (n + 4) * E32 * sigma * torch.mm(dY.abs(), B.abs())
    t_err = HALF * T.abs() + 2 * (k + 4) * E32 * sigma * torch.mm(X.abs(), At.abs())
    ref, mag, _ = gradient([dy], made)
    ref = ref + torch.mm(G, A)
    inner = torch.mm(g_err, A.abs()) + 2 * (n + r + 4) * E32 * (mag + torch.mm(G.abs(), A.abs()))
    tol = inner + HALF * (ref.abs() + inner) + 1e-38
    assert bool(((dX.double() - ref).abs() <= tol).all()), float(((dX.double() - ref).abs() / tol).max())
    assert bool((torch.mm(G, A).abs() > 4 * tol).any())
    Gt, dYt = G.t().contiguous(), dY.t().contiguous()
    tol = torch.mm(g_err.t().contiguous(), X.abs()) + 2 * (m + 4) * E32 * torch.mm(Gt.abs(), X.abs()) + 1e-38
    tol = tol * (1 + HALF)  # G's own rounding meets its fp32 sum
    assert bool(((dA.double() - torch.mm(Gt, X)).abs() <= tol).all())
    tol = torch.mm(dYt.abs(), t_err) + 2 * (m + 4) * E32 * torch.mm(dYt.abs(), T.abs()) + 1e-38
    tol = tol * (1 + HALF)
    assert bool(((dB.double() - torch.mm(dYt, T)).abs() <= tol).all())


@pytest.mark.parametrize("m", [1, 40, 300, 1300])
def test_captured_training_calls(L, m):
    """A set's forward and input gradient and an adapted layer's backward, captured
    together and replayed with new inputs beside eager calls on the same weights;
    then the same calls on two streams at once."""
    k, ns, r = 1088, (512, 64, 192), 24
    made = weights(L, ns, k, 7)
    qws = [qw for qw, _, _ in made]
    g = generator(m)

    def draw(shape, scale):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)

    x, dys = draw((m, k), 1.0), [draw((m, n), 0.01) for n in ns]
    A, B = draw((r, k), 0.05), draw((ns[0], r), 0.05)

    def step():
        ys = L.lbq_linear_fwd_grouped(x, qws)
        return [*ys, L.lbq_linear_bwd_dx_grouped(dys, qws), *L.lbq_lora_bwd(x, dys[0], qws[0], A, B, 0.5)]

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(4):
        x.copy_(draw((m, k), 1.0))
        for d in dys:
            d.copy_(draw(d.shape, 0.01))
        for o in outs:
            o.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    want = step()
    torch.cuda.synchronize()
    streams, runs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for turn in range(6):
        with torch.cuda.stream(streams[turn % 2]):
            runs.append(step())
    torch.cuda.synchronize()
    for run in runs:
        assert all(torch.equal(a, b) for a, b in zip(run, want))
