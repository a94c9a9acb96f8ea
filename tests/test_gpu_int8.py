"""8-bit weights and tokens on the GPU, against the CPU oracle.

The codes, the scales and every product without an adapter are bit-exact: the
integer sums are exact and each fp32 step is one rounding, so no size, split or
kernel may change a bit.  Input gradients and adapter terms are held to bounds
derived from their roundings: a bf16 output is off by at most half a step
(2^-8 of its value), an fp32 sum of n terms by (n + 2) 2^-24 of the sum of
their magnitudes.
"""
import numpy as np
import pytest
import torch

import synth_inputs as SI
from oracle import int8_oracle as I8
from oracle import lbq_oracle as O
from gpu_util import DEV, bf16_bits_host, host, to_dev_bf16, to_dev_f32

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8   # half a bf16 step, relative
E32 = 2.0 ** -24   # half an fp32 step, relative


@pytest.fixture(scope="module")
def L():
    import group_wise_minmax_amd as L
    assert torch.cuda.is_available()
    return L


def tokens(seed, m, k):
    """bf16 bits of tokens with a few hot channels."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[:, rng.random(k) < 0.01] *= 20
    return O.bf16_bits(x)


def weight(L, seed, n, k):
    W = SI.gaussian_weights(seed, n, k, outlier_seed=seed + 1)
    qw = L.lbq_quantize(to_dev_f32(W), "int8")
    return qw, I8.quantize_rows(W)


def bits_equal(y, want):
    got = bf16_bits_host(y)
    assert got.shape == want.shape
    bad = np.flatnonzero((got != want).ravel())
    assert bad.size == 0, f"{bad.size} of {want.size} differ, first at {np.unravel_index(bad[0], want.shape)}"


# ------------------------------------------------------------------ quantizer

@pytest.mark.parametrize("n,k", [(1, 64), (3, 192), (37, 1280), (5, 2048), (4, 2112), (7, 4160), (3, 8192), (2, 8256),
                                 (3, 16384), (2, 16448), (1, 131072)])
def test_rows_bitexact(L, n, k):
    qw, (q, s) = weight(L, 7 * n + k, n, k)
    assert np.array_equal(host(qw.packed).view(np.int8), q)
    assert np.array_equal(host(qw.scales).ravel().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(bf16_bits_host(L.lbq_dequant(qw)), I8.dequant_bf16(q, s))
    x = tokens(n + k, n, k)
    codes, scales = L.lbq_quantize_tokens(to_dev_bf16(x))
    q, s = I8.tokens(x)
    assert np.array_equal(host(codes), q)
    assert np.array_equal(host(scales).view(np.uint32), s.view(np.uint32))


@pytest.mark.parametrize("k", [64, 4096, 20480])
def test_special_rows(L, k):
    """Rows of zeros, subnormal values and steps, exact ties, the largest finite
    values, and rows with an infinity or a NaN at either end."""
    rng = np.random.default_rng(k)
    x = rng.standard_normal((14, k)).astype(np.float32)
    x[0] = 0
    x[1] *= 2.0 ** -135
    x[2] = 0
    x[2, 3] = 2.0 ** -133
    x[3] = 0
    x[3, :6] = [127, 0.5, 1.5, 2.5, -0.5, -1.5]
    x[4, 5] = 3e38
    x[5, 0] = np.inf
    x[6, k - 1] = -np.inf
    x[7, 1] = np.nan
    x[8, k - 1] = np.nan
    x[9] = -2.0
    x[10, :] = np.arange(k) % 255 - 127
    x[11] = 0
    x[11, k - 1] = -1e-40
    bits = O.bf16_bits(x)
    bits[7, 1], bits[8, k - 1] = 0x7FC1, 0xFFC0
    q, s = I8.tokens(bits)
    codes, scales = L.lbq_quantize_tokens(to_dev_bf16(bits))
    assert np.array_equal(host(codes), q)
    assert np.array_equal(np.isnan(host(scales)), np.isnan(s)) and np.isnan(s).sum() == 4
    ok = ~np.isnan(s)
    assert np.array_equal(host(scales)[ok].view(np.uint32), s[ok].view(np.uint32))
    W = x.copy()
    W[1, 0], W[2, 3] = 2.0 ** -149, 2.0 ** -142  # fp32 subnormal steps
    W[12] = 0
    W[12, 3], W[12, 4] = 2.0 ** -142, -2.0 ** -142
    q, s = I8.quantize_rows(W)
    qw = L.lbq_quantize(to_dev_f32(W), "int8")
    assert np.array_equal(host(qw.packed).view(np.int8), q)
    ok = ~np.isnan(s)
    assert np.array_equal(host(qw.scales).ravel()[ok].view(np.uint32), s[ok].view(np.uint32))
    assert np.isnan(host(qw.scales).ravel()[~ok]).all()


def test_codes_near_ties(L):
    """Quotients within an fp32 rounding of k + 1/2, where a product with a
    reciprocal would round to the other side."""
    rng = np.random.default_rng(5)
    k = 2048
    rows = []
    for i in range(64):
        top = np.float32(rng.uniform(0.5, 2.0))
        s = np.float32(top / np.float32(127))
        h = rng.integers(0, 127, k).astype(np.float32) + np.float32(0.5)
        v = (h * s).astype(np.float32)
        v = np.where(rng.random(k) < 0.3, np.nextafter(v, np.float32(9)), np.where(rng.random(k) < 0.4, np.nextafter(v, np.float32(0)), v))
        v[0] = top
        rows.append(np.minimum(v, top))
    W = np.stack(rows).astype(np.float32)
    q, _ = I8.quantize_rows(W)
    assert np.array_equal(host(L.lbq_quantize(to_dev_f32(W), "int8").packed).view(np.int8), q)
    bits = O.bf16_bits(W)
    assert np.array_equal(host(L.lbq_quantize_tokens(to_dev_bf16(bits))[0]), I8.tokens(bits)[0])


def test_tokens_with_row_stride(L):
    x = tokens(3, 9, 512)
    wide = torch.full((9, 648), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 64:576] = to_dev_bf16(x)
    codes, scales = L.lbq_quantize_tokens(wide[:, 64:576])
    q, s = I8.tokens(x)
    assert np.array_equal(host(codes), q) and np.array_equal(host(scales), s)
    with pytest.raises(ValueError):
        L.lbq_quantize_tokens(wide.t())
    with pytest.raises(L.LbqError):
        L.lbq_quantize_tokens(wide[:, 1:513])
    with pytest.raises(L.LbqError):
        L.lbq_quantize_tokens(wide[:, :100])


# ------------------------------------------------------------------ product

MS = [1, 2, 3, 4, 5, 8, 15, 16, 17, 31, 33, 48, 64, 65, 100, 128, 129, 200, 256, 257, 300, 520]


@pytest.mark.parametrize("n,k", [(64, 64), (1, 128), (17, 192), (300, 1024), (1001, 4160), (260, 8192), (4097, 320)])
def test_forward_bitexact(L, n, k):
    qw, (wq, ws) = weight(L, n + k, n, k)
    for m in MS:
        print("m", m, flush=True)
        x = tokens(m, m, k)
        want = I8.product_bf16(*I8.tokens(x), wq, ws)
        X = to_dev_bf16(x)
        bits_equal(L.lbq_linear_fwd(X, qw), want)
        codes, scales = L.lbq_quantize_tokens(X)
        bits_equal(L.lbq_linear_fwd_tokens(codes, scales, qw), want)


@pytest.mark.parametrize("m,n,k", [(5, 8200, 1024), (12, 14336, 1024), (13, 5001, 2048), (16, 28672, 512), (24, 14336, 1088),
                                   (30, 4100, 4096), (48, 9001, 1024), (64, 14336, 512), (90, 4096, 2048)])
def test_forward_of_few_tokens_through_many_channels(L, m, n, k):
    """Every tile shape of the short products: 16 to 64 channels by 16 to 64 tokens."""
    qw, (wq, ws) = weight(L, 8, n, k)
    x = tokens(m, m, k)
    bits_equal(L.lbq_linear_fwd(to_dev_bf16(x), qw), I8.product_bf16(*I8.tokens(x), wq, ws))


@pytest.mark.parametrize("m", [0, 1, 2, 5, 64, 130])
def test_forward_leaves_the_rest_alone(L, m):
    """A strided output, and guard rows before and after it; m = 0 writes nothing."""
    n, k = 100, 448
    qw, (wq, ws) = weight(L, 5, n, k)
    x = tokens(1, m, k)
    buf = torch.full((m + 6, 160), -7.0, dtype=torch.bfloat16, device=DEV)
    L.lbq_linear_fwd(to_dev_bf16(x), qw, out=buf[3:3 + m, :n])
    got = buf.float().cpu().numpy()
    if m:
        bits_equal(buf[3:3 + m, :n], I8.product_bf16(*I8.tokens(x), wq, ws))
    got[3:3 + m, :n] = -7.0
    assert (got == -7.0).all()


@pytest.mark.parametrize("m", [1, 6, 50, 129, 600])
@pytest.mark.parametrize("first,ld", [(1, 311), (3, 312), (2, 315)])
def test_outputs_at_any_address(L, m, first, ld):
    """Rows that begin at any multiple of two bytes, an odd number of values apart."""
    n, k = 301, 704
    qw, (wq, ws) = weight(L, 6, n, k)
    x = tokens(2, m, k)
    buf = torch.full((m, ld), -7.0, dtype=torch.bfloat16, device=DEV)
    L.lbq_linear_fwd(to_dev_bf16(x), qw, out=buf[:, first:first + n])
    bits_equal(buf[:, first:first + n], I8.product_bf16(*I8.tokens(x), wq, ws))
    assert (buf[:, :first] == -7.0).all() and (buf[:, first + n:] == -7.0).all()


@pytest.mark.parametrize("m", [1, 2, 4, 7, 70, 300])
def test_longest_rows_of_largest_codes(L, m):
    """k = 2^17 codes of 127: sums just below 2^31, of either sign."""
    k, n = 1 << 17, 40
    W = np.ones((n, k), dtype=np.float32)
    W[1::2] = -1
    qw = L.lbq_quantize(to_dev_f32(W), "int8")
    x = np.ones((m, k), dtype=np.float32)
    x[m // 2] = -1
    y = L.lbq_linear_fwd(to_dev_bf16(O.bf16_bits(x)), qw)
    q, s = I8.quantize_rows(W)
    bits_equal(y, I8.product_bf16(*I8.quantize_rows(x), q, s))
    assert abs(float(y[0, 0])) == float(k)


@pytest.mark.parametrize("m", [1, 3, 16, 70])
def test_nonfinite_tokens_spoil_their_rows_only(L, m):
    n, k = 80, 320
    qw, (wq, ws) = weight(L, 9, n, k)
    x = tokens(2, m, k)
    x[m // 2, 17] = 0x7F80
    y = bf16_bits_host(L.lbq_linear_fwd(to_dev_bf16(x), qw))
    want = I8.product_bf16(*I8.tokens(np.delete(x, m // 2, 0)), wq, ws)
    assert np.isnan(O.bf16_to_f64(y[m // 2])).all()
    assert np.array_equal(np.delete(y, m // 2, 0), want)


@pytest.mark.parametrize("m", [1, 2, 4, 6, 40, 64, 100, 300])
def test_grouped_equals_single(L, m):
    k = 1152
    made = [weight(L, 20 + i, n, k) for i, n in enumerate((256, 40, 513))]
    other = L.lbq_quantize(to_dev_f32(SI.gaussian_weights(3, 128, k)), "minmax")
    x = tokens(4, m, k)
    X = to_dev_bf16(x)
    t = I8.tokens(x)
    for y, (_, (q, s)) in zip(L.lbq_linear_fwd_grouped(X, [w for w, _ in made]), made):
        bits_equal(y, I8.product_bf16(*t, q, s))
    # beside a weight of another format, in any place
    ys = L.lbq_linear_fwd_grouped(X, [made[0][0], other, made[2][0]])
    bits_equal(ys[0], I8.product_bf16(*t, *made[0][1]))
    bits_equal(ys[2], I8.product_bf16(*t, *made[2][1]))
    assert torch.equal(ys[1], L.lbq_linear_fwd(X, other))
    # the same weight twice
    a, b = L.lbq_linear_fwd_grouped(X, [made[1][0], made[1][0]])
    assert torch.equal(a, b)


@pytest.mark.parametrize("m", [1, 3, 4, 9, 64, 130])
def test_channel_scatter(L, m):
    """INT8 rows and INT4 rows of one layer scatter into one output."""
    n, k = 192, 512
    perm = np.random.default_rng(0).permutation(n)
    a, b = np.sort(perm[:70]), np.sort(perm[70:])
    W = SI.gaussian_weights(8, n, k)
    qa = L.lbq_quantize(to_dev_f32(W[a]), "int8")
    qb = L.lbq_quantize(to_dev_f32(W[b]), "minmax")
    x = tokens(6, m, k)
    X = to_dev_bf16(x)
    plain_b = L.lbq_linear_fwd(X, qb)
    qa.out_rows = torch.from_numpy(a.astype(np.int32)).to(DEV)
    qb.out_rows = torch.from_numpy(b.astype(np.int32)).to(DEV)
    out = torch.full((m, n + 3), 5.0, dtype=torch.bfloat16, device=DEV)
    L.lbq_linear_fwd_grouped(X, [qa, qb], outs=[out, out])
    bits_equal(out[:, torch.from_numpy(a).to(DEV)], I8.product_bf16(*I8.tokens(x), *I8.quantize_rows(W[a])))
    assert torch.equal(out[:, torch.from_numpy(b).to(DEV)], plain_b)
    assert (out[:, n:] == 5.0).all()


def test_workspace_contents_do_not_matter(L):
    n, k = 1024, 4096
    qw, (wq, ws) = weight(L, 30, n, k)
    for m in (3, 20, 64, 130, 300):
        x = tokens(m, m, k)
        w = torch.full((L.lbq_linear_workspace_bytes(qw, m),), 255, dtype=torch.uint8, device=DEV)
        want = I8.product_bf16(*I8.tokens(x), wq, ws)
        for _ in range(2):
            bits_equal(L.lbq_linear_fwd(to_dev_bf16(x), qw, workspace=w), want)


@pytest.mark.parametrize("m", [1, 4, 33, 64, 100])
def test_noalloc_forward(L, m):
    qw, (wq, ws) = weight(L, 31, 300, 2048)
    x = tokens(m, m, 2048)
    bits_equal(L.lbq_linear_fwd_noalloc(to_dev_bf16(x), qw), I8.product_bf16(*I8.tokens(x), wq, ws))


def test_noalloc_forward_refuses_what_does_not_fit(L):
    qw, _ = weight(L, 32, 64, 8192)
    x = torch.zeros((2100, 8192), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(L.LbqError) as e:
        L.lbq_linear_fwd_noalloc(x, qw)
    assert e.value.name == "LBQ_E_WORKSPACE"


@pytest.mark.parametrize("m,n,k", [(64, 11008, 65536), (250, 8192, 8192)])
def test_noalloc_forward_without_room_for_partial_sums(L, m, n, k):
    """The library's array holds the codes but not the partial sums: the same bits."""
    g = torch.Generator(device=DEV).manual_seed(m)
    q = torch.randint(-127, 128, (n, k), generator=g, device=DEV, dtype=torch.int8)
    qw = L.QuantizedWeight(L.make_desc("int8", n, k), q.view(torch.uint8), torch.rand((n, 1), generator=g, device=DEV))
    X = torch.randn((m, k), generator=g, device=DEV).to(torch.bfloat16)
    assert m * (k + 4) < 2 ** 24 < L.lbq_linear_workspace_bytes(qw, m)
    y = L.lbq_linear_fwd(X, qw)
    assert torch.equal(L.lbq_linear_fwd_noalloc(X, qw), y) and y.float().abs().max() > 0


def test_streams_at_once(L):
    """Two weights on two streams in turn, each with its own workspace."""
    k = 2048
    made = [weight(L, 40 + i, n, k) for i, n in enumerate((512, 300))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for m in (1, 3, 16, 200):
        x = tokens(m, m, k)
        X = to_dev_bf16(x)
        torch.cuda.synchronize()
        outs = []
        for i in range(6):
            with torch.cuda.stream(streams[i % 2]):
                outs.append(L.lbq_linear_fwd(X, made[i % 2][0]))
        torch.cuda.synchronize()
        for i, y in enumerate(outs):
            bits_equal(y, I8.product_bf16(*I8.tokens(x), *made[i % 2][1]))


def test_graph_replays(L):
    """Captured forwards of three batch sizes that share one workspace, replayed
    with new inputs and eager work between the replays."""
    k = 1024
    qw, (wq, ws) = weight(L, 50, 700, k)
    ms = (1, 3, 40, 150)
    work = torch.empty(max(L.lbq_linear_workspace_bytes(qw, m) for m in ms) + 16, dtype=torch.uint8, device=DEV)
    xs = [torch.zeros((m, k), dtype=torch.bfloat16, device=DEV) for m in ms]
    ys = [torch.zeros((m, 700), dtype=torch.bfloat16, device=DEV) for m in ms]
    for x, y in zip(xs, ys):
        L.lbq_linear_fwd(x, qw, out=y, workspace=work)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for x, y in zip(xs, ys):
            L.lbq_linear_fwd(x, qw, out=y, workspace=work)
    for turn in range(4):
        host_x = [tokens(100 * turn + m, m, k) for m in ms]
        for x, h in zip(xs, host_x):
            x.copy_(to_dev_bf16(h))
        g.replay()
        eager = [L.lbq_linear_fwd(x, qw) for x in xs]
        torch.cuda.synchronize()
        for y, e, h in zip(ys, eager, host_x):
            want = I8.product_bf16(*I8.tokens(h), wq, ws)
            bits_equal(y, want)
            bits_equal(e, want)


def test_serialization(L):
    qw, (wq, ws) = weight(L, 60, 65, 256)
    back = L.QuantizedWeight.from_bytes(qw.to_bytes(), DEV)
    assert torch.equal(back.packed, qw.packed) and torch.equal(back.scales, qw.scales)
    x = tokens(1, 3, 256)
    bits_equal(L.lbq_linear_fwd(to_dev_bf16(x), back), I8.product_bf16(*I8.tokens(x), wq, ws))


def test_refused_tensors(L):
    qw, _ = weight(L, 61, 64, 256)
    X = torch.zeros((3, 256), dtype=torch.bfloat16, device=DEV)
    codes, scales = L.lbq_quantize_tokens(X)
    with pytest.raises(ValueError):
        L.lbq_linear_fwd(X.cpu(), qw)
    with pytest.raises(ValueError):
        L.lbq_linear_fwd(X.float(), qw)
    with pytest.raises(ValueError):
        L.lbq_linear_fwd_tokens(codes, scales[:2], qw)
    with pytest.raises(ValueError):
        L.lbq_linear_fwd_tokens(codes, scales.double(), qw)
    with pytest.raises(ValueError):
        L.lbq_linear_fwd_tokens(codes, scales, qw, out=torch.empty((3, 63), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        L.lbq_linear_fwd_tokens(codes[:, :128], scales, qw)
    with pytest.raises(L.LbqError):
        L.lbq_linear_fwd_tokens(codes, scales, L.lbq_quantize(torch.zeros((64, 256), device=DEV), "minmax"))
    short = L.QuantizedWeight(qw.desc, qw.packed[:32], qw.scales)
    with pytest.raises(ValueError):
        L.lbq_linear_fwd(X, short)
    with pytest.raises(ValueError):
        L.lbq_linear_fwd(X, L.QuantizedWeight(qw.desc, qw.packed, qw.scales[:32]))
    with pytest.raises(ValueError):
        L.lbq_quantize(torch.zeros((64, 256), device=DEV), "int8", out=L.lbq_quantize(torch.zeros((64, 256), device=DEV)))


def test_refused_outputs(L):
    qw, _ = weight(L, 62, 64, 256)
    X = torch.zeros((3, 256), dtype=torch.bfloat16, device=DEV)
    A, B = X[:2].contiguous(), torch.zeros((64, 2), dtype=torch.bfloat16, device=DEV)
    wide = torch.empty((3, 100), dtype=torch.bfloat16, device=DEV)
    for out in (wide[:, :63], wide[:2, :64], wide[:, :64].float(), wide.t()[:64].t()[:, ::2]):
        for call in (lambda: L.lbq_linear_fwd(X, qw, out=out), lambda: L.lbq_linear_fwd_noalloc(X, qw, out=out),
                     lambda: L.lbq_linear_fwd_grouped(X, [qw], [out]), lambda: L.lbq_lora_fwd(X, qw, A, B, 1.0, out=out)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        L.lbq_lora_fwd(X[:, :128].contiguous(), qw, A, B, 1.0)


# ------------------------------------------------------------------ input gradient

def grad_bound(dys, whats):
    """(reference, bound) of the input gradient in fp64."""
    ref = sum(d @ w for d, w in zip(dys, whats))
    mag = sum(np.abs(d) @ np.abs(w) for d, w in zip(dys, whats))
    terms = sum(d.shape[1] for d in dys)
    return ref, HALF * np.abs(ref) + 2 * (terms + 2) * E32 * mag + 1e-38


@pytest.mark.parametrize("n,k", [(8, 64), (64, 192), (200, 1024), (1000, 4160), (4096, 320)])
def test_bwd_dx(L, n, k):
    qw, (q, s) = weight(L, n + 3 * k, n, k)
    what = O.bf16_to_f64(I8.dequant_bf16(q, s))
    for m in (1, 2, 5, 16, 40, 64, 129, 300):
        print("m", m, flush=True)
        dy = SI.bf16_normal(m + n, (m, n), 0.01)
        dx = O.bf16_to_f64(bf16_bits_host(L.lbq_linear_bwd_dx(to_dev_bf16(dy), qw)))
        ref, tol = grad_bound([O.bf16_to_f64(dy)], [what])
        assert (np.abs(dx - ref) <= tol).all(), np.max(np.abs(dx - ref) / tol)


@pytest.mark.parametrize("n,k,m", [(4096, 4096, 40), (14336, 1024, 16), (6000, 256, 3), (4104, 64, 100), (1000, 8192, 520),
                                   (512, 4096, 1100)])
def test_bwd_dx_workspace_and_without(L, n, k, m):
    """The reduction split over workgroups (workspace, whatever it holds), and
    unsplit through the entry without one or with one byte less."""
    import ctypes
    qw, (q, s) = weight(L, 3 * n + k, n, k)
    dy = SI.bf16_normal(m + n, (m, n), 0.01)
    rows = np.unique(np.linspace(0, m - 1, 16).astype(int))
    ref, tol = grad_bound([O.bf16_to_f64(dy)[rows]], [O.bf16_to_f64(I8.dequant_bf16(q, s))])
    need = L.lbq_linear_bwd_dx_grouped_workspace_bytes([qw], m)
    dY = to_dev_bf16(dy)
    outs = []
    for size in {need, max(need - 1, 0)}:
        w = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        for _ in range(2):
            outs.append(L.lbq_linear_bwd_dx(dY, qw, workspace=w))
            dx = O.bf16_to_f64(bf16_bits_host(outs[-1]))[rows]
            assert (np.abs(dx - ref) <= tol).all()
        assert torch.equal(outs[-1], outs[-2])
    plain = torch.empty((m, k), dtype=torch.bfloat16, device=DEV)
    t = qw.qtensor()
    assert L.lib.lbq_linear_bwd_dx(ctypes.byref(qw.desc), ctypes.byref(t), dY.data_ptr(), m, plain.data_ptr(),
                                   torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    dx = O.bf16_to_f64(bf16_bits_host(plain))[rows]
    assert (np.abs(dx - ref) <= tol).all()
    if need:
        assert torch.equal(plain, outs[-1]) or torch.equal(plain, outs[1])
    else:
        assert torch.equal(plain, outs[0])


@pytest.mark.parametrize("n,k,m", [(72, 128, 5), (72, 128, 200), (40, 4096, 64), (200, 2048, 2100), (72, 4096, 1100), (200, 8192, 1000)])
def test_bwd_dx_next_token_stays_out(L, n, k, m):
    """n % 32 != 0: a token's last slice of rows reads into the next token's
    gradients; an infinity there spoils that token alone, on every path."""
    qw, (q, s) = weight(L, 12, n, k)
    dy = SI.bf16_normal(m, (m, n), 0.01)
    w = torch.empty(L.lbq_linear_bwd_dx_grouped_workspace_bytes([qw], m), dtype=torch.uint8, device=DEV)
    for ws in (w, w[:0]):
        dy[3, :8] = SI.bf16_normal(1, (8,), 0.01)
        clean = bf16_bits_host(L.lbq_linear_bwd_dx(to_dev_bf16(dy), qw, workspace=ws))
        dy[3, :8] = 0x7F80
        dx = bf16_bits_host(L.lbq_linear_bwd_dx(to_dev_bf16(dy), qw, workspace=ws))
        assert np.array_equal(np.delete(dx, 3, 0), np.delete(clean, 3, 0))
        assert not np.isfinite(O.bf16_to_f64(dx[3])).any()


@pytest.mark.parametrize("m", [1, 40, 300])
def test_bwd_dx_grouped(L, m):
    k = 576
    made = [weight(L, 70 + i, n, k) for i, n in enumerate((128, 40, 264))]
    dys = [SI.bf16_normal(80 + i, (m, w.n), 0.01) for i, (w, _) in enumerate(made)]
    dx = L.lbq_linear_bwd_dx_grouped([to_dev_bf16(d) for d in dys], [w for w, _ in made])
    ref, tol = grad_bound([O.bf16_to_f64(d) for d in dys], [O.bf16_to_f64(I8.dequant_bf16(*t)) for _, t in made])
    assert (np.abs(O.bf16_to_f64(bf16_bits_host(dx)) - ref) <= tol).all()
    with pytest.raises(L.LbqError) as e:
        other = L.lbq_quantize(torch.zeros((64, k), device=DEV), "minmax", 4, 64)
        L.lbq_linear_bwd_dx_grouped([torch.zeros((m, 128), dtype=torch.bfloat16, device=DEV),
                                     torch.zeros((m, 64), dtype=torch.bfloat16, device=DEV)], [made[0][0], other])
    assert e.value.name == "LBQ_E_UNSUPPORTED"


def test_bwd_dx_is_the_adjoint_of_differences(L):
    """<dY, deq(W) v> = <dX, v> for a difference v of two inputs: dX is the
    gradient of the product before the tokens are rounded."""
    n, k, m = 64, 128, 3
    qw, (q, s) = weight(L, 77, n, k)
    what = O.bf16_to_f64(I8.dequant_bf16(q, s))
    dy = O.bf16_to_f64(SI.bf16_normal(1, (m, n)))
    dx = O.bf16_to_f64(bf16_bits_host(L.lbq_linear_bwd_dx(to_dev_bf16(O.bf16_bits(dy.astype(np.float32))), qw)))
    rng = np.random.default_rng(0)
    x, h = rng.standard_normal((m, k)), 1e-3

    def loss(v):
        return float(np.sum(dy * (v @ what.T)))

    for _ in range(8):
        v = rng.standard_normal((m, k))
        diff = (loss(x + h * v) - loss(x - h * v)) / (2 * h)
        tol = np.sum((HALF + 2 * (n + 2) * E32) * (np.abs(dy) @ np.abs(what)) * np.abs(v)) + 1e-9 * np.abs(diff)
        assert abs(np.sum(dx * v) - diff) <= tol


# ------------------------------------------------------------------ adapters

def lora_parts(seed, n, k, r):
    return SI.bf16_normal(seed, (r, k), 0.05), SI.bf16_normal(seed + 1, (n, r), 0.05)


@pytest.mark.parametrize("n,k", [(64, 128), (330, 1088)])
@pytest.mark.parametrize("r", [1, 8, 13, 33, 64])
def test_lora_forward(L, n, k, r):
    qw, (q, s) = weight(L, 90 + r, n, k)
    a, b = lora_parts(r, n, k, r)
    A, B = O.bf16_to_f64(a), O.bf16_to_f64(b)
    sigma = 1.5
    for m in (1, 2, 4, 5, 16, 33, 64, 65, 130, 300):
        print("m", m, flush=True)
        x = tokens(m, m, k)
        y = O.bf16_to_f64(bf16_bits_host(L.lbq_lora_fwd(to_dev_bf16(x), qw, to_dev_bf16(a), to_dev_bf16(b), sigma)))
        X = O.bf16_to_f64(x)
        t = sigma * X @ A.T
        base = I8.product(*I8.tokens(x), q, s).astype(np.float64)
        ref = base + t @ B.T
        # T is rounded once to bf16 (and summed in fp32), then r fp32 terms and the base, then bf16
        t_err = HALF * np.abs(t) + (k + 4) * E32 * sigma * np.abs(X) @ np.abs(A).T
        inner = t_err @ np.abs(B).T + 2 * (r + 4) * E32 * (np.abs(base) + np.abs(t) @ np.abs(B).T)
        tol = inner + HALF * (np.abs(ref) + inner) + 1e-38
        assert (np.abs(y - ref) <= tol).all(), np.max(np.abs(y - ref) / tol)


@pytest.mark.parametrize("m", [1, 6, 300])
def test_lora_forward_replayed_and_on_two_streams(L, m):
    """A captured adapted layer replayed with new tokens beside eager calls, and two
    layers on two streams at once: the bits of the calls alone."""
    n, k, r = 520, 1088, 24
    qws = [weight(L, 96 + i, n, k)[0] for i in range(2)]
    parts = [tuple(map(to_dev_bf16, lora_parts(20 + i, n, k, r))) for i in range(2)]
    x = to_dev_bf16(tokens(1, m, k))
    y = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        L.lbq_lora_fwd(x, qws[0], *parts[0], 0.5, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lbq_lora_fwd(x, qws[0], *parts[0], 0.5, out=y)
    for turn in range(4):
        x.copy_(to_dev_bf16(tokens(30 + turn, m, k)))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, L.lbq_lora_fwd(x, qws[0], *parts[0], 0.5))
    want = [L.lbq_lora_fwd(x, q, *p, 0.5) for q, p in zip(qws, parts)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for turn in range(8):
        with torch.cuda.stream(streams[turn % 2]):
            got.append(L.lbq_lora_fwd(x, qws[turn % 2], *parts[turn % 2], 0.5))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[i % 2]) for i, v in enumerate(got))


def test_lora_backward(L):
    n, k, r, m, sigma = 128, 320, 16, 45, 2.0
    qw, (q, s) = weight(L, 95, n, k)
    a, b = lora_parts(5, n, k, r)
    x, dy = tokens(1, m, k), SI.bf16_normal(2, (m, n), 0.1)
    dX, dA, dB = L.lbq_lora_bwd(to_dev_bf16(x), to_dev_bf16(dy), qw, to_dev_bf16(a), to_dev_bf16(b), sigma)
    W = O.bf16_to_f64(I8.dequant_bf16(q, s))
    X, dY, A, B = (O.bf16_to_f64(v) for v in (x, dy, a, b))
    G, T = sigma * dY @ B, sigma * X @ A.T
    g_err = (HALF + (n + 4) * E32) * np.abs(G) + (n + 4) * E32 * sigma * np.abs(dY) @ np.abs(B)
    t_err = (HALF + (k + 4) * E32) * np.abs(T) + (k + 4) * E32 * sigma * np.abs(X) @ np.abs(A).T
    ref = dY @ W + G @ A
    inner = g_err @ np.abs(A) + 2 * (n + r + 4) * E32 * (np.abs(dY) @ np.abs(W) + np.abs(G) @ np.abs(A))
    tol = inner + HALF * (np.abs(ref) + inner) + 1e-38
    assert (np.abs(O.bf16_to_f64(bf16_bits_host(dX)) - ref) <= tol).all()
    tolA = g_err.T @ np.abs(X) + 2 * (m + 4) * E32 * np.abs(G).T @ np.abs(X) + 1e-38
    assert (np.abs(host(dA) - G.T @ X) <= tolA).all()
    tolB = np.abs(dY).T @ t_err + 2 * (m + 4) * E32 * np.abs(dY).T @ np.abs(T) + 1e-38
    assert (np.abs(host(dB) - dY.T @ T) <= tolB).all()


@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (3, 2048, 128), (17, 64, 4096), (40, 1024, 1024), (70, 192, 192), (700, 320, 320)])
@pytest.mark.parametrize("r", [1, 13, 32, 64])
def test_lora_backward_input_gradient(L, m, n, k, r):
    """The input gradient with its adapter term, where the reduction is split over
    waves, workgroups and ranges, and ranks that end inside a step of 32."""
    sigma = 0.5
    qw, (q, s) = weight(L, 195, n, k)
    a, b = lora_parts(r, n, k, r)
    x, dy = tokens(1, m, k), SI.bf16_normal(2, (m, n), 0.1)
    dX, _, _ = L.lbq_lora_bwd(to_dev_bf16(x), to_dev_bf16(dy), qw, to_dev_bf16(a), to_dev_bf16(b), sigma)
    W = O.bf16_to_f64(I8.dequant_bf16(q, s))
    dY, A, B = (O.bf16_to_f64(v) for v in (dy, a, b))
    G = sigma * dY @ B
    g_err = (HALF + (n + 4) * E32) * np.abs(G) + (n + 4) * E32 * sigma * np.abs(dY) @ np.abs(B)
    ref = dY @ W + G @ A
    inner = g_err @ np.abs(A) + 2 * (n + r + 4) * E32 * (np.abs(dY) @ np.abs(W) + np.abs(G) @ np.abs(A))
    tol = inner + HALF * (np.abs(ref) + inner) + 1e-38
    assert (np.abs(O.bf16_to_f64(bf16_bits_host(dX)) - ref) <= tol).all()


def test_training_step(L):
    """An adapted 8-bit layer trained for a few steps as a program does it:
    forward, backward, clipping, optimizer.  Each step's norm is that of its
    gradients, and what the optimizer sees is at most max_norm."""
    n, k, m = 192, 256, 50
    qws = [weight(L, 97 + i, n if i == 0 else k, k if i == 0 else n)[0] for i in range(2)]
    gen = torch.Generator(device=DEV).manual_seed(3)
    layers = [L.LbqLoraLinear(q, r=8, lora_alpha=16, generator=gen) for q in qws]
    params = [p for layer in layers for p in (layer.A, layer.B)]
    opt = torch.optim.SGD(params, lr=1e-3)
    x = torch.randn((2, m // 2, k), device=DEV, generator=gen).to(torch.bfloat16).requires_grad_(True)
    fresh = layers[0](x)
    assert torch.equal(fresh, L.lbq_linear_fwd(x.detach().reshape(m, k), qws[0]).reshape(2, m // 2, n))
    for step in range(4):
        opt.zero_grad(set_to_none=step % 2 == 0)
        x.grad = None
        y = layers[1](layers[0](x))
        (y.float() ** 2).mean().backward()
        grads = [p.grad for p in params]
        before = [g.double().cpu().numpy().copy() for g in grads]
        norm = L.lbq_clip_grad_norm_(grads, 1e-3)
        want = I8.grad_norm(before)
        assert abs(float(norm) - want) <= 2 ** -23 * want
        c = I8.clip_factor(want, 1e-3)
        for g, b in zip(grads, before):
            assert np.allclose(g.double().cpu().numpy(), b * c, rtol=2 ** -21, atol=0)
        assert x.grad is not None and torch.isfinite(x.grad).all() and x.grad.abs().sum() > 0
        opt.step()
    assert all(torch.isfinite(p).all() for p in params) and params[1].abs().sum() > 0


@pytest.mark.parametrize("m", [1, 40])
def test_backward_captured_beside_an_eager_graph(L, m):
    """The backward entry captured while an eager graph of the same leaves is
    alive, replayed between eager steps."""
    n, k = 128, 256
    qw, (q, s) = weight(L, 99, n, k)
    layer = L.LbqLoraLinear(qw, r=8)
    x = torch.randn((m, k), device=DEV).to(torch.bfloat16).requires_grad_(True)
    alive = layer(x)
    dy = torch.randn((m, n), device=DEV).to(torch.bfloat16)
    out = torch.empty((m, k), dtype=torch.bfloat16, device=DEV)
    L.lbq_linear_bwd_dx(dy, qw, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lbq_linear_bwd_dx(dy, qw, out=out)
    for _ in range(3):
        dy.copy_(torch.randn((m, n), device=DEV))
        g.replay()
        want = L.lbq_linear_bwd_dx(dy, qw)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    alive.float().sum().backward()
    assert torch.isfinite(x.grad).all()


# ---------------------------------------------------------------- the largest

def test_more_rows_than_a_grid_has(L):
    """Rows of 64 beyond 2^32 threads of a workgroup a row: tokens, weights and
    the dequantized weight repeat a small block's."""
    block, times = 64, 2 ** 18 + 1
    x = tokens(71, block, 64)
    q, s = I8.tokens(x)
    codes, scales = L.lbq_quantize_tokens(to_dev_bf16(x).repeat(times, 1))
    q, s = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    assert (codes.view(times, block, 64) == q).all() and (scales.view(times, block) == s).all()
    del codes, scales
    W = SI.gaussian_weights(72, block, 64, outlier_seed=73)
    q, s = I8.quantize_rows(W)
    qw = L.lbq_quantize(to_dev_f32(W).repeat(times, 1), "int8")
    dq = torch.from_numpy(I8.dequant_bf16(q, s).view(np.int16)).to(DEV)
    q, s = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    assert (qw.packed.view(torch.int8).view(times, block, 64) == q).all() and (qw.scales.view(times, block) == s).all()
    assert (L.lbq_dequant(qw).view(torch.int16).view(times, block, 64) == dq).all()


def test_more_tokens_than_a_grid_dimension_has_tiles(L):
    """4.2 M tokens of 64 through 8 channels: more than 65535 tiles of 64 tokens."""
    block, times, n = 64, 2 ** 16 + 3, 8
    x = tokens(74, block, 64)
    qw, (q, s) = weight(L, 75, n, 64)
    y = L.lbq_linear_fwd(to_dev_bf16(x).repeat(times, 1), qw)
    xq, xs = I8.tokens(x)
    want = torch.from_numpy(I8.product_bf16(xq, xs, q, s).view(np.int16)).to(DEV)
    assert (y.view(torch.int16).view(times, block, n) == want).all()


def test_gradient_beyond_31_bits_of_bytes(L):
    """4.26 GB of output gradients: the last tokens against the formula in 64 bits."""
    m, n, k = 65000, 32768, 64
    g = torch.Generator(device=DEV).manual_seed(76)
    dY = torch.randn(m, n, generator=g, device=DEV, dtype=torch.bfloat16)
    qw, (q, s) = weight(L, 77, n, k)
    dx = L.lbq_linear_bwd_dx(dY, qw)
    w = L.lbq_dequant(qw).double()
    for rows in (slice(0, 40), slice(32700, 32800), slice(m - 70, m)):
        d = dY[rows].double()
        want, size = d @ w, d.abs() @ w.abs()
        err = (dx[rows].double() - want).abs()
        assert (err <= HALF * want.abs() + (1 + HALF) * (n + 2) * E32 * size).all()
