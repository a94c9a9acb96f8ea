"""Measured cases of the 8-bit linear layer, its input gradient and the global
gradient norm with clipping.

Each case names one operator (``op``) and its sizes:

* ``linear`` -- Y = deq(X_q) . deq(W_q)^T: every token (row of X) is quantized to
  8-bit integers with one scale, every output channel (row of W) holds 8-bit
  integers with one scale, and the products are summed in integers.  ``ns``
  lists the weights that read the same X.  With ``codes`` the tokens are
  quantized once by a call of their own and each weight multiplies the codes;
  with ``rank`` a LoRA branch of that rank is added.
* ``grad`` -- the input gradient through the frozen 8-bit weights,
  dX = sum_i dY_i . deq(W_i).
* ``clip`` -- the 2-norm (or largest magnitude) over all of a step's gradient
  tensors, and the gradients scaled so that it is at most ``max_norm``.

``own`` false computes the plain form in elementary torch operations; ``own``
true makes the calls of ``group_wise_minmax_amd``.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one token through the q or o projection of an 8B layer: the smallest call of decoding, bound by latency
        {"name": "decode_1_q", "op": "linear", "m": 1, "k": 4096, "ns": "4096"},
        # three sequences decoded together through the down projection of a 70B layer: the longest rows
        {"name": "decode_3_down70", "op": "linear", "m": 3, "k": 28672, "ns": "8192"},
        # a decoding batch of 24 through gate of an 8B layer
        {"name": "decode_24_gate", "op": "linear", "m": 24, "k": 4096, "ns": "14336"},
        # a prompt of 333 tokens through q, k and v of a 70B layer, tokens quantized once for the three
        {"name": "prompt_333_qkv70", "op": "linear", "m": 333, "k": 8192, "ns": "8192,1024,1024", "codes": True},
        # odd sizes: a ragged prompt, an odd number of channels, rows that end inside a tile
        {"name": "ragged_130", "op": "linear", "m": 130, "k": 4160, "ns": "1001"},
        # a training batch of 4096 tokens through gate of an 8B layer
        {"name": "train_4096_gate", "op": "linear", "m": 4096, "k": 4096, "ns": "14336"},
        # an adapted q projection of an 8B layer in training, LoRA rank 16
        {"name": "lora_2048_q", "op": "linear", "m": 2048, "k": 4096, "ns": "4096", "rank": 16},
        # input gradient of a short ragged batch through the o projection of an 8B layer
        {"name": "grad_40_o", "op": "grad", "m": 40, "k": 4096, "ns": "4096"},
        # input gradient of 2048 tokens through q, k and v of an 8B layer, summed
        {"name": "grad_2048_qkv", "op": "grad", "m": 2048, "k": 4096, "ns": "4096,1024,1024"},
        # input gradient of a training batch through gate of an 8B layer
        {"name": "grad_4096_gate", "op": "grad", "m": 4096, "k": 4096, "ns": "14336"},
        # the adapters of q and v of one 8B layer, rank 16: four small tensors, bound by launches
        {"name": "clip_qv_r16", "op": "clip", "layers": 1, "linears": "qv", "rank": 16, "bf16": False, "norm": "2"},
        # the adapters of every linear of a 32-layer 8B model, rank 64: 448 tensors, 168 million values
        {"name": "clip_all_r64", "op": "clip", "layers": 32, "linears": "qkvogud", "rank": 64, "bf16": False, "norm": "2"},
    ]


# (out, in) of the linears of an 8B layer, by their first letters
LINEARS = {"q": (4096, 4096), "k": (1024, 4096), "v": (1024, 4096), "o": (4096, 4096), "g": (14336, 4096),
           "u": (14336, 4096), "d": (4096, 14336)}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear", "grad", "clip"))
    if op == "clip":
        names = rng.choice(("qv", "qkvo", "gud", "qkvogud"))
        return {"op": op, "layers": _log_int(rng, 1, 32), "linears": names, "rank": rng.choice((4, 8, 13, 16, 32, 64)),
                "bf16": rng.random() < 0.4, "norm": rng.choice(("2", "2", "inf"))}
    while True:
        m = _log_int(rng, 1, 4096)
        k = 64 * _log_int(rng, 4, 448)
        ns = [_log_int(rng, 256, 14336) for _ in range(rng.choice((1, 1, 2, 3)))]
        if op == "grad":
            ns = [8 * -(-n // 8) for n in ns]
        if m * k * sum(ns) <= 4096 * 4096 * 14336:
            break
    case = {"op": op, "m": m, "k": k, "ns": ",".join(map(str, ns))}
    if op == "linear":
        form = rng.choice(("", "", "codes", "rank"))
        if form == "codes":
            case["codes"] = True
        elif form == "rank":
            case["rank"] = rng.choice((4, 8, 13, 16, 64))
    return case


def _ns(case):
    return [int(v) for v in case["ns"].split(",")]


def _adapter_shapes(case):
    shapes = []
    for layer in range(case["layers"]):
        for name in case["linears"]:
            n, k = LINEARS[name]
            shapes += [(case["rank"], k), (n, case["rank"])]
    return shapes


def _weight(n, k, gen):
    """8-bit rows of a normal weight with rare outliers, one scale a row."""
    w = torch.randn(n, k, generator=gen, device=DEV) * 0.02
    hot = torch.rand(n, k, generator=gen, device=DEV) < 0.001
    w = torch.where(hot, w * 20, w)
    s = w.abs().amax(1) / 127
    return torch.round(w / s[:, None]).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "clip":
        grads = []
        for i, shape in enumerate(_adapter_shapes(case)):
            g = torch.randn(shape, generator=gen, device=DEV) * 0.01
            grads.append(g.to(torch.bfloat16) if case["bf16"] and i % 2 else g)
        # the clipped gradients go to flat buffers, one for each type, that an optimizer reads whole
        flat, outs = [], [None] * len(grads)
        for dtype in (torch.float32, torch.bfloat16):
            at = [i for i, g in enumerate(grads) if g.dtype == dtype]
            if at:
                flat.append(torch.empty(sum(grads[i].numel() for i in at), dtype=dtype, device=DEV))
                for i, part in zip(at, flat[-1].split([grads[i].numel() for i in at])):
                    outs[i] = part.view(grads[i].shape)
        state = {"grads": grads, "outs": outs, "flat": flat, "max_norm": 1.0, "norm": case["norm"]}
        if case["norm"] == "inf":
            state["max_norm"] = 0.01
        if own:
            import group_wise_minmax_amd as L
            # the gradient buffers live as long as the training run: the program lists them once
            state["set"] = L.LbqGradSet(grads, state["outs"])
        return state
    m, k = case["m"], case["k"]
    state = {"m": m, "k": k, "weights": [_weight(n, k, gen) for n in _ns(case)]}
    if case["op"] == "grad":
        state["dys"] = [(torch.randn(m, n, generator=gen, device=DEV) * 0.01).to(torch.bfloat16) for n in _ns(case)]
    else:
        x = torch.randn(m, k, generator=gen, device=DEV)
        # a few input channels are far larger than the rest, as activations of language models have them
        hot = torch.rand(k, generator=gen, device=DEV) < 0.002
        state["x"] = torch.where(hot, x * 20, x).to(torch.bfloat16)
        if "rank" in case:
            r = case["rank"]
            state["lora"] = [((torch.randn(r, k, generator=gen, device=DEV) * 0.01).to(torch.bfloat16),
                              (torch.randn(n, r, generator=gen, device=DEV) * 0.01).to(torch.bfloat16)) for n in _ns(case)]
            state["sigma"] = 16.0 / r
    state["op"], state["codes"] = case["op"], bool(case.get("codes"))
    if own:
        import group_wise_minmax_amd as L
        # the frozen layers: their stored codes and scales, as a program holds them
        state["qws"] = [L.QuantizedWeight(L.make_desc("int8", q.shape[0], k), q.view(torch.uint8), s[:, None])
                        for q, s in state["weights"]]
    return state


def _plain_codes(x):
    """Token codes (as fp32 values) and scales."""
    x = x.float()
    s = x.abs().amax(1) / 127
    s = torch.where(s == 0, torch.ones_like(s), s)
    return torch.clamp(torch.round(x / s[:, None]), -127, 127), s


def _plain_linear(state):
    q, s = _plain_codes(state["x"])
    ys = [(q @ w.float().t()) * s[:, None] * sw for w, sw in state["weights"]]
    if "lora" in state:
        x = state["x"].float()
        ys = [y + state["sigma"] * ((x @ a.float().t()) @ b.float().t()) for y, (a, b) in zip(ys, state["lora"])]
    return [y.to(torch.bfloat16) for y in ys]


def _plain_grad(state):
    parts = [dy.float() @ (w.float() * sw[:, None]) for dy, (w, sw) in zip(state["dys"], state["weights"])]
    return [torch.stack(parts).sum(0).to(torch.bfloat16)] if len(parts) > 1 else [parts[0].to(torch.bfloat16)]


def _plain_clip(state):
    if state["norm"] == "inf":
        norm = torch.stack([g.float().abs().max() for g in state["grads"]]).max()
    else:
        # squares of 10^8 values: summed in 64 bits
        norm = torch.stack([g.double().square().sum() for g in state["grads"]]).sum().sqrt().float()
    c = torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0)
    for g, out in zip(state["grads"], state["outs"]):
        if g.dtype == torch.float32:
            torch.mul(g, c, out=out)
        else:
            out.copy_(g.float() * c)
    return [norm] + state["flat"]


def _own_linear(state):
    import group_wise_minmax_amd as L
    x, qws = state["x"], state["qws"]
    if "lora" in state:
        return [L.lbq_lora_fwd(x, qw, a, b, state["sigma"]) for qw, (a, b) in zip(qws, state["lora"])]
    if state["codes"]:
        q, s = L.lbq_quantize_tokens(x)
        return [L.lbq_linear_fwd_tokens(q, s, qw) for qw in qws]
    if len(qws) > 1:
        return L.lbq_linear_fwd_grouped(x, qws)
    return [L.lbq_linear_fwd(x, qws[0])]


def _own_grad(state):
    import group_wise_minmax_amd as L
    if len(state["qws"]) > 1:
        return [L.lbq_linear_bwd_dx_grouped(state["dys"], state["qws"])]
    return [L.lbq_linear_bwd_dx(state["dys"][0], state["qws"][0])]


def run(state):
    if "grads" in state:
        if own:
            norm = state["set"].clip(state["max_norm"], norm_type=float(state["norm"]))
            return [norm] + state["flat"]
        return _plain_clip(state)
    if state["op"] == "grad":
        return _own_grad(state) if own else _plain_grad(state)
    return _own_linear(state) if own else _plain_linear(state)


def work(case):
    if case["op"] == "clip":
        values = [r * c for r, c in _adapter_shapes(case)]
        size = [2 if case["bf16"] and i % 2 else 4 for i in range(len(values))]
        return {"bytes": 2 * sum(v * b for v, b in zip(values, size)) + 4, "flops": 3 * sum(values)}
    m, k, ns = case["m"], case["k"], _ns(case)
    weights = sum(n * k + 4 * n for n in ns)
    if case["op"] == "grad":
        return {"bytes": weights + 2 * m * sum(ns) + 2 * m * k, "flops": 2 * m * k * sum(ns)}
    r = case.get("rank", 0)
    lora = sum(2 * r * (k + n) for n in ns)
    return {"bytes": weights + lora + 2 * m * k + 2 * m * sum(ns), "flops": 2 * m * k * sum(ns) + sum(2 * m * r * (k + n) for n in ns)}


def exact(case, seed):
    """The definitions in 64 bits.  A token's scale is the 32-bit number nearest
    to its largest magnitude over 127, its codes the whole numbers nearest to
    the values over that scale."""
    global own
    mine, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = mine
    if case["op"] == "clip":
        wide = [g.double() for g in state["grads"]]
        if case["norm"] == "inf":
            norm = max(float(g.abs().max()) for g in wide)
        else:
            norm = math.sqrt(math.fsum(float(torch.dot(g.flatten(), g.flatten())) for g in wide))
        c = min(1.0, state["max_norm"] / (norm + 1e-6))
        flat = [torch.cat([g.flatten() for g, n in zip(wide, state["grads"]) if n.dtype == dtype])
                for dtype in (torch.float32, torch.bfloat16) if any(n.dtype == dtype for n in state["grads"])]
        return [torch.tensor(norm, dtype=torch.float64)] + [f.mul_(c) for f in flat]
    weights = [(w.double(), sw.double()) for w, sw in state["weights"]]
    if case["op"] == "grad":
        dx = torch.zeros(case["m"], case["k"], dtype=torch.float64, device=DEV)
        for dy, (w, sw) in zip(state["dys"], weights):
            dx.addmm_(dy.double() * sw, w)
        return [dx]
    x = state["x"].double()
    s = (x.abs().max(1).values / 127.0).float().double()
    s[s == 0] = 1.0
    q = (x / s.unsqueeze(1)).round().clamp(-127.0, 127.0)
    out = []
    for i, (w, sw) in enumerate(weights):
        y = torch.mm(q, w.t().contiguous()).mul_(s.unsqueeze(1)).mul_(sw.unsqueeze(0))
        if "lora" in state:
            a, b = (v.double() for v in state["lora"][i])
            y.addmm_(x @ a.t(), b.t(), alpha=state["sigma"])
        out.append(y)
    return out
