"""What is measured of the framework's 8-bit integer products and of its router's loss and gradients.

Three kinds of case:

* ``linear``: a projection with INT8 weights (one scale per output channel) of bf16 tokens that are quantised to
  INT8 with one scale per token on the way; out = bf16.
* ``experts``: the routed and shared experts of one MoE layer with INT8 weights, from the routing's outputs to the
  layer's output: gate/up with SwiGLU, down, weighted combine; x and h are quantised per token.
* ``router``: the step that trains or watches a router: the counts of tokens per expert, the balance loss of packed
  sequences, and the gradient of the router's logits from that loss and from the routing weights' gradient.

The definitions are those of ``include/moe_w4a16.h``.  Where ``own`` is false the operators are computed in their
plain form, elementary torch operations in 32 bits (64 where a value is next to a rounding border or a sum is long).
"""
import math

import torch

own = False

HIDDEN = (512, 1024, 2048, 4096)
INTER = (128, 256, 512, 768, 1024, 1536, 2048)


def listed():
    return [
        # one token of a decode step through a square projection of the layer's hidden size: launch latency and the weight stream
        {"name": "linear_1", "op": "linear", "M": 1, "N": 4096, "K": 4096},
        # a small decode batch with ragged widths (a fused projection's odd number of channels)
        {"name": "linear_61", "op": "linear", "M": 61, "N": 8208, "K": 2064},
        # a short prompt, too few rows to fill the card with large tiles
        {"name": "linear_640", "op": "linear", "M": 640, "N": 4096, "K": 2048},
        # a prefill chunk of 8192 tokens through the projection that the FP8_BLOCK benchmark has
        {"name": "linear_8192", "op": "linear", "M": 8192, "N": 4096, "K": 4096},
        # the decode step of one token through the whole layer's experts
        {"name": "experts_1", "op": "experts", "T": 1, "H": 4096, "I": 2048, "E": 256, "k": 6, "ns": 1, "skew": 0.0},
        # a decode batch of 64 tokens with a skewed popularity of experts
        {"name": "experts_64", "op": "experts", "T": 64, "H": 4096, "I": 2048, "E": 256, "k": 6, "ns": 1, "skew": 1.1},
        # a smaller layer with ragged groups
        {"name": "experts_421", "op": "experts", "T": 421, "H": 1024, "I": 512, "E": 40, "k": 3, "ns": 1, "skew": 0.0},
        # a prefill chunk of 8192 tokens through the whole layer's experts
        {"name": "experts_8192", "op": "experts", "T": 8192, "H": 4096, "I": 2048, "E": 256, "k": 6, "ns": 1, "skew": 0.0},
        # a few tokens: launch latency
        {"name": "router_33", "op": "router", "T": 33, "E": 256, "k": 6, "S": 1, "pad": 0.0},
        # many short sequences packed together, some of them empty, an odd number of experts
        {"name": "router_1000", "op": "router", "T": 1000, "E": 41, "k": 3, "S": 48, "pad": 0.1},
        # a prefill chunk of one layer, padded
        {"name": "router_8192", "op": "router", "T": 8192, "E": 256, "k": 6, "S": 8, "pad": 0.05},
        # a training step's tokens on one GPU
        {"name": "router_65536", "op": "router", "T": 65536, "E": 256, "k": 6, "S": 16, "pad": 0.0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("linear", "experts", "router"))
    if op == "linear":
        c = {"op": op, "M": _log(rng, 1, 8192), "N": 16 * _log(rng, 8, 1024), "K": 16 * _log(rng, 8, 512)}
        while c["M"] * c["N"] * c["K"] > 8192 * 4096 * 4096:
            c["M"] = max(1, c["M"] // 2)
        return c
    if op == "experts":
        E = _log(rng, 1, 256)
        c = {"op": op, "T": _log(rng, 1, 8192), "H": rng.choice(HIDDEN), "I": rng.choice(INTER), "E": E,
             "k": rng.randint(1, min(8, E)), "ns": rng.choice((0, 1, 1)), "skew": rng.choice((0.0, 1.1))}
        if c["T"] > 512:  # padded per expert in the plain form
            c["skew"] = 0.0
        while c["T"] * (c["k"] + c["ns"]) * c["H"] * c["I"] > 8192 * 7 * 4096 * 2048:
            c["T"] = max(1, c["T"] // 2)
        return c
    E = _log(rng, 2, 256)
    T = _log(rng, 1, 65536)
    return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(8, E)), "S": min(_log(rng, 1, 64), T + 1), "pad": rng.choice((0.0, 0.1))}


# ---------------------------------------------------------------- inputs
def _weights(G, N, K, gen):
    """INT8 codes [G][N][K] of normally distributed weights, and their scale per channel."""
    w = torch.empty((G, N, K), dtype=torch.int8, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for g in range(0, G, step):
        part = torch.randn(w[g:g + step].shape, device="cuda", generator=gen)
        w[g:g + step] = part.mul_(31.0).round_().clamp_(-127, 127).to(torch.int8)
    scale = (0.5 + torch.rand((G, N), device="cuda", generator=gen)) * (1.0 / 31.0 / math.sqrt(K))
    return w, scale


def _tokens(T, K, gen):
    """bf16 activations: normal, each token at a scale of its own, a few large channels."""
    x = torch.randn((T, K), device="cuda", generator=gen)
    x *= 0.3 + torch.rand((T, 1), device="cuda", generator=gen)
    x[:, :: 97] *= 4.0
    return x.to(torch.bfloat16)


def _choice(T, E, k, skew, gen):
    """k distinct experts of each token, the e-th as popular as 1 / (e + 1) ** skew."""
    noise = -torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=gen).clamp(1e-20, 1 - 1e-7)))
    pop = -skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return (noise + pop).topk(k, dim=1).indices


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"linear": _prepare_linear, "experts": _prepare_experts, "router": _prepare_router}[case["op"]](case, gen)


def _prepare_linear(c, gen):
    M, N, K = c["M"], c["N"], c["K"]
    w, ws = _weights(1, N, K, gen)
    s = dict(c, x=_tokens(M, K, gen), ws=ws[0], w=w[0])
    if own:  # the weights in the kernels' layout instead of the canonical one, and the call's buffers
        import w4a16_routed_expert_moe_amd as moe
        s["w"] = torch.empty(moe.moe_w8a8_packed_bytes(1, N, K), dtype=torch.int8, device="cuda")
        moe.moe_w8a8_prepack(1, N, K, w, s["w"])
        s["codes"] = torch.empty((M, K), dtype=torch.int8, device="cuda")
        s["scales"] = torch.empty(M, dtype=torch.float32, device="cuda")
        s["out"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_experts(c, gen):
    T, H, I, E, k, ns = (c[n] for n in ("T", "H", "I", "E", "k", "ns"))
    G, R = E + ns, T * (k + ns)
    idx = _choice(T, E, k, c["skew"], gen)
    score = torch.sigmoid(torch.randn((T, k), device="cuda", generator=gen))
    slots = torch.cat([idx, torch.full((T, ns), E, device="cuda", dtype=idx.dtype)], 1)
    order = slots.reshape(-1).sort(stable=True).indices  # the slot of each permuted row
    row = torch.empty_like(order)
    row[order] = torch.arange(R, device="cuda")
    sizes = torch.bincount(slots.reshape(-1), minlength=G)
    s = dict(c, x=_tokens(T, H, gen), topk_w=score / score.sum(1, keepdim=True),
             offsets=torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).to(torch.int32),
             token=(order // (k + ns)).to(torch.int32), row=row.reshape(T, k + ns).to(torch.int32))
    w13, s["s13"] = _weights(G, 2 * I, H, gen)
    w2, s["s2"] = _weights(G, H, I, gen)
    if own:  # the experts in the kernels' layout, and the buffers that a layer keeps
        import w4a16_routed_expert_moe_amd as moe
        s["desc"] = moe.MoeLayerDesc.make(H, I, E, k, ns)
        s["experts"] = moe.ExpertWeights(w13=moe.prepack(w13, G, 2 * I, H, fmt="int8"), s13=s.pop("s13"),
                                         w2=moe.prepack(w2, G, H, I, fmt="int8"), s2=s.pop("s2"), fmt="int8")
        s["buf"] = moe.Buffers(s["desc"], T, int8=True)
        return s
    s["w13"], s["w2"] = w13, w2
    # the plain form multiplies the routed experts that have rows as one batch: their row numbers, padded with R
    active = sizes[:E].nonzero()[:, 0]
    most = int(sizes[:E].max())
    at = s["offsets"][:-1].long()[active][:, None] + torch.arange(most, device="cuda")
    s["active"] = None if active.numel() == E else active
    s["rows"] = torch.where(torch.arange(most, device="cuda") < sizes[active][:, None], at, R)
    return s


def _prepare_router(c, gen):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    logits = torch.randn((T, E), device="cuda", generator=gen) * 1.3
    cuts = torch.randint(0, T + 1, (S + 1,), device="cuda", generator=gen).sort().values
    cuts[0] = 0
    cuts[-1] = T
    s = dict(c, logits=logits, idx=logits.topk(k, dim=1).indices.to(torch.int32), offsets=cuts.to(torch.int32),
             mask=(torch.rand(T, device="cuda", generator=gen) >= c["pad"]).to(torch.uint8) if c["pad"] else None,
             d_loss=torch.rand(1, device="cuda", generator=gen) + 0.5,
             d_w=torch.randn((T, k), device="cuda", generator=gen) * (1.0 / T), alpha=0.01)
    if own:
        import w4a16_routed_expert_moe_amd as moe
        s["desc"] = moe.MoeLayerDesc.make(4096, 2048, E, k, 0)
        s["counts"] = torch.empty((S, E), dtype=torch.int32, device="cuda")
        s["prob"] = torch.empty((S, E), dtype=torch.float32, device="cuda")
        s["coef"] = torch.empty(S, dtype=torch.float32, device="cuda")
        s["loss"] = torch.empty(1, dtype=torch.float32, device="cuda")
        s["d_logits"] = torch.empty((T, E), dtype=torch.float32, device="cuda")
        s["ws"] = torch.zeros(moe.moe_balance_workspace_bytes(s["desc"], T, S), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"linear": _plain_linear, "experts": _plain_experts, "router": _plain_router}[s["op"]](s)


def _own(s):
    import w4a16_routed_expert_moe_amd as moe
    if s["op"] == "linear":
        moe.moe_w8a8_linear(s["M"], s["N"], s["K"], s["x"], s["w"], s["ws"], s["codes"], s["scales"], s["out"])
        return s["out"]
    if s["op"] == "experts":
        w, b = s["experts"], s["buf"]
        moe.moe_w8a8_experts(s["desc"], s["T"], s["x"], s["topk_w"], s["offsets"], s["token"], s["row"], w.w13, w.s13,
                             w.w2, w.s2, b.xq8, b.xqs8, b.h, b.hq8, b.hqs8, b.y, b.out)
        return b.out
    moe.moe_balance_loss(s["desc"], s["T"], s["S"], s["offsets"], s["mask"], s["logits"], s["idx"], s["alpha"],
                         s["counts"], s["prob"], s["coef"], s["loss"], s["ws"])
    moe.moe_route_backward(s["desc"], s["T"], s["S"], s["offsets"], s["mask"], s["logits"], s["idx"], s["counts"],
                           s["coef"], s["d_loss"], s["d_w"], s["d_logits"])
    return {"loss": s["loss"], "counts": s["counts"], "prob": s["prob"], "coef": s["coef"], "d_logits": s["d_logits"]}


def _quant(x):
    """INT8 codes (as fp32 values) and the scale of each row; the quotient in 64 bits, for it decides a rounding."""
    amax = x.abs().amax(1, keepdim=True).double()
    codes = torch.where(amax > 0, (x.double() * 127.0 / amax).round(), 0.0)
    return codes.float(), (amax / 127.0).float()


def _plain_linear(s):
    codes, scale = _quant(s["x"])
    return ((codes @ s["w"].float().t()) * scale * s["ws"]).to(torch.bfloat16)


def _product(s, a, scale, w, ws):
    """Rows of each group times its weights, times both scales: the routed groups as one padded batch, the shared one by itself."""
    E, T, R = s["E"], s["T"], a.shape[0]
    pick = slice(0, E) if s["active"] is None else s["active"]
    pad = torch.cat([a, a.new_zeros(1, a.shape[1])])[s["rows"]]
    y = torch.bmm(pad, w[pick].float().transpose(1, 2)) * ws[pick][:, None, :]
    out = a.new_empty((R + 1, w.shape[1]))
    out[s["rows"].reshape(-1)] = y.reshape(-1, w.shape[1])
    if s["ns"]:
        out[R - T:R] = (a[R - T:] @ w[E].float().t()) * ws[E]
    return out[:R] * scale


def _plain_experts(s):
    # h and y are bf16 tensors of the layer, so their rounding belongs to the definition
    I, token, row = s["I"], s["token"].long(), s["row"].long()
    codes, scale = _quant(s["x"])
    g = _product(s, codes[token], scale[token], s["w13"], s["s13"])
    h = (g[:, :I] * torch.sigmoid(g[:, :I]) * g[:, I:]).to(torch.bfloat16)
    y = _product(s, *_quant(h), s["w2"], s["s2"]).to(torch.bfloat16).float()
    out = (y[row[:, :s["k"]]] * s["topk_w"][:, :, None]).sum(1)
    return (out + y[row[:, s["k"]]] if s["ns"] else out).to(torch.bfloat16)


def _member_sums(m, v):
    """sum_t m[s][t] v[t][e] in 64 bits, in blocks of 256 tokens: one long skinny product of a library is many times slower."""
    short = -m.shape[1] % 256
    m = torch.nn.functional.pad(m.double(), (0, short)).reshape(m.shape[0], -1, 256).transpose(0, 1)
    v = torch.nn.functional.pad(v.double(), (0, 0, 0, short)).reshape(-1, 256, v.shape[1])
    return torch.bmm(m.contiguous(), v).sum(0)


def _plain_router(s):
    T, E, k, S = s["T"], s["E"], s["k"], s["S"]
    idx, off = s["idx"].long(), s["offsets"].long()
    t = torch.arange(T, device="cuda")
    member = (t >= off[:-1, None]) & (t < off[1:, None])
    if s["mask"] is not None:
        member = member & (s["mask"] != 0)
    live = member.any(0)[:, None]
    score = torch.sigmoid(s["logits"])
    total = score.sum(1, keepdim=True)
    p = torch.where(live, score / total, 0.0)
    chosen = torch.zeros((T, E), device="cuda").scatter_(1, idx, 1.0)
    counts, prob, n = _member_sums(member, chosen), _member_sums(member, p), member.sum(1).double()
    some = (n > 0).sum().clamp(min=1)
    coef = torch.where(n > 0, s["alpha"] * E / (k * n.clamp(min=1) ** 2 * some), 0.0)
    loss = (coef * (counts * prob).sum(1)).sum()
    c = ((coef * s["d_loss"].double())[:, None] * counts).float()
    seq = member.float().argmax(0)
    ct = c[seq]
    ds = (ct - (ct * p).sum(1, keepdim=True)) / total
    sk = score.gather(1, idx)
    sum_k = sk.sum(1, keepdim=True)
    dw = s["d_w"]
    ds = ds.scatter_add(1, idx, (dw - (dw * sk).sum(1, keepdim=True) / sum_k) / sum_k)
    return {"loss": loss.float().reshape(1), "counts": counts.to(torch.int32), "prob": prob.float(),
            "coef": coef.float(), "d_logits": torch.where(live, ds * score * (1.0 - score), 0.0)}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N, "flops": 2 * M * N * K}
    if case["op"] == "experts":
        T, H, I, E, k, ns = (case[n] for n in ("T", "H", "I", "E", "k", "ns"))
        # the experts that T tokens with k evenly spread choices each reach
        groups = E * (1.0 - (1.0 - k / E) ** T) + ns
        return {"bytes": int(groups * (3 * I * H + 4 * (2 * I + H))) + 4 * T * H + 12 * T * (k + ns),
                "flops": 2 * T * (k + ns) * 3 * I * H}
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    return {"bytes": 8 * T * E + 8 * T * k + (T if case["pad"] else 0) + 8 * S * E, "flops": 30 * T * E}


# ---------------------------------------------------------------- in 64 bits, from the definitions
def _exact_codes(x):
    x = x.double()
    top = x.abs().max(dim=1).values
    v = x * 127 / torch.where(top > 0, top, torch.ones_like(top))[:, None]
    low = torch.floor(v)
    up = (v - low > 0.5) | ((v - low == 0.5) & (torch.remainder(low, 2) == 1))
    return low + up.double(), top / 127


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"linear": _exact_linear, "experts": _exact_experts, "router": _exact_router}[case["op"]](s)


def _exact_linear(s):
    q, a = _exact_codes(s["x"])
    return a[:, None] * s["ws"].double()[None] * torch.matmul(q, s["w"].double().t())


def _exact_experts(s):
    I, k, ns, R = s["I"], s["k"], s["ns"], s["token"].numel()
    token, bounds = s["token"].long(), s["offsets"].tolist()
    q, a = _exact_codes(s["x"])
    y = torch.zeros((R, s["H"]), dtype=torch.float64, device="cuda")
    for g in range(s["E"] + ns):
        lo, hi = bounds[g], bounds[g + 1]
        if lo == hi:
            continue
        r = token[lo:hi]
        z = torch.matmul(q[r], s["w13"][g].double().t()) * a[r][:, None] * s["s13"][g].double()
        gate, up = z[:, :I], z[:, I:]
        hq, ha = _exact_codes((gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16))
        y[lo:hi] = torch.matmul(hq, s["w2"][g].double().t()) * ha[:, None] * s["s2"][g].double()
    weight = torch.cat([s["topk_w"].double(), torch.ones((s["T"], ns), dtype=torch.float64, device="cuda")], 1)
    out = torch.zeros((s["T"], s["H"]), dtype=torch.float64, device="cuda")
    for j in range(k + ns):
        out += weight[:, j:j + 1] * y[s["row"][:, j].long()]
    return out


def _exact_router(s):
    E, k, S = s["E"], s["k"], s["S"]
    x = s["logits"].double().requires_grad_(True)
    score = 1 / (1 + torch.exp(-x))
    share = score / score.sum(1, keepdim=True)
    idx, bounds = s["idx"].long(), s["offsets"].tolist()
    live = torch.ones(s["T"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    parts, counts, prob, sizes = [], [], [], []
    for q in range(S):
        at = torch.arange(bounds[q], bounds[q + 1], device="cuda")
        at = at[live[at]]
        sizes.append(at.numel())
        counts.append(torch.bincount(idx[at].reshape(-1), minlength=E).double())
        prob.append(share[at].sum(0))
        parts.append(E / (k * max(1, at.numel()) ** 2) * torch.dot(counts[-1], prob[-1]))
    some = max(1, sum(n > 0 for n in sizes))
    loss = s["alpha"] * torch.stack(parts).sum() / some
    chosen = score.gather(1, idx)
    weights = chosen / chosen.sum(1, keepdim=True)
    total = s["d_loss"].double() * loss + (s["d_w"].double() * weights)[live].sum()
    grad, = torch.autograd.grad(total, x)
    coef = torch.tensor([s["alpha"] * E / (k * n * n * some) if n else 0.0 for n in sizes], dtype=torch.float64, device="cuda")
    return {"loss": loss.detach().reshape(1), "counts": torch.stack(counts).to(torch.int32), "prob": torch.stack(prob).detach(),
            "coef": coef, "d_logits": grad}
