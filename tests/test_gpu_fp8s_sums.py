"""How far the sums of the fp8 products with block scales may be off, and where they are fp32 sums.

The fp8 matrix instruction cuts each product off at 2^-13 of the power of two of the largest of the eight (aligned) k that
it sums first: seven products may each lose up to 2^-13 of the largest.  The rest are fp32 sums.  SwiGLU's products of few
tokens or outputs are bf16 ones instead, whose products are cut at 2^-24 there."""
import pytest
import torch

import w4a16_routed_expert_moe_amd as moe
from gpu_common import say

pytestmark = pytest.mark.gpu

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
HALF = 2.0 ** -8
MOST = 1 << 23  # rows x columns up to which SwiGLU's sums are fp32 ones


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _nk(N, K):
    return (N + 127) // 128, (K + 127) // 128


def _pack(w):
    G, N, K = w.shape
    out = torch.empty(moe.moe_fp8s_packed_bytes(G, N, K), dtype=torch.uint8, device="cuda")
    moe.moe_fp8s_prepack(G, N, K, w, out)
    return out


def _ints(gen, *shape):
    """e4m3 codes of integers in [-3, 3]."""
    return torch.randint(-3, 4, shape, device="cuda", generator=gen).float().to(F8).view(torch.uint8)


def _twos(gen, *shape):
    return torch.randint(0, 2, shape, device="cuda", generator=gen).float() + 1.0


def _rows(codes, scales):
    return codes.view(F8).double() * scales.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]


def _weights(codes, scales):
    N, K = codes.shape[-2:]
    return codes.view(F8).double() * scales.double().repeat_interleave(128, -1)[..., :K].repeat_interleave(128, -2)[..., :N, :]


# ---------------------------------------------------------------- the bound of the fp8 instruction
@pytest.mark.parametrize("values", ["any", "one large in eight", "integers that cancel"])
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (3, 144, 16), (16, 64, 144), (40, 272, 400), (130, 80, 1040), (64, 4096, 144), (300, 528, 272)])
def test_products_within_their_bound(M, N, K, values):
    say("M=%d N=%d K=%d %s" % (M, N, K, values))
    gen = _gen(M + N + K)
    NB, KB = _nk(N, K)
    a, w = (torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=gen) for s in ((M, K), (N, K)))
    if values == "one large in eight":
        for t in (a, w):
            t[:] = (t & 0x80) | 0x28 + (t & 15)  # 2^-2 to 2^-1
            t[:, 5::8] = 0x78  # 256
    elif values == "integers that cancel":
        a, w = _cancelling(gen, M, K), _cancelling(gen, N, K, True)
    for t in (a, w):
        t[(t & 0x7F) == 0x7F] = 0  # not a number
    sa, sw = (torch.exp(torch.randn(s, device="cuda", generator=gen) * 3) for s in ((M, KB), (NB, KB)))
    out = torch.empty((M, N), dtype=BF16, device="cuda")
    moe.moe_fp8s_gemm(M, N, K, a, sa, _pack(w[None]), sw, out)
    torch.cuda.synchronize()
    x, y = _rows(a, sa), _weights(w, sw)
    want, size = torch.matmul(x, y.t()), torch.matmul(x.abs(), y.abs().t())
    lost = torch.zeros_like(want)
    for k in range(0, K, 8):  # (a block's scales are common to the eight)
        lost += 7 * 2.0 ** -13 * (x[:, None, k:k + 8] * y[None, :, k:k + 8]).abs().amax(2)
    # in fp32: sixteen eights of a block, up to three parts of it joined, the scales' product, its product with a block's sum and
    # the sum over the blocks (k in up to eight parts), each rounded or cut: 2^-23 of the sum of magnitudes
    bound = lost + size * (16 + 3 + 2 + KB + 8) * 2.0 ** -23
    assert ((out.double() - want).abs() <= want.abs() * HALF + bound * (1 + HALF)).all()


# ---------------------------------------------------------------- fp32 sums
def _cancelling(gen, n, K, weights=False):
    """Small integers, and in every 128 k the products 256 x 256 and -256 x 256 in two eights, which cancel: an fp32 sum
    (a cut at 2^-24 of 2^16, a sum of integers below 2^24) is exact, and one that cuts at 2^-13 of 2^16 loses the
    products of up to 7 beside them."""
    c = _ints(gen, n, K)
    c[:, 0::128] = 0x78
    c[:, 8::128] = 0x78 if weights else 0xF8
    return c


def _grouped(T, E, k, ns, N, K, act, n_src=None):
    """SwiGLU's outputs of cancelling products, and what they have to be."""
    gen = _gen(T + N + K)
    G, R = E + ns, T * (k + ns)
    NB, KB = _nk(N, K)
    desc = moe.MoeLayerDesc.make(512, 128, E, k, ns)
    cut = torch.randint(0, R + 1, (G - 1,), device="cuda", generator=gen).sort().values
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), R)]).to(torch.int32)
    if n_src is None:
        src, a = torch.arange(R, device="cuda"), _cancelling(gen, R, K)
        n_src, sa = R, _twos(gen, R, KB)
    else:  # some rows of a tensor of many
        at = torch.tensor([0, 1, n_src // 2, n_src - 2, n_src - 1], device="cuda")
        src, a = at[torch.arange(R, device="cuda") % len(at)], torch.zeros((n_src, K), dtype=torch.uint8, device="cuda")
        a[at] = _cancelling(gen, len(at), K)
        sa = torch.zeros((n_src, KB), device="cuda")
        sa[at] = _twos(gen, len(at), KB)
    w = torch.stack([_cancelling(gen, N, K, True) for _ in range(G)])
    sw = _twos(gen, G, NB, KB) * 2.0 ** -8
    out = torch.full((R + 1, N // 2), 7.0, dtype=BF16, device="cuda")
    moe.moe_fp8s_grouped_gemm(desc, T, a, sa, src.to(torch.int32), n_src, N, K, _pack(w), sw, off, act, out)
    torch.cuda.synchronize()
    assert (out[R] == 7.0).all()
    for g in range(G):
        r = slice(int(off[g]), int(off[g + 1]))
        z = torch.matmul(_rows(a[src[r]], sa[src[r]]), _weights(w[g], sw[g]).t())
        yield out[r].double(), z[:, :N // 2], z[:, N // 2:]


def _off_by_more(got, gate, up):
    """Outputs further from silu(gate) up than its bf16 rounding, and e^-gate, the reciprocal and the products in fp32, allow."""
    want = gate / (1 + torch.exp(-gate)) * up
    tol = want.abs() * (HALF + (2 * gate.abs() + 8) * 2.0 ** -23) + 2.0 ** -133
    return ((got - want).abs() > tol) & (gate > -80)


# tokens, experts, top-k, shared, columns, k: the stream; tiles with k in four parts, in two, and whole
FEW = [(1, 8, 2, 1, 256, 272), (4, 4, 2, 0, 128, 4112), (40, 12, 3, 1, 256, 272), (64, 5, 2, 1, 512, 144), (70, 3, 2, 1, 512, 1040),
       (300, 3, 2, 1, 1024, 1552), (300, 3, 2, 1, 1024, 272), (900, 40, 3, 1, 2048, 400)]


@pytest.mark.parametrize("T,E,k,ns,N,K", FEW)
def test_swiglu_of_few_outputs_sums_in_fp32(T, E, k, ns, N, K):
    assert T <= 64 or T * (k + ns) * N <= MOST
    for g, (got, gate, up) in enumerate(_grouped(T, E, k, ns, N, K, moe.MOE_ACT_SWIGLU)):
        assert not _off_by_more(got, gate, up).any(), g


def test_swiglu_of_few_outputs_of_far_rows_sums_in_fp32():
    """... gathered from more than 4 GB of codes."""
    n_src, K = (1 << 19) + 40, 8208
    assert n_src * K > 1 << 32 and 70 * 2 * 128 <= MOST
    for g, (got, gate, up) in enumerate(_grouped(70, 4, 2, 0, 128, K, moe.MOE_ACT_SWIGLU, n_src)):
        assert not _off_by_more(got, gate, up).any(), g


# more outputs than SwiGLU's sums are fp32 ones for by themselves: tiles of 64 x 128, of 256 x 256, and far rows
@pytest.mark.parametrize("T,E,k,ns,N,K,n_src", [(3000, 2, 2, 1, 1024, 272, None), (4500, 2, 2, 0, 2048, 400, None),
                                                (2100, 40, 3, 1, 1152, 144, None), (2200, 4, 2, 0, 2048, 8208, (1 << 19) + 40)])
def test_swiglu_f32_sums_in_fp32_at_any_size(T, E, k, ns, N, K, n_src):
    assert T * (k + ns) * N > MOST
    for g, (got, gate, up) in enumerate(_grouped(T, E, k, ns, N, K, moe.MOE_ACT_SWIGLU_F32, n_src)):
        assert not _off_by_more(got, gate, up).any(), g


@pytest.mark.parametrize("T,E,k,ns,N,K", FEW)
def test_swiglu_f32_is_swiglu_where_that_sums_in_fp32(T, E, k, ns, N, K):
    for (a, _, _), (b, _, _) in zip(_grouped(T, E, k, ns, N, K, moe.MOE_ACT_SWIGLU), _grouped(T, E, k, ns, N, K, moe.MOE_ACT_SWIGLU_F32)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- whole experts
def _definition(layer, x, buf, w13, w2):
    """The layer's output in 64 bits with the roundings that its definition has: codes of x, h, codes of h, y."""
    from test_gpu_fp8s import _deq_w, _row_ref
    d = layer.desc
    I, H, E, k = d.inter, d.hidden, d.n_routed, d.top_k

    def weights(w, g, N, K):
        codes = torch.empty((1, N, K), dtype=torch.uint8, device="cuda")
        scales = torch.empty((1, *_nk(N, K)), device="cuda")
        moe.moe_fp8s_quant_weights(1, N, K, w[g:g + 1].contiguous(), codes, scales)
        return _deq_w(codes, scales)[0]
    xq, idx = _rows(*_row_ref(x)), buf.topk_idx.long()
    want = torch.zeros((len(x), H), dtype=torch.float64, device="cuda")
    for e in range(d.groups):
        t, j = (idx == e).nonzero(as_tuple=True) if e < E else (torch.arange(len(x), device="cuda"), None)
        if len(t):
            z = xq[t] @ weights(w13, e, 2 * I, H).t()
            h = (z[:, :I] / (1 + torch.exp(-z[:, :I])) * z[:, I:]).to(BF16)
            y = (_rows(*_row_ref(h)) @ weights(w2, e, H, I).t()).to(BF16).double()
            want.index_add_(0, t, y if j is None else y * buf.topk_w.double()[t, j][:, None])
    return want


# Against the definition an output is off by its own rounding, at most 2^-8 / sqrt(3) of the norm, and by flips of y and of h.  A y
# whose sum is off by 2^-19 of its terms' sizes (the cut of the down product), 2^-13 of y with terms of random signs, lands
# beside its value with a chance of 2^-13 / 2^-8 = 2^-5 and is then off by 2^-7 of itself: 2^-7 2^-2.5 = 2^-9.5 at most.  Of fp32
# sums of gate and up (off by 2^-20 of either, the exponential's 2^-20 too) one h in 2^9 lands beside its bf16 value, one in 16 of those
# has another code, off by up to 2^-3: 2^-3 2^-6.5 = 2^-9.5 of h.  Together sqrt((2^-8)^2 / 3 + 2 (2^-9.5)^2) = 0.0030.
@pytest.mark.parametrize("T,H,I,E,k,ns,f32", [(1, 4096, 2048, 8, 6, 1, False), (64, 512, 256, 8, 2, 1, False), (70, 1024, 384, 16, 4, 1, False),
                                              (600, 512, 512, 12, 3, 1, False), (4000, 512, 2048, 8, 4, 1, True), (2500, 1024, 512, 20, 4, 1, True)])
def test_layer_of_fp32_sums(T, H, I, E, k, ns, f32):
    from test_gpu_fp8s import _layer
    case, layer, buf, w13, w2 = _layer(T, H, I, E, k, ns, T + I)
    R = layer.desc.rows(T)
    assert f32 == (T > 64 and R * 2 * I > MOST)
    layer = moe.MoELayer(layer.desc, layer.w_router, layer.gate_bias, layer.experts, f32_sums=f32)
    out = layer.forward(case.xd, buf)
    torch.cuda.synchronize()
    want = _definition(layer, case.xd, buf, w13, w2)
    err = float((out.double() - want).norm() / want.norm())
    say("  out %.2e" % err)
    assert err <= 0.0030


def test_layer_of_fp32_sums_is_the_layer_where_that_sums_in_fp32():
    from test_gpu_fp8s import _layer
    for T in (5, 40, 200):
        case, layer, buf, _, _ = _layer(T, 512, 256, 8, 2, 1, T)
        other = moe.MoELayer(layer.desc, layer.w_router, layer.gate_bias, layer.experts, f32_sums=True)
        a = layer.forward(case.xd, buf).clone()
        assert torch.equal(a, other.forward(case.xd, buf))
    none = moe.Buffers(layer.desc, 0, fp8s=True)
    assert other.forward(case.xd[:0], none).shape == (0, 512)


def test_refusals():
    from test_gpu_fp8s import _layer
    _, layer, buf, w13, w2 = _layer(4, 512, 128, 4, 2, 1, 0)
    with pytest.raises(ValueError, match="f32_sums"):
        moe.MoELayer(layer.desc, layer.w_router, layer.gate_bias, moe.bf16_weights(w13, w2), f32_sums=True)
    with pytest.raises(ValueError, match="out holds"):
        moe.moe_fp8s_grouped_gemm(layer.desc, 4, buf.xq, buf.xqs, buf.sorted_token, 4, 256, 512, layer.experts.w13, layer.experts.s13,
                                  buf.group_offsets, moe.MOE_ACT_SWIGLU_F32, buf.h.reshape(-1)[:-1])
