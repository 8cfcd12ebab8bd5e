"""The products' tiles of 256 rows by 256 columns over many steps of the contraction, with ragged groups and contractions.

Every batch of thousands of tokens runs in these tiles: both stages of their loop, the steps whose contraction ends inside,
row tiles of every fill (they multiply by 64 rows as many as they have) and more than one block of columns.  Inputs are
small integers, so that sums are exact in fp32 and results are compared bit for bit with 64-bit arithmetic.  Each test
asserts the condition on which the library takes the large tile (launch_forward and launch_wide in bf16, launch_tiled in
fp8), so that a changed threshold does not drop the coverage unnoticed."""
import pytest
import torch

import w4a16_routed_expert_moe_amd as moe
from gpu_common import say

pytestmark = pytest.mark.gpu

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
HALF = 2.0 ** -8
# rows of the groups: last tiles of 1, 70, 130, 200, 256, 231, 33 and 188 rows, and a group without
SIZES = [257, 326, 386, 456, 768, 0, 999, 33, 700]
STEPS = [48, 128, 192, 208, 1040, 2048]  # contractions: 1, 2, 3, 4, 17 and 32 steps of 64


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(gen, *shape, top=4):
    return torch.randint(-top, top + 1, shape, device="cuda", generator=gen).to(BF16)


def _up(a, b):
    return -(-a // b)


def _bounds(sizes):
    return torch.tensor([0] + sizes).cumsum(0).tolist()


def _offsets(sizes):
    return torch.tensor(_bounds(sizes), dtype=torch.int32, device="cuda")


def _desc(G):
    return moe.MoeLayerDesc.make(512, 128, G, 1, 0)


def _large_rows(R, G, columns):
    """Of launch_wide, for the products over the permuted rows."""
    return R >= 128 * G and (_up(R, 256) + min(R, G) // 2) * _up(columns, 256) >= 512


def _silu(g):
    return g / (1 + torch.exp(-g))


def _gathered(gen, R, width):
    """Rows of a tensor in another order, one of them without a source."""
    a, at = _ints(gen, R, width), torch.randperm(R, device="cuda", generator=gen)
    at[R // 2] = -1
    rows = torch.where(at[:, None] >= 0, a.double()[at.clamp(min=0)], 0.0)
    return a, at.to(torch.int32), rows


@pytest.mark.parametrize("K", STEPS)
@pytest.mark.parametrize("act", [moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU])
def test_bf16_product(K, act):
    N, G, R = 6688, len(SIZES), sum(SIZES)
    # (SwiGLU's tiles: 128 columns of either projection)
    assert _large_rows(R, G, N) and not R < 64 * G
    say("K=%d act %d" % (K, act))
    gen, at = _gen(K + act), _bounds(SIZES)
    a, gather, rows = _gathered(gen, R, K)
    w = _ints(gen, G, N, K) * (0.125 if act == moe.MOE_ACT_SWIGLU else 1.0)
    C = N // 2 if act == moe.MOE_ACT_SWIGLU else N
    out = torch.full((R + 1, C), 7.0, dtype=BF16, device="cuda")
    gu = torch.full((R + 1, N), 5.0, dtype=BF16, device="cuda") if act == moe.MOE_ACT_SWIGLU else None
    moe.moe_bf16_grouped_gemm(_desc(G), R, a, gather, R, N, K, w, _offsets(SIZES), act, gu, out)
    torch.cuda.synchronize()
    assert (out[R] == 7.0).all() and (gu is None or (gu[R] == 5.0).all())
    for g in range(G):
        r = slice(at[g], at[g + 1])
        z = torch.matmul(rows[r], w[g].double().t())
        if gu is None:
            assert torch.equal(out[r], z.float().to(BF16)), g
            continue
        assert torch.equal(gu[r], z.float().to(BF16)), g
        gate, up = z[:, :C], z[:, C:]
        want = _silu(gate) * up
        # e^-g with its argument rounded, the reciprocal and the products in fp32, one rounding to bf16
        tol = want.abs() * (HALF + (2 * gate.abs() + 8) * 2.0 ** -23) + 2.0 ** -133
        assert (((out[r].double() - want).abs() <= tol) | (gate < -80)).all(), g


@pytest.mark.parametrize("N", STEPS)
@pytest.mark.parametrize("gather", [True, False])
def test_bf16_gradient_of_rows(N, gather):
    K, G, R = 6672, len(SIZES), sum(SIZES)
    assert _large_rows(R, G, K)
    say("contraction %d" % N)
    gen, at = _gen(N), _bounds(SIZES)
    dy, index, rows = _gathered(gen, R, N)
    if not gather:
        index, rows = None, dy.double()
    w = _ints(gen, G, N, K)
    da = torch.full((R + 1, K), 7.0, dtype=BF16, device="cuda")
    moe.moe_bf16_grouped_dgrad(_desc(G), R, dy, index, R, N, K, w, _offsets(SIZES), da)
    torch.cuda.synchronize()
    assert (da[R] == 7.0).all()
    for g in range(G):
        r = slice(at[g], at[g + 1])
        assert torch.equal(da[r], torch.matmul(rows[r], w[g].double()).float().to(BF16)), g


@pytest.mark.parametrize("mode", [moe.MOE_GRAD_BF16, moe.MOE_GRAD_F32, moe.MOE_GRAD_F32_ADD])
@pytest.mark.parametrize("which", ["dy", "a", None])
@pytest.mark.parametrize("N,K", [(3600, 4096), (4096, 3856)])
def test_bf16_gradient_of_weights(N, K, which, mode):
    G, R = len(SIZES), sum(SIZES)
    assert G * _up(N, 256) * _up(K, 256) >= 2048
    say("N=%d K=%d gathered %s mode %d" % (N, K, which, mode))
    gen, at = _gen(N + mode), _bounds(SIZES)
    dy, dy_at, dy_rows = _gathered(gen, R, N)
    a, a_at, a_rows = _gathered(gen, R, K)
    if which != "dy":
        dy_at, dy_rows = None, dy.double()
    if which != "a":
        a_at, a_rows = None, a.double()
    kind = BF16 if mode == moe.MOE_GRAD_BF16 else torch.float32
    dw = torch.full((G * N * K + 64,), 3.0, dtype=kind, device="cuda")
    moe.moe_bf16_grouped_wgrad(_desc(G), R, dy, dy_at, a, a_at, R, N, K, _offsets(SIZES), mode, dw)
    torch.cuda.synchronize()
    assert (dw[G * N * K:] == 3.0).all()
    got = dw[:G * N * K].view(G, N, K)
    for g in range(G):
        r = slice(at[g], at[g + 1])
        want = torch.matmul(dy_rows[r].t(), a_rows[r])
        if mode == moe.MOE_GRAD_F32_ADD:
            want += 3.0
        assert torch.equal(got[g], want.float().to(kind)), g


def _routing(gen, T, E, k, ns):
    """Uneven groups: the e-th expert as popular as 1 / (e + 1); and what moe_permute makes of it."""
    noise = -torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=gen).clamp(1e-20, 1 - 1e-7)))
    idx = (noise - torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))).topk(k, dim=1).indices
    slots = torch.cat([idx, torch.full((T, ns), E, device="cuda")], 1)
    order = slots.reshape(-1).sort(stable=True).indices
    row = torch.empty_like(order)
    row[order] = torch.arange(len(order), device="cuda")
    sizes = torch.bincount(slots.reshape(-1), minlength=E + ns)
    return order // (k + ns), row.reshape(T, k + ns), torch.cat([sizes.new_zeros(1), sizes.cumsum(0)])


@pytest.mark.parametrize("mode", [moe.MOE_GRAD_BF16, moe.MOE_GRAD_F32, moe.MOE_GRAD_F32_ADD])
@pytest.mark.parametrize("T,H,I,E,k,ns,large", [(20, 512, 128, 4, 2, 1, False), (400, 512, 384, 4, 2, 1, False), (300, 1024, 768, 40, 3, 0, False),
                                                (2050, 512, 4096, 4, 3, 1, True), (2050, 2048, 4096, 4, 3, 1, True),
                                                (5600, 1024, 2048, 5, 2, 1, True)])
def test_bf16_backward_bit_exact(T, H, I, E, k, ns, large, mode):
    """The whole backward pass on integers.  Gates are 0 or 18, whose sigmoids are 1/2 and, as 1 + e^-18 rounds to 1, 1: the
    gradients behind the activation are d_h w u / 2 and 0, or d_h w u and 18 d_h w, rounded once.  Routing weights are powers of two."""
    G, R = E + ns, T * (k + ns)
    assert large == _large_rows(R, G, I)
    say("T=%d H=%d I=%d mode %d" % (T, H, I, mode))
    gen = _gen(T + H + mode)
    token, row, bounds = _routing(gen, T, E, k, ns)
    d_out, x = _ints(gen, T, H, top=1), _ints(gen, T, H, top=2)
    w13, w2 = _ints(gen, G, 2 * I, H, top=1), _ints(gen, G, H, I, top=1)
    gu, h = _ints(gen, R, 2 * I, top=2), _ints(gen, R, I, top=3)
    gu[:, :I] = 18.0 * torch.randint(0, 2, (R, I), device="cuda", generator=gen)
    topk_w = torch.exp2(torch.randint(-1, 2, (T, k), device="cuda", generator=gen).float())
    desc = moe.MoeLayerDesc.make(H, I, E, k, ns)
    kind = BF16 if mode == moe.MOE_GRAD_BF16 else torch.float32
    d_w13, d_w2 = torch.full(w13.shape, 3.0, dtype=kind, device="cuda"), torch.full(w2.shape, 3.0, dtype=kind, device="cuda")
    d_x, d_topk_w = torch.empty((T, H), dtype=BF16, device="cuda"), torch.empty((T, k), device="cuda")
    ws = torch.full((moe.moe_bf16_backward_workspace_bytes(desc, T),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_bf16_experts_backward(desc, T, d_out, x, topk_w, bounds.to(torch.int32), token.to(torch.int32), row.to(torch.int32), w13, w2,
                                  gu, h, mode, d_x, d_w13, d_w2, d_topk_w, ws)
    torch.cuda.synchronize()
    weight = torch.ones(R, dtype=torch.float64, device="cuda")
    weight[row[:, :k].reshape(-1)] = topk_w.double().reshape(-1)
    dxs, dot = torch.zeros((R, H), dtype=torch.float64, device="cuda"), torch.zeros(R, dtype=torch.float64, device="cuda")
    start = 3.0 if mode == moe.MOE_GRAD_F32_ADD else 0.0
    cut = bounds.tolist()
    for g in range(G):
        r = slice(cut[g], cut[g + 1])
        d, u = d_out.double()[token[r]], gu[r, I:].double()
        on = gu[r, :I].double() / 18.0
        dh = torch.matmul(d, w2[g].double())
        dot[r] = (dh * h[r].double()).sum(1)
        dw = dh * weight[r, None]
        dgu = torch.cat([dw * u * (0.5 + 0.5 * on), 18.0 * dw * on], 1).float().to(BF16).double()
        dxs[r] = torch.matmul(dgu, w13[g].double()).float().to(BF16).double()
        assert torch.equal(d_w13[g], (start + torch.matmul(dgu.t(), x.double()[token[r]])).float().to(kind)), g
        hw = (weight[r, None] * h[r].double()).float().to(BF16).double()
        assert torch.equal(d_w2[g], (start + torch.matmul(d.t(), hw)).float().to(kind)), g
    assert torch.equal(d_topk_w, dot[row[:, :k]].float())
    assert torch.equal(d_x, dxs[row].sum(1).float().to(BF16))


# ---------------------------------------------------------------- fp8
FP8_SIZES = [257, 326, 386, 456, 768, 0, 999, 33, 700, 1900, 3000, 320]


def _deq_w(codes, scales):
    N, K = codes.shape
    return codes.view(F8).double() * scales.double().repeat_interleave(128, -1)[:, :K].repeat_interleave(128, -2)[:N]


@pytest.mark.parametrize("act", [moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("K", [80, 144, 400, 1040, 2192, 4096])
def test_fp8_product(K, act, gather):
    """(integers of at most 9 are not cut off beside each other: 2^-13 of 2^3)"""
    N, G, R = 2048, len(FP8_SIZES), sum(FP8_SIZES)
    assert R >= 128 * G and (R // 256 + min(R, G)) * _up(N, 256) >= 256 and R * N > 1 << 23
    say("K=%d act %d" % (K, act))
    gen, cut, KB = _gen(K + act), _bounds(FP8_SIZES), _up(K, 128)
    def codes(*shape):
        return torch.randint(-3, 4, shape, device="cuda", generator=gen).float().to(F8).view(torch.uint8)
    def twos(*shape):
        return torch.randint(0, 2, shape, device="cuda", generator=gen).float() + 1.0
    a, sa, w = codes(R, K), twos(R, KB), codes(G, N, K)
    sw = twos(G, _up(N, 128), KB) * (2.0 ** -8 if act == moe.MOE_ACT_SWIGLU else 1.0)
    src = torch.randperm(R, device="cuda", generator=gen) if gather else torch.arange(R, device="cuda")
    if gather:
        src[[5, 1000]] = torch.tensor([-1, R], device="cuda")
    packed = torch.empty(moe.moe_fp8s_packed_bytes(G, N, K), dtype=torch.uint8, device="cuda")
    moe.moe_fp8s_prepack(G, N, K, w, packed)
    C = N // 2 if act == moe.MOE_ACT_SWIGLU else N
    out = torch.full((R + 1, C), 7.0, dtype=BF16, device="cuda")
    moe.moe_fp8s_grouped_gemm(_desc(G), R, a, sa, src.to(torch.int32) if gather else None, R, N, K, packed, sw, _offsets(FP8_SIZES), act, out)
    torch.cuda.synchronize()
    assert (out[R] == 7.0).all()
    ok = (src >= 0) & (src < R)
    x = a.view(F8).double() * sa.double().repeat_interleave(128, 1)[:, :K]
    x = torch.where(ok[:, None], x[src.clamp(0, R - 1)], 0.0)
    for g in range(G):
        r = slice(cut[g], cut[g + 1])
        z = torch.matmul(x[r], _deq_w(w[g], sw[g]).t())
        if act == moe.MOE_ACT_NONE:
            assert torch.equal(out[r], z.float().to(BF16)), g
        else:
            gate, up = z[:, :C], z[:, C:]
            want = _silu(gate) * up
            tol = want.abs() * (HALF + (2 * gate.abs() + 8) * 2.0 ** -23) + 2.0 ** -133
            assert (((out[r].double() - want).abs() <= tol) | (gate < -80)).all(), g
