"""What lies beside an operand of the bf16 products does not reach their results: rows, weights and columns that are not
finite, next to where a group, a row or the contraction ends inside a tile.

The tiles fill up with zeros past the end of a group; whatever is read there instead is multiplied by the zeros of the
other operand, which hides every finite value and shows an infinity or a NaN.  Inputs are small integers, so that the
results of the finite groups are compared bit for bit (see test_gpu_bf16.py)."""
import pytest
import torch

import w4a16_routed_expert_moe_amd as moe
from gpu_common import say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
BAD = (float("nan"), float("inf"), -float("inf"))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(gen, *shape):
    return torch.randint(-4, 5, shape, device="cuda", generator=gen).to(BF16)


def _bad(gen, *shape):
    return torch.tensor(BAD, dtype=BF16, device="cuda")[torch.randint(0, 3, shape, device="cuda", generator=gen)]


def _offsets(sizes):
    return torch.tensor([0] + sizes, dtype=torch.int32).cumsum(0).to(torch.int32)


def _desc(G):
    return moe.MoeLayerDesc.make(512, 128, G, 1, 0)


def _gather(gen, n, on):
    """A gather of n rows from n + 3 sources (a permutation, three of them unused), or None."""
    return torch.randperm(n + 3, device="cuda", generator=gen)[:n].to(torch.int32) if on else None


def _source(rows, gather):
    """The tensor that `gather` reads as rows."""
    if gather is None:
        return rows
    a = torch.full((len(rows) + 3, rows.shape[1]), float("nan"), dtype=BF16, device="cuda")
    a[gather.long()] = rows
    return a


# groups that end inside a step of 64 rows, the first row of every other group and all that follow in it not finite
SHORT = [17, 9, 1, 30, 63, 64, 65, 3, 40, 129, 100, 16]


@pytest.mark.parametrize("mode", [moe.MOE_GRAD_BF16, moe.MOE_GRAD_F32, moe.MOE_GRAD_F32_ADD])
@pytest.mark.parametrize("which", ["dy", "a", None])
@pytest.mark.parametrize("N,K", [(80, 48), (272, 400), (16, 1040), (3600, 4096)])  # the last: tiles of 256 x 256
def test_rows_of_the_next_group(N, K, which, mode):
    say("wgrad N=%d K=%d gathered %s mode %d" % (N, K, which, mode))
    gen, G, R = _gen(N + K), len(SHORT), sum(SHORT)
    if N > 1000:  # as launch_wide counts them
        assert G * -(-N // 256) * -(-K // 256) >= 2048
    off = _offsets(SHORT)
    odd = torch.zeros(R, dtype=torch.bool, device="cuda")
    for g in range(1, G, 2):
        odd[off[g]:off[g + 1]] = True
    rows = {"dy": _ints(gen, R, N), "a": _ints(gen, R, K)}
    for t in rows.values():
        t[odd] = _bad(gen, int(odd.sum()), t.shape[1])
    gather = _gather(gen, R, which is not None)
    at = {n: gather if n == which else None for n in rows}
    kind = BF16 if mode == moe.MOE_GRAD_BF16 else torch.float32
    dw = torch.full((G, N, K), 3.0, dtype=kind, device="cuda")
    moe.moe_bf16_grouped_wgrad(_desc(G), R, _source(rows["dy"], at["dy"]), at["dy"], _source(rows["a"], at["a"]), at["a"], R + 3, N, K,
                               off.cuda(), mode, dw)
    torch.cuda.synchronize()
    for g in range(0, G, 2):
        r = slice(int(off[g]), int(off[g + 1]))
        want = torch.matmul(rows["dy"][r].double().t(), rows["a"][r].double())
        if mode == moe.MOE_GRAD_F32_ADD:
            want += 3.0
        assert torch.equal(dw[g], want.float().to(kind)), g
    for g in range(1, G, 2):
        assert not torch.isfinite(dw[g]).any(), g


@pytest.mark.parametrize("mode", [moe.MOE_GRAD_BF16, moe.MOE_GRAD_F32])
@pytest.mark.parametrize("which", ["dy", "a"])
@pytest.mark.parametrize("N,K", [(80, 48), (272, 400), (3600, 4096)])
def test_rows_without_a_source_add_nothing(N, K, which, mode):
    """... whatever the other operand holds in them."""
    gen, G, R = _gen(N - K), len(SHORT), sum(SHORT)
    off = _offsets(SHORT)
    rows = {"dy": _ints(gen, R, N), "a": _ints(gen, R, K)}
    none = torch.arange(R, device="cuda") % 5 == 2
    for t in rows.values():
        t[none] = _bad(gen, int(none.sum()), t.shape[1])
    at = _gather(gen, R, True)
    source = _source(rows[which], at)
    at[none] = torch.tensor([-1, R + 3, -(1 << 31), (1 << 31) - 1], dtype=torch.int32, device="cuda")[torch.arange(int(none.sum()), device="cuda") % 4]
    given = {n: (source, at) if n == which else (t, None) for n, t in rows.items()}
    kind = BF16 if mode == moe.MOE_GRAD_BF16 else torch.float32
    dw = torch.empty((G, N, K), dtype=kind, device="cuda")
    moe.moe_bf16_grouped_wgrad(_desc(G), R, *given["dy"], *given["a"], R + 3, N, K, off.cuda(), mode, dw)
    torch.cuda.synchronize()
    for g in range(G):
        r = torch.arange(int(off[g]), int(off[g + 1]), device="cuda")
        r = r[~none[r]]
        assert torch.equal(dw[g], torch.matmul(rows["dy"][r].double().t(), rows["a"][r].double()).float().to(kind)), g


# rows a group, output columns: tiles of 64 x 128, 128 x 128 and 256 x 256
@pytest.mark.parametrize("rows,K", [(10, 272), (70, 400), (500, 9040)])
@pytest.mark.parametrize("N", [16, 48, 80, 176, 272])
@pytest.mark.parametrize("gather", [True, False])
def test_weights_of_the_next_group(rows, K, N, gather):
    say("dgrad %d rows N=%d K=%d" % (rows, N, K))
    sizes = [rows, rows + 1, rows - 3, rows + 5, rows + 17, rows]
    gen, G, R = _gen(N + K), len(sizes), sum(sizes)
    if rows == 500:
        assert R >= 128 * G and (-(-R // 256) + G // 2) * -(-K // 256) >= 512
    off = _offsets(sizes)
    w, dy = _ints(gen, G, N, K), _ints(gen, R, N)
    w[1::2] = _bad(gen, *w[1::2].shape)
    at = _gather(gen, R, gather)
    da = torch.empty((R, K), dtype=BF16, device="cuda")
    moe.moe_bf16_grouped_dgrad(_desc(G), R, _source(dy, at), at, R + 3, N, K, w, off.cuda(), da)
    torch.cuda.synchronize()
    for g in range(G):
        r = slice(int(off[g]), int(off[g + 1]))
        if g % 2:
            assert not torch.isfinite(da[r]).all(0).any(), g
        else:
            assert torch.equal(da[r], torch.matmul(dy[r].double(), w[g].double()).float().to(BF16)), g


def _silu(g):
    return g / (1 + torch.exp(-g))


# rows of each group, columns, k: the stream, tiles of 64 x 256 (64 MB of weights), of 64 x 128, 128 x 128 and 256 x 256
@pytest.mark.parametrize("sizes,N,K", [([2, 0, 1, 3], 96, 80), ([20] * 33, 1056, 1040), ([21] * 24, 288, 144), ([70, 65, 60, 80], 288, 208),
                                       ([700, 801, 650, 705], 8224, 336)])
@pytest.mark.parametrize("act", [moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU])
def test_the_next_row_of_weights_and_of_tokens(sizes, N, K, act):
    """Every other weight row and every third token not finite: the columns and rows between them do not see it."""
    say("forward %d groups N=%d K=%d act %d" % (len(sizes), N, K, act))
    gen, G, R = _gen(N + K), len(sizes), sum(sizes)
    off = _offsets(sizes)
    w, a = _ints(gen, G, N, K), _ints(gen, R, K)
    w *= 0.25
    good = torch.arange(0, N, 2, device="cuda")
    w[:, 1::2] = _bad(gen, *w[:, 1::2].shape)
    bad_row = torch.arange(R, device="cuda") % 3 == 1
    a[bad_row] = _bad(gen, int(bad_row.sum()), K)
    C = N // 2 if act == moe.MOE_ACT_SWIGLU else N
    out = torch.empty((R, C), dtype=BF16, device="cuda")
    moe.moe_bf16_grouped_gemm(_desc(G), R, a, None, 0, N, K, w, off.cuda(), act, None, out)
    torch.cuda.synchronize()
    for g in range(G):
        r = torch.arange(int(off[g]), int(off[g + 1]), device="cuda")
        r = r[~bad_row[r]]
        z = torch.matmul(a[r].double(), w[g][good].double().t())
        got = out[r][:, :C:2]
        if act == moe.MOE_ACT_NONE:
            assert torch.equal(got, z.float().to(BF16)), g
        else:  # half a step of bf16, and e^-g, the reciprocal and the products in fp32 (see test_gpu_bf16.py)
            gate, up = z[:, :C // 2], z[:, C // 2:]
            want = _silu(gate) * up
            tol = want.abs() * (2.0 ** -8 + (2 * gate.abs() + 8) * 2.0 ** -23) + 2.0 ** -133
            assert (((got.double() - want).abs() <= tol) | (gate < -80)).all(), g
        assert not torch.isfinite(out[r][:, 1:C:2]).any(), g


@pytest.mark.parametrize("which", ["dy", "a", None])
@pytest.mark.parametrize("N,K", [(80, 48), (3600, 4096)])
def test_gradients_of_groups_without_rows_are_not_touched(N, K, which):
    """Added to, the fp32 gradient of a group without rows keeps its bits (a minus zero with zero added would be plus zero)."""
    sizes = [0, 40, 0, 0, 7, 0, 70, 0, 0]
    gen, G, R = _gen(N), len(sizes), sum(sizes)
    rows = {"dy": _ints(gen, R, N), "a": _ints(gen, R, K)}
    gather = _gather(gen, R, which is not None)
    at = {n: gather if n == which else None for n in rows}
    dw = torch.full((G, N, K), -0.0, device="cuda")
    moe.moe_bf16_grouped_wgrad(_desc(G), R, _source(rows["dy"], at["dy"]), at["dy"], _source(rows["a"], at["a"]), at["a"], R + 3, N, K,
                               _offsets(sizes).cuda(), moe.MOE_GRAD_F32_ADD, dw)
    torch.cuda.synchronize()
    off = _offsets(sizes)
    for g in range(G):
        if not sizes[g]:
            assert (dw[g].view(torch.int32) == -(1 << 31)).all(), g
        else:
            r = slice(int(off[g]), int(off[g + 1]))
            assert torch.equal(dw[g], torch.matmul(rows["dy"][r].double().t(), rows["a"][r].double()).float()), g


@pytest.mark.parametrize("T,H,I,E", [(70, 512, 256, 8), (3000, 512, 4096, 4)])  # tiles of d_h: 128 x 128, 256 x 256
def test_what_is_not_wanted_is_not_written(T, H, I, E):
    """Only the routing weights' gradient, or with frozen weights that of the rows: the workspace holds no more than they need."""
    gen, k = _gen(T), 3
    desc, R = moe.MoeLayerDesc.make(H, I, E, k, 0), T * k
    if T == 3000:
        assert R >= 128 * E and (-(-R // 256) + E // 2) * -(-I // 256) >= 512
    buf = moe.Buffers(desc, T, train=True)
    idx = torch.rand((T, E), device="cuda", generator=gen).topk(k, dim=1).indices.to(torch.int32)
    moe.moe_permute(desc, T, idx, buf.group_offsets, buf.sorted_token, buf.row_of_slot, buf.ws)
    x, d_out = (torch.randn((T, H), device="cuda", generator=gen).to(BF16) for _ in range(2))
    w13 = (torch.randn((E, 2 * I, H), device="cuda", generator=gen) / H ** 0.5).to(BF16)
    w2 = (torch.randn((E, H, I), device="cuda", generator=gen) / I ** 0.5).to(BF16)
    buf.topk_w.fill_(0.5)
    moe.moe_bf16_experts(desc, T, x, buf.topk_w, buf.group_offsets, buf.sorted_token, buf.row_of_slot, w13, w2, buf.gu, buf.h, buf.y, buf.out)
    d2 = torch.empty(w2.shape, device="cuda")

    def written(*outs):
        buf.grad_ws.fill_(171)
        moe.moe_bf16_experts_backward(desc, T, d_out, x, buf.topk_w, buf.group_offsets, buf.sorted_token, buf.row_of_slot, w13, w2, buf.gu,
                                      buf.h, moe.MOE_GRAD_F32, *outs, buf.grad_ws)
        torch.cuda.synchronize()
        return int((buf.grad_ws != 171).sum())
    part, rows_i, rows_h = 4 * R * -(-I // 128), 2 * R * I, 2 * R * H
    assert written(None, None, None, None) == 0
    assert 0 < written(None, None, None, buf.d_topk_w) <= part
    want = buf.d_topk_w.clone()
    assert rows_i < written(buf.d_x, None, None, buf.d_topk_w) <= part + 2 * rows_i + rows_h
    assert torch.equal(buf.d_topk_w, want)
    assert rows_i / 2 < written(None, None, d2, None) <= part + rows_i


@pytest.mark.parametrize("T", [6, 300])
def test_backward_does_not_touch_the_gradients_of_idle_experts(T):
    """The same of the whole backward pass (few tiles: all gradients in one launch; and each in its own)."""
    H, I, E, k = (512, 128, 24, 1) if T == 6 else (4096, 2048, 9, 1)
    gen = _gen(T)
    desc = moe.MoeLayerDesc.make(H, I, E, k, 0)
    buf = moe.Buffers(desc, T, train=True)
    idx = torch.arange(T, dtype=torch.int32, device="cuda")[:, None] % 3 * 2 + 1  # experts 1, 3 and 5
    moe.moe_permute(desc, T, idx, buf.group_offsets, buf.sorted_token, buf.row_of_slot, buf.ws)
    x, d_out = (torch.randn((T, H), device="cuda", generator=gen).to(BF16) for _ in range(2))
    w13 = (torch.randn((E, 2 * I, H), device="cuda", generator=gen) / H ** 0.5).to(BF16)
    w2 = (torch.randn((E, H, I), device="cuda", generator=gen) / I ** 0.5).to(BF16)
    buf.topk_w.fill_(0.5)
    d13, d2 = (torch.full(w.shape, -0.0, device="cuda") for w in (w13, w2))
    moe.moe_bf16_experts(desc, T, x, buf.topk_w, buf.group_offsets, buf.sorted_token, buf.row_of_slot, w13, w2, buf.gu, buf.h, buf.y, buf.out)
    moe.moe_bf16_experts_backward(desc, T, d_out, x, buf.topk_w, buf.group_offsets, buf.sorted_token, buf.row_of_slot, w13, w2, buf.gu,
                                  buf.h, moe.MOE_GRAD_F32_ADD, buf.d_x, d13, d2, buf.d_topk_w, buf.grad_ws)
    torch.cuda.synchronize()
    for e in range(E):
        for d in (d13, d2):
            assert (d[e] != 0).any() if e in (1, 3, 5) else (d[e].view(torch.int32) == -(1 << 31)).all(), e
