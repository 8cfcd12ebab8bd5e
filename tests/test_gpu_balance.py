"""GPU parity of the router's balance (counts, loss) and of the gradient of its
logits, against fp64.

Bounds.  A score's exponential is taken at a product rounded to fp32, so for
|x| <= 8 its relative error is at most 8 * 1.45 * 2^-24 plus a few units of
2^-23 for the hardware exponential, reciprocal and multiplications: below
2^-20 together.  A probability divides by a sum of such scores (positive, so
its relative error is no larger than theirs, plus 8 roundings): 2^-18.  A sum
over n tokens adds n 2^-24.  In the gradient each term is a product of at most
eight such factors, relative to the sum of the absolute values of what it
subtracts: 2^-16 of that."""
import numpy as np
import pytest
import torch

import w4a16_routed_expert_moe_amd as moe
from gpu_common import say

pytestmark = pytest.mark.gpu


def _reference(x, idx, off, mask, k, alpha, scale, d_loss, d_w):
    """fp64 on the host, one token at a time's formulas over whole arrays; also the gradient's bound."""
    T, E = x.shape
    S = len(off) - 1
    x = x.astype(np.float64)
    s = np.zeros_like(x)
    seq = np.full(T, -1)
    for q in range(S):
        seq[off[q]:off[q + 1]] = q
    live = seq >= 0
    if mask is not None:
        live &= mask != 0
    seq[~live] = -1
    s[live] = 1 / (1 + np.exp(-x[live]))
    tot = s.sum(1)
    p = np.divide(s, tot[:, None], out=np.zeros_like(s), where=tot[:, None] > 0)
    counts = np.zeros((S, E), np.int64)
    prob = np.zeros((S, E))
    n = np.zeros(S)
    for q in range(S):
        t = np.nonzero(seq == q)[0]
        n[q] = len(t)
        prob[q] = p[t].sum(0)
        np.add.at(counts[q], idx[t].reshape(-1), 1)
    some = (n > 0).sum()
    coef = np.where(n > 0, alpha * E / (k * np.maximum(n, 1) ** 2 * max(some, 1)), 0.0)
    loss = (coef[:, None] * counts * prob).sum()
    ds, size = np.zeros_like(x), np.zeros_like(x)
    for t in np.nonzero(live)[0]:
        if d_loss is not None and tot[t] > 0:
            c = d_loss * coef[seq[t]] * counts[seq[t]]
            ds[t] += (c - (c * p[t]).sum()) / tot[t]
            size[t] += (np.abs(c) + np.abs(c * p[t]).sum()) / tot[t]
        if d_w is not None:
            si = s[t, idx[t]]
            if si.sum() > 0:
                g = scale * (d_w[t] - (d_w[t] * si).sum() / si.sum()) / si.sum()
                np.add.at(ds[t], idx[t], g)
                np.add.at(size[t], idx[t], np.abs(scale) * (np.abs(d_w[t]) + (np.abs(d_w[t]) * si).sum() / si.sum()) / si.sum())
    slope = s * (1 - s)
    return counts, prob, coef, loss, ds * slope, size * slope, n


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Step:
    """One call of each entry point on host inputs; shift: elements by which logits and their gradient are moved off
    their 16-byte alignment."""

    def __init__(self, x, idx, off, mask, k, alpha=0.01, scale=1.0, d_loss=1.0, d_w=None, shift=0):
        T, E = x.shape
        self.T, self.S, self.alpha = T, len(off) - 1, alpha
        self.desc = moe.MoeLayerDesc.make(512, 128, E, k, 0, scale)
        flat = torch.zeros(T * E + 4, dtype=torch.float32, device="cuda")
        self.x = flat[shift:shift + T * E].view(T, E)
        self.x.copy_(_dev(x))
        self.idx, self.off, self.mask = _dev(idx.astype(np.int32)), _dev(off.astype(np.int32)), _dev(mask)
        self.d_w = _dev(d_w)
        self.d_loss = None if d_loss is None else torch.tensor([d_loss], dtype=torch.float32, device="cuda")
        self.counts = torch.full((self.S + 1, E), -5, dtype=torch.int32, device="cuda")
        self.prob = torch.full((self.S + 1, E), 7.0, device="cuda")
        self.coef = torch.full((self.S + 1,), 7.0, device="cuda")
        self.loss = torch.full((2,), 7.0, device="cuda")
        self.grad = torch.full((T * E + 4 + E,), 7.0, device="cuda")
        self.d_logits = self.grad[shift:shift + (T + 1) * E].view(T + 1, E)
        self.ws = torch.zeros(moe.moe_balance_workspace_bytes(self.desc, T, self.S), dtype=torch.uint8, device="cuda")

    def run(self):
        moe.moe_balance_loss(self.desc, self.T, self.S, self.off, self.mask, self.x, self.idx, self.alpha, self.counts,
                             self.prob, self.coef, self.loss, self.ws)
        moe.moe_route_backward(self.desc, self.T, self.S, self.off, self.mask, self.x, self.idx, self.counts, self.coef,
                               self.d_loss, self.d_w, self.d_logits)
        return self


def _check(st, ref, n_max):
    counts, prob, coef, loss, grad, size, n = ref
    torch.cuda.synchronize()
    tol = 2.0 ** -18 + n_max * 2.0 ** -24
    assert np.array_equal(st.counts[:-1].cpu().numpy(), counts)
    assert (np.abs(st.prob[:-1].double().cpu().numpy() - prob) <= tol * prob).all()
    assert (np.abs(st.coef[:-1].double().cpu().numpy() - coef) <= 2.0 ** -23 * coef).all()
    assert abs(float(st.loss[0]) - loss) <= (tol + 2.0 ** -23) * loss
    got = st.d_logits[:-1].double().cpu().numpy()
    assert (np.abs(got - grad) <= 2.0 ** -16 * size + 1e-38).all()
    # what lies behind the outputs is as it was
    assert (st.counts[-1] == -5).all() and (st.prob[-1] == 7.0).all() and float(st.coef[-1]) == 7.0
    assert float(st.loss[1]) == 7.0 and (st.d_logits[-1] == 7.0).all()


def _inputs(rng, T, E, k, scale=1.5):
    x = np.clip(rng.standard_normal((T, E)) * scale, -8, 8).astype(np.float32)
    idx = np.argsort(-x, 1, kind="stable")[:, :k]
    return x, idx


def _cuts(rng, T, S, first=0, last=None):
    last = T if last is None else last
    return np.concatenate([[first], np.sort(rng.integers(first, last + 1, S - 1)), [last]])


@pytest.mark.parametrize("T,E,k,S,first,last,pad,shift", [
    (1, 1, 1, 1, 0, None, 0.0, 0), (1, 256, 6, 1, 0, None, 0.0, 0), (2, 5, 5, 3, 0, None, 0.0, 0),
    (33, 256, 8, 1, 0, None, 0.2, 0), (128, 64, 2, 64, 0, None, 0.1, 0), (129, 64, 2, 2, 0, None, 0.0, 0),
    (128, 40, 3, 65, 0, None, 0.0, 0), (100, 41, 3, 70, 0, None, 0.3, 0), (300, 256, 6, 7, 17, 250, 0.1, 0),
    (1000, 41, 3, 48, 0, None, 0.1, 0), (513, 63, 4, 5, 100, 100, 0.0, 0), (777, 128, 4, 1, 0, None, 0.0, 1),
    (777, 256, 4, 900, 3, 770, 0.0, 2), (4099, 256, 6, 8, 0, None, 0.05, 0), (20000, 16, 2, 3, 0, None, 0.0, 0),
    (40000, 65, 2, 5, 0, None, 0.1, 0),
])
def test_against_fp64(T, E, k, S, first, last, pad, shift):
    say("balance T=%d E=%d k=%d S=%d" % (T, E, k, S))
    rng = np.random.default_rng(T + E + S)
    x, idx = _inputs(rng, T, E, k)
    off = _cuts(rng, T, S, first, last)
    if S > 6:
        off[3] = off[2]  # empty sequences
        off[4] = off[2]
        off = np.sort(off)
    mask = (rng.random(T) >= pad).astype(np.uint8) * 3 if pad else None
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    st = Step(x, idx, off, mask, k, scale=1.5, d_loss=0.75, d_w=d_w, shift=shift).run()
    _check(st, _reference(x, idx, off, mask, k, 0.01, 1.5, 0.75, d_w), T)


@pytest.mark.parametrize("d_loss,with_w", [(None, True), (2.0, False), (None, False)])
def test_one_term_only(d_loss, with_w):
    rng = np.random.default_rng(1)
    x, idx = _inputs(rng, 200, 48, 4)
    off = np.array([0, 60, 200])
    d_w = rng.standard_normal((200, 4)).astype(np.float32) if with_w else None
    st = Step(x, idx, off, None, 4, d_loss=d_loss, d_w=d_w).run()
    _check(st, _reference(x, idx, off, None, 4, 0.01, 1.0, d_loss, d_w), 200)
    if d_loss is None:  # without that term the counts are not needed
        moe.moe_route_backward(st.desc, st.T, st.S, st.off, None, st.x, st.idx, None, None, None, st.d_w, st.d_logits)
        torch.cuda.synchronize()
        _check(st, _reference(x, idx, off, None, 4, 0.01, 1.0, d_loss, d_w), 200)


@pytest.mark.parametrize("T", [50, 500])
def test_masked_rows_hold_anything(T):
    """NaN, infinities and the lowest value in masked rows and behind the last sequence; an expert masked by the
    lowest value or minus infinity; a sequence whose tokens are all masked; a row whose scores are all zero."""
    rng = np.random.default_rng(T)
    E, k = 32, 4
    x, idx = _inputs(rng, T, E, k)
    off = np.array([2, 10, 20, T - 5])
    mask = np.ones(T, np.uint8)
    mask[10:20] = 0
    mask[[3, 25, 30]] = 0
    clean = x.copy()
    for t, v in ((3, np.nan), (11, np.inf), (12, -np.inf), (25, np.nan), (30, -3.4e38), (0, np.nan), (T - 1, np.nan),
                 (T - 5, np.inf)):
        x[t] = v
        clean[t] = 0
    low = np.float32(-3.4028234663852886e38)
    for a in (x, clean):
        a[:, 7] = np.where(np.isfinite(a[:, 7]), low, a[:, 7])
        a[:, 9] = np.where(np.isfinite(a[:, 9]), -np.inf, a[:, 9])
        a[22] = -np.inf
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    with np.errstate(over="ignore"):
        ref = _reference(clean, idx, off, mask, k, 0.01, 1.0, 1.0, d_w)
    st = Step(x, idx, off, mask, k, d_w=d_w).run()
    _check(st, ref, T)
    assert int(st.counts[1].abs().sum()) == 0 and float(st.coef[1]) == 0.0
    dead = torch.tensor([0, 1, 3, 12, 25, 30, T - 5, T - 1])
    assert (st.d_logits[dead] == 0).all() and (st.d_logits[22] == 0).all()


def test_nan_stays_in_its_sequence():
    rng = np.random.default_rng(8)
    x, idx = _inputs(rng, 600, 64, 2)
    off = np.array([0, 200, 400, 600])
    want = Step(x, idx, off, None, 2).run()
    x[250, 3] = np.nan
    got = Step(x, idx, off, None, 2).run()
    torch.cuda.synchronize()
    assert torch.equal(got.prob[[0, 2]], want.prob[[0, 2]]) and torch.isnan(got.prob[1]).all()
    assert torch.equal(got.d_logits[:200], want.d_logits[:200]) and torch.equal(got.d_logits[400:600], want.d_logits[400:600])
    assert torch.isnan(got.d_logits[250]).any() and not torch.isnan(got.d_logits[251:600]).any()
    assert torch.isnan(got.loss[0])


def test_no_sequences_given_and_empty_calls():
    rng = np.random.default_rng(5)
    x, idx = _inputs(rng, 300, 64, 3)
    st = Step(x, idx, np.array([0, 300]), None, 3).run()
    want = [t.clone() for t in (st.counts, st.prob, st.coef, st.loss, st.d_logits)]
    st.off = None
    for t in (st.counts[:-1], st.prob[:-1], st.loss[:1], st.d_logits[:-1]):
        t.zero_()
    st.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (st.counts, st.prob, st.coef, st.loss, st.d_logits)))
    for S in (1, 70):  # no token at all: zeros in every output, the one-launch form and the other
        z = Step(x[:0], idx[:0], np.zeros(S + 1), None, 3).run()
        torch.cuda.synchronize()
        assert not z.counts[:-1].any() and not z.prob[:-1].any() and not z.coef[:-1].any() and float(z.loss[0]) == 0
        assert (z.d_logits == 7.0).all()


def test_ids_outside_are_not_counted_and_repeats_add():
    rng = np.random.default_rng(6)
    x, idx = _inputs(rng, 400, 24, 3)
    idx[5] = [-1, 24, 3]
    idx[300] = [2, 2, 2]
    st = Step(x, idx, np.array([0, 400]), None, 3, d_w=rng.standard_normal((400, 3)).astype(np.float32)).run()
    torch.cuda.synchronize()
    want = np.zeros(24, np.int64)
    ok = (idx >= 0) & (idx < 24)
    np.add.at(want, idx[ok], 1)
    assert np.array_equal(st.counts[0].cpu().numpy(), want)
    assert torch.isfinite(st.d_logits).all()


def test_nothing_is_left_where_it_cancels():
    """One choice per token: its weight is constant, its gradient exactly zero.  Nearly even counts: the balance term is
    a small difference, still within 1e-6 of its own 2-norm (its parts are about 40 times larger than it; a difference
    formed after rounding them would be off by 40 2^-23)."""
    rng = np.random.default_rng(12)
    x, idx = _inputs(rng, 300, 40, 1)
    d_w = rng.standard_normal((300, 1)).astype(np.float32)
    st = Step(x, idx, np.array([0, 300]), None, 1, d_loss=None, d_w=d_w).run()
    torch.cuda.synchronize()
    assert (st.d_logits[:-1] == 0).all()
    x = (rng.standard_normal((1280, 64)) * 0.02).astype(np.float32)
    idx = np.stack([np.arange(1280) % 64, (np.arange(1280) + 7) % 64], 1)
    idx[:40, 0] = (idx[:40, 0] + 1) % 64
    idx[0] = [5, 9]
    st = Step(x, idx, np.array([0, 1280]), None, 2).run()
    torch.cuda.synchronize()
    grad = _reference(x, idx, np.array([0, 1280]), None, 2, 0.01, 1.0, 1.0, None)[4]
    got = st.d_logits[:-1].double().cpu().numpy()
    assert np.linalg.norm(got - grad) <= 1e-6 * np.linalg.norm(grad)


@pytest.mark.parametrize("T", [700, 9001])
def test_runs_of_empty_sequences(T):
    """Thousands of empty sequences before, between and behind those that hold tokens."""
    rng = np.random.default_rng(T)
    x, idx = _inputs(rng, T, 20, 3)
    cuts = np.sort(rng.integers(0, T + 1, 5))
    off = np.concatenate([[0] * 1000] + [[c] * n for c, n in zip(cuts, (1, 3000, 2, 700, 64))] + [[T] * 900])
    st = Step(x, idx, off, None, 3, d_w=rng.standard_normal((T, 3)).astype(np.float32)).run()
    _check(st, _reference(x, idx, off, None, 3, 0.01, 1.0, 1.0, st.d_w.cpu().numpy()), T)


def test_scores_near_the_smallest():
    """Every score of a token near 2^-120 and large upstream gradients: 1 / sum of scores times them passes fp32's range,
    the gradient itself does not.  At |x| <= 86 the exponential's argument is off by 86 * 1.45 * 2^-24 < 2^-17, a score by
    less than 2^-16, a gradient of eight such factors by 2^-13 of its terms' sizes."""
    rng = np.random.default_rng(21)
    x = -rng.uniform(80, 86, (6, 8)).astype(np.float32)
    idx = np.stack([rng.permutation(8)[:2] for _ in range(6)])
    d_w = (rng.standard_normal((6, 2)) * 1e4).astype(np.float32)
    off = np.array([0, 6])
    for d_loss, w in ((1e6, None), (None, d_w), (1e6, d_w)):
        st = Step(x, idx, off, None, 2, d_loss=d_loss, d_w=w).run()
        torch.cuda.synchronize()
        ref = _reference(x, idx, off, None, 2, 0.01, 1.0, d_loss, w)
        got = st.d_logits[:-1].double().cpu().numpy()
        assert np.isfinite(got).all()
        assert (np.abs(got - ref[4]) <= 2.0 ** -13 * ref[5]).all()


def test_same_bits_every_call():
    rng = np.random.default_rng(7)
    x, idx = _inputs(rng, 9000, 256, 6)
    st = Step(x, idx, _cuts(rng, 9000, 5), None, 6, d_w=rng.standard_normal((9000, 6)).astype(np.float32)).run()
    first = [t.clone() for t in (st.counts, st.prob, st.coef, st.loss, st.d_logits)]
    for _ in range(5):
        st.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (st.counts, st.prob, st.coef, st.loss, st.d_logits)))


def test_gradient_against_differences():
    """Central differences of alpha-loss plus weighted routing weights, both in fp64 (steps of 1e-4: error about
    1e-8 of the third derivative, below 1e-6 of the largest gradient)."""
    rng = np.random.default_rng(11)
    T, E, k = 60, 12, 3
    x, idx = _inputs(rng, T, E, k)
    off = np.array([0, 25, 25, 60])
    d_w = (rng.standard_normal((T, k)) * 0.1).astype(np.float32)
    st = Step(x, idx, off, None, k, alpha=2.0, scale=1.5, d_loss=1.0, d_w=d_w).run()
    torch.cuda.synchronize()
    got = st.d_logits[:-1].double().cpu().numpy()

    def total(v):
        s = 1 / (1 + np.exp(-v))
        p = s / s.sum(1, keepdims=True)
        loss = 0.0
        for a, b in ((0, 25), (25, 60)):
            f = np.bincount(idx[a:b].reshape(-1), minlength=E)
            loss += 2.0 * E / (k * (b - a) ** 2 * 2) * (f * p[a:b].sum(0)).sum()
        si = np.take_along_axis(s, idx, 1)
        return loss + (d_w * 1.5 * si / si.sum(1, keepdims=True)).sum()

    x64, err = x.astype(np.float64), 0.0
    for t, e in zip(rng.integers(0, T, 80), rng.integers(0, E, 80)):
        up, dn = x64.copy(), x64.copy()
        up[t, e] += 1e-4
        dn[t, e] -= 1e-4
        err = max(err, abs((total(up) - total(dn)) / 2e-4 - got[t, e]))
    # the kernel's own error (2^-16 of a term's parts, below 1) comes on top
    assert err <= 1e-6 * np.abs(got).max() + 2.0 ** -16 * np.abs(got).max() * 4


@pytest.mark.parametrize("T,S", [(40, 2), (3000, 4)])
def test_graph_and_side_stream(T, S):
    rng = np.random.default_rng(T)
    x, idx = _inputs(rng, T, 64, 4)
    off = _cuts(rng, T, S)
    d_w = rng.standard_normal((T, 4)).astype(np.float32)
    st, eager = (Step(x, idx, off, None, 4, d_w=d_w) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    for i in range(4):
        v = torch.from_numpy(np.clip(rng.standard_normal((T, 64)), -8, 8).astype(np.float32)).cuda()
        st.x.copy_(v)
        eager.x.copy_(v)
        eager.run()
        st.d_logits[:-1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("counts", "prob", "coef", "loss", "d_logits"):
            assert torch.equal(getattr(st, name), getattr(eager, name)), name


def test_many_tokens():
    """More chunks of tokens than the partial sums' table has at its usual size, and a gradient past 16 tokens per wave:
    sums against fp64, the gradient at sampled tokens."""
    T, E, k = 300001, 8, 2
    rng = np.random.default_rng(4)
    x, idx = _inputs(rng, T, E, k)
    off = np.array([0, 1000, 299000, T])
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    st = Step(x, idx, off, None, k, d_w=d_w).run()
    torch.cuda.synchronize()
    s = 1 / (1 + np.exp(-x.astype(np.float64)))
    p = s / s.sum(1, keepdims=True)
    for q in range(3):
        a, b = off[q], off[q + 1]
        assert np.array_equal(st.counts[q].cpu().numpy(), np.bincount(idx[a:b].reshape(-1), minlength=E))
        want = p[a:b].sum(0)
        # fp32 sums in blocks: 128 tokens in a chunk, then its 16 chunk groups
        assert (np.abs(st.prob[q].double().cpu().numpy() - want) <= (2.0 ** -18 + 400 * 2.0 ** -24) * want).all()
    at = np.unique(np.concatenate([rng.integers(0, T, 300), [0, 999, 1000, 298999, 299000, T - 1]]))
    counts, coef = st.counts.cpu().numpy(), st.coef.double().cpu().numpy()
    got = st.d_logits.double().cpu().numpy()
    for t in at:
        q = int(np.searchsorted(off, t, side="right") - 1)
        c = coef[q] * counts[q]
        si = s[t, idx[t]]
        ds = (c - (c * p[t]).sum()) / s[t].sum()
        size = (np.abs(c) + (np.abs(c) * p[t]).sum()) / s[t].sum()
        np.add.at(ds, idx[t], (d_w[t] - (d_w[t] * si).sum() / si.sum()) / si.sum())
        np.add.at(size, idx[t], (np.abs(d_w[t]) + (np.abs(d_w[t]) * si).sum() / si.sum()) / si.sum())
        slope = s[t] * (1 - s[t])
        assert (np.abs(got[t] - ds * slope) <= 2.0 ** -16 * size * slope).all()


def test_with_the_router():
    """moe_route, the balance loss and the gradient together: the weights' term is that of moe_route's own weights."""
    T, H, E, k = 700, 512, 32, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    desc = moe.MoeLayerDesc.make(H, 128, E, k, 1, 2.5)
    xt = torch.randn((T, H), device="cuda", generator=gen).to(torch.bfloat16)
    wr = (torch.randn((E, H), device="cuda", generator=gen) * 0.04).to(torch.bfloat16)
    bias = torch.zeros(E, device="cuda")
    logits, w = torch.empty((T, E), device="cuda"), torch.empty((T, k), device="cuda")
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    moe.moe_route(desc, T, xt, wr, bias, logits, idx, w)
    d_w = torch.randn((T, k), device="cuda", generator=gen)
    x, ix = logits.cpu().numpy(), idx.cpu().numpy().astype(np.int64)
    assert np.abs(x).max() < 8
    st = Step(x, ix, np.array([0, 300, T]), None, k, scale=2.5, d_w=d_w.cpu().numpy()).run()
    _check(st, _reference(x, ix, np.array([0, 300, T]), None, k, 0.01, 2.5, 1.0, d_w.cpu().numpy()), T)
    v = logits.double().cpu().requires_grad_(True)
    s = torch.sigmoid(v).gather(1, idx.long().cpu())
    got_w = 2.5 * s / s.sum(1, keepdim=True)
    assert float((got_w.detach() - w.double().cpu()).abs().max()) < 1e-6


def test_binding_refusals():
    desc = moe.MoeLayerDesc.make(512, 128, 8, 2, 0)
    f, i = torch.zeros(4096, device="cuda"), torch.zeros(4096, dtype=torch.int32, device="cuda")
    ws = torch.zeros(moe.moe_balance_workspace_bytes(desc, 64, 2), dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeError):  # several sequences without their offsets
        moe.moe_balance_loss(desc, 64, 2, None, None, f, i, 0.01, i, f, f, f, ws)
    with pytest.raises(moe.MoeError):  # workspace
        moe.moe_balance_loss(desc, 64, 2, i, None, f, i, 0.01, i, f, f, f, ws[:64])
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(desc, 64, 2, i, None, f, i, float("nan"), i, f, f, f, ws)
    with pytest.raises(ValueError):    # mask type
        moe.moe_balance_loss(desc, 64, 2, i, i, f, i, 0.01, i, f, f, f, ws)
    with pytest.raises(ValueError):    # counts are needed with d_loss
        moe.moe_route_backward(desc, 64, 2, i, None, f, i, None, f, f, None, f)


def test_one_workspace_for_every_smaller_call():
    """A workspace sized for 8193 tokens and 9 sequences, allocated once, in turn through calls of other sizes, those with
    more partial sums among them."""
    say("balance, one workspace")
    rng = np.random.default_rng(13)
    E, k = 64, 3
    ws = None
    for T, S in ((8193, 9), (8192, 9), (2048, 2), (8193, 1), (100, 3), (4096, 8), (0, 9), (8000, 9)):
        x, idx = _inputs(rng, T, E, k)
        off = _cuts(rng, T, S)
        d_w = rng.standard_normal((T, k)).astype(np.float32)
        st = Step(x, idx, off, None, k, d_w=d_w)
        if ws is None:
            ws = st.ws
        st.ws = ws
        st.run()
        _check(st, _reference(x, idx, off, None, k, 0.01, 1.0, 1.0, d_w), T)


def _token_by_token(x, idx, k, alpha, d_loss, d_w):
    """_reference where every token is a sequence of its own, with the slope s (1 - s) as e / (1 + e)^2, e = exp(-|x|):
    1 - s is 0 in fp64 from x = 37 on."""
    T, E = x.shape
    counts, prob, coef, loss, _, _, n = _reference(x, idx, np.arange(T + 1), None, k, alpha, 1.0, d_loss, d_w)
    x = x.astype(np.float64)
    e = np.exp(-np.abs(x))
    s, slope = np.where(x < 0, e, 1.0) / (1 + e), e / (1 + e) ** 2
    ds, size = np.zeros_like(x), np.zeros_like(x)
    for t in range(T):
        if d_loss is not None:
            c = d_loss * coef[t] * counts[t]
            ds[t] = (c - (c * prob[t]).sum()) / s[t].sum()
            size[t] = (np.abs(c) + np.abs(c * prob[t]).sum()) / s[t].sum()
        si = s[t, idx[t]]
        ds[t, idx[t]] += (d_w[t] - (d_w[t] * si).sum() / si.sum()) / si.sum()
        size[t, idx[t]] += (np.abs(d_w[t]) + (np.abs(d_w[t]) * si).sum() / si.sum()) / si.sum()
    return counts, prob, coef, loss, ds * slope, size * slope, n


@pytest.mark.parametrize("T", [24, 300])
@pytest.mark.parametrize("low,high", [(-80.0, -20.0), (-80.0, 80.0), (-30.0, -8.0)])
def test_far_logits(T, low, high):
    """The bounds hold whatever the logits' size.  In units of 2^-23 a score is within 5 (exponential 1, its argument 2, the
    rest of that and the sum with 1 a half each, reciprocal 1), a probability within 17 (score 5, the sum's scores 5 and its
    ten levels a half each, reciprocal 1, product a half); the gradient's factors as before.  Every sequence is one token,
    so that no average hides an error; no probability is below 2^-126."""
    rng = np.random.default_rng(int(T + high))
    E, k = 256, 6
    x = rng.uniform(low, high, (T, E)).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    st = Step(x, idx, np.arange(T + 1), None, k, d_w=d_w).run()
    ref = _token_by_token(x, idx, k, 0.01, 1.0, d_w)
    _check(st, ref, 1)
    assert (np.abs(st.prob[:-1].double().cpu().numpy() - ref[1]) <= 17 * 2.0 ** -23 * ref[1]).all()
    one = Step(x[:6], idx[:6], np.arange(7), None, k, d_loss=None, d_w=d_w[:6]).run()  # the one-launch form
    _check(one, _token_by_token(x[:6], idx[:6], k, 0.01, None, d_w[:6]), 1)


def test_mask_of_truth_values():
    """A torch.bool mask, which comparisons give, is the uint8 mask of the same bytes; a strided one is refused as any."""
    rng = np.random.default_rng(17)
    T, E, k = 200, 24, 2
    x, idx = _inputs(rng, T, E, k)
    mask = (rng.random(T) >= 0.3).astype(np.uint8)
    off = np.array([0, 90, T])
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    want = Step(x, idx, off, mask, k, d_w=d_w).run()
    got = Step(x, idx, off, mask, k, d_w=d_w)
    got.mask = got.mask != 0
    assert got.mask.dtype is torch.bool
    got.run()
    _check(got, _reference(x, idx, off, mask, k, 0.01, 1.0, 1.0, d_w), T)
    assert torch.equal(got.d_logits, want.d_logits) and torch.equal(got.prob, want.prob)
    got.mask = (torch.zeros(2 * T, device="cuda") == 0)[::2]
    with pytest.raises(ValueError, match="token_mask must be contiguous"):
        got.run()
