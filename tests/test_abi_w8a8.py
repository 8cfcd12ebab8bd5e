"""Host-side argument checks of the W8A8 and router-balance entry points: each
returns its documented status before anything is enqueued (the pointers are
placeholders that are never dereferenced; no GPU is needed)."""
import ctypes

import pytest
import torch

import w4a16_routed_expert_moe_amd as moe
from w4a16_routed_expert_moe_amd import _lib

OK, NULL, SHAPE, UNSUP, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 7
P = ctypes.c_void_p
A, ODD = P(0x10000), P(0x10002)  # aligned, and not

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder-pointer checks run without a GPU")


def _desc(**kw):
    base = dict(hidden=4096, inter=2048, n_routed=256, top_k=6, n_shared=1, routed_scale=1.0)
    base.update(kw)
    return ctypes.byref(moe.MoeLayerDesc.make(**base))


def _call(name, args, **at):
    """The entry point on its valid placeholder arguments, some of them replaced (by position)."""
    args = list(args)
    for i, v in at.items():
        args[int(i[1:])] = v
    return getattr(_lib.lib(), name)(*args)


QUANT = (4, 4096, A, A, A, None)


@pytest.mark.parametrize("at,status", [
    (dict(_0=-1), SHAPE), (dict(_0=(1 << 20) * 9 + 1), SHAPE), (dict(_1=0), SHAPE), (dict(_1=40), SHAPE),
    (dict(_1=65552), SHAPE), (dict(_2=None), NULL), (dict(_3=None), NULL), (dict(_4=None), NULL),
    (dict(_2=ODD), ALIGN), (dict(_3=ODD), ALIGN), (dict(_4=ODD), ALIGN), (dict(_0=0, _2=None), OK),
])
def test_quant(at, status):
    assert _call("moe_act_quant_int8", QUANT, **at) == status


PACK = (2, 80, 400, A, P(0x10000000), None)


@pytest.mark.parametrize("at,status", [
    (dict(_0=0), SHAPE), (dict(_0=258), SHAPE), (dict(_1=72), SHAPE), (dict(_1=0), SHAPE), (dict(_2=8), SHAPE),
    (dict(_2=65552), SHAPE), (dict(_3=None), NULL), (dict(_4=None), NULL), (dict(_3=ODD), ALIGN), (dict(_4=ODD), ALIGN),
    (dict(_4=P(0x10000 + 2 * 80 * 400 - 16)), SHAPE), (dict(_3=P(0x10000000 + 2 * 128 * 512 - 16)), SHAPE),
])
def test_prepack(at, status):
    assert _call("moe_w8a8_prepack", PACK, **at) == status


def test_packed_bytes():
    f = moe.moe_w8a8_packed_bytes
    assert f(1, 16, 16) == 64 * 128 and f(1, 64, 128) == 64 * 128 and f(3, 80, 400) == 3 * 128 * 512
    assert f(257, 65536, 65536) == 257 << 32
    assert f(0, 64, 64) == f(1, 60, 64) == f(1, 64, 60) == f(1, 65552, 64) == f(258, 64, 64) == 0


GEMM = (4, 4096, 4096, A, A, A, A, A, None)


@pytest.mark.parametrize("at,status", [
    (dict(_0=-1), SHAPE), (dict(_0=(1 << 20) + 1), SHAPE), (dict(_1=100), SHAPE), (dict(_1=65552), SHAPE),
    (dict(_2=100), SHAPE), (dict(_2=0), SHAPE), (dict(_3=None), NULL), (dict(_4=None), NULL), (dict(_5=None), NULL),
    (dict(_6=None), NULL), (dict(_7=None), NULL), (dict(_3=ODD), ALIGN), (dict(_4=ODD), ALIGN), (dict(_5=ODD), ALIGN),
    (dict(_6=ODD), ALIGN), (dict(_7=ODD), ALIGN), (dict(_0=0, _3=None), OK),
])
def test_gemm(at, status):
    assert _call("moe_w8a8_gemm", GEMM, **at) == status


LINEAR = (4, 4096, 4096, A, A, A, A, A, A, None)


@pytest.mark.parametrize("at,status", [
    (dict(_0=-1), SHAPE), (dict(_1=24), SHAPE), (dict(_2=24), SHAPE), (dict(_0=0, _3=None), OK),
] + [({"_%d" % i: None}, NULL) for i in range(3, 9)] + [({"_%d" % i: ODD}, ALIGN) for i in range(3, 9)])
def test_linear(at, status):
    assert _call("moe_w8a8_linear", LINEAR, **at) == status


def _grouped(**kw):
    return (_desc(**kw), 4, A, A, A, 4, 4096, 4096, A, A, A, 1, A, None)


@pytest.mark.parametrize("at,status", [
    (dict(_1=-1), SHAPE), (dict(_5=0), SHAPE), (dict(_5=(1 << 20) + 1), SHAPE), (dict(_6=192), SHAPE),
    (dict(_6=24, _11=0), SHAPE), (dict(_7=24), SHAPE), (dict(_11=2), UNSUP), (dict(_1=0, _2=None), OK),
] + [({"_%d" % i: None}, NULL) for i in (2, 3, 8, 9, 10, 12)] + [({"_%d" % i: ODD}, ALIGN) for i in (2, 3, 4, 8, 9, 10, 12)])
def test_grouped(at, status):
    assert _call("moe_w8a8_grouped_gemm", _grouped(), **at) == status
    assert _call("moe_w8a8_grouped_gemm", _grouped(top_k=9)) == SHAPE
    assert _call("moe_w8a8_grouped_gemm", (None,) + _grouped()[1:]) == NULL


EXPERTS = (4,) + (A,) * 16 + (None,)


@pytest.mark.parametrize("at,status", [
    (dict(_1=-1), SHAPE), (dict(_1=(1 << 20) + 1), SHAPE), (dict(_1=0, _2=None), OK),
] + [({"_%d" % i: None}, NULL) for i in range(2, 18)] + [({"_%d" % i: ODD}, ALIGN) for i in range(2, 18)])
def test_experts(at, status):
    assert _call("moe_w8a8_experts", (_desc(),) + EXPERTS, **at) == status
    assert _call("moe_w8a8_experts", (_desc(hidden=300),) + EXPERTS) == SHAPE


LOSS = (64, 2, A, A, A, A, 0.01, A, A, A, A, A, 1 << 20, None)


@pytest.mark.parametrize("at,status", [
    (dict(_1=-1), SHAPE), (dict(_1=(1 << 20) + 1), SHAPE), (dict(_2=0), SHAPE), (dict(_2=(1 << 20) + 1), SHAPE),
    (dict(_3=None), NULL), (dict(_5=None), NULL), (dict(_6=None), NULL), (dict(_7=float("nan")), SHAPE),
    (dict(_7=float("inf")), SHAPE), (dict(_8=None), NULL), (dict(_9=None), NULL), (dict(_10=None), NULL),
    (dict(_11=None), NULL), (dict(_12=None), NULL), (dict(_13=64), WORKSPACE), (dict(_12=P(0x10004)), ALIGN),
] + [({"_%d" % i: ODD}, ALIGN) for i in (3, 5, 6, 8, 9, 10, 11)])
def test_balance_loss(at, status):
    assert _call("moe_balance_loss", (_desc(),) + LOSS, **at) == status
    assert _call("moe_balance_loss", (_desc(n_routed=300),) + LOSS) == SHAPE


def test_balance_workspace():
    f = moe.moe_balance_workspace_bytes
    d = moe.MoeLayerDesc.make(4096, 2048, 256, 6, 1)
    assert f(d, 0, 1) > 0 and f(d, -1, 1) == 0 and f(d, 5, 0) == 0 and f(d, (1 << 20) + 1, 1) == 0
    assert f(d, 1 << 20, 1) >= 512 * 256 * 8  # at most 512 chunks of partial sums


BACKWARD = (64, 2, A, A, A, A, A, A, A, A, A, None)


@pytest.mark.parametrize("at,status", [
    (dict(_1=-1), SHAPE), (dict(_2=0), SHAPE), (dict(_3=None), NULL), (dict(_5=None), NULL), (dict(_6=None), NULL),
    (dict(_7=None), NULL), (dict(_8=None), NULL), (dict(_11=None), NULL), (dict(_1=0, _5=None), OK),
] + [({"_%d" % i: ODD}, ALIGN) for i in (3, 5, 6, 7, 8, 9, 10, 11)])
def test_route_backward(at, status):
    assert _call("moe_route_backward", (_desc(),) + BACKWARD, **at) == status


def _partial_sums_bytes(T, n_seq, E, chunk):
    """The header, a double per sequence and 64 experts, and per chunk and sequence E sums, E counts and a token count."""
    rows = -(-T // chunk) + n_seq
    return 64 + 8 * n_seq * -(-E // 64) + rows * (8 * E + 4) + 4 * n_seq


def test_balance_workspace_serves_smaller_calls():
    """It never shrinks with more tokens or sequences (the tokens of a chunk, and with them the number of chunks, jump at
    powers of two), and it holds the partial sums of the smallest chunks that a call of that size takes."""
    f = moe.moe_balance_workspace_bytes
    edges = sorted({max(0, (1 << i) + j) for i in range(21) for j in (-129, -1, 0, 1, 2, 129)} | {3000, 12289, 50000})
    edges = [t for t in edges if t <= 1 << 20]
    for E in (1, 41, 256):
        d = moe.MoeLayerDesc.make(4096, 2048, E, 1, 0)
        for S in (1, 7, 65, 3000):
            sizes = [f(d, t, S) for t in edges]
            assert all(a <= b for a, b in zip(sizes, sizes[1:])), (E, S)
            assert all(f(d, t, S) <= f(d, t, S + 1) for t in edges), (E, S)
        for T, chunk in ((2048, 8), (4096, 16), (8192, 32), (16384, 64), (32768, 64), (65536, 128), (1 << 20, 128)):
            for S in (1, 65):
                assert f(d, T, S) >= _partial_sums_bytes(T, S, E, chunk), (E, T, S)


def test_balance_workspace_of_another_call_is_accepted():
    """A call refuses a workspace only where its own partial sums do not fit.  (That of T + 1 tokens was smaller than
    that of T past 2048, 4096 and 8192 tokens.)"""
    d = moe.MoeLayerDesc.make(4096, 2048, 256, 6, 1)
    for T in (2048, 4096, 8192, 32768):
        least = _partial_sums_bytes(T, 2, 256, 8 * max(1, T // 2048) if T <= 16384 else 64)
        args = (ctypes.byref(d), T) + LOSS[1:]
        assert _call("moe_balance_loss", args, _13=least - 1) == WORKSPACE
        assert moe.moe_balance_workspace_bytes(d, T + 1, 2) >= least
