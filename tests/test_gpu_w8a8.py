"""GPU parity of the W8A8 calls (INT8 weights with a scale per output channel,
activations quantised to INT8 per token) against plain 64-bit arithmetic.

What is decided by the definition is compared bit for bit: codes and scales of
the quantisation (integer arithmetic on the host), the exact integer sums, and
the two fp32 multiplications and the bf16 rounding of an output without an
activation.  The SwiGLU output is compared with fp64: its value passes through
the hardware exponential and reciprocal (a few units of 2^-23) and is rounded
to bf16 (2^-8 of its size at most), hence 2^-8 + 2^-18.  The one-call forms
are compared bit for bit with the calls that they stand for."""
import numpy as np
import pytest
import torch

import w4a16_routed_expert_moe_amd as moe
from gpu_common import Case, bf16_to_np_bits, say, to_dev_bf16

pytestmark = pytest.mark.gpu

SWIGLU_TOL = 2.0 ** -8 + 2.0 ** -18


def _bits(x32):
    """fp32 array -> bf16 bits, round to nearest even."""
    return torch.from_numpy(np.ascontiguousarray(x32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _f32(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def _quant_ref(bits):
    """Codes and scales of bf16 rows, the quotients compared as integers."""
    x = _f32(bits).astype(np.float64)
    codes = np.zeros(x.shape, np.int64)
    scales = np.zeros(x.shape[0], np.float32)
    for r in range(x.shape[0]):
        if not np.isfinite(x[r]).all():
            scales[r] = np.nan
            continue
        amax = np.abs(x[r]).max()
        scales[r] = np.float32(amax) / np.float32(127)
        if amax == 0:
            continue
        v = 127.0 * np.abs(x[r])           # 15 significant bits: exact
        n = np.floor(v / amax)             # off by one at most: settled below
        n -= n * amax > v                  # (products of 7 and 8 bits, exact)
        n += (n + 1) * amax <= v
        twice = 2.0 * (v - n * amax)       # exact: against a half
        n += (twice > amax) | ((twice == amax) & (n % 2 == 1))
        codes[r] = np.where(x[r] < 0, -n, n).astype(np.int64)
    return codes.astype(np.int8), scales


def _rows(rng, rows, K, spread=1.0):
    mag = np.exp(rng.uniform(-np.log(spread), np.log(spread), (rows, 1))) if spread > 1 else 1.0
    return _bits((rng.standard_normal((rows, K)) * mag).astype(np.float32))


def _quantise(bits):
    rows, K = bits.shape
    codes = torch.full((rows, K), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((rows,), 7.0, dtype=torch.float32, device="cuda")
    moe.moe_act_quant_int8(rows, K, to_dev_bf16(bits), codes, scales)
    return codes, scales


@pytest.mark.parametrize("rows,K,spread", [
    (1, 16, 1.0), (3, 48, 1.0), (37, 400, 1e3), (300, 4096, 1.0), (5, 2048, 1e30), (9, 8208, 1.0), (2, 65536, 1.0),
    (2051, 2064, 10.0), (2050, 512, 1.0), (2049, 4096, 1e4),
])
def test_quant_bit_exact(rows, K, spread):
    say("quant %dx%d" % (rows, K))
    rng = np.random.default_rng(rows * 7 + K)
    x = _rows(rng, rows, K, spread)
    if rows > 2:
        x[1] = 0                                                            # a row of zeros
        x[1, 3] = 0x8000
        x[rows - 1] = (np.arange(K) % 128).astype(np.uint16) | 0x8000       # a row of subnormals
        x[2] = _bits(((np.arange(K) % 255) - 127).astype(np.float32) * 1.0)
        x[2, 0] = _bits(np.float32([254.0]))[0]                             # every odd value is a tie
    if rows > 8:
        x[5] = np.where(np.arange(K) % 2, 0x7F7F, 0xFF7F).astype(np.uint16)  # the largest finite bf16
        x[6, K // 2] = 0x7F80                                               # an infinity
        x[7, K - 1] = 0x7FC1                                                # a NaN
        x[8] = 0
        x[8, 5] = 0x0001                                                    # only the smallest subnormal
    codes, scales = _quantise(x)
    torch.cuda.synchronize()
    rc, rs = _quant_ref(x)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32)[~np.isnan(rs)], rs.view(np.uint32)[~np.isnan(rs)])
    assert np.array_equal(np.isnan(scales.cpu().numpy()), np.isnan(rs))
    assert np.array_equal(codes.cpu().numpy(), rc)


def test_quant_every_quotient():
    """Every bf16 mantissa against every maximum's, over the exponents whose codes are not all zero."""
    top = _f32((0x3F80 + np.arange(128)).astype(np.uint16))
    x = np.concatenate([_f32(((127 - d) * 128 + np.arange(128)).astype(np.uint16)) for d in range(0, 9)])
    rows = np.zeros((128, 16 * ((x.size + 16) // 16)), np.float32)
    rows[:, 1:x.size + 1] = x
    rows = np.where(rows > top[:, None], 0.0, rows).astype(np.float32)
    rows[:, 0] = -top
    bits = _bits(rows)
    codes, scales = _quantise(bits)
    torch.cuda.synchronize()
    rc, rs = _quant_ref(bits)
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)


def _packed_ref(w):
    G, N, K = w.shape
    NT, KB = 4 * -(-N // 64), 2 * -(-K // 128)
    full = np.zeros((G, NT * 16, KB * 64), np.int8)
    full[:, :N, :K] = w
    out = np.zeros((G, NT, KB, 64, 16), np.int8)
    for t in range(NT):
        for lane in range(64):
            n = 64 * (t // 4) + 16 * ((lane % 16) // 4) + 4 * (t % 4) + lane % 4
            out[:, t, :, lane] = full[:, n].reshape(G, KB, 4, 16)[:, :, lane // 16]
    return out.reshape(-1)


def _pack(w):
    G, N, K = w.shape
    out = torch.full((moe.moe_w8a8_packed_bytes(G, N, K),), 55, dtype=torch.int8, device="cuda")
    moe.moe_w8a8_prepack(G, N, K, torch.from_numpy(w).cuda(), out)
    return out


@pytest.mark.parametrize("G,N,K", [(1, 16, 16), (1, 64, 128), (3, 80, 400), (2, 272, 144)])
def test_prepack_layout(G, N, K):
    rng = np.random.default_rng(N)
    w = rng.integers(-128, 128, (G, N, K), dtype=np.int8)
    got = _pack(w)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), _packed_ref(w))


def test_layout_and_quantisation_past_32_bit_threads():
    """Sizes whose pieces, and whose rows times 1024 threads, pass 2^32 in one call."""
    G, N, K = 9, 65536, 65536
    rng = np.random.default_rng(11)
    w = torch.zeros((G, N, K), dtype=torch.int8, device="cuda")
    at = [(0, 64, 128), (3, N - 64, 0), (7, N - 64, K - 128), (8, 0, 0), (8, N - 64, K - 128)]
    parts = [rng.integers(-128, 128, (1, 64, 128), dtype=np.int8) for _ in at]
    for (g, n, k), part in zip(at, parts):
        w[g, n:n + 64, k:k + 128] = torch.from_numpy(part[0]).cuda()
    out = torch.empty(moe.moe_w8a8_packed_bytes(G, N, K), dtype=torch.int8, device="cuda")
    moe.moe_w8a8_prepack(G, N, K, w, out)
    blocks = out.view(G, N // 16, K // 64, 1024)
    for (g, n, k), part in zip(at, parts):
        got = blocks[g, n // 16:n // 16 + 4, k // 64:k // 64 + 2].cpu().numpy()
        assert np.array_equal(got.reshape(-1), _packed_ref(part)), (g, n, k)
    del w, out, blocks
    torch.cuda.empty_cache()
    rows, K = (1 << 22) + 3, 16400
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    at = [0, (1 << 21) - 1, 1 << 21, rows - 4, rows - 1]
    part = _rows(rng, len(at), K, 10.0)
    for i, r in enumerate(at):
        x[r] = to_dev_bf16(part[i:i + 1])[0]
    codes = torch.empty((rows, K), dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, device="cuda")
    moe.moe_act_quant_int8(rows, K, x, codes, scales)
    torch.cuda.synchronize()
    rc, rs = _quant_ref(part)
    assert np.array_equal(codes[at].cpu().numpy(), rc) and np.array_equal(scales[at].cpu().numpy(), rs)
    assert int((scales != 0).sum()) == len(at)
    del x, codes
    torch.cuda.empty_cache()


def _int_product(a, w):
    """int64 sums of int8 codes (fp64 holds every partial sum exactly)."""
    return (a.astype(np.float64) @ w.astype(np.float64).T).astype(np.int64)


def _scaled(acc, sa, sw):
    """The kernels' epilogue in the same fp32 operations."""
    return _bits(acc.astype(np.float32) * sa[:, None] * sw[None, :])


# one and several m-tiles of every kernel, ragged N and K, K of a single and of many blocks
@pytest.mark.parametrize("M", [1, 15, 16, 17, 33, 64, 65, 97, 128, 130, 300])
@pytest.mark.parametrize("N,K", [(16, 16), (64, 64), (80, 80), (272, 400), (1040, 2064), (528, 8192)])
def test_gemm_bit_exact(M, N, K):
    say("gemm %d %d %d" % (M, N, K))
    rng = np.random.default_rng(M * 1000 + N + K)
    a = rng.integers(-127, 128, (M, K), dtype=np.int8)
    w = rng.integers(-128, 128, (N, K), dtype=np.int8)
    sa = rng.uniform(0.001, 0.02, M).astype(np.float32)
    sw = rng.uniform(0.0001, 0.01, N).astype(np.float32)
    out = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_w8a8_gemm(M, N, K, torch.from_numpy(a).cuda(), torch.from_numpy(sa).cuda(), _pack(w[None]),
                      torch.from_numpy(sw).cuda(), out)
    torch.cuda.synchronize()
    assert np.array_equal(bf16_to_np_bits(out[:M]), _scaled(_int_product(a, w), sa, sw))
    assert (out[M:] == 7.0).all()  # rows behind the last one: as they were


# wide enough outputs that the rows choose each of the tiles: 32 x 64, 32 x 128, 64 x 128, 64 x 256, 128 x 256
@pytest.mark.parametrize("M", [40, 200, 300, 640, 1100, 1500])
@pytest.mark.parametrize("N,K", [(4096, 16), (4096, 400), (4112, 640)])
def test_gemm_every_tile(M, N, K):
    test_gemm_bit_exact(M, N, K)


@pytest.mark.parametrize("M", [1, 40, 200])
def test_gemm_extreme_codes(M):
    """The largest sums: 65536 products of -128 and -128 (2^30)."""
    N, K = 32, 65536
    a = np.full((M, K), -128, np.int8)
    w = np.full((N, K), -128, np.int8)
    w[1::2] = 127
    one = np.ones(M, np.float32)
    sw = np.ones(N, np.float32)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_w8a8_gemm(M, N, K, torch.from_numpy(a).cuda(), torch.from_numpy(one).cuda(), _pack(w[None]),
                      torch.from_numpy(sw).cuda(), out)
    torch.cuda.synchronize()
    want = np.where(np.arange(N) % 2, -128 * 127 * K, 128 * 128 * K)
    assert np.array_equal(bf16_to_np_bits(out), _scaled(np.broadcast_to(want, (M, N)), one, sw))


def test_gemm_past_32_bit_offsets():
    """Rows of a beyond 2^32 bytes and outputs on both sides of that row."""
    M, N, K = (1 << 19) + 40, 16, 8208
    a = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    rng = np.random.default_rng(3)
    rows = [0, 1, (1 << 32) // K - 1, (1 << 32) // K, (1 << 32) // K + 1, M - 129, M - 2, M - 1]
    part = rng.integers(-127, 128, (len(rows), K), dtype=np.int8)
    a[rows] = torch.from_numpy(part).cuda()
    w = rng.integers(-128, 128, (N, K), dtype=np.int8)
    sw = rng.uniform(0.001, 0.01, N).astype(np.float32)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_w8a8_gemm(M, N, K, a, torch.ones(M, device="cuda"), _pack(w[None]), torch.from_numpy(sw).cuda(), out)
    torch.cuda.synchronize()
    got = bf16_to_np_bits(out[rows])
    assert np.array_equal(got, _scaled(_int_product(part, w), np.ones(len(rows), np.float32), sw))
    assert int((out != 0).any(1).sum()) == len(rows)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (5, 208, 144), (16, 512, 2064), (16, 64, 4096), (16, 64, 4112),
                                   (17, 64, 256), (61, 208, 2064), (150, 640, 1024), (2100, 128, 512)])
def test_linear_is_quantise_then_product(M, N, K):
    rng = np.random.default_rng(M + N + K)
    x = _rows(rng, M, K, 30.0)
    if M > 3:
        x[1] = 0
        x[2, 7] = 0x7F80  # its products are NaN, the other rows' are not
    w = rng.integers(-127, 128, (N, K), dtype=np.int8)
    wp, sw = _pack(w[None]), torch.from_numpy(rng.uniform(0.001, 0.02, N).astype(np.float32)).cuda()
    codes, scales = _quantise(x)
    want = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_w8a8_gemm(M, N, K, codes, scales, wp, sw, want)
    got = torch.full((M + 1, N), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_w8a8_linear(M, N, K, to_dev_bf16(x), wp, sw, torch.empty_like(codes), torch.empty_like(scales), got)
    torch.cuda.synchronize()
    assert torch.equal(got[:M].view(torch.int16), want.view(torch.int16)) or torch.equal(
        torch.nan_to_num(got[:M].float()), torch.nan_to_num(want.float()))
    assert torch.equal(torch.isnan(got[:M]), torch.isnan(want)) and (got[M] == 3.0).all()
    if M > 3:
        assert torch.isnan(got[2]).all() and not torch.isnan(got[[0, 1, 3]]).any() and (got[1] == 0).all()


@pytest.mark.parametrize("N,K", [(208, 16), (80, 512), (1024, 528), (80, 1024), (272, 1040), (80, 2048), (80, 2064),
                                 (80, 4096), (9216, 512), (9216, 1024), (9216, 2048)])
def test_linear_of_few_rows(N, K):
    """Every row count of the one-launch products (a row is quantised by one to eight waves) and those past them."""
    rng = np.random.default_rng(N + K)
    x = _rows(rng, 17, K, 30.0)
    x[3] = 0
    w = rng.integers(-128, 128, (N, K), dtype=np.int8)
    wp, sw = _pack(w[None]), torch.from_numpy(rng.uniform(0.001, 0.02, N).astype(np.float32)).cuda()
    codes, scales = _quantise(x)
    want = torch.empty((17, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_w8a8_gemm(17, N, K, codes, scales, wp, sw, want)
    xd = to_dev_bf16(x)
    for M in range(1, 18):
        got = torch.full((M + 1, N), 3.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_w8a8_linear(M, N, K, xd, wp, sw, torch.empty_like(codes), torch.empty_like(scales), got)
        torch.cuda.synchronize()
        assert torch.equal(got[:M].view(torch.int16), want[:M].view(torch.int16)) and (got[M] == 3.0).all(), M


@pytest.mark.parametrize("T", [5, 6, 7, 9, 12, 13, 16, 17])
@pytest.mark.parametrize("H,I,E,k,ns", [(1024, 512, 16, 4, 1), (512, 128, 16, 1, 0), (4096, 128, 12, 2, 1), (512, 1024, 1, 1, 1)])
def test_experts_of_few_tokens(T, H, I, E, k, ns):
    """moe_w8a8_experts of small experts gives the bits of its parts at the token counts around its one-launch products."""
    case, layer, _ = _experts_case(T, H, I, E, k, ns, T + H)
    buf = moe.Buffers(case.desc, T, int8=True)
    layer.forward(case.xd, buf)
    d, w, R = case.desc, layer.experts, case.desc.rows(T)
    o = moe.Buffers(d, T, int8=True)
    moe.moe_act_quant_int8(T, H, case.xd, o.xq8, o.xqs8)
    moe.moe_w8a8_grouped_gemm(d, T, o.xq8, o.xqs8, buf.sorted_token, T, 2 * I, H, w.w13, w.s13, buf.group_offsets,
                              moe.MOE_ACT_SWIGLU, o.h)
    moe.moe_act_quant_int8(R, I, o.h, o.hq8, o.hqs8)
    moe.moe_w8a8_grouped_gemm(d, T, o.hq8, o.hqs8, None, 0, H, I, w.w2, w.s2, buf.group_offsets, moe.MOE_ACT_NONE, o.y)
    moe.moe_combine(d, T, o.y, buf.row_of_slot, buf.topk_w, o.out)
    torch.cuda.synchronize()
    for name in ("h", "y", "out"):
        assert torch.equal(getattr(o, name).view(torch.int16), getattr(buf, name).view(torch.int16)), name


def _groups(rng, G, R, empty):
    cut = np.sort(rng.integers(0, R + 1, G - 1))
    off = np.concatenate([[0], cut, [R]]).astype(np.int32)
    if empty and G > 2:
        off[2] = off[1]
    return off


# groups of one to hundreds of rows, empty ones among them; T picks the kernel
@pytest.mark.parametrize("T,E,k,ns,N,K,gather", [
    (1, 8, 2, 1, 256, 512, True), (7, 16, 4, 0, 128, 80, True), (16, 8, 8, 1, 384, 1040, False),
    (40, 12, 3, 1, 256, 256, True), (64, 5, 2, 1, 512, 144, False), (65, 6, 2, 1, 640, 400, True),
    (200, 3, 2, 1, 1152, 512, True), (421, 40, 3, 1, 1024, 1024, True), (500, 200, 6, 0, 128, 128, True),
    (700, 1, 1, 1, 1024, 2064, False),
    (300, 1, 1, 1, 256, 272, True), (1200, 1, 1, 1, 1024, 400, True), (2500, 1, 1, 1, 2048, 144, True),
    (2500, 3, 2, 1, 1024, 80, False), (900, 4, 2, 0, 4096, 48, True),
])
@pytest.mark.parametrize("act", [moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU])
def test_grouped_every_element(T, E, k, ns, N, K, gather, act):
    say("grouped T=%d E=%d N=%d K=%d act=%d" % (T, E, N, K, act))
    rng = np.random.default_rng(T + N)
    desc = moe.MoeLayerDesc.make(512, 128, E, k, ns)
    G, R = E + ns, T * (k + ns)
    n_src = T if gather else R
    off = _groups(rng, G, R, True)
    a = rng.integers(-127, 128, (n_src, K), dtype=np.int8)
    sa = rng.uniform(0.002, 0.02, n_src).astype(np.float32)
    idx = rng.integers(0, T, R).astype(np.int32)
    if gather and R > 4:
        idx[[1, R - 2]] = [-1, T]  # no such row: zeros
    w = rng.integers(-128, 128, (G, N, K), dtype=np.int8)
    sw = rng.uniform(0.0005, 0.005, (G, N)).astype(np.float32)
    cols = N // 2 if act == moe.MOE_ACT_SWIGLU else N
    out = torch.full((R + 2, cols), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_w8a8_grouped_gemm(desc, T, torch.from_numpy(a).cuda(), torch.from_numpy(sa).cuda(),
                              torch.from_numpy(idx).cuda() if gather else None, n_src if gather else 0, N, K, _pack(w),
                              torch.from_numpy(sw).cuda(), torch.from_numpy(off).cuda(), act, out)
    torch.cuda.synchronize()
    assert (out[R:] == 9.0).all()
    src = idx if gather else np.arange(R, dtype=np.int32)
    ok = (src >= 0) & (src < n_src)
    ar = np.where(ok[:, None], a[np.clip(src, 0, n_src - 1)], 0)
    sr = sa[np.clip(src, 0, n_src - 1)]
    got = bf16_to_np_bits(out[:R])
    for g in range(G):
        lo, hi = off[g], off[g + 1]
        if lo == hi:
            continue
        acc = _int_product(ar[lo:hi], w[g])
        if act == moe.MOE_ACT_NONE:
            assert np.array_equal(_f32(got[lo:hi]), _f32(_scaled(acc, sr[lo:hi], sw[g])))
            continue
        v = acc * sr[lo:hi, None].astype(np.float64) * sw[g].astype(np.float64)
        gate, up = v[:, :cols], v[:, cols:]
        ref = gate / (1 + np.exp(-gate)) * up
        assert (np.abs(_f32(got[lo:hi]) - ref) <= SWIGLU_TOL * np.abs(ref) + 1e-30).all()
    assert not got[:R][~ok].any()


def _experts_case(T, H, I, E, k, ns, seed):
    rng = np.random.default_rng(seed)
    G = E + ns
    w13 = rng.integers(-127, 128, (G, 2 * I, H), dtype=np.int8)
    w2 = rng.integers(-127, 128, (G, H, I), dtype=np.int8)
    s13 = rng.uniform(0.5, 1.5, (G, 2 * I)).astype(np.float32) / np.float32(74 * np.sqrt(H))
    s2 = rng.uniform(0.5, 1.5, (G, H)).astype(np.float32) / np.float32(74 * np.sqrt(I))
    case = Case("shape", T=T, H=H, E=E, k=k, I=I, n_shared=ns, seed=seed)
    experts = moe.upload_weights(w13, s13, w2, s2, fmt="int8")
    layer = moe.MoELayer(case.desc, case.layer_obj.w_router, case.layer_obj.gate_bias, experts)
    return case, layer, (w13, s13, w2, s2)


@pytest.mark.parametrize("T,H,I,E,k,ns", [
    (1, 512, 256, 8, 2, 1), (1, 2048, 512, 16, 4, 0), (1, 512, 128, 1, 1, 0), (2, 512, 4096, 8, 8, 0),
    (2, 1024, 512, 20, 6, 1), (4, 512, 256, 8, 2, 1), (4, 4096, 128, 12, 3, 1), (4, 512, 2048, 9, 8, 1), (9, 1024, 384, 12, 3, 1), (16, 512, 128, 4, 4, 1),
    (17, 512, 256, 8, 2, 1), (64, 1024, 512, 10, 3, 1), (90, 512, 256, 6, 2, 0), (421, 1024, 512, 40, 3, 1),
])
def test_layer_stage_by_stage(T, H, I, E, k, ns):
    """The layer with INT8 experts: routing as moe_route_permute alone gives it,
    h against fp64, y bit for bit from the layer's own h, out against fp64 from
    its own y (k + 1 products and sums in fp32 and one rounding: 2^-8 of the
    result plus (k + 2) 2^-24 of the sum of the terms' sizes)."""
    case, layer, (w13, s13, w2, s2) = _experts_case(T, H, I, E, k, ns, T + E)
    buf = moe.Buffers(case.desc, T, int8=True)
    layer.forward(case.xd, buf)
    d = case.desc
    ref = moe.Buffers(d, T)
    moe.moe_route_permute(d, T, case.xd, layer.w_router, layer.gate_bias, ref.logits, ref.topk_idx, ref.topk_w,
                          ref.group_offsets, ref.sorted_token, ref.row_of_slot, ref.ws)
    torch.cuda.synchronize()
    for name in ("logits", "topk_idx", "topk_w", "group_offsets", "sorted_token", "row_of_slot"):
        assert torch.equal(getattr(buf, name), getattr(ref, name)), name
    off, tok = buf.group_offsets.cpu().numpy(), buf.sorted_token.cpu().numpy()
    h, y = bf16_to_np_bits(buf.h), bf16_to_np_bits(buf.y)
    xc, xs = _quant_ref(case.x)
    hc, hs = _quant_ref(h)
    for g in range(E + ns):
        lo, hi = off[g], off[g + 1]
        if lo == hi:
            continue
        v = _int_product(xc[tok[lo:hi]], w13[g]) * xs[tok[lo:hi], None].astype(np.float64) * s13[g].astype(np.float64)
        want = v[:, :I] / (1 + np.exp(-v[:, :I])) * v[:, I:]
        assert (np.abs(_f32(h[lo:hi]) - want) <= SWIGLU_TOL * np.abs(want) + 1e-30).all()
        assert np.array_equal(_f32(y[lo:hi]), _f32(_scaled(_int_product(hc[lo:hi], w2[g]), hs[lo:hi], s2[g])))
    wt = np.concatenate([buf.topk_w.cpu().numpy(), np.ones((T, ns), np.float32)], 1).astype(np.float64)
    terms = wt[:, :, None] * _f32(y)[buf.row_of_slot.cpu().numpy()].astype(np.float64)
    want = terms.sum(1)
    bound = 2.0 ** -8 * np.abs(want) + (k + 2) * 2.0 ** -24 * np.abs(terms).sum(1) * 2
    assert (np.abs(_f32(bf16_to_np_bits(buf.out)) - want) <= bound).all()


@pytest.mark.parametrize("T", [1, 3, 600, 3000])
def test_full_size_layer(T):
    """The layer at hidden 4096, inter 2048, 256 experts, 6 per token: sampled rows of h, y and out from the codes."""
    H, I, E, k = 4096, 2048, 256, 6
    case = Case("shape", T=T, H=H, E=E, k=k, I=I, n_shared=1, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    G = E + 1
    w13 = torch.empty((G, 2 * I, H), dtype=torch.int8, device="cuda")
    w2 = torch.empty((G, H, I), dtype=torch.int8, device="cuda")
    for g in range(G):
        w13[g] = torch.randint(-127, 128, (2 * I, H), device="cuda", generator=gen, dtype=torch.int8)
        w2[g] = torch.randint(-127, 128, (H, I), device="cuda", generator=gen, dtype=torch.int8)
    s13 = (torch.rand((G, 2 * I), device="cuda", generator=gen) + 0.5) / (74 * 64)
    s2 = (torch.rand((G, H), device="cuda", generator=gen) + 0.5) / (74 * 45)
    experts = moe.ExpertWeights(w13=moe.prepack(w13, G, 2 * I, H, fmt="int8"), s13=s13,
                                w2=moe.prepack(w2, G, H, I, fmt="int8"), s2=s2, fmt="int8")
    layer = moe.MoELayer(case.desc, case.layer_obj.w_router, case.layer_obj.gate_bias, experts)
    buf = moe.Buffers(case.desc, T, int8=True)
    layer.forward(case.xd, buf)
    torch.cuda.synchronize()
    off, tok = buf.group_offsets.cpu().numpy(), buf.sorted_token.cpu().numpy()
    R = case.desc.rows(T)
    rows = np.unique(np.concatenate([np.arange(min(R, 6)), [R - 1, R - T], np.random.default_rng(T).integers(0, R, 40)]))
    h, y = bf16_to_np_bits(buf.h[rows]), bf16_to_np_bits(buf.y[rows])
    xc, xs = _quant_ref(case.x[tok[rows]])
    hc, hs = _quant_ref(h)
    for i, r in enumerate(rows):
        g = int(np.searchsorted(off, r, side="right") - 1)
        v = _int_product(xc[i:i + 1], w13[g].cpu().numpy())[0] * float(xs[i]) * s13[g].double().cpu().numpy()
        want = v[:I] / (1 + np.exp(-v[:I])) * v[I:]
        assert (np.abs(_f32(h[i]) - want) <= SWIGLU_TOL * np.abs(want) + 1e-30).all()
        acc = _int_product(hc[i:i + 1], w2[g].cpu().numpy())
        assert np.array_equal(_f32(y[i:i + 1]), _f32(_scaled(acc, hs[i:i + 1], s2[g].cpu().numpy())))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 8, 40, 200])
def test_experts_call_is_its_parts(T):
    """moe_w8a8_experts gives the bits of quantise, product, quantise, product, combine."""
    case, layer, _ = _experts_case(T, 1024, 512, 16, 4, 1, 5)
    buf = moe.Buffers(case.desc, T, int8=True)
    layer.forward(case.xd, buf)
    d, w, R = case.desc, layer.experts, case.desc.rows(T)
    o = moe.Buffers(d, T, int8=True)
    moe.moe_act_quant_int8(T, d.hidden, case.xd, o.xq8, o.xqs8)
    moe.moe_w8a8_grouped_gemm(d, T, o.xq8, o.xqs8, buf.sorted_token, T, 2 * d.inter, d.hidden, w.w13, w.s13,
                              buf.group_offsets, moe.MOE_ACT_SWIGLU, o.h)
    moe.moe_act_quant_int8(R, d.inter, o.h, o.hq8, o.hqs8)
    moe.moe_w8a8_grouped_gemm(d, T, o.hq8, o.hqs8, None, 0, d.hidden, d.inter, w.w2, w.s2, buf.group_offsets,
                              moe.MOE_ACT_NONE, o.y)
    moe.moe_combine(d, T, o.y, buf.row_of_slot, buf.topk_w, o.out)
    torch.cuda.synchronize()
    for name in ("h", "y", "out"):
        assert torch.equal(getattr(o, name).view(torch.int16), getattr(buf, name).view(torch.int16)), name


def test_quantised_weights_layer():
    """bf16 expert weights through quantize_weights_int8: the layer stays near the same layer in fp64 without
    quantisation (each of the four roundings to 1/254 of a row's maximum, at most 3.5 standard deviations here, adds
    noise of 3.5 / 254 / sqrt(3) of the signal: 1.6% for the four together; 4% is over twice that)."""
    T, H, I, E, k = 30, 512, 256, 8, 2
    case = Case("shape", T=T, H=H, E=E, k=k, I=I, n_shared=1, seed=2)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    w13 = torch.randn((E + 1, 2 * I, H), device="cuda", generator=gen).to(torch.bfloat16)
    w2 = torch.randn((E + 1, H, I), device="cuda", generator=gen).to(torch.bfloat16)
    layer = moe.MoELayer(case.desc, case.layer_obj.w_router, case.layer_obj.gate_bias,
                         moe.quantize_weights_int8(w13, w2))
    buf = moe.Buffers(case.desc, T, int8=True)
    out = layer.forward(case.xd, buf).double().cpu()
    x, a, b = case.xd.double().cpu(), w13.double().cpu(), w2.double().cpu()
    idx, wt = buf.topk_idx.long().cpu(), buf.topk_w.double().cpu()
    want = torch.zeros_like(out)
    for t in range(T):
        for j in range(k + 1):
            e = int(idx[t, j]) if j < k else E
            v = a[e] @ x[t]
            want[t] += (wt[t, j] if j < k else 1.0) * (b[e] @ (v[:I] * torch.sigmoid(v[:I]) * v[I:]))
    err = float((out - want).norm() / want.norm())
    say("  relative 2-norm against the layer without quantisation: %.4f" % err)
    assert err < 0.04


@pytest.mark.parametrize("T", [1, 200])
def test_graph_and_side_stream(T):
    """Captured once, replayed on new inputs with eager work between, each replay against the eager result; and the
    same calls on another stream."""
    case, layer, _ = _experts_case(T, 1024, 256, 8, 2, 1, 9)
    eager, buf = moe.Buffers(case.desc, T, int8=True), moe.Buffers(case.desc, T, int8=True)
    x = case.xd.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer.forward(x, buf)
    side.synchronize()
    layer.forward(x, eager)
    torch.cuda.synchronize()
    assert torch.equal(buf.out, eager.out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, buf)
    for i in range(4):
        x.copy_(case.xd * (0.5 + i) if i % 2 else case.xd.flip(1))
        layer.forward(x, eager)
        buf.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf.out, eager.out)
        assert float(buf.out.float().abs().max()) > 0


def test_binding_refusals(monkeypatch):
    desc = moe.MoeLayerDesc.make(512, 128, 4, 2, 1)
    i8, f, b = (torch.zeros(1 << 17, dtype=t, device="cuda") for t in (torch.int8, torch.float32, torch.bfloat16))
    with pytest.raises(ValueError):
        moe.moe_act_quant_int8(4, 64, b.float(), i8, f)                   # type
    with pytest.raises(ValueError):
        moe.moe_act_quant_int8(1 << 13, 64, b, i8, f)                     # too small
    with pytest.raises(moe.MoeError):
        moe.moe_act_quant_int8(4, 40, b, i8, f)                           # K
    with pytest.raises(moe.MoeError):
        moe.moe_w8a8_gemm(4, 40, 64, i8, f, i8, f, b)                     # N
    with pytest.raises(moe.MoeError):
        moe.moe_w8a8_gemm(4, 64, 64, i8[1:], f, i8, f, b)                 # alignment
    with pytest.raises(ValueError):
        moe.moe_w8a8_gemm(4, 64, 64, i8, f, i8.cpu(), f, b)               # host memory
    with pytest.raises(moe.MoeError):
        moe.moe_w8a8_grouped_gemm(desc, 4, i8, f, None, 0, 192, 64, i8, f,
                                  torch.zeros(6, dtype=torch.int32, device="cuda"), moe.MOE_ACT_SWIGLU, b)
    moe.moe_w8a8_gemm(0, 64, 64, i8, f, i8, f, b)                         # nothing to do
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        moe.moe_w8a8_gemm(4, 64, 64, i8, f, i8, f, b)                     # tensors of another device
    monkeypatch.undo()
    with pytest.raises(ValueError):
        layer = moe.MoELayer(desc, b, f, moe.ExpertWeights(i8, f, i8, f, fmt="int8"))
        layer.forward(b, moe.Buffers(desc, 4))


def test_every_tensor_is_on_the_current_device():
    """Each tensor of each call, one at a time, on another device than the rest: refused."""
    class Away(torch.Tensor):
        def get_device(self):
            return 1

    n = 1 << 18
    t = {k: torch.zeros(n, dtype=v, device="cuda") for k, v in
         dict(b=torch.bfloat16, f=torch.float32, i=torch.int32, c=torch.int8, u=torch.uint8).items()}
    desc = moe.MoeLayerDesc.make(128, 128, 4, 2, 1)
    for fn, args in ((moe.moe_act_quant_int8, [4, 64, "b", "c", "f"]),
                     (moe.moe_w8a8_prepack, [1, 64, 128, "c", "c"]),
                     (moe.moe_w8a8_gemm, [4, 64, 128, "c", "f", "c", "f", "b"]),
                     (moe.moe_w8a8_linear, [4, 64, 128, "b", "c", "f", "c", "f", "b"]),
                     (moe.moe_w8a8_grouped_gemm, [desc, 2, "c", "f", "i", 2, 128, 128, "c", "f", "i", 0, "b"]),
                     (moe.moe_w8a8_experts, [desc, 1, "b", "f", "i", "i", "i", "c", "f", "c", "f", "c", "f", "b", "c",
                                             "f", "b", "b"]),
                     (moe.moe_balance_loss, [desc, 4, 1, "i", "u", "f", "i", 0.1, "i", "f", "f", "f", "u"]),
                     (moe.moe_route_backward, [desc, 4, 1, "i", "u", "f", "i", "i", "f", "f", "f", "f"])):
        for at, a in enumerate(args):
            if isinstance(a, str):
                call = [t[x] if isinstance(x, str) else x for x in args]
                call[at] = call[at].as_subclass(Away)
                with pytest.raises(ValueError, match="device"):
                    fn(*call)


@pytest.mark.parametrize("T", [1, 6, 200, 900])
def test_another_stream_that_waits_for_the_inputs(T):
    """The layer on a stream of its own, which waits for the stream that filled the inputs, the weights and the workspaces,
    as a caller has to: the bits of the eager call, also after another batch in the same buffers."""
    case, layer, _ = _experts_case(T, 1024, 256, 8, 2, 1, 9)
    eager, buf = moe.Buffers(case.desc, T, int8=True), moe.Buffers(case.desc, T, int8=True)
    x = case.xd.clone()
    side = torch.cuda.Stream()
    for i in range(3):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.forward(x, buf)
        torch.cuda.current_stream().wait_stream(side)
        layer.forward(x, eager)
        torch.cuda.synchronize()
        for name in ("h", "y", "out"):
            assert torch.equal(getattr(buf, name).view(torch.int16), getattr(eager, name).view(torch.int16)), (i, name)
        x.copy_(case.xd.flip(1) * (i + 2.0))
