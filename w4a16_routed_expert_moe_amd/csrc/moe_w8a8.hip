// moe_w8a8.hip -- matrix products in 8-bit integers with a scale for each
// token and each output channel (W8A8): the per-token quantisation, the
// weight layout, the weight-stream kernel for few rows per group, and the
// ABI entry points.  The LDS-tiled kernel for many rows is in
// moe_w8a8_tiled.hip.
//
//   acc[m][n] = sum_k a[m][k] w[n][k]            exact, in int32
//   out[m][n] = bf16( (float)acc * as[m] * ws[n] )
//
// |a| <= 127 and |w| <= 128, so the sum stays below 2^31 up to K = 65536 and
// its order does not matter: every kernel and every split of K gives the same
// bits.
#include "moe_w8a8.h"

namespace moe {
namespace w8 {
namespace {

// ---------------------------------------------------------------- quantise
// W waves per row, NV 16-byte words of it per lane: the row is read once and
// stays in registers between its maximum and its codes.  3 bytes per
// element: bound by HBM.
template <int W, int NV>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void k_act_quant_int8(const uint16_t *__restrict__ a, int rows,
                                                                          int K, int8_t *__restrict__ codes,
                                                                          float *__restrict__ scales) {
    constexpr int RPB = W < 4 ? 4 / W : 1;  // rows per workgroup
    const int l = lane_id(), wave = threadIdx.x >> 6;
    const int row = blockIdx.x * RPB + wave / W, part = wave % W;
    const bool in = row < rows;
    const int chunks = K >> 3;
    const uint16_t *src = a + (size_t)(in ? row : 0) * K;
    u32x4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * W + part) * kWave + l;
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (c < chunks) v[i] = *(const u32x4 *)(src + 8 * c);
    }
    uint32_t mx = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = pk_max_abs(mx, v[i][j]);
    mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, d, kWave));
    if constexpr (W > 1) {
        __shared__ uint32_t smx[W < 4 ? 4 : W];
        smx[wave] = mx;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) mx = max(mx, smx[wave - part + i]);
    }
    if (!in) return;
    const RowScale s = row_scale(mx);
    if (part == 0 && l == 0) scales[row] = s.scale;
    int8_t *dst = codes + (size_t)row * K;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * W + part) * kWave + l;
        if (c < chunks) *(uint2 *)(dst + 8 * c) = quant8(v[i], s);
    }
}

// A wave per row up to 4096 elements where there are rows for every SIMD,
// else four waves per row (few rows: the latency of one row is what counts);
// 16 waves past 16384 elements.
void launch_quant(int rows, int K, const uint16_t *a, int8_t *codes, float *scales, hipStream_t st) {
#define QUANT(W, NV)                                                                                            \
    hipLaunchKernelGGL((k_act_quant_int8<W, NV>), dim3((unsigned)(W < 4 ? (rows + 4 / W - 1) / (4 / W) : rows)), \
                       dim3(W < 4 ? 256 : 64 * W), 0, st, a, rows, K, codes, scales)
    if (rows >= 2048 && K <= 4096) {
        if (K <= 1024)
            QUANT(1, 2);
        else if (K <= 2048)
            QUANT(1, 4);
        else
            QUANT(1, 8);
    } else if (K <= 2048) {
        QUANT(4, 1);
    } else if (K <= 4096) {
        QUANT(4, 2);
    } else if (K <= 16384) {
        QUANT(4, 8);
    } else {
        QUANT(16, 8);
    }
#undef QUANT
}

// ---------------------------------------------------------------- prepack
__global__ void k_w8a8_prepack(const int8_t *__restrict__ src, int8_t *__restrict__ dst, int G, int N, int K, int NT,
                               int KB) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;  // one 16-byte piece each
    const long long total = (long long)G * NT * KB * 64;
    if (i >= total) return;
    const int lane = (int)(i & 63);
    const long long blk = i >> 6;
    const int kb = (int)(blk % KB);
    const long long gt = blk / KB;
    const int t = (int)(gt % NT), g = (int)(gt / NT);
    const int n = packed_row(t, lane & 15), k = 64 * kb + 16 * (lane >> 4);
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (n < N && k < K) v = *(const u32x4 *)(src + ((size_t)g * N + n) * K + k);
    *(u32x4 *)(dst + 16 * i) = v;
}

// ---------------------------------------------------------------- weight stream
// Few rows per group: the weights' bytes are the bound.  A workgroup of W
// waves takes NS subtiles (16 weight rows each; SwiGLU: NS/2 of the gate and
// the same NS/2 of the up projection) and at most 16 C rows of one group;
// the waves split K: wave w takes k blocks w, w + W, ..., every weight byte
// goes straight from HBM into the registers of the one wave that multiplies
// it, U blocks ahead, and the waves' int32 partial sums meet in LDS.
// Q (C = 1, K <= 64 W U): the rows come in bf16 and are quantised here, each
// workgroup its own copy (a row is 2K bytes, in L2), while the weights are
// in flight: one launch less.
template <int ACT, int NS, int C, int W, int U, bool Q>
__global__ __launch_bounds__(64 * W) void k_w8a8_stream(Args p) {
    static_assert(!Q || C == 1, "the fused quantisation takes one m-tile");
    __shared__ int sred[W * NS * C * 256];
    __shared__ int srow[16 * C];
    __shared__ uint32_t smax[Q ? 16 * W : 1];
    __shared__ float sscale[16];  // Q: the rows' scales
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id();
    const int m = l & 15, q = l >> 4;
    TileItem it;
    if (p.offsets) {
        if (!workgroup_tile_item(p.NB, 16 * C, p.offsets, p.G, p.R, it)) return;
    } else {  // one group: the blocks in order, the m-tiles of an n-block side by side
        const int mt = (p.R + 16 * C - 1) / (16 * C);
        it.g = 0;
        it.nb = blockIdx.x / mt;
        it.m0 = (blockIdx.x - it.nb * mt) * 16 * C;
        if (it.nb >= p.NB) return;
        it.mrows = min(16 * C, p.R - it.m0);
    }
    const int K = p.K, KB = p.KB, NTH = p.NT >> 1;
    // subtile j of the workgroup
    auto tile_of = [&](int j) {
        const int t = ACT == MOE_ACT_SWIGLU ? (j < NS / 2 ? it.nb * (NS / 2) + j : NTH + it.nb * (NS / 2) + j - NS / 2)
                                            : it.nb * NS + j;
        return min(t, p.NT - 1);
    };
    const int8_t *wb[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) wb[j] = p.wq + ((size_t)it.g * p.NT + tile_of(j)) * KB * kBlockBytes;
    u32x4 b[U][NS];
    auto load_b = [&](int kb0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t off = (uint32_t)min(kb0 + u * W + wave, KB - 1) * kBlockBytes + 16 * l;
#pragma unroll
            for (int j = 0; j < NS; ++j) b[u][j] = __builtin_nontemporal_load((const u32x4 *)(wb[j] + off));
        }
    };
    load_b(0);
    // the source row of row 16 c + m of the tile (-1: none)
    int sr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int r = 16 * c + m;
        sr[c] = -1;
        if (r < it.mrows) {
            sr[c] = it.m0 + r;
            if (p.gather) {
                const int t = p.gather[it.m0 + r];
                sr[c] = (unsigned)t < (unsigned)p.n_src ? t : -1;
            }
        }
        if (wave == 0 && q == 0) srow[r] = sr[c];
    }
    v4i acc[C][NS];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < NS; ++j) acc[c][j] = v4i{0, 0, 0, 0};
    float rscale = 0.0f;  // Q: the scale of row m

    if constexpr (Q) {
        const uint16_t *xr = p.x + (size_t)max(sr[0], 0) * K;
        u32x4 v[U][2];
        uint32_t mx = 0u;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = 64 * (u * W + wave) + 16 * q;
            const bool in = k < K && sr[0] >= 0;
            v[u][0] = v[u][1] = u32x4{0u, 0u, 0u, 0u};
            if (in) {
                v[u][0] = *(const u32x4 *)(xr + k);
                v[u][1] = *(const u32x4 *)(xr + k + 8);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = pk_max_abs(pk_max_abs(mx, v[u][0][i]), v[u][1][i]);
        mx = max(mx & 0xFFFFu, mx >> 16);
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, kWave));
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, kWave));
        if (q == 0) smax[16 * wave + m] = mx;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) mx = max(mx, smax[16 * w + m]);
        const RowScale s = row_scale(mx);
        rscale = s.scale;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * W + wave >= KB) break;
            const uint2 lo = quant8(v[u][0], s), hi = quant8(v[u][1], s);
            const u32x4 av = u32x4{lo.x, lo.y, hi.x, hi.y};
#pragma unroll
            for (int j = 0; j < NS; ++j) acc[0][j] = mfma_i8(b[u][j], av, acc[0][j]);
        }
    } else {
        const int8_t *ar[C];
#pragma unroll
        for (int c = 0; c < C; ++c) ar[c] = p.a + (size_t)max(sr[c], 0) * K;
        for (int kb0 = 0;;) {
            u32x4 av[U][C];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // past the end of a row whose K is not a multiple of 128: any
                // 16 bytes of the row, the packed weights there are zero
                const int k = min(64 * (kb0 + u * W + wave) + 16 * q, K - 16);
#pragma unroll
                for (int c = 0; c < C; ++c) av[u][c] = *(const u32x4 *)(ar[c] + k);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (kb0 + u * W + wave < KB)
#pragma unroll
                    for (int j = 0; j < NS; ++j)
#pragma unroll
                        for (int c = 0; c < C; ++c) acc[c][j] = mfma_i8(b[u][j], av[u][c], acc[c][j]);
            kb0 += U * W;
            if (kb0 >= KB) break;
            load_b(kb0);
        }
    }
    // the waves' partial sums: [wave][j][c][i][lane]
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c)
            *(v4i *)&sred[((wave * NS + j) * C + c) * 256 + 4 * l] = acc[c][j];
    if constexpr (Q) {
        if (wave == 0 && q == 0) sscale[m] = rscale;
    }
    __syncthreads();
    constexpr int NO = ACT == MOE_ACT_SWIGLU ? NS / 2 : NS;  // output subtiles
    for (int i = tid; i < NO * C * 64; i += 64 * W) {
        const int ln = i & 63, jc = i >> 6, c = jc % C, j = jc / C;
        const int mm = ln & 15, qq = ln >> 4, r = 16 * c + mm;
        v4i s0 = v4i{0, 0, 0, 0}, s1 = v4i{0, 0, 0, 0};
        for (int w = 0; w < W; ++w) {
            s0 += *(const v4i *)&sred[((w * NS + j) * C + c) * 256 + 4 * ln];
            if (ACT == MOE_ACT_SWIGLU) s1 += *(const v4i *)&sred[((w * NS + j + NS / 2) * C + c) * 256 + 4 * ln];
        }
        if (r >= it.mrows) continue;
        const int t = ACT == MOE_ACT_SWIGLU ? it.nb * (NS / 2) + j : it.nb * NS + j;
        const int n = packed_row(t, 4 * qq);
        const int NC = ACT == MOE_ACT_SWIGLU ? p.N >> 1 : p.N;
        if (n >= NC) continue;
        const int src = srow[r];
        const float sa = Q ? sscale[mm] : p.as[max(src, 0)];
        const float *ws = p.ws + (size_t)it.g * p.N + n;
        float o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[k] = (float)s0[k] * sa * ws[k];
            if (ACT == MOE_ACT_SWIGLU) o[k] = silu_mul(o[k], (float)s1[k] * sa * ws[NC + k]);
            if (src < 0) o[k] = 0.0f;  // a row without a source
        }
        *(uint2 *)(p.out + (size_t)(it.m0 + r) * NC + n) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
}

template <int ACT, int NS, int C, bool Q>
void launch_stream(Args a, hipStream_t st) {
    constexpr int W = 8, U = 8;
    a.NB = (ACT == MOE_ACT_SWIGLU ? a.NT / 2 : a.NT) / (ACT == MOE_ACT_SWIGLU ? NS / 2 : NS);
    const int64_t tiles = a.offsets ? (int64_t)a.R / (16 * C) + (a.R < a.G ? a.R : a.G) : (a.R + 16 * C - 1) / (16 * C);
    const dim3 grid((unsigned)((tiles * a.NB + 7) / 8 * 8));
    hipLaunchKernelGGL((k_w8a8_stream<ACT, NS, C, W, U, Q>), grid, dim3(64 * W), 0, st, a);
}

constexpr int kFusedRows = 16;     // rows of one m-tile
constexpr int kFusedMaxK = 4096;   // 64 W U
constexpr int kStreamRows = 64;

// rows: an upper bound of the rows of one group
void launch_gemm(int act, const Args &a, int rows, hipStream_t st) {
    if (a.x) {
        if (act == MOE_ACT_SWIGLU)
            launch_stream<MOE_ACT_SWIGLU, 2, 1, true>(a, st);
        else
            launch_stream<MOE_ACT_NONE, 2, 1, true>(a, st);
    } else if (rows <= 16) {
        if (act == MOE_ACT_SWIGLU)
            launch_stream<MOE_ACT_SWIGLU, 2, 1, false>(a, st);
        else
            launch_stream<MOE_ACT_NONE, 2, 1, false>(a, st);
    } else if (rows <= kStreamRows) {
        if (act == MOE_ACT_SWIGLU)
            launch_stream<MOE_ACT_SWIGLU, 2, 4, false>(a, st);
        else
            launch_stream<MOE_ACT_NONE, 2, 4, false>(a, st);
    } else {
        launch_tiled(act, a, st);
    }
}

moe_status check_nk(int32_t N, int32_t K) {
    if (N < 16 || N % 16 || N > 65536 || K < 16 || K % 16 || K > 65536) return MOE_ERR_SHAPE;
    return MOE_OK;
}

Args make_args(int G, int R, int N, int K, const int8_t *wq, const float *ws, uint16_t *out) {
    Args x = {};
    x.wq = wq;
    x.ws = ws;
    x.G = G;
    x.R = R;
    x.N = N;
    x.K = K;
    x.out = out;
    x.KB = kblocks(K);
    x.NT = subtiles(N);
    return x;
}

}  // namespace
}  // namespace w8
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_act_quant_int8(int32_t rows, int32_t K, const uint16_t *a, int8_t *codes, float *scales,
                                         void *stream) {
    if (rows < 0 || rows > MOE_MAX_TOKENS * 9 || K < 16 || K % 16 || K > 65536) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!a || !codes || !scales) return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
    w8::launch_quant(rows, K, a, codes, scales, (hipStream_t)stream);
    return launch_status();
}

extern "C" size_t moe_w8a8_packed_bytes(int32_t n_groups, int32_t N, int32_t K) {
    if (n_groups < 1 || n_groups > 257 || w8::check_nk(N, K) != MOE_OK) return 0;
    return (size_t)n_groups * w8::subtiles(N) * w8::kblocks(K) * w8::kBlockBytes;
}

extern "C" moe_status moe_w8a8_prepack(int32_t n_groups, int32_t N, int32_t K, const int8_t *w_canonical,
                                       int8_t *w_packed, void *stream) {
    const size_t bytes = moe_w8a8_packed_bytes(n_groups, N, K);
    if (bytes == 0) return MOE_ERR_SHAPE;
    if (!w_canonical || !w_packed) return MOE_ERR_NULL;
    if (!aligned(w_canonical, 16) || !aligned(w_packed, 16)) return MOE_ERR_ALIGN;
    const uintptr_t s0 = (uintptr_t)w_canonical, d0 = (uintptr_t)w_packed;
    if (s0 < d0 + bytes && d0 < s0 + (size_t)n_groups * N * K) return MOE_ERR_SHAPE;  // overlapping buffers
    const size_t pieces = bytes / 16;
    if ((pieces + 255) / 256 > 0x7FFFFFFF) return MOE_ERR_SHAPE;
    hipLaunchKernelGGL(w8::k_w8a8_prepack, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, (hipStream_t)stream,
                       w_canonical, w_packed, n_groups, N, K, w8::subtiles(N), w8::kblocks(K));
    return launch_status();
}

extern "C" moe_status moe_w8a8_gemm(int32_t M, int32_t N, int32_t K, const int8_t *a, const float *a_scales,
                                    const int8_t *w_packed, const float *w_scales, uint16_t *out, void *stream) {
    if (M < 0 || M > MOE_MAX_TOKENS) return MOE_ERR_SHAPE;
    MOE_TRY(w8::check_nk(N, K));
    if (M == 0) return MOE_OK;
    if (!a || !a_scales || !w_packed || !w_scales || !out) return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(w_packed, 16) || !aligned(out, 16) || !aligned(w_scales, 16) || !aligned(a_scales, 4))
        return MOE_ERR_ALIGN;
    w8::Args x = w8::make_args(1, M, N, K, w_packed, w_scales, out);
    x.a = a;
    x.as = a_scales;
    w8::launch_gemm(MOE_ACT_NONE, x, M, (hipStream_t)stream);
    return launch_status();
}

extern "C" moe_status moe_w8a8_linear(int32_t M, int32_t N, int32_t K, const uint16_t *x, const int8_t *w_packed,
                                      const float *w_scales, int8_t *codes, float *scales, uint16_t *out,
                                      void *stream) {
    if (M < 0 || M > MOE_MAX_TOKENS) return MOE_ERR_SHAPE;
    MOE_TRY(w8::check_nk(N, K));
    if (M == 0) return MOE_OK;
    if (!x || !w_packed || !w_scales || !codes || !scales || !out) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(out, 16) || !aligned(w_scales, 16) ||
        !aligned(codes, 16) || !aligned(scales, 4))
        return MOE_ERR_ALIGN;
    hipStream_t st = (hipStream_t)stream;
    w8::Args p = w8::make_args(1, M, N, K, w_packed, w_scales, out);
    if (M <= w8::kFusedRows && K <= w8::kFusedMaxK) {
        p.x = x;
    } else {
        w8::launch_quant(M, K, x, codes, scales, st);
        p.a = codes;
        p.as = scales;
    }
    w8::launch_gemm(MOE_ACT_NONE, p, M, st);
    return launch_status();
}

namespace {
// N and K limits of the grouped product (SwiGLU: both halves whole 64-row tiles)
moe_status check_grouped(int32_t act, int32_t N, int32_t K) {
    if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return MOE_ERR_UNSUPPORTED;
    MOE_TRY(w8::check_nk(N, K));
    if (act == MOE_ACT_SWIGLU && N % 128) return MOE_ERR_SHAPE;
    return MOE_OK;
}
}  // namespace

extern "C" moe_status moe_w8a8_grouped_gemm(const moe_layer_desc *desc, int32_t T, const int8_t *a,
                                            const float *a_scales, const int32_t *a_gather, int32_t n_src, int32_t N,
                                            int32_t K, const int8_t *w_packed, const float *w_scales,
                                            const int32_t *group_offsets, int32_t act, uint16_t *out, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_tokens(T));
    MOE_TRY(check_grouped(act, N, K));
    if (a_gather && (n_src < 1 || n_src > MOE_MAX_TOKENS)) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!a || !a_scales || !w_packed || !w_scales || !group_offsets || !out) return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(a_scales, 4) || !aligned(w_packed, 16) || !aligned(w_scales, 16) ||
        !aligned(out, 16) || !aligned(group_offsets, 4) || (a_gather && !aligned(a_gather, 4)))
        return MOE_ERR_ALIGN;
    w8::Args x = w8::make_args(desc->n_routed + desc->n_shared, T * (desc->top_k + desc->n_shared), N, K, w_packed,
                               w_scales, out);
    x.a = a;
    x.as = a_scales;
    x.gather = a_gather;
    x.n_src = n_src;
    x.offsets = group_offsets;
    w8::launch_gemm(act, x, T, (hipStream_t)stream);
    return launch_status();
}

extern "C" moe_status moe_w8a8_experts(const moe_layer_desc *desc, int32_t T, const uint16_t *x, const float *topk_w,
                                       const int32_t *group_offsets, const int32_t *sorted_token,
                                       const int32_t *row_of_slot, const int8_t *w13_packed, const float *w13_scales,
                                       const int8_t *w2_packed, const float *w2_scales, int8_t *xq, float *xqs,
                                       uint16_t *h, int8_t *hq, float *hqs, uint16_t *y, uint16_t *out, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_tokens(T));
    if (T == 0) return MOE_OK;
    if (!x || !topk_w || !group_offsets || !sorted_token || !row_of_slot || !w13_packed || !w13_scales || !w2_packed ||
        !w2_scales || !xq || !xqs || !h || !hq || !hqs || !y || !out)
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(topk_w, 4) || !aligned(group_offsets, 4) || !aligned(sorted_token, 4) ||
        !aligned(row_of_slot, 4) || !aligned(w13_packed, 16) || !aligned(w13_scales, 16) || !aligned(w2_packed, 16) ||
        !aligned(w2_scales, 16) || !aligned(xq, 16) || !aligned(xqs, 4) || !aligned(h, 16) || !aligned(hq, 16) ||
        !aligned(hqs, 4) || !aligned(y, 16) || !aligned(out, 16))
        return MOE_ERR_ALIGN;
    const int H = desc->hidden, I = desc->inter, G = desc->n_routed + desc->n_shared;
    const int R = T * (desc->top_k + desc->n_shared);
    hipStream_t st = (hipStream_t)stream;
    const bool fused = T <= w8::kFusedRows;  // H and I are at most 4096 = kFusedMaxK
    w8::Args p = w8::make_args(G, R, 2 * I, H, w13_packed, w13_scales, h);
    p.gather = sorted_token;
    p.n_src = T;
    p.offsets = group_offsets;
    if (fused) {
        p.x = x;
    } else {
        w8::launch_quant(T, H, x, xq, xqs, st);
        p.a = xq;
        p.as = xqs;
    }
    w8::launch_gemm(MOE_ACT_SWIGLU, p, T, st);
    w8::Args d = w8::make_args(G, R, H, I, w2_packed, w2_scales, y);
    d.offsets = group_offsets;
    if (fused) {
        d.x = h;
    } else {
        w8::launch_quant(R, I, h, hq, hqs, st);
        d.a = hq;
        d.as = hqs;
    }
    w8::launch_gemm(MOE_ACT_NONE, d, T, st);
    MOE_TRY(launch_status());
    return moe_combine(desc, T, y, row_of_slot, topk_w, out, stream);
}
