// moe_fp8s.hip -- matrix products in 8-bit floating point (e4m3) with an fp32
// scale for each block of 128: of a token's row in the activations, 128 x 128
// in the weights.  Here: the quantisation of rows and of weights, the
// weight-stream kernel for few rows per group, and the ABI entry points.  The
// LDS-tiled kernel for many rows is in moe_fp8s_tiled.hip.
//
//   out[m][n] = bf16( sum_b as[m][b] ws[n / 128][b] sum_{k in b} a[m][k] w[n][k] )
//
// with b the blocks of 128 k; the sums over a block come out of the matrix
// cores in fp32, and so do the sums over the blocks.
#include <algorithm>

#include "moe_fp8s.h"

namespace moe {
namespace f8 {
namespace {

// ---------------------------------------------------------------- quantise
// Sixteen lanes per block of 128, eight elements each; the chunks of a row are
// counted up to whole blocks.  Bound by HBM: 8192 x 4096 in 19.4 us, 5.2 TB/s;
// below a MB by its launch (4 us).
__global__ __launch_bounds__(256) void k_act_quant_fp8s(const uint16_t *__restrict__ a, int rows, int K, int KG,
                                                        uint8_t *__restrict__ codes, float *__restrict__ scales) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int row = (int)(i / (16 * KG)), c = (int)(i - (int64_t)row * (16 * KG));
    const bool in = row < rows && 8 * c < K;
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (in) v = *(const u32x4 *)(a + (size_t)row * K + 8 * c);
    const BlockScale s = block_scale(max_of_16(max8(v)));
    if (!in) return;
    *(uint2 *)(codes + (size_t)row * K + 8 * c) = quant8(v, s);
    if ((c & 15) == 0) scales[(size_t)row * KG + (c >> 4)] = s.scale;
}

// A workgroup per block of 128 x 128 weights.  Bound by HBM: 257 x 4096 x 4096 in
// 2425 us, 5.3 TB/s; 4096 x 4096 in 11.9.
__global__ __launch_bounds__(256) void k_weight_quant_fp8s(const uint16_t *__restrict__ w, int N, int K, int NBK, int KG,
                                                           uint8_t *__restrict__ codes, float *__restrict__ scales) {
    __shared__ uint32_t smax[4];
    const int tid = threadIdx.x, kg = blockIdx.x, nb = blockIdx.y, c = 8 * (tid & 15) + 128 * kg;
    const size_t g = blockIdx.z;
    u32x4 v[8];
    uint32_t mx = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = 128 * nb + 16 * i + (tid >> 4);
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (n < N && c < K) v[i] = *(const u32x4 *)(w + (g * N + n) * K + c);
        mx = max(mx, max8(v[i]));
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, d, kWave));
    if ((tid & 63) == 0) smax[tid >> 6] = mx;
    __syncthreads();
    const BlockScale s = block_scale(max(max(smax[0], smax[1]), max(smax[2], smax[3])));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = 128 * nb + 16 * i + (tid >> 4);
        if (n < N && c < K) *(uint2 *)(codes + (g * N + n) * K + c) = quant8(v[i], s);
    }
    if (tid == 0) scales[(g * NBK + nb) * KG + kg] = s.scale;
}

// ---------------------------------------------------------------- weight stream
// Few rows per group.  A workgroup of eight waves takes NS subtiles (16 weight
// rows each; SwiGLU: NS/2 of the gate and the same NS/2 of the up projection)
// and at most 16 rows of one group; the waves split K by blocks of 128: wave w
// takes blocks w, w + 8, ..., U of them in flight; every weight byte goes
// straight from HBM into the registers of the one wave that multiplies it,
// and the waves' partial sums meet in LDS.  1 token of the 256-expert layer of
// 4096/2048: gate/up 22 us, down 14.6, 5.3 and 4.0 TB/s; 1 x 4096 x 4096 4.5.  Q
// (K <= kFusedMaxK): the rows come in bf16 and every workgroup quantises its own
// copy of them into LDS while its first weights are in flight: one launch less.
constexpr int kFusedMaxK = 4096, kW = 8;

template <int ACT, int NS, int U, bool Q>
__global__ __launch_bounds__(64 * kW) void k_fp8s_stream(Args p) {
    __shared__ float sred[kW * NS * 256];
    __shared__ int srow[16];
    extern __shared__ __attribute__((aligned(16))) uint8_t sq[];  // Q: codes [rows][128 KG + 16], scales [rows][KG]
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id();
    const int m = l & 15, q = l >> 4;
    TileItem it;
    const int TM = Q ? p.qrows : 16;  // rows of a tile (Q: as many as the launch gave LDS for)
    if (p.offsets) {
        if (!workgroup_tile_item(p.NB, TM, p.offsets, p.G, p.R, it)) return;
    } else {  // one group: the blocks in order, the m-tiles of an n-block side by side
        const int mt = (p.R + TM - 1) / TM;
        it.g = 0;
        it.nb = blockIdx.x / mt;
        it.m0 = (blockIdx.x - it.nb * mt) * TM;
        if (it.nb >= p.NB) return;
        it.mrows = min(TM, p.R - it.m0);
    }
    const int K = p.K, KG = p.KG, NTH = p.NT >> 1, NBK = (p.N + 127) >> 7;
    auto tile_of = [&](int j) {  // subtile j of the workgroup
        const int t = ACT == MOE_ACT_SWIGLU ? (j < NS / 2 ? it.nb * (NS / 2) + j : NTH + it.nb * (NS / 2) + j - NS / 2)
                                            : it.nb * NS + j;
        return min(t, p.NT - 1);
    };
    const uint8_t *wb[NS];
    const float *ws[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        wb[j] = p.wq + ((size_t)it.g * p.NT + tile_of(j)) * (2 * KG) * kBlockBytes;
        ws[j] = p.ws + ((size_t)it.g * NBK + (tile_of(j) >> 3)) * KG;
    }
    u32x4 b[U][NS][2];
    float sw[U][NS];
    auto load_b = [&](int kg0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kg = kg0 + u * kW + wave;
            if (kg < KG) {
                const uint32_t off = (uint32_t)kg * (2 * kBlockBytes) + 16 * l;
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    b[u][j][0] = __builtin_nontemporal_load((const u32x4 *)(wb[j] + off));
                    b[u][j][1] = __builtin_nontemporal_load((const u32x4 *)(wb[j] + off + kBlockBytes));
                    sw[u][j] = ws[j][kg];
                }
            }
        }
    };
    load_b(0);
    if (tid < 16) {  // the source row of each row of the tile (-1: none)
        int src = -1;
        if (tid < it.mrows) {
            src = it.m0 + tid;
            if (p.gather) {
                const int t = p.gather[it.m0 + tid];
                src = (unsigned)t < (unsigned)p.n_src ? t : -1;
            }
        }
        srow[tid] = src;
    }
    __syncthreads();
    f32x4 acc[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](int u, v8i a, float sa) {
        Wide aw;
        if constexpr (ACT == MOE_ACT_SWIGLU) aw = widen(a);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const v8i w = join(b[u][j][0], b[u][j][1]);
            f32x4 t;
            if constexpr (ACT == MOE_ACT_SWIGLU)
                t = mfma_wide(widen(w), aw);
            else
                t = mfma_fp8(w, a);
            const float f = sa * sw[u][j];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = __builtin_fmaf(t[e], f, acc[j][e]);
        }
    };

    if constexpr (Q) {
        const int LD = 128 * KG + 16;
        float *ssc = (float *)(sq + (size_t)it.mrows * LD);
        for (int i = tid; i < it.mrows * 16 * KG; i += 64 * kW) {  // (16 KG a multiple of the 16 lanes of a block)
            const int r = i / (16 * KG), c = i - r * (16 * KG), src = srow[r];
            u32x4 v = u32x4{0u, 0u, 0u, 0u};
            if (src >= 0 && 8 * c < K) v = *(const u32x4 *)(p.x + (size_t)src * K + 8 * c);
            const BlockScale s = block_scale(max_of_16(max8(v)));
            *(uint2 *)(sq + (size_t)r * LD + 8 * c) = quant8(v, s);
            if ((c & 15) == 0) ssc[r * KG + (c >> 4)] = s.scale;
        }
        __syncthreads();
        const int mr = min(m, it.mrows - 1);
        const uint8_t *ar = sq + (size_t)mr * LD + 16 * q;
        for (int kg0 = 0;;) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kg = kg0 + u * kW + wave;
                if (kg < KG) {
                    const u32x4 *at = (const u32x4 *)(ar + 128 * kg);
                    multiply(u, join(at[0], at[4]), ssc[mr * KG + kg]);
                }
            }
            kg0 += U * kW;
            if (kg0 >= KG) break;
            load_b(kg0);
        }
    } else {
        const size_t src = (size_t)max(srow[m], 0);
        const uint8_t *ar = p.a + src * K;
        const float *as = p.as + src * KG;
        for (int kg0 = 0;;) {
            u32x4 lo[U], hi[U];
            float sa[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kg = kg0 + u * kW + wave;
                if (kg < KG) {  // past the end of a row: any of its codes, the weights there are zero
                    lo[u] = *(const u32x4 *)(ar + min(128 * kg + 16 * q, K - 16));
                    hi[u] = *(const u32x4 *)(ar + min(128 * kg + 16 * q + 64, K - 16));
                    sa[u] = as[kg];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (kg0 + u * kW + wave < KG) multiply(u, join(lo[u], hi[u]), sa[u]);
            kg0 += U * kW;
            if (kg0 >= KG) break;
            load_b(kg0);
        }
    }
    // the waves' partial sums: [wave][j][lane][i]
#pragma unroll
    for (int j = 0; j < NS; ++j) *(f32x4 *)&sred[(wave * NS + j) * 256 + 4 * l] = acc[j];
    __syncthreads();
    constexpr int NO = ACT == MOE_ACT_SWIGLU ? NS / 2 : NS;  // output subtiles
    if (tid < NO * 64) {
        const int j = tid >> 6;
        if (m >= it.mrows) return;
        f32x4 s0 = f32x4{0.0f, 0.0f, 0.0f, 0.0f}, s1 = s0;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            const f32x4 v = *(const f32x4 *)&sred[(w * NS + j) * 256 + 4 * l];
            const f32x4 u = ACT == MOE_ACT_SWIGLU ? *(const f32x4 *)&sred[(w * NS + j + NS / 2) * 256 + 4 * l] : v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s0[e] += v[e];
                s1[e] += u[e];
            }
        }
        const int t = ACT == MOE_ACT_SWIGLU ? it.nb * (NS / 2) + j : it.nb * NS + j;
        const int n = packed_row(t, 4 * q), NC = ACT == MOE_ACT_SWIGLU ? p.N >> 1 : p.N;
        if (n >= NC) return;
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[e] = ACT == MOE_ACT_SWIGLU ? silu_mul(s0[e], s1[e]) : s0[e];
            if (srow[m] < 0) o[e] = 0.0f;  // a row without a source
        }
        *(uint2 *)(p.out + (size_t)(it.m0 + m) * NC + n) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
}

template <int ACT, int NS, int U, bool Q>
void launch_stream_u(Args a, int rows, hipStream_t st) {
    a.NB = (ACT == MOE_ACT_SWIGLU ? a.NT / 2 : a.NT) / (ACT == MOE_ACT_SWIGLU ? NS / 2 : NS);
    const int TM = Q ? rows : 16;
    a.qrows = rows;
    int64_t tiles = a.offsets ? (int64_t)a.R / TM + (a.R < a.G ? a.R : a.G) : (a.R + TM - 1) / TM;
    if (tiles > a.R) tiles = a.R;  // every tile has a row
    const dim3 grid((unsigned)((tiles * a.NB + 7) / 8 * 8));
    const size_t lds = Q ? (size_t)rows * (132 * a.KG + 16) : 0;
    hipLaunchKernelGGL((k_fp8s_stream<ACT, NS, U, Q>), grid, dim3(64 * kW), lds, st, a);
}

// U: the k blocks that each wave has in flight.  One where workgroups follow each
// other on the CUs, as many as K gives a wave (up to 4) where one round of them
// is all there is: 1 x 4096 x 4096 6.1, 5.9 us, 1 x 16384 x 4096 12.4, 13.1 (U = 1,
// 4; weights from HBM); experts of 1 token of the 256-expert layer 43.6, 49.9.
// NS: two subtiles of y's columns to a workgroup there, one 43.6 -> 41.6.
template <bool Q>
void launch_stream_dense(const Args &a, int rows, hipStream_t st) {
    const bool deep = a.NT <= 512;
    if (!deep || a.KG <= kW)
        launch_stream_u<MOE_ACT_NONE, 1, 1, Q>(a, rows, st);
    else if (a.KG <= 2 * kW)
        launch_stream_u<MOE_ACT_NONE, 1, 2, Q>(a, rows, st);
    else
        launch_stream_u<MOE_ACT_NONE, 1, 4, Q>(a, rows, st);
}
template <bool Q>
void launch_stream(int act, const Args &a, int rows, hipStream_t st) {
    if (act == MOE_ACT_SWIGLU)  // (grouped: products of one group have no SwiGLU)
        launch_stream_u<MOE_ACT_SWIGLU, 2, 1, Q>(a, rows, st);
    else if (a.offsets)
        launch_stream_u<MOE_ACT_NONE, 2, 1, Q>(a, rows, st);
    else
        launch_stream_dense<Q>(a, rows, st);
}

// Where the weight stream is the faster kernel, by measured times (us; stream,
// tiles of 64 x 128 or 32 x 64): one group, 16 and 17 rows of 4096 x 4096 9.7, 10.3
// and 9.0, 9.0; 7, 28, 112, 224 and 252 (skewed) rows of 257 groups, gate/up 25, 66, 209,
// 359, 263 and 29, 91, 262, 384, 256, down 14, 38, 111, 189, 146 and 16, 34, 123, 191, 133;
// 64 and 96 rows of 41 groups, gate/up 1024 x 1024 9.6, 12 and 12, 17, down 7.5, 9.4 and
// 6.8, 8.1; 48 rows of 9 groups, gate/up 4096 x 4096 30 and 51, down 18 and 25.  SwiGLU's
// products are in bf16 here (see mfma_wide): 64 tokens with a skewed choice 380,
// in tiles 421, and 371 as they are.
bool few(int act, int rows) { return rows <= (act == MOE_ACT_SWIGLU ? 64 : 16); }
// Where a product's workgroups quantise its few rows for themselves instead of a
// launch before.
bool fuse(int rows, int K) { return K <= kFusedMaxK && rows <= 4; }

// rows: an upper bound of the rows of one group.  Returns whether a.hq and a.hqs
// were written instead of a.out.
bool launch_gemm(int act, const Args &a, int rows, hipStream_t st) {
    if (a.x) {
        launch_stream<true>(act, a, rows, st);
    } else if (few(act, rows)) {
        launch_stream<false>(act, a, rows, st);
    } else {
        return launch_tiled(act, a, st);
    }
    return false;
}

void launch_quant(int rows, int K, const uint16_t *a, uint8_t *codes, float *scales, hipStream_t st) {
    const int KG = (K + 127) / 128, most = (1 << 24) / KG;  // rows whose chunks number at most 2^28
    for (int r = 0; r < rows; r += most) {
        const int n = std::min(most, rows - r);
        hipLaunchKernelGGL(k_act_quant_fp8s, dim3((unsigned)(((int64_t)n * 16 * KG + 255) / 256)), dim3(256), 0, st,
                           a + (size_t)r * K, n, K, KG, codes + (size_t)r * K, scales + (size_t)r * KG);
    }
}

moe_status check_nk(int32_t N, int32_t K) {
    if (N < 16 || N % 16 || N > 65536 || K < 16 || K % 16 || K > 65536) return MOE_ERR_SHAPE;
    return MOE_OK;
}

Args make_args(int G, int R, int N, int K, const uint8_t *wq, const float *ws, uint16_t *out) {
    Args x = {};
    x.wq = wq;
    x.ws = ws;
    x.G = G;
    x.R = R;
    x.N = N;
    x.K = K;
    x.out = out;
    x.KG = kblocks(K) / 2;
    x.NT = subtiles(N);
    return x;
}

}  // namespace
}  // namespace f8
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_act_quant_fp8s(int32_t rows, int32_t K, const uint16_t *a, uint8_t *codes, float *scales,
                                         void *stream) {
    if (rows < 0 || rows > MOE_MAX_TOKENS * 9 || K < 16 || K % 16 || K > 65536) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!a || !codes || !scales) return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
    f8::launch_quant(rows, K, a, codes, scales, (hipStream_t)stream);
    return launch_status();
}

extern "C" moe_status moe_fp8s_quant_weights(int32_t n_groups, int32_t N, int32_t K, const uint16_t *w, uint8_t *codes,
                                             float *scales, void *stream) {
    if (n_groups < 1 || n_groups > 257) return MOE_ERR_SHAPE;
    MOE_TRY(f8::check_nk(N, K));
    if (!w || !codes || !scales) return MOE_ERR_NULL;
    if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
    const int NBK = (N + 127) / 128, KG = (K + 127) / 128;
    hipLaunchKernelGGL(f8::k_weight_quant_fp8s, dim3(KG, NBK, n_groups), dim3(256), 0, (hipStream_t)stream, w, N, K, NBK, KG,
                       codes, scales);
    return launch_status();
}

extern "C" size_t moe_fp8s_packed_bytes(int32_t n_groups, int32_t N, int32_t K) { return moe_w8a8_packed_bytes(n_groups, N, K); }

extern "C" moe_status moe_fp8s_prepack(int32_t n_groups, int32_t N, int32_t K, const uint8_t *w_canonical,
                                       uint8_t *w_packed, void *stream) {
    return moe_w8a8_prepack(n_groups, N, K, (const int8_t *)w_canonical, (int8_t *)w_packed, stream);  // bytes in the same places
}

extern "C" moe_status moe_fp8s_gemm(int32_t M, int32_t N, int32_t K, const uint8_t *a, const float *a_scales,
                                    const uint8_t *w_packed, const float *w_scales, uint16_t *out, void *stream) {
    if (M < 0 || M > MOE_MAX_TOKENS) return MOE_ERR_SHAPE;
    MOE_TRY(f8::check_nk(N, K));
    if (M == 0) return MOE_OK;
    if (!a || !a_scales || !w_packed || !w_scales || !out) return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(w_packed, 16) || !aligned(out, 16) || !aligned(w_scales, 4) || !aligned(a_scales, 4))
        return MOE_ERR_ALIGN;
    f8::Args x = f8::make_args(1, M, N, K, w_packed, w_scales, out);
    x.a = a;
    x.as = a_scales;
    f8::launch_gemm(MOE_ACT_NONE, x, M, (hipStream_t)stream);
    return launch_status();
}

extern "C" moe_status moe_fp8s_linear(int32_t M, int32_t N, int32_t K, const uint16_t *x, const uint8_t *w_packed,
                                      const float *w_scales, uint8_t *codes, float *scales, uint16_t *out,
                                      void *stream) {
    if (M < 0 || M > MOE_MAX_TOKENS) return MOE_ERR_SHAPE;
    MOE_TRY(f8::check_nk(N, K));
    if (M == 0) return MOE_OK;
    if (!x || !w_packed || !w_scales || !codes || !scales || !out) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(out, 16) || !aligned(w_scales, 4) || !aligned(codes, 16) ||
        !aligned(scales, 4))
        return MOE_ERR_ALIGN;
    hipStream_t st = (hipStream_t)stream;
    f8::Args p = f8::make_args(1, M, N, K, w_packed, w_scales, out);
    if (f8::fuse(M, K)) {
        p.x = x;
    } else {
        f8::launch_quant(M, K, x, codes, scales, st);
        p.a = codes;
        p.as = scales;
    }
    f8::launch_gemm(MOE_ACT_NONE, p, M, st);
    return launch_status();
}

extern "C" moe_status moe_fp8s_grouped_gemm(const moe_layer_desc *desc, int32_t T, const uint8_t *a,
                                            const float *a_scales, const int32_t *a_gather, int32_t n_src, int32_t N,
                                            int32_t K, const uint8_t *w_packed, const float *w_scales,
                                            const int32_t *group_offsets, int32_t act, uint16_t *out, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_tokens(T));
    if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU && act != MOE_ACT_SWIGLU_F32) return MOE_ERR_UNSUPPORTED;
    MOE_TRY(f8::check_nk(N, K));
    if (act != MOE_ACT_NONE && N % 128) return MOE_ERR_SHAPE;  // both halves whole 64-row tiles
    if (a_gather && (n_src < 1 || n_src > MOE_MAX_TOKENS)) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!a || !a_scales || !w_packed || !w_scales || !group_offsets || !out) return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(a_scales, 4) || !aligned(a_gather, 4) || !aligned(w_packed, 16) ||
        !aligned(w_scales, 4) || !aligned(group_offsets, 4) || !aligned(out, 16))
        return MOE_ERR_ALIGN;
    f8::Args p = f8::make_args(desc->n_routed + desc->n_shared, T * (desc->top_k + desc->n_shared), N, K, w_packed,
                               w_scales, out);
    p.a = a;
    p.as = a_scales;
    p.gather = a_gather;
    p.n_src = n_src;
    p.offsets = group_offsets;
    p.f32 = act == MOE_ACT_SWIGLU_F32;
    f8::launch_gemm(act == MOE_ACT_NONE ? act : MOE_ACT_SWIGLU, p, T, (hipStream_t)stream);
    return launch_status();
}

extern "C" moe_status moe_fp8s_experts(const moe_layer_desc *desc, int32_t T, const uint16_t *x, const float *topk_w,
                                       const int32_t *group_offsets, const int32_t *sorted_token,
                                       const int32_t *row_of_slot, const uint8_t *w13_packed, const float *w13_scales,
                                       const uint8_t *w2_packed, const float *w2_scales, uint8_t *xq, float *xqs,
                                       uint16_t *h, uint8_t *hq, float *hqs, uint16_t *y, uint16_t *out, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_tokens(T));
    if (T == 0) return MOE_OK;
    if (!x || !topk_w || !group_offsets || !sorted_token || !row_of_slot || !w13_packed || !w13_scales || !w2_packed ||
        !w2_scales || !xq || !xqs || !h || !hq || !hqs || !y || !out)
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(topk_w, 4) || !aligned(group_offsets, 4) || !aligned(sorted_token, 4) ||
        !aligned(row_of_slot, 4) || !aligned(w13_packed, 16) || !aligned(w13_scales, 4) || !aligned(w2_packed, 16) ||
        !aligned(w2_scales, 4) || !aligned(xq, 16) || !aligned(xqs, 4) || !aligned(h, 16) || !aligned(hq, 16) ||
        !aligned(hqs, 4) || !aligned(y, 16) || !aligned(out, 16))
        return MOE_ERR_ALIGN;
    const int H = desc->hidden, I = desc->inter, G = desc->n_routed + desc->n_shared;
    const int R = T * (desc->top_k + desc->n_shared);
    hipStream_t st = (hipStream_t)stream;
    f8::Args p = f8::make_args(G, R, 2 * I, H, w13_packed, w13_scales, h);
    p.gather = sorted_token;
    p.n_src = T;
    p.offsets = group_offsets;
    const bool fused = f8::fuse(T, std::max(H, I));
    if (fused) {
        p.x = x;
    } else {
        f8::launch_quant(T, H, x, xq, xqs, st);
        p.a = xq;
        p.as = xqs;
    }
    if (!fused) {
        p.hq = hq;
        p.hqs = hqs;
    }
    const bool quantised = f8::launch_gemm(MOE_ACT_SWIGLU, p, T, st);
    f8::Args d = f8::make_args(G, R, H, I, w2_packed, w2_scales, y);
    d.offsets = group_offsets;
    if (fused) {
        d.x = h;
    } else {
        if (!quantised) f8::launch_quant(R, I, h, hq, hqs, st);
        d.a = hq;
        d.as = hqs;
    }
    f8::launch_gemm(MOE_ACT_NONE, d, T, st);
    MOE_TRY(launch_status());
    return moe_combine(desc, T, y, row_of_slot, topk_w, out, stream);
}
