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
#include <algorithm>

#include "moe_route_common.h"
#include "moe_w8a8.h"

namespace moe {
namespace w8 {
namespace {

// ---------------------------------------------------------------- quantise
// W waves per row, NV 16-byte words of it per lane: the row is read once and
// stays in registers between its maximum and its codes.  3 bytes per
// element: bound by HBM (8192 x 4096: 100 MB in 22 us, 4.6 TB/s; 57344 x 2048
// behind the product that wrote it: 53 us, 6.6 TB/s).
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
// One 16-byte piece per thread, a group per blockIdx.y.
__global__ void k_w8a8_prepack(const int8_t *__restrict__ src, int8_t *__restrict__ dst, int N, int K, int NT, int KB) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x, total = NT * KB * 64, g = blockIdx.y;
    if (i >= total) return;
    const int lane = i & 63, blk = i >> 6, kb = blk % KB, t = blk / KB;
    const int n = packed_row(t, lane & 15), k = 64 * kb + 16 * (lane >> 4);
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (n < N && k < K) v = *(const u32x4 *)(src + ((size_t)g * N + n) * K + k);
    *(u32x4 *)(dst + 16 * ((size_t)g * total + i)) = v;
}

// ---------------------------------------------------------------- weight stream
// Few rows per group: the weights' bytes are the bound (the gate/up product of
// 7 rows at hidden 4096, inter 2048: 117 MB in 27 to 28 us, 4.2 TB/s, the
// first requests' latency and the launch with it).  A workgroup of W
// waves takes NS subtiles (16 weight rows each; SwiGLU: NS/2 of the gate and
// the same NS/2 of the up projection) and at most 16 rows of one group; the
// waves split K: wave w takes k blocks w, w + W, ..., every weight byte
// goes straight from HBM into the registers of the one wave that multiplies
// it, U blocks ahead, and the waves' int32 partial sums meet in LDS.
// Q (K <= kFusedMaxK): the rows come in bf16 and every workgroup
// quantises its own copy of them into LDS while its weights are in flight (a
// row is 2K bytes, in L2): one launch less.
constexpr int kFusedMaxK = 4096;  // 8 elements per thread of 8 waves

// `rows` bf16 rows (row r from source row src_of(r) of x, zeros if that is
// negative) to INT8 codes in LDS, row r at sq + r (K + 16) -- 16 bytes of
// padding: 16 rows at one k sit on distinct banks -- and their scales.  A row
// takes as many waves as it needs (1, 2, 4 or 8; eight elements per thread),
// the W waves W divided by that many rows at a time and kQuantRows times as
// many between two barriers.  Ends with a barrier.
constexpr int kQuantRows = 4;
__host__ __device__ inline int log2_waves_per_row(int K) { return K <= 512 ? 0 : K <= 1024 ? 1 : K <= 2048 ? 2 : 3; }
template <int W, typename F>
__device__ __forceinline__ void quantise_rows(const uint16_t *__restrict__ x, int K, int rows, F src_of, int8_t *sq,
                                              float *sscale, uint32_t (&smax)[kQuantRows * W]) {
    constexpr int RB = kQuantRows;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id(), LD = K + 16;
    const int lw = log2_waves_per_row(K), GR = W >> lw, gr = wave >> lw, part = wave & ((1 << lw) - 1);
    const int tid = 64 * part + l;  // of the threads of the row
    const bool in = 8 * tid < K;
    for (int r0 = gr; r0 - gr < rows; r0 += RB * GR) {
        u32x4 v[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            v[i] = u32x4{0u, 0u, 0u, 0u};
            const int r = r0 + i * GR, src = r < rows ? __builtin_amdgcn_readfirstlane(src_of(r)) : -1;
            if (in && src >= 0) v[i] = *(const u32x4 *)(x + (size_t)src * K + 8 * tid);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            if (r0 + i * GR < rows) {
                uint32_t mx = pk_max_abs(pk_max_abs(pk_max_abs(pk_max_abs(0u, v[i][0]), v[i][1]), v[i][2]), v[i][3]);
                mx = route::wave_max32(max(mx & 0xFFFFu, mx >> 16));
                if (l == 0) smax[i * W + wave] = mx;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int r = r0 + i * GR;
            if (r < rows) {
                uint32_t mx = 0u;
#pragma unroll
                for (int w = 0; w < 8; ++w) mx = max(mx, smax[i * W + (gr << lw) + (w & ((1 << lw) - 1))]);
                const RowScale s = row_scale(mx);
                if (tid == 0) sscale[r] = s.scale;
                if (in) *(uint2 *)(sq + (size_t)r * LD + 8 * tid) = quant8(v[i], s);
            }
        }
        __syncthreads();
    }
}

template <int ACT, int NS, int W, int U, bool Q>
__global__ __launch_bounds__(64 * W) void k_w8a8_stream(Args p) {
    static_assert(!Q || W == 8, "the fused quantisation gives each thread 8 of 4096 elements");
    __shared__ int sred[W * NS * 256];
    __shared__ int srow[16];
    __shared__ float sscale[16];
    __shared__ uint32_t smax[kQuantRows * W];
    extern __shared__ __attribute__((aligned(16))) int8_t sq[];  // Q: codes [rows][K + 16]
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
            if (kb0 + u * W + wave < KB) {
                const uint32_t off = (uint32_t)(kb0 + u * W + wave) * kBlockBytes + 16 * l;
#pragma unroll
                for (int j = 0; j < NS; ++j) b[u][j] = __builtin_nontemporal_load((const u32x4 *)(wb[j] + off));
            }
        }
    };
    load_b(0);
    // the source row of each row of the tile (-1: none) and its scale
    if (tid < 16) {
        int src = -1;
        if (tid < it.mrows) {
            src = it.m0 + tid;
            if (p.gather) {
                const int t = p.gather[it.m0 + tid];
                src = (unsigned)t < (unsigned)p.n_src ? t : -1;
            }
        }
        srow[tid] = src;
        if (!Q) sscale[tid] = p.as[max(src, 0)];
    }
    __syncthreads();
    v4i acc[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[j] = v4i{0, 0, 0, 0};

    if constexpr (Q) {
        const int LD = K + 16;
        quantise_rows<W>(p.x, K, it.mrows, [&](int r) { return srow[r]; }, sq, sscale, smax);
        const int8_t *ar = sq + (size_t)min(m, it.mrows - 1) * LD + 16 * q;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = u * W + wave;
            if (kb < KB) {
                // past the end of a row: any of its bytes, the weights there are zero
                const u32x4 av = *(const u32x4 *)(ar + min(64 * kb, K - 16 - 16 * q));
#pragma unroll
                for (int j = 0; j < NS; ++j) acc[j] = mfma_i8(b[u][j], av, acc[j]);
            }
        }
    } else {
        const int8_t *ar = p.a + (size_t)max(srow[m], 0) * K;
        for (int kb0 = 0;;) {
            u32x4 av[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (kb0 + u * W + wave < KB)
                    av[u] = *(const u32x4 *)(ar + min(64 * (kb0 + u * W + wave) + 16 * q, K - 16));
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (kb0 + u * W + wave < KB) {
#pragma unroll
                    for (int j = 0; j < NS; ++j) acc[j] = mfma_i8(b[u][j], av[u], acc[j]);
                }
            kb0 += U * W;
            if (kb0 >= KB) break;
            load_b(kb0);
        }
    }
    // the waves' partial sums: [wave][j][lane][i]
#pragma unroll
    for (int j = 0; j < NS; ++j) *(v4i *)&sred[(wave * NS + j) * 256 + 4 * l] = acc[j];
    __syncthreads();
    constexpr int NO = ACT == MOE_ACT_SWIGLU ? NS / 2 : NS;  // output subtiles
    if (tid < NO * 64) {
        const int j = tid >> 6, r = l & 15, qq = l >> 4;
        if (r >= it.mrows) return;
        v4i s0 = v4i{0, 0, 0, 0}, s1 = v4i{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < W; ++w) {
            s0 += *(const v4i *)&sred[(w * NS + j) * 256 + 4 * l];
            if (ACT == MOE_ACT_SWIGLU) s1 += *(const v4i *)&sred[(w * NS + j + NS / 2) * 256 + 4 * l];
        }
        const int t = ACT == MOE_ACT_SWIGLU ? it.nb * (NS / 2) + j : it.nb * NS + j;
        const int n = packed_row(t, 4 * qq);
        const int NC = ACT == MOE_ACT_SWIGLU ? p.N >> 1 : p.N;
        if (n >= NC) return;
        const int src = srow[r];
        const float sa = sscale[r];
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

// ---------------------------------------------------------------- down + combine
// Few rows of h (R = T (k + ns) <= 16): the down product and the combine in
// one launch.  A workgroup takes one subtile (16 output channels) of every
// row's expert, two waves per row (and the one eight later), each half of K,
// so that every slot of a token meets in one workgroup: it quantises all rows
// of h, streams each row's own weights, rounds y as the separate product does
// and adds it up in moe_combine's order.  59 MB at hidden 4096, inter 2048, 7
// rows: 14.9 us, against 14.6 + 4.1 us and a launch with the combine apart.
constexpr int kCombineRows = 16;

struct CombineArgs {
    const int32_t *row_of_slot;
    const float *topk_w;
    int T, k, ns;
    uint16_t *out;
};

template <int U>
__global__ __launch_bounds__(1024) void k_w8a8_down_combine(Args p, CombineArgs c) {
    constexpr int W = 16;
    __shared__ float sscale[kCombineRows];
    __shared__ __attribute__((aligned(16))) int sacc[kCombineRows][2][16];
    __shared__ float sy[kCombineRows][16];
    __shared__ uint32_t smax[kQuantRows * W];
    __shared__ int sgroup[kCombineRows];
    extern __shared__ __attribute__((aligned(16))) int8_t sq[];  // codes [R][K + 16]
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id();
    const int q = l >> 4, t = blockIdx.x, K = p.K, KH = p.KB >> 1, R = p.R;
    const int half = wave & 1;
    // the group of row r: the number of group ends at or before it
    int lo[kGroupChunks], cnt[kGroupChunks];
    load_group_sizes(p.offsets, p.G, lo, cnt);
    auto group_of = [&](int r) {
        int g = 0;
#pragma unroll
        for (int i = 0; i < kGroupChunks; ++i) {
            const bool past = kWave * i + l < p.G && lo[i] + cnt[i] <= r;
            g += __popcll(__ballot(past));
        }
        return min(g, p.G - 1);
    };
    u32x4 b[U];
    auto load_b = [&](int g, int kb0) {  // k blocks kb0 .. of the wave's half
        const int8_t *wb = p.wq + (((size_t)g * p.NT + t) * p.KB + half * KH) * kBlockBytes + 16 * l;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (kb0 + u < KH) b[u] = __builtin_nontemporal_load((const u32x4 *)(wb + (size_t)(kb0 + u) * kBlockBytes));
    };
    int r = wave >> 1, g = group_of(r);
    if (r < R) load_b(g, 0);
    quantise_rows<W>(p.x, K, R, [](int i) { return i; }, sq, sscale, smax);
    for (; r < R; r += W / 2) {
        const int8_t *ar = sq + (size_t)r * (K + 16) + 16 * q;
        v4i acc = v4i{0, 0, 0, 0};
        if (r >= W / 2) {
            g = group_of(r);
            load_b(g, 0);
        }
        for (int kb0 = 0;;) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (kb0 + u < KH)  // past the end of a row: any of its bytes, the weights there are zero
                    acc = mfma_i8(b[u], *(const u32x4 *)(ar + min(64 * (half * KH + kb0 + u), K - 16 - 16 * q)), acc);
            kb0 += U;
            if (kb0 >= KH) break;
            load_b(g, kb0);
        }
        if ((l & 15) == 0) *(v4i *)&sacc[r][half][4 * q] = acc;  // every column of the result is this row
        if (l == 0) sgroup[r] = g;
    }
    __syncthreads();
    if (tid < 4 * R) {  // y: four channels of a row per thread
        const int yr = tid >> 2, e = 4 * (tid & 3), n = packed_row(t, e);
        const float *ws = p.ws + (size_t)sgroup[yr] * p.N + n;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] = f32_to_bf16((float)(sacc[yr][0][e + i] + sacc[yr][1][e + i]) * sscale[yr] * ws[i]);
            sy[yr][e + i] = __uint_as_float(o[i] << 16);
        }
        *(uint2 *)(p.out + (size_t)yr * p.N + n) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
    }
    __syncthreads();
    if (tid < 16 * c.T) {
        const int tk = tid >> 4, e = tid & 15, S = c.k + c.ns;
        const int32_t *row = c.row_of_slot + (size_t)tk * S;
        float acc = 0.0f;
        if (c.ns && (unsigned)row[c.k] < (unsigned)R) acc = sy[row[c.k]][e];
        for (int j = 0; j < c.k; ++j)
            if ((unsigned)row[j] < (unsigned)R)
                acc = __builtin_fmaf(c.topk_w[(size_t)tk * c.k + j], sy[row[j]][e], acc);
        c.out[(size_t)tk * p.N + packed_row(t, e)] = f32_to_bf16(acc);
    }
}

void launch_down_combine(const Args &a, const CombineArgs &c, hipStream_t st) {
    const size_t lds = (size_t)a.R * (a.K + 16);
    if (a.KB <= 8)
        hipLaunchKernelGGL(k_w8a8_down_combine<4>, dim3(a.NT), dim3(1024), lds, st, a, c);
    else  // (16: registers spill)
        hipLaunchKernelGGL(k_w8a8_down_combine<8>, dim3(a.NT), dim3(1024), lds, st, a, c);
}

template <int ACT, int NS, int U, bool Q>
void launch_stream_u(Args a, int rows, hipStream_t st) {
    constexpr int W = 8;
    a.NB = (ACT == MOE_ACT_SWIGLU ? a.NT / 2 : a.NT) / (ACT == MOE_ACT_SWIGLU ? NS / 2 : NS);
    const int TM = Q ? rows : 16;
    a.qrows = rows;
    int64_t tiles = a.offsets ? (int64_t)a.R / TM + (a.R < a.G ? a.R : a.G) : (a.R + TM - 1) / TM;
    if (tiles > a.R) tiles = a.R;  // every tile has a row
    const dim3 grid((unsigned)((tiles * a.NB + 7) / 8 * 8));
    const size_t lds = Q ? (size_t)rows * (a.K + 16) : 0;
    hipLaunchKernelGGL((k_w8a8_stream<ACT, NS, W, U, Q>), grid, dim3(64 * W), lds, st, a);
}

// U: the k blocks that each wave has in flight, as many as K gives it (up to 8)
template <int ACT, int NS, bool Q>
void launch_stream(const Args &a, int rows, hipStream_t st) {
    if (a.KB <= 16)
        launch_stream_u<ACT, NS, 2, Q>(a, rows, st);
    else if (a.KB <= 32)
        launch_stream_u<ACT, NS, 4, Q>(a, rows, st);
    else
        launch_stream_u<ACT, NS, 8, Q>(a, rows, st);
}

// Where a product's workgroups quantise its few rows for themselves instead of
// a launch before.  Dense: up to 4 rows, and as many as quantise_rows takes in
// one pass, half of that past 8192 columns, where a CU has several workgroups
// (captured / called one by one, us, against two launches: 4096 x 1024 at 8
// rows 4.2 / 6.1 against 5.3 / 8.5, at 16 5.2 / 6.1 against 5.5 / 8.6; 4096 x
// 2048 at 8 5.4 / 6.1 against 6.1 / 8.4, at 12 6.8 / 6.7 against 6.2 / 8.5;
// 16384 x 2048 at 8 9.6 / 9.3 against 8.4 / 8.4; 4096 x 4096 at 4 6.1 / 6.1
// against 8.1 / 8.3, at 8 8.5 / 8.5 against 8.1 / 8.3).
bool fuse_dense(int M, int N, int K) {
    if (K > kFusedMaxK) return false;
    return M <= 4 || (M <= 16 && M << log2_waves_per_row(K) <= (N <= 8192 ? 32 : 16));
}
// Experts: up to 4 tokens, and up to 16 (12 with longer rows) where the weights
// are few: then the five launches' latency counts, else the tiled products
// stream the weights faster (hidden 1024, inter 512, 17 groups, 27 MB: 15.7
// against 17.1 us captured, 16.1 against 20.6 called one by one at 8 tokens,
// 17.9 / 18.2 against 17.5 / 20.5 at 16; hidden 4096, inter 128, 12 groups:
// 13.7 against 21.1 at 12; hidden 2048, inter 256, 9 groups: 13.6 against 18.4
// at 5, 18.7 against 18.6 at 12, 21.0 against 18.8 at 16; hidden 2048, inter
// 512, 25 groups, 79 MB: 26.9 against 25.1 at 12; the layer at hidden 4096: 42
// against 49 at 1 token, 126 against 131 at 4, 149 against 125 at 5).
bool fuse_experts(int T, int G, int H, int I) {  // H and I are at most 4096 = kFusedMaxK
    return T <= 4 || (T <= (H <= 1024 ? 16 : 12) && (size_t)3 * G * H * I <= (size_t)32 << 20);
}
// Rows up to which the weight stream is the faster kernel.  Dense, 4096 x
// 4096: 6.2 against 9.5 us at 16 rows.  Grouped: the tiled kernel needs no
// more bytes and has more of them in flight (the layer's experts: 207 against
// 220 us at 8 tokens, 354 against 380 at 16).
constexpr int kStreamRows = 16, kStreamRowsGrouped = 4;

// rows: an upper bound of the rows of one group
void launch_gemm(int act, const Args &a, int rows, hipStream_t st) {
    const bool swiglu = act == MOE_ACT_SWIGLU;
    // two subtiles per workgroup, or one where two would leave CUs without
    // work (4096 columns: 5.5 against 6.2 us; 8192: 4.8 against 4.7)
    const bool one = !swiglu && !a.offsets && a.NT <= 256;
    if (a.x) {
        swiglu ? launch_stream<MOE_ACT_SWIGLU, 2, true>(a, rows, st)
        : one  ? launch_stream<MOE_ACT_NONE, 1, true>(a, rows, st)
               : launch_stream<MOE_ACT_NONE, 2, true>(a, rows, st);
    } else if (rows <= (a.offsets ? kStreamRowsGrouped : kStreamRows)) {
        swiglu ? launch_stream<MOE_ACT_SWIGLU, 2, false>(a, rows, st)
        : one  ? launch_stream<MOE_ACT_NONE, 1, false>(a, rows, st)
               : launch_stream<MOE_ACT_NONE, 2, false>(a, rows, st);
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
    constexpr int most = 1 << 21;  // of 1024 threads a row: fewer than 2^32 in a launch
    for (int r = 0; r < rows; r += most) {
        w8::launch_quant(std::min(most, rows - r), K, a + (size_t)r * K, codes + (size_t)r * K, scales + r,
                         (hipStream_t)stream);
        MOE_TRY(launch_status());
    }
    return MOE_OK;
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
    // up to 2^31 threads in a launch (a group has at most 2^28)
    const size_t pieces = bytes / 16 / n_groups, out = bytes / n_groups;
    const int most = (int)std::min<size_t>(n_groups, ((size_t)1 << 31) / pieces);
    for (int g = 0; g < n_groups; g += most) {
        hipLaunchKernelGGL(w8::k_w8a8_prepack, dim3((unsigned)((pieces + 255) / 256), std::min(most, n_groups - g)),
                           dim3(256), 0, (hipStream_t)stream, w_canonical + (size_t)g * N * K, w_packed + g * out, N, K,
                           w8::subtiles(N), w8::kblocks(K));
        MOE_TRY(launch_status());
    }
    return MOE_OK;
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
    if (w8::fuse_dense(M, N, K)) {
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
    const bool fused = w8::fuse_experts(T, G, H, I);
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
        if (R <= w8::kCombineRows) {
            w8::launch_down_combine(d, {row_of_slot, topk_w, T, desc->top_k, desc->n_shared, out}, st);
            return launch_status();
        }
    } else {
        w8::launch_quant(R, I, h, hq, hqs, st);
        d.a = hq;
        d.as = hqs;
    }
    w8::launch_gemm(MOE_ACT_NONE, d, T, st);
    MOE_TRY(launch_status());
    return moe_combine(desc, T, y, row_of_slot, topk_w, out, stream);
}
