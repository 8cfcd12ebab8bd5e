// moe_bf16.hip -- the experts in bf16, forward and backward: the ABI entry
// points and the kernels beside the products (moe_bf16_tiled.hip).
#include <algorithm>

#include "moe_bf16.h"

namespace moe {
namespace b16 {
namespace {

// d_x[t] = sum over the slots of t of dxs[row] (fp32, slot order), and
// d_topk_w[t][j] = the sum of its row's partial sums over NB column blocks.
__global__ __launch_bounds__(256) void k_slot_sums(const uint16_t *__restrict__ dxs, const float *__restrict__ part,
                                                   const int32_t *__restrict__ row_of_slot, int H, int k, int ns, int R,
                                                   int NB, uint16_t *__restrict__ d_x, float *__restrict__ d_topk_w) {
    const int t = blockIdx.x, S = k + ns, tid = threadIdx.x;
    if (d_topk_w && blockIdx.y == 0 && tid < k) {
        const int r = row_of_slot[(size_t)t * S + tid];
        float s = 0.0f;
        if ((unsigned)r < (unsigned)R)
            for (int b = 0; b < NB; ++b) s += part[(size_t)b * R + r];
        d_topk_w[(size_t)t * k + tid] = s;
    }
    const int h0 = (blockIdx.y * 256 + tid) * 8;
    if (!d_x || h0 >= H) return;
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < S; ++j) {
        const int r = row_of_slot[(size_t)t * S + j];
        if ((unsigned)r >= (unsigned)R) continue;
        const u32x4 v = *(const u32x4 *)(dxs + (size_t)r * H + h0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[2 * i] += bf16lo_to_f32(v[i]);
            acc[2 * i + 1] += bf16hi_to_f32(v[i]);
        }
    }
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
    *(u32x4 *)(d_x + (size_t)t * H + h0) = o;
}

// ---------------------------------------------------------------- weight stream
// kNT with few rows per group: the weights' bytes are the bound.  A workgroup
// of eight waves takes NS subtiles (16 weight rows each; SwiGLU: NS/2 of the
// gate and the same NS/2 of the up projection) and at most 16 rows of one
// group; the waves split K by blocks of 64: wave w takes blocks w, w + 8, ...,
// two of them in flight; every weight byte goes straight from HBM into the
// registers of the one wave that multiplies it (32 consecutive bytes a lane,
// so that a row's 128 are read together), and the waves' partial sums meet in
// LDS.  1 token of the 256-expert layer of 4096/2048 (7 groups; NS = 4, 2, 1):
// gate/up 50, 51 us, down 34, 30, 27, 4.7 and 4.3 TB/s; with all of a wave's blocks
// in flight at once, a workgroup per CU, 60 and 30.
constexpr int kStreamWaves = 8, U = 2;

template <int EPI, int NS>
__global__ __launch_bounds__(64 * kStreamWaves) void k_bf16_stream(Args p) {
    __shared__ float sred[kStreamWaves * NS * 256];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id();
    const int m = l & 15, q = l >> 4;
    TileItem it;
    if (!workgroup_tile_item(p.NB, 16, p.offsets, p.G, p.R, it)) return;
    const int K = p.K, KB = (K + 63) >> 6, half = p.N >> 1;
    constexpr int NO = EPI == kSwiglu ? NS / 2 : NS;  // output subtiles
    const int cols = EPI == kSwiglu ? half : p.N;
    const uint16_t *w[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = min((it.nb * NO + j % NO) * 16 + m, cols - 1) + (j >= NO ? half : 0);
        w[j] = p.b + ((size_t)it.g * p.N + n) * K + 16 * q;
    }
    int src = it.m0 + min(m, it.mrows - 1);
    bool live = true;  // a row without a source is zeros
    if (p.gather) {
        src = p.gather[src];
        live = (unsigned)src < (unsigned)p.n_src;
        if (!live) src = 0;
    }
    const uint16_t *x = p.a + (size_t)src * K + 16 * q;
    f32x4 acc[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb0 = wave; kb0 < KB; kb0 += U * kStreamWaves) {
        u32x4 b[U][NS][2], a[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * kStreamWaves;
            // past the end of a row: zeros (a multiple of 16 is left of it)
            if (kb < KB && 64 * kb + 16 * q < K) {
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    const u32x4 *at = (const u32x4 *)(w[j] + 64 * kb);
                    b[u][j][0] = __builtin_nontemporal_load(at);
                    b[u][j][1] = __builtin_nontemporal_load(at + 1);
                }
                const u32x4 *at = (const u32x4 *)(x + 64 * kb);
                a[u][0] = at[0];
                a[u][1] = at[1];
            } else {
#pragma unroll
                for (int j = 0; j < NS; ++j) b[u][j][0] = b[u][j][1] = u32x4{0u, 0u, 0u, 0u};
                a[u][0] = a[u][1] = u32x4{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    acc[j] = mfma16(__builtin_bit_cast(bf16x8, b[u][j][h]), __builtin_bit_cast(bf16x8, a[u][h]), acc[j]);
    }
    // the waves' partial sums: [wave][j][lane][i]
#pragma unroll
    for (int j = 0; j < NS; ++j) *(f32x4 *)&sred[(wave * NS + j) * 256 + 4 * l] = acc[j];
    __syncthreads();
    if (tid < NO * 64) {
        const int j = tid >> 6;
        f32x4 s0 = f32x4{0.0f, 0.0f, 0.0f, 0.0f}, s1 = s0;
#pragma unroll
        for (int v = 0; v < kStreamWaves; ++v) {
            const f32x4 g = *(const f32x4 *)&sred[(v * NS + j) * 256 + 4 * l];
            const f32x4 u = EPI == kSwiglu ? *(const f32x4 *)&sred[(v * NS + j + NO) * 256 + 4 * l] : g;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s0[e] += live ? g[e] : 0.0f;
                s1[e] += live ? u[e] : 0.0f;
            }
        }
        const int n = (it.nb * NO + j) * 16 + 4 * q;
        if (m >= it.mrows || n >= cols) return;
        const size_t row = (size_t)it.m0 + m;
        const uint2 g = make_uint2(pack_bf16x2(s0[0], s0[1]), pack_bf16x2(s0[2], s0[3]));
        if constexpr (EPI == kSwiglu) {
            *(uint2 *)((uint16_t *)p.out + row * cols + n) =
                make_uint2(pack_bf16x2(silu_mul(s0[0], s1[0]), silu_mul(s0[1], s1[1])),
                           pack_bf16x2(silu_mul(s0[2], s1[2]), silu_mul(s0[3], s1[3])));
            if (p.gu) {
                *(uint2 *)(p.gu + row * p.N + n) = g;
                *(uint2 *)(p.gu + row * p.N + half + n) = make_uint2(pack_bf16x2(s1[0], s1[1]), pack_bf16x2(s1[2], s1[3]));
            }
        } else {
            *(uint2 *)((uint16_t *)p.out + row * cols + n) = g;
        }
    }
}

template <int EPI, int NS>
void launch_stream(Args p, hipStream_t st) {
    constexpr int NO = EPI == kSwiglu ? NS / 2 : NS;
    const int cols = EPI == kSwiglu ? p.N / 2 : p.N;
    p.NB = (cols + 16 * NO - 1) / (16 * NO);
    const int64_t tiles = std::min<int64_t>((int64_t)p.R / 16 + std::min(p.R, p.G), p.R);
    hipLaunchKernelGGL((k_bf16_stream<EPI, NS>), dim3((unsigned)((tiles * p.NB + 7) / 8 * 8)), dim3(64 * kStreamWaves), 0,
                       st, p);
}

}  // namespace

void launch_stream(int epi, const Args &p, hipStream_t st) {
    epi == kSwiglu ? launch_stream<kSwiglu, 4>(p, st) : launch_stream<kStore, 1>(p, st);
}

namespace {

// ---------------------------------------------------------------- host side
bool size_ok(int32_t n) { return n >= 16 && n <= 65536 && n % 16 == 0; }

Args make_args(const moe_layer_desc *d, int32_t T, int N, int K, const int32_t *offsets) {
    Args p{};
    p.G = d->n_routed + d->n_shared;
    p.R = T * (d->top_k + d->n_shared);
    p.N = N;
    p.K = K;
    p.offsets = offsets;
    return p;
}

// The forward product, by measured times (us; stream, 64 x 256 tiles, 64 x 128
// tiles; rows, groups, layer):
//   gate/up   7 of 257, 4096/2048  50, 67, 59    28  144, 156, 151    112  453, 451, 537    448, skewed  1049, 700, 799
//            64 of  41, 1024/512   16, 21, 19   240   23,  21,  21
//           150 of  65, 2048/768   75, 91, 87  1500  152,  99, 139   5000   374, 120, 130
//            60 of  17, 512/256   7.9, 13, 10
//   down      7 of 257, 4096/2048  27, 36, 32    14   43,  36,  37    112  272, 223, 260
//            64 of  41, 1024/512   13, 12, 10;  60 of 17, 512/256  5.7, 8.5, 6.4
//           150 of  65, 2048/768   54, 31, 39  1500  133,  45,  42
// The stream reads a group's weights again for every 16 of its rows and starts
// at once; the tiles whose weights go straight into registers
// (moe_bf16_tiled.hip) are for the few rows of many weights.
void launch_forward(int epi, const Args &p, hipStream_t st) {
    const int64_t weights = (int64_t)p.G * p.N * p.K * 2, G = p.G, MB = 1 << 20;
    const bool stream = epi == kSwiglu ? p.R <= 32 || (p.R <= 3 * G && weights <= 512 * MB)
                                       : p.R <= 8 || (p.R <= 4 * G && weights <= 32 * MB);
    if (stream)
        launch_stream(epi, p, st);
    else if (p.R < 64 * G && weights >= 64 * MB)
        launch_tiled(epi, p, st);
    else
        launch_wide(kNT, epi, p, st);
}

int gradient_epi(int32_t mode) { return mode == MOE_GRAD_BF16 ? kStore : mode == MOE_GRAD_F32 ? kStoreF32 : kAddF32; }

// dw_g[n][k]: whichever operand is gathered goes through LDS row by row (a),
// the other by consecutive rows (b); the result is written transposed where
// that is the second.
Args weight_args(const moe_layer_desc *d, int32_t T, const uint16_t *dy, const int32_t *dy_gather, const uint16_t *a,
                 const int32_t *a_gather, int n_src, int N, int K, const int32_t *offsets, void *dw) {
    const bool swap = a_gather != nullptr;
    Args p = make_args(d, T, swap ? N : K, 0, offsets);
    p.swap = swap;
    p.M = swap ? K : N;
    p.a = swap ? a : dy;
    p.gather = swap ? a_gather : dy_gather;
    p.b = swap ? dy : a;
    p.n_src = n_src;
    p.out = dw;
    return p;
}

// The workspace of the backward pass: where each part begins.
struct Workspace {
    size_t dgu, hw, dxs, part, bytes;
};
Workspace workspace(const moe_layer_desc *d, int32_t T) {
    const size_t R = (size_t)T * (d->top_k + d->n_shared), I = d->inter, H = d->hidden;
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    Workspace w;
    w.dgu = 0;
    w.hw = w.dgu + up(R * 2 * I * 2);
    w.dxs = w.hw + up(R * I * 2);
    w.part = w.dxs + up(R * H * 2);
    w.bytes = w.part + up(R * ((I + 127) / 128) * 4);
    return w;
}

}  // namespace
}  // namespace b16
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_bf16_grouped_gemm(const moe_layer_desc *desc, int32_t T, const uint16_t *a,
                                            const int32_t *a_gather, int32_t n_src, int32_t N, int32_t K,
                                            const uint16_t *w, const int32_t *group_offsets, int32_t act,
                                            uint16_t *gu, uint16_t *out, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_tokens(T));
    if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return MOE_ERR_UNSUPPORTED;
    if (!b16::size_ok(N) || !b16::size_ok(K) || (act == MOE_ACT_SWIGLU && N % 32)) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!a || !w || !group_offsets || !out) return MOE_ERR_NULL;
    if (a_gather && (n_src < 1 || n_src > MOE_MAX_TOKENS)) return MOE_ERR_SHAPE;
    if (!aligned(a, 16) || !aligned(a_gather, 4) || !aligned(w, 16) || !aligned(group_offsets, 4) || !aligned(gu, 16) ||
        !aligned(out, 16))
        return MOE_ERR_ALIGN;
    b16::Args p = b16::make_args(desc, T, N, K, group_offsets);
    p.a = a;
    p.gather = a_gather;
    p.n_src = n_src;
    p.b = w;
    p.out = out;
    p.gu = act == MOE_ACT_SWIGLU ? gu : nullptr;
    b16::launch_forward(act == MOE_ACT_SWIGLU ? b16::kSwiglu : b16::kStore, p, (hipStream_t)stream);
    return launch_status();
}

extern "C" moe_status moe_bf16_grouped_dgrad(const moe_layer_desc *desc, int32_t T, const uint16_t *dy,
                                             const int32_t *dy_gather, int32_t n_src, int32_t N, int32_t K,
                                             const uint16_t *w, const int32_t *group_offsets, uint16_t *da,
                                             void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_tokens(T));
    if (!b16::size_ok(N) || !b16::size_ok(K)) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!dy || !w || !group_offsets || !da) return MOE_ERR_NULL;
    if (dy_gather && (n_src < 1 || n_src > MOE_MAX_TOKENS)) return MOE_ERR_SHAPE;
    if (!aligned(dy, 16) || !aligned(dy_gather, 4) || !aligned(w, 16) || !aligned(group_offsets, 4) || !aligned(da, 16))
        return MOE_ERR_ALIGN;
    b16::Args p = b16::make_args(desc, T, K, N, group_offsets);  // K columns out, N summed over
    p.a = dy;
    p.gather = dy_gather;
    p.n_src = n_src;
    p.b = w;
    p.out = da;
    b16::launch_wide(b16::kNN, b16::kStore, p, (hipStream_t)stream);
    return launch_status();
}

extern "C" moe_status moe_bf16_grouped_wgrad(const moe_layer_desc *desc, int32_t T, const uint16_t *dy,
                                             const int32_t *dy_gather, const uint16_t *a, const int32_t *a_gather,
                                             int32_t n_src, int32_t N, int32_t K, const int32_t *group_offsets,
                                             int32_t mode, void *dw, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_tokens(T));
    if (mode != MOE_GRAD_BF16 && mode != MOE_GRAD_F32 && mode != MOE_GRAD_F32_ADD) return MOE_ERR_UNSUPPORTED;
    if (!b16::size_ok(N) || !b16::size_ok(K)) return MOE_ERR_SHAPE;
    if (dy_gather && a_gather) return MOE_ERR_UNSUPPORTED;
    if (T == 0 && mode == MOE_GRAD_F32_ADD) return MOE_OK;
    if (!group_offsets || !dw || (T > 0 && (!dy || !a))) return MOE_ERR_NULL;
    if ((dy_gather || a_gather) && T > 0 && (n_src < 1 || n_src > MOE_MAX_TOKENS)) return MOE_ERR_SHAPE;
    if (!aligned(dy, 16) || !aligned(dy_gather, 4) || !aligned(a, 16) || !aligned(a_gather, 4) ||
        !aligned(group_offsets, 4) || !aligned(dw, 16))
        return MOE_ERR_ALIGN;
    b16::launch_wide(b16::kTN, b16::gradient_epi(mode),
                     b16::weight_args(desc, T, dy, dy_gather, a, a_gather, n_src, N, K, group_offsets, dw), (hipStream_t)stream);
    return launch_status();
}

extern "C" moe_status moe_bf16_experts(const moe_layer_desc *desc, int32_t T, const uint16_t *x, const float *topk_w,
                                       const int32_t *group_offsets, const int32_t *sorted_token,
                                       const int32_t *row_of_slot, const uint16_t *w13, const uint16_t *w2, uint16_t *gu,
                                       uint16_t *h, uint16_t *y, uint16_t *out, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_tokens(T));
    if (T == 0) return MOE_OK;
    if (!x || !topk_w || !group_offsets || !sorted_token || !row_of_slot || !w13 || !w2 || !h || !y || !out)
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(topk_w, 4) || !aligned(group_offsets, 4) || !aligned(sorted_token, 4) ||
        !aligned(row_of_slot, 4) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(gu, 16) || !aligned(h, 16) ||
        !aligned(y, 16) || !aligned(out, 16))
        return MOE_ERR_ALIGN;
    const int H = desc->hidden, I = desc->inter;
    MOE_TRY(moe_bf16_grouped_gemm(desc, T, x, sorted_token, T, 2 * I, H, w13, group_offsets, MOE_ACT_SWIGLU, gu, h, stream));
    MOE_TRY(moe_bf16_grouped_gemm(desc, T, h, nullptr, 0, H, I, w2, group_offsets, MOE_ACT_NONE, nullptr, y, stream));
    return moe_combine(desc, T, y, row_of_slot, topk_w, out, stream);
}

extern "C" size_t moe_bf16_backward_workspace_bytes(const moe_layer_desc *desc, int32_t T) {
    if (check_desc(desc) != MOE_OK || check_tokens(T) != MOE_OK) return 0;
    return b16::workspace(desc, T).bytes;
}

extern "C" moe_status moe_bf16_experts_backward(const moe_layer_desc *desc, int32_t T, const uint16_t *d_out,
                                                const uint16_t *x, const float *topk_w, const int32_t *group_offsets,
                                                const int32_t *sorted_token, const int32_t *row_of_slot,
                                                const uint16_t *w13, const uint16_t *w2, const uint16_t *gu,
                                                const uint16_t *h, int32_t mode, uint16_t *d_x, void *d_w13, void *d_w2,
                                                float *d_topk_w, void *ws, size_t ws_bytes, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_tokens(T));
    if (mode != MOE_GRAD_BF16 && mode != MOE_GRAD_F32 && mode != MOE_GRAD_F32_ADD) return MOE_ERR_UNSUPPORTED;
    const int H = desc->hidden, I = desc->inter, k = desc->top_k, ns = desc->n_shared;
    if (!aligned(d_out, 16) || !aligned(x, 16) || !aligned(topk_w, 4) || !aligned(group_offsets, 4) ||
        !aligned(sorted_token, 4) || !aligned(row_of_slot, 4) || !aligned(w13, 16) || !aligned(w2, 16) ||
        !aligned(gu, 16) || !aligned(h, 16) || !aligned(d_x, 16) || !aligned(d_w13, 16) || !aligned(d_w2, 16) ||
        !aligned(d_topk_w, 4) || !aligned(ws, 16))
        return MOE_ERR_ALIGN;
    hipStream_t st = (hipStream_t)stream;
    const uint16_t *dgu = nullptr, *hw = nullptr;
    bool done = false;  // with the weights' gradients
    if (T > 0) {
        if (!d_out || !x || !topk_w || !group_offsets || !sorted_token || !row_of_slot || !w13 || !w2 || !gu || !h || !ws)
            return MOE_ERR_NULL;
        const b16::Workspace at = b16::workspace(desc, T);
        if (ws_bytes < at.bytes) return MOE_ERR_WORKSPACE;
        if (!d_x && !d_w13 && !d_w2 && !d_topk_w) return MOE_OK;
        char *base = (char *)ws;
        const int R = T * (k + ns);
        float *part = (float *)(base + at.part);
        uint16_t *dxs = (uint16_t *)(base + at.dxs);
        // dh = d_out W2 and what follows from it
        b16::Args p = b16::make_args(desc, T, I, H, group_offsets);
        p.a = d_out;
        p.gather = sorted_token;
        p.n_src = T;
        p.b = w2;
        p.gu_in = gu;
        p.h = h;
        p.row_of_slot = row_of_slot;
        p.topk_w = topk_w;
        p.k = k;
        p.ns = ns;
        p.dgu = d_x || d_w13 ? (uint16_t *)(base + at.dgu) : nullptr;
        p.hw = d_w2 ? (uint16_t *)(base + at.hw) : nullptr;
        p.part = part;
        const int NB = b16::launch_wide(b16::kNN, b16::kSwigluBwd, p, st);
        dgu = p.dgu;
        hw = p.hw;
        b16::Args q = b16::make_args(desc, T, H, 2 * I, group_offsets);
        q.a = dgu;
        q.b = w13;
        q.out = dxs;
        if (d_x && d_w13 && d_w2)
            done = b16::launch_gradients(
                b16::gradient_epi(mode), q, b16::weight_args(desc, T, dgu, nullptr, x, sorted_token, T, 2 * I, H, group_offsets, d_w13),
                b16::weight_args(desc, T, d_out, sorted_token, hw, nullptr, T, H, I, group_offsets, d_w2), st);
        if (d_x && !done) b16::launch_wide(b16::kNN, b16::kStore, q, st);
        if (d_x || d_topk_w)
            hipLaunchKernelGGL(b16::k_slot_sums, dim3(T, d_x ? (H + 2047) / 2048 : 1), dim3(256), 0, st, dxs, part,
                               row_of_slot, H, k, ns, R, NB, d_x, d_topk_w);
        MOE_TRY(launch_status());
    }
    if (done || (!d_w13 && !d_w2) || (T == 0 && mode == MOE_GRAD_F32_ADD)) return MOE_OK;
    if (!group_offsets) return MOE_ERR_NULL;
    if (d_w13)
        b16::launch_wide(b16::kTN, b16::gradient_epi(mode),
                         b16::weight_args(desc, T, dgu, nullptr, x, sorted_token, T, 2 * I, H, group_offsets, d_w13), st);
    if (d_w2)
        b16::launch_wide(b16::kTN, b16::gradient_epi(mode),
                         b16::weight_args(desc, T, d_out, sorted_token, hw, nullptr, T, H, I, group_offsets, d_w2), st);
    return launch_status();
}
