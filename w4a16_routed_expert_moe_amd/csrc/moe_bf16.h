// moe_bf16.h -- what the kernels of the bf16 experts share: the launch
// arguments of the grouped products and the entries to their kernels.
#pragma once

#include "moe_gemm_common.h"

namespace moe {
namespace b16 {

// The three products over the permuted rows of each group g:
//   kNT  c[r][n] = sum_k a[r][k] b_g[n][k]      (forward: b the weights)
//   kNN  c[r][n] = sum_k a[r][k] b_g[k][n]      (gradient of the rows)
//   kTN  c_g[m][n] = sum_r a[r][m] b[r][n]      (gradient of the weights)
enum { kNT = 0, kNN = 1, kTN = 2 };

// What is done with a finished tile.
enum {
    kStore = 0,      // bf16(c)
    kSwiglu = 1,     // kNT: bf16(silu(gate) * up), and bf16 of both where gu is given
    kSwigluBwd = 2,  // kNN: the gradients behind the activation (see moe_bf16_tiled.hip)
    kStoreF32 = 3,   // kTN: c in fp32
    kAddF32 = 4      // kTN: added to the fp32 values there
};

struct Args {
    const uint16_t *a;        // kNT, kNN: [n_src or R][K]; kTN: [n_src or R][M]
    const int32_t *gather;    // row r reads a[gather[r]] (null: a[r]); a row outside [0, n_src) is zeros
    const uint16_t *b;        // kNT: [G][N][K]; kNN: [G][K][N]; kTN: [R][N]
    int n_src;
    const int32_t *offsets;   // [G+1]
    int G, R, M, N, K;        // (K: kNT, kNN; M: kTN)
    bool swap;                // kTN: c_g is written transposed
    void *out;                // [R][N], [R][N/2] (kSwiglu), [G][M][N] or (swap) [G][N][M]
    uint16_t *gu;             // kSwiglu: [R][N] or null
    // kSwigluBwd (N columns of h)
    const uint16_t *gu_in, *h;  // [R][2N], [R][N]
    const int32_t *row_of_slot;  // [T][k + ns]; row r is one of token gather[r]'s
    const float *topk_w;         // [T][k]
    int k, ns;
    uint16_t *dgu, *hw;         // [R][2N], [R][N]; null: not wanted
    float *part;                // [NB][R]
    int MB, NB;                 // tiles along M (kTN) and N, set by the launch
};

void launch_stream(int epi, const Args &p, hipStream_t st);  // moe_bf16.hip: kNT, a few rows per group
void launch_tiled(int epi, const Args &p, hipStream_t st);   // moe_bf16_tiled.hip: kNT, few rows of many weights
// moe_bf16_wide.hip: everything else.  Returns the number of column blocks
// (kSwigluBwd: of partial sums per row), at most ceil(N / 128).
int launch_wide(int form, int epi, const Args &p, hipStream_t st);
// The gradients of the rows (kNN) and of both weights (kTN, the first one
// swapped) in one launch; false, and nothing launched, where three are faster.
bool launch_gradients(int epi, const Args &x, const Args &w13, const Args &w2, hipStream_t st);

// What the gradient d of one element of h (before the routing weight w) gives:
// h = silu(g) u with s = sigmoid(g), silu'(g) = s (1 + g (1 - s)).
__device__ __forceinline__ void swiglu_gradient(float d, float w, float g, float u, float h, float &dot, float &dg,
                                                float &du, float &hw) {
    const float dw = d * w, s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
    dot = __builtin_fmaf(d, h, dot);
    dg = dw * u * s * (1.0f + g * (1.0f - s));
    du = dw * g * s;
    hw = h * w;
}

}  // namespace b16
}  // namespace moe
