// moe_w8a8.h -- what the W8A8 (INT8 weights, INT8 activations) kernels share:
// the packed weight layout, the launch arguments, the quantisation of one
// row's elements, and the entry to the LDS-tiled kernel.
#pragma once

#include "moe_gemm_common.h"

namespace moe {
namespace w8 {

typedef int v4i __attribute__((ext_vector_type(4)));

// Packed weights.  One 1 KB block per (16-row subtile, 64-wide k block): lane
// l of a wave owns bytes [16l, 16l+16), the instruction's operand of row
// r = l % 16 and k = 64 kb + 16 (l / 16) + [0, 16).  Four subtiles share 64
// consecutive weight rows: row r = 4q + i of subtile 4 st + j is weight row
// n = 64 st + 16 q + 4 j + i, so that lane (m, q) of the four results holds
// the 16 consecutive outputs n = 64 st + 16 q + [0, 16) of token m and stores
// them as two 16-byte words, four lanes filling a 128-byte line (with the
// rows in order a store would write two bytes per lane).  N is padded with
// zero rows to a multiple of 64, K with zeros to a multiple of 128.
constexpr int kBlockBytes = 1024;
inline int subtiles(int N) { return (N + 63) / 64 * 4; }
inline int kblocks(int K) { return (K + 127) / 128 * 2; }
__host__ __device__ inline int packed_row(int t, int r) {  // the weight row of row r of subtile t
    return 64 * (t >> 2) + 16 * (r >> 2) + 4 * (t & 3) + (r & 3);
}

struct Args {
    const int8_t *a;         // int8 codes [n_src or R][K]
    const float *as;         // fp32 [n_src or R]
    const uint16_t *x;       // fused quantisation: bf16 rows instead of a, as
    const int32_t *gather;   // row r reads a[gather[r]] (or null: a[r])
    int n_src;
    const int8_t *wq;        // packed weights
    const float *ws;         // fp32 [G][N]
    const int32_t *offsets;  // group offsets [G+1]; null: one group of rows [0, R)
    int G, R, N, K;
    uint16_t *out;           // bf16 [R][N] or [R][N/2] (SwiGLU)
    int KB, NT;              // 64-wide k blocks and 16-row subtiles per group in the packed weights
    int NB;                  // n-blocks (the instance's tile width)
    int qrows;               // fused quantisation: rows of a tile
};

__device__ __forceinline__ v4i mfma_i8(u32x4 a, u32x4 b, v4i c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), c, 0, 0, 0);
}

// The largest |x| of bf16 pairs, as bit patterns: for non-negative values
// the order of the patterns is the order of the values, infinities and NaNs
// above every finite one.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_max_abs(uint32_t m, uint32_t v) {
    const u16x2 a = __builtin_bit_cast(u16x2, m), b = __builtin_bit_cast(u16x2, v & 0x7FFF7FFFu);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
}

// One row's quantisation: scale = amax / 127 (fp32), code = 127 x / amax
// rounded to nearest, ties to even, exactly.  With amax = m 2^e (m in
// [1/2, 1)) and t = 127 (x 2^-e), all exact, the code is t / m rounded.
// Where 127 x / amax is not a tie it is at least 2^-17 of its size away
// from one (the quotient of a 15-bit and an 8-bit integer), far more than
// the error of q = t r, r ~ 1/m; where it is a tie, it is a float, and one
// correction step q + (t - q m) r returns it exactly.
// A row with an infinity or NaN gets a NaN scale and codes 0, a row of
// zeros scale 0 and codes 0.
struct RowScale {
    float m, r, scale;
    int e;
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {  // bf16 bits of max |x|
    RowScale s;
    if (amax_bits >= 0x7F80u) {
        s.m = 1.0f;
        s.r = 0.0f;
        s.e = 0;
        s.scale = __uint_as_float(0x7FC00000u);
        return s;
    }
    const float amax = __uint_as_float(amax_bits << 16);
    s.e = __builtin_amdgcn_frexp_expf(amax);
    s.m = __builtin_amdgcn_frexp_mantf(amax);
    s.r = amax_bits ? __builtin_amdgcn_rcpf(s.m) : 0.0f;
    s.scale = __fdiv_rn(amax, 127.0f);
    return s;
}
__device__ __forceinline__ uint32_t quant1(float x, const RowScale &s) {
    const float t = 127.0f * __builtin_amdgcn_ldexpf(x, -s.e);
    const float q = t * s.r;
    const float d = __builtin_fmaf(__builtin_fmaf(-q, s.m, t), s.r, q);
    // adding 1.5 * 2^23 rounds to the integer (nearest, ties to even) and
    // leaves it in the low bits
    return __float_as_uint(d + 12582912.0f);
}
// eight bf16 -> eight int8 codes
__device__ __forceinline__ uint2 quant8(u32x4 v, const RowScale &s) {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[2 * i] = quant1(bf16lo_to_f32(v[i]), s);
        c[2 * i + 1] = quant1(bf16hi_to_f32(v[i]), s);
    }
    uint2 w;
    // bytes 0 of four words: (c0, c1) and (c2, c3) pairwise, then joined
    const uint32_t p0 = __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u), p1 = __builtin_amdgcn_perm(c[3], c[2], 0x04000C0Cu);
    const uint32_t p2 = __builtin_amdgcn_perm(c[5], c[4], 0x0C0C0400u), p3 = __builtin_amdgcn_perm(c[7], c[6], 0x04000C0Cu);
    w.x = p0 | p1;
    w.y = p2 | p3;
    // a row with an infinity or NaN (r = 0 with a NaN scale): 0 times inf is
    // NaN, whose low byte is not 0
    if (s.r == 0.0f) w = make_uint2(0u, 0u);
    return w;
}

void launch_tiled(int act, Args a, hipStream_t st);

}  // namespace w8
}  // namespace moe
