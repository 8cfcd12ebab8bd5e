// moe_fp8s.h -- what the kernels of the products in 8-bit floating point with
// an fp32 scale for each block of 128 share: the launch arguments, the matrix
// instruction, and the quantisation of one block's elements.
#pragma once

#include "moe_w8a8.h"

namespace moe {
namespace f8 {

typedef int v8i __attribute__((ext_vector_type(8)));

// The weights lie as the W8A8 products' (moe_w8a8.h): 1 KB blocks of 16 rows x
// 64 k.  Two neighbouring blocks are the matrix instruction's operand for 128
// k: lane l's 32 bytes are k = 16 (l / 16) + [0, 16) and 64 more.  Which k a
// byte of the operand stands for does not matter while both operands agree:
// the activations are read at the same k.
using w8::kblocks;
using w8::kBlockBytes;
using w8::packed_row;
using w8::subtiles;

struct Args {
    const uint8_t *a;        // e4m3 codes [n_src or R][K]
    const float *as;         // fp32 [n_src or R][KG]
    const uint16_t *x;       // fused quantisation: bf16 rows instead of a, as
    const int32_t *gather;   // row r reads a[gather[r]] (or null: a[r])
    int n_src;
    const uint8_t *wq;       // packed weights
    const float *ws;         // fp32 [G][ceil(N/128)][KG]
    const int32_t *offsets;  // group offsets [G+1]; null: one group of rows [0, R)
    int G, R, N, K;
    uint16_t *out;           // bf16 [R][N] or [R][N/2] (SwiGLU)
    uint8_t *hq;             // SwiGLU: e4m3 [R][N/2] and fp32 [R][N/256] that may be written instead of out, or null
    float *hqs;
    int KG, NT;              // 128-wide blocks of k, 16-row subtiles per group in the packed weights
    int NB;                  // n-blocks (the instance's tile width)
    int qrows;               // fused quantisation: rows of a tile
    bool f32;                // SwiGLU: sums in fp32 at any size
};

// The products of 128 k, without scales (the instruction's own are powers of
// two; fp32 scales are applied to its result).
__device__ __forceinline__ f32x4 mfma_fp8(v8i a, v8i b) {
    const f32x4 z = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v8i join(u32x4 lo, u32x4 hi) {
    return __builtin_bit_cast(v8i, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The same in bf16, to which e4m3 converts exactly.  mfma_fp8 sums eight
// neighbouring products after cutting each off at 2^-13 of the largest one's
// power of two (measured: off by 2e-6 of the sum of the products' sizes, root
// mean square), which moves a few in a thousand of SwiGLU's outputs to their
// bf16 neighbour and some of those to another code when they are quantised for
// the next product.  That adds as much to the error of a layer's output as its
// bf16 rounding does (0.0017 -> 0.0024 of its norm), and more where few values
// make up the output.  The products that SwiGLU follows are therefore these
// where its outputs are few (launch_tiled), in the weight stream, and where the
// caller asks for them (they take twice the matrix instructions' time and the
// conversions).
__device__ __forceinline__ bf16x8 to_bf16(int lo, int hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    const u32x4 v = {__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                     __builtin_bit_cast(uint32_t, d)};
    return __builtin_bit_cast(bf16x8, v);
}
struct Wide {  // 128 k of an operand
    bf16x8 v[4];
};
__device__ __forceinline__ Wide widen(v8i a) {
    Wide w;
#pragma unroll
    for (int p = 0; p < 4; ++p) w.v[p] = to_bf16(a[2 * p], a[2 * p + 1]);
    return w;
}
__device__ __forceinline__ f32x4 mfma_wide(const Wide &a, const Wide &b) {
    f32x4 c = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < 4; ++p) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[p], b.v[p], c, 0, 0, 0);
    return c;
}

// Quantisation of a block: scale = amax / 448 (fp32), code = the e4m3 value
// nearest 448 x / amax, ties to even, exactly.  With amax = m 2^e (m in [1/2,
// 1)) and t = 448 (x 2^-e), all exact, the code is t / m rounded.  t has 11
// significant bits, m 8 and a value between two codes 5: where t / m is not
// such a value it is at least 2^-14 of its size away from one, far more than
// the error of q = t r, r ~ 1/m; where it is, it is a float, and one
// correction step returns it exactly.  A block with an infinity or NaN gets a
// NaN scale and codes 0, a block of zeros scale 0 and codes 0.
struct BlockScale {
    float m, r, scale;
    int e;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {  // bf16 bits of max |x|
    BlockScale s;
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
    s.scale = __fdiv_rn(amax, 448.0f);
    return s;
}
__device__ __forceinline__ float quotient(float x, const BlockScale &s) {
    const float t = 448.0f * __builtin_amdgcn_ldexpf(x, -s.e);
    const float q = t * s.r;
    return __builtin_fmaf(__builtin_fmaf(-q, s.m, t), s.r, q);
}
// eight bf16 -> eight e4m3 codes
__device__ __forceinline__ uint2 quant8(u32x4 v, const BlockScale &s) {
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(bf16lo_to_f32(v[2 * i]), s), quotient(bf16hi_to_f32(v[2 * i]), s), 0,
                                                false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(bf16lo_to_f32(v[2 * i + 1]), s), quotient(bf16hi_to_f32(v[2 * i + 1]), s),
                                            w, true);
        c[i] = (uint32_t)w;
    }
    return s.r == 0.0f ? make_uint2(0u, 0u) : make_uint2(c[0], c[1]);
}
// the largest |x| of eight bf16, as bits
__device__ __forceinline__ uint32_t max8(u32x4 v) {
    const uint32_t m = w8::pk_max_abs(w8::pk_max_abs(w8::pk_max_abs(w8::pk_max_abs(0u, v[0]), v[1]), v[2]), v[3]);
    return max(m & 0xFFFFu, m >> 16);
}
// ... of the sixteen lanes that share a block of 128
__device__ __forceinline__ uint32_t max_of_16(uint32_t m) {
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, kWave));
    return m;
}

// Returns whether hq and hqs were written instead of out.
bool launch_tiled(int act, Args a, hipStream_t st);

}  // namespace f8
}  // namespace moe
