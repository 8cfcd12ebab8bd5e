// moe_bf16_tiled.hip -- the grouped bf16 product (kNT) for few rows per group of
// a layer with many weights, on tiles of 64 rows by 256 columns.
//
// Bound by the weights' bytes.  Four waves side by side along the columns.  The
// permuted rows, which all four multiply with, go from global memory straight
// into LDS, 64 of K a step, two steps ahead; the weights, which no two waves of
// a workgroup share, go straight into the registers of the one wave that
// multiplies them, a lane taking 32 consecutive bytes of a weight row a step, a
// step ahead.  64 tokens of the 256-expert layer with a skewed choice (123
// groups): gate/up 700 us, down 355 us, 5.9 TB/s; through LDS both (64 x 128
// and 256 x 256 tiles of moe_bf16_wide.hip) 800 and 395.  2048 tokens (56 rows a
// group): 1694 and 846 us, 5.1 TB/s, against 1840 and 930.
// Row r of the matrix instruction's first operand stands for column 4 r + j of
// the wave's columns in its subtile j, so that a lane's results are 16
// consecutive columns of one row.
#include <algorithm>

#include "moe_bf16.h"
#include "moe_dma.h"

namespace moe {
namespace b16 {
namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kBK = 64;  // contraction per step

// What lanes without an element of a row load.
__device__ const u32x4 kZeros = {0u, 0u, 0u, 0u};

// The buffer of moe_dma.h for loads into registers.
__device__ __forceinline__ rsrc_t resource(const void *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, buffer_size(bytes), kBufferFlags);
}
__device__ __forceinline__ u32x4 load16(rsrc_t r, uint32_t voff) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, 0, 0));
}
// s_waitcnt immediate: at most n vector loads outstanding, no LDS operation.
constexpr int wait_imm(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0070; }

// Place x of row r of a [row][64 k] stage holds chunk (16 bytes) chunk_at(x ^
// swz(r)).  An operand read takes one place of sixteen rows in each of its
// four lane groups; the lanes that one pass serves (see lds_swz), two rows to
// each 256 bytes of banks, then lie on distinct banks.  Lane group q takes
// chunk 2 q + h, the 32 bytes that it loads of a weight row.
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int chunk_at(int x) { return (x & 3) << 1 | x >> 2; }
// The matrix instruction written as assembly, so that each accumulator stays
// in its registers: the compiler's own form rotates the accumulators of a
// large tile through copies and spills.  The two wait states in front cover an
// operand that the instruction before it wrote (they pass in the shadow of the
// previous matrix instruction's 16 cycles); an accumulator comes up again only
// after every other one, and mfma_drain precedes the first use of the sums.
__device__ __forceinline__ void mfma_acc(f32x4 &acc, bf16x8 a, bf16x8 b) {
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_drain() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

template <int EPI>
__global__ __launch_bounds__(256, 2) void k_bf16_tiled(Args p) {
    constexpr int NSW = 4, MC = 4, TM = 16 * MC, HS = NSW / 2;  // subtiles and m-tiles of a wave
    constexpr int ABYTES = TM * kBK * 2, LA = ABYTES / 4096;     // loads into LDS per wave and step, 1 KB each
    __shared__ __attribute__((aligned(16))) char sA[3 * ABYTES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id();
    const int m = l & 15, q = l >> 4;
    TileItem it;
    if (!workgroup_tile_item(p.NB, TM, p.offsets, p.G, p.R, it)) return;
    const int K = p.K, KG = (K + kBK - 1) / kBK;
    // the wave's first column (SwiGLU: of the gate projection, and as many of the up projection)
    const int n0 = (it.nb * 4 + wave) * (EPI == kSwiglu ? 16 * HS : 16 * NSW);

    f32x4 acc[MC][NSW];
#pragma unroll
    for (int c = 0; c < MC; ++c)
#pragma unroll
        for (int j = 0; j < NSW; ++j) acc[c][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // ---- the rows: load j of a wave brings eight of them
    const char *zero = (const char *)&kZeros, *asrc[LA];
    auto chunk = [&](int j) { return chunk_at((l & 7) ^ swz(8 * (LA * wave + j) + (l >> 3))); };
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        const int r = 8 * (LA * wave + j) + (l >> 3);
        int src = it.m0 + min(r, it.mrows - 1);
        if (p.gather) src = p.gather[src];
        // (a row without a source, or past the tile's last: zeros)
        const bool in = r < it.mrows && (unsigned)src < (unsigned)(p.gather ? p.n_src : p.R);
        asrc[j] = in ? (const char *)p.a + 2 * ((size_t)src * K + 8 * chunk(j)) : nullptr;
    }
    auto dma = [&](int kg, int stage) {
#pragma unroll
        for (int j = 0; j < LA; ++j) {
            const bool in = asrc[j] && kBK * kg + 8 * chunk(j) < K;
            dma16_untracked(in ? asrc[j] + 2 * kBK * (size_t)kg : zero, sA + stage * ABYTES + 1024 * (LA * wave + j));
        }
    };
    auto read_a = [&](int stage, int h, int c) -> bf16x8 {
        return *(const bf16x8 *)(sA + stage * ABYTES + (16 * c + m) * 128 + 16 * ((4 * h + q) ^ swz(m)));
    };

    // ---- the weights: row NSW m + j of the wave's columns in subtile j
    const size_t ld = 2 * (size_t)K;
    const char *w = (const char *)p.b + (size_t)it.g * p.N * ld;
    const int up = (p.N >> 1) + n0;
    const rsrc_t b0 = resource(w + n0 * ld, (int64_t)(p.N - n0) * ld);
    const rsrc_t b1 = EPI == kSwiglu ? resource(w + up * ld, (int64_t)(p.N - up) * ld) : b0;
    const uint32_t voff = (uint32_t)((EPI == kSwiglu ? HS : NSW) * m * ld) + 32 * q;
    auto load_b = [&](u32x4 (&part)[2 * NSW], int kg, int i) {  // half i & 1 of the 32 bytes of subtile i / 2
        const int j = i >> 1;
        const uint32_t far = kBK * kg + 16 * q >= K ? kFar : 0u;  // past the row's end: zeros
        const bool u = EPI == kSwiglu && j >= HS;
        part[i] = load16(u ? b1 : b0, voff + 16 * (i & 1) + far + (uint32_t)((u ? j - HS : j) * ld) + 128 * kg);
    };
    u32x4 raw[2][2 * NSW];  // of two steps
    constexpr int PFD = 3, WIN = 4;  // m-tiles that an operand read is ahead of its use
    bf16x8 win[WIN][2];              // the operands of the next m-tiles
    dma(0, 0);
    dma(min(1, KG - 1), 1);
    dma(min(2, KG - 1), 2);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 2 * NSW; ++i) load_b(raw[t], t, i);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_imm(4 * NSW));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < PFD; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) win[c][h] = read_a(0, h, c);
    int s0 = 0;
    auto step = [&](u32x4 (&part)[2 * NSW], int kg) {
        const int s1 = s0 == 2 ? 0 : s0 + 1;
#pragma unroll
        for (int c = 0; c < MC; ++c) {
            if (c == MC - PFD) {
                // Everything that this wave reads of step kg's stage is in
                // registers, and step kg + 1 has landed (older than the
                // weights in flight); after the barrier that holds for every
                // wave, and the stage takes step kg + 3.
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_waitcnt(wait_imm(4 * NSW));
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                dma(min(kg + 3, KG - 1), s0);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) win[(c + PFD) % WIN][h] = read_a(c < MC - PFD ? s0 : s1, h, (c + PFD) % MC);
#pragma unroll
            for (int j = 0; j < NSW; ++j) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mfma_acc(acc[c][j], __builtin_bit_cast(bf16x8, part[2 * j + h]), win[c % WIN][h]);
                if (c == MC - 1) {
                    load_b(part, kg + 2, 2 * j);
                    load_b(part, kg + 2, 2 * j + 1);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        s0 = s1;
    };
    static_assert(MC % WIN == 0, "a step begins at the window's first place");
    int kg = 0;
#pragma unroll 1
    for (; kg + 2 <= KG; kg += 2) {
        step(raw[0], kg);
        step(raw[1], kg + 1);
    }
    if (kg < KG) step(raw[0], kg);
    mfma_drain();
#pragma unroll
    for (int c = 0; c < MC; ++c)
#pragma unroll
        for (int j = 0; j < NSW; ++j) asm volatile("" : "+a"(acc[c][j]));  // no use before the drain
    __builtin_amdgcn_s_waitcnt(wait_imm(0));                                // no load into LDS outlives the block
    __builtin_amdgcn_sched_barrier(0);

    // ---- epilogue: lane (m, q) holds, of row 16 c + m, the columns 4 NSW q + NSW i + j of its wave's
#pragma unroll
    for (int c = 0; c < MC; ++c) {
        const int r = 16 * c + m;
        if (r >= it.mrows) continue;
        const size_t row = (size_t)it.m0 + r;
        if constexpr (EPI == kSwiglu) {
            const int NC = p.N >> 1, n = n0 + 4 * HS * q;
            if (n >= NC) continue;
            uint32_t o[4], g[4], u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // columns HS e + {0, 1} are subtiles 0 and 1 of element e
                const float g0 = acc[c][0][e], g1 = acc[c][1][e], u0 = acc[c][2][e], u1 = acc[c][3][e];
                o[e] = pack_bf16x2(silu_mul(g0, u0), silu_mul(g1, u1));
                g[e] = pack_bf16x2(g0, g1);
                u[e] = pack_bf16x2(u0, u1);
            }
            *(u32x4 *)((uint16_t *)p.out + row * NC + n) = u32x4{o[0], o[1], o[2], o[3]};
            if (p.gu) {
                *(u32x4 *)(p.gu + row * p.N + n) = u32x4{g[0], g[1], g[2], g[3]};
                *(u32x4 *)(p.gu + row * p.N + NC + n) = u32x4{u[0], u[1], u[2], u[3]};
            }
        } else {
            const int n = n0 + 4 * NSW * q;
            if (n >= p.N) continue;
            u32x4 v[2];
#pragma unroll
            for (int x = 0; x < 8; ++x)  // columns 2 x and 2 x + 1
                v[x >> 2][x & 3] = pack_bf16x2(acc[c][2 * x % NSW][2 * x / NSW], acc[c][(2 * x + 1) % NSW][(2 * x + 1) / NSW]);
            u32x4 *out = (u32x4 *)((uint16_t *)p.out + row * p.N + n);
            out[0] = v[0];
            out[1] = v[1];
        }
    }
}

template <int EPI>
void launch(Args p, hipStream_t st) {
    constexpr int TM = 64, TN = EPI == kSwiglu ? 128 : 256;
    p.NB = ((EPI == kSwiglu ? p.N / 2 : p.N) + TN - 1) / TN;
    const int64_t tiles = std::min<int64_t>((int64_t)p.R / TM + std::min(p.R, p.G), p.R);  // every tile has a row
    hipLaunchKernelGGL((k_bf16_tiled<EPI>), dim3((unsigned)((tiles * p.NB + 7) / 8 * 8)), dim3(256), 0, st, p);
}

}  // namespace

void launch_tiled(int epi, const Args &p, hipStream_t st) { epi == kSwiglu ? launch<kSwiglu>(p, st) : launch<kStore>(p, st); }

}  // namespace b16
}  // namespace moe
