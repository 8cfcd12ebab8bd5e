// moe_w8a8_tiled.hip -- the W8A8 product for many rows per group: tiles of up
// to 16 MC permuted rows by 64 NSW weight rows, four waves side by side along
// the weight rows.
//
// Per 128-wide k step the tile's activation codes (128 bytes a row) go from
// global memory straight into one of ST LDS stages, ST - 1 steps ahead, and
// every wave reads all of them; the weights, which no two waves of a
// workgroup share, go from global memory into registers, PF half steps (64 k)
// ahead, so that per matrix instruction of 16 cycles only 1024 / NSW bytes
// come out of LDS.  ONCE: groups of one tile, whose weights are read by one
// workgroup and not kept in the caches.  The sums are exact in int32, so the
// k loop holds nothing but loads and matrix instructions; both scales are
// applied in the epilogue.
// The wave multiplies only the m-tiles (16 rows) that have rows: the count is
// a constant of each instance of the k loop, chosen once per work item.
//
// What bounds it.  Dense with many rows: power.  The matrix instruction alone,
// on random bytes, runs at 3800 TOPS here (4830 on zeros); an 8192 x 4096 x
// 4096 product takes 113 to 134 us (2050 to 2430 TOPS) at 2.03 GHz with the
// matrix units busy 57% of the time, and the same k loop without its loads 90.
// Groups of 200 rows (the layer's experts at 8192 tokens): HBM, 4.96 GB read
// and 0.24 written in 1.04 ms and 2.5 + 0.47 GB in 0.60 ms, 5.0 TB/s, a copy's
// rate.  Few rows per group: the weights' bytes (64 tokens: 6.6 TB/s read).
#include <algorithm>
#include <type_traits>

#include "moe_w8a8.h"

namespace moe {
namespace w8 {
namespace {

// Chunk c (16 bytes) of row r of a stage sits at chunk c ^ swz(r): the eight
// rows of each parity that one 16-lane group of an operand read takes then
// lie on eight distinct chunks (two 128-byte rows share the 64 banks).
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// The matrix instruction written as assembly, so that each accumulator stays
// in its registers and the loads between the instructions stay where they are
// written: the compiler's own form rotates the accumulators of a large tile
// through copies.  The two wait states in
// front cover a copy that the compiler may place before it (they pass in the
// shadow of the previous instruction's 16 cycles); an accumulator comes up
// again only after every other one, and mfma_drain precedes the first use of
// the sums.
__device__ __forceinline__ void mfma_acc(v4i &acc, u32x4 a, u32x4 b) {
    asm volatile("s_nop 1\n\tv_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+v"(acc) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_drain() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// The work item of this workgroup in a dense product: find_tile_item's list
// (m-tiles in chunks of four, n-block-major inside a chunk; a contiguous
// slice per XCD) for one group, without its search.
__device__ __forceinline__ bool dense_item(int NB, int TM, int R, TileItem &it) {
    const int mt = (R + TM - 1) / TM, total = mt * NB, per = (total + 7) >> 3;
    const int item = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || item >= total) return false;
    const int ch = item / (4 * NB), rem = item - ch * 4 * NB, mc = min(4, mt - 4 * ch);
    it.g = 0;
    it.nb = rem / mc;
    it.m0 = (4 * ch + rem - it.nb * mc) * TM;
    it.mrows = min(TM, R - it.m0);
    return true;
}

template <int ACT, int NSW, int MC, int PF, int ST, int OCC, bool ONCE>
__global__ __launch_bounds__(256, OCC) void k_w8a8_tiled(Args p) {
    constexpr int TM = 16 * MC;  // times 64 NSW weight rows
    constexpr int HSW = NSW / 2;
    static_assert(2 * (ST - 2) * NSW < 64, "the wait counts 64 loads");
    __shared__ u32x4 sA[ST * TM * 8];
    constexpr int NO = ACT == MOE_ACT_SWIGLU ? HSW : NSW;  // output subtiles per wave
    constexpr int NWS = NSW / 4 > 0 ? NSW / 4 : 1;         // weight scales per thread
    __shared__ int srow[TM];
    __shared__ float sas[TM], sws[256 * NWS];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id();
    const int m = l & 15, q = l >> 4;
    TileItem it;
    if (p.offsets ? !workgroup_tile_item(p.NB, TM, p.offsets, p.G, p.R, it) : !dense_item(p.NB, TM, p.R, it)) return;
    const int K = p.K, KB = p.KB, KG = KB >> 1, NTH = p.NT >> 1;
    if (tid < TM) {
        int sr = -1;
        if (tid < it.mrows) {
            sr = it.m0 + tid;
            if (p.gather) {
                const int t = p.gather[it.m0 + tid];
                sr = (unsigned)t < (unsigned)p.n_src ? t : -1;
            }
        }
        srow[tid] = sr;
    }
    __syncthreads();
    const int mc = (it.mrows + 15) >> 4;  // m-tiles that have rows
    // The epilogue's scales: one row scale and NWS weight scales per thread.
    // Scale x of the tile belongs to output x % (64 NO) of the tile's columns
    // (SwiGLU: first the gate columns', then the up columns').
    const float my_as = tid < TM ? p.as[max(srow[tid], 0)] : 0.0f;
    float my_ws[NWS];
#pragma unroll
    for (int i = 0; i < NWS; ++i) {
        const int x = 256 * i + tid, col = min(it.nb * (64 * NO) + x % (64 * NO), (ACT == MOE_ACT_SWIGLU ? p.N >> 1 : p.N) - 1);
        my_ws[i] = p.ws[(size_t)it.g * p.N + (ACT == MOE_ACT_SWIGLU && x >= 64 * NO ? p.N >> 1 : 0) + col];
    }

    // the wave's subtiles: NSW consecutive ones, or (SwiGLU) NSW/2 of the
    // gate projection and the same of the up projection
    auto tile_of = [&](int j) {
        if (ACT == MOE_ACT_SWIGLU)
            return (j < HSW ? 0 : NTH) + min((it.nb * 4 + wave) * HSW + (j < HSW ? j : j - HSW), NTH - 1);
        return min((it.nb * 4 + wave) * NSW + j, p.NT - 1);
    };
    const int8_t *wb[NSW];
#pragma unroll
    for (int j = 0; j < NSW; ++j) wb[j] = p.wq + ((size_t)it.g * p.NT + tile_of(j)) * KB * kBlockBytes;

    const int a_lane[2] = {m * 8 + (q ^ swz(m)), m * 8 + ((q + 4) ^ swz(m))};

    auto body = [&](auto mcc) {
        constexpr int C = decltype(mcc)::value;
        // activation loads: wave w moves rows 4 C w .., eight rows a load.
        // Past the end of a row whose K is not a multiple of 128 they take
        // any 16 bytes of the row (the packed weights there are zero).
        constexpr int NLA = C / 2;
        const int8_t *asrc[NLA];
        int achunk[NLA];
#pragma unroll
        for (int j = 0; j < NLA; ++j) {
            const int r = 4 * C * wave + 8 * j + (l >> 3);
            achunk[j] = 16 * ((l & 7) ^ swz(r));
            asrc[j] = p.a + (size_t)max(srow[r], 0) * K;
        }
        auto dma_a = [&](int stage, int kg) {
#pragma unroll
            for (int j = 0; j < NLA; ++j)
                dma16_untracked(asrc[j] + min(128 * kg + achunk[j], K - 16), &sA[stage * (TM * 8) + (4 * C * wave + 8 * j) * 8]);
        };
        v4i acc[C][NSW];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < NSW; ++j) acc[c][j] = v4i{0, 0, 0, 0};
        u32x4 b[PF][NSW], a0[C], a1[C];  // the weights of PF half steps
        auto load_b = [](const int8_t *at) {
            return ONCE ? __builtin_nontemporal_load((const u32x4 *)at) : *(const u32x4 *)at;
        };
        auto boff = [&](int kb) { return (uint32_t)min(kb, KB - 1) * kBlockBytes + 16 * l; };
        auto read_a = [&](u32x4(&av)[C], int stage, int h) {
#pragma unroll
            for (int c = 0; c < C; ++c) av[c] = sA[stage * (TM * 8) + 128 * c + a_lane[h]];
        };
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) dma_a(i, min(i, KG - 1));
#pragma unroll
        for (int h = 0; h < PF; ++h) {
            const uint32_t o = boff(h);
#pragma unroll
            for (int j = 0; j < NSW; ++j) b[h][j] = load_b(wb[j] + o);
        }
        __builtin_amdgcn_sched_barrier(0);
        // the activation loads of the first ST - 1 steps have landed, then every wave's
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(PF * NSW));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        read_a(a0, 0, 0);

        // half a step: the m-tiles times one 64-wide k block; each subtile's
        // operand is replaced by the one of PF half steps later once its
        // last matrix instruction is issued
        auto half = [&](u32x4(&bv)[NSW], u32x4(&av)[C], int kb_next) {
            const uint32_t o = boff(kb_next);
#pragma unroll
            for (int j = 0; j < NSW; ++j) {
#pragma unroll
                for (int c = 0; c < C; ++c) mfma_acc(acc[c][j], bv[j], av[c]);
                bv[j] = load_b(wb[j] + o);
            }
        };
        int s0 = 0;  // the stage of step kg
        // This wave's activation loads of step kg + 1 have landed: they are
        // older than the weight loads of the last 2 (ST - 2) half steps.
        // After the barrier every wave's have, and every wave is done with
        // the stage of step kg - 1, which step kg + ST - 1 takes.
        auto turn = [&](int kg) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * (ST - 2) * NSW));
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            dma_a((s0 + ST - 1) & (ST - 1), min(kg + ST - 1, KG - 1));
            __builtin_amdgcn_sched_barrier(0);
            s0 = (s0 + 1) & (ST - 1);
        };
        auto step = [&](u32x4(&bl)[NSW], u32x4(&bh)[NSW], int kg) {
            read_a(a1, s0, 1);
            half(bl, a0, 2 * kg + PF);
            turn(kg);
            read_a(a0, s0, 0);
            half(bh, a1, 2 * kg + PF + 1);
            __builtin_amdgcn_sched_barrier(0);
        };
        constexpr int NS = PF / 2;  // steps whose weights are in registers
        int kg = 0;
#pragma unroll 1
        for (; kg + NS <= KG; kg += NS)
#pragma unroll
            for (int i = 0; i < NS; ++i) step(b[2 * i], b[2 * i + 1], kg + i);
#pragma unroll
        for (int i = 0; i < NS - 1; ++i)
            if (kg + i < KG) step(b[2 * i], b[2 * i + 1], kg + i);
        mfma_drain();
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < NSW; ++j) asm volatile("" : "+v"(acc[c][j]));  // no use before the drain
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // no load into LDS outlives the block

        // epilogue: the scales, requested before the k loop, go through LDS;
        // lane (m, q) holds, of token 16 c + m, the 16 outputs at 64 st + 16 q
        // of each four subtiles (packed_row), four per subtile
        if (tid < TM) sas[tid] = my_as;
#pragma unroll
        for (int i = 0; i < NWS; ++i) sws[256 * i + tid] = my_ws[i];
        __syncthreads();
        const int NC = ACT == MOE_ACT_SWIGLU ? p.N >> 1 : p.N;
        const int t0 = (it.nb * 4 + wave) * NO;  // the wave's first output subtile
        f32x4 wg[NO], wu[NO];
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            wg[j] = *(const f32x4 *)&sws[packed_row(wave * NO + j, 4 * q)];
            wu[j] = ACT == MOE_ACT_SWIGLU ? *(const f32x4 *)&sws[64 * NO + packed_row(wave * NO + j, 4 * q)] : f32x4{};
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int r = 16 * c + m;
            const bool live = srow[r] >= 0;  // a row without a source is zero
            const float sa = sas[r];
            uint2 w[NO];
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                float o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i] = (float)acc[c][j][i] * sa * wg[j][i];
                    if (ACT == MOE_ACT_SWIGLU) o[i] = silu_mul(o[i], (float)acc[c][j + HSW][i] * sa * wu[j][i]);
                }
                w[j] = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
                if (!live) w[j] = make_uint2(0u, 0u);
            }
            if (r >= it.mrows) continue;
            uint16_t *row = p.out + (size_t)(it.m0 + r) * NC;
            if constexpr (NO == 1) {
                const int n = packed_row(t0, 4 * q);
                if (n < NC) *(uint2 *)(row + n) = w[0];
            } else {
#pragma unroll
                for (int j = 0; j < NO; j += 2) {
                    const int n = packed_row(t0 + j, 4 * q);
                    if (n < NC) *(u32x4 *)(row + n) = u32x4{w[j].x, w[j].y, w[j + 1].x, w[j + 1].y};
                }
            }
        }
    };
    if constexpr (MC == 2) {
        body(std::integral_constant<int, 2>());
    } else if constexpr (MC == 8) {
        if (mc > 6)
            body(std::integral_constant<int, 8>());
        else if (mc > 4)
            body(std::integral_constant<int, 6>());
        else if (mc > 2)
            body(std::integral_constant<int, 4>());
        else
            body(std::integral_constant<int, 2>());
    } else {
        if (mc > 2)
            body(std::integral_constant<int, 4>());
        else
            body(std::integral_constant<int, 2>());
    }
}

template <int NSW, int MC, int PF, int ST, int OCC, bool ONCE = false>
void launch(int act, Args a, hipStream_t st) {
    constexpr int TM = 16 * MC;
    a.NB = (a.NT + 4 * NSW - 1) / (4 * NSW);
    int64_t tiles = a.offsets ? (int64_t)a.R / TM + (a.R < a.G ? a.R : a.G) : (a.R + TM - 1) / TM;
    if (tiles > a.R) tiles = a.R;  // every tile has a row
    const dim3 grid((unsigned)((tiles * a.NB + 7) / 8 * 8));  // a whole slice per XCD
    if constexpr (NSW > 1) {  // SwiGLU: a gate and an up subtile per wave at least
        if (act == MOE_ACT_SWIGLU) {
            hipLaunchKernelGGL((k_w8a8_tiled<MOE_ACT_SWIGLU, NSW, MC, PF, ST, OCC, ONCE>), grid, dim3(256), 0, st, a);
            return;
        }
    }
    hipLaunchKernelGGL((k_w8a8_tiled<MOE_ACT_NONE, NSW, MC, PF, ST, OCC, ONCE>), grid, dim3(256), 0, st, a);
}

}  // namespace

// Which tile: the one with the least cost times rounds of one workgroup per
// CU.  A larger tile reads fewer bytes per product (what bounds a CU that has
// its workgroup), a smaller one fills the CUs with fewer rows; where every CU
// gets a second workgroup that costs nearly a second round, and a few too many
// are counted as one too, which was not measured (61 rows of 8208 columns: 258
// workgroups of 32 x 64 count as two rounds, so 130 of 32 x 128 are taken).
// The costs are the times of one round at N = K = 4096, 8 to 30 us; us there
// (tiles of rows x weight rows):
//   rows       128 x 256   64 x 256   64 x 128   32 x 128   32 x 64
//   61              18.1       16.7       12.2        9.8       7.7
//   256             28.5       17.0       12.8       10.6      12.6
//   512             29.0       17.9       13.9       17.7      22.6
//   1024            30.0       21.7       22.6       31.6      40.7
//   2048            36.9       40.5       46.9       61.6
//   8192             119        149        169        246       293
// (32 x 64 without an activation only: a wave has one subtile.)
// Groups of few rows are bound by the weights' bytes: 64 x 128 tiles keep the
// most of them in flight (the layer's experts at hidden 4096, 256 experts, 6
// per token: 1162 us against 1177 with 128 x 256 at 1024 tokens, 1279 against
// 1249 at 2048, where a group has 48 rows; 64 x 256 there: 1282), and loads
// that pass the caches by stream them faster (512 tokens: 1057 against 1110
// us; 8 tokens: 196 against 207; with a skewed choice of experts 491 against
// 519 at 64 tokens, 1101 against 1064 at 512).  Not where several tiles share
// a group's weights (8192 tokens: 2824 against 1990), nor where the layer's
// weights may still be in the 256 MB last-level cache from the call before
// (hidden 1024, 40 experts, 43 MB: 34.8 against 30.5 us at 421 tokens).
void launch_tiled(int act, Args a, hipStream_t st) {
    auto workgroups = [&](int TM, int TN) {
        const int64_t tiles = (a.R + TM - 1) / TM + (a.offsets ? (a.R < a.G ? a.R : a.G) / 2 : 0);
        return tiles * ((16 * a.NT + TN - 1) / TN);
    };
    auto cost = [&](int TM, int TN, int of_a_round) { return (workgroups(TM, TN) + 255) / 256 * of_a_round; };
    const int64_t c128x256 = cost(128, 256, 30), c64x256 = cost(64, 256, 20), c64x128 = cost(64, 128, 12),
                  c32x128 = cost(32, 128, 10), c32x64 = act == MOE_ACT_NONE ? cost(32, 64, 8) : INT64_MAX;
    const int64_t least = std::min({c128x256, c64x256, c64x128, c32x128, c32x64});
    const size_t weights = (size_t)a.G * a.NT * a.KB * kBlockBytes;
    if (a.offsets && a.R < 48 * (int64_t)a.G && weights >= (size_t)128 << 20)
        launch<2, 4, 4, 4, 3, true>(act, a, st);
    else if (a.offsets && a.R < 48 * (int64_t)a.G)
        launch<2, 4, 4, 4, 3>(act, a, st);
    else if (c128x256 == least || (a.offsets && workgroups(128, 256) >= 256))
        launch<4, 8, 2, 4, 2>(act, a, st);
    else if (c64x256 == least)
        launch<4, 4, 4, 4, 2>(act, a, st);
    else if (c64x128 == least)
        launch<2, 4, 4, 4, 3>(act, a, st);
    else if (c32x128 == least)
        launch<2, 2, 4, 4, 4>(act, a, st);
    else
        launch<1, 2, 8, 8, 4>(act, a, st);
}

}  // namespace w8
}  // namespace moe
