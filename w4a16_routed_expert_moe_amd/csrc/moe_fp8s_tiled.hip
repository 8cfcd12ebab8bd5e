// moe_fp8s_tiled.hip -- the fp8 product with fp32 block scales for more than a
// few rows per group, on tiles of 16 MW WM permuted rows by 64 WN weight rows.
//
// WM x WN waves (rows x weight rows) compute a tile, each 16 MW x 64 of it.
// Per 128-wide k block the activation codes and the weights go from global
// memory straight into one of two LDS stages; one matrix instruction multiplies
// 16 x 16 over the block, and its result is added to the sums times both
// scales (a product per row and block, a multiply-add per element).
//
// A wave works on two m-tiles at a time while the next two come from LDS, the
// additions of one product filling the time of the next.  When it works on the
// last two of a step all of the stage is in registers, so that one barrier
// there lets the loads of the step after the next begin; the weights' registers are
// read anew, for the next step, as each has served the last two.
//
// 8192 x 4096 x 4096 124 us, 20 in a row 137 to 142, 1.95 to 2.2 PFLOP/s; 57344 rows of
// 33 groups, gate/up 991 to 1114 us, 1.7 to 1.9.  The matrix units are busy 53% of
// that at 2.08 GHz, the waves wait for 24% of their cycles and bank conflicts take
// 12% of those in which LDS works: the eight waves of the one workgroup on a CU
// meet at a barrier every step and read LDS at the same time.  The four
// multiply-adds for each matrix instruction cost a cycle of its 33 where only they
// run; without them the kernel takes 105 us.  Few rows of many weights: HBM, 5.7
// TB/s.
#include <algorithm>
#include <type_traits>

#include "moe_dma.h"
#include "moe_fp8s.h"

namespace moe {
namespace f8 {
namespace {

// What rows without a source are read as: the longest row that there is.
__device__ const u32x4 kZeros[65536 / 16] = {};

// Offsets from kNone, which lies past the end of every buffer, give zeros.
constexpr uint32_t kNone = 0xFFFF0000u;
__device__ __forceinline__ i32x4 buffer_all(const char *p, uint64_t bytes) {
    const uint32_t n = bytes > kNone ? kNone : (uint32_t)bytes;
    return i32x4{(int)(uint32_t)(uintptr_t)p, (int)((uintptr_t)p >> 32), (int)n, 0x00027000};
}

// Chunk c (16 bytes) of row r of a stage sits at chunk c ^ swz(r).
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ void dma4_pointer(uint64_t src, uint32_t lds) {  // 4 bytes a lane (see dma16_pointer)
    asm volatile(
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %0, off"
        :
        : "v"(src), "s"(lds)
        : "memory");
}
__device__ __forceinline__ void dma4_buffer(i32x4 r, uint32_t voff, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %0, %1, 0 offen lds"
        :
        : "v"(voff), "s"(r), "s"(lds)
        : "memory");
}

// The workgroup's tile.  One group needs no search (2 us for the 245 tiles of 300
// x 6160 x 2064): the list of find_tile_item, of whole columns.
__device__ __forceinline__ bool find_item(const Args &p, int TM, TileItem &it) {
    if (p.offsets) return workgroup_tile_item(p.NB, TM, p.offsets, p.G, p.R, it);
    const int mt = (p.R + TM - 1) / TM, total = mt * p.NB, per = (total + 7) >> 3;
    const int j = blockIdx.x >> 3, item = (blockIdx.x & 7) * per + j;
    if (j >= per || item >= total) return false;
    const int ch = item / (4 * p.NB), rem = item - ch * 4 * p.NB, mc = min(4, mt - 4 * ch);
    it.g = 0;
    it.nb = rem / mc;
    it.m0 = (4 * ch + rem - it.nb * mc) * TM;
    it.mrows = min(TM, p.R - it.m0);
    return true;
}

// FAR: rows and scales at an address each (more than 4 GB of codes to gather
// from), else at an offset into a buffer.
// EXACT: the products in bf16 (see mfma_wide).
// QUANT: SwiGLU's outputs go quantised into hq and hqs, as moe_act_quant_fp8s
// would from bf16: the workgroup's 128 columns are a block (57344 rows of 2048: 69
// us of a launch less, and 235 MB written and read).
// KS: the workgroup has KS times the waves, each WM x WN of them with stages of
// their own and with every KS-th k block; their sums meet in LDS.
template <int ACT, int MW, int WM, int WN, int KS, int OCC, bool FAR, bool EXACT, bool QUANT>
__global__ __launch_bounds__(64 * WM * WN * KS, OCC) void k_fp8s_tiled(Args p) {
    constexpr int NW = WM * WN, TM = 16 * MW * WM, TN = 64 * WN;
    constexpr bool SWIGLU = ACT == MOE_ACT_SWIGLU;
    constexpr int LA = TM / 8 / NW, LB = TN / 8 / NW, L = LA + LB;  // loads into LDS per wave and step, 1 KB each
    constexpr int LS = TM / 8 / NW;                                 // ... of scales per eight steps
    constexpr int ABYTES = 128 * TM, BBYTES = 128 * TN;
    __shared__ __attribute__((aligned(16))) char sAll[KS * 2 * (ABYTES + BBYTES)];
    __shared__ __attribute__((aligned(16))) float sScale[KS][2][TM * 8];  // scales of eight k blocks, of the next eight
    __shared__ float sWeights[KS * WN][2][16];  // the weights' scales of as many blocks, of both projections
    const int tid = threadIdx.x, wave_id = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id();
    const int wave = wave_id % NW, ks = wave_id / NW;
    char *const sA = sAll + ks * 2 * (ABYTES + BBYTES), *const sB = sA + 2 * ABYTES;
    const int wm = wave / WN, wn = wave % WN, m = l & 15, q = l >> 4;
    float(*const sS)[TM * 8] = sScale[ks], (*const sW)[16] = sWeights[ks * WN + wn];
    int *const sRow = (int *)sScale[0][1];  // source rows, -1: none, until the first step
    TileItem it;
    if (!find_item(p, TM, it)) return;
    const int K = p.K, KG = p.KG, steps = (KG + KS - 1) / KS, NTH = p.NT >> 1, NBK = (p.N + 127) >> 7;
    // ---- the weights.  Slot x = 4 wave column + j of the tile is a subtile: 16
    // consecutive ones, or (SwiGLU) two of the gate projection and the same two
    // of the up projection.  A wave loads LB blocks, in the order of the slots.
    auto tile_of = [&](int x) {
        if (SWIGLU) return ((x & 2) ? NTH : 0) + min(it.nb * (2 * WN) + 2 * (x >> 2) + (x & 1), NTH - 1);
        return min(it.nb * (4 * WN) + x, p.NT - 1);
    };
    // (offsets from the wave's first slot stay below the buffer's 1 GB: only where a
    // workgroup has one column of waves has a wave slots of both projections, and
    // such a tile is for at most 320 columns of 64)
    const int slot0 = LB / 2 * wave, t0 = tile_of(slot0);
    const i32x4 bsrc =
        buffer((const char *)p.wq + ((size_t)p.NT * it.g + t0) * (2 * KG) * kBlockBytes, (int64_t)kFar);
    uint32_t boff[LB / 2];
#pragma unroll
    for (int j = 0; j < LB / 2; ++j) boff[j] = (uint32_t)(tile_of(slot0 + j) - t0) * (2 * KG) * kBlockBytes;

    const uint32_t ldsA = lds_address(sA) + 1024 * LA * wave, ldsB = lds_address(sB) + 1024 * LB * wave;
    const uint32_t ldsS = lds_address((const char *)sS), ldsW = lds_address((const char *)sW);
    auto load_b = [&](int x, int kg, int s) {
        const int at = min(kg * KS + ks, KG - 1);
        dma16_buffer(bsrc, 16 * l, boff[x >> 1] + (2 * at + (x & 1)) * kBlockBytes, ldsB + s * BBYTES + 1024 * x);
    };
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < LB; ++x) load_b(x, t, t);
    // the scales of the wave's weight rows (its subtiles lie in one block of 128
    // rows; SwiGLU: one of each projection): eight blocks of each
    const i32x4 wbuf = buffer_all((const char *)(p.ws + (size_t)it.g * NBK * KG), (uint64_t)NBK * KG * 4);
    const uint32_t wsrc = (((l & 8 ? tile_of(4 * wn + 2) : tile_of(4 * wn)) >> 3) * KG + (l & 7) * KS + ks) * 4;

    if (tid < TM) {
        int src = it.m0 + tid;
        if (tid >= it.mrows)
            src = -1;
        else if (p.gather) {
            src = p.gather[src];
            if ((unsigned)src >= (unsigned)p.n_src) src = -1;
        }
        sRow[tid] = src;
    }
    __syncthreads();

    // ---- the rows: load j of a wave brings eight of them.  Their scales: eight
    // rows' of eight blocks a load; in every other eight rows blocks 4 to 7 come
    // first, so that the rows that a wave reads lie on distinct banks.
    const size_t first = p.gather ? 0 : (size_t)it.m0, rows = (p.gather ? p.n_src : p.R) - first;
    const char *codes = (const char *)p.a + first * K, *scales = (const char *)(p.as + first * KG);
    const uint64_t zero = (uint64_t)(uintptr_t)kZeros;
    const i32x4 abuf = buffer_all(codes, rows * K), sbuf = buffer_all(scales, rows * KG * 4);
    typename std::conditional<FAR, uint64_t, uint32_t>::type asrc[LA], ssrc[LS];
    auto chunk = [&](int j) { return (l & 7) ^ swz(8 * (LA * wave + j) + (l >> 3)); };
    auto sblock = [&](int i) { return (l >> 3) ^ 4 * ((i * NW + wave) & 1); };
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        const int src = sRow[8 * (LA * wave + j) + (l >> 3)];
        if constexpr (FAR)
            asrc[j] = (src < 0 ? zero : (uint64_t)(uintptr_t)p.a + (uint64_t)src * K) + 16 * chunk(j);
        else
            asrc[j] = src < 0 ? kNone : (uint32_t)(src - (int)first) * K + 16 * chunk(j);
    }
#pragma unroll
    for (int i = 0; i < LS; ++i) {
        const int src = sRow[8 * (i * NW + wave) + (l & 7)];
        if constexpr (FAR)
            ssrc[i] = src < 0 ? zero : (uint64_t)(uintptr_t)(p.as + (uint64_t)src * KG);
        else
            ssrc[i] = src < 0 ? kNone : ((uint32_t)(src - (int)first) * KG + sblock(i) * KS + ks) * 4;
    }
    uint32_t live = 0;  // of the wave's m-tiles, whether lane m's row has a source
#pragma unroll
    for (int i = 0; i < MW; ++i) live |= (uint32_t)(sRow[16 * (WM * i + wm) + m] >= 0) << i;
    // the scales of steps [8 kg8, 8 kg8 + 8); those past the last block are not used
    // (they may lie past the buffers' ends, so that none of the offset is scalar)
    auto load_scales = [&](int kg8) {
        if (wm == 0 && l < 16) dma4_buffer(wbuf, wsrc + 32 * KS * kg8, ldsW + (kg8 & 1) * 64);
#pragma unroll
        for (int i = 0; i < LS; ++i) {
            const uint32_t to = __builtin_amdgcn_readfirstlane(ldsS + (kg8 & 1) * (TM * 32) + 256 * (i * NW + wave));
            if constexpr (FAR)
                dma4_pointer(ssrc[i] + 4 * min((8 * kg8 + sblock(i)) * KS + ks, KG - 1), to);
            else
                dma4_buffer(sbuf, ssrc[i] + 32 * KS * kg8, to);
        }
    };
    // load x of step kg into stage s; past the end of the rows: zeros
    uint64_t cut[2];  // lanes that the last block does not have, of even and odd loads
#pragma unroll
    for (int x = 0; x < 2; ++x) cut[x] = __ballot(16 * chunk(x) >= K - 128 * (KG - 1));
    auto load = [&](int x, int kg, int s) {
        const int at = min(kg * KS + ks, KG - 1);
        if (x < LA) {
            const uint64_t none = at == KG - 1 ? cut[x & 1] : 0;
            const bool in = !(none >> l & 1);
            if constexpr (FAR)
                dma16_pointer(in ? asrc[x] + 128 * (uint64_t)at : zero, ldsA + s * ABYTES + 1024 * x);
            else
                dma16_buffer(abuf, in ? asrc[x] : kNone, 128 * at, ldsA + s * ABYTES + 1024 * x);
        } else {
            load_b(x - LA, kg, s);
        }
    };
    auto read_b = [&](int s, int j) -> v8i {
        const u32x4 *at = (const u32x4 *)(sB + s * BBYTES + 2048 * (4 * wn + j) + 16 * l);
        return join(at[0], at[64]);
    };
    auto read_a = [&](int s, int i) -> v8i {
        const u32x4 *row = (const u32x4 *)(sA + s * ABYTES + 128 * (16 * (WM * i + wm) + m));
        return join(row[q ^ swz(m)], row[(q + 4) ^ swz(m)]);
    };
    auto read_s = [&](int kg, int i) { 
        return sS[(kg >> 3) & 1][64 * (2 * (WM * i + wm) + (m >> 3)) + 8 * ((kg & 7) ^ 4 * (m >> 3)) + (m & 7)];
    };

    auto body = [&](auto cc) {
        constexpr int C = decltype(cc)::value, P = C / 2;  // m-tiles, pairs
        f32x4 acc[C][4];
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        load_scales(0);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < LA; ++x) load(x, t, t);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(LA));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        v8i b[4], a[2];
        float sg = sW[0][0], su = sW[0][8];
        float sa[2], fg[2] = {0.0f, 0.0f}, fu[2] = {0.0f, 0.0f};
        f32x4 t[4];  // products that are yet to be added
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            b[j] = read_b(0, j);
            t[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[i] = read_a(0, i);
            sa[i] = read_s(0, i);
        }
        auto add = [&](int pair, int n) {  // product n of a pair: subtile n / 2, m-tile n % 2
            f32x4 &c = acc[2 * pair + (n & 1)][n >> 1];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = __builtin_fmaf(t[n & 3][e], SWIGLU && n >= 4 ? fu[n & 1] : fg[n & 1], c[e]);
            asm volatile("" : "+v"(c));  // here, not when the sums are next needed
        };
        // What the barrier frees is loaded anew between the products up to the
        // next one, one load for two of them: all at once would hold the wave
        // up.  (In the first step the pairs before the last load the last
        // stage once more.)
        constexpr int SLOTS = 8 * P < 2 * L ? 8 * P : 2 * L;
        auto load_at = [&](int slot, int kg, int s) {  // after barrier kg, which freed stage s
            if (slot == 0 && (kg & 7) == 0) load_scales((kg >> 3) + 1);
#pragma unroll
            for (int x = 0; x < L; ++x)
                if (x * SLOTS / L == slot) load(x, kg + 2, s);
        };
        int s = 0;
#pragma unroll 1
        for (int kg = 0; kg < steps; ++kg) {
            const bool real = KS == 1 || kg * KS + ks < KG;  // (the last step of some waves is none)
            const int s1 = s ^ 1;
#pragma unroll
            for (int pair = 0; pair < P; ++pair) {
                const bool last = pair == P - 1;
                if (last) {
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0) & ~0x0F00);  // and no read of LDS outstanding
                    __builtin_amdgcn_s_barrier();
                    __builtin_amdgcn_sched_barrier(0);
                }
                v8i an[2];
                float sn[2], sgn = sg, sun = su;
                if (last) {
                    sgn = sW[((kg + 1) >> 3) & 1][(kg + 1) & 7];
                    sun = sW[((kg + 1) >> 3) & 1][8 + ((kg + 1) & 7)];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int kn = last ? kg + 1 : kg, x = last ? i : 2 * pair + 2 + i;
                    an[i] = read_a(last ? s1 : s, x);
                    sn[i] = read_s(kn, x);
                }
                Wide aw[2], bw;
                if constexpr (EXACT) {
                    aw[0] = widen(a[0]);
                    aw[1] = widen(a[1]);
                }
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    f32x4 r;
                    if constexpr (EXACT) {
                        if ((n & 1) == 0) bw = widen(b[n >> 1]);
                        r = mfma_wide(bw, aw[n & 1]);
                    } else {
                        r = mfma_fp8(b[n >> 1], a[n & 1]);
                    }
                    // the product three before this one's
                    n < 3 ? add(pair ? pair - 1 : P - 1, n + 5) : add(pair, n - 3);
                    if (n == 1 || n == 2) {
                        fg[n - 1] = real ? sa[n - 1] * sg : 0.0f;
                        fu[n - 1] = real ? sa[n - 1] * (SWIGLU ? su : sg) : 0.0f;
                    }
                    t[n & 3] = r;
                    last ? load_at(n, kg, s) : load_at(8 * (pair + 1) + n, kg - 1, s1);
                    if (last && (n & 1)) b[n >> 1] = read_b(s1, n >> 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    a[i] = an[i];
                    sa[i] = sn[i];
                }
                sg = sgn;
                su = sun;
            }
            s = s1;
        }
#pragma unroll
        for (int n = 5; n < 8; ++n) add(P - 1, n);
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // no load into LDS outlives the block
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (KS > 1) {  // the sums over the other waves' blocks, in their order
            f32x4 *part = (f32x4 *)sAll;
            static_assert((KS - 1) * NW * MW * 4096 <= KS * 2 * (ABYTES + BBYTES), "they fit in the stages");
            __syncthreads();
            if (ks)
#pragma unroll
                for (int i = 0; i < C; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[(((ks - 1) * NW + wave) * C + i) * 256 + 64 * j + l] = acc[i][j];
            __syncthreads();
            if (ks) return;
#pragma unroll
            for (int x = 0; x < KS - 1; ++x)
#pragma unroll
                for (int i = 0; i < C; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f32x4 v = part[((x * NW + wave) * C + i) * 256 + 64 * j + l];
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][e] += v[e];
                    }
        }

        // epilogue: lane (m, q) holds, of row 16 (WM i + wm) + m, the outputs at packed_row(subtile, 4 q)
        constexpr int NO = SWIGLU ? 2 : 4;
        const int NC = SWIGLU ? p.N >> 1 : p.N, n0 = (it.nb * WN + wn) * NO;
        auto output = [&](int i) -> u32x4 {  // SwiGLU: eight consecutive columns
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = x >> 1, e = 2 * (x & 1);
                w[x] = pack_bf16x2(silu_mul(acc[i][j][e], acc[i][j + 2][e]), silu_mul(acc[i][j][e + 1], acc[i][j + 2][e + 1]));
            }
            return live >> i & 1 ? u32x4{w[0], w[1], w[2], w[3]} : u32x4{0u, 0u, 0u, 0u};
        };
        if constexpr (QUANT) {
            static_assert(SWIGLU && WN == 4, "a block of 128 columns");
            uint32_t(*const smax)[WN] = (uint32_t(*)[WN])sAll;  // of each row, of each wave's columns
            u32x4 o[C];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < C; ++i) {
                o[i] = output(i);
                uint32_t most = max8(o[i]);
                most = max(most, (uint32_t)__shfl_xor((int)most, 16, kWave));
                most = max(most, (uint32_t)__shfl_xor((int)most, 32, kWave));
                if (q == 0) smax[16 * (WM * i + wm) + m][wn] = most;
            }
            __syncthreads();
            const int n = packed_row(n0, 4 * q);  // (N / 2 is whole blocks)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int r = 16 * (WM * i + wm) + m;
                if (r >= it.mrows) continue;
                const u32x4 v = *(const u32x4 *)smax[r];
                const BlockScale bs = block_scale(max(max(v[0], v[1]), max(v[2], v[3])));
                const size_t row = (size_t)it.m0 + r;
                *(uint2 *)(p.hq + row * NC + n) = quant8(o[i], bs);
                if (q == 0 && wn == 0) p.hqs[row * (NC >> 7) + it.nb] = bs.scale;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int r = 16 * (WM * i + wm) + m;
            if (r >= it.mrows) continue;
            uint16_t *row = p.out + (size_t)(it.m0 + r) * NC;
            if constexpr (SWIGLU) {
                const int n = packed_row(n0, 4 * q);
                if (n < NC) *(u32x4 *)(row + n) = output(i);
            } else {
                uint2 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[j] = make_uint2(pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3]));
                    if (!(live >> i & 1)) w[j] = make_uint2(0u, 0u);
                }
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const int n = packed_row(n0 + j, 4 * q);
                    if (n < NC) *(u32x4 *)(row + n) = u32x4{w[j].x, w[j].y, w[j + 1].x, w[j + 1].y};
                }
            }
        }
    };
    // (the products of rows that the tile does not have are left out, 32 WM rows at a time)
    const int need = (it.mrows + 32 * WM - 1) / (32 * WM);
    if constexpr (MW == 8) {
        if (need >= 4)
            body(std::integral_constant<int, 8>{});
        else if (need == 3)
            body(std::integral_constant<int, 6>{});
        else if (need == 2)
            body(std::integral_constant<int, 4>{});
        else
            body(std::integral_constant<int, 2>{});
    } else if constexpr (MW == 4) {
        if (need >= 2)
            body(std::integral_constant<int, 4>{});
        else
            body(std::integral_constant<int, 2>{});
    } else {
        body(std::integral_constant<int, 2>{});
    }
}

template <int ACT, int MW, int WM, int WN, int KS, int OCC, bool FAR = false, bool EXACT = false, bool QUANT = false>
void launch(Args a, hipStream_t st) {
    constexpr int TM = 16 * MW * WM;
    a.NB = (a.NT + 4 * WN - 1) / (4 * WN);
    int64_t tiles = a.offsets ? (int64_t)a.R / TM + (a.R < a.G ? a.R : a.G) : (a.R + TM - 1) / TM;
    if (tiles > a.R) tiles = a.R;  // every tile has a row
    const dim3 grid((unsigned)((tiles * a.NB + 7) / 8 * 8)), block(64 * WM * WN * KS);  // a whole slice per XCD
    hipLaunchKernelGGL((k_fp8s_tiled<ACT, MW, WM, WN, KS, OCC, FAR, EXACT, QUANT>), grid, block, 0, st, a);
}

}  // namespace

// Which tile, by measured times (us; 256 x 256, 64 x 128, the latter with k in two
// parts, 32 x 64 with k in four; rows x outputs x inputs, or rows a group of
// groups, outputs x inputs, in SwiGLU):
//   8192 x 4096 x 4096        142, 226, 296, 570
//   1024 x 4096 x 4096         46,  30,  36,  74
//    300 x 6160 x 2064         28, 14.4, 13.5, 29
//    128 x 4096 x 4096         32,  17,  14,  9.9
//    512 x 4096 x 1024         17, 7.9, 8.1,  20
//    256 x 1024 x 1024         17, 6.7, 6.8, 5.9
//   1738 of  33, 4096 x 4096 1114, 1579, 2278, 4898
//     72 of 257, 4096 x 4096 1017, 974, 1285, 2441
//    100 of  41, 1024 x 1024  20,  16,  27,  61
// The large tile multiplies most per byte brought in, but a CU holds one of
// them only; the others fill the CUs where tiles are few, and parts of k
// shorten the steps in a row where they would not fill them.
bool launch_tiled(int act, Args a, hipStream_t st) {
    const int64_t G = a.offsets ? a.G : 1;
    auto tiles = [&](int TM, int TN) {
        return (a.R / TM + (a.offsets ? std::min(a.R, a.G) : 1)) * (int64_t)((16 * a.NT + TN - 1) / TN);
    };
    constexpr int kSilu = MOE_ACT_SWIGLU, kPlain = MOE_ACT_NONE;
    const bool swiglu = act == MOE_ACT_SWIGLU;
    // SwiGLU's products in bf16 where its outputs are so few that the ones of
    // another code show in the layer's output, which a few large tokens can make
    // up (64 tokens of the 256-expert layer: error against 64 bits 0.0020 to 0.0033
    // without, 0.0017 with; 8192 tokens 0.0024), and where k in parts leaves the time
    // for them.  800 rows of 41 groups, 1024 x 1024: 13 -> 17 us, 18432 of 257,
    // 4096 x 4096, would be 974 -> 1259.  (MOE_ACT_SWIGLU_F32: always; 8192 tokens of the
    // 256-expert layer 2140 -> 3730.)
    const bool exact = swiglu && (a.f32 || (int64_t)a.R * a.N <= 1 << 23);
    if (a.gather && (int64_t)a.n_src * a.K > kNone) {
        if (exact)
            launch<kSilu, 2, 2, 2, 1, 2, true, true>(a, st);
        else
            swiglu ? launch<kSilu, 2, 2, 2, 1, 3, true>(a, st) : launch<kPlain, 2, 2, 2, 1, 3, true>(a, st);
    } else if (a.R >= 128 * G && tiles(256, 256) >= 256 && !exact) {
        if (swiglu && a.hq) {
            launch<kSilu, 8, 2, 4, 1, 2, false, false, true>(a, st);
            return true;
        }
        swiglu ? launch<kSilu, 8, 2, 4, 1, 2>(a, st) : launch<kPlain, 8, 2, 4, 1, 2>(a, st);
    } else if (a.KG >= 8 && tiles(32, 64) <= 320) {
        swiglu ? launch<kSilu, 2, 1, 1, 4, 2, false, true>(a, st) : launch<kPlain, 2, 1, 1, 4, 2>(a, st);
    } else if (a.KG >= 12 && tiles(64, 128) <= 320) {
        swiglu ? launch<kSilu, 2, 2, 2, 2, 2, false, true>(a, st) : launch<kPlain, 2, 2, 2, 2, 2>(a, st);
    } else if (exact) {
        launch<kSilu, 2, 2, 2, 1, 2, false, true>(a, st);
    } else {
        swiglu ? launch<kSilu, 2, 2, 2, 1, 3>(a, st) : launch<kPlain, 2, 2, 2, 1, 3>(a, st);
    }
    return false;
}

}  // namespace f8
}  // namespace moe
