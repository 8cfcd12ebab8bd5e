// moe_bf16_wide.hip -- the grouped bf16 products of the experts and of their
// gradients, on tiles of 32 MW rows by 32 NW columns.
//
// Four waves (2 x 2: rows x columns) compute a tile, each 16 MW x 16 NW of it, a
// wave per SIMD with its sums in the accumulation registers.  Per 64-wide step
// of the contraction both operands go from global memory straight into one of
// two LDS stages.  An operand whose rows run along the contraction (kNT: both;
// kNN: a) lies there as [row][64 k] and is read 16 bytes a lane; one whose rows
// run across it (kNN: b; kTN: both) lies as [64 k][column] and is read through
// the transposing LDS load, which hands each lane four k of one column.
//
// Half a step's operands are in registers while the half before it multiplies.
// In the middle of a step all of its stage is in registers, so that one barrier
// there lets the loads of the step after the next one begin, a whole step
// before they are needed.
//
// 57344 rows of 33 groups of 4096/2048: gate/up 1839 us, 1.05 PFLOP/s, rows'
// gradient 1604 to 1711, 1.13 to 1.20 (matrix units busy 53% at 2.2 GHz), weights' 1910
// and 950, 1.0 (44%); the library's product of 8192 x 8192 x 8192 does 0.97 to 1.36 in
// these forms.  The rest of the matrix units' time goes to what a CU's one large
// tile has nothing to overlap with, the first loads and the epilogue of each tile,
// and to waits at the barrier of a step (15 to 18% of the waves' cycles).  SwiGLU's
// gradient moves 1.4 GB in its epilogue: 1090 us where the product alone takes 825.
// Gradients added to fp32 read the old values there: the whole backward pass of
// 8192 tokens on these experts takes 5770 us with them in bf16, 6010 in fp32, 6940 added.
#include <algorithm>
#include <type_traits>

#include "moe_bf16.h"
#include "moe_dma.h"

namespace moe {
namespace b16 {
namespace {

typedef short v4s __attribute__((ext_vector_type(4)));

constexpr int kBK = 64;  // contraction per step

// What rows without a source are read as: the longest row that there is.
__device__ const u32x4 kZeros[2 * 65536 / 16] = {};

// Chunk c (16 bytes) of row r of a [row][64 k] stage sits at chunk c ^ swz(r);
// the lanes that one pass of an operand read serves (see lds_swz), two rows to
// each 256 bytes of banks, then lie on distinct banks.  The weights' rows are
// read in the order 16 (r / 4) + 4 j + r % 4 of each 64, so that a lane's
// results of four subtiles are 16 consecutive columns: their swizzle follows.
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int wswz(int r) { return ((r >> 1) & 1) | ((r >> 4) & 3) << 1; }
// Chunk c of row k of a [64 k][column] stage sits at chunk c ^ tswz(k): the
// eight rows that 32 lanes of a transposing read take, 32 bytes of each, then
// lie on distinct banks.
__device__ __forceinline__ int tswz(int k) { return 2 * ((k & 3) | ((k >> 3) & 1) << 2); }
// Load j of wave w brings the rows stage_row .. of such a stage of `width`
// columns (1 KB: two rows of 256, four of 128, eight of 64), in an order in
// which tswz is the same for all loads of a lane.
__device__ __forceinline__ int stage_row(int width, int j, int w) {
    if (width == 256) return 16 * (j >> 1) + 8 * (w >> 1) + 4 * (j & 1) + 2 * (w & 1);
    return 512 / width * (4 * j + w);
}

__device__ __forceinline__ v4s read_tr(const char *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)(uintptr_t)(lds_void_t *)p);
}
__device__ __forceinline__ bf16x8 read_tr2(const char *p, int next) {
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(read_tr(p), read_tr(p + next), 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ uint64_t choose(bool c, uint64_t a, uint64_t b) {
    const uint32_t lo = c ? (uint32_t)a : (uint32_t)b, hi = c ? (uint32_t)(a >> 32) : (uint32_t)(b >> 32);
    return (uint64_t)hi << 32 | lo;
}

// The matrix instructions of one operand with four or eight, written as
// assembly so that each accumulator stays in its registers: the compiler's own
// form rotates the accumulators of a large tile through copies and spills.
// The two wait states in front cover an operand that the instruction before
// wrote; an accumulator comes up again only after every other one (eight of
// them at least), and mfma_drain precedes the first use of the sums.  FIRST:
// the single operand is the first one.
template <bool FIRST>
__device__ __forceinline__ void mfma_row(f32x4 (&c)[8], bf16x8 a, bf16x8 (&b)[8]) {
    if constexpr (FIRST)
        asm volatile("s_nop 1\n\t"
                     "v_mfma_f32_16x16x32_bf16 %0, %8, %9, %0\n\t"
                     "v_mfma_f32_16x16x32_bf16 %1, %8, %10, %1\n\t"
                     "v_mfma_f32_16x16x32_bf16 %2, %8, %11, %2\n\t"
                     "v_mfma_f32_16x16x32_bf16 %3, %8, %12, %3\n\t"
                     "v_mfma_f32_16x16x32_bf16 %4, %8, %13, %4\n\t"
                     "v_mfma_f32_16x16x32_bf16 %5, %8, %14, %5\n\t"
                     "v_mfma_f32_16x16x32_bf16 %6, %8, %15, %6\n\t"
                     "v_mfma_f32_16x16x32_bf16 %7, %8, %16, %7"
                     : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3]), "+a"(c[4]), "+a"(c[5]), "+a"(c[6]), "+a"(c[7])
                     : "v"(a), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(b[4]), "v"(b[5]), "v"(b[6]), "v"(b[7]));
    else
        asm volatile("s_nop 1\n\t"
                     "v_mfma_f32_16x16x32_bf16 %0, %9, %8, %0\n\t"
                     "v_mfma_f32_16x16x32_bf16 %1, %10, %8, %1\n\t"
                     "v_mfma_f32_16x16x32_bf16 %2, %11, %8, %2\n\t"
                     "v_mfma_f32_16x16x32_bf16 %3, %12, %8, %3\n\t"
                     "v_mfma_f32_16x16x32_bf16 %4, %13, %8, %4\n\t"
                     "v_mfma_f32_16x16x32_bf16 %5, %14, %8, %5\n\t"
                     "v_mfma_f32_16x16x32_bf16 %6, %15, %8, %6\n\t"
                     "v_mfma_f32_16x16x32_bf16 %7, %16, %8, %7"
                     : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3]), "+a"(c[4]), "+a"(c[5]), "+a"(c[6]), "+a"(c[7])
                     : "v"(a), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(b[4]), "v"(b[5]), "v"(b[6]), "v"(b[7]));
}
template <bool FIRST>
__device__ __forceinline__ void mfma_row(f32x4 (&c)[4], bf16x8 a, bf16x8 (&b)[4]) {
    if constexpr (FIRST)
        asm volatile("s_nop 1\n\t"
                     "v_mfma_f32_16x16x32_bf16 %0, %4, %5, %0\n\t"
                     "v_mfma_f32_16x16x32_bf16 %1, %4, %6, %1\n\t"
                     "v_mfma_f32_16x16x32_bf16 %2, %4, %7, %2\n\t"
                     "v_mfma_f32_16x16x32_bf16 %3, %4, %8, %3"
                     : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3])
                     : "v"(a), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]));
    else
        asm volatile("s_nop 1\n\t"
                     "v_mfma_f32_16x16x32_bf16 %0, %5, %4, %0\n\t"
                     "v_mfma_f32_16x16x32_bf16 %1, %6, %4, %1\n\t"
                     "v_mfma_f32_16x16x32_bf16 %2, %7, %4, %2\n\t"
                     "v_mfma_f32_16x16x32_bf16 %3, %8, %4, %3"
                     : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3])
                     : "v"(a), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]));
}
__device__ __forceinline__ void mfma_drain() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

struct Item {
    int g, m0, mrows, nb, lo, hi;  // kTN: m0 the first column of a; [lo, hi) the group's rows
};

template <int FORM>
__device__ __forceinline__ bool find_item(const Args &p, int block, int TM, Item &it) {
    if constexpr (FORM == kTN) {
        // Every group's tiles are dealt to the eight XCDs in equal parts, the
        // groups last to first (the shared expert's, the longest, begins), so
        // that groups of different lengths keep all of them busy; in a part
        // four rows of tiles at a time, column by column.
        const int per_group = p.MB * p.NB, part = (per_group + 7) >> 3, j = block >> 3;
        const int local = (block & 7) * part + j % part;
        it.g = p.G - 1 - j / part;
        if (it.g < 0 || local >= per_group) return false;
        const int ch = local / (4 * p.NB), rem = local - ch * 4 * p.NB;
        const int mc = min(4, p.MB - 4 * ch);
        it.nb = rem / mc;
        it.m0 = (4 * ch + rem - it.nb * mc) * TM;
        it.mrows = min(TM, p.M - it.m0);
        it.lo = max(__builtin_amdgcn_readfirstlane(p.offsets[it.g]), 0);
        it.hi = min(__builtin_amdgcn_readfirstlane(p.offsets[it.g + 1]), p.R);
        return true;
    } else {
        TileItem t;
        if (!workgroup_tile_item(p.NB, TM, p.offsets, p.G, p.R, t)) return false;
        it.g = t.g;
        it.m0 = t.m0;
        it.mrows = t.mrows;
        it.nb = t.nb;
        it.lo = it.hi = 0;
        return true;
    }
}

// SWAP (kTN): the result is written transposed, out[G][N][M].
// A wave has MW m-tiles (16 rows) and NW subtiles (16 columns).
// (kNT, kNN: `block` is blockIdx.x.)
template <int MW, int NW>
constexpr int kStages = 2 * 32 * (MW + NW) * kBK * 2;  // bytes of the LDS stages
template <int FORM, int EPI, bool SWAP, int MW, int NW>
__device__ __forceinline__ void multiply(const Args &p, int block, char *stages) {
    constexpr int TM = 32 * MW, kCols = 32 * NW;  // rows and columns of a tile
    constexpr bool TRA = FORM == kTN, TRB = FORM != kNT;
    constexpr int ABYTES = TM * kBK * 2, BBYTES = kCols * kBK * 2;  // of a stage
    constexpr int LA = MW, LB = NW;                                 // loads of a and b per wave and step
    char *const sA = stages, *const sB = stages + 2 * ABYTES;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = lane_id();
    const int wm = wave >> 1, wn = wave & 1, m = l & 15, q = l >> 4;
    Item it;
    if (!find_item<FORM>(p, block, TM, it)) return;
    const int KC = FORM == kTN ? max(it.hi - it.lo, 0) : p.K;  // contraction
    if (EPI == kAddF32 && KC == 0) return;  // a group without rows: its gradient stays as it is
    const int KG = (KC + kBK - 1) / kBK;
    // columns of the tile: of the output, or (SwiGLU) half of them of the gate
    // projection and the same of the up projection
    const int n0 = it.nb * (EPI == kSwiglu ? kCols / 2 : kCols);
    const uint32_t ldsA = lds_address(sA), ldsB = lds_address(sB);
    const uint64_t zero = (uint64_t)kZeros;

    // ---- a into LDS.  Rows along the contraction: load j brings eight of
    // them; across it: 1 KB of the stage.
    constexpr int RPL = 1024 / (2 * TM), LPR = 64 / RPL;  // kTN: rows of a load, lanes of a row
    uint64_t asrc[LA], acol = 0;
    int arow[LA];
    auto a_row = [&](int j) {  // kTN: the lane's row of load j
        return stage_row(TM, j, wave) + l / LPR;
    };
    auto a_chunk = [&](int j) { return (l & 7) ^ swz(8 * (LA * wave + j) + (l >> 3)); };
    const int n_rows = p.gather ? p.n_src : FORM == kTN ? it.hi : p.R;
    if constexpr (!TRA) {
#pragma unroll
        for (int j = 0; j < LA; ++j) {
            const int r = 8 * (LA * wave + j) + (l >> 3);
            int src = it.m0 + min(r, it.mrows - 1);
            if (p.gather) src = p.gather[src];
            // (a row without a source, or past the tile's last: zeros)
            asrc[j] = r < it.mrows && (unsigned)src < (unsigned)n_rows
                          ? (uint64_t)(p.a + (size_t)src * p.K + 8 * a_chunk(j)) : zero;
        }
    } else {
        // columns past the last are any of the others
        acol = (uint64_t)(p.a + min(it.m0 + 8 * ((l % LPR) ^ tswz(a_row(0)) & (LPR - 1)), p.M - 8));
    }
    auto rows_of = [&](int kg) {  // kTN: the rows of the next step to be loaded
        if constexpr (TRA) {
#pragma unroll
            for (int j = 0; j < LA; ++j) {
                const int r = it.lo + kBK * kg + a_row(j);
                arow[j] = p.gather ? p.gather[min(r, p.R - 1)] : r;
            }
        }
    };
    // (cut: step kg may have less than 64 of the contraction left, the rest is zeros)
    auto load_a = [&](auto cut, int kg, int stage, int j) {
        if constexpr (!TRA) {
            uint64_t at = asrc[j] + 2 * kBK * (uint64_t)kg;
            if (cut) at = choose(kBK * kg + 8 * a_chunk(j) < KC, at, zero);
            dma16_pointer(at, ldsA + stage * ABYTES + 1024 * (LA * wave + j));
        } else {
            uint64_t at = acol + (uint64_t)(uint32_t)arow[j] * (uint32_t)(2 * p.M);
            asm volatile("" : "+v"(at));  // (formed in all lanes, not under the condition below)
            const bool in = (unsigned)arow[j] < (unsigned)n_rows && (!cut || kBK * kg + a_row(j) < KC);
            dma16_pointer(choose(in, at, zero), ldsA + stage * ABYTES + 2 * TM * stage_row(TM, j, wave));
        }
    };
    // ---- b into LDS
    const size_t ld = 2 * (size_t)(FORM == kNT ? p.K : p.N);
    constexpr int LPB = kCols / 8;  // lanes of a row of a [64 k][column] stage
    const char *bbase;
    int64_t bbytes;
    uint32_t boff[4];
    i32x4 bbuf, ubuf;
    if constexpr (!TRB) {
        // Load j of a wave brings rows 8 (NW wave + j) + l / 8 of the stage,
        // of which each 16 NW are a wave column's.  SwiGLU: four subtiles of
        // the gate rows and four of the up rows in turn (NW = 8), or two and
        // two, every other eight rows, so that a lane's results of either are
        // consecutive columns there too.
        const int row = EPI == kSwiglu ? n0 + 8 * NW * (wave >> 1) + (NW == 8 ? ((wave & 1) ? p.N >> 1 : 0) : 16 * (wave & 1))
                                       : n0 + 8 * NW * wave;
        bbase = (const char *)p.b + ((size_t)it.g * p.N + row) * ld;
        bbytes = (int64_t)(p.N - row) * ld;
        bbuf = buffer(bbase, bbytes);
        if (EPI == kSwiglu && NW == 4) ubuf = buffer(bbase + (size_t)(p.N >> 1) * ld, bbytes - (int64_t)(p.N >> 1) * ld);
#pragma unroll
        for (int x = 0; x < 4; ++x) boff[x] = (uint32_t)((l >> 3) * ld) + 16 * ((l & 7) ^ wswz(16 * x + (l >> 3)));
    } else {
        bbase = (const char *)p.b + (FORM == kNN ? (size_t)it.g * p.K : (size_t)it.lo) * ld + 2 * (size_t)n0;
        bbytes = (int64_t)KC * ld - 2 * (int64_t)n0;
        const int k = stage_row(kCols, 0, wave) + l / LPB;
        boff[0] = (uint32_t)(k * ld) + 16 * ((l % LPB) ^ (tswz(k) & (LPB - 1)));
    }
    auto load_b = [&](auto cut, int kg, int stage, int j) {
        const uint32_t lds = ldsB + stage * BBYTES;
        if constexpr (!TRB) {
            const int r = 8 * (NW * wave + j);  // (the swizzle goes by its place in 64 rows)
            const int x = NW == 8 ? j >> 1 : (2 * wave + (j >> 1)) & 3;
            const bool u = EPI == kSwiglu && NW == 4 && (j & 1);
            const int row = EPI == kSwiglu && NW == 4 ? 8 * (j >> 1) : 8 * j;
            uint32_t voff = (NW == 8 ? boff[j >> 1] : (wave & 1) ? boff[2 + (j >> 1)] : boff[j >> 1]) + (uint32_t)(row * ld) + 128 * kg;
            if (cut && kBK * kg + 8 * ((l & 7) ^ wswz(16 * x + (l >> 3))) >= KC) voff = kFar;
            dma16_buffer(u ? ubuf : bbuf, voff, lds + 128 * r);
        } else {
            if (j == 0) bbuf = buffer(bbase + (size_t)kg * kBK * ld, bbytes - (int64_t)kg * kBK * ld);
            uint32_t voff = boff[0] + (uint32_t)(stage_row(kCols, j, 0) * ld);
            if constexpr (FORM == kTN) {  // a row that a has no source for adds nothing, whatever b has there
                static_assert(TM == kCols, "load j brings the same rows of both");
                if ((unsigned)arow[j] >= (unsigned)n_rows) voff = kFar;
            }
            dma16_buffer(bbuf, voff, lds + 2 * kCols * stage_row(kCols, j, wave));
        }
    };

    // kSwigluBwd: the routing weight of one of the tile's rows per thread
    float row_w = 1.0f;
    if constexpr (EPI == kSwigluBwd) {
        if (tid < it.mrows) {
            const int r = it.m0 + tid, t = p.gather[r], S = p.k + p.ns;
            if ((unsigned)t < (unsigned)p.n_src)
                for (int j = 0; j < p.k; ++j)
                    if (p.row_of_slot[(size_t)t * S + j] == r) row_w = p.topk_w[(size_t)t * p.k + j];
        }
    }
    __shared__ float sW[EPI == kSwigluBwd ? TM : 1];

    auto body = [&](auto cc) {
        constexpr int C = decltype(cc)::value;  // m-tiles of a wave that have rows
        // ---- operand reads.  Wave row wm takes the m-tiles 2 c + wm of the
        // tile, so that a tile of few rows is shared by both (kTN: C wm + c).
        auto m_tile = [&](int c) { return FORM == kTN ? C * wm + c : 2 * c + wm; };
        auto read_a = [&](int stage, int h, int c) -> bf16x8 {
            const char *A = sA + stage * ABYTES;
            const int t = m_tile(c);
            if constexpr (!TRA) {
                return *(const bf16x8 *)(A + (16 * t + m) * 128 + 16 * ((4 * h + q) ^ swz(m)));
            } else {
                const int k = 8 * q + (m >> 2), x = (2 * t + ((m & 3) >> 1)) ^ (tswz(k) & (TM / 8 - 1));
                return read_tr2(A + (k + 32 * h) * (2 * TM) + 16 * x + 8 * (m & 1), 4 * (2 * TM));
            }
        };
        auto read_b = [&](int stage, int h, int j) -> bf16x8 {
            const char *B = sB + stage * BBYTES;
            if constexpr (!TRB) {
                const int r = 16 * NW * wn + 64 * (j >> 2) + 16 * (m >> 2) + 4 * (j & 3) + (m & 3);
                return *(const bf16x8 *)(B + r * 128 + 16 * ((4 * h + q) ^ swz(m)));
            } else {
                const int k = 8 * q + (m >> 2), x = (2 * NW * wn + 2 * j + ((m & 3) >> 1)) ^ (tswz(k) & (LPB - 1));
                return read_tr2(B + (k + 32 * h) * (2 * kCols) + 16 * x + 8 * (m & 1), 4 * (2 * kCols));
            }
        };
        f32x4 acc[C][NW];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < NW; ++j) acc[c][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        bf16x8 a0[C], a1[C], b0[NW], b1[NW];
        if (KG > 0) {
            rows_of(0);
#pragma unroll
            for (int j = 0; j < LA; ++j) load_a(std::true_type(), 0, 0, j);
#pragma unroll
            for (int j = 0; j < LB; ++j) load_b(std::true_type(), 0, 0, j);
            rows_of(1);
#pragma unroll
            for (int j = 0; j < LA; ++j) load_a(std::true_type(), min(1, KG - 1), 1, j);
#pragma unroll
            for (int j = 0; j < LB; ++j) load_b(std::true_type(), min(1, KG - 1), 1, j);
            rows_of(2);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(LA + LB));
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < C; ++c) a0[c] = read_a(0, 0, c);
#pragma unroll
            for (int j = 0; j < NW; ++j) b0[j] = read_b(0, 0, j);
        }
        // The matrix instructions of m-tile c of half a step
        auto multiply = [&](int c, bf16x8(&a)[C], bf16x8(&b)[NW]) {
            mfma_row<SWAP>(acc[c], a[c], b);
        };
        constexpr int PB = (NW + C - 1) / C > 2 ? (NW + C - 1) / C : 2;  // operand reads of b per m-tile
        constexpr int PL = (LA + LB + C - 1) / C;  // loads into LDS per m-tile
        auto step = [&](auto cut, int kg, int s) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                a1[c] = read_a(s, 1, c);
#pragma unroll
                for (int j = PB * c; j < PB * (c + 1) && j < NW; ++j) b1[j] = read_b(s, 1, j);
                multiply(c, a0, b0);
                __builtin_amdgcn_sched_barrier(0);
            }
            // This step's stage is in registers, the next one's has landed;
            // past the barrier that holds for every wave.
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(0) & ~0x0F00);
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            const int next = min(kg + 2, KG - 1);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                a0[c] = read_a(s ^ 1, 0, c);
#pragma unroll
                for (int j = PB * c; j < PB * (c + 1) && j < NW; ++j) b0[j] = read_b(s ^ 1, 0, j);
#pragma unroll
                for (int x = PL * c; x < PL * (c + 1) && x < LA + LB; ++x) x < LA ? load_a(cut, next, s, x) : load_b(cut, next, s, x - LA);
                if (c == C - 1) rows_of(kg + 3);
                multiply(c, a1, b1);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        const int plain = KC % kBK ? KG - 3 : KG;  // steps that load whole ones
        int kg = 0;
#pragma unroll 1
        for (; kg + 2 <= plain; kg += 2) {
            step(std::false_type(), kg, 0);
            step(std::false_type(), kg + 1, 1);
        }
#pragma unroll 1
        for (; kg < KG; ++kg) step(std::true_type(), kg, kg & 1);
        mfma_drain();
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < NW; ++j) asm volatile("" : "+a"(acc[c][j]));  // no use before the drain
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));                              // no load into LDS outlives the block
        __builtin_amdgcn_sched_barrier(0);

        // ---- epilogue.  Lane (m, q) holds, of row 16 (2 c + wm) + m, four
        // columns of each of its wave's subtiles.
        if constexpr (SWAP) {  // ... of column 16 j + m, four rows of each m-tile
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const int n = n0 + 16 * NW * wn + 16 * j + m;
                const size_t at = ((size_t)it.g * p.N + n) * p.M + it.m0;
                if constexpr (EPI == kStore) {
                    // pairs of m-tiles: after the exchange a lane has eight consecutive rows of one of the two
#pragma unroll
                    for (int c = 0; c < C; c += 2) {
                        const auto x = __builtin_amdgcn_permlane16_swap(pack_bf16x2(acc[c][j][0], acc[c][j][1]),
                                                                        pack_bf16x2(acc[c + 1][j][0], acc[c + 1][j][1]), false, false);
                        const auto y = __builtin_amdgcn_permlane16_swap(pack_bf16x2(acc[c][j][2], acc[c][j][3]),
                                                                        pack_bf16x2(acc[c + 1][j][2], acc[c + 1][j][3]), false, false);
                        const int r = 16 * m_tile(c) + 16 * (q & 1) + 8 * (q >> 1);
                        if (n < p.N && r < it.mrows) *(u32x4 *)((uint16_t *)p.out + at + r) = u32x4{x[0], y[0], x[1], y[1]};
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int r = 16 * m_tile(c) + 4 * q;
                        if (n >= p.N || r >= it.mrows) continue;
                        f32x4 *out = (f32x4 *)((float *)p.out + at + r);
                        *out = EPI == kAddF32 ? *out + acc[c][j] : acc[c][j];
                    }
                }
            }
            return;
        }
        float *red = (float *)sA;  // kSwigluBwd: [2][TM]
        if constexpr (EPI == kSwigluBwd) {
            if (tid < TM) sW[tid] = row_w;
            __syncthreads();
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int r = 16 * m_tile(c) + m;
            const bool in = r < it.mrows;
            const size_t row = FORM == kTN ? (size_t)it.g * p.M + it.m0 + r : (size_t)it.m0 + r;
            if constexpr (EPI == kSwigluBwd) {
                // pairs of subtiles: after the exchange a lane has eight
                // consecutive columns of one of the two
                const float w = sW[r];
                float dot = 0.0f;
                u32x4 gv[NW / 2], uv[NW / 2], hv[NW / 2];
#pragma unroll
                for (int j = 0; j < NW / 2; ++j) {
                    const int n = n0 + 16 * NW * wn + 32 * j + 16 * (q & 1) + 8 * (q >> 1);
                    gv[j] = uv[j] = hv[j] = u32x4{0u, 0u, 0u, 0u};
                    if (in && n < p.N) {
                        gv[j] = *(const u32x4 *)(p.gu_in + row * 2 * p.N + n);
                        uv[j] = *(const u32x4 *)(p.gu_in + row * 2 * p.N + p.N + n);
                        hv[j] = *(const u32x4 *)(p.h + row * p.N + n);
                    }
                }
#pragma unroll
                for (int j = 0; j < NW / 2; ++j) {
                    const int n = n0 + 16 * NW * wn + 32 * j + 16 * (q & 1) + 8 * (q >> 1);
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[c][2 * j][e]),
                                                                        __float_as_uint(acc[c][2 * j + 1][e]), false, false);
                        d[e] = __uint_as_float(x[0]);
                        d[4 + e] = __uint_as_float(x[1]);
                    }
                    u32x4 og, ou, oh;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float dg[2], du[2], hw[2];
                        swiglu_gradient(d[2 * e], w, bf16lo_to_f32(gv[j][e]), bf16lo_to_f32(uv[j][e]),
                                        bf16lo_to_f32(hv[j][e]), dot, dg[0], du[0], hw[0]);
                        swiglu_gradient(d[2 * e + 1], w, bf16hi_to_f32(gv[j][e]), bf16hi_to_f32(uv[j][e]),
                                        bf16hi_to_f32(hv[j][e]), dot, dg[1], du[1], hw[1]);
                        og[e] = pack_bf16x2(dg[0], dg[1]);
                        ou[e] = pack_bf16x2(du[0], du[1]);
                        oh[e] = pack_bf16x2(hw[0], hw[1]);
                    }
                    if (p.dgu && in && n < p.N) {
                        *(u32x4 *)(p.dgu + row * 2 * p.N + n) = og;
                        *(u32x4 *)(p.dgu + row * 2 * p.N + p.N + n) = ou;
                    }
                    if (p.hw && in && n < p.N) *(u32x4 *)(p.hw + row * p.N + n) = oh;
                }
                dot += __shfl_xor(dot, 16, kWave);
                dot += __shfl_xor(dot, 32, kWave);
                if (q == 0) red[wn * TM + r] = dot;
            } else if constexpr (EPI == kSwiglu) {
                constexpr int HS = NW / 2;  // a lane has 4 HS consecutive columns of either projection
                if (!in) continue;
                const int NC = p.N >> 1, n = n0 + 16 * HS * wn + 4 * HS * q;
                if (n >= NC) continue;
                uint32_t o[2 * HS], g[2 * HS], u[2 * HS];
#pragma unroll
                for (int j = 0; j < HS; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float g0 = acc[c][j][2 * e], g1 = acc[c][j][2 * e + 1];
                        const float u0 = acc[c][j + HS][2 * e], u1 = acc[c][j + HS][2 * e + 1];
                        g[2 * j + e] = pack_bf16x2(g0, g1);
                        u[2 * j + e] = pack_bf16x2(u0, u1);
                        o[2 * j + e] = pack_bf16x2(silu_mul(g0, u0), silu_mul(g1, u1));
                    }
                uint16_t *out = (uint16_t *)p.out + row * NC + n, *gu = p.gu + row * p.N + n;
#pragma unroll
                for (int x = 0; x < HS / 2; ++x) {
                    ((u32x4 *)out)[x] = u32x4{o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]};
                    if (p.gu) {
                        ((u32x4 *)gu)[x] = u32x4{g[4 * x], g[4 * x + 1], g[4 * x + 2], g[4 * x + 3]};
                        ((u32x4 *)(gu + NC))[x] = u32x4{u[4 * x], u[4 * x + 1], u[4 * x + 2], u[4 * x + 3]};
                    }
                }
            } else if constexpr (EPI == kStore) {
#pragma unroll
                for (int j = 0; j < NW; j += 2) {
                    const uint32_t a0 = pack_bf16x2(acc[c][j][0], acc[c][j][1]), a1 = pack_bf16x2(acc[c][j][2], acc[c][j][3]);
                    const uint32_t b0 = pack_bf16x2(acc[c][j + 1][0], acc[c][j + 1][1]);
                    const uint32_t b1 = pack_bf16x2(acc[c][j + 1][2], acc[c][j + 1][3]);
                    u32x4 v;
                    int n;
                    if constexpr (TRB) {  // eight consecutive columns of one of the two subtiles
                        const auto x = __builtin_amdgcn_permlane16_swap(a0, b0, false, false);
                        const auto y = __builtin_amdgcn_permlane16_swap(a1, b1, false, false);
                        v = u32x4{x[0], y[0], x[1], y[1]};
                        n = n0 + 16 * NW * wn + 16 * j + 16 * (q & 1) + 8 * (q >> 1);
                    } else {  // sixteen in four subtiles
                        v = u32x4{a0, a1, b0, b1};
                        n = n0 + 16 * NW * wn + 64 * (j >> 2) + 16 * q + 4 * (j & 3);
                    }
                    if (in && n < p.N) *(u32x4 *)((uint16_t *)p.out + row * p.N + n) = v;
                }
            } else {
                if (!in) continue;
#pragma unroll
                for (int j = 0; j < NW; ++j) {
                    const int n = n0 + 16 * NW * wn + 16 * j + 4 * q;
                    if (n >= p.N) continue;
                    f32x4 *at = (f32x4 *)((float *)p.out + row * p.N + n);
                    *at = EPI == kAddF32 ? *at + acc[c][j] : acc[c][j];
                }
            }
        }
        if constexpr (EPI == kSwigluBwd) {
            __syncthreads();
            if (tid < it.mrows) p.part[(size_t)it.nb * p.R + it.m0 + tid] = red[tid] + red[TM + tid];
        }
    };
    const int pairs = (it.mrows + 31) >> 5;  // m-tiles of a wave that have rows
    if constexpr (FORM == kTN || MW <= 4) {
        body(std::integral_constant<int, MW>());
    } else {
        if (pairs > 6)
            body(std::integral_constant<int, 8>());
        else if (pairs > 4)
            body(std::integral_constant<int, 6>());
        else if (pairs > 2)
            body(std::integral_constant<int, 4>());
        else
            body(std::integral_constant<int, 2>());
    }
}

// OCC workgroups share a CU.
template <int FORM, int EPI, bool SWAP, int MW, int NW, int OCC>
__global__ __launch_bounds__(256, OCC) void k_bf16_wide(Args p) {
    __shared__ __attribute__((aligned(16))) char stages[kStages<MW, NW>];
    multiply<FORM, EPI, SWAP, MW, NW>(p, blockIdx.x, stages);
}

// What the backward pass computes from d_gu and hw, in one launch: the first n_x
// workgroups the rows' gradients, n_w13 and the others the weights'.
template <int EPI>
__global__ __launch_bounds__(256, 2) void k_bf16_gradients(Args x, Args w13, Args w2, int n_x, int n_w13) {
    __shared__ __attribute__((aligned(16))) char stages[kStages<4, 4>];
    const int b = blockIdx.x;
    if (b < n_x)
        multiply<kNN, kStore, false, 2, 4>(x, b, stages);
    else if (b < n_x + n_w13)
        multiply<kTN, EPI, true, 4, 4>(w13, b - n_x, stages);
    else
        multiply<kTN, EPI, false, 4, 4>(w2, b - n_x - n_w13, stages);
}

// Workgroups of a launch; sets the numbers of tiles.
template <int FORM, int EPI, int MW, int NW>
unsigned count(Args &p) {
    constexpr int TM = 32 * MW, TN = EPI == kSwiglu ? 16 * NW : 32 * NW;
    const int cols = EPI == kSwiglu ? p.N / 2 : p.N;
    p.NB = (cols + TN - 1) / TN;
    int64_t items;
    if (FORM == kTN) {
        p.MB = (p.M + TM - 1) / TM;
        items = (int64_t)p.G * ((p.MB * p.NB + 7) / 8 * 8);
    } else {
        int64_t tiles = (int64_t)p.R / TM + std::min(p.R, p.G);
        tiles = std::min<int64_t>(tiles, p.R);  // every tile has a row
        items = (tiles * p.NB + 7) / 8 * 8;
    }
    return (unsigned)items;
}

template <int FORM, int EPI, bool SWAP, int MW, int NW, int OCC>
int launch(Args p, hipStream_t st) {
    const unsigned items = count<FORM, EPI, MW, NW>(p);
    hipLaunchKernelGGL((k_bf16_wide<FORM, EPI, SWAP, MW, NW, OCC>), dim3(items), dim3(256), 0, st, p);
    return p.NB;
}

template <int EPI>
void launch_gradients(Args x, Args w13, Args w2, hipStream_t st) {
    const unsigned n_x = count<kNN, kStore, 2, 4>(x), n_w13 = count<kTN, EPI, 4, 4>(w13), n_w2 = count<kTN, EPI, 4, 4>(w2);
    hipLaunchKernelGGL(k_bf16_gradients<EPI>, dim3(n_x + n_w13 + n_w2), dim3(256), 0, st, x, w13, w2, (int)n_x, (int)n_w13);
}

template <int MW, int NW, int OCC>
int launch_rows(int form, int epi, const Args &p, hipStream_t st) {
    if (form == kNT && epi == kSwiglu) return launch<kNT, kSwiglu, false, MW, NW, OCC>(p, st);
    if (form == kNT) return launch<kNT, kStore, false, MW, NW, OCC>(p, st);
    if (epi == kSwigluBwd) return launch<kNN, kSwigluBwd, false, MW, NW, OCC>(p, st);
    return launch<kNN, kStore, false, MW, NW, OCC>(p, st);
}

template <int MW, int NW, int OCC>
int launch_weights(int epi, const Args &p, hipStream_t st) {
    if (p.swap) {
        if (epi == kStore) return launch<kTN, kStore, true, MW, NW, OCC>(p, st);
        if (epi == kStoreF32) return launch<kTN, kStoreF32, true, MW, NW, OCC>(p, st);
        return launch<kTN, kAddF32, true, MW, NW, OCC>(p, st);
    }
    if (epi == kStore) return launch<kTN, kStore, false, MW, NW, OCC>(p, st);
    if (epi == kStoreF32) return launch<kTN, kStoreF32, false, MW, NW, OCC>(p, st);
    return launch<kTN, kAddF32, false, MW, NW, OCC>(p, st);
}

}  // namespace

namespace {
int64_t tiles(const Args &p, int form, int epi, int TM, int TN) {
    const int64_t nb = ((epi == kSwiglu ? p.N / 2 : p.N) + (epi == kSwiglu ? TN / 2 : TN) - 1) / (epi == kSwiglu ? TN / 2 : TN);
    if (form == kTN) return (int64_t)p.G * ((p.M + TM - 1) / TM) * nb;
    return ((p.R + TM - 1) / TM + std::min(p.R, p.G) / 2) * nb;
}
}  // namespace

// Which tile, by measured times (us; 256 x 256, 128 x 128, 64 x 128; rows a
// group, groups, layer):
//   gate/up, 1738 rows, 33 groups, 4096/2048: 1839, 2769, 3371; 434 rows: 498, 711, 905
//   gate/up, 390 rows, 41 groups, 1024/512:   59, 61, 60;  100 rows: 31, 25, 24;  39 rows: 30, 24, 22
//   dxs,     1738 rows, 33 groups, 4096/2048: 1711, 2137, 2726; 56 rows, 257 groups: 1690, 1584, 1696
//   dxs,     390 rows, 41 groups, 1024/512:   59, 50, 52;  9 rows, 17 groups, 512/256: 11, 8.3, 7.3
//   d_w13,   1738 rows, 33 groups, 4096/2048: 1998, 2405, 2765; 23 rows, 65 groups, 2048/768: 130, 148, 170
//   d_w13,   390 rows, 41 groups, 1024/512:   111, 70, 76; d_w2 there: 103, 54, 47
// The large tile reads least per product and needs two rounds of them to fill
// the CUs (each has one); the middle one, two to a CU, hides its start and its
// end behind the other's work; the small one is for a few rows.
int launch_wide(int form, int epi, const Args &p, hipStream_t st) {
    const int64_t large = tiles(p, form, epi, 256, 256);
    if (form == kTN) return large >= 2048 ? launch_weights<8, 8, 1>(epi, p, st) : launch_weights<4, 4, 2>(epi, p, st);
    if (p.R >= 128 * (int64_t)p.G && large >= 512) return launch_rows<8, 8, 1>(form, epi, p, st);
    if (p.R >= 48 * (int64_t)p.G) return launch_rows<4, 4, 2>(form, epi, p, st);
    return launch_rows<2, 4, 3>(form, epi, p, st);
}

// One launch in place of three where none of them is of the large tile (50
// tokens on 17 experts of 512/256: 37.4 -> 26.2 us for the backward pass, 1021 on
// 41 of 1024/512: 133 -> 124).
bool launch_gradients(int epi, const Args &x, const Args &w13, const Args &w2, hipStream_t st) {
    if (tiles(w13, kTN, epi, 256, 256) >= 2048 || tiles(w2, kTN, epi, 256, 256) >= 2048) return false;
    if (x.R >= 128 * (int64_t)x.G && tiles(x, kNN, kStore, 256, 256) >= 512) return false;
    epi == kStore      ? launch_gradients<kStore>(x, w13, w2, st)
    : epi == kStoreF32 ? launch_gradients<kStoreF32>(x, w13, w2, st)
                       : launch_gradients<kAddF32>(x, w13, w2, st);
    return true;
}

}  // namespace b16
}  // namespace moe
