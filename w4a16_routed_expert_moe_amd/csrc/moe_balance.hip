// moe_balance.hip -- the router's balance: tokens per expert, the balance
// loss of packed sequences, and the gradient of the router's logits.
//
//   s[t][e] = sigmoid(logits[t][e]),  p[t][e] = s[t][e] / sum_j s[t][j]
//   counts[q][e], prob_sums[q][e]: per sequence q, over its live tokens
//   loss = sum_q coef[q] sum_e counts[q][e] prob_sums[q][e],
//   coef[q] = alpha E / (k n_q^2 Q')
//
// The loss reads every logit once and the gradient reads and writes every
// one once: at 65536 x 256, 67 MB in 19 to 24 us plus 6 us for the sums of the
// chunks, and 134 MB in 28 to 29 us (4.7 TB/s, near a copy's rate).  Up to 8192
// tokens both are bound by latency: 4 to 9 us a launch.  A wave takes a token;
// a lane holds four experts, so the sum over a token's experts is one wave
// reduction and the sums over tokens stay in registers.
#include <algorithm>

#include "moe_route_common.h"

namespace moe {
namespace {

constexpr int kSlots = 4;          // experts per lane: E <= 256
constexpr int kMaxExperts = kSlots * kWave;
// Up to here the loss is one workgroup's work, one launch: about 0.8 us per
// sequence.  Loss + gradient of 256 experts, us, captured / called one by one,
// against two launches for the loss:
//   8 tokens, 6 sequences     9.0 / 10.3   12.8 / 12.9
//   33 tokens, 1 sequence     8.2 / 10.4   10.7 / 12.9
//              4             10.6 / 10.7   11.9 / 12.9
//              6             12.1 / 12.3   12.1 / 12.9
//   128 tokens, 1 sequence   10.7 / 11.0   11.2 / 15.0
//               4            13.1 / 13.4   11.6 / 14.6
//               6            14.7 / 15.1   11.7 / 14.9
// The bounds are where the calls one by one, which the host's launches weigh
// on, break even.
constexpr int kOneTokens = 128, kOneSeqs = 6;
// Token chunks of the partial sums: one per CU, past 16384 tokens two, of at
// least 8 tokens and at most as many as fit the registers (past 65536 tokens
// the chunks stay as long and get more: 8192 at 2^20).
constexpr int kChunks = 256;
constexpr int kMinChunk = 8, kMaxChunk = 128;

// the tokens of one chunk, a power of two
int chunk_tokens(int T) {
    int C = kMinChunk;
    while (C < kMaxChunk && (int64_t)C * kChunks * (T > 16384 ? 2 : 1) < T) C *= 2;
    return C;
}
int chunk_count(int T) { return (T + chunk_tokens(T) - 1) / chunk_tokens(T); }
// The most chunks of any call with up to T tokens, which is not always that of
// T: where the chunk's length doubles (past 2048, 4096, ..., 32768 tokens) the
// count halves.
int most_chunks(int T) {
    int n = chunk_count(T);
    for (int64_t t = (int64_t)kMinChunk * kChunks; t < T; t *= 2) n = std::max(n, chunk_count((int)t));
    return n;
}

// e^y = 2^p (1 + d): p is y log2(e) rounded to fp32, which alone would leave a
// relative error that grows with |y| (4e-6 at 80), and d = y - p ln 2 is what
// the rounding left out (with ln 2 itself rounded: 2 units of 2^-23 at |y| =
// 87, where e^-y leaves the normal range).  The loss of 65536 x 256 takes 23.8
// us with it and 22.9 without, its gradient 33.3 and 32.8; the probabilities'
// errors at 60 <= |y| <= 87 are 3.5 units of 2^-23 at most instead of 32.
// Where y is infinite, so is p, and d would be inf - inf: any small number does.
__device__ __forceinline__ float exp_split(float y, float &d) {
    const float p = y * route::kLog2e;
    d = fminf(__builtin_fmaf(-p, (float)route::kLn2, y), 0.5f);
    return __builtin_amdgcn_exp2f(p);
}
// Sigmoid s and its slope s (1 - s) from e = exp(-|x|), which neither
// overflows nor cancels: s = 1 / (1 + e) or e / (1 + e), slope = e / (1 + e)^2.
// Within five (s) and eight (slope) units of 2^-23: the hardware exponential
// and reciprocal are good to one each.  Nothing is selected by these scores.
// Scores below 2^-126 become 0; a NaN stays one.
__device__ __forceinline__ float score(float x, float &slope) {
    float d;
    const float e0 = exp_split(-fabsf(x), d), e = __builtin_fmaf(e0, d, e0);
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    slope = e * r * r;
    return x < 0.0f ? e * r : r;
}
// the score alone (exp(-x) = inf gives 0)
__device__ __forceinline__ float score(float x) {
    float d;
    const float e = exp_split(-x, d);
    return __builtin_amdgcn_rcpf(__builtin_fmaf(e, 1.0f + d, 1.0f));
}

// the expert of slot i of a lane: VEC four consecutive ones (16-byte loads),
// else one in each block of 64 (any E, any alignment)
template <bool VEC>
__device__ __forceinline__ int expert_of(int i) {
    return VEC ? 4 * lane_id() + i : lane_id() + kWave * i;
}
// A row's logits; past its end the lane takes others of the row, which no
// caller uses: a load under a condition would be waited for before the next.
template <bool VEC>
__device__ __forceinline__ void load_row(const float *__restrict__ row, int E, float (&x)[kSlots]) {
    if (VEC) {
        const float4 v = *(const float4 *)(row + min(4 * lane_id(), E - 4));
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) x[i] = row[min(expert_of<VEC>(i), E - 1)];
    }
}

struct Seqs {
    const int32_t *offsets;  // null: one sequence [0, T)
    const uint8_t *mask;     // null: every token is live
    int n, T;
};
__device__ __forceinline__ int seq_begin(const Seqs &q, int s) {
    return q.offsets ? min(max(q.offsets[s], 0), q.T) : 0;
}
__device__ __forceinline__ int seq_end(const Seqs &q, int s) {
    return q.offsets ? min(max(q.offsets[s + 1], 0), q.T) : q.T;
}

// The first sequence that ends past token t (n if none): each round the 64
// lanes probe 64 equally spaced ends, so 64 sequences take one memory round
// trip and a million take four.
__device__ __forceinline__ int seq_of(const Seqs &q, int t) {
    if (!q.offsets) return t < q.T ? 0 : 1;
    int lo = 0, hi = q.n;
    while (lo < hi) {
        const int step = (hi - lo + kWave - 1) / kWave;
        const int at = lo + (lane_id() + 1) * step - 1;  // the last of the lane's share
        const bool before = at < hi && q.offsets[min(at, q.n - 1) + 1] <= t;
        const int skip = __popcll(__ballot(before));
        lo += skip * step;
        if (step == 1) break;
        hi = min(hi, lo + step);  // the answer is among the next share's
    }
    return __builtin_amdgcn_readfirstlane(min(lo, q.n));
}

// seq_of with that sequence's bounds (the last one's where there is none):
// up to 64 sequences take one memory round trip together.
__device__ __forceinline__ int seq_at(const Seqs &q, int t, int &begin, int &end) {
    if (q.offsets && q.n <= kWave) {
        const int i = min(lane_id(), q.n - 1), b = q.offsets[i], e = q.offsets[i + 1];
        const int s = __popcll(__ballot(lane_id() < q.n && e <= t)), at = min(s, q.n - 1);
        begin = min(max(__builtin_amdgcn_readlane(b, at), 0), q.T);
        end = min(max(__builtin_amdgcn_readlane(e, at), 0), q.T);
        return s;
    }
    const int s = seq_of(q, t), at = min(s, q.n - 1);
    begin = seq_begin(q, at);
    end = seq_end(q, at);
    return s;
}

struct Out {
    int32_t *counts;
    float *prob, *coef, *loss;
};
// Workspace: 64 bytes of header (word 0: arrival counter), then for each of
// chunks + n partial sums its experts' probabilities and counts and its live
// tokens, then per sequence its live tokens and per 64-expert block a double.
struct Parts {
    int32_t *counter;
    double *dot;    // [n][EB]
    float *prob;    // [chunks + n][E]
    int32_t *cnt;   // [chunks + n][E]
    int32_t *live;  // [chunks + n]
    int32_t *nq;    // [n]
};
size_t parts_bytes(int chunks, int n, int E) {
    const size_t rows = (size_t)chunks + n, EB = (E + 63) / 64;
    return 64 + (size_t)n * EB * 8 + rows * E * 8 + rows * 4 + (size_t)n * 4;
}
Parts parts_of(void *ws, int chunks, int n, int E) {
    const size_t rows = (size_t)chunks + n, EB = (E + 63) / 64;
    Parts p;
    char *c = (char *)ws;
    p.counter = (int32_t *)c;
    c += 64;
    p.dot = (double *)c;
    c += (size_t)n * EB * 8;
    p.prob = (float *)c;
    c += rows * E * 4;
    p.cnt = (int32_t *)c;
    c += rows * E * 4;
    p.live = (int32_t *)c;
    c += rows * 4;
    p.nq = (int32_t *)c;
    return p;
}

// ---------------------------------------------------------------- loss
// A workgroup of W waves holds the probabilities of its W U tokens in
// registers (wave w those of tokens t0 + w, t0 + w + W, ...) and, each
// thread, NI of their choices; then it goes through the segments, the parts of
// sequences that lie among them.  A segment's sums: each wave adds its tokens
// that belong to it, the waves meet in LDS and are added in order.  Two LDS
// buffers in turn: one barrier per segment.
template <int W>
struct SegmentLds {
    float red[2][W][kMaxExperts];
    int32_t hist[2][kMaxExperts];
    int32_t live[2][W];
};
template <bool VEC, int W, int U>
struct Tokens {
    static constexpr int NI = (W * U * 8 + 64 * W - 1) / (64 * W);  // choices per thread (k <= 8)
    float p[U][kSlots];
    bool on[U];
    int e[NI], te[NI];  // choice, its token

    __device__ __forceinline__ void load(const Seqs &q, const float *__restrict__ logits,
                                         const int32_t *__restrict__ idx, int E, int k, int t0, int t1) {
        const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        float x[U][kSlots];
#pragma unroll
        for (int u = 0; u < U; ++u) on[u] = t0 + wave + u * W < t1;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            te[i] = t0 + (tid + 64 * W * i) / k;
            e[i] = -1;
        }
        if (t0 < t1) {  // there is a token: every load is of one, and all are in flight together
#pragma unroll
            for (int u = 0; u < U; ++u) load_row<VEC>(logits + (size_t)min(t0 + wave + u * W, t1 - 1) * E, E, x[u]);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                e[i] = idx[(size_t)t0 * k + min(tid + 64 * W * i, (t1 - t0) * k - 1)];
            if (q.mask) {
                uint8_t m[U], me[NI];
#pragma unroll
                for (int u = 0; u < U; ++u) m[u] = q.mask[min(t0 + wave + u * W, t1 - 1)];
#pragma unroll
                for (int i = 0; i < NI; ++i) me[i] = q.mask[min(te[i], t1 - 1)];
#pragma unroll
                for (int u = 0; u < U; ++u) on[u] = on[u] & (m[u] != 0);
#pragma unroll
                for (int i = 0; i < NI; ++i) e[i] = me[i] != 0 ? e[i] : -1;
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (te[i] >= t1 || (unsigned)e[i] >= (unsigned)E) e[i] = -1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t0 + wave + u * W >= t1) continue;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                p[u][i] = expert_of<VEC>(i) < E ? score(x[u][i]) : 0.0f;
                sum += p[u][i];
            }
            sum = route::wave_tree_sum(sum);
            const float inv = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
#pragma unroll
            for (int i = 0; i < kSlots; ++i) p[u][i] *= inv;
        }
    }
    // The sums over tokens [a, b): on return thread e < E has expert e's, and
    // every thread below 64 * 4 the number of live tokens.  `buf` alternates.
    __device__ __forceinline__ void segment(int t0, int a, int b, SegmentLds<W> &sh, int buf, float &prob, int &cnt,
                                            int &live) const {
        const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        float acc[kSlots] = {0.f, 0.f, 0.f, 0.f};
        int n = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + wave + u * W;
            if (t >= a && t < b && on[u]) {
                ++n;
#pragma unroll
                for (int i = 0; i < kSlots; ++i) acc[i] += p[u][i];
            }
        }
        if (VEC) {
            *(float4 *)&sh.red[buf][wave][4 * lane_id()] = float4{acc[0], acc[1], acc[2], acc[3]};
        } else {
#pragma unroll
            for (int i = 0; i < kSlots; ++i) sh.red[buf][wave][expert_of<VEC>(i)] = acc[i];
        }
        if (lane_id() == 0) sh.live[buf][wave] = n;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (e[i] >= 0 && te[i] >= a && te[i] < b) atomicAdd(&sh.hist[buf][e[i]], 1);
        __syncthreads();
        prob = 0.0f;
        cnt = 0;
        live = 0;
        if (tid < kMaxExperts) {
#pragma unroll
            for (int w = 0; w < W; ++w) live += sh.live[buf][w];
#pragma unroll
            for (int w = 0; w < W; ++w) prob += sh.red[buf][w][tid];
            cnt = sh.hist[buf][tid];
            sh.hist[buf][tid] = 0;  // for the segment after the next, past its barrier
        }
    }
};

// One workgroup per chunk of C = W U tokens; a chunk's segments go to partial
// sum c + s, which no other segment shares.
template <bool VEC, int W, int U>
__global__ __launch_bounds__(64 * W) void k_balance_part(Seqs q, const float *__restrict__ logits,
                                                         const int32_t *__restrict__ idx, int E, int k, Parts p) {
    __shared__ __attribute__((aligned(16))) SegmentLds<W> sh;
    const int t0 = blockIdx.x * (W * U), t1 = min(t0 + W * U, q.T);
    const int tid = threadIdx.x;
    if (tid < kMaxExperts) sh.hist[0][tid] = sh.hist[1][tid] = 0;
    Tokens<VEC, W, U> tok;
    tok.load(q, logits, idx, E, k, t0, t1);
    __syncthreads();
    int buf = 0;
    int begin, end;
    for (int s = seq_at(q, t0, begin, end); s < q.n && begin < t1;) {
        const int a = max(begin, t0), b = min(end, t1);
        if (a >= b) {  // empty, and any number after it: on to the one that holds token a
            const int to = seq_at(q, a, begin, end);
            if (to <= s) break;  // (bounds that decrease)
            s = to;
            continue;
        }
        float prob;
        int cnt, live;
        tok.segment(t0, a, b, sh, buf, prob, cnt, live);
        buf ^= 1;
        const size_t row = (size_t)blockIdx.x + s;
        if (tid < E) {
            p.prob[row * E + tid] = prob;
            p.cnt[row * E + tid] = cnt;
        }
        if (tid == 0) p.live[row] = live;
        if (b == t1 || ++s >= q.n) break;  // the chunk ends in this sequence
        begin = seq_begin(q, s);
        end = seq_end(q, s);
    }
}

// the sum of one double per thread of the workgroup, in a fixed order; the
// result is thread 0's
template <int NT>
__device__ __forceinline__ double block_sum(double v, double *sh) {
    sh[threadIdx.x] = v;
    __syncthreads();
#pragma unroll
    for (int d = NT / 2; d >= 1; d >>= 1) {
        if ((int)threadIdx.x < d) sh[threadIdx.x] += sh[threadIdx.x + d];
        __syncthreads();
    }
    const double r = sh[0];
    __syncthreads();
    return r;
}

__device__ __forceinline__ double coef_of(float alpha, int E, int k, int n, int some) {
    return n > 0 ? (double)alpha * E / ((double)k * n * n * some) : 0.0;
}

// Partial sums -> counts, prob_sums and each sequence's product, 64 experts
// of one sequence per workgroup: GR groups of 64 threads add every GR-th
// chunk, then the groups in order.  The last workgroup to arrive adds the
// sequences up.
template <int GR>
__global__ __launch_bounds__(64 * GR) void k_balance_reduce(Seqs q, int E, int k, int C, int EB, float alpha, Parts p,
                                                            Out o) {
    constexpr int NT = 64 * GR;
    __shared__ float sp[GR][64];
    __shared__ int32_t sc[GR][64];
    __shared__ int32_t sl[GR];
    __shared__ double sd[NT];
    __shared__ int last;
    const int s = blockIdx.x / EB, eb = blockIdx.x - s * EB;
    const int tid = threadIdx.x, ex = tid & 63, gr = tid >> 6, e = 64 * eb + ex;
    const int a = seq_begin(q, s), b = seq_end(q, s);
    float prob = 0.0f;
    int cnt = 0, live = 0;
    if (a < b) {
        const int c1 = (b - 1) / C;
        const int ec = min(e, E - 1);
#pragma unroll 8
        for (int c = a / C + gr; c <= c1; c += GR) {
            const size_t row = (size_t)c + s;
            prob += p.prob[row * E + ec];
            cnt += p.cnt[row * E + ec];
            live += p.live[row];
        }
    }
    sp[gr][ex] = prob;
    sc[gr][ex] = cnt;
    if (ex == 0) sl[gr] = live;
    __syncthreads();
    double dot = 0.0;
    if (tid < 64) {
        prob = 0.0f;
        cnt = 0;
        live = 0;
        for (int g = 0; g < GR; ++g) {
            prob += sp[g][ex];
            cnt += sc[g][ex];
            live += sl[g];
        }
        if (e < E) {
            o.counts[(size_t)s * E + e] = cnt;
            o.prob[(size_t)s * E + e] = prob;
            dot = (double)cnt * (double)prob;
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, kWave);
        if (tid == 0) {
            // The sums go to memory by atomic exchanges whose results are
            // waited for, then the arrival is counted: whoever sees the last
            // count and reads with atomic loads reads the sums, with no
            // write-back of the whole L2 (a releasing count took 3 us more).
            const double was = __hip_atomic_exchange(&p.dot[(size_t)s * EB + eb], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (eb == 0) {
                const int nwas = __hip_atomic_exchange(&p.nq[s], live, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                asm volatile("" ::"v"(nwas) : "memory");
            }
            asm volatile("" ::"v"(was) : "memory");
            last = __hip_atomic_fetch_add(p.counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                   (int)gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    if (tid == 0) __hip_atomic_store(p.counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    auto dot_of = [&](int i) {
        double d = 0.0;
        for (int j = 0; j < EB; ++j)
            d += __hip_atomic_load(&p.dot[(size_t)i * EB + j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return d;
    };
    auto nq_of = [&](int i) { return __hip_atomic_load(&p.nq[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    if (q.n <= kWave) {  // a lane per sequence
        if (tid >= kWave) return;
        const int n = tid < q.n ? nq_of(tid) : 0;
        const double c = coef_of(alpha, E, k, n, __popcll(__ballot(n > 0)));
        if (tid < q.n) o.coef[tid] = (float)c;
        double sum = c != 0.0 ? c * dot_of(tid) : 0.0;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, kWave);
        if (tid == 0) *o.loss = (float)sum;
        return;
    }
    int some = 0;
    for (int i = tid; i < q.n; i += NT) some += nq_of(i) > 0;
    const int total = (int)block_sum<NT>((double)some, sd);
    double sum = 0.0;
    for (int i = tid; i < q.n; i += NT) {
        const double c = coef_of(alpha, E, k, nq_of(i), total);
        o.coef[i] = (float)c;
        sum += c != 0.0 ? c * dot_of(i) : 0.0;
    }
    sum = block_sum<NT>(sum, sd);
    if (tid == 0) *o.loss = (float)sum;
}

// Few tokens and sequences: everything in one workgroup, in one launch.  The
// sequences' bounds are read once; a thread adds its expert's products over
// the sequences, divided by n_q^2, and one reduction at the end gives the loss.
template <bool VEC, int U>
__global__ __launch_bounds__(1024) void k_balance_one(Seqs q, const float *__restrict__ logits,
                                                      const int32_t *__restrict__ idx, int E, int k, float alpha,
                                                      Out o) {
    constexpr int W = 16;
    __shared__ __attribute__((aligned(16))) SegmentLds<W> sh;
    __shared__ double sdot[4];
    __shared__ int snq[kOneSeqs], sbegin[kOneSeqs], send[kOneSeqs];
    const int tid = threadIdx.x;
    if (tid < kMaxExperts) sh.hist[0][tid] = sh.hist[1][tid] = 0;
    if (tid < q.n) {
        sbegin[tid] = seq_begin(q, tid);
        send[tid] = seq_end(q, tid);
    }
    Tokens<VEC, W, U> tok;
    tok.load(q, logits, idx, E, k, 0, q.T);
    __syncthreads();
    double dot = 0.0;
    for (int s = 0; s < q.n; ++s) {
        float prob;
        int cnt, live;
        tok.segment(0, sbegin[s], send[s], sh, s & 1, prob, cnt, live);
        if (tid < E) {
            o.counts[(size_t)s * E + tid] = cnt;
            o.prob[(size_t)s * E + tid] = prob;
            if (live) dot += (double)cnt * (double)prob / ((double)live * live);
        }
        if (tid == 0) snq[s] = live;
    }
    if (tid < kMaxExperts) {
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, kWave);
        if (lane_id() == 0) sdot[tid >> 6] = dot;
    }
    __syncthreads();
    if (tid < kWave) {
        const int n = tid < q.n ? snq[tid] : 0;
        const int some = __popcll(__ballot(n > 0));
        if (tid < q.n) o.coef[tid] = (float)coef_of(alpha, E, k, n, some);
        const double c = coef_of(alpha, E, k, 1, some), sum = ((sdot[0] + sdot[1]) + sdot[2]) + sdot[3];
        if (tid == 0) *o.loss = some && c != 0.0 ? (float)(c * sum) : 0.0f;
    }
}

// ---------------------------------------------------------------- gradient
// v of the lane whose number differs in the bits of X, within each aligned
// group of eight lanes.
template <int X>
__device__ __forceinline__ float lane_xor(float v) {
    if constexpr (X >= 4) {  // row_half_mirror is X = 7
        return lane_xor<7 - X>(__uint_as_float(route::dpp32<0x141>(__float_as_uint(v))));
    } else if constexpr (X > 0) {  // quad_perm 0^X, 1^X, 2^X, 3^X
        return __uint_as_float(route::dpp32<(0 ^ X) | (1 ^ X) << 2 | (2 ^ X) << 4 | (3 ^ X) << 6>(__float_as_uint(v)));
    }
    return v;
}
// The routing-weight term of a token's gradient, whose choices (score s, its
// slope, gradient g of the weight) sit in eight lanes:
// (g_j - sum_l g_l s_l / S) / S slope_j, written
// (sum_l s_l (g_j - g_l) / S) (slope_j / S) so that nothing cancels (one choice
// gives 0) and nothing overflows where every score is tiny (slope <= s <= S).
__device__ __forceinline__ float weight_term(float s, float slope, float g) {
    float S = s, d = 0.0f;
#define MOE_PAIR(X)                                \
    {                                                             \
        const float so = lane_xor<X>(s), go = lane_xor<X>(g);     \
        S += so;                                                  \
        d = so != 0.0f ? __builtin_fmaf(so, g - go, d) : d;       \
    }
    MOE_PAIR(1) MOE_PAIR(2) MOE_PAIR(3) MOE_PAIR(4) MOE_PAIR(5) MOE_PAIR(6) MOE_PAIR(7)
#undef MOE_PAIR
    const float r = S == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(S);
    return (d * r) * (r * slope);
}

// A wave takes TW consecutive tokens, U of them at a time (1, or 8: the
// requests of eight rows in flight).  The routing-weight term first, of all U
// tokens at once: lane 8 u + j has token u's j-th choice, its score comes from
// its logit by itself, the two sums over a token's choices are sums over
// eight lanes, and the terms go to the lanes that hold those experts through
// a row of zeros in LDS per token.  Then per token the scores of all experts,
// their sum and the sum of c s (two wave reductions), and the balance term.
template <bool VEC, int U>
__global__ __launch_bounds__(256) void k_route_backward(Seqs q, const float *__restrict__ logits,
                                                        const int32_t *__restrict__ idx,
                                                        const int32_t *__restrict__ counts,
                                                        const float *__restrict__ coef,
                                                        const float *__restrict__ d_loss,
                                                        const float *__restrict__ d_w, int E, int k, float scale,
                                                        int TW, float *__restrict__ d_logits) {
    __shared__ __attribute__((aligned(16))) float sterm[4][U][kMaxExperts];
    const int l = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t0 = (blockIdx.x * 4 + wave) * TW, t1 = min(t0 + TW, q.T);
    if (t0 >= t1) return;
    float(&term)[U][kMaxExperts] = sterm[wave];
    const int lu = l >> 3, lj = l & 7;  // the lane's token and choice
    float c[kSlots] = {0.f, 0.f, 0.f, 0.f};
    int s = -1, begin = 0, end = 0;
    float dl = 0.0f;
    // The sequence s: its bounds and c of the lane's experts, less their
    // average: c[e] - sum_j c[j] p[j] is the same for c less any constant, and
    // with nearly even counts little is left to cancel.
    auto enter = [&]() {
        if (s >= q.n) begin = end = q.T;
        if (!d_loss || s >= q.n) return;
        float n[kSlots], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int e = expert_of<VEC>(i);
            n[i] = e < E ? (float)counts[(size_t)s * E + e] : 0.0f;
            sum += n[i];
        }
        const float f = dl * coef[s], even = __builtin_rintf(route::wave_tree_sum(sum) / (float)E);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) c[i] = expert_of<VEC>(i) < E ? f * (n[i] - even) : 0.0f;
    };
    if (d_w) {
#pragma unroll
        for (int u = 0; u < U; ++u) *(float4 *)&term[u][4 * l] = float4{0.f, 0.f, 0.f, 0.f};
    }
    for (int tb = t0; tb < t1; tb += U) {
        float x[U][kSlots];
        bool on[U];
        int ek = -1;
        float dw = 0.0f, xk = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            on[u] = true;
            load_row<VEC>(logits + (size_t)min(tb + u, t1 - 1) * E, E, x[u]);
        }
        if (d_w && lu < U && lj < k && tb + lu < t1) {
            ek = idx[(size_t)(tb + lu) * k + lj];
            dw = d_w[(size_t)(tb + lu) * k + lj];
        }
        if (q.mask) {
#pragma unroll
            for (int u = 0; u < U; ++u) on[u] = q.mask[min(tb + u, t1 - 1)] != 0;
        }
        if (s < 0) {
            dl = d_loss ? *d_loss : 0.0f;
            s = seq_at(q, t0, begin, end);
            enter();
        }
        if ((unsigned)ek >= (unsigned)E) ek = -1;
        if (d_w) {
            if (ek >= 0) xk = logits[(size_t)(tb + lu) * E + ek];
            float slope_k;
            const float sk = score(xk, slope_k);
            const float term_k = weight_term(ek >= 0 ? sk : 0.0f, slope_k, dw);
            // (the same index twice in a row: its terms add)
            if (ek >= 0) atomicAdd(&term[lu < U ? lu : 0][ek], scale * term_k);
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = tb + u;
            if (t >= t1) break;
            if (s < q.n && t >= end) {  // the sequence that holds t, past any number of empty ones
                s = seq_at(q, t, begin, end);
                enter();
            }
            const bool live = on[u] && s < q.n && t >= begin;
            float slope[kSlots], sum = 0.0f, cs = 0.0f, ds[kSlots] = {0.f, 0.f, 0.f, 0.f};
            if (d_w) {
                if (VEC) {
                    const float4 v = *(const float4 *)&term[u][4 * l];
                    ds[0] = v.x;
                    ds[1] = v.y;
                    ds[2] = v.z;
                    ds[3] = v.w;
                } else {
#pragma unroll
                    for (int i = 0; i < kSlots; ++i) ds[i] = term[u][expert_of<VEC>(i)];
                }
            }
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                float sc = score(x[u][i], slope[i]);
                if (expert_of<VEC>(i) >= E) sc = 0.0f;
                sum += sc;
                cs = __builtin_fmaf(c[i], sc, cs);
            }
            if (d_loss) {
                sum = route::wave_tree_sum(sum);
                cs = route::wave_tree_sum(cs);
                const float inv = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
                const float mean = cs * inv;
#pragma unroll
                for (int i = 0; i < kSlots; ++i) ds[i] = __builtin_fmaf(c[i] - mean, slope[i] * inv, ds[i]);
            }
            float *row = d_logits + (size_t)t * E;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) ds[i] = live ? ds[i] : 0.0f;
            if (VEC) {
                if (4 * l < E) *(float4 *)(row + 4 * l) = float4{ds[0], ds[1], ds[2], ds[3]};
            } else {
#pragma unroll
                for (int i = 0; i < kSlots; ++i)
                    if (expert_of<VEC>(i) < E) row[expert_of<VEC>(i)] = ds[i];
            }
        }
        if (d_w) {  // the rows are zeros again before the next tokens' terms
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            if (ek >= 0) term[lu < U ? lu : 0][ek] = 0.0f;
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
    }
}

moe_status check_seqs(int32_t T, int32_t n_seq, const int32_t *seq_offsets) {
    MOE_TRY(check_tokens(T));
    if (n_seq < 1 || n_seq > MOE_MAX_TOKENS) return MOE_ERR_SHAPE;
    if (!seq_offsets && n_seq != 1) return MOE_ERR_NULL;
    if (!aligned(seq_offsets, 4)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_balance_workspace_bytes(const moe_layer_desc *desc, int32_t T, int32_t n_seq) {
    if (check_desc(desc) != MOE_OK || check_tokens(T) != MOE_OK || n_seq < 1 || n_seq > MOE_MAX_TOKENS) return 0;
    return (parts_bytes(most_chunks(T), n_seq, desc->n_routed) + 255) / 256 * 256;
}

extern "C" moe_status moe_balance_loss(const moe_layer_desc *desc, int32_t T, int32_t n_seq,
                                       const int32_t *seq_offsets, const uint8_t *token_mask, const float *logits,
                                       const int32_t *topk_idx, float alpha, int32_t *counts, float *prob_sums,
                                       float *seq_coef, float *loss, void *ws, size_t ws_bytes, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_seqs(T, n_seq, seq_offsets));
    if (!(alpha - alpha == 0.0f)) return MOE_ERR_SHAPE;
    if (!counts || !prob_sums || !seq_coef || !loss || !ws || (T > 0 && (!logits || !topk_idx))) return MOE_ERR_NULL;
    if (!aligned(ws, 16) || !aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(counts, 4) ||
        !aligned(prob_sums, 4) || !aligned(seq_coef, 4) || !aligned(loss, 4))
        return MOE_ERR_ALIGN;
    const int E = desc->n_routed, k = desc->top_k;
    if (ws_bytes < parts_bytes(chunk_count(T), n_seq, E)) return MOE_ERR_WORKSPACE;  // what this call uses
    hipStream_t st = (hipStream_t)stream;
    const Seqs q{seq_offsets, token_mask, n_seq, T};
    const Out o{counts, prob_sums, seq_coef, loss};
    const bool vec = E % 4 == 0 && aligned(logits, 16);
    if (T <= kOneTokens && n_seq <= kOneSeqs) {
        const auto one = vec ? (T <= 32 ? k_balance_one<true, 2> : k_balance_one<true, 8>)
                             : (T <= 32 ? k_balance_one<false, 2> : k_balance_one<false, 8>);
        hipLaunchKernelGGL(one, dim3(1), dim3(1024), 0, st, q, logits, topk_idx, E, k, alpha, o);
        return launch_status();
    }
    const int C = chunk_tokens(T), chunks = chunk_count(T), EB = (E + 63) / 64;
    const Parts p = parts_of(ws, chunks, n_seq, E);
    if (chunks > 0) {
        void (*part)(Seqs, const float *, const int32_t *, int, int, Parts) = nullptr;
        switch (C) {
            case 8: part = vec ? k_balance_part<true, 8, 1> : k_balance_part<false, 8, 1>; break;
            case 16: part = vec ? k_balance_part<true, 16, 1> : k_balance_part<false, 16, 1>; break;
            case 32: part = vec ? k_balance_part<true, 16, 2> : k_balance_part<false, 16, 2>; break;
            case 64: part = vec ? k_balance_part<true, 16, 4> : k_balance_part<false, 16, 4>; break;
            default: part = vec ? k_balance_part<true, 16, 8> : k_balance_part<false, 16, 8>; break;
        }
        hipLaunchKernelGGL(part, dim3(chunks), dim3(C == 8 ? 512 : 1024), 0, st, q, logits, topk_idx, E, k, p);
        MOE_TRY(launch_status());
    }
    // 16 groups of threads where a sequence spans many chunks, else 4
    if (chunks > 8 * (int64_t)n_seq)
        hipLaunchKernelGGL(k_balance_reduce<16>, dim3(n_seq * EB), dim3(1024), 0, st, q, E, k, C, EB, alpha, p, o);
    else
        hipLaunchKernelGGL(k_balance_reduce<4>, dim3(n_seq * EB), dim3(256), 0, st, q, E, k, C, EB, alpha, p, o);
    return launch_status();
}

extern "C" moe_status moe_route_backward(const moe_layer_desc *desc, int32_t T, int32_t n_seq,
                                         const int32_t *seq_offsets, const uint8_t *token_mask, const float *logits,
                                         const int32_t *topk_idx, const int32_t *counts, const float *seq_coef,
                                         const float *d_loss, const float *d_topk_w, float *d_logits, void *stream) {
    MOE_TRY(check_desc(desc));
    MOE_TRY(check_seqs(T, n_seq, seq_offsets));
    if (T == 0) return MOE_OK;
    if (!logits || !topk_idx || !d_logits || (d_loss && (!counts || !seq_coef))) return MOE_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(counts, 4) || !aligned(seq_coef, 4) ||
        !aligned(d_loss, 4) || !aligned(d_topk_w, 4) || !aligned(d_logits, 4))
        return MOE_ERR_ALIGN;
    const int E = desc->n_routed, k = desc->top_k;
    const Seqs q{seq_offsets, token_mask, n_seq, T};
    const bool vec = E % 4 == 0 && aligned(logits, 16) && aligned(d_logits, 16);
    // a token per wave while that takes at most eight waves per SIMD, else
    // eight at a time (256 experts, 8192 tokens: 7.5 us either way and 3.4
    // against 6.0 at 128; 16384: 13.2 against 11.8; 65536: 47 against 33)
    const int TW = T <= 8192 ? 1 : T <= 32768 ? 8 : 16;
    const dim3 grid((unsigned)((T + 4 * TW - 1) / (4 * TW)));
    hipStream_t st = (hipStream_t)stream;
    const auto back = vec ? (TW == 1 ? k_route_backward<true, 1> : k_route_backward<true, 8>)
                          : (TW == 1 ? k_route_backward<false, 1> : k_route_backward<false, 8>);
    hipLaunchKernelGGL(back, grid, dim3(256), 0, st, q, logits, topk_idx, counts, seq_coef, d_loss, d_topk_w, E, k,
                       desc->routed_scale, TW, d_logits);
    return launch_status();
}
