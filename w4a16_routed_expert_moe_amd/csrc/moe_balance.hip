// moe_balance.hip -- the router's balance: tokens per expert, the balance
// loss of packed sequences, and the gradient of the router's logits.
//
//   s[t][e] = sigmoid(logits[t][e]),  p[t][e] = s[t][e] / sum_j s[t][j]
//   counts[q][e], prob_sums[q][e]: per sequence q, over its live tokens
//   loss = sum_q coef[q] sum_e counts[q][e] prob_sums[q][e],
//   coef[q] = alpha E / (k n_q^2 Q')
//
// The loss reads every logit once and the gradient reads and writes every
// one once: both are bound by HBM (at 65536 x 256: 67 MB and 134 MB).  A wave
// takes a token; a lane holds four experts, so the sum over a token's experts
// is one wave reduction and the sums over tokens stay in registers.
#include "moe_route_common.h"

namespace moe {
namespace {

constexpr int kSlots = 4;          // experts per lane: E <= 256
constexpr int kMaxExperts = kSlots * kWave;
constexpr int kOneTokens = 128;    // up to here the loss is one workgroup's work, one launch
constexpr int kOneSeqs = 64;
constexpr int kMaxChunks = 512;    // token chunks of the partial sums

// the tokens of one chunk: at most kMaxChunks of them (two per CU), 32 tokens at least
int chunk_tokens(int T) { return T <= 32 * kMaxChunks ? 32 : (T + kMaxChunks - 1) / kMaxChunks; }
int chunk_count(int T) { return (T + chunk_tokens(T) - 1) / chunk_tokens(T); }

// Sigmoid s and its slope s (1 - s) from e = exp(-|x|), which neither
// overflows nor cancels: s = 1 / (1 + e) or e / (1 + e), slope = e / (1 + e)^2.
// The hardware exponential and reciprocal are good to an ulp or two, and
// nothing is selected by these scores.  Scores below 2^-126 become 0.
__device__ __forceinline__ float score(float x, float &slope) {
    const float e = __expf(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e);
    slope = e * r * r;
    return x < 0.0f ? e * r : r;
}
__device__ __forceinline__ float score(float x) {
    float slope;
    return score(x, slope);
}

// the expert of slot i of a lane: VEC four consecutive ones (16-byte loads),
// else one in each block of 64 (any E, any alignment)
template <bool VEC>
__device__ __forceinline__ int expert_of(int i) {
    return VEC ? 4 * lane_id() + i : lane_id() + kWave * i;
}
template <bool VEC>
__device__ __forceinline__ void load_row(const float *__restrict__ row, int E, float (&x)[kSlots]) {
    if (VEC) {
        const float4 v = 4 * lane_id() < E ? *(const float4 *)(row + 4 * lane_id()) : float4{0.f, 0.f, 0.f, 0.f};
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) x[i] = expert_of<VEC>(i) < E ? row[expert_of<VEC>(i)] : 0.0f;
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
__device__ __forceinline__ bool token_live(const Seqs &q, int t) { return !q.mask || q.mask[t] != 0; }

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
// Tokens [a, b) of one sequence: the workgroup's sums over its live tokens.
// On return thread e < E has the expert's probability sum and count, every
// thread the number of live tokens.  Fixed order: wave w adds tokens a + w,
// a + w + W, ..., then the waves are added in order.
template <bool VEC, int W>
struct SegmentLds {
    float red[W][kMaxExperts];
    int32_t hist[kMaxExperts];
    int32_t live[W];
};
template <bool VEC, int W>
__device__ __forceinline__ void segment_sums(const Seqs &q, const float *__restrict__ logits,
                                             const int32_t *__restrict__ idx, int E, int k, int a, int b,
                                             SegmentLds<VEC, W> &sh, float &prob, int &cnt, int &live) {
    constexpr int U = 4;  // tokens in flight per wave
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int e = tid; e < kMaxExperts; e += 64 * W) sh.hist[e] = 0;
    __syncthreads();
    float acc[kSlots] = {0.f, 0.f, 0.f, 0.f};
    int n = 0;
    for (int t0 = a + wave; t0 < b; t0 += U * W) {
        float x[U][kSlots];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * W;
            on[u] = t < b && token_live(q, t);
            load_row<VEC>(logits + (size_t)min(t, b - 1) * E, E, x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s[kSlots], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                s[i] = expert_of<VEC>(i) < E ? score(x[u][i]) : 0.0f;
                sum += s[i];
            }
            sum = route::wave_tree_sum(sum);
            const float inv = sum > 0.0f ? __builtin_amdgcn_rcpf(sum) : sum == 0.0f ? 0.0f : sum;  // NaN stays
            if (on[u]) {
                ++n;
#pragma unroll
                for (int i = 0; i < kSlots; ++i) acc[i] += s[i] * inv;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) sh.red[wave][expert_of<VEC>(i)] = acc[i];
    if (lane_id() == 0) sh.live[wave] = n;
    for (int i = tid; i < (b - a) * k; i += 64 * W) {
        const int t = a + i / k;
        const int e = idx[(size_t)a * k + i];
        if ((unsigned)e < (unsigned)E && token_live(q, t)) atomicAdd(&sh.hist[e], 1);
    }
    __syncthreads();
    prob = 0.0f;
    cnt = 0;
    live = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) live += sh.live[w];
    if (tid < kMaxExperts) {
#pragma unroll
        for (int w = 0; w < W; ++w) prob += sh.red[w][tid];
        cnt = sh.hist[tid];
    }
    __syncthreads();  // the next segment writes the arrays again
}

// One workgroup per chunk of C tokens; a chunk's segments (one per sequence
// that it meets) go to partial sum c + s, which no other segment shares.
template <bool VEC>
__global__ __launch_bounds__(256) void k_balance_part(Seqs q, const float *__restrict__ logits,
                                                      const int32_t *__restrict__ idx, int E, int k, int C, Parts p) {
    __shared__ SegmentLds<VEC, 4> sh;
    const int t0 = blockIdx.x * C, t1 = min(t0 + C, q.T);
    for (int s = seq_of(q, t0); s < q.n; ++s) {
        const int a = max(seq_begin(q, s), t0), b = min(seq_end(q, s), t1);
        if (seq_begin(q, s) >= t1) break;
        if (a >= b) continue;
        float prob;
        int cnt, live;
        segment_sums<VEC, 4>(q, logits, idx, E, k, a, b, sh, prob, cnt, live);
        const size_t row = (size_t)blockIdx.x + s;
        if ((int)threadIdx.x < E) {
            p.prob[row * E + threadIdx.x] = prob;
            p.cnt[row * E + threadIdx.x] = cnt;
        }
        if (threadIdx.x == 0) p.live[row] = live;
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
            __hip_atomic_store(&p.dot[(size_t)s * EB + eb], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (eb == 0) __hip_atomic_store(&p.nq[s], live, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(p.counter, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                   (int)gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    auto nq_of = [&](int i) { return __hip_atomic_load(&p.nq[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    int some = 0;
    for (int i = tid; i < q.n; i += NT) some += nq_of(i) > 0;
    const int total = (int)block_sum<NT>((double)some, sd);
    double sum = 0.0;
    for (int i = tid; i < q.n; i += NT) {
        const double c = coef_of(alpha, E, k, nq_of(i), total);
        double d = 0.0;
        for (int j = 0; j < EB; ++j)
            d += __hip_atomic_load(&p.dot[(size_t)i * EB + j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        o.coef[i] = (float)c;
        sum += c != 0.0 ? c * d : 0.0;
    }
    sum = block_sum<NT>(sum, sd);
    if (tid == 0) {
        *o.loss = (float)sum;
        __hip_atomic_store(p.counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// Few tokens and sequences: everything in one workgroup.
template <bool VEC>
__global__ __launch_bounds__(512) void k_balance_one(Seqs q, const float *__restrict__ logits,
                                                     const int32_t *__restrict__ idx, int E, int k, float alpha, Out o) {
    __shared__ SegmentLds<VEC, 8> sh;
    __shared__ double sdot[kOneSeqs], sd[8];
    __shared__ int snq[kOneSeqs];
    const int tid = threadIdx.x;
    for (int s = 0; s < q.n; ++s) {
        const int a = seq_begin(q, s), b = seq_end(q, s);
        float prob = 0.0f;
        int cnt = 0, live = 0;
        if (a < b) segment_sums<VEC, 8>(q, logits, idx, E, k, a, b, sh, prob, cnt, live);
        double dot = 0.0;
        if (tid < E) {
            o.counts[(size_t)s * E + tid] = cnt;
            o.prob[(size_t)s * E + tid] = prob;
            dot = (double)cnt * (double)prob;
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, kWave);
        if (lane_id() == 0) sd[tid >> 6] = dot;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < 8; ++w) dot += sd[w];
            sdot[s] = dot;
            snq[s] = live;
        }
        __syncthreads();
    }
    if (tid < kWave) {
        const int n = tid < q.n ? snq[tid] : 0;
        const int some = __popcll(__ballot(n > 0));
        const double c = coef_of(alpha, E, k, n, some);
        if (tid < q.n) o.coef[tid] = (float)c;
        double sum = n > 0 && c != 0.0 ? c * sdot[tid] : 0.0;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, kWave);
        if (tid == 0) *o.loss = (float)sum;
    }
}

// ---------------------------------------------------------------- gradient
// A wave takes TW consecutive tokens, four in flight.  Per token: the scores
// of its experts, their sum S and the sum of c s (two wave reductions), the
// balance term, and the k chosen experts' weight terms, computed by lanes
// j < k from the chosen logits and handed to the lanes that hold them.
template <bool VEC>
__global__ __launch_bounds__(256) void k_route_backward(Seqs q, const float *__restrict__ logits,
                                                        const int32_t *__restrict__ idx,
                                                        const int32_t *__restrict__ counts,
                                                        const float *__restrict__ coef,
                                                        const float *__restrict__ d_loss,
                                                        const float *__restrict__ d_w, int E, int k, float scale,
                                                        int TW, float *__restrict__ d_logits) {
    constexpr int U = 4;
    const int l = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t0 = (blockIdx.x * 4 + wave) * TW, t1 = min(t0 + TW, q.T);
    if (t0 >= t1) return;
    const float dl = d_loss ? *d_loss : 0.0f;
    int s = seq_of(q, t0), begin = 0, end = 0;
    float c[kSlots] = {0.f, 0.f, 0.f, 0.f};
    auto enter = [&]() {  // the sequence s: its bounds and c of the lane's experts
        begin = s < q.n ? seq_begin(q, s) : q.T;
        end = s < q.n ? seq_end(q, s) : q.T;
        const float f = d_loss && s < q.n ? dl * coef[s] : 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int e = expert_of<VEC>(i);
            c[i] = d_loss && s < q.n && e < E ? f * (float)counts[(size_t)s * E + e] : 0.0f;
        }
    };
    enter();
    for (int tb = t0; tb < t1; tb += U) {
        float x[U][kSlots], xk[U], dw[U];
        int ek[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = min(tb + u, t1 - 1);
            on[u] = token_live(q, t);
            load_row<VEC>(logits + (size_t)t * E, E, x[u]);
            ek[u] = -1;
            dw[u] = 0.0f;
            if (d_w && l < k) {
                ek[u] = idx[(size_t)t * k + l];
                dw[u] = d_w[(size_t)t * k + l];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = min(tb + u, t1 - 1);
            if ((unsigned)ek[u] >= (unsigned)E) ek[u] = -1;
            xk[u] = ek[u] >= 0 ? logits[(size_t)t * E + ek[u]] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = tb + u;
            if (t >= t1) break;
            while (s < q.n && t >= end) {
                ++s;
                enter();
            }
            const bool live = on[u] && s < q.n && t >= begin;
            float slope[kSlots], sum = 0.0f, cs = 0.0f;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                float sc = score(x[u][i], slope[i]);
                if (expert_of<VEC>(i) >= E) sc = 0.0f;
                sum += sc;
                cs = __builtin_fmaf(c[i], sc, cs);
            }
            sum = route::wave_tree_sum(sum);
            cs = route::wave_tree_sum(cs);
            const float inv = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
            const float mean = cs * inv;
            float ds[kSlots];
#pragma unroll
            for (int i = 0; i < kSlots; ++i) ds[i] = d_loss ? (c[i] - mean) * inv : 0.0f;
            if (d_w) {
                const float sk = ek[u] >= 0 ? score(xk[u]) : 0.0f;
                const float S = route::wave_tree_sum(sk), A = route::wave_tree_sum(dw[u] * sk);
                const float ik = S == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(S);
                const float g = scale * ik * (dw[u] - A * ik);
                for (int j = 0; j < k; ++j) {
                    const int e = __builtin_amdgcn_readlane(ek[u], j);
                    const float gj = route::readlane_f32(g, j);
#pragma unroll
                    for (int i = 0; i < kSlots; ++i)
                        if (expert_of<VEC>(i) == e) ds[i] += gj;
                }
            }
            float *row = d_logits + (size_t)t * E;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) ds[i] = live ? ds[i] * slope[i] : 0.0f;
            if (VEC) {
                if (4 * l < E) *(float4 *)(row + 4 * l) = float4{ds[0], ds[1], ds[2], ds[3]};
            } else {
#pragma unroll
                for (int i = 0; i < kSlots; ++i)
                    if (expert_of<VEC>(i) < E) row[expert_of<VEC>(i)] = ds[i];
            }
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
    return (parts_bytes(chunk_count(T), n_seq, desc->n_routed) + 255) / 256 * 256;
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
    if (ws_bytes < moe_balance_workspace_bytes(desc, T, n_seq)) return MOE_ERR_WORKSPACE;
    const int E = desc->n_routed, k = desc->top_k;
    hipStream_t st = (hipStream_t)stream;
    const Seqs q{seq_offsets, token_mask, n_seq, T};
    const Out o{counts, prob_sums, seq_coef, loss};
    const bool vec = E % 4 == 0 && aligned(logits, 16);
    if (T <= kOneTokens && n_seq <= kOneSeqs) {
        if (vec)
            hipLaunchKernelGGL(k_balance_one<true>, dim3(1), dim3(512), 0, st, q, logits, topk_idx, E, k, alpha, o);
        else
            hipLaunchKernelGGL(k_balance_one<false>, dim3(1), dim3(512), 0, st, q, logits, topk_idx, E, k, alpha, o);
        return launch_status();
    }
    const int C = chunk_tokens(T), chunks = chunk_count(T), EB = (E + 63) / 64;
    const Parts p = parts_of(ws, chunks, n_seq, E);
    if (chunks > 0) {
        if (vec)
            hipLaunchKernelGGL(k_balance_part<true>, dim3(chunks), dim3(256), 0, st, q, logits, topk_idx, E, k, C, p);
        else
            hipLaunchKernelGGL(k_balance_part<false>, dim3(chunks), dim3(256), 0, st, q, logits, topk_idx, E, k, C, p);
        MOE_TRY(launch_status());
    }
    // 16 groups of threads where a sequence spans many chunks, else 4
    if (chunks > 16 * (int64_t)n_seq)
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
    // four tokens per wave while that does not fill the card, else 16
    const int TW = T <= 32768 ? 4 : 16;
    const dim3 grid((unsigned)((T + 4 * TW - 1) / (4 * TW)));
    hipStream_t st = (hipStream_t)stream;
    if (vec)
        hipLaunchKernelGGL(k_route_backward<true>, grid, dim3(256), 0, st, q, logits, topk_idx, counts, seq_coef, d_loss,
                           d_topk_w, E, k, desc->routed_scale, TW, d_logits);
    else
        hipLaunchKernelGGL(k_route_backward<false>, grid, dim3(256), 0, st, q, logits, topk_idx, counts, seq_coef,
                           d_loss, d_topk_w, E, k, desc->routed_scale, TW, d_logits);
    return launch_status();
}
