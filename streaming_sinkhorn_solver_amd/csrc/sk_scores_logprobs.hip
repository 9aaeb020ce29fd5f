// sk_scores_logprobs.hip -- log-probabilities of given columns of a score
// matrix, entropy and the largest alternatives (sk_scores_logprobs), and their
// gradient (sk_scores_logprobs_grad).
//
// With z = s / eps and M = max_j s_j, S = sum_j exp((s_j - M)/eps) of a row,
//     lse = M/eps + log S,   log p_j = (s_j - M)/eps - log S,
//     H = -sum_j p_j log p_j = log S - (sum_j e_j d_j) / S,  d = (s - M)/eps, e = exp(d).
// The scores are read once.  A workgroup holds a chunk of a row in registers
// (16-byte loads), so the maximum is known before the sum and nothing is
// rescaled; longer rows are cut into chunks whose (M, S, sum e d) and sorted
// candidate lists a second kernel joins.
//
// The largest entries of a chunk: the maximum of every lane number over the
// workgroup's waves gives 64 disjoint classes; the k-th largest of their
// maxima is at most the k-th largest score, so only entries above it (about
// k + k^2 / 100 of them) and the first ones equal to it are candidates, whose ranks are
// counted in LDS.  Ties go to the lowest index.
#include "sk_scores.hpp"

#include <algorithm>

namespace sk {
namespace {

constexpr int kMaxTop = 64;
constexpr int64_t kTopMaxCols = (int64_t)1 << 20;  // columns, where alternatives are asked for
constexpr int64_t kLpGrid = 1 << 20;               // workgroups of one launch (each may serve several chunks)

struct LpArgs {
    const void* s;
    int64_t ld, n;
    int m;
    float eps, c;  // c = log2e / eps
    const int64_t* targets;
    int top;
    float *logp, *lse, *entropy, *top_logp, *stats;
    int32_t* top_idx;
    int splits;
    // partial results of the chunks, [n * splits] each, lists [n * splits][top]
    float *pm, *ps, *px;
    uint64_t* plist;
};

// A candidate: larger score first, then lower column.
__device__ __forceinline__ uint64_t cand(float v, uint32_t j) { return (uint64_t)ordered(v) << 32 | (uint32_t)~j; }
__device__ __forceinline__ uint32_t cand_col(uint64_t k) { return ~(uint32_t)k; }

// The row's outputs from its maximum and sums.  Called by one lane.
template <class T>
__device__ void finish_row(const LpArgs& A, int64_t i, float M, float S, float X) {
    const bool empty = S == 0.0f;
    const float top = empty ? -INFINITY : M;
    const float log_s = empty ? 0.0f : logf(S);
    A.lse[i] = top / A.eps + log_s;
    A.stats[2 * i] = top;
    A.stats[2 * i + 1] = log_s;
    if (A.entropy) {
        const float h = log_s - X / S * kLn2;
        A.entropy[i] = empty || h < 0.0f ? 0.0f : h;
    }
    if (A.targets) {
        const int64_t t = A.targets[i];
        float lp = 0.0f;  // no token given
        if (t >= A.m)
            lp = NAN;
        else if (t >= 0)
            lp = empty ? -INFINITY : (T::to(static_cast<const typename T::type*>(A.s)[i * A.ld + t]) - M) / A.eps - log_s;
        A.logp[i] = lp;
    }
}

template <class T>
__device__ __forceinline__ void finish_top(const LpArgs& A, int64_t i, int r, uint64_t key, float M, float S) {
    const uint32_t j = cand_col(key);
    const float s = T::to(static_cast<const typename T::type*>(A.s)[i * A.ld + j]);
    A.top_idx[i * A.top + r] = (int32_t)j;
    A.top_logp[i * A.top + r] = S == 0.0f ? -INFINITY : (s - M) / A.eps - logf(S);
}

template <class T>
struct Vec {
    static constexpr int n = 16 / sizeof(typename T::type);
    uint4 raw;
    __device__ float at(int i) const {
        if constexpr (n == 4) {
            const uint32_t w = i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w;
            return __builtin_bit_cast(float, w);
        } else {
            const uint32_t w = i / 2 == 0 ? raw.x : i / 2 == 1 ? raw.y : i / 2 == 2 ? raw.z : raw.w;
            return T::to((uint16_t)(i % 2 ? w >> 16 : w & 0xffffu));
        }
    }
};

// One chunk of a row per workgroup of W waves: NV 16-byte vectors per thread.
// The first chunk also takes the row's few entries before the first and after
// the last aligned 16 bytes, one per thread.
template <class T, int W, int NV>
__global__ __launch_bounds__(W * 64) void k_logprobs(LpArgs A) {
    constexpr int kThreads = W * 64, VE = Vec<T>::n;
    constexpr int kCap = W == 1 ? 256 : 1024;  // candidates above the threshold
    __shared__ uint64_t list[kCap + W * kMaxTop];
    __shared__ float red[W][3];
    __shared__ uint32_t lane_max[W][64];
    __shared__ uint32_t shared_t;
    __shared__ int count;
    using E = typename T::type;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    for (int64_t item = blockIdx.x; item < A.n * A.splits; item += gridDim.x) {
        const int64_t i = item / A.splits;
        const int split = (int)(item % A.splits);
        const E* row = static_cast<const E*>(A.s) + i * A.ld;
        const int mis = (int)(reinterpret_cast<uintptr_t>(row) / sizeof(E) % VE);
        const int head = min(A.m, (VE - mis) % VE);
        const int vecs = (A.m - head) / VE, tail = A.m - head - vecs * VE;
        const int v0 = split * (kThreads * NV);
        const E* body = row + head;
        Vec<T> v[NV];
        float x = -INFINITY;
        int xj = -1;  // column of the single entry
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int at = v0 + q * kThreads + tid;
            v[q].raw = make_uint4(T::kNegInfBits, T::kNegInfBits, T::kNegInfBits, T::kNegInfBits);
            if (at < vecs) v[q].raw = *reinterpret_cast<const uint4*>(body + (int64_t)at * VE);
        }
        if (split == 0) {
            if (tid < head)
                xj = tid;
            else if (tid < head + tail)
                xj = vecs * VE + tid;
            if (xj >= 0) x = T::to(row[xj]);
        }
        // maximum
        float vm[NV], tm = x;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            vm[q] = v[q].at(0);
#pragma unroll
            for (int e = 1; e < VE; ++e) vm[q] = fmaxf(vm[q], v[q].at(e));
            tm = fmaxf(tm, vm[q]);
        }
        if (A.top) lane_max[wave][lane] = ordered(tm);
        const float wm = lanes_max<64>(tm);
        if (lane == 0) red[wave][0] = wm;
        if (tid == 0) count = 0;
        __syncthreads();
        float M = kNegBig;
        for (int w = 0; w < W; ++w) M = fmaxf(M, red[w][0]);
        if (A.top && wave == 0) {
            uint32_t k = lane_max[0][lane];
            for (int w = 1; w < W; ++w) k = max(k, lane_max[w][lane]);
            k = kth_of_wave(k, A.top);
            if (lane == 0) shared_t = k;
        }
        // sums; an entry of -inf adds nothing
        float S = 0.0f, X = 0.0f;
        if (A.entropy) {
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float d = (v[q].at(e) - M) * A.c, ex = s_ex2(d);
                    S += ex;
                    X = fmaf(ex, fmaxf(d, -16384.0f), X);
                }
            const float d = (x - M) * A.c, ex = s_ex2(d);
            S += ex;
            X = fmaf(ex, fmaxf(d, -16384.0f), X);
        } else {
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int e = 0; e < VE; ++e) S += s_ex2((v[q].at(e) - M) * A.c);
            S += s_ex2((x - M) * A.c);
        }
        S = lanes_sum<64>(S);
        X = lanes_sum<64>(X);
        if (lane == 0) red[wave][1] = S, red[wave][2] = X;
        __syncthreads();
        S = X = 0.0f;
        for (int w = 0; w < W; ++w) S += red[w][1], X += red[w][2];

        if (tid == 0) {
            if (A.splits == 1)
                finish_row<T>(A, i, M, S, X);
            else
                A.pm[item] = M, A.ps[item] = S, A.px[item] = X;
        }
        if (A.top) {
            const uint32_t t = shared_t;
            const int jv = head + (v0 + tid) * VE;  // column of the thread's first entry
            // entries above the threshold, in any order
            if (__any(ordered(tm) > t)) {
                if (xj >= 0 && ordered(x) > t) {
                    const int at = atomicAdd(&count, 1);
                    if (at < kCap) list[at] = cand(x, xj);
                }
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    if (!__any(ordered(vm[q]) > t)) continue;
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float s = v[q].at(e);
                        if (ordered(s) > t) {
                            const int at = atomicAdd(&count, 1);
                            if (at < kCap) list[at] = cand(s, jv + q * kThreads * VE + e);
                        }
                    }
                }
            }
            __syncthreads();
            int have = count;
            uint64_t* out = A.splits == 1 ? nullptr : A.plist + item * A.top;
            if (have <= kCap) {
                // the first entries equal to the threshold: each wave its own first ones, in order of the column
                const int need = A.top - have;
                int mine = 0;  // found by this wave
                if (need > 0) {
                    uint64_t* eq = list + have + wave * need;
                    const uint64_t below = (1ull << lane) - 1;
                    // the single entries: the ones before the vectors come first, the ones after them last
                    for (int part = 0; part < 3; ++part) {
                        if (part == 1) {
#pragma unroll
                            for (int q = 0; q < NV; ++q) {
                                const bool in = v0 + q * kThreads + tid < vecs;
                                if (mine >= need || !__any(in && ordered(vm[q]) >= t)) continue;
                                uint32_t hit = 0;
                                int before = 0, total = 0;
#pragma unroll
                                for (int e = 0; e < VE; ++e) {
                                    const bool h = in && ordered(v[q].at(e)) == t;
                                    const uint64_t mask = __ballot(h);
                                    hit |= h ? 1u << e : 0u;
                                    before += __popcll(mask & below);
                                    total += __popcll(mask);
                                }
                                int at = mine + before;
#pragma unroll
                                for (int e = 0; e < VE; ++e)
                                    if (hit >> e & 1) {
                                        if (at < need) eq[at] = cand(v[q].at(e), jv + q * kThreads * VE + e);
                                        ++at;
                                    }
                                mine += total;
                            }
                        } else if (wave == 0 && split == 0 && mine < need) {
                            const bool h = xj >= 0 && (part == 0) == (xj < head) && ordered(x) == t;
                            const uint64_t mask = __ballot(h);
                            const int at = mine + __popcll(mask & below);
                            if (h && at < need) eq[at] = cand(x, xj);
                            mine += __popcll(mask);
                        }
                    }
                    mine = min(mine, need);
                    // close the gaps between the waves' entries with keys that rank last
                    for (int at = mine + lane; at < need; at += 64) eq[at] = 0;
                    have += W * need;
                }
                __syncthreads();
                for (int a = tid; a < have; a += kThreads) {
                    const uint64_t key = list[a];
                    int rank = 0;
                    for (int b = 0; b < have; ++b) rank += list[b] > key ? 1 : 0;
                    if (key && rank < A.top) {
                        if (out)
                            out[rank] = key;
                        else
                            finish_top<T>(A, i, rank, key, M, S);
                    }
                }
                // a chunk with fewer entries than asked for (only a cut row has one): the rest ranks last
                if (out) {
                    int found = 0;
                    for (int b = lane; b < have; b += 64) found += list[b] ? 1 : 0;
                    for (int o = 1; o < 64; o *= 2) found += __shfl_xor(found, o);
                    for (int r = found + tid; r < A.top; r += kThreads) out[r] = 0;
                }
            } else {
                // the largest entries crowd into a few lane classes: one round of the workgroup for each
                uint64_t last = ~0ull;
                for (int r = 0; r < A.top; ++r) {
                    uint64_t best = 0;
                    if (xj >= 0) {
                        const uint64_t k = cand(x, xj);
                        best = k < last ? k : 0;
                    }
#pragma unroll
                    for (int q = 0; q < NV; ++q)
                        if (v0 + q * kThreads + tid < vecs) {
#pragma unroll
                            for (int e = 0; e < VE; ++e) {
                                const uint64_t k = cand(v[q].at(e), jv + q * kThreads * VE + e);
                                best = k < last && k > best ? k : best;
                            }
                        }
                    const uint32_t hi = lanes_max<64>((uint32_t)(best >> 32));
                    const uint32_t lo = lanes_max<64>((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
                    if (lane == 0) list[wave] = (uint64_t)hi << 32 | lo;
                    __syncthreads();
                    best = list[0];
                    for (int w = 1; w < W; ++w) best = max(best, list[w]);
                    if (tid == 0) {
                        if (out)
                            out[r] = best;
                        else
                            finish_top<T>(A, i, r, best, M, S);
                    }
                    last = best;
                    __syncthreads();
                }
            }
        }
        __syncthreads();
    }
}

// Joins the chunks of a cut row: one workgroup per row.
template <class T>
__global__ __launch_bounds__(kBlock) void k_logprobs_join(LpArgs A) {
    extern __shared__ uint64_t list[];  // [splits][top]
    __shared__ float red[kBlock / 64][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    for (int64_t i = blockIdx.x; i < A.n; i += gridDim.x) {
        const int64_t p0 = i * A.splits;
        float M = kNegBig;
        for (int k = tid; k < A.splits; k += kBlock) M = fmaxf(M, A.pm[p0 + k]);
        M = lanes_max<64>(M);
        if (lane == 0) red[wave][0] = M;
        __syncthreads();
        for (int w = 0; w < kBlock / 64; ++w) M = fmaxf(M, red[w][0]);
        __syncthreads();
        float S = 0.0f, X = 0.0f;
        for (int k = tid; k < A.splits; k += kBlock) {
            const float s = A.ps[p0 + k], d = (A.pm[p0 + k] - M) * A.c, w = s_ex2(d);
            if (s == 0.0f) continue;
            S = fmaf(s, w, S);
            X = fmaf(w, fmaf(s, fmaxf(d, -16384.0f), A.px[p0 + k]), X);
        }
        S = lanes_sum<64>(S);
        X = lanes_sum<64>(X);
        if (lane == 0) red[wave][0] = S, red[wave][1] = X;
        const int total = A.splits * A.top;
        for (int a = tid; a < total; a += kBlock) list[a] = A.plist[p0 * A.top + a];
        __syncthreads();
        S = X = 0.0f;
        for (int w = 0; w < kBlock / 64; ++w) S += red[w][0], X += red[w][1];
        if (tid == 0) finish_row<T>(A, i, M, S, X);
        for (int a = tid; a < total; a += kBlock) {
            const uint64_t key = list[a];
            int rank = 0;
            for (int b = 0; b < total; ++b) rank += list[b] > key ? 1 : 0;
            if (key && rank < A.top) finish_top<T>(A, i, rank, key, M, S);
        }
        __syncthreads();
    }
}

struct LpGradArgs {
    const void* s;
    int64_t ld, ldg, n;
    int m;
    float eps, inv_eps, c;
    const int64_t* targets;
    const float *stats, *entropy;
    int top;
    const int32_t* top_idx;
    const float *d_logp, *d_lse, *d_entropy, *d_top;
    void* grad;
    int splits;
};

// ds_j = (1/eps) [ p_j (a0 + a1 y_j) + sum of the d of the picks at j ],
// y = c (s - M), p = 2^(y - log2 S), a1 = -d_H ln2,
// a0 = d_lse - sum of the picks' d - d_H (H - log S).
// One pass: a thread loads and stores the same entries (so the gradient may
// take the scores' place); the picks are put in afterwards by the workgroup
// whose chunk they lie in.
template <class T, int NV>
__global__ __launch_bounds__(kBlock) void k_logprobs_grad(LpGradArgs A) {
    constexpr int VE = Vec<T>::n;
    using E = typename T::type;
    __shared__ int pick_j[kMaxTop + 1];
    __shared__ float pick_d[kMaxTop + 1], pick_s[kMaxTop + 1];
    const int tid = threadIdx.x;
    for (int64_t item = blockIdx.x; item < A.n * A.splits; item += gridDim.x) {
        const int64_t i = item / A.splits;
        const int split = (int)(item % A.splits);
        const E* row = static_cast<const E*>(A.s) + i * A.ld;
        E* out = static_cast<E*>(A.grad) + i * A.ldg;
        const int picks = A.top + 1;
        float pull = 0.0f;
        {
            const int64_t t = A.targets ? A.targets[i] : -1;
            const float d = A.d_logp && t >= 0 ? A.d_logp[i] : 0.0f;
            if (A.d_logp && t >= A.m) pull = NAN;
            if (tid == 0) {
                pick_j[0] = t >= 0 && t < A.m && A.d_logp ? (int)t : -1;
                pick_d[0] = d;
            }
            for (int r = tid; r < A.top; r += kBlock) {
                const int j = A.d_top ? A.top_idx[i * A.top + r] : -1;
                pick_j[1 + r] = (unsigned)j < (unsigned)A.m ? j : -1;
                pick_d[1 + r] = A.d_top ? A.d_top[i * A.top + r] : 0.0f;
            }
        }
        __syncthreads();
        for (int r = 0; r < picks; ++r) pull += pick_j[r] >= 0 ? pick_d[r] : 0.0f;
        for (int r = tid; r < picks; r += kBlock) pick_s[r] = pick_j[r] >= 0 ? T::to(row[pick_j[r]]) : 0.0f;
        const float top = A.stats[2 * i], log_s = A.stats[2 * i + 1];
        const float M = top == -INFINITY ? 0.0f : top;  // an empty row: every y is -inf
        const float dh = A.d_entropy ? A.d_entropy[i] : 0.0f;
        const float a1 = -dh * kLn2 * A.inv_eps;
        const float a0 = ((A.d_lse ? A.d_lse[i] : 0.0f) - pull - (A.d_entropy ? dh * (A.entropy[i] - log_s) : 0.0f)) * A.inv_eps;
        const float inv_s = expf(-log_s);
        const float k0 = a0 * inv_s, k1 = a1 * inv_s;
        auto value = [&](float s) {
            const float y = (s - M) * A.c;
            return s_ex2(y) * fmaf(k1, fmaxf(y, -16384.0f), k0);
        };
        const int mis = (int)(reinterpret_cast<uintptr_t>(row) / sizeof(E) % VE);
        const int mis_out = (int)(reinterpret_cast<uintptr_t>(out) / sizeof(E) % VE);
        int64_t lo, hi;  // columns of this workgroup
        __syncthreads();  // the picks' scores are read before any of them may be overwritten
        if (mis == mis_out) {
            const int head = min(A.m, (VE - mis) % VE);
            const int vecs = (A.m - head) / VE, tail = A.m - head - vecs * VE;
            const int v0 = split * (kBlock * NV);
            Vec<T> v[NV];
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int at = v0 + q * kBlock + tid;
                if (at < vecs) v[q].raw = *reinterpret_cast<const uint4*>(row + head + (int64_t)at * VE);
            }
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int at = v0 + q * kBlock + tid;
                if (at >= vecs) break;
                union {
                    E e[VE];
                    uint4 raw;
                } o;
#pragma unroll
                for (int e = 0; e < VE; ++e) o.e[e] = T::from(value(v[q].at(e)));
                *reinterpret_cast<uint4*>(out + head + (int64_t)at * VE) = o.raw;
            }
            if (split == 0 && tid < head + tail) {
                const int j = tid < head ? tid : vecs * VE + tid;
                out[j] = T::from(value(T::to(row[j])));
            }
            // the row's first and last single entries belong to the first workgroup
            lo = split == 0 ? 0 : head + (int64_t)v0 * VE;
            hi = head + min((int64_t)vecs, (int64_t)v0 + kBlock * NV) * VE;
        } else {  // rows aligned differently: entry by entry
            const int width = kBlock * NV * VE;
            lo = min((int64_t)A.m, (int64_t)split * width);
            hi = split + 1 == A.splits ? A.m : min((int64_t)A.m, lo + width);
            for (int64_t j = lo + tid; j < hi; j += kBlock) out[j] = T::from(value(T::to(row[j])));
        }
        __syncthreads();
        for (int r = tid; r < picks; r += kBlock) {
            const int j = pick_j[r];
            if (j < 0) continue;
            bool mine = j >= lo && j < hi;
            if (mis == mis_out && split == 0) {
                const int head = min(A.m, (VE - mis) % VE), vecs = (A.m - head) / VE;
                mine = mine || j >= head + vecs * VE;
            }
            if (!mine) continue;
            float total = 0.0f;
            bool first = true;
            for (int u = 0; u < picks; ++u)
                if (pick_j[u] == j) {
                    if (u < r) first = false;
                    total += pick_d[u];
                }
            if (first) out[j] = T::from(fmaf(total, A.inv_eps, value(pick_s[r])));
        }
        __syncthreads();
    }
}

// Chunks of a row of m scores when a workgroup takes `vecs` vectors of 16 bytes.
int64_t chunks(int64_t m, int es, int vecs) {
    const int64_t v = m * es / 16;
    return std::max<int64_t>(1, (v + vecs - 1) / vecs);
}

constexpr int kLpWide = 8 * 64 * 8;  // vectors of the widest chunk

int64_t lp_splits(int64_t m, int es) { return chunks(m, es, kLpWide); }

struct LpLayout {
    int64_t splits;
    size_t pm, ps, px, plist, total;
};

LpLayout lp_layout(int es, int64_t n, int64_t m, int top) {
    LpLayout L{lp_splits(m, es), 0, 0, 0, 0, 256};
    if (L.splits == 1) return L;
    const size_t items = (size_t)n * (size_t)L.splits;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    L.ps = up(items * 4);
    L.px = L.ps + up(items * 4);
    L.plist = L.px + up(items * 4);
    L.total = L.plist + up(items * (size_t)top * 8) + 256;
    return L;
}

template <class T, int W, int NV>
void launch_lp(const LpArgs& A, hipStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>(A.n * A.splits, kLpGrid);
    hipLaunchKernelGGL((k_logprobs<T, W, NV>), dim3(grid), dim3(W * 64), 0, s, A);
}

template <class T>
hipError_t logprobs(const LpArgs& A, hipStream_t s) {
    const int64_t vecs = A.m * (int64_t)sizeof(typename T::type) / 16;
    if (vecs <= 64 * 2)
        launch_lp<T, 1, 2>(A, s);
    else if (vecs <= 64 * 8)
        launch_lp<T, 1, 8>(A, s);
    else if (vecs <= 512 * 2)
        launch_lp<T, 8, 2>(A, s);
    else
        launch_lp<T, 8, 8>(A, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || A.splits == 1) return e;
    hipLaunchKernelGGL((k_logprobs_join<T>), dim3((unsigned)std::min<int64_t>(A.n, kLpGrid)), dim3(kBlock),
                       (size_t)A.splits * A.top * 8, s, A);
    return hipGetLastError();
}

constexpr int kLpGradVecs = 4;

template <class T>
hipError_t logprobs_grad(const LpGradArgs& A, hipStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>(A.n * A.splits, kLpGrid);
    hipLaunchKernelGGL((k_logprobs_grad<T, kLpGradVecs>), dim3(grid), dim3(kBlock), 0, s, A);
    return hipGetLastError();
}

int check_top(int32_t top, int64_t m) {
    if (top < 0 || top > kMaxTop || top > m || (top > 0 && m > kTopMaxCols)) return SK_ERR_SHAPE;
    return SK_OK;
}

}  // namespace
}  // namespace sk

using namespace sk;

extern "C" {

size_t sk_scores_logprobs_workspace_bytes(int32_t dtype, int64_t n, int64_t m, int32_t top) {
    if (dtype != SK_F32 && dtype != SK_BF16 && dtype != SK_F16) return 0;
    if (n < 0 || m < 1 || n > INT32_MAX || m > INT32_MAX || check_top(top, m) != SK_OK) return 0;
    return lp_layout(elem_size(dtype), n, m, top).total;
}

int sk_scores_logprobs(const void* scores, int32_t dtype, int64_t n, int64_t m, int64_t ld, float eps,
                       const int64_t* targets, int32_t top, float* logp, float* lse, float* entropy, int32_t* top_idx,
                       float* top_logp, float* stats, void* ws, size_t ws_bytes, void* stream) {
    int st = check_scores(scores, dtype, n, m, ld);
    if (st) return st;
    if ((st = check_temperature(eps))) return st;
    if ((st = check_top(top, m))) return st;
    const LpLayout L = lp_layout(elem_size(dtype), n, m, top);
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < L.total) return SK_ERR_WORKSPACE;
    if (n == 0) return SK_OK;
    if (!lse || !stats || (targets && !logp) || (top > 0 && (!top_idx || !top_logp))) return SK_ERR_NULL;
    char* base = static_cast<char*>(ws);
    LpArgs A{};
    A.s = scores;
    A.ld = ld;
    A.n = n;
    A.m = (int)m;
    A.eps = eps;
    A.c = (float)(1.4426950408889634 / (double)eps);
    A.targets = targets;
    A.top = top;
    A.logp = logp;
    A.lse = lse;
    A.entropy = entropy;
    A.top_logp = top_logp;
    A.stats = stats;
    A.top_idx = top_idx;
    A.splits = (int)L.splits;
    A.pm = reinterpret_cast<float*>(base + L.pm);
    A.ps = reinterpret_cast<float*>(base + L.ps);
    A.px = reinterpret_cast<float*>(base + L.px);
    A.plist = reinterpret_cast<uint64_t*>(base + L.plist);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SK_TRY_LAUNCH(dtype == SK_F32    ? logprobs<F32>(A, s)
                  : dtype == SK_BF16 ? logprobs<Bf16>(A, s)
                                     : logprobs<F16>(A, s));
    return SK_OK;
}

int sk_scores_logprobs_grad(const void* scores, int32_t dtype, int64_t n, int64_t m, int64_t ld, float eps,
                            const int64_t* targets, const float* stats, const float* entropy, int32_t top,
                            const int32_t* top_idx, const float* d_logp, const float* d_lse, const float* d_entropy,
                            const float* d_top, void* grad, int64_t ld_grad, void* stream) {
    int st = check_scores(scores, dtype, n, m, ld);
    if (st) return st;
    if ((st = check_temperature(eps))) return st;
    if ((st = check_top(top, m))) return st;
    if ((st = check_grad(scores, ld, grad, ld_grad, dtype, n, m))) return st;
    if (n == 0) return SK_OK;
    if (!stats || (d_logp && !targets) || (d_entropy && !entropy) || (d_top && top > 0 && !top_idx)) return SK_ERR_NULL;
    LpGradArgs A{};
    A.s = scores;
    A.ld = ld;
    A.ldg = ld_grad;
    A.n = n;
    A.m = (int)m;
    A.eps = eps;
    A.inv_eps = (float)(1.0 / (double)eps);
    A.c = (float)(1.4426950408889634 / (double)eps);
    A.targets = targets;
    A.stats = stats;
    A.entropy = entropy;
    A.top = d_top ? top : 0;
    A.top_idx = top_idx;
    A.d_logp = d_logp;
    A.d_lse = d_lse;
    A.d_entropy = d_entropy;
    A.d_top = d_top;
    A.grad = grad;
    A.splits = (int)chunks(m, elem_size(dtype), kBlock * kLpGradVecs);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SK_TRY_LAUNCH(dtype == SK_F32    ? logprobs_grad<F32>(A, s)
                  : dtype == SK_BF16 ? logprobs_grad<Bf16>(A, s)
                                     : logprobs_grad<F16>(A, s));
    return SK_OK;
}

}  // extern "C"
