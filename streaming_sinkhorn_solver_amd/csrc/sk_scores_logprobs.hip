// sk_scores_logprobs.hip -- log-probabilities of given columns of a score
// matrix, entropy and the largest alternatives (sk_scores_logprobs), and their
// gradient (sk_scores_logprobs_grad).
//
// With z = s / eps and M = max_j s_j, S = sum_j exp((s_j - M)/eps) of a row,
//     lse = M/eps + log S,   log p_j = (s_j - M)/eps - log S,
//     H = -sum_j p_j log p_j = log S - (sum_j e_j d_j) / S,  d = (s - M)/eps, e = exp(d).
// The scores are read once: a thread keeps a running maximum and rescales its
// sums once per block of four 16-byte loads.  Rows are cut only where there are too few to
// fill the GPU, or where a row has more blocks than LDS has room for; a second
// kernel joins the cuts' (M, S, sum e d) and sorted lists of their largest entries.
//
// The largest entries: every thread leaves the maximum of each of its blocks in
// LDS.  The threads (in rows that a wave takes alone, its threads' blocks) are
// classes of entries; the k-th largest of the classes' maxima is at most the
// k-th largest score, so only blocks that reach it are looked at again, and of
// their entries only those above it (with 256 classes 21 at k = 20, 74 at k = 64 in
// the mean) and the first ones equal to it are candidates, whose ranks are counted.
// Ties go to the lowest column.  Where the largest entries crowd into few
// classes, or more entries equal the bound than the list holds, the cut is read
// again.
#include "sk_scores.hpp"

#include <algorithm>

namespace sk {
namespace {

constexpr int kMaxTop = 64;
constexpr int64_t kTopMaxCols = (int64_t)1 << 20;  // columns, where alternatives are asked for
constexpr int64_t kLpGrid = 1 << 20;               // workgroups of one launch (each may serve several rows)
constexpr int kLpVecs = 4;                         // 16-byte loads of a thread's block
constexpr int kLpBlocks = 32;                      // blocks whose maxima LDS holds: 32 KB

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
    int cut;  // vectors of 16 bytes in a cut of k_logprobs_stream
    // partial results of the chunks, [n * splits] each, lists [n * splits][top]
    float *pm, *ps, *px;
    uint64_t* plist;
};

// A candidate: larger score first, then lower column.
__device__ __forceinline__ uint64_t cand(float v, uint32_t j) { return (uint64_t)ordered(v) << 32 | (uint32_t)~j; }
__device__ __forceinline__ uint32_t cand_col(uint64_t k) { return ~(uint32_t)k; }

// The row's target and its score, loaded ahead of the sums they are needed after.  Called by one lane.
struct Target {
    int64_t t;
    float s;
};
template <class T>
__device__ __forceinline__ Target load_target(const LpArgs& A, int64_t i) {
    Target g{-1, 0.0f};
    if (A.targets) {
        g.t = A.targets[i];
        if (g.t >= 0 && g.t < A.m) g.s = T::to(static_cast<const typename T::type*>(A.s)[i * A.ld + g.t]);
    }
    return g;
}

// The row's outputs from its maximum and sums.  Called by one lane.
__device__ __forceinline__ void finish_row(const LpArgs& A, int64_t i, const Target& g, float M, float S, float X) {
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
        float lp = 0.0f;  // no token given
        if (g.t >= A.m)
            lp = NAN;
        else if (g.t >= 0)
            lp = empty ? -INFINITY : (g.s - M) / A.eps - log_s;
        A.logp[i] = lp;
    }
}

// (The key holds the score; a NaN's says -inf, but then S is NaN.)
__device__ __forceinline__ void finish_top(const LpArgs& A, int64_t i, int r, uint64_t key, float M, float S) {
    A.top_idx[i * A.top + r] = (int32_t)cand_col(key);
    A.top_logp[i * A.top + r] = S == 0.0f ? -INFINITY : (unordered((uint32_t)(key >> 32)) - M) / A.eps - logf(S);
}

template <class T>
struct Vec {
    static constexpr int n = 16 / sizeof(typename T::type);
    uint4 raw;
    __device__ __forceinline__ float at(int i) const {
        if constexpr (n == 4) {
            const uint32_t w = i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w;
            return __builtin_bit_cast(float, w);
        } else {
            const uint32_t w = i / 2 == 0 ? raw.x : i / 2 == 1 ? raw.y : i / 2 == 2 ? raw.z : raw.w;
            return T::to((uint16_t)(i % 2 ? w >> 16 : w & 0xffffu));
        }
    }
};

// Joins the (M, S, X) of lanes or waves: sums relative to the common maximum top.
__device__ __forceinline__ void rescale(float M, float top, float c, float& S, float& X) {
    const float d = fmaxf((M - top) * c, -16384.0f), w = s_ex2(d);
    X = w * fmaf(S, d, X);
    S *= w;
}

// The k-th largest of the classes' maxima: of all W * 64 threads', or, for small k, of the 64 lane numbers', which
// takes W times fewer steps and leaves about k^2 / 128 entries more (measured alike at k = 24).
template <int LOW, int W>
__device__ __forceinline__ uint32_t kth_of_classes(const uint32_t (*class_max)[64], int lane, int k) {
    uint32_t key[W], most[1] = {0};
#pragma unroll
    for (int w = 0; w < W; ++w) {
        key[w] = class_max[w][lane];
        most[0] = max(most[0], key[w]);
    }
    return k <= 24 ? kth_of_wave<LOW>(most, k) : kth_of_wave<LOW>(key, k);
}

// A row, or a cut of one, per W waves (4 / W rows per workgroup).  Dynamic LDS with TOP: the blocks' maxima,
// [blocks][256].
template <class T, int W, int NV, bool ENT, bool TOP>
__global__ __launch_bounds__(kBlock) void k_logprobs(LpArgs A) {
    constexpr int VE = Vec<T>::n, kThreads = W * 64, kRows = kBlock / kThreads, kStep = kThreads * NV;
    constexpr int kCap = W == 1 ? 704 : 1024;                  // candidates above the bound
    constexpr int kEqual = W * kMaxTop, kHits = TOP ? 512 : 1;  // entries equal to it; blocks that reach it
    __shared__ float red[kBlock / 64][3];
    __shared__ uint32_t class_max[TOP ? kBlock / 64 : 1][64];
    __shared__ uint64_t lists[TOP ? kRows : 1][TOP ? kCap + kEqual : 1];
    __shared__ uint16_t hit_lists[TOP ? kRows : 1][kHits];
    __shared__ int counts[kRows][3];
    extern __shared__ float block_max[];
    using E = typename T::type;
    const int t = threadIdx.x % kThreads, lane = threadIdx.x & 63, wave = threadIdx.x / 64, slot = threadIdx.x / kThreads;
    auto sync = [] {
        if constexpr (W == 1)
            wave_sync();
        else
            __syncthreads();
    };
    const int64_t items = A.n * A.splits;
    for (int64_t item0 = (int64_t)blockIdx.x * kRows; item0 < items; item0 += (int64_t)gridDim.x * kRows) {
        const int64_t item = item0 + slot;
        const bool on = item < items;
        const int64_t i = (on ? item : item0) / A.splits;
        const int split = (int)((on ? item : item0) - i * A.splits);
        const E* row = static_cast<const E*>(A.s) + i * A.ld;
        const int mis = (int)(reinterpret_cast<uintptr_t>(row) / sizeof(E) % VE);
        const int head = min(A.m, (VE - mis) % VE);
        const int vecs = (A.m - head) / VE, tail = A.m - head - vecs * VE;
        const int v0 = split * A.cut, v1 = min(vecs, v0 + A.cut);
        const uint4* body = reinterpret_cast<const uint4*>(row + head);
        const int blocks = v1 > v0 ? (v1 - v0 + kStep - 1) / kStep : 0;
        Target target{-1, 0.0f};
        if (t == 0 && A.splits == 1) target = load_target<T>(A, i);
        Vec<T> next[NV], v[NV];
        auto fetch = [&](int b) {
#pragma unroll
            for (int q = 0; q < NV; ++q) next[q].raw = body[min(v0 + b * kStep + q * kThreads + t, v1 - 1)];
        };
        if (blocks > 0) fetch(0);
        float M = kNegBig, S = 0.0f, X = 0.0f, single = -INFINITY, largest = -INFINITY;  // (M starts above -inf)
        int single_j = -1;
        if (split == 0 && t < head + tail) {  // the row's single entries, one per thread
            single_j = t < head ? t : vecs * VE + t;
            single = T::to(row[single_j]);
            M = fmaxf(M, single);
            largest = fmaxf(largest, single);
            const float d = (single - M) * A.c;
            S = s_ex2(d);
            X = S * fmaxf(d, -16384.0f);
        }
        for (int b = 0; b < blocks; ++b) {
#pragma unroll
            for (int q = 0; q < NV; ++q) v[q] = next[q];
            if (b + 1 < blocks) {
                fetch(b + 1);
            } else {  // vectors behind the end
#pragma unroll
                for (int q = 0; q < NV; ++q)
                    if (v0 + b * kStep + q * kThreads + t >= v1)
                        v[q].raw = make_uint4(T::kNegInfBits, T::kNegInfBits, T::kNegInfBits, T::kNegInfBits);
            }
            float top = -INFINITY;
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int e = 0; e < VE; ++e) top = fmaxf(top, v[q].at(e));
            if (TOP) {
                block_max[b * kBlock + threadIdx.x] = top;
                largest = fmaxf(largest, top);
            }
            top = fmaxf(M, top);
            rescale(M, top, A.c, S, X);
            M = top;
            float s = 0.0f, x = 0.0f;
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float d = (v[q].at(e) - M) * A.c, ex = s_ex2(d);
                    s += ex;
                    if (ENT) x = fmaf(ex, fmaxf(d, -16384.0f), x);  // an entry of -inf adds nothing
                }
            S += s;
            X += x;
        }
        float top = lanes_max<64>(M);
        if (TOP) class_max[wave][lane] = blocks > 0 || single_j >= 0 ? ordered(largest) : 0u;
        if (TOP && t == 0) counts[slot][0] = counts[slot][1] = counts[slot][2] = 0;
        if (W > 1) {
            if (lane == 0) red[wave][0] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < W; ++w) top = fmaxf(top, red[w][0]);
        }
        rescale(M, top, A.c, S, X);
        S = lanes_sum<64>(S);
        if (ENT) X = lanes_sum<64>(X);
        if (W > 1) {
            if (lane == 0) red[wave][1] = S, red[wave][2] = X;
            __syncthreads();
            S = X = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) S += red[w][1], X += red[w][2];
        }
        if (t == 0 && on) {
            if (A.splits == 1)
                finish_row(A, i, target, top, S, X);
            else
                A.pm[item] = top, A.ps[item] = S, A.px[item] = X;
        }
        if constexpr (TOP) {
            if (W == 1) wave_sync();
            uint64_t* list = lists[slot];
            uint16_t* hits = hit_lists[slot];
            int* count = counts[slot];  // candidates above the bound, blocks that reach it, entries that equal it
            uint32_t bound;
            if constexpr (W == 1) {
                const float second = blocks > 1 ? block_max[kBlock + threadIdx.x] : -INFINITY;
                const uint32_t first = blocks > 1 ? ordered(fmaxf(block_max[threadIdx.x], single)) : class_max[wave][lane];
                const uint32_t key[2] = {first, blocks > 1 ? ordered(second) : 0u};
                bound = kth_of_wave<T::kLowBits>(key, A.top);
            } else {
                bound = kth_of_classes<T::kLowBits, W>(class_max, lane, A.top);
            }
            // a mask that leaves fewer classes than k: the entries equal to the bound are the masked ones
            const bool masked = bound <= ordered(-INFINITY);
            auto column = [&](int at, int e) { return (uint32_t)(head + at * VE + e); };
            auto see = [&](float s, uint32_t j, bool equals) {
                const uint32_t k = ordered(s);
                if (k > bound) {
                    const int at = atomicAdd(&count[0], 1);
                    if (at < kCap) list[at] = cand(s, j);
                } else if (equals && k == bound) {
                    const int at = atomicAdd(&count[2], 1);
                    if (at < kEqual) list[kCap + at] = cand(s, j);
                }
            };
            if (single_j >= 0) see(single, (uint32_t)single_j, true);
            for (int b = 0; b < blocks; ++b)
                if (ordered(block_max[b * kBlock + threadIdx.x]) >= bound + (masked ? 1 : 0)) {
                    const int at = atomicAdd(&count[1], 1);
                    if (at < kHits) hits[at] = (uint16_t)(b * kThreads + t);
                }
            sync();
            const int reached = count[1];
            if (reached <= kHits) {
                for (int h = t; h < reached * NV; h += kThreads) {
                    const int hit = hits[h / NV], at = v0 + hit / kThreads * kStep + h % NV * kThreads + hit % kThreads;
                    if (at >= v1) continue;
                    Vec<T> x;
                    x.raw = body[at];
#pragma unroll
                    for (int e = 0; e < VE; ++e) see(x.at(e), column(at, e), !masked);
                }
            } else {
                for (int at = v0 + t; at < v1; at += kThreads) {
                    Vec<T> x;
                    x.raw = body[at];
#pragma unroll
                    for (int e = 0; e < VE; ++e) see(x.at(e), column(at, e), false);
                }
            }
            sync();
            const int above = count[0], equal = count[2];
            uint64_t* out = A.splits == 1 ? nullptr : A.plist + (on ? item : item0) * A.top;
            auto place = [&](int rank, uint64_t key) {
                if (!on) return;
                if (out)
                    out[rank] = key;
                else
                    finish_top(A, i, rank, key, top, S);
            };
            if (above <= kCap) {
                const int need = A.top - above;
                int have = above;
                if (need > 0 && !masked && reached <= kHits && equal <= kEqual) {
                    for (int a = t; a < equal; a += kThreads) {
                        const uint64_t key = list[kCap + a];  // moved up behind the others; kCap is far behind them
                        list[above + a] = key;
                    }
                    have = above + equal;
                } else if (need > 0) {
                    // masked ones, or more than the list holds: each wave its own first ones, in order of the column
                    uint64_t* eq = list + above + (wave % W) * need;
                    const uint64_t below = (1ull << lane) - 1;
                    int mine = 0;
                    auto take = [&](bool hit, uint64_t key, int before, int total) {
                        if (hit && mine + before < need) eq[mine + before] = key;
                        mine += total;
                    };
                    auto take_single = [&](bool in) {
                        const bool hit = in && ordered(single) == bound;
                        const uint64_t mask = __ballot(hit);
                        take(hit, cand(single, (uint32_t)single_j), __popcll(mask & below), __popcll(mask));
                    };
                    take_single(single_j >= 0 && single_j < head);
                    for (int at0 = v0 + (wave % W) * 64; at0 < v1 && mine < need; at0 += kThreads) {
                        const int at = at0 + lane;
                        Vec<T> x;
                        x.raw = body[min(at, v1 - 1)];
                        uint32_t hit = 0;
                        int before = 0, total = 0;
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            const bool h = at < v1 && ordered(x.at(e)) == bound;
                            const uint64_t mask = __ballot(h);
                            hit |= h ? 1u << e : 0u;
                            before += __popcll(mask & below);
                            total += __popcll(mask);
                        }
                        int to = mine + before;
#pragma unroll
                        for (int e = 0; e < VE; ++e)
                            if (hit >> e & 1) {
                                if (to < need) eq[to] = cand(x.at(e), column(at, e));
                                ++to;
                            }
                        mine += total;
                    }
                    if (mine < need) take_single(single_j >= head);
                    for (int at = min(mine, need) + lane; at < need; at += 64) eq[at] = 0;  // ranks last
                    have = above + W * need;
                }
                sync();
                int found = 0;
                for (int a = t; a < have; a += kThreads) {
                    const uint64_t key = list[a];
                    int rank = 0;
#pragma unroll 4
                    for (int b = 0; b < have; ++b) rank += list[b] > key ? 1 : 0;
                    if (key && rank < A.top) place(rank, key);
                }
                if (out) {  // a cut with fewer entries than asked for: the rest ranks last
                    for (int b = lane; b < have; b += 64) found += list[b] ? 1 : 0;
                    found = (int)lanes_sum_u<64>((uint32_t)found);
                    for (int r = found + t; r < A.top; r += kThreads) place(r, 0);
                }
            } else {
                // the largest entries crowd into a few classes: one reading of the cut for each
                uint64_t last = ~0ull;
                for (int r = 0; r < A.top; ++r) {
                    uint64_t best = 0;
                    auto look = [&](uint64_t k) { best = k < last && k > best ? k : best; };
                    if (single_j >= 0) look(cand(single, (uint32_t)single_j));
                    for (int at = v0 + t; at < v1; at += kThreads) {
                        Vec<T> x;
                        x.raw = body[at];
#pragma unroll
                        for (int e = 0; e < VE; ++e) look(cand(x.at(e), column(at, e)));
                    }
                    const uint32_t hi = lanes_max<64>((uint32_t)(best >> 32));
                    const uint32_t lo = lanes_max<64>((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
                    best = (uint64_t)hi << 32 | lo;
                    if (W > 1) {
                        if (lane == 0) list[wave] = best;
                        __syncthreads();
#pragma unroll
                        for (int w = 0; w < W; ++w) best = max(best, list[w]);
                        __syncthreads();
                    }
                    if (t == 0) place(r, best);
                    last = best;
                }
            }
            sync();
        }
    }
}

// Joins the chunks of a cut row: one wave per row, or (TOP) one workgroup.
template <class T, bool TOP>
__global__ __launch_bounds__(kBlock) void k_logprobs_join(LpArgs A) {
    constexpr int kWaves = TOP ? kBlock / 64 : 1, kRows = kBlock / 64 / kWaves;
    extern __shared__ uint64_t list[];  // [splits][top] entries, then those near the top
    const int tid = threadIdx.x, lane = tid & 63;
    for (int64_t i0 = (int64_t)blockIdx.x * kRows; i0 < A.n; i0 += (int64_t)gridDim.x * kRows) {
        const int64_t i = min(i0 + (TOP ? 0 : tid / 64), A.n - 1);
        const int64_t p0 = i * A.splits;
        const Target target = load_target<T>(A, i);
        const int total = A.splits * A.top;
        if (TOP)
            for (int a = tid; a < total; a += kBlock) list[a] = A.plist[p0 * A.top + a];
        // every wave joins the sums for itself
        float M = kNegBig, S = 0.0f, X = 0.0f;
        for (int k = lane; k < A.splits; k += 64) {
            const float m = A.pm[p0 + k], s = A.ps[p0 + k], x = A.px[p0 + k], top = fmaxf(M, m);
            float s1 = s, x1 = x;
            rescale(m, top, A.c, s1, x1);
            rescale(M, top, A.c, S, X);
            S += s1;
            X += x1;
            M = top;
        }
        const float top = lanes_max<64>(M);
        rescale(M, top, A.c, S, X);
        S = lanes_sum<64>(S);
        X = lanes_sum<64>(X);
        if (TOP ? tid == 0 : lane == 0 && i0 + tid / 64 < A.n) finish_row(A, i, target, top, S, X);
        if constexpr (TOP) {
            // as in k_logprobs: the entries' upper halves reach the k-th largest thread's maximum, then ranks
            __shared__ uint32_t class_max[kBlock / 64][64];
            __shared__ int count;
            if (tid == 0) count = 0;
            __syncthreads();
            uint32_t most = 0;
            for (int a = tid; a < total; a += kBlock) most = max(most, (uint32_t)(list[a] >> 32));
            class_max[tid / 64][lane] = most;
            __syncthreads();
            const uint32_t bound = max(kth_of_classes<T::kLowBits, kBlock / 64>(class_max, lane, A.top), 1u);  // (0: no entry)
            uint64_t* near = list + total;
            for (int a = tid; a < total; a += kBlock)
                if ((uint32_t)(list[a] >> 32) >= bound) near[atomicAdd(&count, 1)] = list[a];
            __syncthreads();
            const int have = count;
            for (int a = tid; a < have; a += kBlock) {
                const uint64_t mine = near[a];
                int rank = 0;
#pragma unroll 4
                for (int b = 0; b < have; ++b) rank += near[b] > mine ? 1 : 0;
                if (rank < A.top) finish_top(A, i, rank, mine, top, S);
            }
            __syncthreads();
        }
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
// whose chunk they lie in.  Rows whose scores and gradient lie differently to 16
// bytes go entry by entry: 4096 rows of 50257 bf16 scores out of 50304 take 400 us
// into a gradient of 50257, 152 into one of the scores' own row stride (7 rows of 8
// of the former are such rows), 144 in place.
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

// How a forward pass cuts its rows: whole where there are kFill of them, else to make kFill pieces, none below kCutMin
// vectors.  With alternatives a piece has at most kLpBlocks blocks, and a row no more pieces than
// the joining workgroup ranks the lists of, kJoin entries, where that leaves pieces of kLpBlocks.
constexpr int kFill = 1024, kCutMin = 1024, kJoin = 1024;

struct LpCut {
    int64_t splits;
    int cut;
};

LpCut lp_cut(int es, int64_t n, int64_t m, int top) {
    const int64_t vecs = std::max<int64_t>(1, m * es / 16);
    int64_t most = std::min((kFill + n - 1) / std::max<int64_t>(n, 1), vecs / kCutMin);
    if (top > 0) {
        const int64_t longest = (int64_t)kLpBlocks * kLpVecs * kBlock;
        most = std::max(std::min<int64_t>(most, kJoin / top), (vecs + longest - 1) / longest);
    }
    most = std::max<int64_t>(1, most);
    const int64_t cut = (vecs + most - 1) / most;
    return {(vecs + cut - 1) / cut, (int)cut};
}

struct LpLayout {
    LpCut cut;
    size_t pm, ps, px, plist, total;
};

LpLayout lp_layout(int es, int64_t n, int64_t m, int top) {
    LpLayout L{lp_cut(es, n, m, top), 0, 0, 0, 0, 256};
    if (L.cut.splits == 1) return L;
    const size_t items = (size_t)n * (size_t)L.cut.splits;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    L.ps = up(items * 4);
    L.px = L.ps + up(items * 4);
    L.plist = L.px + up(items * 4);
    L.total = L.plist + up(items * (size_t)top * 8) + 256;
    return L;
}

template <class T, int W, int NV>
void launch_rows(const LpArgs& A, hipStream_t s) {
    const int rows = kBlock / (W * 64);
    const unsigned grid = (unsigned)std::min<int64_t>((A.n * A.splits + rows - 1) / rows, kLpGrid);
    auto kernel = A.top ? (A.entropy ? k_logprobs<T, W, NV, true, true> : k_logprobs<T, W, NV, false, true>)
                        : (A.entropy ? k_logprobs<T, W, NV, true, false> : k_logprobs<T, W, NV, false, false>);
    const int step = W * 64 * NV;
    const size_t lds = A.top ? (size_t)((A.cut + step - 1) / step) * kBlock * sizeof(float) : 0;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kBlock), lds, s, A);
}

template <class T>
hipError_t logprobs(const LpArgs& A, hipStream_t s) {
    // a wave takes a row alone up to two blocks (512 vectors), with one vector per lane where that is all of it
    const int64_t vecs = A.m * (int64_t)sizeof(typename T::type) / 16;
    if (vecs <= 64)
        launch_rows<T, 1, 1>(A, s);
    else if (vecs <= 2 * 64 * kLpVecs)
        launch_rows<T, 1, kLpVecs>(A, s);
    else
        launch_rows<T, 4, kLpVecs>(A, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || A.splits == 1) return e;
    if (A.top > 0)
        hipLaunchKernelGGL((k_logprobs_join<T, true>), dim3((unsigned)std::min<int64_t>(A.n, kLpGrid)), dim3(kBlock),
                           (size_t)A.splits * A.top * 16, s, A);
    else
        hipLaunchKernelGGL((k_logprobs_join<T, false>), dim3((unsigned)std::min<int64_t>((A.n + 3) / 4, kLpGrid)),
                           dim3(kBlock), 0, s, A);
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
    A.splits = (int)L.cut.splits;
    A.cut = L.cut.cut;
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
