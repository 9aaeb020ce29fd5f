// sk_route_rows.hip -- token rows under a routing: the choices sorted by expert
// (sk_route_sort), token rows copied into that order (sk_route_dispatch), the
// experts' rows summed back onto their tokens (sk_route_combine), and the
// gradient of that sum (sk_route_combine_grad).
//
// A choice, or pair, t = i k + r is the r-th expert of token i.  The plan is a
// 0/1 matrix with one entry per pair; dispatch applies it, combine its transpose,
// both with the routing's weights or without.
#include "sk_scores.hpp"

#include <algorithm>
#include <type_traits>

namespace sk {
namespace {

constexpr int kRowsMaxExperts = 1024;
constexpr int kRowsMaxTop = 64;

// ----- the choices sorted by expert ---------------------------------------------------
// A stable counting sort.  A wave takes its pairs 64 at a time, in order; lanes of
// equal expert find one another by one ballot per bit of its number, so a pair's rank
// among the wave's pairs of its expert is a count of lower lanes beside the wave's own
// counter in LDS.  Adding the counts of the waves and workgroups before gives the rank
// among all.  131072 choices among 256 take 10.6 us: two launches of 128 workgroups.  The second
// (8.0) issues vector instructions in 56 % of its CUs' cycles, 570 in each wave, and its waves
// wait for the tables' loads and for one another in 58 % of theirs.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortMost = 16;      // pairs per thread at most: a wave's counter fits 16 bits
constexpr int kSortOne = 4096;     // pairs that one workgroup takes alone
// Workgroups whose counts the others add up themselves: 64, and up to 256 where that is no more than 32768 counts
// (524288 choices among 128: 256 take 12.8 us, 128 13.5; among 256: 128 take 15.1, 64 18.3, 256 15.5; among 512: 64 take
// 20.4, 128 18.1, where 131072 take 12.1 and 13.1; 131072 among 1024: 64 take 14.9, 128 18.0, 32 15.4).
int sort_groups(int64_t m) { return (int)std::min<int64_t>(256, std::max<int64_t>(64, 32768 / m)); }

struct SortArgs {
    const int32_t* idx;
    int64_t pairs, rows;
    int m, bits, align, capacity;
    int per;  // pairs of a workgroup
    int groups, scanned;
    int wide;  // power of two >= m
    int32_t *slot, *source, *counts, *offsets;
    int32_t* hist;  // [groups][m] counts of the workgroups (scanned: of those before), then [m] totals
};

__device__ __forceinline__ int expert_of(const SortArgs& A, int64_t t) {
    const int e = t < A.pairs ? A.idx[t] : A.m;
    return (unsigned)e < (unsigned)A.m ? e : A.m;  // m: dropped
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs A) {
    __shared__ int hist[kRowsMaxExperts];
    for (int e = threadIdx.x; e < A.m; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * A.per;
    for (int q = threadIdx.x; q < A.per; q += kSortThreads) {
        const int e = expert_of(A, t0 + q);
        if (e < A.m) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < A.m; e += kSortThreads) A.hist[(int64_t)blockIdx.x * A.m + e] = hist[e];
}

// Counts of each workgroup to those of the workgroups before it, 64 experts per workgroup.
__global__ __launch_bounds__(kSortThreads) void k_sort_scan(SortArgs A) {
    __shared__ int part[kSortWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64, e = blockIdx.x * 64 + lane;
    const int64_t per = (A.groups + kSortWaves - 1) / kSortWaves;
    const int64_t g0 = min(per * wave, (int64_t)A.groups), g1 = min(g0 + per, (int64_t)A.groups);
    int sum = 0;
    if (e < A.m)
        for (int64_t g = g0; g < g1; ++g) sum += A.hist[g * A.m + e];
    part[wave][lane] = sum;
    __syncthreads();
    int run = 0, total = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        run += w < wave ? part[w][lane] : 0;
        total += part[w][lane];
    }
    if (e >= A.m) return;
    for (int64_t g = g0; g < g1; ++g) {
        const int here = A.hist[g * A.m + e];
        A.hist[g * A.m + e] = run;
        run += here;
    }
    if (wave == 0) A.hist[(int64_t)A.groups * A.m + e] = total;
}

template <int J>
__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortArgs A) {
    __shared__ uint16_t count[kSortWaves][kRowsMaxExperts];  // then: of the waves before
    __shared__ int first[kRowsMaxExperts], stop[kRowsMaxExperts], before[kRowsMaxExperts], all[kRowsMaxExperts];
    __shared__ int sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64, group = blockIdx.x;
    // the other workgroups' counts: each thread some of them for one expert, requested before all else
    int prior = 0, total = 0;
    if (A.groups > 1) {
        const int q = tid & (A.wide - 1), parts = kSortThreads / A.wide;
        if (A.scanned) {
            if (tid < A.m) {
                prior = A.hist[(int64_t)group * A.m + tid];
                total = A.hist[(int64_t)A.groups * A.m + tid];
            }
        } else if (q < A.m) {
#pragma unroll 16
            for (int g = tid / A.wide; g < A.groups; g += parts) {
                const int here = A.hist[g * A.m + q];
                prior += g < group ? here : 0;
                total += here;
            }
        }
    }
    for (int e = tid; e < A.m; e += kSortThreads) before[e] = all[e] = 0;
    for (int e = lane; e < A.m; e += 64) count[wave][e] = 0;
    wave_sync();
    const int64_t t0 = (int64_t)group * A.per + wave * (64 * J) + lane;
    int e[J], rank[J];
#pragma unroll
    for (int j = 0; j < J; ++j) e[j] = expert_of(A, t0 + j * 64);
#pragma unroll
    for (int j = 0; j < J; ++j) {
        uint64_t same = ~0ull;
        for (int b = 0; b < A.bits; ++b) {
            const bool set = e[j] >> b & 1;
            const uint64_t with = __ballot(set);
            same &= set ? with : ~with;
        }
        const int lower = __popcll(same & ((1ull << lane) - 1));
        rank[j] = lower + (e[j] < A.m ? count[wave][e[j]] : 0);
        wave_sync();
        if (e[j] < A.m && (same >> lane) == 1) count[wave][e[j]] = (uint16_t)(rank[j] + 1);  // the highest of them
        wave_sync();
    }
    __syncthreads();
    if (A.groups > 1 && (tid & (A.wide - 1)) < A.m) {
        atomicAdd(&before[tid & (A.wide - 1)], prior);
        atomicAdd(&all[tid & (A.wide - 1)], total);
    }
    __syncthreads();
    // each thread an expert: its pairs in this workgroup's waves, and in all; then the segments' first rows
    int kept = 0, padded = 0;
    if (tid < A.m) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const int here = count[w][tid];
            count[w][tid] = (uint16_t)run;
            run += here;
        }
        total = A.groups == 1 ? run : all[tid];
        kept = A.capacity ? min(total, A.capacity) : total;
        padded = (int)(((int64_t)kept + A.align - 1) / A.align * A.align);
    }
    int upto = padded;
    for (int o = 1; o < 64; o *= 2) {
        const int low = __shfl_up(upto, o);
        if (lane >= o) upto += low;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int end = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        const int s = sums[w];
        upto += w < wave ? s : 0;
        end += s;
    }
    if (tid < A.m) {
        first[tid] = upto - padded;
        stop[tid] = upto - padded + kept;
        if (group == 0) {
            A.counts[tid] = kept;
            A.offsets[tid + 1] = upto;
            if (tid == 0) A.offsets[0] = 0;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int64_t t = t0 + j * 64;
        if (t >= A.pairs) continue;
        int at = -1;
        if (e[j] < A.m) {
            const int r = before[e[j]] + count[wave][e[j]] + rank[j];
            if (!A.capacity || r < A.capacity) at = first[e[j]] + r;
        }
        A.slot[t] = at;
        if (at >= 0) A.source[at] = (int32_t)t;
    }
    // rows of no pair: the segments' padding, and what lies behind the last segment
    if (A.align > 1)
        for (int q = group * kSortWaves + wave; q < A.m; q += A.groups * kSortWaves) {
            const int next = q + 1 < A.m ? first[q + 1] : end;
            for (int s = stop[q] + lane; s < next; s += 64) A.source[s] = -1;
        }
    for (int64_t s = end + (int64_t)group * kSortThreads + tid; s < A.rows; s += (int64_t)A.groups * kSortThreads) A.source[s] = -1;
}

template <int J>
hipError_t launch_place(const SortArgs& A, hipStream_t s) {
    hipLaunchKernelGGL((k_sort_place<J>), dim3((unsigned)A.groups), dim3(kSortThreads), 0, s, A);
    return hipGetLastError();
}

// How the pairs are shared out: per workgroup a power-of-two number of pairs per thread.
struct SortPlan {
    int per_thread, groups;
    size_t total;
};

SortPlan sort_plan(int64_t pairs, int64_t m) {
    SortPlan P{1, 1, 256};
    const int64_t most = pairs <= kSortOne ? 1 : sort_groups(m);
    while (P.per_thread < kSortMost && (int64_t)P.per_thread * kSortThreads * most < pairs) P.per_thread *= 2;
    const int64_t per = (int64_t)P.per_thread * kSortThreads;
    P.groups = (int)std::max<int64_t>(1, (pairs + per - 1) / per);
    if (P.groups > 1) P.total = ((size_t)(P.groups + 1) * (size_t)m * 4 + 255) / 256 * 256;
    return P;
}

// Rows of the sorted pairs at most, every segment rounded up to align; -1 for invalid arguments or beyond 2^31 - 1.
int64_t sort_rows(int64_t n, int32_t k, int64_t m, int32_t align, int32_t capacity) {
    if (n < 0 || n > INT32_MAX || k < 1 || k > kRowsMaxTop || m < 1 || m > kRowsMaxExperts || align < 1 || capacity < 0)
        return -1;
    const int64_t pairs = n * k;
    int64_t rows = pairs + std::min(pairs, m) * ((int64_t)align - 1);
    if (capacity) rows = std::min(rows, m * (((int64_t)capacity + align - 1) / align * align));
    return rows <= INT32_MAX && pairs <= INT32_MAX ? rows : -1;
}

// ----- token rows -----------------------------------------------------------------------
// A row goes in pieces of 16 bytes at any address.  Where it does not end with one, the copy and the sum let the last
// piece end with the row and overlap the one before, whose elements are then stored twice, the same; but for a sum
// over what is added, which stores the last elements one by one, as the gradient does, which counts each once.  Rows
// shorter than a piece go element by element.
constexpr int64_t kRowsMaxCols = (int64_t)1 << 28;  // (32-bit offsets inside a row)

struct RowsArgs {
    int64_t n, rows;
    int d, k, m;
    int lanes;         // of a token: a power of two up to the workgroup
    int whole, pieces, rest;  // whole pieces of a row, all of them, and the elements behind the whole ones
    bool apart;        // the output is no input
    int parts, span;       // workgroups that share a token's row, and the pieces of each
    int64_t token_groups;  // groups of kBlock / lanes tokens, times parts
    int64_t grid;          // workgroups that take them in turn
    int pad_parts;         // workgroups behind them for each expert's padding, 0: there is none
    const int32_t *slot, *counts, *offsets;
    const float* weights;
    const void *tokens, *add, *in;  // (n, d); (n, d); (rows, d)
    int64_t ld_tokens, ld_add, ld_in;
    void* out;
    int64_t ld_out;
    float* d_weights;
};

__device__ __forceinline__ bool in_rows(const RowsArgs& A, int s) { return (uint64_t)(int64_t)s < (uint64_t)A.rows; }
// First element of piece q.
template <class T>
__device__ __forceinline__ int piece_at(const RowsArgs& A, int q) {
    return q < A.whole ? q * Run16<T>::n : A.d - Run16<T>::n;
}
// The workgroups behind those of the tokens: zeros into the segments' padding.
template <class T>
__device__ void clear_padding(const RowsArgs& A) {
    using E = typename T::type;
    const int item = (int)(blockIdx.x - A.grid), e = item % A.m, part = item / A.m;
    const int64_t s0 = max((int64_t)A.offsets[e] + A.counts[e], (int64_t)0), s1 = min((int64_t)A.offsets[e + 1], A.rows);
    Run16<T> zero;
    zero.fill(0);
    for (int64_t s = s0 + part; s < s1; s += A.pad_parts) {
        E* row = static_cast<E*>(A.out) + s * A.ld_out;
        for (int q = threadIdx.x; q < A.pieces; q += kBlock) zero.put(row + piece_at<T>(A, q));
        if (A.pieces == 0 && (int)threadIdx.x < A.d) row[threadIdx.x] = E(0);
    }
}

// f(token, lane in the token's group, first and last piece) for the thread's tokens.  ONE: all lanes of a wave have the
// same token.
template <bool ONE, class F>
__device__ __forceinline__ void each_token(const RowsArgs& A, F f) {
    int in_group = threadIdx.x / A.lanes;
    const int lane = threadIdx.x % A.lanes;
    if (ONE) in_group = __builtin_amdgcn_readfirstlane(in_group);
    for (int64_t g = blockIdx.x; g < A.token_groups; g += A.grid) {
        int64_t i = g * (kBlock / A.lanes) + in_group;
        int q0 = 0, q1 = A.pieces;
        if (ONE && A.parts > 1) {
            i = (uint32_t)g / (uint32_t)A.parts;
            q0 = (int)(g - i * A.parts) * A.span;
            q1 = min(A.pieces, q0 + A.span);
        }
        if (i < A.n) f(i, lane, q0 + lane, q1);
    }
}

// rows[slot] = (w) x: a token's piece is read once and stored to each of its rows.
// ONCE: the stores pass the caches by, for rows of whole cache lines (16384 x 8 rows of 2048 bf16: 105 us against 119;
// of 2040, whose lines two rows share: 143 against 134).
template <class T, bool ONE, bool ONCE>
__global__ __launch_bounds__(kBlock) void k_dispatch(RowsArgs A) {
    using E = typename T::type;
    constexpr int VE = Run16<T>::n;
    if (blockIdx.x >= A.grid) return clear_padding<T>(A);
    each_token<ONE>(A, [&](int64_t i, int lane, int q0, int q1) {
        const E* x = static_cast<const E*>(A.tokens) + i * A.ld_tokens;
        const int32_t* slot = A.slot + i * A.k;
        const float* weights = A.weights ? A.weights + i * A.k : nullptr;
        auto each_row = [&](auto f) {
            for (int r = 0; r < A.k; ++r) {
                const int s = slot[r];
                if (in_rows(A, s)) f(static_cast<E*>(A.out) + s * A.ld_out, weights ? weights[r] : 1.0f);
            }
        };
        for (int q = q0; q < q1; q += A.lanes) {
            const int j = piece_at<T>(A, q);
            Run16<T> v;
            v.get(x + j);
            each_row([&](E* row, float w) {
                Run16<T> o = v;
                if (weights) {
                    float f[VE];
#pragma unroll
                    for (int c = 0; c < VE; ++c) f[c] = w * v.at(c);
                    o.round(f);
                }
                o.template store<ONCE>(row + j);
            });
        }
        if (A.pieces == 0 && lane < A.d) {
            const E v = x[lane];
            each_row([&](E* row, float w) { row[lane] = weights ? T::from(w * T::to(v)) : v; });
        }
    });
}

constexpr int kAheadMost = 8;  // rows of a token whose pieces are in flight

// y = add + sum_r w_r rows[slot_r], in the order of r, float32, rounded once.  Bound by the rows' reads: 16384 x 8 rows
// of 2048 f16 take 105 us, 6.4 TB/s.
// ONCE: the rows are read past the caches (131 us otherwise).  REST: they do not end with a whole piece.
template <class T, bool ONE, bool ONCE, bool REST>
__global__ __launch_bounds__(kBlock) void k_combine(RowsArgs A) {
    using E = typename T::type;
    constexpr int VE = Run16<T>::n, kAhead = kAheadMost;
    each_token<ONE>(A, [&](int64_t i, int lane, int q0, int q1) {
        const int32_t* slot = A.slot + i * A.k;
        const float* weights = A.weights ? A.weights + i * A.k : nullptr;
        const E* add = A.add ? static_cast<const E*>(A.add) + i * A.ld_add : nullptr;
        E* out = static_cast<E*>(A.out) + i * A.ld_out;
        for (int q = q0; q < q1; q += A.lanes) {
            const int j = REST ? piece_at<T>(A, q) : q * VE;
            float y[VE];
            Run16<T> v[kAhead];
            if (add) v[0].get(add + j);
#pragma unroll
            for (int c = 0; c < VE; ++c) y[c] = add ? v[0].at(c) : 0.0f;
            for (int r0 = 0; r0 < A.k; r0 += kAhead) {
                float w[kAhead];
#pragma unroll
                for (int r = 0; r < kAhead; ++r) {
                    const int s = r0 + r < A.k ? slot[r0 + r] : -1;
                    const bool in = in_rows(A, s);
                    w[r] = !in ? 0.0f : weights ? weights[r0 + r] : 1.0f;
                    v[r].fill(0);
                    if (in) v[r].template fetch<ONCE>(static_cast<const E*>(A.in) + s * A.ld_in + j);
                }
#pragma unroll
                for (int r = 0; r < kAhead; ++r) {
                    v[r].held();
#pragma unroll
                    for (int c = 0; c < VE; ++c) y[c] = fmaf(w[r], v[r].at(c), y[c]);
                }
            }
            v[0].round(y);
            if (!REST || q < A.whole || A.apart) {
                v[0].template store<ONCE>(out + j);
            } else {
#pragma unroll
                for (int c = 1; c < VE; ++c)
                    if (c >= VE - A.rest) out[j + c] = v[0].bits(c);
            }
        }
        if (A.pieces == 0 && lane < A.d) {
            float y = add ? T::to(add[lane]) : 0.0f;
            for (int r = 0; r < A.k; ++r) {
                const int s = slot[r];
                if (in_rows(A, s))
                    y = fmaf(weights ? weights[r] : 1.0f, T::to(static_cast<const E*>(A.in)[s * A.ld_in + lane]), y);
            }
            out[lane] = T::from(y);
        }
    });
}

// d_rows[slot_r] = w_r d_y and d_w_r = <rows[slot_r], d_y>: d_y is read once per kAhead rows, eight or four.  A thread reads a piece of
// a row before it stores the gradient's, so that the gradient may take the rows' place.  Bound by memory: 16384 x 8 rows
// of 2048 bf16 take 200 us, 5.7 TB/s.
// Rows of less than a wave's pieces go four at a time: 65536 x 8 rows of 203 bf16 208 us with dispatch's gradient, 239 by eights.
template <class T, int L, bool ONCE>
__global__ __launch_bounds__(kBlock) void k_combine_grad(RowsArgs A) {
    using E = typename T::type;
    constexpr int VE = Run16<T>::n, kWaves = L > 64 ? L / 64 : 1, kAhead = L < 64 ? 4 : kAheadMost;
    __shared__ float part[kAhead][kWaves];
    if (blockIdx.x >= A.grid) return clear_padding<T>(A);
    int in_group = threadIdx.x / L;
    const int lane = threadIdx.x % L;
    if (L >= 64) in_group = __builtin_amdgcn_readfirstlane(in_group);
    for (int64_t g = blockIdx.x; g < A.token_groups; g += A.grid) {
        const int64_t at = g * (kBlock / L) + in_group, i = min(at, A.n - 1);
        const bool on = at < A.n;  // (the others repeat the last token and store nothing)
        const E* dy = static_cast<const E*>(A.tokens) + i * A.ld_tokens;
        const int32_t* slot = A.slot + i * A.k;
        for (int r0 = 0; r0 < A.k; r0 += kAhead) {
            float dot[kAhead], w[kAhead];
            int s[kAhead];
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
                s[r] = r0 + r < A.k ? slot[r0 + r] : -1;
                if (!in_rows(A, s[r])) s[r] = -1;
                w[r] = s[r] < 0 ? 0.0f : A.weights ? A.weights[i * A.k + r0 + r] : 1.0f;
                dot[r] = 0.0f;
            }
            for (int q = lane; q < A.whole; q += L) {
                Run16<T> dyr, v[kAhead];
                dyr.get(dy + q * VE);
                if (A.d_weights) {
#pragma unroll
                    for (int r = 0; r < kAhead; ++r) {
                        v[r].fill(0);
                        if (s[r] >= 0) v[r].template fetch<ONCE>(static_cast<const E*>(A.in) + s[r] * A.ld_in + q * VE);
                    }
                }
                float gf[VE];
#pragma unroll
                for (int c = 0; c < VE; ++c) gf[c] = dyr.at(c);
#pragma unroll
                for (int r = 0; r < kAhead; ++r) {
                    if (s[r] < 0) continue;
                    if (A.d_weights) {
                        v[r].held();
#pragma unroll
                        for (int c = 0; c < VE; ++c) dot[r] = fmaf(v[r].at(c), gf[c], dot[r]);
                    }
                    if (A.out && on) {
                        float o[VE];
#pragma unroll
                        for (int c = 0; c < VE; ++c) o[c] = w[r] * gf[c];
                        Run16<T> scaled;
                        scaled.round(o);
                        scaled.put(static_cast<E*>(A.out) + s[r] * A.ld_out + q * VE);
                    }
                }
            }
            if (lane < A.rest) {  // (fewer than the lanes)
                const int j = A.whole * VE + lane;
                const float gf = T::to(dy[j]);
                float x[kAhead];
#pragma unroll
                for (int r = 0; r < kAhead; ++r)
                    x[r] = s[r] >= 0 && A.d_weights ? T::to(static_cast<const E*>(A.in)[s[r] * A.ld_in + j]) : 0.0f;
#pragma unroll
                for (int r = 0; r < kAhead; ++r) {
                    if (s[r] < 0) continue;
                    if (A.d_weights) dot[r] = fmaf(x[r], gf, dot[r]);
                    if (A.out && on) static_cast<E*>(A.out)[s[r] * A.ld_out + j] = T::from(w[r] * gf);
                }
            }
            if (!A.d_weights) continue;
#pragma unroll
            for (int r = 0; r < kAhead; ++r) dot[r] = lanes_sum<(L < 64 ? L : 64)>(dot[r]);
            if constexpr (L > 64) {
                const int wave = threadIdx.x / 64;
                __syncthreads();
                if ((threadIdx.x & 63) == 0)
#pragma unroll
                    for (int r = 0; r < kAhead; ++r) part[r][wave] = dot[r];
                __syncthreads();
#pragma unroll
                for (int r = 0; r < kAhead; ++r) {
                    dot[r] = 0.0f;
#pragma unroll
                    for (int w2 = 0; w2 < kWaves; ++w2) dot[r] += part[r][w2];
                }
            }
#pragma unroll
            for (int r = 0; r < kAhead; ++r)
                if (lane == 0 && on && r0 + r < A.k) A.d_weights[i * A.k + r0 + r] = s[r] < 0 ? 0.0f : dot[r];
        }
    }
}

// ----- host side ------------------------------------------------------------------------
constexpr int64_t kRowsGrid = 1 << 20;  // workgroups of one launch at most

// How a row of d elements goes, and the fewest lanes, a power of two from `least` on, that hold its pieces.
template <class T>
void share(RowsArgs& A, int least) {
    constexpr int VE = Run16<T>::n;
    A.whole = A.d / VE;
    A.rest = A.d % VE;
    A.pieces = A.whole + (A.whole > 0 && A.rest > 0 ? 1 : 0);
    A.lanes = least;
    while (A.lanes < kBlock && A.lanes < (A.whole > 0 ? A.pieces : A.d)) A.lanes *= 2;
    A.parts = 1;
    A.span = A.pieces;
    A.pad_parts = A.counts ? std::min(16, std::max(1, 1024 / A.m)) : 0;
}

// Whether rows take whole cache lines, that no two share.
template <class T>
bool whole_lines(const void* p, int64_t ld, int d) {
    const int64_t es = sizeof(typename T::type);
    return reinterpret_cast<uintptr_t>(p) % 128 == 0 && ld * es % 128 == 0 && d * es % 128 == 0;
}

// Whether the rows that are summed are read past the caches: where no two share a line, or where rows are so long that few
// of their lines are shared.  65536 x 8 rows of 203 bf16: the sum takes 49 us through the caches and 61 past them, 16384 x 8 of
// 2040 122 and 107; both gradients of 300 286 and 315, of 2040 362 and 330.  Between them, 32768 x 8 rows: the sum of 600 89
// and 88, of 1010 124 and 110, of 1040 152 and 149, of 1500 184 and 172; both gradients of 600 245 and 232, of 1010 393 and 377, of 1040
// 409 and 402, of 1500 557 and 591.
template <class T>
bool past_caches(const RowsArgs& A) {
    return A.pieces > 128 || whole_lines<T>(A.in, A.ld_in, A.d);
}

// Few tokens with long rows: several workgroups for each, every one with a run of pieces (1 x 8 rows of 8192 bf16: the sum
// takes 4.7 us so, 10.5 in one workgroup; 64 x 8 6.9 and 22.4, dispatch with its sort 8.3 and 13.2; 512 x 8 of 4096 10.4 and 15.4, dispatch
// 14.5 and 14.3, of 8192 19.3 and 28.2, 20.5 and 21.5).  Of more tokens only the sum would gain (768 x 8 of 4096 12.9 in halves and 17.3, 1024
// 18.9 and 19.0; dispatch 17.4 and 17.0, 20.9 and 20.1).  The gradient's rows are not shared out: partial dot products would have to be joined.
void split_rows(RowsArgs& A) {
    const int most = (A.pieces + kBlock - 1) / kBlock;
    if (A.lanes < kBlock || A.n > 512 || most < 2) return;
    const int each = (most + std::min(most, (int)(1024 / A.n)) - 1) / std::min(most, (int)(1024 / A.n));
    A.span = each * kBlock;
    A.parts = (A.pieces + A.span - 1) / A.span;
}

template <class K>
hipError_t launch_rows(RowsArgs A, K kernel, hipStream_t s) {
    const int per = kBlock / A.lanes;
    A.token_groups = (A.n + per - 1) / per * A.parts;
    A.grid = std::min(A.token_groups, kRowsGrid);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(A.grid + (int64_t)A.pad_parts * A.m)), dim3(kBlock), 0, s, A);
    return hipGetLastError();
}

template <class T>
hipError_t dispatch(RowsArgs A, hipStream_t s) {
    share<T>(A, 4);
    split_rows(A);
    auto kernel = A.lanes < 64                                 ? k_dispatch<T, false, false>
                  : whole_lines<T>(A.out, A.ld_out, A.d) ? k_dispatch<T, true, true>
                                                               : k_dispatch<T, true, false>;
    return launch_rows(A, kernel, s);
}

template <class T>
hipError_t combine(RowsArgs A, hipStream_t s) {
    share<T>(A, 4);
    split_rows(A);
    A.apart = A.add != A.out;
    const bool once = past_caches<T>(A);
    auto kernel = A.lanes < 64 ? (A.rest ? k_combine<T, false, false, true>
                                  : once ? k_combine<T, false, true, false>
                                         : k_combine<T, false, false, false>)
                  : once       ? (A.rest ? k_combine<T, true, true, true> : k_combine<T, true, true, false>)
                               : (A.rest ? k_combine<T, true, false, true> : k_combine<T, true, false, false>);
    return launch_rows(A, kernel, s);
}

template <class T>
hipError_t combine_grad(RowsArgs A, hipStream_t s) {
    share<T>(A, 8);
    if (A.lanes == 128) A.lanes = 64;  // (a wave alone needs no barrier)
    if (!A.out) A.pad_parts = 0;
    auto by_lanes = [&](auto once) {
        constexpr bool O = decltype(once)::value;
        return A.lanes == 8    ? k_combine_grad<T, 8, O>
               : A.lanes == 16 ? k_combine_grad<T, 16, O>
               : A.lanes == 32 ? k_combine_grad<T, 32, O>
               : A.lanes == 64 ? k_combine_grad<T, 64, O>
                               : k_combine_grad<T, 256, O>;
    };
    return launch_rows(A, past_caches<T>(A) ? by_lanes(std::true_type()) : by_lanes(std::false_type()), s);
}

// Sizes shared by the three row operators.
int check_rows(int32_t dtype, int64_t n, int64_t d, int32_t k, int64_t rows) {
    if (dtype != SK_F32 && dtype != SK_BF16 && dtype != SK_F16) return SK_ERR_DTYPE;
    if (n < 0 || n > INT32_MAX || d < 1 || d > kRowsMaxCols || rows < 0 || rows > INT32_MAX) return SK_ERR_SHAPE;
    if (k < 1 || k > kRowsMaxTop) return SK_ERR_ROUTE;
    return SK_OK;
}

int check_matrix(const void* p, int32_t dtype, int64_t rows, int64_t d, int64_t ld) {
    if (!good_stride(ld, rows, d)) return SK_ERR_SHAPE;
    if (rows > 0 && !p) return SK_ERR_NULL;
    return reinterpret_cast<uintptr_t>(p) % elem_size(dtype) != 0 ? SK_ERR_DTYPE : SK_OK;
}

// Whether an output meets what a plan and its weights hold.
bool meet_plan(Span out, const int32_t* slot, const float* weights, int64_t pairs, const int32_t* counts, const int32_t* offsets,
               int64_t m) {
    return meet(span_of(slot, pairs, 4), out) || (weights && meet(span_of(weights, pairs, 4), out)) ||
           (counts && (meet(span_of(counts, m, 4), out) || meet(span_of(offsets, m + 1, 4), out)));
}

// counts and offsets are given together, with m.
int check_padding(const int32_t* counts, const int32_t* offsets, int64_t m) {
    if (!counts && !offsets) return SK_OK;
    if (!counts || !offsets) return SK_ERR_NULL;
    return m < 1 || m > kRowsMaxExperts ? SK_ERR_SHAPE : SK_OK;
}

}  // namespace
}  // namespace sk

using namespace sk;

extern "C" {

int64_t sk_route_sort_rows(int64_t n, int32_t k, int64_t m, int32_t align, int32_t capacity) {
    return sort_rows(n, k, m, align, capacity);
}

size_t sk_route_sort_workspace_bytes(int64_t n, int32_t k, int64_t m) {
    return sort_rows(n, k, m, 1, 0) < 0 ? 0 : sort_plan(n * k, m).total;
}

int sk_route_sort(const int32_t* idx, int64_t n, int32_t k, int64_t m, int32_t align, int32_t capacity, int32_t* slot,
                  int32_t* source, int64_t rows, int32_t* counts, int32_t* offsets, void* ws, size_t ws_bytes,
                  void* stream) {
    if (n < 0 || n > INT32_MAX || m < 1 || m > kRowsMaxExperts) return SK_ERR_SHAPE;
    if (k < 1 || k > kRowsMaxTop || align < 1 || capacity < 0) return SK_ERR_ROUTE;
    const int64_t most = sort_rows(n, k, m, align, capacity);
    if (most < 0 || rows < most || rows > INT32_MAX) return SK_ERR_SHAPE;
    if ((n > 0 && (!idx || !slot)) || (rows > 0 && !source) || !counts || !offsets) return SK_ERR_NULL;
    const SortPlan P = sort_plan(n * k, m);
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < P.total) return SK_ERR_WORKSPACE;
    const Span choices = span_of(idx, n * k, 4);
    if ((slot != idx && meet(span_of(slot, n * k, 4), choices)) || meet(span_of(source, rows, 4), choices) ||
        meet(span_of(counts, m, 4), choices) || meet(span_of(offsets, m + 1, 4), choices))
        return SK_ERR_OVERLAP;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SortArgs A{};
    A.idx = idx;
    A.pairs = n * k;
    A.rows = rows;
    A.m = (int)m;
    while ((m >> A.bits) > 0) ++A.bits;  // the numbers 0 to m
    A.align = align;
    A.capacity = capacity;
    A.per = P.per_thread * kSortThreads;
    A.groups = P.groups;
    A.scanned = P.groups > sort_groups(m);
    A.wide = 1;
    while (A.wide < m) A.wide *= 2;
    A.slot = slot;
    A.source = source;
    A.counts = counts;
    A.offsets = offsets;
    A.hist = static_cast<int32_t*>(ws);
    if (A.groups > 1) {
        hipLaunchKernelGGL(k_sort_count, dim3((unsigned)A.groups), dim3(kSortThreads), 0, s, A);
        SK_TRY_LAUNCH(hipGetLastError());
    }
    if (A.scanned) {
        hipLaunchKernelGGL(k_sort_scan, dim3((unsigned)((m + 63) / 64)), dim3(kSortThreads), 0, s, A);
        SK_TRY_LAUNCH(hipGetLastError());
    }
    SK_TRY_LAUNCH(P.per_thread == 1   ? launch_place<1>(A, s)
                  : P.per_thread == 2 ? launch_place<2>(A, s)
                  : P.per_thread == 4 ? launch_place<4>(A, s)
                  : P.per_thread == 8 ? launch_place<8>(A, s)
                                      : launch_place<16>(A, s));
    return SK_OK;
}

int sk_route_dispatch(const void* x, int32_t dtype, int64_t n, int64_t d, int64_t ld, const int32_t* slot, int32_t k,
                      const float* weights, const int32_t* counts, const int32_t* offsets, int64_t m, void* out,
                      int64_t rows, int64_t ld_out, void* stream) {
    int st = check_rows(dtype, n, d, k, rows);
    if (st) return st;
    if ((st = check_matrix(x, dtype, n, d, ld)) || (st = check_matrix(out, dtype, rows, d, ld_out))) return st;
    if ((st = check_padding(counts, offsets, m))) return st;
    if (n == 0 || rows == 0) return SK_OK;
    if (!slot) return SK_ERR_NULL;
    const Span to = span_of(out, rows, d, ld_out, elem_size(dtype));
    if (meet(span_of(x, n, d, ld, elem_size(dtype)), to) || meet_plan(to, slot, weights, n * k, counts, offsets, m))
        return SK_ERR_OVERLAP;
    RowsArgs A{};
    A.n = n;
    A.d = (int)d;
    A.rows = rows;
    A.k = k;
    A.m = (int)m;
    A.slot = slot;
    A.counts = counts;
    A.offsets = offsets;
    A.weights = weights;
    A.tokens = x;
    A.ld_tokens = ld;
    A.out = out;
    A.ld_out = ld_out;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SK_TRY_LAUNCH(dtype == SK_F32 ? dispatch<F32>(A, s) : dtype == SK_BF16 ? dispatch<Bf16>(A, s) : dispatch<F16>(A, s));
    return SK_OK;
}

int sk_route_combine(const void* in, int32_t dtype, int64_t rows, int64_t d, int64_t ld_in, const int32_t* slot,
                     int64_t n, int32_t k, const float* weights, const void* add, int64_t ld_add, void* y, int64_t ld_y,
                     void* stream) {
    int st = check_rows(dtype, n, d, k, rows);
    if (st) return st;
    if ((st = check_matrix(in, dtype, rows, d, ld_in)) || (st = check_matrix(y, dtype, n, d, ld_y))) return st;
    if (add && (st = check_matrix(add, dtype, n, d, ld_add))) return st;
    if (n == 0) return SK_OK;
    if (!slot) return SK_ERR_NULL;
    const int es = elem_size(dtype);
    const Span out = span_of(y, n, d, ld_y, es);
    if (meet(span_of(in, rows, d, ld_in, es), out) || meet_plan(out, slot, weights, n * k, nullptr, nullptr, 0))
        return SK_ERR_OVERLAP;
    const bool in_place = add == y && (ld_add == ld_y || n == 1);
    if (add && !in_place && meet(span_of(add, n, d, ld_add, es), out)) return SK_ERR_OVERLAP;
    RowsArgs A{};
    A.n = n;
    A.d = (int)d;
    A.rows = rows;
    A.k = k;
    A.slot = slot;
    A.weights = weights;
    A.add = add;
    A.ld_add = ld_add;
    A.in = in;
    A.ld_in = ld_in;
    A.out = y;
    A.ld_out = ld_y;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SK_TRY_LAUNCH(dtype == SK_F32 ? combine<F32>(A, s) : dtype == SK_BF16 ? combine<Bf16>(A, s) : combine<F16>(A, s));
    return SK_OK;
}

int sk_route_combine_grad(const void* in, int32_t dtype, int64_t rows, int64_t d, int64_t ld_in, const int32_t* slot,
                          int64_t n, int32_t k, const float* weights, const int32_t* counts, const int32_t* offsets,
                          int64_t m, const void* d_y, int64_t ld_dy, void* d_rows, int64_t ld_out, float* d_weights,
                          void* stream) {
    int st = check_rows(dtype, n, d, k, rows);
    if (st) return st;
    if (d_weights && (st = check_matrix(in, dtype, rows, d, ld_in))) return st;
    if ((st = check_matrix(d_y, dtype, n, d, ld_dy))) return st;
    if (d_rows && (st = check_matrix(d_rows, dtype, rows, d, ld_out))) return st;
    if ((st = check_padding(counts, offsets, m))) return st;
    if (n == 0) return SK_OK;
    if (!slot || (!d_rows && !d_weights)) return SK_ERR_NULL;
    const int es = elem_size(dtype);
    if (d_rows) {
        const Span out = span_of(d_rows, rows, d, ld_out, es);
        if (meet(span_of(d_y, n, d, ld_dy, es), out)) return SK_ERR_OVERLAP;
        const bool in_place = in == d_rows && (ld_in == ld_out || rows == 1);
        if (d_weights && !in_place && meet(span_of(in, rows, d, ld_in, es), out)) return SK_ERR_OVERLAP;
        if (meet_plan(out, slot, weights, n * k, counts, offsets, m)) return SK_ERR_OVERLAP;
    }
    if (d_weights) {
        const Span out = span_of(d_weights, n * k, 4);
        if (meet(span_of(in, rows, d, ld_in, es), out) || meet(span_of(d_y, n, d, ld_dy, es), out)) return SK_ERR_OVERLAP;
        if (meet_plan(out, slot, d_weights == weights ? nullptr : weights, n * k, counts, offsets, m)) return SK_ERR_OVERLAP;
    }
    RowsArgs A{};
    A.n = n;
    A.d = (int)d;
    A.rows = rows;
    A.k = k;
    A.m = (int)m;
    A.slot = slot;
    A.counts = counts;
    A.offsets = offsets;
    A.weights = weights;
    A.tokens = d_y;
    A.ld_tokens = ld_dy;
    A.in = in;
    A.ld_in = ld_in;
    A.out = rows > 0 ? d_rows : nullptr;
    A.ld_out = ld_out;
    A.d_weights = d_weights;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SK_TRY_LAUNCH(dtype == SK_F32 ? combine_grad<F32>(A, s) : dtype == SK_BF16 ? combine_grad<Bf16>(A, s) : combine_grad<F16>(A, s));
    return SK_OK;
}

}  // extern "C"
