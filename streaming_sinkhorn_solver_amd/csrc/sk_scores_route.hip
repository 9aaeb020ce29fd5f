// sk_scores_route.hip -- routing of tokens to experts from a given score
// matrix (sk_scores_route) and its gradient (sk_scores_route_grad).
//
// act_ij is softmax_j(s_i.) or sigmoid(s_ij); the experts of row i are the k
// largest v_ij = (act_ij or s_ij) + bias_j, inside the topk_group best of
// n_group equal groups of columns when there are groups (a group's score is
// the sum of its group_top largest v); ties go to the lowest index.  The
// weights come from act at the chosen experts, without the bias.
//
// One row per L lanes with E scores each, in registers.  Wide rows find the k-th
// largest of the lanes' maxima, a lower bound of the k-th largest value, and rank
// the few entries above it by counting; narrow rows, and rows whose largest entries
// crowd into a few lanes, take k rounds of an argmax (16384 x 256, k = 8: 30 us in
// rounds alone, 14 ranked; with k = 16 of 16 lanes, where the bound is not used, 23).
// The kernel is bound by latency and issue, not by the 16.8 MB that it reads: about
// 650 vector instructions per wave of four rows.
//
// The order of two values that are closer than the float32 rounding of act or
// of the sum with the bias would depend on that rounding.  The choice is
// therefore checked against error bounds (one entry more than k is ranked for it),
// and rows where a pair that decides is too close are marked: their first index is
// stored as its complement.  Entries of equal score and equal bias tie exactly and
// are not in doubt (16384 x 256 bf16 scores under a bias of zeros: 18 us; 186 with
// their ties taken as doubt).  A second kernel, which also counts the rows per
// expert, chooses the marked rows again in float64, a workgroup each: the result is
// that of the definition.  (With the float64 code in the first kernel its registers
// leave two waves per SIMD, or spill, and one doubtful row holds up the end of the
// launch.)  Groups whose sums tie are in doubt: 16384 x 256 equal scores in 8 groups
// send every row there and take 1.0 ms.
#include "sk_scores.hpp"

#include <algorithm>

namespace sk {
namespace {

constexpr int kRouteMaxCols = 1024;
constexpr int kRouteMaxTop = 64;
constexpr int kRouteMaxGroups = 64;
constexpr int kRouteGroupsOfGrid = 2048;  // workgroups: eight per CU
constexpr int kFinishRows = 128;          // rows that a workgroup of the second kernel takes at a time
constexpr int kFinishGroups = 128;        // its workgroups, each of which adds up to m counts to memory

struct RouteArgs {
    const void* s;
    int64_t ld;
    int n, m;
    int sigmoid;       // act: 0 softmax, 1 sigmoid
    const float* bias; // null: none
    int raw;           // v from the raw score (also where act alone decides: act keeps the scores' order)
    int by_score;      // act without a bias: v for the groups' scores, the scores themselves inside them
    int n_group, topk_group, group_top, group_size;
    uint32_t group_magic;  // ceil(2^20 / group_size): (j * magic) >> 20 = j / group_size for j < 1024
    int k, renorm;
    float scale;
    int32_t* idx;
    float* weights;
    int32_t* counts;   // null: not wanted
    int doubt;         // values are rounded: a row may be marked
    int count_here;    // one workgroup and no doubt: the routing kernel counts
};

__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float exp_of(float x) { return s_ex2(kLog2e * x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float sigmoid_of(float x) { return rcp(1.0f + exp_of(-x)); }
__device__ __forceinline__ double sigmoid_of(double x) { return 1.0 / (1.0 + exp(-x)); }
// act exp(-shift) with shift >= the largest exponent of the row's choice, so that it does not underflow
// together: exp(x - shift), or exp(min(x, 0) - shift) / (1 + exp(-|x|)).
__device__ __forceinline__ float act_exponent(bool sigmoid, float x) { return sigmoid ? fminf(x, 0.0f) : x; }
__device__ __forceinline__ float act_shifted(bool sigmoid, float x, float shift) {
    const float e = exp_of(act_exponent(sigmoid, x) - shift);
    return sigmoid ? e * rcp(1.0f + exp_of(-fabsf(x))) : e;
}

// The value that decides the choice, from the row's maximum M and the reciprocal of the
// sum of its exponentials.  The same expression in float32 and float64.
template <class R>
__device__ __forceinline__ R choice_value(const RouteArgs& A, float s, float bias, float M, R inv_S) {
    R v = (R)s;
    if (!A.raw) v = A.sigmoid ? sigmoid_of((R)s) : exp_of((R)s - (R)M) * inv_S;
    return A.bias ? v + (R)bias : v;
}

// How far the float32 choice_value may be off.  One step is 2^-23.
//  softmax: an exponent d carries less than 1.25 d steps, the hardware's exp2 one;
//    the sum of at most 16 + 6 additions 11 steps and its terms' own mean error, at most
//    1.25 log m + 1 < 10; reciprocal and product 2: less than act (2 d + 32) steps.
//  sigmoid: the exponential's relative error, less than 1.25 |s| + 1 steps, enters by the factor 1 - sigmoid, where
//    |s| (1 - sigmoid) < 0.28 for s > 0; sum and reciprocal add 1.5: less than act (4 + 1.25 max(0, -s)) steps.
//    That is less than 4 steps, as s falls from 0 act falls faster than the factor rises.
//  the sum with the bias adds half a step of the value.
// An act below 2^-126 may be off by that much (subnormal, or flushed). A masked score's act and an expert switched off
// by a bias of -inf are exact.
constexpr float kStep = 0x1p-23f, kLost = 0x1p-126f;
__device__ __forceinline__ float choice_error(const RouteArgs& A, float s, float v, float M, float inv_S) {
    if (v == -INFINITY) return 0.0f;
    float err = A.bias ? fabsf(v) * kStep : 0.0f;
    if (!A.raw) {
        err += kLost + kStep * (A.sigmoid ? sigmoid_of(s) * (4.0f + 1.25f * fminf(fmaxf(0.0f, -s), 128.0f))
                                          : exp_of(s - M) * inv_S * (2.0f * fminf(M - s, 128.0f) + 32.0f));
    }
    return err;
}
// The most that act's part of it can be in the row (act (2 d + 32) falls with d).
__device__ __forceinline__ float act_error(const RouteArgs& A, float inv_S) {
    return A.raw ? 0.0f : A.sigmoid ? 4.0f * kStep : 32.0f * kStep * inv_S;
}

// The float32 keys of the routing kernel are the values themselves: a NaN value
// has been made -inf, and a column that takes no part is a NaN, which the
// hardware's maximum and every comparison pass over.
__device__ __forceinline__ float key_of(float v) { return fmaxf(v, -INFINITY); }

// LDS of one wave (64 / L rows): the rows' scores (their keys while groups are chosen), and small arrays.
template <int L, int E>
struct alignas(16) RouteWave {
    static constexpr int kRows = 64 / L, kList = 2 * L;
    float s[kRows][L * E];
    union {  // at different times: candidates, lanes' maxima, the groups' scores
        uint64_t list[kRows][kList];
        float lane_key[kRows][L];
        float gscore[kRows][kRouteMaxGroups];
    };
    int count[kRows];
    uint16_t won[kRows][kRouteMaxTop + 1];
};

// The kk-th largest of the row's lanes' keys (NaN for a lane without one), kk at most the lanes that have one;
// -inf if there are fewer.  Counted through LDS.
template <int L, int E>
__device__ __forceinline__ float kth_of_lanes(RouteWave<L, E>& W, float key, int l, int row, int kk) {
    W.lane_key[row][l] = key;
    wave_sync();
    int rank = 0;
#pragma unroll
    for (int q = 0; q < L; q += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&W.lane_key[row][q]);
        rank += (x.x > key ? 1 : 0) + (x.y > key ? 1 : 0) + (x.z > key ? 1 : 0) + (x.w > key ? 1 : 0);
    }
    wave_sync();
    // the ranks below kk belong to the kk largest and what equals the last of them
    const float low = -lanes_max<L>(rank < kk ? -key : -INFINITY);
    const uint32_t some = lanes_sum_u<L>(key == key && rank < kk ? 1u : 0u);
    return some >= (uint32_t)kk ? low : -INFINITY;
}

// Sets to NaN the keys of columns outside the row's best groups.  close: whether the
// last group taken and the first left out are within their errors.
template <class Rw, int L, int E>
__device__ __forceinline__ void keep_groups(const RouteArgs& A, RouteWave<L, E>& W, float (&key)[E], int l, int row,
                                            float act_err, float inv_S, bool* close) {
    // the lanes of a row share its groups out, `per` lanes to a group (a power of two)
    int per = 1;
    while (2 * per * A.n_group <= L) per *= 2;
    const int share = (A.group_size + per - 1) / per;  // columns of one lane
    uint64_t taken = 0;                                // bit g: group g is one of the best
    float worst_err = 0.0f;
    for (int g0 = 0; g0 < A.n_group; g0 += L / per) {
        const int g = g0 + l / per, sub = l % per;
        float k1 = -INFINITY, k2 = -INFINITY;
        if (g < A.n_group) {
            // each lane starts somewhere else in its group, so the lanes do not meet in one bank
            int q = l % share;
            for (int n = 0; n < share; ++n) {
                const int at = sub * share + q;
                const float x = at < A.group_size ? W.s[row][g * A.group_size + at] : -INFINITY;
                k2 = fmaxf(k2, fminf(k1, x));
                k1 = fmaxf(k1, x);
                if (++q == share) q = 0;
            }
        }
        for (int o = 1; o < per; o *= 2) {
            const float y1 = __shfl_xor(k1, o), y2 = __shfl_xor(k2, o);
            k2 = fmaxf(fminf(k1, y1), fmaxf(k2, y2));
            k1 = fmaxf(k1, y1);
        }
        // (half the sum of two values, which does not overflow, and is exact but for subnormal ones)
        const float v1 = A.group_top == 2 ? 0.5f * k1 : k1, v2 = A.group_top == 2 ? 0.5f * k2 : 0.0f;
        const float sum = key_of(v1 + v2);
        float err = fabsf(sum) * kStep + kLost;
        if (A.bias) err += (fabsf(v1) + fabsf(v2)) * kStep + 2.0f * act_err;
        // without a bias v is act itself, and both are off by no more than the smaller one's factor: 2 d + 32 steps with
        // d = log(1 / (act S)), or 4 + 1.25 max(0, -s) with -s <= log(1 / act); each may have lost kLost
        if (!A.bias && !A.raw) {
            const float far = -s_lg2(fmaxf(k2, 0x1p-126f));  // log2(1 / act)
            const float steps = A.sigmoid ? 4.0f + 1.25f * kLn2 * far : 32.0f + 2.0f * kLn2 * fmaxf(0.0f, s_lg2(inv_S) + far);
            err += (v1 + v2) * kStep * steps + kLost;
        }
        if (g < A.n_group) {
            if (sum > -INFINITY) worst_err = fmaxf(worst_err, err);  // (a masked group's score is exact)
            if (sub == 0) W.gscore[row][g] = sum;
        }
    }
    worst_err = lanes_max<L>(worst_err);
    wave_sync();
    float in = INFINITY, out = -INFINITY;  // the last score taken, the first left out
    for (int g = l; g < A.n_group; g += L) {
        const float mine = W.gscore[row][g];
        int rank = 0;
        for (int q = 0; q < A.n_group; ++q) {
            const float x = W.gscore[row][q];
            rank += x > mine || (x == mine && q < g) ? 1 : 0;
        }
        if (rank < A.topk_group) {
            taken |= 1ull << g;
            in = fminf(in, mine);
        } else {
            out = fmaxf(out, mine);
        }
    }
    const uint32_t lo = lanes_reduce<L>((uint32_t)taken, OpOr()), hi = lanes_reduce<L>((uint32_t)(taken >> 32), OpOr());
    in = -lanes_max<L>(-in);
    out = lanes_max<L>(out);
    if (A.doubt && A.topk_group < A.n_group && in - out <= 2.0f * worst_err) *close = true;
    wave_sync();
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint32_t j = Rw::col(e, l), g = (j * A.group_magic) >> 20;
        const uint32_t bit = (g < 32 ? lo >> g : hi >> (g - 32)) & 1u;
        key[e] = bit ? key[e] : NAN;
    }
}

// The rows' first `rounds` columns in descending order of their keys, ties by the lower column, into W.won.
template <class Rw, int L, int E, class Key>
__device__ __forceinline__ void choose(RouteWave<L, E>& W, float (&key)[E], int l, int row, int rounds, Key key_at) {
    if constexpr (L >= 16) {
        // The bound is loose when nearly every lane's maximum is wanted, and for two rounds a plain argmax is as short.
        if (rounds > 2 && rounds <= L - L / 4) {
            float best = key[0];
#pragma unroll
            for (int e = 1; e < E; ++e) best = fmaxf(best, key[e]);
            const float t = kth_of_lanes<L, E>(W, best, l, row, rounds);
            if (l == 0) W.count[row] = 0;
            W.list[row][l] = 0;
            W.list[row][l + L] = 0;
            uint32_t mask = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) mask |= key[e] >= t ? 1u << e : 0u;
            wave_sync();
            int at = mask ? atomicAdd(&W.count[row], __popc(mask)) : 0;
            wave_sync();
            const int have = W.count[row];
            if (!__any(have > RouteWave<L, E>::kList)) {
                while (mask) {
                    const int j = Rw::col(__builtin_ctz(mask), l);
                    mask &= mask - 1;
                    W.list[row][at++] = (uint64_t)ordered(key_at(j)) << 32 | (uint32_t)~j;
                }
                wave_sync();
                const uint64_t a = W.list[row][l], b = W.list[row][l + L];
                int ra = 0, rb = 0;
                const int most = (int)lanes_max<64>((uint32_t)have);
                if (most <= L) {
                    for (int c = 0; c < most; ++c) ra += W.list[row][c] > a ? 1 : 0;
                } else {
                    for (int c = 0; c < most; ++c) {
                        const uint64_t x = W.list[row][c];
                        ra += x > a ? 1 : 0;
                        rb += x > b ? 1 : 0;
                    }
                }
                if (a && ra < rounds) W.won[row][ra] = (uint16_t)~(uint32_t)a;
                if (b && rb < rounds) W.won[row][rb] = (uint16_t)~(uint32_t)b;
                wave_sync();
                return;
            }
        }
    }
    for (int r = 0; r < rounds; ++r) {
        float best = key[0];
#pragma unroll
        for (int e = 1; e < E; ++e) best = fmaxf(best, key[e]);
        best = lanes_max<L>(best);
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int e = E - 1; e >= 0; --e) at = key[e] == best ? (uint32_t)Rw::col(e, l) : at;
        at = lanes_min<L>(at);
#pragma unroll
        for (int e = 0; e < E; ++e) key[e] = (uint32_t)Rw::col(e, l) == at ? NAN : key[e];
        if (l == 0) W.won[row][r] = (uint16_t)at;
    }
    wave_sync();
}

// Weights of the lane's entries r = l, l + L, ... of the row's choice `won`; score(j) is the row's score at j.
template <int L, class Score>
__device__ __forceinline__ void store_weights(const RouteArgs& A, const uint16_t* won, int l, int64_t i, bool on, float M,
                                              float inv_S, Score score) {
    float shift = 0.0f, inv = 1.0f;
    if (A.renorm) {
        shift = kNegBig;
        for (int r = l; r < A.k; r += L) shift = fmaxf(shift, act_exponent(A.sigmoid, score(won[r])));
        shift = lanes_max<L>(shift);
        float sum = 0.0f;
        for (int r = l; r < A.k; r += L) sum += act_shifted(A.sigmoid, score(won[r]), shift);
        sum = lanes_sum<L>(sum);
        inv = sum == 0.0f ? 1.0f : 1.0f / sum;  // every chosen score is masked: weights 0
    }
    if (!on) return;
    for (int r = l; r < A.k; r += L) {
        const float x = score(won[r]);
        const float q = A.renorm ? act_shifted(A.sigmoid, x, shift) * inv : A.sigmoid ? sigmoid_of(x) : exp_of(x - M) * inv_S;
        A.weights[i * A.k + r] = A.scale * q;
    }
}

// Four waves per SIMD hide the latency of its short chains (16384 x 256: 13.9 us, 16.3 at the two that the
// compiler's own choice of registers leaves; 8192 x 1024: 20.1 and 23.4).
template <class T, int L, int E, bool V>
__global__ __launch_bounds__(kBlock, 4) void k_route(RouteArgs A) {
    constexpr int kSlots = kBlock / L;
    using Rw = Row<T, L, E, V>;
    using Elem = typename T::type;
    __shared__ RouteWave<L, E> waves[kBlock / 64];
    __shared__ int32_t hist[L * E];
    __shared__ float bias[L * E];
    __shared__ int wave_huge[kBlock / 64];
    const int lane = threadIdx.x & 63, l = threadIdx.x % L, row = lane / L;
    RouteWave<L, E>& W = waves[threadIdx.x / 64];
    if (A.counts) {
        for (int j = threadIdx.x; j < A.m; j += kBlock) {
            if (A.count_here)
                hist[j] = 0;
            else if (blockIdx.x == 0)
                A.counts[j] = 0;  // cleared here for the kernel that counts
        }
    }
    // Whether a finite bias may take its sum with a finite score out of the float32 range (by half its last step, 2^103).
    bool huge = false;
    for (int j = threadIdx.x; j < L * E; j += kBlock) {
        const float b = A.bias && j < A.m ? A.bias[j] : 0.0f;
        bias[j] = b;
        huge = huge || (fabsf(b) >= 0x1p102f && fabsf(b) < INFINITY);
    }
    const bool sums = A.raw && A.bias;
    if (sums) {
        const bool any = __any(huge);
        if (lane == 0) wave_huge[threadIdx.x / 64] = any ? 1 : 0;
    }
    __syncthreads();
    huge = false;
    if (sums) {
#pragma unroll
        for (int w = 0; w < kBlock / 64; ++w) huge = huge || wave_huge[w] != 0;
    }
    const int left = A.n_group > 1 ? A.topk_group * A.group_size : A.m;
    // where values are rounded, one more than k shows whether the last one chosen is apart from the first left out
    const bool check = A.doubt && A.bias;
    const int rounds = check ? min(left, A.k + 1) : A.k;
    for (int64_t i0 = (int64_t)blockIdx.x * kSlots; i0 < A.n; i0 += (int64_t)gridDim.x * kSlots) {
        const int64_t i = i0 + threadIdx.x / L;
        const bool on = i < A.n;
        float s[E];
        Rw::load(static_cast<const Elem*>(A.s) + (on ? i : i0) * A.ld, l, A.m, s);
        // softmax statistics; an empty row keeps S = 0
        float M = kNegBig, inv_S = 1.0f;
        if (!A.sigmoid && (!A.raw || !A.renorm)) {
            float S = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) M = fmaxf(M, s[e]);
            M = lanes_max<L>(M);
#pragma unroll
            for (int e = 0; e < E; ++e) S += exp_of(s[e] - M);
            S = lanes_sum<L>(S);
            inv_S = S == 0.0f ? 1.0f : 1.0f / S;  // act = 0 in an empty row
        }
        auto key_at = [&](int j) {
            return key_of(A.by_score ? W.s[row][j] : choice_value<float>(A, W.s[row][j], bias[j], M, inv_S));
        };
        float key[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = Rw::col(e, l);
            key[e] = j < A.m ? key_of(choice_value<float>(A, s[e], bias[j], M, inv_S)) : NAN;
        }
        bool close = false;
        if (huge) {  // sums that are finite, whatever float32 makes of them, are left to float64
#pragma unroll
            for (int e = 0; e < E; ++e)
                close = close || (fabsf(key[e]) == INFINITY && fabsf(s[e]) < INFINITY && fabsf(bias[Rw::col(e, l)]) < INFINITY);
        }
        const float act_err = act_error(A, inv_S);
        if (A.n_group > 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) W.s[row][Rw::col(e, l)] = key[e];
            wave_sync();
            keep_groups<Rw, L, E>(A, W, key, l, row, act_err, inv_S, &close);
            if (A.by_score) {
#pragma unroll
                for (int e = 0; e < E; ++e) key[e] = key[e] == key[e] ? key_of(s[e]) : NAN;
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) W.s[row][Rw::col(e, l)] = s[e];
        wave_sync();
        choose<Rw, L, E>(W, key, l, row, rounds, key_at);
        if (check) {  // neighbours in the order must be apart, or equal in score and bias: then the column decides
            auto tie = [&](int p, int q) { return W.s[row][p] == W.s[row][q] && bias[p] == bias[q]; };
            auto error = [&](int j, float v) { return choice_error(A, W.s[row][j], v, M, inv_S); };
            for (int r = l; r + 1 < A.k; r += L) {
                const int j0 = W.won[row][r], j1 = W.won[row][r + 1];
                const float v0 = key_at(j0), v1 = key_at(j1);
                if (v0 - v1 <= error(j0, v0) + error(j1, v1) && !tie(j0, j1)) close = true;
            }
            if (rounds > A.k) {
                // the first column left out stands for all others, whose act may be larger; where it ties with the last
                // one chosen, the largest that does not
                const int j0 = W.won[row][A.k - 1], j1 = W.won[row][A.k];
                const float v0 = key_at(j0);
                float below = key_at(j1);
                const bool tied = tie(j0, j1);
                if (__any(tied)) {
                    float other = -INFINITY;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int j = Rw::col(e, l);
                        if (j < A.m && key[e] <= v0 && !tie(j0, j)) other = fmaxf(other, key[e]);
                    }
                    other = lanes_max<L>(other);
                    below = tied ? other : below;
                }
                if (v0 - below <= error(j0, v0) + (below > -INFINITY ? fabsf(below) * kStep + act_err : 0.0f)) close = true;
            }
        }
        const bool marked = lanes_max<L>(close ? 1u : 0u) != 0;
        for (int r = l; on && r < A.k; r += L) {
            const int j = W.won[row][r];
            A.idx[i * A.k + r] = marked && r == 0 ? ~j : j;
            if (A.count_here) atomicAdd(&hist[j], 1);
        }
        store_weights<L>(A, W.won[row], l, i, on, M, inv_S, [&](int j) { return W.s[row][j]; });
        wave_sync();
    }
    if (A.count_here) {
        __syncthreads();
        for (int j = threadIdx.x; j < A.m; j += kBlock) A.counts[j] = hist[j];
    }
}

// After k_route: chooses the marked rows in float64 and counts the rows per expert into cleared counts (whole numbers,
// so the order does not matter).  A workgroup takes kFinishRows rows at a time.
template <class T>
__global__ __launch_bounds__(kBlock) void k_route_finish(RouteArgs A) {
    constexpr int kWaves = kBlock / 64;
    __shared__ unsigned long long key[kRouteMaxCols], first[kRouteMaxGroups], second[kRouteMaxGroups];
    __shared__ int owner[kRouteMaxGroups];
    __shared__ double red[kWaves];
    __shared__ uint32_t lane_top[kWaves][64];
    __shared__ uint16_t list[kRouteMaxCols];
    __shared__ int have;
    __shared__ uint16_t won[kRouteMaxTop];
    __shared__ int32_t hist[kRouteMaxCols];
    __shared__ uint8_t todo[kFinishRows];
    __shared__ int many;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    // One row by the whole workgroup: values, ranks by counting, weights.
    auto exact = [&](int64_t i) {
        const typename T::type* s = static_cast<const typename T::type*>(A.s) + i * A.ld;
        float M = kNegBig, S1 = 1.0f;
        double inv_S = 1.0;
        if (!A.sigmoid) {
            for (int j = lane; j < A.m; j += 64) M = fmaxf(M, T::to(s[j]));
            M = lanes_max<64>(M);
            double S = 0.0;
            for (int j = tid; j < A.m; j += kBlock) S += exp((double)T::to(s[j]) - (double)M);
            S = lanes_sum<64>(S);
            if (lane == 0) red[wave] = S;
            __syncthreads();
            S = 0.0;
            for (int w = 0; w < kWaves; ++w) S += red[w];
            if (S != 0.0) inv_S = 1.0 / S, S1 = (float)S;
        }
        for (int j = tid; j < A.m; j += kBlock)
            key[j] = ordered(choice_value<double>(A, T::to(s[j]), A.bias ? A.bias[j] : 0.0f, M, inv_S));
        __syncthreads();
        if (A.n_group > 1) {
            // the groups' two largest keys; of equal largest ones the lowest column is the first
            for (int g = tid; g < A.n_group; g += kBlock) first[g] = second[g] = 0, owner[g] = INT_MAX;
            __syncthreads();
            for (int j = tid; j < A.m; j += kBlock) atomicMax(&first[j / A.group_size], key[j]);
            __syncthreads();
            if (A.group_top == 2) {
                for (int j = tid; j < A.m; j += kBlock)
                    if (key[j] == first[j / A.group_size]) atomicMin(&owner[j / A.group_size], j);
                __syncthreads();
                for (int j = tid; j < A.m; j += kBlock)
                    if (owner[j / A.group_size] != j) atomicMax(&second[j / A.group_size], key[j]);
                __syncthreads();
                for (int g = tid; g < A.n_group; g += kBlock) first[g] = ordered(unordered((uint64_t)first[g]) + unordered((uint64_t)second[g]));
                __syncthreads();
            }
            for (int j = tid; j < A.m; j += kBlock) {
                const int g = j / A.group_size;
                int rank = 0;
                for (int q = 0; q < A.n_group; ++q) rank += first[q] > first[g] || (first[q] == first[g] && q < g) ? 1 : 0;
                if (rank >= A.topk_group)
                    key[j] = 0;
                else if (A.by_score)
                    key[j] = ordered((double)T::to(s[j]));
            }
        }
        // the k-th largest of 64 classes' maxima (upper halves of the keys) bounds the k-th largest key from below
        uint32_t top = 0;
        for (int j = tid; j < A.m; j += kBlock) top = max(top, (uint32_t)(key[j] >> 32));
        lane_top[wave][lane] = top;
        if (tid == 0) have = 0;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) top = max(top, lane_top[w][lane]);
        const uint32_t lane_best[1] = {top};
        top = max(kth_of_wave<0>(lane_best, A.k), 1u);
        for (int j = tid; j < A.m; j += kBlock)
            if ((uint32_t)(key[j] >> 32) >= top) list[atomicAdd(&have, 1)] = (uint16_t)j;
        __syncthreads();
        const int count = have;
        for (int c = tid; c < count; c += kBlock) {
            const int j = list[c];
            const uint64_t mine = key[j];
            int rank = 0;
#pragma unroll 8
            for (int q = 0; q < count; ++q) {
                const int jq = list[q];
                const uint64_t x = key[jq];
                rank += (x > mine ? 1 : 0) + (((x == mine) & (jq < j)) ? 1 : 0);
            }
            if (rank < A.k) {
                won[rank] = (uint16_t)j;
                A.idx[i * A.k + rank] = j;
            }
        }
        __syncthreads();
        if (wave == 0) store_weights<64>(A, won, lane, i, true, M, 1.0f / S1, [&](int j) { return T::to(s[j]); });
        __syncthreads();
    };
    if (A.counts)
        for (int j = tid; j < A.m; j += kBlock) hist[j] = 0;
    for (int64_t i0 = (int64_t)blockIdx.x * kFinishRows; i0 < A.n; i0 += (int64_t)gridDim.x * kFinishRows) {
        if (A.doubt) {
            if (tid == 0) many = 0;
            __syncthreads();
            const int64_t i = i0 + tid;
            if (tid < kFinishRows && i < A.n && A.idx[i * A.k] < 0) todo[atomicAdd(&many, 1)] = (uint8_t)tid;
            __syncthreads();
            for (int q = 0; q < many; ++q) exact(i0 + todo[q]);
        }
        __syncthreads();
        if (A.counts) {
            const int64_t end = min((int64_t)A.n, i0 + kFinishRows) * A.k;
            for (int64_t q = i0 * A.k + tid; q < end; q += kBlock) atomicAdd(&hist[A.idx[q]], 1);
        }
        __syncthreads();
    }
    if (A.counts)
        for (int j = tid; j < A.m; j += kBlock)
            if (hist[j]) atomicAdd(&A.counts[j], hist[j]);
}

struct RouteGradArgs {
    const void* s;
    int64_t ld, ldg;
    int n, m, sigmoid, k, renorm;
    float scale;
    const int32_t* idx;
    const float* dw;
    void* grad;
};

// With q = weight / scale and dq = scale d_weight, inner = sum q dq over the row's choice:
//   softmax: ds_j = p_j (dq_j - inner); renormalised, p is the softmax over the choice alone (zero elsewhere);
//   sigmoid: ds_j = dq_j q_j (1 - sigmoid(s_j)); renormalised q_j (dq_j - inner)(1 - sigmoid(s_j)).
// The row is put together in LDS (dense term, then the choice's terms) and stored once.
template <class T, int L, int E, bool V>
__global__ __launch_bounds__(kBlock) void k_route_grad(RouteGradArgs A) {
    constexpr int kSlots = kBlock / L;
    using Rw = Row<T, L, E, V>;
    using Elem = typename T::type;
    __shared__ float term[kSlots][kRouteMaxTop];
    __shared__ int16_t place[kSlots][kRouteMaxTop];
    __shared__ float tile[kSlots][L * E];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const bool dense = !A.sigmoid && !A.renorm;
    for (int64_t i0 = (int64_t)blockIdx.x * kSlots; i0 < A.n; i0 += (int64_t)gridDim.x * kSlots) {
        const int64_t i = i0 + slot < A.n ? i0 + slot : i0;
        const bool on = i0 + slot < A.n;
        const Elem* row = static_cast<const Elem*>(A.s) + i * A.ld;
        const int32_t* idx = A.idx + i * A.k;
        const float* dw = A.dw + i * A.k;
        // the choice: column (an entry outside the row was dropped: -1), score and gradient; the lane's first in registers
        auto column = [&](int r) {
            const int j = idx[r];
            return (unsigned)j < (unsigned)A.m ? j : -1;
        };
        const int j0 = l < A.k ? column(l) : -1;
        const float x0 = j0 >= 0 ? T::to(row[j0]) : -INFINITY, d0 = j0 >= 0 ? dw[l] : 0.0f;
        auto each = [&](auto f) {
            if (l < A.k) f(l, j0, x0, d0);
            for (int r = l + L; r < A.k; r += L) {
                const int j = column(r);
                f(r, j, j >= 0 ? T::to(row[j]) : -INFINITY, dw[r]);
            }
        };
        float p[E], M = kNegBig, inv_S = 1.0f;
        if (dense) {
            Rw::load(row, l, A.m, p);
            float S = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) M = fmaxf(M, p[e]);
            M = lanes_max<L>(M);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                p[e] = exp_of(p[e] - M);
                S += p[e];
            }
            S = lanes_sum<L>(S);
            inv_S = S == 0.0f ? 1.0f : 1.0f / S;
        }
        float shift = kNegBig, inv = 1.0f;
        if (A.renorm) {
            each([&](int, int, float x, float) { shift = fmaxf(shift, act_exponent(A.sigmoid, x)); });
            shift = lanes_max<L>(shift);
            float sum = 0.0f;
            each([&](int, int, float x, float) { sum += act_shifted(A.sigmoid, x, shift); });
            sum = lanes_sum<L>(sum);
            inv = sum == 0.0f ? 1.0f : 1.0f / sum;
        }
        auto weight = [&](float x) {  // q; 0 for a dropped entry (x = -inf)
            return A.renorm ? act_shifted(A.sigmoid, x, shift) * inv : A.sigmoid ? sigmoid_of(x) : exp_of(x - M) * inv_S;
        };
        float inner = 0.0f;
        each([&](int r, int j, float x, float d) {
            const float qd = j >= 0 ? weight(x) * (A.scale * d) : 0.0f;
            place[slot][r] = (int16_t)j;
            term[slot][r] = qd;
            inner += qd;
        });
        inner = lanes_sum<L>(inner);
        const float all = dense ? -inv_S * inner : 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) tile[slot][Rw::col(e, l)] = dense ? p[e] * all : 0.0f;
        wave_sync();
        each([&](int r, int j, float x, float) {
            if (j < 0) return;
            // an expert that stands twice in the row: its first entry takes the sum of all
            float total = 0.0f;
            int copies = 0;
            bool first = true;
            for (int u = 0; u < A.k; ++u) {
                if (place[slot][u] != j) continue;
                if (u < r) first = false;
                total += term[slot][u];
                ++copies;
            }
            if (!first) return;
            if (A.renorm) total -= (float)copies * weight(x) * inner;
            if (A.sigmoid) total *= sigmoid_of(-x);
            tile[slot][j] += total;
        });
        wave_sync();
        if (on) {
            float out[E];
#pragma unroll
            for (int e = 0; e < E; ++e) out[e] = tile[slot][Rw::col(e, l)];
            Rw::store(static_cast<Elem*>(A.grad) + i * A.ldg, l, A.m, out);
        }
        wave_sync();
    }
}

// f(lanes per row, scores per lane) for rows of m scores.  8 scores per lane up to 128 columns: with half the lanes and
// 16 scores each, 32768 x 64 f32, k = 6 takes 14.0 us and one row 7.2, against 13.6 and 5.7 so; 32768 x 128 bf16, k = 8
// takes 17.7 and one row 7.4, against 18.7 and 5.7.  256 columns take 16 x 16 (14 us; 32 x 8 takes 27).  For 257 to 512
// columns 64 x 8 is the shorter for one row (6.2 us; 32 x 16: 6.6) and the longer for many: 16384 x 512 f32, k = 8
// takes 27 us, 21 with 32 x 16.
template <class F>
void by_width(int m, F f) {
    using std::integral_constant;
    if (m <= 8)
        f(integral_constant<int, 4>(), integral_constant<int, 2>());
    else if (m <= 16)
        f(integral_constant<int, 4>(), integral_constant<int, 4>());
    else if (m <= 32)
        f(integral_constant<int, 4>(), integral_constant<int, 8>());
    else if (m <= 64)
        f(integral_constant<int, 8>(), integral_constant<int, 8>());
    else if (m <= 128)
        f(integral_constant<int, 16>(), integral_constant<int, 8>());
    else if (m <= 256)
        f(integral_constant<int, 16>(), integral_constant<int, 16>());
    else if (m <= 512)
        f(integral_constant<int, 64>(), integral_constant<int, 8>());
    else
        f(integral_constant<int, 64>(), integral_constant<int, 16>());
}

unsigned route_grid(int64_t n, int lanes) {
    const int slots = kBlock / lanes;
    return (unsigned)std::min<int64_t>((n + slots - 1) / slots, kRouteGroupsOfGrid);
}

template <class T>
hipError_t launch_route(RouteArgs A, hipStream_t s) {
    by_width(A.m, [&](auto lanes, auto per_lane) {
        constexpr int L = decltype(lanes)::value, E = decltype(per_lane)::value;
        const unsigned grid = route_grid(A.n, L);
        A.count_here = A.counts && grid == 1 && !A.doubt;
        auto kernel = Row<T, L, E, true>::fits(A.s, A.ld, A.m) ? k_route<T, L, E, true> : k_route<T, L, E, false>;
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(kBlock), 0, s, A);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(A.doubt || (A.counts && !A.count_here))) return e;
    const int64_t grid = std::min<int64_t>(((int64_t)A.n + kFinishRows - 1) / kFinishRows, kFinishGroups);
    hipLaunchKernelGGL((k_route_finish<T>), dim3((unsigned)grid), dim3(kBlock), 0, s, A);
    return hipGetLastError();
}

template <class T>
hipError_t launch_route_grad(const RouteGradArgs& A, hipStream_t s) {
    by_width(A.m, [&](auto lanes, auto per_lane) {
        constexpr int L = decltype(lanes)::value, E = decltype(per_lane)::value;
        const bool runs = Row<T, L, E, true>::fits(A.s, A.ld, A.m) && Row<T, L, E, true>::fits(A.grad, A.ldg, A.m);
        auto kernel = runs ? k_route_grad<T, L, E, true> : k_route_grad<T, L, E, false>;
        hipLaunchKernelGGL(kernel, dim3(route_grid(A.n, L)), dim3(kBlock), 0, s, A);
    });
    return hipGetLastError();
}

__global__ __launch_bounds__(kBlock) void k_clear_counts(int32_t* counts, int m) {
    const int j = blockIdx.x * kBlock + threadIdx.x;
    if (j < m) counts[j] = 0;
}

}  // namespace
}  // namespace sk

using namespace sk;

extern "C" {

int sk_scores_route(const void* scores, int32_t dtype, int64_t n, int64_t m, int64_t ld, int32_t score_fn,
                    const float* bias, int32_t select_on, int32_t n_group, int32_t topk_group, int32_t group_top,
                    int32_t k, int32_t renorm, float scale, int32_t* idx, float* weights, int32_t* counts,
                    void* stream) {
    int st = check_scores(scores, dtype, n, m, ld);
    if (st) return st;
    if (m > kRouteMaxCols) return SK_ERR_SHAPE;
    if (score_fn < 0 || score_fn > 1 || select_on < 0 || select_on > 1 || renorm < 0 || renorm > 1 ||
        !std::isfinite(scale))
        return SK_ERR_ROUTE;
    if (n_group < 1 || n_group > kRouteMaxGroups || m % n_group != 0 || topk_group < 1 || topk_group > n_group)
        return SK_ERR_ROUTE;
    if (group_top < 1 || group_top > 2 || group_top > m / n_group) return SK_ERR_ROUTE;
    if (k < 1 || k > kRouteMaxTop || k > topk_group * (m / n_group)) return SK_ERR_ROUTE;
    if (n > 0 && (!idx || !weights)) return SK_ERR_NULL;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    RouteArgs A{};
    A.s = scores;
    A.ld = ld;
    A.n = (int)n;
    A.m = (int)m;
    A.sigmoid = score_fn == 1;
    A.bias = bias;
    A.n_group = n_group;
    A.topk_group = topk_group;
    A.group_top = group_top;
    A.group_size = (int)(m / n_group);
    A.group_magic = (uint32_t)(((1u << 20) + A.group_size - 1) / A.group_size);
    // act rises with the score: without a bias and without sums of it, the scores decide, exactly
    A.raw = select_on == 1 || (!bias && (n_group == 1 || group_top == 1));
    A.by_score = !A.raw && !bias;
    A.doubt = bias || !A.raw || (n_group > 1 && topk_group < n_group && group_top == 2);
    A.k = k;
    A.renorm = renorm;
    A.scale = scale;
    A.idx = idx;
    A.weights = weights;
    A.counts = counts;
    if (n == 0) {
        if (!counts) return SK_OK;
        hipLaunchKernelGGL(k_clear_counts, dim3((unsigned)((m + kBlock - 1) / kBlock)), dim3(kBlock), 0, s, counts, (int)m);
        SK_TRY_LAUNCH(hipGetLastError());
        return SK_OK;
    }
    SK_TRY_LAUNCH(dtype == SK_F32    ? launch_route<F32>(A, s)
                  : dtype == SK_BF16 ? launch_route<Bf16>(A, s)
                                     : launch_route<F16>(A, s));
    return SK_OK;
}

int sk_scores_route_grad(const void* scores, int32_t dtype, int64_t n, int64_t m, int64_t ld, int32_t score_fn,
                         const int32_t* idx, const float* d_weights, int32_t k, int32_t renorm, float scale, void* grad,
                         int64_t ld_grad, void* stream) {
    int st = check_scores(scores, dtype, n, m, ld);
    if (st) return st;
    if (m > kRouteMaxCols) return SK_ERR_SHAPE;
    if (score_fn < 0 || score_fn > 1 || renorm < 0 || renorm > 1 || !std::isfinite(scale)) return SK_ERR_ROUTE;
    if (k < 1 || k > kRouteMaxTop || k > m) return SK_ERR_ROUTE;
    if (n > 0 && (!idx || !d_weights)) return SK_ERR_NULL;
    if ((st = check_grad(scores, ld, grad, ld_grad, dtype, n, m))) return st;
    if (n == 0) return SK_OK;
    RouteGradArgs A{scores, ld, ld_grad, (int)n, (int)m, score_fn == 1, k, renorm, scale, idx, d_weights, grad};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SK_TRY_LAUNCH(dtype == SK_F32    ? launch_route_grad<F32>(A, s)
                  : dtype == SK_BF16 ? launch_route_grad<Bf16>(A, s)
                                     : launch_route_grad<F16>(A, s));
    return SK_OK;
}

}  // extern "C"
