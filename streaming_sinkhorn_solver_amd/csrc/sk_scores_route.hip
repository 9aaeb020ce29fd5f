// sk_scores_route.hip -- routing of tokens to experts from a given score
// matrix (sk_scores_route) and its gradient (sk_scores_route_grad).
//
// act_ij is softmax_j(s_i.) or sigmoid(s_ij); the experts of row i are the k
// largest v_ij = (act_ij or s_ij) + bias_j, inside the topk_group best of
// n_group equal groups of columns when there are groups (a group's score is
// the sum of its group_top largest v); ties go to the lowest index.  The
// weights come from act at the chosen experts, without the bias.
//
// One row per L lanes with E scores each (column e L + l), in registers; k
// rounds of an argmax over ordered 32-bit keys, each a scan of the lane's keys
// and four or six cross-lane steps.  The rounds are what the kernel spends
// its time on, not the n m scores it reads.
//
// The order of two values that are closer than the float32 rounding of act or
// of the sum with the bias would depend on that rounding.  Rows where a pair
// that decides the result is that close are chosen again with everything in
// float64, so the result is that of the definition.
#include "sk_scores.hpp"

#include <algorithm>

namespace sk {
namespace {

constexpr int kRouteMaxCols = 1024;
constexpr int kRouteMaxTop = 64;
constexpr int kRouteMaxGroups = 64;
constexpr int kRouteGroupsOfGrid = 2048;  // workgroups: eight per CU

struct RouteArgs {
    const void* s;
    int64_t ld;
    int n, m;
    int sigmoid;       // act: 0 softmax, 1 sigmoid
    const float* bias; // null: none
    int raw;           // v from the raw score (also where act alone decides: act keeps the scores' order)
    int n_group, topk_group, group_top, group_size;
    uint32_t group_magic;  // ceil(2^20 / group_size): (j * magic) >> 20 = j / group_size for j < 1024
    int k, renorm;
    float scale;
    int32_t* idx;
    float* weights;
    int32_t* counts;   // null: not wanted
    int fill;          // counts were cleared before: add to them (else store)
};

__device__ __forceinline__ float sigmoid_of(float x) { return 1.0f / (1.0f + s_ex2(-kLog2e * x)); }
__device__ __forceinline__ double sigmoid_of(double x) { return 1.0 / (1.0 + exp(-x)); }
__device__ __forceinline__ float exp_of(float x) { return s_ex2(kLog2e * x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
// log sigmoid(x), accurate where sigmoid itself leaves the float32 range
__device__ __forceinline__ float log_sigmoid(float x) { return fminf(x, 0.0f) - log1pf(exp_of(-fabsf(x))); }

template <class R>
struct KeyOf;
template <>
struct KeyOf<float> {
    using type = uint32_t;
};
template <>
struct KeyOf<double> {
    using type = uint64_t;
};

template <int L>
__device__ __forceinline__ uint32_t key_max(uint32_t k) {
    return lanes_max<L>(k);
}
template <int L>
__device__ __forceinline__ uint64_t key_max(uint64_t k) {
    const uint32_t hi = lanes_max<L>((uint32_t)(k >> 32));
    const uint32_t lo = lanes_max<L>((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The value that decides the choice, from the row's maximum M and sum S of
// exponentials.  The same expression in float32 and float64.
template <class R>
__device__ __forceinline__ R choice_value(const RouteArgs& A, float s, float bias, float M, R S) {
    R v = (R)s;
    if (!A.raw) v = A.sigmoid ? sigmoid_of((R)s) : exp_of((R)s - (R)M) / S;
    return A.bias ? v + (R)bias : v;
}

// How far the float32 choice_value may be off, in steps of 2^-23.  The
// exponential's argument d log2e carries three half-step roundings of |d| at
// most, relative to act in the result; the exponentials, the sum of at most
// 16 + 6 terms in turn, and the division add less than 30 half steps of act; the
// sum with the bias adds half a step of v.
__device__ __forceinline__ float choice_error(const RouteArgs& A, float s, float v, float M, float S) {
    const float step = 0x1p-23f;
    float err = A.bias ? fabsf(v) * step : 0.0f;
    if (!A.raw) {
        const float d = A.sigmoid ? fabsf(s) : M - s;
        const float act = A.sigmoid ? sigmoid_of(s) : exp_of(s - M) / S;
        err += act * (2.0f * d + 32.0f) * step;
    }
    return err;
}

struct RouteLds {
    uint16_t* won;    // [kRouteMaxTop + 1] this row's choice, in order
    void* tile;       // [m] keys of the row (groups only)
    // of the n_group groups: keys of their scores, the scores and their float32 errors by rank, chosen or not
    uint64_t* gkey;
    float *gscore, *gerr;
    uint8_t* gsel;
};

// Chooses the row's k experts (and, where one is left, the next after them)
// into lds.won.  Returns the number of entries written; sets close when two
// groups that decide were within their float32 error.
template <class R, int L, int E>
__device__ __forceinline__ int choose(const RouteArgs& A, const float (&s)[E], const float (&bias)[E], int l, float M,
                                      R S, const RouteLds& lds, bool* close) {
    using K = typename KeyOf<R>::type;
    K key[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int j = e * L + l;
        key[e] = j < A.m ? ordered(choice_value<R>(A, s[e], bias[e], M, S)) : (K)0;
    }
    int left = A.m;
    if (A.n_group > 1) {
        K* tile = static_cast<K*>(lds.tile);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e * L + l < A.m) tile[e * L + l] = key[e];
        wave_sync();
        float err[kRouteMaxGroups / L];
#pragma unroll
        for (int gl = 0; gl < kRouteMaxGroups / L; ++gl) {
            const int g = gl * L + l;
            if (g >= A.n_group) break;
            K k1 = 0, k2 = 0;
            for (int q = 0; q < A.group_size; ++q) {
                const K x = tile[g * A.group_size + q];
                k2 = x > k1 ? k1 : (x > k2 ? x : k2);
                k1 = x > k1 ? x : k1;
            }
            const R v1 = unordered(k1), v2 = A.group_top == 2 ? unordered(k2) : (R)0;
            lds.gkey[g] = (uint64_t)ordered(v1 + v2);
            // choice_error of both values and the sum's rounding.  act (2 d + 32) is at most 33 where a bias
            // hides act, and at most 2^8 v where it does not (d <= 104, or act is zero)
            const float size = fabsf((float)v1) + fabsf((float)v2);
            err[gl] = size * 0x1p-22f + (A.raw ? 0.0f : A.bias ? 0x1p-16f : size * 0x1p-15f);
        }
        wave_sync();
#pragma unroll
        for (int gl = 0; gl < kRouteMaxGroups / L; ++gl) {
            const int g = gl * L + l;
            if (g >= A.n_group) break;
            const uint64_t mine = lds.gkey[g];
            int rank = 0;
            for (int q = 0; q < A.n_group; ++q) {
                const uint64_t x = lds.gkey[q];
                rank += x > mine || (x == mine && q < g) ? 1 : 0;
            }
            lds.gsel[g] = rank < A.topk_group;
            lds.gscore[rank] = (float)unordered((K)mine);
            lds.gerr[rank] = err[gl];
        }
        wave_sync();
        if (A.topk_group < A.n_group) {
            const float in = lds.gscore[A.topk_group - 1], out = lds.gscore[A.topk_group];
            const float tol = lds.gerr[A.topk_group - 1] + lds.gerr[A.topk_group];
            if (in - out <= tol && (A.bias || !A.raw || A.group_top == 2)) *close = true;
        }
        left = A.topk_group * A.group_size;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t j = e * L + l;
            if ((int)j < A.m && !lds.gsel[(j * A.group_magic) >> 20]) key[e] = 0;
        }
    }
    const int rounds = left > A.k ? A.k + 1 : A.k;
    for (int r = 0; r < rounds; ++r) {
        K best = key[0];
#pragma unroll
        for (int e = 1; e < E; ++e) best = key[e] > best ? key[e] : best;
        best = key_max<L>(best);
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int e = E - 1; e >= 0; --e) at = key[e] == best ? (uint32_t)(e * L + l) : at;
        at = lanes_min<L>(at);
#pragma unroll
        for (int e = 0; e < E; ++e) key[e] = (uint32_t)(e * L + l) == at ? (K)0 : key[e];
        if (l == 0) lds.won[r] = (uint16_t)at;
    }
    wave_sync();
    return rounds;
}

template <class T, int L, int E>
__global__ __launch_bounds__(kBlock) void k_route(RouteArgs A) {
    constexpr int kSlots = kBlock / L;
    extern __shared__ uint64_t dyn[];
    __shared__ uint16_t won[kSlots][kRouteMaxTop + 2];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    // dynamic: counts [m], then, with groups, per row slot the keys [m] and the groups' keys, scores and flags
    int32_t* hist = reinterpret_cast<int32_t*>(dyn);
    char* p = reinterpret_cast<char*>(dyn) + (A.counts ? ((size_t)A.m * 4 + 7) / 8 * 8 : 0);
    RouteLds lds{won[slot], nullptr, nullptr, nullptr, nullptr, nullptr};
    if (A.n_group > 1) {
        const size_t row = (size_t)A.m * 8 + (size_t)A.n_group * 24;
        char* q = p + (size_t)slot * row;
        lds.tile = q;
        lds.gkey = reinterpret_cast<uint64_t*>(q + (size_t)A.m * 8);
        lds.gscore = reinterpret_cast<float*>(lds.gkey + A.n_group);
        lds.gerr = lds.gscore + A.n_group;
        lds.gsel = reinterpret_cast<uint8_t*>(lds.gerr + A.n_group);
    }
    if (A.counts) {
        for (int j = threadIdx.x; j < A.m; j += kBlock) hist[j] = 0;
        __syncthreads();
    }
    float bias[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int j = e * L + l;
        bias[e] = A.bias && j < A.m ? A.bias[j] : 0.0f;
    }
    for (int64_t i0 = (int64_t)blockIdx.x * kSlots; i0 < A.n; i0 += (int64_t)gridDim.x * kSlots) {
        const int64_t i = i0 + slot;
        const bool on = i < A.n;
        const typename T::type* row = static_cast<const typename T::type*>(A.s) + (on ? i : i0) * A.ld;
        float s[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = e * L + l;
            s[e] = T::to(row[j < A.m ? j : A.m - 1]);
            if (j >= A.m) s[e] = -INFINITY;
        }
        // softmax statistics; an empty row keeps S = 0
        float M = kNegBig, S = 0.0f;
        if (!A.sigmoid) {
#pragma unroll
            for (int e = 0; e < E; ++e) M = fmaxf(M, s[e]);
            M = lanes_max<L>(M);
#pragma unroll
            for (int e = 0; e < E; ++e) S += exp_of(s[e] - M);
            S = lanes_sum<L>(S);
        }
        const float S1 = S == 0.0f ? 1.0f : S;  // act = 0 in an empty row
        bool close = false;
        int rounds = choose<float, L, E>(A, s, bias, l, M, S1, lds, &close);
        if (A.bias || !A.raw) {  // values that were rounded: neighbours in the order must be apart
            for (int r = l; r + 1 < rounds; r += L) {
                const int j0 = lds.won[r], j1 = lds.won[r + 1];
                const float s0 = T::to(row[j0]), s1 = T::to(row[j1]);
                const float v0 = choice_value<float>(A, s0, A.bias ? A.bias[j0] : 0.0f, M, S1);
                const float v1 = choice_value<float>(A, s1, A.bias ? A.bias[j1] : 0.0f, M, S1);
                const float tol = choice_error(A, s0, v0, M, S1) + choice_error(A, s1, v1, M, S1);
                if (v0 - v1 <= tol) close = true;
            }
        }
        if (__any(close)) {
            double S2 = 0.0;
            if (!A.sigmoid) {
#pragma unroll
                for (int e = 0; e < E; ++e) S2 += exp((double)s[e] - (double)M);
                S2 = lanes_sum<L>(S2);
                if (S2 == 0.0) S2 = 1.0;
            }
            wave_sync();
            bool ignored = false;
            choose<double, L, E>(A, s, bias, l, M, S2, lds, &ignored);
        }
        // weights of the chosen: q = act, or act over its sum taken relative to the largest
        float top = kNegBig, sum = 0.0f;
        if (A.renorm) {
            for (int r = l; r < A.k; r += L) {
                const float x = T::to(row[lds.won[r]]);
                top = fmaxf(top, A.sigmoid ? log_sigmoid(x) : x);
            }
            top = lanes_max<L>(top);
            for (int r = l; r < A.k; r += L) {
                const float x = T::to(row[lds.won[r]]);
                sum += exp_of((A.sigmoid ? log_sigmoid(x) : x) - top);
            }
            sum = lanes_sum<L>(sum);
            if (sum == 0.0f) sum = 1.0f;  // every chosen score is masked: weights 0
        }
        if (on) {
            for (int r = l; r < A.k; r += L) {
                const int j = lds.won[r];
                const float x = T::to(row[j]);
                float q;
                if (A.renorm)
                    q = exp_of((A.sigmoid ? log_sigmoid(x) : x) - top) / sum;
                else
                    q = A.sigmoid ? sigmoid_of(x) : exp_of(x - M) / S1;
                A.idx[i * A.k + r] = j;
                A.weights[i * A.k + r] = A.scale * q;
                if (A.counts) atomicAdd(&hist[j], 1);
            }
        }
        wave_sync();
    }
    if (A.counts) {
        __syncthreads();
        for (int j = threadIdx.x; j < A.m; j += kBlock) {
            if (!A.fill)
                A.counts[j] = hist[j];
            else if (hist[j])
                atomicAdd(&A.counts[j], hist[j]);  // whole numbers: the order does not matter
        }
    }
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
template <class T, int L, int E>
__global__ __launch_bounds__(kBlock) void k_route_grad(RouteGradArgs A) {
    constexpr int kSlots = kBlock / L;
    __shared__ float term[kSlots][kRouteMaxTop];
    __shared__ int place[kSlots][kRouteMaxTop];
    __shared__ float tile[kSlots][L * E];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const bool dense = !A.sigmoid && !A.renorm;
    for (int64_t i0 = (int64_t)blockIdx.x * kSlots; i0 < A.n; i0 += (int64_t)gridDim.x * kSlots) {
        const int64_t i = i0 + slot < A.n ? i0 + slot : i0;
        const bool on = i0 + slot < A.n;
        const typename T::type* row = static_cast<const typename T::type*>(A.s) + i * A.ld;
        const int32_t* idx = A.idx + i * A.k;
        const float* dw = A.dw + i * A.k;
        float s[E], M = kNegBig, S = 0.0f;
        if (dense) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j = e * L + l;
                s[e] = T::to(row[j < A.m ? j : A.m - 1]);
                if (j >= A.m) s[e] = -INFINITY;
                M = fmaxf(M, s[e]);
            }
            M = lanes_max<L>(M);
#pragma unroll
            for (int e = 0; e < E; ++e) S += exp_of(s[e] - M);
            S = lanes_sum<L>(S);
            if (S == 0.0f) S = 1.0f;
        }
        float top = kNegBig, sum = 0.0f, inner = 0.0f;
        if (A.renorm) {
            for (int r = l; r < A.k; r += L) {
                const int j = idx[r];
                if ((unsigned)j >= (unsigned)A.m) continue;
                const float x = T::to(row[j]);
                top = fmaxf(top, A.sigmoid ? log_sigmoid(x) : x);
            }
            top = lanes_max<L>(top);
            for (int r = l; r < A.k; r += L) {
                const int j = idx[r];
                if ((unsigned)j >= (unsigned)A.m) continue;
                const float x = T::to(row[j]);
                sum += exp_of((A.sigmoid ? log_sigmoid(x) : x) - top);
            }
            sum = lanes_sum<L>(sum);
            if (sum == 0.0f) sum = 1.0f;
        }
        for (int r = l; r < A.k; r += L) {
            const int j = idx[r];
            const bool in = (unsigned)j < (unsigned)A.m;  // an entry outside the row was dropped: no part
            const float x = in ? T::to(row[j]) : -INFINITY;
            float q = 0.0f;
            if (in) {
                if (A.renorm)
                    q = exp_of((A.sigmoid ? log_sigmoid(x) : x) - top) / sum;
                else
                    q = A.sigmoid ? sigmoid_of(x) : exp_of(x - M) / S;
            }
            const float qd = in ? q * (A.scale * dw[r]) : 0.0f;
            place[slot][r] = in ? j : -1;
            term[slot][r] = qd;
            inner += qd;
        }
        inner = lanes_sum<L>(inner);
        wave_sync();
#pragma unroll
        for (int e = 0; e < E; ++e) tile[slot][e * L + l] = dense ? -(exp_of(s[e] - M) / S) * inner : 0.0f;
        wave_sync();
        for (int r = l; r < A.k; r += L) {
            const int j = place[slot][r];
            if (j < 0) continue;
            // an expert that stands twice in the row: its first entry takes the sum of all
            float total = 0.0f;
            bool first = true;
            for (int u = 0; u < A.k; ++u) {
                if (place[slot][u] != j) continue;
                if (u < r) first = false;
                total += term[slot][u];
            }
            if (!first) continue;
            const float x = T::to(row[j]);
            if (A.renorm) {
                int copies = 0;
                for (int u = 0; u < A.k; ++u) copies += place[slot][u] == j ? 1 : 0;
                const float q = exp_of((A.sigmoid ? log_sigmoid(x) : x) - top) / sum;
                total -= (float)copies * q * inner;
            }
            if (A.sigmoid) total *= sigmoid_of(-x);
            tile[slot][j] += total;
        }
        wave_sync();
        if (on) {
            typename T::type* out = static_cast<typename T::type*>(A.grad) + i * A.ldg;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j = e * L + l;
                if (j < A.m) out[j] = T::from(tile[slot][j]);
            }
        }
        wave_sync();
    }
}

template <class F>
void by_width(int m, F f) {
    if (m <= 8)
        f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    else if (m <= 16)
        f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    else if (m <= 32)
        f(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
    else if (m <= 64)
        f(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
    else if (m <= 128)
        f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
    else if (m <= 256)
        f(std::integral_constant<int, 16>(), std::integral_constant<int, 16>());
    else if (m <= 512)
        f(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
    else
        f(std::integral_constant<int, 64>(), std::integral_constant<int, 16>());
}

int route_slots(int m) { return m <= 8 ? kBlock / 8 : m <= 256 ? kBlock / 16 : kBlock / 64; }

unsigned route_grid(int64_t n, int m) {
    const int slots = route_slots(m);
    return (unsigned)std::min<int64_t>((n + slots - 1) / slots, kRouteGroupsOfGrid);
}

template <class T>
hipError_t launch_route(const RouteArgs& A, hipStream_t s) {
    size_t lds = A.counts ? ((size_t)A.m * 4 + 7) / 8 * 8 : 0;
    if (A.n_group > 1) lds += (size_t)route_slots(A.m) * ((size_t)A.m * 8 + (size_t)A.n_group * 24);
    by_width(A.m, [&](auto l, auto e) {
        hipLaunchKernelGGL((k_route<T, decltype(l)::value, decltype(e)::value>), dim3(route_grid(A.n, A.m)),
                           dim3(kBlock), lds, s, A);
    });
    return hipGetLastError();
}

template <class T>
hipError_t launch_route_grad(const RouteGradArgs& A, hipStream_t s) {
    by_width(A.m, [&](auto l, auto e) {
        hipLaunchKernelGGL((k_route_grad<T, decltype(l)::value, decltype(e)::value>), dim3(route_grid(A.n, A.m)),
                           dim3(kBlock), 0, s, A);
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
    A.k = k;
    A.renorm = renorm;
    A.scale = scale;
    A.idx = idx;
    A.weights = weights;
    A.counts = counts;
    A.fill = n == 0 || route_grid(n, A.m) > 1;
    if (counts && A.fill) {
        hipLaunchKernelGGL(k_clear_counts, dim3((unsigned)((m + kBlock - 1) / kBlock)), dim3(kBlock), 0, s, counts, (int)m);
        SK_TRY_LAUNCH(hipGetLastError());
    }
    if (n == 0) return SK_OK;
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
