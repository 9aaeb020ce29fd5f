// sk_scores_solve.hip -- log-domain Sinkhorn on a given score matrix
// (sk_scores_solve): the potentials that balance a router's scores.
//
// With the cost C = -s the half-steps of the library are
//     f_i = -eps LSE_j[(g_j + s_ij)/eps + log b_j],
//     g_j = -eps LSE_i[(f_i + s_ij)/eps + log a_i].
// One read of the scores serves both.  In base 2 (c = log2e / eps),
//     t_ij = c s_ij + h_j,  h_j = c g_j + log2 b_j,  M_i = max_j t_ij,
//     S_i = sum_j 2^(t_ij - M_i),  f_i = -(M_i + log2 S_i) / c,
// and q_ij = 2^(t_ij - M_i) / S_i is the row-normalised plan, so
//     c_j = sum_i a_i q_ij = b_j exp(g_j/eps) sum_i a_i exp((f_i + s_ij)/eps),
// and the column half-step is g_j <- g_j + eps log(b_j / c_j): one exponential
// per score and iteration, no running maximum over the long axis.  What the
// exponential flushes below 2^-126 is lost to c_j; a column whose sum is too
// small to be sure of it (or whose b_j is zero) takes its log-sum-exp over the
// rows directly.  Sums over rows run in a fixed order (per lane, lanes, waves,
// workgroups): results are deterministic.
//
// The direct sum is one strided read of a column by one workgroup, which takes its
// columns in turn.  A column that is masked in every row has a sum of zero and takes it
// in every iteration: 10 iterations of 32768 x 256 bfloat16 take 90 us without such a
// column, 560 with one or with one in each of eight workgroups, 3550 with eight
// neighbouring ones.  A column switched off by b_j = 0 takes it in the last iteration
// alone: 139 us with one, 437 with eight neighbouring ones.
//
// An iteration is two launches: the pass leaves each workgroup's column sums,
// the update joins them.  At 32768 x 256 bfloat16 an iteration takes 8.9 us: 6.6
// the pass (16.8 MB from the caches in 2 row steps per wave, about 3 us of
// instruction issue; the rest is latency: launch, column terms, first rows, joining in LDS)
// and 2.3 the update.  Problems of at most 32 scores per thread of one workgroup
// run all their iterations in a single launch: 8 iterations of 200 x 16 take 12 us
// against 40 in two launches each, and at the limit 30 against 43 (2048 x 16), 28
// against 47 (512 x 64), 30 against 56 (128 x 256).
#include "sk_scores.hpp"

#include <algorithm>

namespace sk {
namespace {

constexpr int kSolveMaxCols = 1024;
constexpr int kSolveThreads = 1024;  // of a pass: 16 waves, whose sums are joined in LDS before they reach memory
constexpr int kSolveGroups = 256;    // workgroups of a pass: one per CU, so the update joins at most 256 partials
constexpr int kSmallScores = 32;     // scores per thread of the single-workgroup kernel

struct SolveArgs {
    const void* s;
    int64_t ld;
    int n, m;
    const float *a, *b;  // null: uniform 1/n, 1/m
    const float* g_in;   // potentials before the iteration (null: zeros)
    float *f, *g;
    float* part;         // [groups][m] sums over each workgroup's rows
    float c, inv_c;      // log2e / eps, eps ln2
    int groups;
    int last;            // the iteration is the last one
    int iters;           // of the single-workgroup kernel
};

// The row half-step of a row held as t (scores in base 2 with the column
// terms): t becomes 2^(t - M), and the row's potential and the factor a / S of
// its share in the column sums are returned.  A row that the mask leaves empty has S = 0: its
// potential is 0 and it sends nothing; nor does a row of weight zero, whatever
// it holds.
template <int L, int E>
__device__ __forceinline__ float row_step(const SolveArgs& A, float (&t)[E], float w, float* f) {
    float M = kNegBig;
#pragma unroll
    for (int e = 0; e < E; ++e) M = fmaxf(M, t[e]);
    M = lanes_max<L>(M);
    float S = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        t[e] = s_ex2(t[e] - M);
        S += t[e];
    }
    S = lanes_sum<L>(S);
    *f = S == 0.0f ? 0.0f : -A.inv_c * (M + s_lg2(S));
    return S == 0.0f || w == 0.0f ? 0.0f : w * __builtin_amdgcn_rcpf(S);
}

__device__ __forceinline__ float log2_b(const SolveArgs& A, int j) { return A.b ? s_lg2(A.b[j]) : -s_lg2((float)A.m); }

// Whether the sum c_j is sure to hold what its n terms a_i q_ij add up to: a term loses at most a_i 2^-126 to the
// exponential's flush and 2^-126 to its own, so above (mass + n) 2^-100 less than a rounding is lost.
__device__ __forceinline__ bool safe(const SolveArgs& A, float cj, float mass) { return cj >= (mass + (float)A.n) * 0x1p-100f; }

// The mass of the weights, by the whole workgroup (through its columns' side, which is the shorter one).
template <int THREADS>
__device__ float total_mass(const SolveArgs& A) {
    if (!A.b) return 1.0f;
    __shared__ float part[THREADS / 64];
    float sum = 0.0f;
    for (int j = threadIdx.x; j < A.m; j += THREADS) sum += A.b[j];
    sum = lanes_sum<64>(sum);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int w = 0; w < THREADS / 64; ++w) sum += part[w];
    return sum;
}

// The column half-step of one column by its log-sum-exp over the rows, by the whole workgroup.
template <class T, int THREADS>
__device__ float column_direct(const SolveArgs& A, int col, const float* f) {
    __shared__ float wave_m[THREADS / 64], wave_s[THREADS / 64];
    const float l2n = -s_lg2((float)A.n);
    float M = kNegBig, S = 0.0f;
    for (int64_t i = threadIdx.x; i < A.n; i += THREADS) {
        if (A.a && A.a[i] == 0.0f) continue;
        const float s = T::to(static_cast<const typename T::type*>(A.s)[i * A.ld + col]);
        const float t = fmaf(s + f[i], A.c, A.a ? s_lg2(A.a[i]) : l2n);
        const float top = fmaxf(M, t);
        S = S * s_ex2(M - top) + s_ex2(t - top);
        M = top;
    }
    const float top = lanes_max<64>(M);
    const float s = lanes_sum<64>(S * s_ex2(M - top));
    __syncthreads();
    if (threadIdx.x % 64 == 0) wave_m[threadIdx.x / 64] = top, wave_s[threadIdx.x / 64] = s;
    __syncthreads();
    float m2 = kNegBig, s2 = 0.0f;
    for (int w = 0; w < THREADS / 64; ++w) m2 = fmaxf(m2, wave_m[w]);
    for (int w = 0; w < THREADS / 64; ++w) s2 += wave_s[w] * s_ex2(wave_m[w] - m2);
    return s2 == 0.0f ? 0.0f : -A.inv_c * (m2 + s_lg2(s2));
}

// One row per L lanes, E scores per lane, 1024 / L rows of a workgroup at a time.
template <class T, int L, int E, bool V>
__global__ __launch_bounds__(kSolveThreads) void k_solve_pass(SolveArgs A) {
    constexpr int kSlots = kSolveThreads / L, kWaves = kSolveThreads / 64;
    using R = Row<T, L, E, V>;
    __shared__ float red[kWaves][L * E];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const float uniform = 1.0f / (float)A.n;
    const int64_t step = (int64_t)A.groups * kSlots;
    int64_t i = (int64_t)blockIdx.x * kSlots + slot;
    typename R::Raw next;  // the next row, loaded while this one is worked on
    auto fetch = [&](int64_t row) {
        R::fetch(static_cast<const typename T::type*>(A.s) + (row < A.n ? row : 0) * A.ld, l, A.m, next);
    };
    fetch(i);
    // the columns' terms, each loaded once and passed on through LDS
    for (int j = threadIdx.x; j < L * E; j += kSolveThreads)
        red[0][j] = j < A.m ? fmaf(A.g_in ? A.g_in[j] : 0.0f, A.c, log2_b(A, j)) : -INFINITY;
    __syncthreads();
    float h[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        h[e] = red[0][R::col(e, l)];
        acc[e] = 0.0f;
    }
    __syncthreads();
    for (int64_t i0 = (int64_t)blockIdx.x * kSlots; i0 < A.n; i0 += step, i += step) {
        const bool on = i < A.n;
        float t[E], f;
        R::template get<false>(next, l, A.m, t);  // (behind the row h is -inf)
        if (i0 + step < A.n) fetch(i + step);
        const float w = on ? (A.a ? A.a[i] : uniform) : 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) t[e] = fmaf(t[e], A.c, h[e]);
        const float scale = row_step<L, E>(A, t, w, &f);
        if (on && l == 0) A.f[i] = f;
        if (scale != 0.0f) {
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(t[e], scale, acc[e]);
        }
    }
    // rows of the wave, then the waves
#pragma unroll
    for (int e = 0; e < E; ++e) {
        acc[e] = groups_sum<L>(acc[e]);
        if ((threadIdx.x & 63) < L) red[threadIdx.x / 64][R::col(e, l)] = acc[e];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < A.m; j += kSolveThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += red[w][j];
        A.part[(int64_t)blockIdx.x * A.m + j] = sum;
    }
}

// The column half-step from the passes' partial sums: 8 columns per workgroup, 32 slices of the partials.
template <class T>
__global__ __launch_bounds__(kBlock) void k_solve_update(SolveArgs A) {
    constexpr int kCols = 8, kSlices = kBlock / kCols;
    __shared__ float sum[kSlices][kCols];
    __shared__ int direct[kCols];
    const int x = threadIdx.x % kCols, y = threadIdx.x / kCols;
    const int j = blockIdx.x * kCols + x;
    const int jc = j < A.m ? j : 0;
    const float g = A.g_in ? A.g_in[jc] : 0.0f, lb = log2_b(A, jc);
    float part = 0.0f;
    if (j < A.m) {
#pragma unroll
        for (int k = 0; k < kSolveGroups / kSlices; ++k) {
            const int w = k * kSlices + y;
            const float p = A.part[(int64_t)min(w, A.groups - 1) * A.m + j];
            part += w < A.groups ? p : 0.0f;
        }
    }
    sum[y][x] = part;
    const float mass = total_mass<kBlock>(A);
    __syncthreads();
    if (y == 0) {
        float cj = 0.0f;
#pragma unroll
        for (int k = 0; k < kSlices; ++k) cj += sum[k][x];
        int need = 0;
        if (j < A.m) {
            if (lb > -INFINITY && safe(A, cj, mass))
                A.g[j] = fmaf(A.inv_c, lb - s_lg2(cj), g);
            else if (lb == -INFINITY && !A.last)
                A.g[j] = g;  // a column of weight zero enters no row before the last iteration
            else
                need = 1;
        }
        direct[x] = need;
    }
    __syncthreads();
    for (int k = 0; k < kCols; ++k) {
        if (!direct[k]) continue;  // the same for the whole workgroup
        const int col = blockIdx.x * kCols + k;
        const float g = column_direct<T, kBlock>(A, col, A.f);
        if (threadIdx.x == 0) A.g[col] = g;
    }
}

// All iterations in one workgroup, the scores in registers (R rows per slot).
template <class T, int L, int E, bool V>
__global__ __launch_bounds__(kSolveThreads) void k_solve_small(SolveArgs A) {
    constexpr int kSlots = kSolveThreads / L, kWaves = kSolveThreads / 64, R = kSmallScores / E;
    using Rw = Row<T, L, E, V>;
    __shared__ float red[kWaves][L * E];
    __shared__ float g[L * E], fs[kSlots * R];
    __shared__ int direct[2];  // of this iteration and the next one
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    float s[R][E], lb[E], w[R];
    const float uniform = 1.0f / (float)A.n;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = r * kSlots + slot;
        const bool on = i < A.n;
        typename Rw::Raw raw;
        Rw::fetch(static_cast<const typename T::type*>(A.s) + (int64_t)(on ? i : 0) * A.ld, l, A.m, raw);
        Rw::template get<false>(raw, l, A.m, s[r]);  // (behind the row lb is -inf)
        w[r] = on ? (A.a ? A.a[i] : uniform) : 0.0f;
    }
    const float b2 = (int)threadIdx.x < A.m ? log2_b(A, threadIdx.x) : -INFINITY;  // of this thread's column
    if (threadIdx.x < L * E) {
        g[threadIdx.x] = (int)threadIdx.x < A.m && A.g_in ? A.g_in[threadIdx.x] : 0.0f;
        red[0][threadIdx.x] = b2;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) lb[e] = red[0][Rw::col(e, l)];
    if (threadIdx.x < 2) direct[threadIdx.x] = 0;
    const float mass = total_mass<kSolveThreads>(A);
    for (int k = 0; k < A.iters; ++k) {
        __syncthreads();
        float h[E], acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            h[e] = fmaf(g[Rw::col(e, l)], A.c, lb[e]);
            acc[e] = 0.0f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r * kSlots >= A.n) break;
            float t[E], f;
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = fmaf(s[r][e], A.c, h[e]);
            const float scale = row_step<L, E>(A, t, w[r], &f);
            if (l == 0) fs[r * kSlots + slot] = f;
            if (scale != 0.0f) {
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(t[e], scale, acc[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[e] = groups_sum<L>(acc[e]);
            if ((threadIdx.x & 63) < L) red[threadIdx.x / 64][Rw::col(e, l)] = acc[e];
        }
        __syncthreads();
        const int j = threadIdx.x;
        const bool last = k + 1 == A.iters;
        bool need = false;
        // (every thread has read the last iteration's flag before this iteration's first barrier)
        if (threadIdx.x == 0) direct[(k + 1) & 1] = 0;
        if (j < A.m) {
            float cj = 0.0f;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) cj += red[q][j];
            if (b2 > -INFINITY && safe(A, cj, mass))
                g[j] = fmaf(A.inv_c, b2 - s_lg2(cj), g[j]);
            else
                need = b2 > -INFINITY || last;
            if (need) direct[k & 1] = 1;
            red[0][j] = need ? 1.0f : 0.0f;
        }
        __syncthreads();
        if (direct[k & 1]) {
            for (int q = 0; q < A.m; ++q) {
                if (red[0][q] == 0.0f) continue;
                const float x = column_direct<T, kSolveThreads>(A, q, fs);
                if (threadIdx.x == 0) g[q] = x;
            }
            __syncthreads();
        }
    }
    if ((int)threadIdx.x < A.m) A.g[threadIdx.x] = g[threadIdx.x];
    for (int i = threadIdx.x; i < A.n; i += kSolveThreads) A.f[i] = fs[i];
}

// n_iters = 0: f = 0, g = g_init or 0.
__global__ __launch_bounds__(kBlock) void k_solve_start(SolveArgs A) {
    const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (i < A.n) A.f[i] = 0.0f;
    if (i < A.m) A.g[i] = A.g_in ? A.g_in[i] : 0.0f;
}

// f(lanes per row, scores per lane) for rows of m scores.  Every lane of a row
// repeats the row's own work (reductions, reciprocal); fewer lanes with more scores
// each have longer chains.  8 iterations of 32768 x 64 f32 take 51 us (58 with 4 x 16),
// of 32768 x 128 bf16 57.7 (58.8 with 8 x 16), of 16384 x 512 bf16 75.6 (70.8 with
// 32 x 16); in one workgroup 200 x 64 takes 19.5 (23.8) and 30 x 512 19.3 (21.0).
template <class F>
void solve_width(int m, F f) {
    using std::integral_constant;
    if (m <= 16)
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

int solve_groups(int64_t n, int64_t m) {
    int64_t rows = 0;
    solve_width((int)m, [&](auto lanes, auto) { rows = kSolveThreads / decltype(lanes)::value; });
    return (int)std::min<int64_t>((n + rows - 1) / rows, kSolveGroups);
}

template <class T>
int solve(SolveArgs A, int n_iters, hipStream_t s) {
    if (n_iters == 0) {
        const int64_t most = std::max(A.n, A.m);
        hipLaunchKernelGGL(k_solve_start, dim3((unsigned)((most + kBlock - 1) / kBlock)), dim3(kBlock), 0, s, A);
        SK_TRY_LAUNCH(hipGetLastError());
        return SK_OK;
    }
    int st = SK_OK;
    solve_width(A.m, [&](auto lanes, auto per_lane) {
        constexpr int L = decltype(lanes)::value, E = decltype(per_lane)::value;
        auto small = k_solve_small<T, L, E, false>;
        auto pass = k_solve_pass<T, L, E, false>;
        if (Row<T, L, E, true>::fits(A.s, A.ld, A.m)) {
            small = k_solve_small<T, L, E, true>;
            pass = k_solve_pass<T, L, E, true>;
        }
        if (A.n <= kSolveThreads / L * (kSmallScores / E)) {
            A.iters = n_iters;
            hipLaunchKernelGGL(small, dim3(1), dim3(kSolveThreads), 0, s, A);
            if (hipGetLastError() != hipSuccess) st = SK_ERR_HIP;
            return;
        }
        for (int k = 0; k < n_iters && st == SK_OK; ++k) {
            A.last = k + 1 == n_iters;
            hipLaunchKernelGGL(pass, dim3(A.groups), dim3(kSolveThreads), 0, s, A);
            if (hipGetLastError() != hipSuccess) st = SK_ERR_HIP;
            hipLaunchKernelGGL((k_solve_update<T>), dim3((unsigned)((A.m + 7) / 8)), dim3(kBlock), 0, s, A);
            if (hipGetLastError() != hipSuccess) st = SK_ERR_HIP;
            A.g_in = A.g;
        }
    });
    return st;
}

size_t solve_ws_bytes(int64_t n, int64_t m) {
    return ((size_t)solve_groups(n, m) * (size_t)m * sizeof(float) + 255) / 256 * 256;
}

}  // namespace
}  // namespace sk

using namespace sk;

extern "C" {

size_t sk_scores_solve_workspace_bytes(int64_t n, int64_t m) {
    if (n < 1 || m < 1 || n > INT32_MAX || m > kSolveMaxCols) return 0;
    return solve_ws_bytes(n, m);
}

int sk_scores_solve(const void* scores, int32_t dtype, int64_t n, int64_t m, int64_t ld, const float* a,
                    const float* b, float eps, int32_t n_iters, const float* g_init, float* f, float* g, void* ws,
                    size_t ws_bytes, void* stream) {
    if (!scores || !f || !g) return SK_ERR_NULL;
    if (n < 1 || m > kSolveMaxCols) return SK_ERR_SHAPE;
    int st = check_scores(scores, dtype, n, m, ld);
    if (st) return st;
    if ((st = check_temperature(eps))) return st;
    if (n_iters < 0) return SK_ERR_ITERS;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < solve_ws_bytes(n, m)) return SK_ERR_WORKSPACE;
    SolveArgs A{};
    A.s = scores;
    A.ld = ld;
    A.n = (int)n;
    A.m = (int)m;
    A.a = a;
    A.b = b;
    A.g_in = g_init;
    A.f = f;
    A.g = g;
    A.part = static_cast<float*>(ws);
    A.c = (float)(1.4426950408889634 / (double)eps);
    A.inv_c = (float)(0.6931471805599453 * (double)eps);
    A.groups = solve_groups(n, m);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    switch (dtype) {
        case SK_F32: return solve<F32>(A, n_iters, s);
        case SK_BF16: return solve<Bf16>(A, n_iters, s);
        default: return solve<F16>(A, n_iters, s);
    }
}

}  // extern "C"
