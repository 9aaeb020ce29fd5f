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
#include "sk_scores.hpp"

#include <algorithm>

namespace sk {
namespace {

constexpr int kSolveMaxCols = 1024;
constexpr int kSolveGroups = 512;  // workgroups of a pass: two per CU

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
    int last;
};

// One row per L lanes, E scores per lane (column e L + l), 64 / L rows per wave.
template <class T, int L, int E>
__global__ __launch_bounds__(kBlock) void k_solve_pass(SolveArgs A) {
    constexpr int kSlots = kBlock / L;  // rows of one workgroup at a time
    __shared__ float red[kBlock / 64][L * E];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const float l2b = -s_lg2((float)A.m);
    float h[E], acc[E];
    int col[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int j = e * L + l;
        col[e] = j < A.m ? j : A.m - 1;  // loads of the padding lanes stay inside the row
        const float g = A.g_in ? A.g_in[col[e]] : 0.0f;
        const float lb = A.b ? s_lg2(A.b[col[e]]) : l2b;
        h[e] = j < A.m ? fmaf(g, A.c, lb) : -INFINITY;
        acc[e] = 0.0f;
    }
    const float uniform = 1.0f / (float)A.n;
    for (int64_t i0 = (int64_t)blockIdx.x * kSlots; i0 < A.n; i0 += (int64_t)A.groups * kSlots) {
        const int64_t i = i0 + slot;
        const bool on = i < A.n;
        const typename T::type* row = static_cast<const typename T::type*>(A.s) + (on ? i : 0) * A.ld;
        float t[E];
        float M = kNegBig;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            t[e] = fmaf(T::to(row[col[e]]), A.c, h[e]);
            M = fmaxf(M, t[e]);
        }
        M = lanes_max<L>(M);
        float S = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            t[e] = s_ex2(t[e] - M);
            S += t[e];
        }
        S = lanes_sum<L>(S);
        // a row that the mask leaves empty has S = 0: its potential is 0 and it sends nothing; nor does a row
        // of weight zero, whatever it holds
        const float w = on ? (A.a ? A.a[i] : uniform) : 0.0f;
        const float scale = S == 0.0f || w == 0.0f ? 0.0f : w / S;
        if (on && l == 0) A.f[i] = S == 0.0f ? 0.0f : -A.inv_c * (M + s_lg2(S));
        if (scale != 0.0f) {
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(t[e], scale, acc[e]);
        }
    }
    // rows of the wave, then the waves
#pragma unroll
    for (int e = 0; e < E; ++e) {
        for (int o = L; o < 64; o *= 2) acc[e] += __shfl_xor(acc[e], o);
        if ((threadIdx.x & 63) < L) red[threadIdx.x / 64][e * L + l] = acc[e];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < A.m; j += kBlock) {
        float sum = 0.0f;
        for (int w = 0; w < kBlock / 64; ++w) sum += red[w][j];
        A.part[(int64_t)blockIdx.x * A.m + j] = sum;
    }
}

// The column half-step from the passes' partial sums: 32 columns per workgroup, 8 slices of the partials.
template <class T>
__global__ __launch_bounds__(kBlock) void k_solve_update(SolveArgs A) {
    constexpr int kCols = 32, kSlices = kBlock / kCols;
    __shared__ float sum[kSlices][kCols];
    __shared__ float wave_m[kBlock / 64], wave_s[kBlock / 64];
    __shared__ int direct[kCols];
    const int x = threadIdx.x % kCols, y = threadIdx.x / kCols;
    const int j = blockIdx.x * kCols + x;
    float part = 0.0f;
    if (j < A.m)
        for (int w = y; w < A.groups; w += kSlices) part += A.part[(int64_t)w * A.m + j];
    sum[y][x] = part;
    __syncthreads();
    if (y == 0) {
        float cj = 0.0f;
        for (int k = 0; k < kSlices; ++k) cj += sum[k][x];
        int need = 0;
        if (j < A.m) {
            const float g = A.g_in ? A.g_in[j] : 0.0f;
            const float bj = A.b ? A.b[j] : 1.0f / (float)A.m;
            // each of the n terms loses at most 2^-126: above n 2^-100 that is below a rounding
            if (bj > 0.0f && cj >= (float)A.n * 0x1p-100f)
                A.g[j] = fmaf(A.inv_c, s_lg2(bj) - s_lg2(cj), g);
            else if (bj == 0.0f && !A.last)
                A.g[j] = g;  // enters no row before the last iteration
            else
                need = 1;
        }
        direct[x] = need;
    }
    __syncthreads();
    for (int k = 0; k < kCols; ++k) {
        if (!direct[k]) continue;  // the same for the whole workgroup
        const int col = blockIdx.x * kCols + k;
        const float l2n = -s_lg2((float)A.n);
        float M = kNegBig, S = 0.0f;
        for (int64_t i = threadIdx.x; i < A.n; i += kBlock) {
            if (A.a && A.a[i] == 0.0f) continue;
            const float s = T::to(static_cast<const typename T::type*>(A.s)[i * A.ld + col]);
            const float t = fmaf(s + A.f[i], A.c, A.a ? s_lg2(A.a[i]) : l2n);
            const float top = fmaxf(M, t);
            S = S * s_ex2(M - top) + s_ex2(t - top);
            M = top;
        }
        const float top = lanes_max<64>(M);
        const float s = lanes_sum<64>(S * s_ex2(M - top));
        if (threadIdx.x % 64 == 0) wave_m[threadIdx.x / 64] = top, wave_s[threadIdx.x / 64] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            float m2 = kNegBig, s2 = 0.0f;
            for (int w = 0; w < kBlock / 64; ++w) m2 = fmaxf(m2, wave_m[w]);
            for (int w = 0; w < kBlock / 64; ++w) s2 += wave_s[w] * s_ex2(wave_m[w] - m2);
            A.g[col] = s2 == 0.0f ? 0.0f : -A.inv_c * (m2 + s_lg2(s2));
        }
        __syncthreads();
    }
}

// n_iters = 0: f = 0, g = g_init or 0.
__global__ __launch_bounds__(kBlock) void k_solve_start(SolveArgs A) {
    const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (i < A.n) A.f[i] = 0.0f;
    if (i < A.m) A.g[i] = A.g_in ? A.g_in[i] : 0.0f;
}

int solve_rows_per_group(int m) { return m <= 256 ? kBlock / 16 : kBlock / 64; }

int solve_groups(int64_t n, int64_t m) {
    const int rows = solve_rows_per_group((int)m);
    return (int)std::min<int64_t>((n + rows - 1) / rows, kSolveGroups);
}

template <class T>
hipError_t launch_solve_pass(const SolveArgs& A, hipStream_t s) {
    const dim3 grid(A.groups), block(kBlock);
    if (A.m <= 16)
        hipLaunchKernelGGL((k_solve_pass<T, 16, 1>), grid, block, 0, s, A);
    else if (A.m <= 32)
        hipLaunchKernelGGL((k_solve_pass<T, 16, 2>), grid, block, 0, s, A);
    else if (A.m <= 64)
        hipLaunchKernelGGL((k_solve_pass<T, 16, 4>), grid, block, 0, s, A);
    else if (A.m <= 128)
        hipLaunchKernelGGL((k_solve_pass<T, 16, 8>), grid, block, 0, s, A);
    else if (A.m <= 256)
        hipLaunchKernelGGL((k_solve_pass<T, 16, 16>), grid, block, 0, s, A);
    else if (A.m <= 512)
        hipLaunchKernelGGL((k_solve_pass<T, 64, 8>), grid, block, 0, s, A);
    else
        hipLaunchKernelGGL((k_solve_pass<T, 64, 16>), grid, block, 0, s, A);
    return hipGetLastError();
}

template <class T>
int solve(SolveArgs A, int n_iters, hipStream_t s) {
    if (n_iters == 0) {
        const int64_t most = std::max(A.n, A.m);
        hipLaunchKernelGGL(k_solve_start, dim3((unsigned)((most + kBlock - 1) / kBlock)), dim3(kBlock), 0, s, A);
        SK_TRY_LAUNCH(hipGetLastError());
        return SK_OK;
    }
    for (int k = 0; k < n_iters; ++k) {
        A.last = k + 1 == n_iters;
        SK_TRY_LAUNCH(launch_solve_pass<T>(A, s));
        hipLaunchKernelGGL((k_solve_update<T>), dim3((unsigned)((A.m + 31) / 32)), dim3(kBlock), 0, s, A);
        SK_TRY_LAUNCH(hipGetLastError());
        A.g_in = A.g;
    }
    return SK_OK;
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
