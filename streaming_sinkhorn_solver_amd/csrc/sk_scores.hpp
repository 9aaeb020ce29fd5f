// sk_scores.hpp -- what the operators on a given score matrix share
// (sk_scores_solve.hip, sk_scores_route.hip, sk_scores_logprobs.hip,
// sk_scores_verify.hip) and on rows of tokens (sk_route_rows.hip): element
// types, reductions inside a wave without LDS, argument checks.
//
// A score matrix is row-major, n rows of m scores with a row stride of ld
// elements (ld >= m), in float32, bfloat16 or float16; every sum, maximum and
// exponential is in float32, whatever the type.  Offsets are 64-bit.
#pragma once

#include "sk.h"
#include "sk_internal.hpp"

#include <climits>
#include <cmath>

#define SK_TRY_LAUNCH(expr)                       \
    do {                                          \
        if ((expr) != hipSuccess) return SK_ERR_HIP; \
    } while (0)

namespace sk {
namespace {

// ----- element types ----------------------------------------------------------------
struct F32 {
    using type = float;
    static constexpr uint32_t kNegInfBits = 0xff800000u;  // one 32-bit word of -inf elements
    static constexpr int kLowBits = 0;                    // of the float32 value that are always zero
    __device__ static float to(float v) { return v; }
    __device__ static float from(float v) { return v; }
};
struct Bf16 {
    using type = uint16_t;
    static constexpr uint32_t kNegInfBits = 0xff80ff80u;
    static constexpr int kLowBits = 16;
    __device__ static float to(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
    __device__ static uint16_t from(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }  // nearest even
};
struct F16 {
    using type = uint16_t;
    static constexpr uint32_t kNegInfBits = 0xfc00fc00u;
    static constexpr int kLowBits = 13;
    __device__ static float to(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
    // Nearest even, of the float32 value: the product that made it is not contracted with the conversion, which the
    // compiler does in some of a kernel's paths and not in others.
    __device__ static uint16_t from(float v) {
        asm("" : "+v"(v));
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    }
};

inline int elem_size(int32_t dtype) { return dtype == SK_F32 ? 4 : 2; }

// ----- base-2 exponential and logarithm -----------------------------------------------
__device__ __forceinline__ float s_ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float s_lg2(float x) { return __builtin_amdgcn_logf(x); }

// ----- reductions over groups of L consecutive lanes (L = 4, 8, 16, 32 or 64), result in every lane --------
// Inside a row of 16 lanes by quad permutations, half-row mirror and rotation;
// across the four rows of a wave by the row swaps.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, true);
}
constexpr int kQuadXor1 = 0xb1;     // quad_perm [1, 0, 3, 2]
constexpr int kQuadXor2 = 0x4e;     // quad_perm [2, 3, 0, 1]
constexpr int kHalfMirror = 0x141;  // row_half_mirror: lane i <- 7 - i in each 8 lanes
constexpr int kRor4 = 0x124;        // row_ror:4
constexpr int kRor8 = 0x128;        // row_ror:8

template <int L, class Op>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t x, Op op) {
    static_assert(L == 4 || L == 8 || L == 16 || L == 32 || L == 64, "lanes per row");
    x = op(x, dpp<kQuadXor1>(x));
    x = op(x, dpp<kQuadXor2>(x));
    if constexpr (L >= 8) x = op(x, dpp<kHalfMirror>(x));
    if constexpr (L >= 16) x = op(x, dpp<kRor8>(x));
    if constexpr (L >= 32) {
        auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = op((uint32_t)r[0], (uint32_t)r[1]);
    }
    if constexpr (L == 64) {
        auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        x = op((uint32_t)r[0], (uint32_t)r[1]);
    }
    return x;
}

struct OpMaxF {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
    }
};
struct OpAddF {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }
};
struct OpMaxU {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
struct OpOr {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a | b; }
};
struct OpAddU {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a + b; }
};
struct OpMinU {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a < b ? a : b; }
};

// Sum over the 64 / L groups of L lanes of a wave (lanes with the same number in their groups), in every lane.
template <int L>
__device__ __forceinline__ float groups_sum(float x) {
    asm("" : "+v"(x));  // (as in lanes_sum)
    uint32_t u = __builtin_bit_cast(uint32_t, x);
    OpAddF add;
    if constexpr (L <= 8) u = add(u, dpp<kRor8>(u));
    if constexpr (L <= 4) u = add(u, dpp<kRor4>(u));
    if constexpr (L <= 16) {
        auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        u = add((uint32_t)r[0], (uint32_t)r[1]);
        r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        u = add((uint32_t)r[0], (uint32_t)r[1]);
    }
    return __builtin_bit_cast(float, u);
}

template <int L>
__device__ __forceinline__ float lanes_max(float x) {
    return __builtin_bit_cast(float, lanes_reduce<L>(__builtin_bit_cast(uint32_t, x), OpMaxF()));
}
// The order of the additions is fixed by the lane numbers alone, and every lane gets the same bits: a product in x is
// rounded first (contracted with the first addition, each lane would round only its neighbour's).
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
    asm("" : "+v"(x));
    return __builtin_bit_cast(float, lanes_reduce<L>(__builtin_bit_cast(uint32_t, x), OpAddF()));
}
template <int L>
__device__ __forceinline__ double lanes_sum(double x) {
    for (int o = 1; o < L; o *= 2) x += __shfl_xor(x, o);
    return x;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
    return lanes_reduce<L>(x, OpMaxU());
}
template <int L>
__device__ __forceinline__ uint32_t lanes_sum_u(uint32_t x) {
    return lanes_reduce<L>(x, OpAddU());
}
template <int L>
__device__ __forceinline__ uint32_t lanes_min(uint32_t x) {
    return lanes_reduce<L>(x, OpMinU());
}

// ----- a row in the registers of L lanes, E scores per lane -------------------------------
// With V the lane takes runs of W neighbouring scores (16 bytes at most) from
// rows whose runs are aligned and whose m is a multiple of W; without, single
// scores L apart, from any row.
template <class T, int L, int E, bool V>
struct Row {
    using Elem = typename T::type;
    static constexpr int kMost = 16 / (int)sizeof(Elem);
    static constexpr int W = V ? (E < kMost ? E : kMost) : 1;
    __device__ static int col(int e, int l) { return (e / W * L + l) * W + e % W; }
    struct alignas(W * sizeof(Elem)) Run {
        Elem v[W];
    };
    // fetch only issues the loads; get converts what arrived (MASK: -inf behind the row, else some score of it).
    struct Raw {
        Run r[E / W];
    };
    __device__ static void fetch(const Elem* row, int l, int m, Raw& raw) {
#pragma unroll
        for (int q = 0; q < E / W; ++q) {
            const int j = col(q * W, l);
            raw.r[q] = *reinterpret_cast<const Run*>(row + (j < m ? j : W == 1 ? m - 1 : 0));
        }
    }
    template <bool MASK = true>
    __device__ static void get(const Raw& raw, int l, int m, float (&s)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            s[e] = !MASK || col(e / W * W, l) < m ? T::to(raw.r[e / W].v[e % W]) : -INFINITY;
    }
    __device__ static void load(const Elem* row, int l, int m, float (&s)[E]) {
        Raw raw;
        fetch(row, l, m, raw);
        get(raw, l, m, s);
    }
    __device__ static void store(Elem* row, int l, int m, const float (&s)[E]) {
#pragma unroll
        for (int q = 0; q < E / W; ++q) {
            const int j = col(q * W, l);
            Run r;
#pragma unroll
            for (int e = 0; e < W; ++e) r.v[e] = T::from(s[q * W + e]);
            if (j < m) *reinterpret_cast<Run*>(row + j) = r;
        }
    }
    // Whether the rows of a matrix can be read and written in runs.
    static bool fits(const void* p, int64_t ld, int64_t m) {
        return W > 1 && m % W == 0 && ld % W == 0 && reinterpret_cast<uintptr_t>(p) % (W * sizeof(Elem)) == 0;
    }
};

// ----- 16 bytes of a row, at any address of its element type ------------------------------
// Such loads and stores need no alignment on this GPU, so rows of odd length or at odd addresses go the same way.
template <class T>
struct Run16 {
    using Elem = typename T::type;
    static constexpr int n = 16 / (int)sizeof(Elem);
    uint4 raw;
    __device__ __forceinline__ uint32_t word(int w) const { return w == 0 ? raw.x : w == 1 ? raw.y : w == 2 ? raw.z : raw.w; }
    __device__ __forceinline__ Elem bits(int i) const {
        if constexpr (n == 4)
            return __builtin_bit_cast(float, word(i));
        else
            return (uint16_t)(i % 2 ? word(i / 2) >> 16 : word(i / 2) & 0xffffu);
    }
    __device__ __forceinline__ float at(int i) const { return T::to(bits(i)); }
    __device__ __forceinline__ void set(const Elem (&v)[n]) { __builtin_memcpy(&raw, v, 16); }
    __device__ __forceinline__ void round(const float (&v)[n]) {
        Elem e[n];
#pragma unroll
        for (int i = 0; i < n; ++i) e[i] = T::from(v[i]);
        set(e);
    }
    __device__ __forceinline__ void fill(uint32_t w) { raw = make_uint4(w, w, w, w); }
    __device__ __forceinline__ void get(const Elem* p) { __builtin_memcpy(&raw, p, 16); }
    __device__ __forceinline__ void put(Elem* p) const { __builtin_memcpy(p, &raw, 16); }
    // ONCE: what this launch touches once, past what the caches hold.
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    typedef Words AnyWords __attribute__((aligned(2)));
    template <bool ONCE>
    __device__ __forceinline__ void fetch(const Elem* p) {
        if constexpr (ONCE) {
            const Words w = __builtin_nontemporal_load(reinterpret_cast<const AnyWords*>(p));
            raw = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            get(p);
        }
    }
    template <bool ONCE>
    __device__ __forceinline__ void store(Elem* p) const {
        if constexpr (ONCE)
            __builtin_nontemporal_store(Words{raw.x, raw.y, raw.z, raw.w}, reinterpret_cast<AnyWords*>(p));
        else
            put(p);
    }
    // Holds the run as it was loaded up to here: its conversions to float32, twice the registers, stay behind.
    __device__ __forceinline__ void held() { asm("" : "+v"(raw.x), "+v"(raw.y), "+v"(raw.z), "+v"(raw.w)); }
};

// LDS written by this wave's lanes is visible to its other lanes (one wave's
// LDS operations complete in order; this stops the compiler from moving them).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// ----- ordered keys: larger value = larger unsigned key, never 0; -0 equals +0, a NaN ranks as -inf -----
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return v == v ? k : 0x007fffffu;
}
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    const uint64_t k = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
    return v == v ? k : 0x000fffffffffffffull;
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __builtin_bit_cast(float, k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ double unordered(uint64_t k) {
    return __builtin_bit_cast(double, k ^ ((k >> 63) ? 0x8000000000000000ull : 0xffffffffffffffffull));
}

// The k-th largest of the 64 lanes' N keys each (the same in every lane), 0 if they are fewer.  LOW: the lowest
// bits that are all alike in every key, 0 above the sign's and 1 below it (ordered keys of 16-bit scores).
template <int LOW, int N>
__device__ __forceinline__ uint32_t kth_of_wave(const uint32_t (&key)[N], int k) {
    uint32_t t = 0;
    for (int b = 31; b >= LOW; --b) {
        const uint32_t x = t | (1u << b);
        int have = 0;
#pragma unroll
        for (int c = 0; c < N; ++c) have += __popcll(__ballot(key[c] >= x));
        if (have >= k) t = x;
    }
    return LOW > 0 && t && !(t >> 31) ? t | ((1u << LOW) - 1) : t;
}

// ----- host-side checks ---------------------------------------------------------------
// A row stride of at least m elements whose n rows stay below 2^60 elements.
inline bool good_stride(int64_t ld, int64_t n, int64_t m) {
    return ld >= m && ld <= ((int64_t)1 << 60) / (n > 0 ? n : 1);
}

inline int check_scores(const void* scores, int32_t dtype, int64_t n, int64_t m, int64_t ld) {
    if (dtype != SK_F32 && dtype != SK_BF16 && dtype != SK_F16) return SK_ERR_DTYPE;
    if (n < 0 || m < 1 || n > INT32_MAX || m > INT32_MAX || !good_stride(ld, n, m)) return SK_ERR_SHAPE;
    if (n == 0) return SK_OK;
    if (!scores) return SK_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(scores) % elem_size(dtype) != 0) return SK_ERR_DTYPE;
    return SK_OK;
}

// The gradient may be written over the scores (same address and row stride);
// any other overlap of the two n x m windows is refused.
inline int check_grad(const void* scores, int64_t ld, const void* grad, int64_t ld_grad, int32_t dtype, int64_t n,
                      int64_t m) {
    if (!good_stride(ld_grad, n, m)) return SK_ERR_SHAPE;
    if (n == 0) return SK_OK;
    if (!grad) return SK_ERR_NULL;
    const int64_t es = elem_size(dtype);
    const uintptr_t p = reinterpret_cast<uintptr_t>(scores), q = reinterpret_cast<uintptr_t>(grad);
    if (q % es != 0) return SK_ERR_DTYPE;
    if (p == q && (ld == ld_grad || n == 1)) return SK_OK;
    const uintptr_t lp = (uintptr_t)(((n - 1) * ld + m) * es), lq = (uintptr_t)(((n - 1) * ld_grad + m) * es);
    if (p + lp <= q || q + lq <= p) return SK_OK;
    if (ld == ld_grad) {  // two column windows of one buffer
        const uintptr_t row = (uintptr_t)(ld * es), w = (uintptr_t)(m * es);
        const uintptr_t off = (p > q ? p - q : q - p) % row;
        if (off >= w && off + w <= row) return SK_OK;
    }
    return SK_ERR_OVERLAP;
}

// Rows of d elements, stride ld, at address p.
struct Span {
    uintptr_t lo, hi, row, width;  // in bytes: what they span, the stride (0: a single row), a row
};
inline Span span_of(const void* p, int64_t n, int64_t d, int64_t ld, int es) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, n > 0 ? a + (uintptr_t)(((n - 1) * ld + d) * es) : a, n > 1 ? (uintptr_t)(ld * es) : 0, (uintptr_t)(d * es)};
}
inline Span span_of(const void* p, int64_t n, int es) { return span_of(p, 1, n, n, es); }
// Whether they have an element in common; two windows of columns of one buffer have none.
inline bool meet(Span a, Span b) {
    if (a.lo == a.hi || b.lo == b.hi || a.hi <= b.lo || b.hi <= a.lo) return false;
    const uintptr_t row = a.row ? a.row : b.row;
    if (row == 0 || (b.row && b.row != row)) return true;
    if (a.lo > b.lo) {
        const Span c = a;
        a = b;
        b = c;
    }
    const uintptr_t off = (b.lo - a.lo) % row;
    return !(off >= a.width && off + b.width <= row);
}

inline int check_temperature(float eps) {
    if (!std::isfinite(eps) || eps <= 0.0f) return SK_ERR_EPS;
    // log2e / eps, the factor of every exponent, must be finite and nonzero in fp32
    const double c = (double)kLog2e / (double)eps;
    if (!(c < 3.4e38) || !(c > 1.2e-38)) return SK_ERR_EPS;
    return SK_OK;
}

}  // namespace
}  // namespace sk
