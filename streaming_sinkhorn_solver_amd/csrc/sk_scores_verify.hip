// sk_scores_verify.hip -- drafted tokens against the target's probabilities
// (sk_scores_verify).
//
// With p = softmax(s / eps) of the target's row and q = softmax(t / eps_draft) of
// the draft's, or q one at the drafted token, a token x drawn from q is taken if
// u q(x) < p(x); in its place, at the first row where it is not, comes a draw from
// the residual max(p - q, 0).  That pair of draws is the maximal coupling of q and
// p, the transport plan of least cost 1[x != y].
//
// A decision or a draw next to a border must not depend on how sums are taken.  All
// rows' sums are taken in float32, at the rate that the scores arrive; a decision that
// lies within the bound of their error (some 2^-15 of p / q) takes its row's sums again
// in float64.  What is drawn from, one row per request, goes in float64 throughout: the
// error of a probability is some 2^-38 of it, where a row of 131072 has borders 2^-17
// apart in the mean and the random numbers are multiples of 2^-24.  With e and h the
// exponentials of p's and q's row and rho the quotient of their sums, the residual is
// max(e - rho h, 0).  One pass takes sum e and sum h, which give rho, and with rho0 from the
// float32 sums R = sum max(e - rho0 h, 0) and B = sum of h where e > rho0 h.  The residual's
// sum is then R + (rho0 - rho) B but for entries whose e / h lies between the two quotients:
// each is off by |rho0 - rho| h at most, some 2^-22 of itself, and must lie within the bound
// of the float32 error of rho0 (2^-15 to 2^-17), where the pass leaves a mark on its chunk.  A
// draw that is nearer to a border than these errors can add up to has the marked chunks summed
// again with rho itself: few draws, but many where p and q are proportional over much of the row.
#include "sk_scores.hpp"

#include <algorithm>

namespace sk {
namespace {

constexpr int64_t kVfGrid = 1 << 20;  // workgroups of one launch (each may serve several rows)
constexpr int64_t kVfMaxCols = (int64_t)1 << 30;
constexpr int kVfVecs = 4;             // 16-byte loads of a thread's block
constexpr int kVfChunkMost = 2048;     // entries of a chunk: 512, 1024 or this
constexpr int kVfFill = 1024;          // workgroups that a launch is cut into where it has fewer,
constexpr int kVfCutMin = 1024;        // no part of a row below so many 16-byte loads
constexpr double kFloor = -1000.0;     // exponents below count as zero; in the chunks' sums they count as 2^-1000,
constexpr double kNothing = 0x1p-900;  // and sums below this as zero
constexpr double kUnset = -1.0e300;    // reference of what is no part of a row

// What is needed of a row, or a part of one: sum of 2^(c (s - ref)), NaN if a score is NaN or +inf.  The reference is the
// largest score, and the difference to it is taken first: rows of a type's lowest value lose nothing.
struct Sum {
    double ref, s;
};

// What a request's draw needs.
struct Draw {
    double ref_p, log_p;  // reference of the row's sum, and the sum's log2
    double ref_q, rho;    // of the draft's row; the quotient of the two sums
    int64_t row;          // where the request stops, -1: nothing is drawn
    int64_t out;          // column that the residual leaves out, or -1
    int64_t with_q;
};

struct VfArgs {
    const void *s, *q;
    int64_t ld, ldq, n, b;
    int m;
    double c, cq;    // log2e / eps
    float cf, cqf;   // in float32: c over scale
    float scale, scale_q;  // of the scores before their differences: 1, or 1/2 at temperatures where one beyond float32 counts
    double floor, floor_q;  // kFloor / c
    double doubt;    // relative error of p / q from the float32 sums at most
    const int64_t *tokens, *starts;
    const float *u_accept, *u_sample;
    int32_t* accepted;
    int64_t *next, *out_tokens;
    float *ratio, *logp;
    int splits, cut;  // parts of a row, and the runs of 16 bytes of one
    int width;        // lanes that join a row's parts: a power of two
    int chunk_len, chunks, parts;
    Sum* sums;        // [n][2][splits]
    double* chunk;    // [b][chunks][4]
    Draw* draw;       // [b]
};

// 2^(d c) for d c in [kFloor, 1000]: the exponent is k + f with |f| <= 1/2, 2^f by the polynomial that meets it at the
// eight Chebyshev points and at 0 (within 2^-38.7), k added to the exponent.  2^0 is 1 exactly.
__device__ __forceinline__ double pow2(double d, double c) {
    constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52: the sum's low word is the nearest integer
    const double t = fma(d, c, kRound);
    const double f = fma(d, c, -(t - kRound));
    double p = 0x1.63b2d7971923fp-20;
    p = fma(p, f, 0x1.00c0e4e15189cp-16);
    p = fma(p, f, 0x1.4308c7183d6a2p-13);
    p = fma(p, f, 0x1.5d877598350dep-10);
    p = fma(p, f, 0x1.3b2ab70ad2565p-7);
    p = fma(p, f, 0x1.c6b08da70cce3p-5);
    p = fma(p, f, 0x1.ebfbdff82a734p-3);
    p = fma(p, f, 0x1.62e42fef9cc69p-1);
    p = fma(p, f, 1.0);
    const uint64_t bits = __builtin_bit_cast(uint64_t, p);
    const uint32_t k = (uint32_t)__builtin_bit_cast(uint64_t, t);
    const uint32_t high = (uint32_t)(bits >> 32) + (k << 20);
    return __builtin_bit_cast(double, (uint64_t)high << 32 | (uint32_t)bits);
}
// 2^y; 0 below the floor (a masked score's exponent is -inf).
__device__ __forceinline__ double pow2_or_zero(double y) {
    const double v = pow2(fmax(y, kFloor), 1.0);
    return y > kFloor ? v : 0.0;
}

// log2 of x > 0: float32's logarithm of the mantissa, and one step from what 2 to that power leaves of it.
__device__ __forceinline__ double log2_of(double x) {
    const int e = __builtin_amdgcn_frexp_exp(x);
    const double m = __builtin_amdgcn_frexp_mant(x);  // [1/2, 1)
    const double guess = (double)s_lg2((float)m);
    const double z = fma(m, pow2(-guess, 1.0), -1.0);  // some 2^-22
    return (double)e + (guess + z * fma(z, -0.7213475204444817, 1.4426950408889634));
}

// A sum taken to another, no lower reference; an unset one is 0 there.
__device__ __forceinline__ double moved(Sum a, double ref, double c) {
    return a.ref == ref ? a.s : a.s * pow2_or_zero((a.ref - ref) * c);
}
__device__ __forceinline__ Sum join(Sum a, Sum b, double c) {
    const double ref = fmax(a.ref, b.ref);
    return {ref, moved(a, ref, c) + moved(b, ref, c)};
}

// Whether row i is one that a request looks at.  All lanes of a wave, i the same in each.
__device__ __forceinline__ bool row_counts(const VfArgs& A, int64_t i, int lane) {
    const int64_t lowest = A.starts[0], end = A.starts[A.b], before = A.tokens[i > 0 ? i - 1 : 0];
    if (i < lowest || i >= end) return false;
    if (i == 0 || before >= 0) return true;  // (row 0 is the first of its request, also where that starts below 0)
    // behind a row without a drafted token only a request's first row counts: a search by 64 at a time
    int64_t lo = 0, size = A.b;
    while (size > 64) {
        const int64_t step = (size + 63) / 64, at = lo + lane * step;
        const uint64_t mask = __ballot(at < lo + size && A.starts[min(at, A.b)] <= i);
        const int below = __popcll(mask);
        if (below == 0) return false;
        const int64_t rest = size - (int64_t)(below - 1) * step;
        lo += (int64_t)(below - 1) * step;
        size = min(step, rest);
    }
    return __ballot(lane < size && A.starts[min(lo + lane, A.b)] == i) != 0;
}

// 2^(c (x - top)) with the difference taken of the scaled values (exact products: one rounding, that of the difference).
__device__ __forceinline__ float ex2_below(float x, float top, float scale, float c) { return s_ex2(fmaf(x, scale, -(top * scale)) * c); }
// S for the reference M to the same for top >= M.
__device__ __forceinline__ float rescaled(float S, float M, float top, float scale, float c) { return S * ex2_below(M, top, scale, c); }

// Sums of the rows' exponentials in float32: a row, or a part of one, per W waves, each thread with a running maximum
// that it moves once per kVfVecs loads.  (A NaN or +inf score makes the sum NaN by itself.)  Bound by memory: 512 rows
// of 131072 bf16 take 26 us, 5.2 TB/s; in float64 they took 59, bound by 17 instructions per score of 5 to 6 cycles each.
template <class T, int W>
__global__ __launch_bounds__(kBlock) void k_verify_sums(VfArgs A) {
    using E = typename T::type;
    constexpr int VE = Run16<T>::n, kThreads = W * 64, kRows = kBlock / kThreads, NV = kVfVecs, kStep = kThreads * NV;
    __shared__ float red[kBlock / 64][2];
    const int t = threadIdx.x % kThreads, lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int slot = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    // the grid's second dimension: parts of a row, of the target's and then of the draft's
    const int kind = blockIdx.y >= (unsigned)A.splits, split = (int)blockIdx.y - kind * A.splits;
    const bool draft = kind == 1;
    const float c = draft ? A.cqf : A.cf, scale = draft ? A.scale_q : A.scale;
    for (int64_t i = (int64_t)blockIdx.x * kRows + slot; i < A.n; i += (int64_t)gridDim.x * kRows) {
        const E* row = static_cast<const E*>(draft ? A.q : A.s) + i * (draft ? A.ldq : A.ld);
        const int runs = A.m / VE, tail = A.m - runs * VE;
        const int v0 = split * A.cut, v1 = min(runs, v0 + A.cut);
        const int blocks = v1 > v0 ? (v1 - v0 + kStep - 1) / kStep : 0;
        Run16<T> next[NV], v[NV];
        auto fetch = [&](int b) {
#pragma unroll
            for (int q = 0; q < NV; ++q) next[q].get(row + (int64_t)min(v0 + b * kStep + q * kThreads + t, v1 - 1) * VE);
        };
        if (draft && A.tokens[i] < 0) continue;  // (such a row of the draft need not be there)
        if (blocks > 0) fetch(0);                // (before it is known whether the row counts)
        if (!row_counts(A, i, lane)) continue;
        float M = kNegBig, S = 0.0f;  // (M starts above -inf)
        if (split == 0 && t < tail) {
            const float x = T::to(row[runs * VE + t]);
            M = fmaxf(M, x);
            S = ex2_below(x, M, scale, c);
        }
        for (int b = 0; b < blocks; ++b) {
#pragma unroll
            for (int q = 0; q < NV; ++q) v[q] = next[q];
            if (b + 1 < blocks) {
                fetch(b + 1);
            } else {
#pragma unroll
                for (int q = 0; q < NV; ++q)
                    if (v0 + b * kStep + q * kThreads + t >= v1) v[q].fill(T::kNegInfBits);
            }
            float top = M;
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int e = 0; e < VE; ++e) top = fmaxf(top, v[q].at(e));
            S = rescaled(S, M, top, scale, c);
            M = top;
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int e = 0; e < VE; ++e) s += ex2_below(v[q].at(e), M, scale, c);
            S += s;
        }
        float top = lanes_max<64>(M);
        if (W > 1) {
            __syncthreads();
            if (lane == 0) red[wave][0] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < W; ++w) top = fmaxf(top, red[w][0]);
        }
        S = lanes_sum<64>(rescaled(S, M, top, scale, c));
        if (W > 1) {
            if (lane == 0) red[wave][1] = S;
            __syncthreads();
            S = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) S += red[w][1];
        }
        if (t == 0) A.sums[(i * 2 + kind) * A.splits + split] = {(double)top, (double)S};
    }
}

// A row's reference and the log2 of its sum; log2 of a column's probability.
struct RowLog {
    double ref, log_sum;  // -inf: no unmasked entry; NaN: a NaN or +inf score
};
__device__ __forceinline__ double column_log(float s, double c, const RowLog& r) {
    if (r.log_sum != r.log_sum) return r.log_sum;
    return s == -INFINITY ? -(double)INFINITY : fma((double)s - r.ref, c, -r.log_sum);
}

struct Rows {
    int64_t lo, hi;
};
__device__ __forceinline__ Rows rows_of(const VfArgs& A, int64_t r) {
    const int64_t lo = min(max(A.starts[r], (int64_t)0), A.n), hi = min(max(A.starts[r + 1], lo), A.n);
    return {lo, hi};
}

struct Look {
    RowLog row[2][64];
    Draw draw;
    double part[kBlock / 64];
    int stop, none, again;  // in a block of 64 rows: the first that is not taken, that has no drafted token (64: not
                            // there); one to be summed again (-1: none)
};

// A row's log2 sum in float64, by a whole workgroup; ref is the row's largest score.
template <class T>
__device__ double exact_log(const void* m, int64_t ld, int64_t i, int cols, double c, double ref, double* part) {
    using E = typename T::type;
    constexpr int VE = Run16<T>::n;
    const E* row = static_cast<const E*>(m) + i * ld;
    double sum = 0.0;
    Run16<T> v;
#pragma unroll 1
    for (int q = threadIdx.x; q < cols / VE; q += kBlock) {
        v.get(row + (int64_t)q * VE);
#pragma unroll
        for (int e = 0; e < VE; ++e) sum += pow2_or_zero(((double)v.at(e) - ref) * c);
    }
    const int j = cols / VE * VE + threadIdx.x;
    if (j < cols) sum += pow2_or_zero(((double)T::to(row[j]) - ref) * c);
    sum = lanes_sum<64>(sum);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kBlock / 64; ++w) sum += part[w];
    return log2_of(sum);
}

// Where a request stops, by a whole workgroup: the first row whose token is not taken or that has none.  64 rows at a
// time: A.width lanes join the parts of a row's sum, then a wave has a row per lane.  With write, the request's outputs
// but what is drawn; the row where it stops keeps its drafted token until then, for the other workgroups that look at it.
template <class T>
__device__ Draw look(const VfArgs& A, int64_t r, bool write, Look& L) {
    using E = typename T::type;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64, kinds = A.q ? 2 : 1;
    const Rows R = rows_of(A, r);
    Draw d{0.0, 0.0, 0.0, 0.0, -1, -1, 0};
    bool stopped = false, ended = false;
    for (int64_t i0 = R.lo; i0 < R.hi; i0 += 64) {
        const int rows = (int)min((int64_t)64, R.hi - i0);
        const int64_t i = i0 + lane;
        const bool on = wave == 0 && lane < rows;
        int64_t token = 0;
        float s = 0.0f, q = 0.0f, u = 0.0f;
        bool known = false;  // a token of the vocabulary
        if (on) {
            token = A.tokens[i];
            u = A.u_accept[i];
            known = token >= 0 && token < A.m;
            if (known) s = T::to(static_cast<const E*>(A.s)[i * A.ld + token]);
            if (known && A.q) q = T::to(static_cast<const E*>(A.q)[i * A.ldq + token]);
        }
        // (rows behind one without a drafted token, and draft rows of one, have no sums and are not looked at)
        for (int item = tid / A.width; item < rows * kinds; item += kBlock / A.width) {
            const int row = item / kinds, kind = item % kinds, part = tid % A.width;
            const double c = kind ? A.cq : A.c;
            const Sum* p = A.sums + ((i0 + row) * 2 + kind) * A.splits;
            Sum sum = part < A.splits ? p[part] : Sum{kUnset, 0.0};
            for (int k = part + A.width; k < A.splits; k += A.width) sum = join(sum, p[k], c);
            double ref = sum.ref;
            for (int o = 1; o < A.width; o *= 2) ref = fmax(ref, __shfl_xor(ref, o));
            double all = moved(sum, ref, c);
            for (int o = 1; o < A.width; o *= 2) all += __shfl_xor(all, o);
            if (part == 0) L.row[kind][row] = {ref, all == 0.0 ? -(double)INFINITY : all != all ? all : log2_of(all)};
        }
        uint64_t exact = 0;  // rows whose sums were taken again
        for (int tries = 0; tries <= 64; ++tries) {  // (each row is summed again once at most)
            __syncthreads();
            if (wave == 0) {
                const RowLog P = L.row[0][lane], Q = L.row[A.q ? 1 : 0][lane];
                const double lp = known ? column_log(s, A.c, P) : P.log_sum == P.log_sum ? -(double)INFINITY : P.log_sum;
                const double lq = !A.q ? 0.0 : known ? column_log(q, A.cq, Q) : Q.log_sum;
                // p(x) / q(x), at most 2; NaN where one of the rows holds a NaN or +inf
                const double quotient = lp != lp || lq != lq ? (double)NAN
                                        : lp < kFloor        ? 0.0
                                        : lq < kFloor        ? 2.0
                                                             : pow2_or_zero(fmin(lp - lq, 1.0));
                const bool taken = token >= 0 && (double)u < quotient && quotient > 0.0;
                const bool near = token >= 0 && !(exact >> lane & 1) && quotient > 0.0 &&
                                  fabs((double)u - quotient) <= A.doubt * quotient;
                const uint64_t stops = __ballot(on && !taken), nears = __ballot(on && near), nones = __ballot(on && token < 0);
                const int stop = stops ? __ffsll((unsigned long long)stops) - 1 : 64;
                const int none = nones ? __ffsll((unsigned long long)nones) - 1 : 64;
                const int first_near = nears ? __ffsll((unsigned long long)nears) - 1 : 64;
                const int again = !stopped && nears && first_near <= stop ? first_near : -1;
                if (lane == 0) L.again = again;
                if (again < 0) {
                    if (lane == stop) {
                        const bool with_q = A.q && token >= 0 && !(Q.log_sum == -(double)INFINITY);
                        const double gap = P.log_sum - Q.log_sum;  // (of sums from 1 to m, where there is something to draw)
                        const double rho = !with_q ? 0.0 : gap == gap ? pow2(fmin(fmax(gap, -64.0), 64.0), 1.0) : gap;
                        L.draw = {P.ref, P.log_sum, Q.ref, rho, i, A.q || !known ? -1 : token, with_q};
                    }
                    if (lane == 0) L.stop = stop, L.none = none;
                    if (write && on) {
                        const bool emits = !stopped && lane < stop;
                        if (stopped || lane > stop) A.out_tokens[i] = -1;
                        if (emits) A.out_tokens[i] = token;
                        A.ratio[i] = ended || lane >= none ? 0.0f : quotient > 1.0 ? 1.0f : (float)quotient;
                        A.logp[i] = emits ? (float)(lp * 0.6931471805599453094) : 0.0f;
                    }
                }
            }
            __syncthreads();
            const int row = L.again;
            if (row < 0) break;
            exact |= 1ull << row;
            for (int kind = 0; kind < kinds; ++kind) {
                const double ref = L.row[kind][row].ref;
                const double log_sum = exact_log<T>(kind ? A.q : A.s, kind ? A.ldq : A.ld, i0 + row, A.m, kind ? A.cq : A.c, ref, L.part);
                if (tid == 0 && L.row[kind][row].log_sum > -(double)INFINITY) L.row[kind][row].log_sum = log_sum;
            }
        }
        if (!stopped && L.stop < 64) {
            d = L.draw;
            stopped = true;
        }
        ended = ended || L.none < 64;
        __syncthreads();
        if (stopped && !write) break;
    }
    if (write && tid == 0) {
        A.accepted[r] = (int32_t)((stopped ? d.row : R.hi) - R.lo);
        A.next[r] = -1;
    }
    return d;
}

// The same in scalar registers; all threads have the same.
__device__ __forceinline__ Draw uniform(const Draw& d) {
    struct Words {
        int w[sizeof(Draw) / 4];
    };
    Words x = __builtin_bit_cast(Words, d);
#pragma unroll
    for (int& w : x.w) w = __builtin_amdgcn_readfirstlane(w);
    return __builtin_bit_cast(Draw, x);
}

__device__ __forceinline__ bool drawable(const Draw& d) {
    return d.row >= 0 && d.log_p > -(double)INFINITY && (!d.with_q || d.rho == d.rho);  // (NaN: no)
}

// The exponential of a score over its row's largest, floor / c below it: 2^-1000, where that is told apart later; or 0.
__device__ __forceinline__ double exp_near(float s, double ref, double c, double floor) {
    return pow2(fmax((double)s - ref, floor), c);
}
__device__ __forceinline__ double exp_of(float s, double ref, double c, double floor) {
    return (double)s - ref > floor ? exp_near(s, ref, c, floor) : 0.0;
}

// Sums over a chunk, by a wave: of e, of h, of max(e - rho h, 0) and of h where that is positive (without q: of e).  With
// near > 0 the second is negative where an entry has |e - rho h| <= near h.
template <class T>
__device__ __forceinline__ void chunk_sums(const VfArgs& A, const Draw& d, double near, int chunk, int lane, double* out) {
    using E = typename T::type;
    constexpr int VE = Run16<T>::n;
    const int start = chunk * A.chunk_len, j0 = start + lane * VE, size = min(A.chunk_len, A.m - start);
    const E* s = static_cast<const E*>(A.s) + d.row * A.ld + j0;
    const E* q = static_cast<const E*>(d.with_q ? A.q : A.s) + d.row * (d.with_q ? A.ldq : A.ld) + j0;
    double e = 0.0, h = 0.0, rest = 0.0, hot = 0.0, gap = 1.0;
    auto add_both = [&](float x, float y) {
        const double a = exp_near(x, d.ref_p, A.c, A.floor), b = exp_near(y, d.ref_q, A.cq, A.floor_q), w = fma(-d.rho, b, a);
        e += a;
        h += b;
        const double over = fmin(fmax(w * 0x1p1020, 0.0), 1.0);  // 1 where w > 0 (one instruction, where a choice takes three)
        rest = fma(w, over, rest);
        hot = fma(b, over, hot);
        gap = fmin(gap, fma(-near, b, fabs(w)));
    };
    const int whole = size / (64 * VE) * (64 * VE);  // entries in whole runs of all lanes
    // (the loops are not unrolled: a wave has few chunks, and cold code takes longer to fetch than to run)
    if (d.with_q) {
        Run16<T> a, b, a1, b1;
        if (whole > 0) a1.get(s), b1.get(q);
#pragma unroll 1
        for (int at = 0; at < whole; at += 64 * VE) {
            a = a1;
            b = b1;
            const int next = at + 64 * VE < whole ? at + 64 * VE : at;
            a1.get(s + next);
            b1.get(q + next);
#pragma unroll
            for (int c = 0; c < VE; ++c) add_both(a.at(c), b.at(c));
        }
#pragma unroll 1
        for (int j = whole + lane; j < size; j += 64) add_both(T::to(s[j - lane * VE]), T::to(q[j - lane * VE]));
    } else {
        double floor = A.floor;
        asm("" : "+v"(floor));  // (in vector registers, where the comparison takes it as it is: 17 us against 18 for 64 rows of 131072)
        auto add_one = [&](float x, int j) { e += j == d.out ? 0.0 : exp_near(x, d.ref_p, A.c, floor); };
        Run16<T> a, a1;
        if (whole > 0) a1.get(s);
#pragma unroll 1
        for (int at = 0; at < whole; at += 64 * VE) {
            a = a1;
            a1.get(s + (at + 64 * VE < whole ? at + 64 * VE : at));
#pragma unroll
            for (int c = 0; c < VE; ++c) add_one(a.at(c), j0 + at + c);
        }
#pragma unroll 1
        for (int j = whole + lane; j < size; j += 64) add_one(T::to(s[j - lane * VE]), start + j);
    }
    if (!d.with_q) {
        e = lanes_sum<64>(e);
        if (lane == 0) out[0] = e;
        return;
    }
    // four sums over the lanes at once: half of the lanes take two of them, a quarter one each
    const bool high = lane & 32, odd = lane & 16;
    double x0 = high ? rest : e, x1 = high ? hot : h;
    x0 += __shfl_xor(high ? e : rest, 32);
    x1 += __shfl_xor(high ? h : hot, 32);
    double x = odd ? x1 : x0;
    x += __shfl_xor(odd ? x0 : x1, 16);
    for (int o = 8; o > 0; o /= 2) x += __shfl_xor(x, o);
    if (near > 0.0 && __any(gap <= 0.0) && lane / 16 == 1) x = -x;
    if ((lane & 15) == 0) out[lane / 16] = x;
}

// Inclusive sums over the workgroup's threads; the last is the same in every thread.
__device__ __forceinline__ double block_scan(double x, double* lds, double& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    for (int o = 1; o < 64; o *= 2) {
        const double low = __shfl_up(x, o);
        if (lane >= o) x += low;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = x;
    __syncthreads();
    double before = 0.0;
    total = 0.0;
#pragma unroll
    for (int w = 0; w < kBlock / 64; ++w) {
        if (w == wave) before = total;
        total += lds[w];
    }
    return before + x;
}

// Sums of x and of y over the workgroup's threads, the same in every thread.
__device__ __forceinline__ void block_sums(double x, double y, double (*lds)[2], double& sum_x, double& sum_y) {
    x = lanes_sum<64>(x);
    y = lanes_sum<64>(y);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64][0] = x, lds[threadIdx.x / 64][1] = y;
    __syncthreads();
    sum_x = sum_y = 0.0;
#pragma unroll
    for (int w = 0; w < kBlock / 64; ++w) sum_x += lds[w][0], sum_y += lds[w][1];
}

struct Pick {
    double scan[kBlock / 64], two[kBlock / 64][2], prior, room;
    uint64_t over[kBlock / 64], some[kBlock / 64];
};

// Of the threads for which over holds the first, else the last of those for which some does (-1: none), in every thread.
__device__ __forceinline__ int first_over(bool over, bool some, Pick& L, bool& found) {
    const uint64_t a = __ballot(over), b = __ballot(some);
    const int wave = threadIdx.x / 64;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) L.over[wave] = a, L.some[wave] = b;
    __syncthreads();
    int first = -1, last = -1;
#pragma unroll
    for (int w = 0; w < kBlock / 64; ++w) {
        const uint64_t x = L.over[w], y = L.some[w];
        if (first < 0 && x) first = w * 64 + __ffsll((unsigned long long)x) - 1;
        if (y) last = w * 64 + 63 - __clzll((long long)y);
    }
    found = first >= 0;
    return found ? first : last;
}

// The draw of a request from its chunks' sums, by a whole workgroup.  False where it is nearer to a border than the marked
// chunks' sums allow: they are to be taken again, with rho; after that (exact) they are as good as the others.
template <class T>
__device__ bool draw(const VfArgs& A, int64_t r, Draw d, bool exact, double& rho, Pick& L) {
    using E = typename T::type;
    constexpr int kPer = kVfChunkMost / kBlock;
    const int tid = threadIdx.x;
    const double* sums = A.chunk + r * A.chunks * 4;
    if (tid == 0) A.out_tokens[d.row] = -1;  // (until the draw)
    double shift = 0.0, all = 0.0;  // rho0 - rho; the sum of e
    double slack = 0.0;             // what a sum of chunks' weights is off by at most
    if (d.with_q) {
        double h = 0.0;
        for (int k0 = 0; k0 < A.chunks; k0 += kBlock) {
            const int k = k0 + tid;
            double e_here, h_here;
            block_sums(k < A.chunks ? sums[4 * k] : 0.0, k < A.chunks ? fabs(sums[4 * k + 1]) : 0.0, L.two, e_here, h_here);
            all += e_here;
            h += h_here;
        }
        shift = d.rho - all / h;
        rho = d.rho = all / h;
        slack = exact ? 0.0 : fabs(shift) * h;
    }
    double mine = 0.0, upto = 0.0, here, total = 0.0;
    auto weight_of = [&](int k) {
        if (k >= A.chunks) return 0.0;
        const double w = d.with_q ? fma(shift, sums[4 * k + 3], sums[4 * k + 2]) : sums[4 * k];
        return w > kNothing ? w : 0.0;
    };
    // only the marked chunks' weights are off
    auto sum_marked = [&]() {
        double h = 0.0;
        for (int k0 = 0; k0 < A.chunks; k0 += kBlock) {
            const double marked = k0 + tid < A.chunks ? fmax(-sums[4 * (k0 + tid) + 1], 0.0) : 0.0;
            block_scan(marked, L.scan, here);
            h += here;
        }
        slack = fabs(shift) * h;
    };
    for (int k0 = 0; k0 < A.chunks; k0 += kBlock) {
        mine = weight_of(k0 + tid);
        upto = block_scan(mine, L.scan, here);
        total += here;
    }
    if (d.with_q && !(total - slack > 0x1p-40 * all)) {
        if (slack > 0.0) return false;
        // p - q leaves nothing (q = p, but for roundings): the draw is from p itself
        d.with_q = 0;
        total = all;
        if (A.chunks <= kBlock) {
            mine = weight_of(tid);
            upto = block_scan(mine, L.scan, here);
        }
    }
    if (!(total > 0.0)) {
        // all of p is at the column left out: that is drawn
        if (tid == 0 && d.out >= 0) {
            A.next[r] = A.out_tokens[d.row] = d.out;
            A.logp[d.row] = 0.0f;
        }
        return true;
    }
    // the first chunk whose sum with those before exceeds the mark; where none does (u_sample = 1), the last whose sum
    // is more than roundings
    const double mark = (double)fminf(fmaxf(A.u_sample[r], 0.0f), 1.0f) * total;
    int at = -1;
    double before = 0.0;
    bool found = false;
    for (int k0 = 0; k0 < A.chunks && !found; k0 += kBlock) {
        if (A.chunks > kBlock) {  // (else both are there)
            mine = weight_of(k0 + tid);
            upto = before + block_scan(mine, L.scan, here);
            before += here;
        }
        const int hit = first_over(mine > 0.0 && upto > mark, mine > 0x1p-44 * all, L, found);
        if (hit >= 0) at = k0 + hit;
        if (tid == hit) L.prior = upto - mine;
    }
    __syncthreads();
    const double prior = at < 0 ? total : L.prior;
    if (at < 0) at = A.chunks - 1;
    // inside it, each thread some neighbouring entries
    const E* s = static_cast<const E*>(A.s) + d.row * A.ld;
    const E* t = static_cast<const E*>(d.with_q ? A.q : A.s) + d.row * (d.with_q ? A.ldq : A.ld);
    const int j0 = at * A.chunk_len + tid * kPer, end = min(A.m, (at + 1) * A.chunk_len);
    double w[kPer];
    mine = 0.0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) w[e] = 0.0;
    if (j0 < end) {  // (a short chunk leaves waves without)
        E a[kPer], b[kPer];
        if (j0 + kPer <= end) {
            __builtin_memcpy(a, s + j0, sizeof(a));
            __builtin_memcpy(b, t + j0, sizeof(b));
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                a[e] = s[min(j0 + e, end - 1)];
                b[e] = t[min(j0 + e, end - 1)];
            }
        }
        // (as in the chunk's sums: what counts there counts here)
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const double p = j0 + e == d.out ? 0.0 : exp_of(T::to(a[e]), d.ref_p, A.c, A.floor);
            const double q = d.with_q ? exp_of(T::to(b[e]), d.ref_q, A.cq, A.floor_q) : 0.0;
            w[e] = j0 + e < end ? fmax(fma(-d.rho, q, p), 0.0) : 0.0;
            mine += w[e];
        }
    }
    double run = prior + (block_scan(mine, L.scan, here) - mine), room = -1.0;
    int first = -1, possible = -1;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const double below = run;
        run += w[e];
        if (w[e] > 0.0) {
            possible = j0 + e;
            if (run > mark && first < 0) {
                first = j0 + e;
                room = fmin(mark - below, run - mark);
            }
        }
    }
    const int hit = first_over(first >= 0, possible >= 0, L, found);
    if (slack > 0.0) {
        // the distance to the nearest border against what the mark and the sum before may be off by
        if (tid == hit) L.room = room;
        __syncthreads();
        const double least = hit < 0 ? -1.0 : L.room;
        if (!(least > 2.0 * slack)) {
            sum_marked();
            if (slack > 0.0 && !(least > 2.0 * slack)) return false;
        }
    }
    if (tid == hit) {
        const int token = found ? first : possible;  // (roundings: the last possible entry of the chunk)
        A.next[r] = token;
        A.out_tokens[d.row] = token;
        A.logp[d.row] = (float)(column_log(T::to(s[token]), A.c, {d.ref_p, d.log_p}) * 0.6931471805599453094);
    }
    __syncthreads();
    return true;
}

// Where each request stops and the sums of the chunks of what it draws from: a wave per chunk, A.parts workgroups per
// request; one that has all the chunks (ALONE) draws too.  Bound by the issue of some 40 float64 instructions per entry: 64
// requests over 131072 columns take 21 us, 5 of them to look where each stops.
template <class T, bool ALONE>
__global__ __launch_bounds__(kBlock, 4) void k_verify_chunks(VfArgs A) {
    __shared__ Look L;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    for (int64_t item = blockIdx.x; item < A.b * A.parts; item += gridDim.x) {
        const int64_t r = item / A.parts;
        const int part = (int)(item % A.parts);
        Draw d = uniform(look<T>(A, r, part == 0, L));
        if (!ALONE && part == 0 && threadIdx.x == 0) A.draw[r] = d;
        if (!drawable(d)) {
            if (ALONE && d.row >= 0 && threadIdx.x == 0) A.out_tokens[d.row] = -1;
            continue;
        }
        for (double near = A.doubt * d.rho;; near = 0.0) {
            for (int k = part * (kBlock / 64) + wave; k < A.chunks; k += A.parts * (kBlock / 64))
                chunk_sums<T>(A, d, near, k, lane, A.chunk + (r * A.chunks + k) * 4);
            if constexpr (ALONE) {
                __shared__ Pick P;
                __syncthreads();
                double rho = d.rho;
                if (draw<T>(A, r, d, near == 0.0, rho, P)) break;
                d.rho = rho;  // (all chunks again)
            } else {
                break;
            }
        }
    }
}

// Bound by the latency of its loads and of three sums over the workgroup: 7 us for one request, 9 for 64.
template <class T>
__global__ __launch_bounds__(kBlock) void k_verify_draw(VfArgs A) {
    __shared__ Pick P;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    for (int64_t r = blockIdx.x; r < A.b; r += gridDim.x) {
        const Draw d = uniform(A.draw[r]);
        if (!drawable(d)) {
            if (d.row >= 0 && threadIdx.x == 0) A.out_tokens[d.row] = -1;
            continue;
        }
        double* sums = A.chunk + r * A.chunks * 4;
        Draw again = d;
        for (bool exact = false; !draw<T>(A, r, d, exact, again.rho, P); exact = true) {
            // the marked chunks, which need no correction then
            __syncthreads();
            for (int k = wave; k < A.chunks; k += kBlock / 64) {
                if (!(sums[4 * k + 1] < 0.0)) continue;
                chunk_sums<T>(A, again, 0.0, k, lane, sums + 4 * k);
                if (lane == 48) sums[4 * k + 3] = 0.0;  // (the lane that wrote it)
            }
            __syncthreads();
        }
    }
}

// ----- greedy: p is one at the row's largest score, the first of equal ones -----------------
// Part: (ordered score, ~column) of the largest entry; 0: no unmasked entry; all ones: a NaN or +inf score.
// Bound by memory: 320 rows of 65536 f16 take 8 us, 5.2 TB/s.
template <class T, int W>
__global__ __launch_bounds__(kBlock) void k_verify_best(VfArgs A) {
    using E = typename T::type;
    constexpr int VE = Run16<T>::n, kThreads = W * 64, kRows = kBlock / kThreads, NV = kVfVecs, kStep = kThreads * NV;
    __shared__ uint64_t red[kBlock / 64];
    const int t = threadIdx.x % kThreads, lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int slot = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    uint64_t* best_of = reinterpret_cast<uint64_t*>(A.sums);
    const int split = (int)blockIdx.y;
    for (int64_t i = (int64_t)blockIdx.x * kRows + slot; i < A.n; i += (int64_t)gridDim.x * kRows) {
        if (!row_counts(A, i, lane)) continue;
        const E* row = static_cast<const E*>(A.s) + i * A.ld;
        const int runs = A.m / VE, tail = A.m - runs * VE;
        const int v0 = split * A.cut, v1 = min(runs, v0 + A.cut);
        float best = -INFINITY;
        int at = -1;  // run of the largest; its entries are looked at again below
        auto see = [&](float top, int v) {
            // a NaN takes the lead and keeps it
            if (!(top <= best) && best == best) best = top, at = v;
        };
        for (int b = v0 + t; b < v1; b += kStep) {
            Run16<T> v[NV];
#pragma unroll
            for (int q = 0; q < NV; ++q) v[q].get(row + (int64_t)min(b + q * kThreads, v1 - 1) * VE);
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                float top = v[q].at(0);
#pragma unroll
                for (int e = 1; e < VE; ++e) top = __builtin_elementwise_maximum(top, v[q].at(e));
                see(top, min(b + q * kThreads, v1 - 1));
            }
        }
        int column = at * VE;
        if (at >= 0) {
            Run16<T> v;
            v.get(row + (int64_t)at * VE);
#pragma unroll
            for (int e = VE - 1; e >= 0; --e)
                if (v.at(e) == best) column = at * VE + e;
        }
        if (split == 0 && t < tail) {
            const float x = T::to(row[runs * VE + t]);
            see(x, runs);
            if (at == runs) column = runs * VE + t;
        }
        uint64_t key = at < 0 ? 0 : !(best < INFINITY) ? ~0ull : (uint64_t)ordered(best) << 32 | (uint32_t)~column;
        for (int o = 1; o < 64; o *= 2) {
            const uint64_t other = (uint64_t)__shfl_xor((unsigned long long)key, o);
            key = key > other ? key : other;
        }
        if (W > 1) {
            __syncthreads();
            if (lane == 0) red[wave] = key;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < W; ++w) key = key > red[w] ? key : red[w];
        }
        if (t == 0) best_of[i * A.splits + split] = key;
    }
}

// A wave per request.
__global__ __launch_bounds__(kBlock) void k_verify_greedy(VfArgs A) {
    const int lane = threadIdx.x & 63;
    const uint64_t* best_of = reinterpret_cast<const uint64_t*>(A.sums);
    for (int64_t r = (int64_t)blockIdx.x * (kBlock / 64) + threadIdx.x / 64; r < A.b; r += (int64_t)gridDim.x * (kBlock / 64)) {
        const Rows R = rows_of(A, r);
        int64_t stop = -1, token = -1;
        bool ended = false;
        for (int64_t i0 = R.lo; i0 < R.hi; i0 += 64) {
            const int64_t i = i0 + lane;
            const bool on = i < R.hi;
            const int64_t drafted = on ? A.tokens[i] : 0;
            const uint64_t none = __ballot(on && drafted < 0);
            const int first_none = none ? __ffsll((unsigned long long)none) - 1 : 64;
            const bool in = on && !ended && lane <= first_none;
            uint64_t key = 0;
            if (in)
                for (int k = 0; k < A.splits; ++k) key = max(key, best_of[i * A.splits + k]);
            const bool bad = key == ~0ull;
            const int64_t best = key == 0 || bad ? -1 : (int64_t)(uint32_t)~(uint32_t)key;
            const bool hit = drafted >= 0 && drafted == best;
            if (stop < 0) {
                const uint64_t mask = __ballot(in && !hit);
                if (mask) {
                    const int at = __ffsll((unsigned long long)mask) - 1;
                    stop = i0 + at;
                    token = __shfl((long long)best, at);
                }
            }
            if (on) {
                A.out_tokens[i] = ended ? -1 : stop < 0 || i < stop ? drafted : i == stop ? token : -1;
                A.ratio[i] = !in || drafted < 0 ? 0.0f : bad ? NAN : hit ? 1.0f : 0.0f;
                A.logp[i] = 0.0f;
            }
            ended = ended || none != 0;
        }
        if (lane == 0) {
            A.accepted[r] = (int32_t)((stop < 0 ? R.hi : stop) - R.lo);
            A.next[r] = token;
        }
    }
}

// ----- host side ------------------------------------------------------------------------
// A row of two blocks at most is one wave's.
bool one_wave(int es, int64_t m) { return m / (16 / es) <= 2 * 64 * kVfVecs; }

struct VfPlan {
    int splits, cut, chunk_len, chunks, parts;
    size_t sums, chunk, draw, total;
};

VfPlan vf_plan(int es, int64_t n, int64_t m, int64_t b) {  // (the same with and without draft scores)
    VfPlan P{};
    const int64_t runs = std::max<int64_t>(1, m * es / 16);
    const int64_t most = std::max<int64_t>(1, std::min((kVfFill + n - 1) / std::max<int64_t>(n, 1), runs / kVfCutMin));
    const int64_t cut = (runs + most - 1) / most;
    P.cut = (int)cut;
    P.splits = (int)((runs + cut - 1) / cut);
    // shorter chunks where they leave waves idle
    for (P.chunk_len = 512; P.chunk_len < kVfChunkMost && b * m > (int64_t)P.chunk_len * 4 * kVfFill; P.chunk_len *= 2) {}
    P.chunks = (int)((m + P.chunk_len - 1) / P.chunk_len);
    const int64_t whole = (P.chunks + 3) / 4;
    P.parts = (int)std::max<int64_t>(1, std::min<int64_t>(whole, (kVfFill + b - 1) / std::max<int64_t>(b, 1)));
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    P.chunk = up((size_t)n * 2 * (size_t)P.splits * sizeof(Sum));
    P.draw = P.chunk + up((size_t)b * (size_t)P.chunks * 4 * sizeof(double));
    P.total = P.draw + up((size_t)b * sizeof(Draw)) + 256;
    return P;
}

template <class T>
hipError_t verify(const VfArgs& A, bool greedy, hipStream_t s) {
    const bool wave = one_wave((int)sizeof(typename T::type), A.m);
    const int kinds = A.q ? 2 : 1, rows = wave ? kBlock / 64 : 1;
    const dim3 grid((unsigned)std::min<int64_t>((A.n + rows - 1) / rows, kVfGrid), (unsigned)(A.splits * kinds));
    hipError_t e;
    if (greedy) {
        if (A.n == 0)
            ;
        else if (wave)
            hipLaunchKernelGGL((k_verify_best<T, 1>), grid, dim3(kBlock), 0, s, A);
        else
            hipLaunchKernelGGL((k_verify_best<T, 4>), grid, dim3(kBlock), 0, s, A);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(k_verify_greedy, dim3((unsigned)std::min<int64_t>((A.b + 3) / 4, kVfGrid)), dim3(kBlock), 0, s, A);
        return hipGetLastError();
    }
    if (A.n == 0)
        ;
    else if (wave)
        hipLaunchKernelGGL((k_verify_sums<T, 1>), grid, dim3(kBlock), 0, s, A);
    else
        hipLaunchKernelGGL((k_verify_sums<T, 4>), grid, dim3(kBlock), 0, s, A);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    auto chunks = A.parts == 1 ? k_verify_chunks<T, true> : k_verify_chunks<T, false>;
    hipLaunchKernelGGL(chunks, dim3((unsigned)std::min<int64_t>(A.b * A.parts, kVfGrid)), dim3(kBlock), 0, s, A);
    if ((e = hipGetLastError()) != hipSuccess || A.parts == 1) return e;
    hipLaunchKernelGGL((k_verify_draw<T>), dim3((unsigned)std::min<int64_t>(A.b, kVfGrid)), dim3(kBlock), 0, s, A);
    return hipGetLastError();
}

bool good_sizes(int64_t n, int64_t m, int64_t b) {
    return n >= 0 && n <= INT32_MAX && m >= 1 && m <= kVfMaxCols && b >= 0 && b <= INT32_MAX;
}

}  // namespace
}  // namespace sk

using namespace sk;

extern "C" {

size_t sk_scores_verify_workspace_bytes(int32_t dtype, int64_t n, int64_t m, int64_t b) {
    if (dtype != SK_F32 && dtype != SK_BF16 && dtype != SK_F16) return 0;
    return good_sizes(n, m, b) ? vf_plan(elem_size(dtype), n, m, b).total : 0;
}

int sk_scores_verify(const void* scores, int32_t dtype, int64_t n, int64_t m, int64_t ld, float eps, const void* draft,
                     int64_t ld_draft, float eps_draft, const int64_t* tokens, const int64_t* starts, int64_t b,
                     const float* u_accept, const float* u_sample, int32_t* accepted, int64_t* next, int64_t* out_tokens,
                     float* ratio, float* logp, void* ws, size_t ws_bytes, void* stream) {
    int st = check_scores(scores, dtype, n, m, ld);
    if (st) return st;
    if (!good_sizes(n, m, b)) return SK_ERR_SHAPE;
    if (draft && (st = check_scores(draft, dtype, n, m, ld_draft))) return st;
    const bool greedy = eps == 0.0f;
    if (!greedy && (st = check_temperature(eps))) return st;
    if (draft && (st = check_temperature(eps_draft))) return st;
    const VfPlan P = vf_plan(elem_size(dtype), n, m, b);
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < P.total) return SK_ERR_WORKSPACE;
    if (b == 0) return SK_OK;
    if (!starts || !accepted || !next || (!greedy && !u_sample)) return SK_ERR_NULL;
    if (n > 0 && (!tokens || !out_tokens || !ratio || !logp || (!greedy && !u_accept))) return SK_ERR_NULL;
    const int es = elem_size(dtype);
    // (not the draft's rows: which of them are there is not known here)
    const Span inputs[] = {span_of(tokens, n, 8), span_of(starts, b + 1, 8), span_of(scores, n, m, ld, es),
                           span_of(u_accept, greedy ? 0 : n, 4), span_of(u_sample, greedy ? 0 : b, 4)};
    const Span outputs[] = {span_of(out_tokens, n, 8), span_of(accepted, b, 4), span_of(next, b, 8), span_of(ratio, n, 4),
                            span_of(logp, n, 4)};
    for (const Span& in : inputs)
        for (const Span& out : outputs)
            if (meet(in, out) && !(&in == inputs && &out == outputs && out_tokens == tokens)) return SK_ERR_OVERLAP;
    char* base = static_cast<char*>(ws);
    VfArgs A{};
    A.s = scores;
    A.q = greedy ? nullptr : draft;
    A.ld = ld;
    A.ldq = ld_draft;
    A.n = n;
    A.b = b;
    A.m = (int)m;
    A.c = greedy ? 1.0 : 1.4426950408889634074 / (double)eps;
    A.cq = draft ? 1.4426950408889634074 / (double)eps_draft : 1.0;
    A.floor = kFloor / A.c;
    A.floor_q = kFloor / A.cq;
    A.scale = A.c < 1.0 ? 0.5f : 1.0f;  // (from c = 1 on, twice c may leave float32, and an infinite difference is none that counts)
    A.scale_q = A.cq < 1.0 ? 0.5f : 1.0f;
    A.cf = (float)(A.c / A.scale);
    A.cqf = (float)(A.cq / A.scale_q);
    // the float32 sums: an exponent carries 3 u of itself, and as much again by the moves of the maximum, of which the
    // weighted mean is at most ln m; 2 u the exponential; then the additions of a block, of the blocks (with 3 u for each
    // move), lanes and waves
    const int64_t blocks = P.cut / ((one_wave(elem_size(dtype), m) ? 64 : kBlock) * kVfVecs) + 1;
    A.doubt = 2.5 * (6.0 * std::log((double)m) + 60.0 + 4.0 * (double)blocks) * 0x1p-24;
    A.tokens = tokens;
    A.starts = starts;
    A.u_accept = u_accept;
    A.u_sample = u_sample;
    A.accepted = accepted;
    A.next = next;
    A.out_tokens = out_tokens;
    A.ratio = ratio;
    A.logp = logp;
    A.splits = P.splits;
    A.cut = P.cut;
    A.width = 1;
    while (A.width < 64 && A.width < P.splits) A.width *= 2;
    A.chunk_len = P.chunk_len;
    A.chunks = P.chunks;
    A.parts = P.parts;
    A.sums = reinterpret_cast<Sum*>(base + P.sums);
    A.chunk = reinterpret_cast<double*>(base + P.chunk);
    A.draw = reinterpret_cast<Draw*>(base + P.draw);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SK_TRY_LAUNCH(dtype == SK_F32 ? verify<F32>(A, greedy, s) : dtype == SK_BF16 ? verify<Bf16>(A, greedy, s) : verify<F16>(A, greedy, s));
    return SK_OK;
}

}  // extern "C"
