// loss.hpp -- shared by the loss operators (top.hip, distill.hip,
// balance.hip): the workers' rows as one index space, 16-byte row accesses at
// any element alignment, wave and workgroup reductions, and the host checks
// of their arguments.
#pragma once
#include <algorithm>
#include <cmath>

#include "../../include/ga_loss.h"
#include "common.hpp"

namespace ga {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The rows of all workers, one after another: worker w holds rows
// start[w] .. start[w + 1] - 1.
struct RowMap {
    int32_t P;
    int32_t start[GA_MAX_WORKERS + 1];
};

// The worker that holds `row` (wave-uniform): the last one whose start is not
// above it, so workers without rows are passed over.
__device__ __forceinline__ int worker_of(const RowMap& m, int32_t row) {
    int lo = 0, hi = m.P;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (m.start[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ------------------------------------------------------------------ rows
// 16 bytes of a row. Rows start at any multiple of the element size (an odd
// vocabulary, a padded stride): gfx950 takes global accesses of 16 bytes at
// such addresses in one instruction.
typedef unsigned int u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));

typedef __attribute__((address_space(1))) char g_char;

template <ga_dtype DT> struct RowVec;

template <> struct RowVec<GA_F32> {
    static constexpr int kElems = 4;
    static constexpr uint32_t kEmpty = 0xFF800000u;      // -inf
    typedef u32x4_e4 vec;
    typedef __attribute__((address_space(1))) vec g_vec;
    typedef float elem;
    __device__ static __forceinline__ float value(elem x) { return x; }
    __device__ static __forceinline__ elem narrow1(float f) { return f; }
    __device__ static __forceinline__ void widen(uint4 r, float* f) {
        f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
    }
    __device__ static __forceinline__ uint4 narrow(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
    // element e of a vector as raw bits
    __device__ static __forceinline__ void put(uint32_t* w, int e, elem x) { w[e] = __float_as_uint(x); }
};

template <> struct RowVec<GA_BF16> {
    static constexpr int kElems = 8;
    static constexpr uint32_t kEmpty = 0xFF80FF80u;
    typedef u32x4_e2 vec;
    typedef __attribute__((address_space(1))) vec g_vec;
    typedef uint16_t elem;
    __device__ static __forceinline__ float value(elem x) { return __uint_as_float((uint32_t)x << 16); }
    // round to nearest even in one instruction per pair (v_cvt_pk_bf16_f32)
    __device__ static __forceinline__ uint32_t narrow2(float a, float b) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 v = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    __device__ static __forceinline__ elem narrow1(float f) { return (elem)(narrow2(f, 0.0f) & 0xFFFFu); }
    __device__ static __forceinline__ void widen(uint4 r, float* f) {
        f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
        f[4] = bf16_lo(r.z); f[5] = bf16_hi(r.z); f[6] = bf16_lo(r.w); f[7] = bf16_hi(r.w);
    }
    __device__ static __forceinline__ uint4 narrow(const float* f) {
        return make_uint4(narrow2(f[0], f[1]), narrow2(f[2], f[3]), narrow2(f[4], f[5]),
                          narrow2(f[6], f[7]));
    }
    __device__ static __forceinline__ void put(uint32_t* w, int e, elem x) {
        const int s = (e & 1) * 16;
        w[e >> 1] = (w[e >> 1] & ~(0xFFFFu << s)) | ((uint32_t)x << s);
    }
};

// Vector v of a row of n elements; elements past the row's end read as -inf.
template <ga_dtype DT, bool STREAM>
__device__ __forceinline__ uint4 load_row_vec(const void* row, int64_t v, int64_t n) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    const typename R::elem* x = static_cast<const typename R::elem*>(row) + v * E;
    if ((v + 1) * E <= n) {
        const auto* p = (const typename R::g_vec*)x;
        const typename R::vec r = STREAM ? __builtin_nontemporal_load(p) : *p;
        return make_uint4(r.x, r.y, r.z, r.w);
    }
    uint32_t w[4] = {R::kEmpty, R::kEmpty, R::kEmpty, R::kEmpty};
#pragma unroll
    for (int e = 0; e < E; e++)
        if (v * E + e < n) R::put(w, e, x[e]);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <ga_dtype DT>
__device__ __forceinline__ void store_row_vec(void* row, int64_t v, int64_t n, const float* f) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    typename R::elem* x = static_cast<typename R::elem*>(row) + v * E;
    if ((v + 1) * E <= n) {
        const uint4 u = R::narrow(f);
        const typename R::vec r = {u.x, u.y, u.z, u.w};
        __builtin_nontemporal_store(r, (typename R::g_vec*)x);
        return;
    }
#pragma unroll
    for (int e = 0; e < E; e++)
        if (v * E + e < n) x[e] = R::narrow1(f[e]);
}

// A whole vector of a row without a check, `at` bytes (the same for the whole
// wave) and `lane` bytes from its start: one 32-bit register of address, for
// kernels that hold many vectors at once.
template <ga_dtype DT, bool STREAM>
__device__ __forceinline__ uint4 load_whole_vec(const void* row, int64_t at, uint32_t lane) {
    using R = RowVec<DT>;
    const auto* p = (const typename R::g_vec*)((const g_char*)row + at + lane);
    const typename R::vec r = STREAM ? __builtin_nontemporal_load(p) : *p;
    return make_uint4(r.x, r.y, r.z, r.w);
}
template <ga_dtype DT>
__device__ __forceinline__ void store_whole_vec(void* row, int64_t at, uint32_t lane, uint4 u) {
    using R = RowVec<DT>;
    const typename R::vec r = {u.x, u.y, u.z, u.w};
    __builtin_nontemporal_store(r, (typename R::g_vec*)((g_char*)row + at + lane));
}
// Element `tid` of those behind a row's whole vectors, -inf where there is none.
template <ga_dtype DT>
__device__ __forceinline__ float load_last(const void* row, int64_t n, int64_t n_whole, int tid) {
    using R = RowVec<DT>;
    const int64_t at = n_whole * R::kElems + tid;
    const float x = R::value(static_cast<const typename R::elem*>(row)[min(at, n - 1)]);
    return at < n ? x : -INFINITY;
}
// Values kept in registers from one pass over them to the next: what a pass
// made of them is not to be kept as well (the compiler would, and spill).
__device__ __forceinline__ void forget_derived(uint4& r) {
    asm volatile("" : "+v"(r.x), "+v"(r.y), "+v"(r.z), "+v"(r.w));
}
// ------------------------------------------------------------------ reductions
// Over the 2^k lanes that a lane forms a team with (lane index aligned to the
// team): lane permutes of the vector unit, no LDS. Every lane gets the result.
struct OpMax {
    __device__ static __forceinline__ float f(float a, float b) { return fmaxf(a, b); }
};
struct OpSum {
    __device__ static __forceinline__ float f(float a, float b) { return a + b; }
};

template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}

template <int L, class OP> __device__ __forceinline__ float team_reduce(float v) {
    static_assert(L == 1 || L == 2 || L == 4 || L == 8 || L == 16 || L == 32 || L == 64, "team size");
    if (L >= 2) v = OP::f(v, dpp<0xB1>(v));      // quad_perm 1,0,3,2
    if (L >= 4) v = OP::f(v, dpp<0x4E>(v));      // quad_perm 2,3,0,1
    if (L >= 8) v = OP::f(v, dpp<0x141>(v));     // half-row mirror: quads are uniform
    if (L >= 16) v = OP::f(v, dpp<0x140>(v));    // row mirror
    if (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = OP::f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    if (L >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = OP::f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Sum over a workgroup of T threads, in a fixed order; every thread gets it.
// sh: T / 64 doubles.
template <int T> __device__ __forceinline__ double group_sum_f64(double v, double* sh) {
    v = wave_sum_f64(v);
    if (T == 64) return v;
    __syncthreads();                                   // sh may still be read
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < T / 64; i++) t += sh[i];
    return t;
}

// exp2 of the hardware (1 ulp; 0 below the smallest normal number).
__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// A softmax's running maximum m and the sum s of its terms
// exp((x - max) / temp), in powers of two: with c = log2(e) / temp, m is the
// product max * c, rounded, and a term is exp2(fma(x, c, -m)), one instruction
// and one rounding before the exp2. m itself is the reference, so its rounding
// is in every term and cancels. Nothing but -inf: m = -inf, s = 0.
// m is rounded up, two steps or three: the exact product is never above it, so
// no term is above 1 and no part of a sum overflows, however large the logits
// (a mask of -1e10, of the type's lowest value: to the nearest, exact products
// of that size lie hundreds or more above m, and inf * 0 = NaN follows
// where another part has the maximum). They may all vanish instead: at
// |max| c above 2^27 a row's s is small or 0 although its maximum is finite,
// and where max * c overflows too. The callers see that (out_of_range), and
// subtract the maximum from the row first. (s above 2^-60: what is lost below
// the smallest normal number is 2^-35 of 2^31 terms together.)
// The maximum m from here on. (Of -inf the fma makes NaN: the median of three
// is then the least number among them, m; otherwise the larger of m and the
// new one, the largest number at most.)
__device__ __forceinline__ float scaled_max(float m, float max, float c) {
    const float p = max * c;
    return __builtin_amdgcn_fmed3f(m, __builtin_fmaf(fabsf(p), 0x1p-22f, p), 3.402823466e38f);
}
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

struct MaxSum {
    float m, s;
};

__device__ __forceinline__ bool out_of_range(const MaxSum& v) { return v.s < 0x1p-60f || v.s == INFINITY; }

// m: the maximum so far, before the product with c. The terms are added up by
// themselves first: the running sum, which is larger, rounds once for E of them.
template <int E>
__device__ __forceinline__ void add_terms(MaxSum& v, const float* x, float max, float c) {
    const float m = scaled_max(v.m, max, c), b = base_of(m);
    float t = fast_exp2(__builtin_fmaf(x[0], c, -b));
#pragma unroll
    for (int e = 1; e < E; e++) t += fast_exp2(__builtin_fmaf(x[e], c, -b));
    v.s = __builtin_fmaf(v.s, fast_exp2(v.m - b), t);
    v.m = m;
}

// Adds what v holds to `total` and starts its sum anew: after kRun additions of
// a thread, so that a row of 2^31 columns rounds its sum some 1300 times, not
// 262144 (each by up to half a step).
constexpr int kRun = 256;
__device__ __forceinline__ void fold(MaxSum& total, MaxSum& v) {
    total.s = __builtin_fmaf(total.s, fast_exp2(total.m - base_of(v.m)), v.s);
    total.m = v.m;
    v.s = 0.0f;
}

template <int L> __device__ __forceinline__ MaxSum team_max_sum(MaxSum v) {
    MaxSum r;
    r.m = team_reduce<L, OpMax>(v.m);
    r.s = team_reduce<L, OpSum>(v.s * fast_exp2(v.m - base_of(r.m)));
    return r;
}

// Over a workgroup of T threads. sh: T / 64 entries; holds a barrier.
template <int T> __device__ __forceinline__ MaxSum group_max_sum(MaxSum v, MaxSum* sh) {
    constexpr int W = T / 64;
    v = team_max_sum<64>(v);
    if (W == 1) return v;
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return team_max_sum<W>(sh[threadIdx.x & (W - 1)]);
}

template <int T> __device__ __forceinline__ float group_max(float v, float* sh) {
    constexpr int W = T / 64;
    v = team_reduce<64, OpMax>(v);
    if (W == 1) return v;
    __syncthreads();                                   // sh may still be read
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return team_reduce<W, OpMax>(sh[threadIdx.x & (W - 1)]);
}

// ------------------------------------------------------------------ host checks
// Row counts: 0 <= tokens[i], fewer than 2^31 rows together.
inline ga_status make_rows(const int64_t* tokens, int32_t P, RowMap* m, const char* what) {
    if (P < 1 || P > GA_MAX_WORKERS)
        return fail(GA_EINVAL, "%s: P = %d outside [1, %d]", what, P, GA_MAX_WORKERS);
    if (!tokens) return fail(GA_EINVAL, "%s: null row counts", what);
    m->P = P;
    int64_t sum = 0;
    for (int i = 0; i < P; i++) {
        m->start[i] = (int32_t)sum;
        if (tokens[i] < 0 || tokens[i] > INT32_MAX || (sum += tokens[i]) > INT32_MAX)
            return fail(GA_EINVAL, "%s: row counts must be >= 0 and below 2^31 together", what);
    }
    for (int i = P; i <= GA_MAX_WORKERS; i++) m->start[i] = (int32_t)sum;
    return GA_OK;
}

// The address ranges of one call, to find outputs that overlap anything.
struct Regions {
    struct R {
        uintptr_t lo, hi;
        bool write;
    };
    R r[8 * GA_MAX_WORKERS + 8];
    int n = 0;
    bool wraps = false;
    void add(const void* p, int64_t bytes, bool write) {
        if (bytes <= 0) return;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (lo + (uintptr_t)bytes < lo) wraps = true;
        r[n++] = {lo, lo + (uintptr_t)bytes, write};
    }
    bool clash() {
        if (wraps) return true;
        std::sort(r, r + n, [](const R& a, const R& b) { return a.lo < b.lo; });
        uintptr_t any = 0, written = 0;                // ends of what came before
        for (int i = 0; i < n; i++) {
            if (r[i].lo < written || (r[i].write && r[i].lo < any)) return true;
            any = std::max(any, r[i].hi);
            if (r[i].write) written = std::max(written, r[i].hi);
        }
        return false;
    }
};

// P matrices of rows of n elements of `es` bytes, row stride ld: pointers
// there and aligned where a worker has rows, addresses in range. Fills t and
// adds the ranges to reg.
inline ga_status check_rows(const void* const* bufs, const int64_t* tokens, int32_t P, int64_t n,
                            int64_t ld, size_t es, bool write, const char* name, const char* what,
                            PtrTable* t, Regions* reg) {
    if (!bufs) return fail(GA_EINVAL, "%s: null %s array", what, name);
    if (ld < n) return fail(GA_EINVAL, "%s: row stride %lld of %s is below %lld", what, (long long)ld, name, (long long)n);
    for (int i = 0; i < P; i++) {
        t->p[i] = nullptr;
        if (tokens[i] == 0) continue;
        if (!bufs[i]) return fail(GA_EINVAL, "%s: worker %d %s pointer is null", what, i, name);
        if (!aligned(bufs[i], es))
            return fail(GA_EINVAL, "%s: worker %d %s pointer not aligned to %zu bytes", what, i, name, es);
        int64_t bytes;
        if (__builtin_mul_overflow(tokens[i] - 1, ld, &bytes) || __builtin_add_overflow(bytes, n, &bytes) ||
            __builtin_mul_overflow(bytes, (int64_t)es, &bytes) || bytes > (int64_t)1 << 47)
            return fail(GA_EINVAL, "%s: %s of worker %d is too large", what, name, i);
        t->p[i] = const_cast<void*>(bufs[i]);
        reg->add(bufs[i], bytes, write);
    }
    for (int i = P; i < GA_MAX_WORKERS; i++) t->p[i] = nullptr;
    return GA_OK;
}

// A gradient that replaces the logits has one range, which is written. (No
// rows: nothing is replaced, and the strides are free.)
inline bool in_place(const void* const* logits, void* const* grad, const int64_t* tokens, int32_t P) {
    bool any = false;
    for (int i = 0; i < P; i++) {
        if (tokens[i] == 0) continue;
        if (logits[i] != grad[i]) return false;
        any = true;
    }
    return any;
}

inline bool valid_scalar(float f) { return std::isfinite(f); }

// The kernels multiply by log2(e) / temp.
inline bool valid_temp(float t) { return t > 0.0f && std::isfinite(t) && std::isfinite(kLog2e / t); }

}  // namespace
}  // namespace ga
