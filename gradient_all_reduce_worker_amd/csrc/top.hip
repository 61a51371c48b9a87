// top.hip -- the K largest logits of every row, in order, with the row's
// log-sum-exp (ga_loss.h): what a student is distilled from.
//
// A value's place in the order is an integer key: its 32 bits made monotone
// (-0 taken as +0) above the complement of its column, so that no two
// elements of a row have the same key and equal values go by column.
//
// One read of the row finds the maximum of every thread's batches of it. The
// K-th largest of the threads' maxima is a bound that at least K elements reach
// and few others do (some T ln(T / (T - K)) of T threads where the row is in no
// order); it is found by bisection, roughly. Only batches whose maximum reaches
// it are looked at again. What reaches it is ranked by counting, or sorted. A
// row that has too many such elements (all equal, sorted) is selected digit by
// digit instead.
#include "loss.hpp"

namespace ga {
namespace {

constexpr int kBatches = 8;           // batches of a row per thread, at most
constexpr int kCands = 2048;          // candidates held in LDS
constexpr int kCount = 192;           // up to as many are ranked by counting

struct TopArgs {
    PtrTable logits, vals, idx, lse;
    RowMap rows;
    int32_t K, has_lse;
    int64_t V, ld;
    float temp;
};

// binary32 -> uint32 whose unsigned order is the values' order; -0 as +0.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint64_t full_key(float f, int32_t col) {
    return (uint64_t)order_key(f) << 32 | (uint32_t)~col;
}


// The K-th largest key of the row, digit by digit (8 bits, most significant
// first), reading the row once per digit: exact for any row.
template <ga_dtype DT, int T>
__device__ uint64_t select_by_digits(const void* z, int64_t V, int K, uint32_t* hist, uint64_t* sh_key) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    const int tid = threadIdx.x;
    const int n_vec = (int)((V + E - 1) / E);
    uint64_t prefix = 0;
    int need = K;                                      // the K-th of those with the prefix
    for (int shift = 56; shift >= 0; shift -= 8) {
        const uint64_t above = shift == 56 ? 0 : ~0ull << (shift + 8);
        for (int i = tid; i < 256; i += T) hist[i] = 0;
        __syncthreads();
        for (int j = tid; j < n_vec; j += T) {
            float x[E];
            R::widen(load_row_vec<DT, false>(z, j, V), x);
            for (int e = 0; e < E; e++) {
                const int64_t col = (int64_t)j * E + e;
                const uint64_t k = full_key(x[e], (int32_t)col);
                if (col < V && ((k ^ prefix) & above) == 0) atomicAdd(&hist[(k >> shift) & 255], 1u);
            }
        }
        __syncthreads();
        if (tid == 0) {
            int d = 255, left = need;
            while (d > 0 && (int)hist[d] < left) left -= hist[d--];
            *sh_key = prefix | (uint64_t)d << shift;
            hist[256] = left;
        }
        __syncthreads();
        prefix = *sh_key;
        need = hist[256];
    }
    return prefix;
}

// A bound that at least K and not many more of the workgroup's T keys reach
// (K <= T): the K-th largest, or one between it and the (K + slack)-th.
// sh: 2 T / 64 counts.
template <int T> __device__ uint32_t bound_of(uint32_t key, int K, int slack, uint32_t (*sh)[T / 64]) {
    uint32_t lo = 0, hi = 0xFFFFFFFFu;                 // K keys reach lo; hi: fewer, or not known
    for (int turn = 0; hi - lo > 1; turn ^= 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const uint32_t n = (uint32_t)__popcll(__ballot(key >= mid));
        if ((threadIdx.x & 63) == 0) sh[turn][threadIdx.x >> 6] = n;
        __syncthreads();
        int sum = 0;
#pragma unroll
        for (int i = 0; i < T / 64; i++) sum += sh[turn][i];
        if (sum >= K) {
            lo = mid;
            if (sum <= K + slack) break;
        } else {
            hi = mid;
        }
    }
    return lo;
}

// The n keys of c, descending, by a bitonic network over the next power of two.
template <int T> __device__ void sort_keys(uint64_t* c, int n) {
    int size = 64;
    while (size < n) size *= 2;
    for (int i = n + threadIdx.x; i < size; i += T) c[i] = 0;
    for (int k = 2; k <= size; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
            __syncthreads();
            for (int i = threadIdx.x; i < size / 2; i += T) {
                const int lo = (i & ~(j - 1)) * 2 + (i & (j - 1)), hi = lo + j;
                const uint64_t a = c[lo], b = c[hi];
                if (((lo & k) == 0) == (a < b)) {
                    c[lo] = b;
                    c[hi] = a;
                }
            }
        }
    __syncthreads();
}

// One workgroup of T threads per row.
template <ga_dtype DT, int T, bool LSE>
__global__ __launch_bounds__(T) void top_kernel(TopArgs a) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    constexpr int U = 4;                               // vectors in flight
    __shared__ uint64_t cand[kCands];
    __shared__ float batch_max[kBatches * T];
    __shared__ uint32_t hist[257];
    __shared__ uint32_t counts[2][T / 64];
    __shared__ uint64_t sh_key;
    __shared__ uint32_t n_cand;
    __shared__ MaxSum sh[T / 64];
    __shared__ float sh_f[T / 64];
    const int tid = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.rows.start[GA_MAX_WORKERS]) return;
    const int64_t V = a.V;
    const int n_vec = (int)((V + E - 1) / E);
    // a batch is `per` rounds of U vectors, T apart; kBatches of them hold a row
    const int rounds = (n_vec + U * T - 1) / (U * T);
    const int per = (rounds + kBatches - 1) / kBatches;
    const int n_batch = (rounds + per - 1) / per;
    const float c = kLog2e / a.temp;
    const int K = a.K;
    const int w = worker_of(a.rows, (int32_t)row);
    const int64_t r = row - a.rows.start[w];
    const typename R::elem* z = static_cast<const typename R::elem*>(a.logits.p[w]) + r * a.ld;
    int32_t* out_i = static_cast<int32_t*>(a.idx.p[w]) + r * K;
    typename R::elem* out_v = static_cast<typename R::elem*>(a.vals.p[w]) + r * K;

    if (tid == 0) n_cand = 0;
    // one read: batch maxima, and the sum of exponentials
    MaxSum ms = {-INFINITY, 0.0f};
    float top = -INFINITY;
    for (int b = 0; b < n_batch; b++) {
        float bm = -INFINITY;
        for (int p = b * per; p < (b + 1) * per && p < rounds; p++) {
            const int j0 = p * U * T + tid;
            float x[U * E];
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; u++)
                raw[u] = j0 + u * T < n_vec ? load_row_vec<DT, false>(z, j0 + u * T, V)
                                            : make_uint4(R::kEmpty, R::kEmpty, R::kEmpty, R::kEmpty);
#pragma unroll
            for (int u = 0; u < U; u++) R::widen(raw[u], x + u * E);
#pragma unroll
            for (int e = 0; e < U * E; e++) bm = fmaxf(bm, x[e]);
            if (LSE) {
                top = fmaxf(top, bm);
                add_terms<U * E>(ms, x, top, c);
            }
        }
        batch_max[b * T + tid] = bm;
        if (!LSE) top = fmaxf(top, bm);
    }
    if (LSE) {
        ms = group_max_sum<T>(ms, sh);
        float lse = (base_of(ms.m) + log2f(ms.s)) * kLn2;
        if (overflowed(ms)) {
            // nothing but -inf, or a maximum next to an end of the type, where
            // the products with c overflow: subtracted first
            const float all = group_max<T>(top, sh_f);
            lse = -INFINITY;
            if (all != -INFINITY) {
                ms = {-INFINITY, 0.0f};
                for (int j = tid; j < n_vec; j += T) {
                    float x[E];
                    R::widen(load_row_vec<DT, false>(z, j, V), x);
#pragma unroll
                    for (int e = 0; e < E; e++) x[e] -= all;
                    add_terms<E>(ms, x, 0.0f, c);
                }
                ms = group_max_sum<T>(ms, sh);
                lse = all / a.temp + logf(ms.s);
            }
        }
        if (tid == 0) static_cast<float*>(a.lse.p[w])[r] = lse;
    }
    // Too many slots for T threads' maxima: everything is a candidate (all of
    // a short row fits).
    uint32_t least = 0;
    if (K <= T * 3 / 4) least = bound_of<T>(order_key(top), K, K / 8, counts);
    else __syncthreads();                              // n_cand

    // what reaches the bound
    for (int b = 0; b < n_batch; b++) {
        if (order_key(batch_max[b * T + tid]) < least) continue;
        for (int p = b * per; p < (b + 1) * per && p < rounds; p++)
            for (int u = 0; u < U; u++) {
                const int j = (p * U + u) * T + tid;
                if (j >= n_vec) continue;
                float x[E];
                R::widen(load_row_vec<DT, false>(z, j, V), x);
                for (int e = 0; e < E; e++) {
                    const int64_t col = (int64_t)j * E + e;
                    if (col < V && order_key(x[e]) >= least) {
                        const uint32_t at = atomicAdd(&n_cand, 1u);
                        if (at < kCands) cand[at] = full_key(x[e], (int32_t)col);
                    }
                }
            }
    }
    __syncthreads();
    int n = (int)n_cand;
    if (n < K || n > kCands) {
        // fewer than K: NaN below every number hid from the maxima
        const uint64_t key = select_by_digits<DT, T>(z, V, K, hist, &sh_key);
        if (tid == 0) n_cand = 0;
        __syncthreads();
        for (int j = tid; j < n_vec; j += T) {
            float x[E];
            R::widen(load_row_vec<DT, false>(z, j, V), x);
            for (int e = 0; e < E; e++) {
                const int64_t col = (int64_t)j * E + e;
                const uint64_t k = full_key(x[e], (int32_t)col);
                if (col < V && k >= key) {
                    const uint32_t at = atomicAdd(&n_cand, 1u);
                    if (at < kCands) cand[at] = k;
                }
            }
        }
        __syncthreads();
        n = K;                                         // keys differ: exactly K reach the K-th
    }
    if (n > kCount) {
        sort_keys<T>(cand, n);
        for (int k = tid; k < K; k += T) {
            const int32_t col = (int32_t)~(uint32_t)cand[k];
            out_i[k] = col;
            out_v[k] = z[col];
        }
        return;
    }
    // H threads count the keys above one
    int H = 1;
    while (H < 64 && 2 * H * n <= T) H *= 2;
    for (int k0 = 0; k0 < n; k0 += T / H) {
        const int k = k0 + tid / H;
        const uint64_t mine = k < n ? cand[k] : 0;
        int rank = 0;
        for (int j = tid & (H - 1); j < n; j += H) rank += cand[j] > mine;
        for (int o = 1; o < H; o *= 2) rank += __shfl_xor(rank, o);
        if (k < n && rank < K && (tid & (H - 1)) == 0) {
            const int32_t col = (int32_t)~(uint32_t)mine;
            out_i[rank] = col;
            out_v[rank] = z[col];
        }
    }
}

template <ga_dtype DT, int T> void launch_top(const TopArgs& a, hipStream_t s) {
    // (a launch takes fewer than 2^32 work-items along x)
    const int64_t n = a.rows.start[GA_MAX_WORKERS], wide = std::min<int64_t>(n, 1 << 20);
    const dim3 grid((unsigned)wide, (unsigned)ceil_div(n, wide));
    if (a.has_lse) top_kernel<DT, T, true><<<grid, T, 0, s>>>(a);
    else top_kernel<DT, T, false><<<grid, T, 0, s>>>(a);
}

template <ga_dtype DT> void launch_rows(const TopArgs& a, hipStream_t s) {
    if (a.K > 192 || a.V / RowVec<DT>::kElems > 4096) launch_top<DT, 1024>(a, s);
    else launch_top<DT, 256>(a, s);
}

}  // namespace
}  // namespace ga

using namespace ga;

extern "C" ga_status ga_top_logits(const void* const* logits, const int64_t* tokens, int32_t P, int64_t V,
                                   int64_t ld, ga_dtype dt, int32_t K, float temp, void* const* vals,
                                   int32_t* const* idx, float* const* lse, void* stream) {
    const char* what = "ga_top_logits";
    TopArgs a = {};
    if (ga_status s = make_rows(tokens, P, &a.rows, what)) return s;
    if (!valid_dtype(dt)) return fail(GA_EINVAL, "%s: bad dtype", what);
    if (V < 1 || V > INT32_MAX) return fail(GA_EINVAL, "%s: V = %lld outside [1, 2^31)", what, (long long)V);
    if (K < 1 || K > GA_TOP_MAX || K > V)
        return fail(GA_EINVAL, "%s: K = %d outside [1, min(V, %d)]", what, K, GA_TOP_MAX);
    if (!(temp > 0.0f) || !valid_scalar(temp) || !valid_scalar(1.0f / temp))
        return fail(GA_EINVAL, "%s: temp must be a positive normal number", what);
    Regions reg;
    ga_status s;
    if ((s = check_rows(logits, tokens, P, V, ld, elem_size(dt), false, "logits", what, &a.logits, &reg))) return s;
    if ((s = check_rows(vals, tokens, P, K, K, elem_size(dt), true, "vals", what, &a.vals, &reg))) return s;
    if ((s = check_rows((const void* const*)idx, tokens, P, K, K, 4, true, "idx", what, &a.idx, &reg))) return s;
    if (lse && (s = check_rows((const void* const*)lse, tokens, P, 1, 1, 4, true, "lse", what, &a.lse, &reg))) return s;
    if (reg.clash()) return fail(GA_EINVAL, "%s: an output overlaps another buffer", what);
    const int64_t n_rows = a.rows.start[GA_MAX_WORKERS];
    if (n_rows == 0) return GA_OK;
    a.K = K;
    a.has_lse = lse != nullptr;
    a.V = V;
    a.ld = ld;
    a.temp = temp;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dt == GA_BF16) launch_rows<GA_BF16>(a, st);
    else launch_rows<GA_F32>(a, st);
    return check_launch(what);
}
