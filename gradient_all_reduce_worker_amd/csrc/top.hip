// top.hip -- the K largest logits of every row, in order, with the row's
// log-sum-exp (ga_loss.h): what a student is distilled from.
//
// A value's place in the order is an integer key: its 32 bits made monotone
// (-0 taken as +0) above the complement of its column, so that no two
// elements of a row have the same key and equal values go by column.
//
// One read of the row finds the maximum of every thread's batches of it. Of
// G groups of threads, G >= K, the K-th largest group maximum is a bound that
// at least K elements reach and few others do (some G ln(G / (G - K)) where
// the row is in no order); only batches whose maximum reaches it are looked
// at again. What reaches it is ranked by counting. A row that has too many
// such elements (all equal, sorted) is selected digit by digit instead.
#include "loss.hpp"

namespace ga {
namespace {

constexpr int kMaxTopGroups = 16384;  // workgroups; each walks its rows
constexpr int kBatches = 8;           // batches of a row per thread, at most
constexpr int kCands = 2048;          // candidates held in LDS

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
    const int64_t n_vec = (V + E - 1) / E;
    uint64_t prefix = 0;
    int need = K;                                      // the K-th of those with the prefix
    for (int shift = 56; shift >= 0; shift -= 8) {
        const uint64_t above = shift == 56 ? 0 : ~0ull << (shift + 8);
        for (int i = tid; i < 256; i += T) hist[i] = 0;
        __syncthreads();
        for (int64_t j = tid; j < n_vec; j += T) {
            float x[E];
            R::widen(load_row_vec<DT, false>(z, j, V), x);
            for (int e = 0; e < E; e++) {
                const int64_t col = j * E + e;
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

// One workgroup of T threads per row.
template <ga_dtype DT, int T>
__global__ __launch_bounds__(T) void top_kernel(TopArgs a) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    constexpr int U = 4;                               // vectors in flight
    __shared__ uint64_t cand[kCands];
    __shared__ float batch_max[kBatches * T];
    __shared__ uint32_t group_key[T];
    __shared__ uint32_t hist[257];
    __shared__ uint64_t sh_key;
    __shared__ uint32_t n_cand, bound;
    __shared__ MaxSum sh[T / 64];
    const int tid = threadIdx.x;
    const int32_t n_rows = a.rows.start[GA_MAX_WORKERS];
    const int64_t V = a.V, n_vec = (V + E - 1) / E;
    // a batch is `per` rounds of U vectors, T apart; kBatches of them hold a row
    const int64_t rounds = (n_vec + (int64_t)U * T - 1) / ((int64_t)U * T);
    const int64_t per = (rounds + kBatches - 1) / kBatches;
    const int n_batch = (int)((rounds + per - 1) / per);
    const float c = kLog2e / a.temp;
    const int K = a.K;
    int G = 64;                                        // groups: a power of two, 2 K or T of them
    while (G < 2 * K && G < T) G *= 2;
    const int span = T / G;                            // threads of a group

    for (int32_t row = blockIdx.x; row < n_rows; row += gridDim.x) {
        const int w = worker_of(a.rows, row);
        const int64_t r = row - a.rows.start[w];
        const typename R::elem* z = static_cast<const typename R::elem*>(a.logits.p[w]) + r * a.ld;
        int32_t* out_i = static_cast<int32_t*>(a.idx.p[w]) + r * K;
        typename R::elem* out_v = static_cast<typename R::elem*>(a.vals.p[w]) + r * K;

        // one read: batch maxima, and the sum of exponentials
        MaxSum ms = {-INFINITY, 0.0f};
        for (int b = 0; b < n_batch; b++) {
            float bm = -INFINITY;
            for (int64_t p = b * per; p < (b + 1) * per && p < rounds; p++) {
                uint4 raw[U];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int64_t j = (p * U + u) * T + tid;
                    raw[u] = j < n_vec ? load_row_vec<DT, false>(z, j, V)
                                       : make_uint4(R::kEmpty, R::kEmpty, R::kEmpty, R::kEmpty);
                }
                float m = -INFINITY;
#pragma unroll
                for (int u = 0; u < U; u++) {
                    float x[E];
                    R::widen(raw[u], x);
#pragma unroll
                    for (int e = 0; e < E; e++) m = fmaxf(m, x[e]);
                }
                bm = fmaxf(bm, m);
                if (a.has_lse) {
                    m = fmaxf(m, ms.m);
                    const float base = base_of(m);
                    float s = ms.s * fast_exp2((ms.m - base) * c);
#pragma unroll
                    for (int u = 0; u < U; u++) {
                        float x[E];
                        R::widen(raw[u], x);
#pragma unroll
                        for (int e = 0; e < E; e++) s += fast_exp2((x[e] - base) * c);
                    }
                    ms.m = m;
                    ms.s = s;
                }
            }
            batch_max[b * T + tid] = bm;
        }
        if (tid == 0) {
            n_cand = 0;
            bound = 0;
        }
        // the groups' maxima, and the K-th largest of them
        float gm = -INFINITY;
        for (int b = 0; b < n_batch; b++) gm = fmaxf(gm, batch_max[b * T + tid]);
        for (int o = 1; o < span; o *= 2) gm = fmaxf(gm, __shfl_xor(gm, o));
        if (tid % span == 0) group_key[tid / span] = order_key(gm);
        if (a.has_lse) {
            ms = group_max_sum<T>(ms, c, sh);
            if (tid == 0)
                static_cast<float*>(a.lse.p[w])[r] = ms.s == 0.0f ? -INFINITY : base_of(ms.m) / a.temp + logf(ms.s);
        }
        __syncthreads();
        if (tid < G && K <= G) {
            const uint32_t mine = group_key[tid];
            int before = 0;
            for (int j = 0; j < G; j++) {
                const uint32_t o = group_key[j];
                before += o > mine || (o == mine && j < tid);
            }
            if (before == K - 1) bound = mine;
        }
        __syncthreads();
        const uint32_t least = bound;

        // what reaches the bound
        for (int b = 0; b < n_batch; b++) {
            if (order_key(batch_max[b * T + tid]) < least) continue;
            for (int64_t p = b * per; p < (b + 1) * per && p < rounds; p++)
                for (int u = 0; u < U; u++) {
                    const int64_t j = (p * U + u) * T + tid;
                    if (j >= n_vec) continue;
                    float x[E];
                    R::widen(load_row_vec<DT, false>(z, j, V), x);
                    for (int e = 0; e < E; e++) {
                        const int64_t col = j * E + e;
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
            for (int64_t j = tid; j < n_vec; j += T) {
                float x[E];
                R::widen(load_row_vec<DT, false>(z, j, V), x);
                for (int e = 0; e < E; e++) {
                    const int64_t col = j * E + e;
                    const uint64_t k = full_key(x[e], (int32_t)col);
                    if (col < V && k >= key) {
                        const uint32_t at = atomicAdd(&n_cand, 1u);
                        if (at < kCands) cand[at] = k;
                    }
                }
            }
            __syncthreads();
            n = K;                                     // keys differ: exactly K reach the K-th
        }
        for (int k = tid; k < n; k += T) {
            const uint64_t mine = cand[k];
            int rank = 0;
            for (int j = 0; j < n; j++) rank += cand[j] > mine;
            if (rank < K) {
                const int32_t col = (int32_t)~(uint32_t)mine;
                out_i[rank] = col;
                out_v[rank] = z[col];
            }
        }
        __syncthreads();                               // the candidates are read
    }
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
    const int blocks = (int)std::min<int64_t>(n_rows, kMaxTopGroups);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dt == GA_BF16) top_kernel<GA_BF16, 256><<<blocks, 256, 0, st>>>(a);
    else top_kernel<GA_F32, 256><<<blocks, 256, 0, st>>>(a);
    return check_launch(what);
}
