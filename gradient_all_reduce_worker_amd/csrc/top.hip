// top.hip -- the K largest logits of every row, in order, with the row's
// log-sum-exp (ga_loss.h): what a student is distilled from.
//
// A value's place in the order is an integer key: its 32 bits made monotone
// (-0 taken as +0) above the complement of its column, so that no two
// elements of a row have the same key and equal values go by column.
//
// One read of the row finds every thread's maximum. The K-th largest of those is
// a bound that at least K elements reach and few others do (some
// T ln(T / (T - K)) of T threads where the row is in no order); it is found by
// bisection, roughly. Only batches of a thread's vectors whose maximum reaches
// it are looked at again, shared out among all threads. (Short rows with many
// slots: the elements themselves are bisected.) What reaches the bound is
// ranked by counting, or sorted. A row that has too many such elements (all
// equal, sorted), or one in rounds with more than some 570 slots, which the
// threads' maxima do not bound, is selected digit by digit instead: six reads
// of it or more (1024 rows of 131072 bf16: K = 500 89 us, 600 303, 1024 553).
//
// Bound: reading the row, and close behind it the vector unit: widening, maximum,
// product, exp2 and sum are 6 instructions' time per element, and the selection
// some 700 per wave and row. 2048 rows of 131072 bf16, K = 128: 112 us, 4.8 TB/s (a
// kernel that only reads gets 7); 2048 rows of 32000 f32, K = 32: 48 us, 5.4; about
// 1100 rows of 50003 bf16, K = 64: 35 us, 3.2, where a workgroup's selection
// has few others beside it; one row of 32768 bf16: 7.5 us, all latency. The second look
// takes 1.5 us on an idle device and up to 12 behind the other workgroups'
// loads. 8192 rows of 131072 f32 come to 5.9 TB/s.
// Not kept: the bound from a sample of the row, so that one pass collects
// (2048 rows of 32000 f32 47 -> 65 us: too many pass a loose bound); rows of up
// to 65536 held in registers without a second look (50003: 38 -> 50 us, two
// workgroups fit a CU instead of four); two rounds on their way (131072: 115 ->
// 121 us); all waves bisecting together, a barrier per step (8192 rows of
// 32000 bf16: 107 -> 119 us).
#include "loss.hpp"

namespace ga {
namespace {

constexpr int kBatches = 8;           // batches of a row per thread, at most
constexpr int kMostCands = 2048;      // candidates held in LDS
constexpr int kMostBatches = 1024;    // batches that are looked at again
constexpr int kCount = 192;           // up to as many are ranked by counting (no barrier), more sorted

struct TopArgs {
    PtrTable logits, vals, idx, lse;
    RowMap rows;
    int32_t K, has_lse;
    int64_t V, ld;
    float temp;
};

// binary32 -> uint32 whose unsigned order is the values' order, -0 as +0; and
// back.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ uint64_t full_key(float f, int32_t col) {
    return (uint64_t)order_key(f) << 32 | (uint32_t)~col;
}


// The K-th largest key of the row, digit by digit (8 bits, most significant
// first), reading the row once per digit: exact for any row. (1024 rows of
// 131072 equal bf16: 530 us, 65 in random order.) Digits that all
// keys with the prefix share are passed over: the lower half of a bf16 value
// (0, or all ones for a negative one), the upper digits of a small column.
template <ga_dtype DT, int T>
__device__ uint64_t select_by_digits(const void* z, int64_t V, int K, uint32_t* hist, uint64_t* sh_key) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    const int tid = threadIdx.x, lane = tid & 63;
    const int n_vec = (int)((V + E - 1) / E);
    uint64_t prefix = 0;
    int need = K;                                      // the K-th of those with the prefix
    for (int shift = 56; shift >= 0; shift -= 8) {
        if (DT == GA_BF16 && (shift == 40 || shift == 32)) {
            prefix |= prefix >> 63 ? 0 : 0xFFull << shift;
            continue;
        }
        if (shift < 32 && V <= (int64_t)1 << shift) {
            prefix |= 0xFFull << shift;
            continue;
        }
        const uint64_t above = shift == 56 ? 0 : ~0ull << (shift + 8);
        for (int i = tid; i < 256; i += T) hist[i] = 0;
        __syncthreads();
        for (int j = tid; j < n_vec; j += T) {
            float x[E];
            R::widen(load_row_vec<DT, false>(z, j, V), x);
            for (int e = 0; e < E; e++) {
                const int64_t col = (int64_t)j * E + e;
                const uint64_t k = full_key(x[e], (int32_t)col);
                if (col < V && ((k ^ prefix) & above) == 0) {
                    // rows that come here hold many equal values: lanes that
                    // share the first one's digit are counted at once
                    const int d = (int)((k >> shift) & 255), d0 = __builtin_amdgcn_readfirstlane(d);
                    const uint64_t same = __ballot(d == d0);
                    if (d != d0) atomicAdd(&hist[d], 1u);
                    else if (lane == __ffsll((unsigned long long)same) - 1) atomicAdd(&hist[d0], (uint32_t)__popcll(same));
                }
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

// A bound that at least K and not many more of a set of values reach: the K-th
// largest, or one between it and the (K + slack)-th; 0 (what anything reaches,
// NaN too) where fewer than K values reach `least`. `most` is their maximum.
// count(b, c) sets c to how many values reach each of the three bounds b.
template <class COUNT>
__device__ __forceinline__ uint32_t bound_of(COUNT count, int K, int slack, float least, float most) {
    uint32_t lo = order_key(least), hi = order_key(most) + 1;
    bool known = false;                                // K values reach lo
    for (;;) {
        const uint32_t q = max((hi - lo) / 4, 1u);
        const uint32_t at[3] = {known ? lo + q : lo, lo + 2 * q, lo + 3 * q};
        const float b[3] = {key_value(at[0]), key_value(at[1]), key_value(at[2])};
        int c[3];
        count(b, c);
#pragma unroll
        for (int k = 0; k < 3; k++)
            if (at[k] >= hi) c[k] = 0;
        if (c[0] < K) {
            if (!known) return 0;
            hi = at[0];
        } else {
            const int k = c[2] >= K ? 2 : c[1] >= K ? 1 : 0;
            lo = at[k];
            if (k < 2) hi = min(hi, at[k + 1]);
            if (c[k] <= K + slack) return lo;
        }
        known = true;
        if (hi - lo <= 1) return lo;
    }
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

// One workgroup of T threads per row, which is read in rounds of U vectors per
// thread, T apart; a round is on its way while the one before is looked at. ONE:
// the row is one round, and stays in registers; else it has one whole round at
// least (the launches see to it). Rows pass once: nontemporal
// loads, two per round (4096 rows of 131072 bf16, K = 8: 177 us; plain, one per round: 218).
template <ga_dtype DT, int T, int U, bool ONE, bool LSE>
__global__ __launch_bounds__(T) __attribute__((amdgpu_waves_per_eu(T == 64 ? 4 : 8))) void top_kernel(TopArgs a) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems, N = U * E;
    constexpr int kRounds = ONE ? 1 : kBatches;
    // (a power of two, as the sort needs; a row that stays has N T elements at most)
    constexpr int kCands = ONE && N * T < kMostCands ? N * T : kMostCands;
    __shared__ uint64_t cand[kCands];
    __shared__ float batch_max[ONE ? 1 : kRounds * T];
    __shared__ uint16_t batches[ONE ? 1 : kMostBatches];
    __shared__ uint32_t hist[257];
    __shared__ uint32_t counts[2][3][T / 64];
    __shared__ uint64_t sh_key;
    __shared__ uint32_t n_cand, n_again, sh_bound;
    __shared__ MaxSum sh[T / 64];
    __shared__ float tops[T], sh_most;
    const int tid = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.rows.start[GA_MAX_WORKERS]) return;
    const int V = (int)a.V, n_vec = (V - 1) / E + 1, n_whole = V / E;
    // a batch is `per` rounds; kBatches of them hold a row
    const int rounds = ONE ? 1 : (n_whole - 1) / (U * T) + 1;
    const int per = ONE ? 1 : (rounds + kBatches - 1) / kBatches;
    const float c = kLog2e / a.temp;
    const int K = a.K;
    const int w = worker_of(a.rows, (int32_t)row);
    const int64_t r = row - a.rows.start[w];
    const typename R::elem* z = static_cast<const typename R::elem*>(a.logits.p[w]) + r * a.ld;
    int32_t* out_i = static_cast<int32_t*>(a.idx.p[w]) + r * K;
    typename R::elem* out_v = static_cast<typename R::elem*>(a.vals.p[w]) + r * K;

    if (tid == 0) n_cand = n_again = 0;
    // one read: the threads' maxima (and those of their batches), and the sum
    // of exponentials
    MaxSum ms = {-INFINITY, 0.0f};
    float top = -INFINITY, last = -INFINITY;
    uint4 raw[U];
    if constexpr (ONE) {
#pragma unroll
        for (int u = 0; u < U; u++) raw[u] = make_uint4(R::kEmpty, R::kEmpty, R::kEmpty, R::kEmpty);
        // (no load under a mask, which would be waited for at once)
        if (n_whole > 0) {
#pragma unroll
            for (int u = 0; u < U; u++)
                raw[u] = load_whole_vec<DT, true>(z, 0, (uint32_t)min(u * T + tid, n_whole - 1) * 16u);
        }
        last = load_last<DT>(z, V, n_whole, tid);
        float x[N];
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (u * T + tid >= n_whole) raw[u] = make_uint4(R::kEmpty, R::kEmpty, R::kEmpty, R::kEmpty);
            R::widen(raw[u], x + u * E);
            forget_derived(raw[u]);
        }
#pragma unroll
        for (int e = 0; e < N; e++) top = fmaxf(top, x[e]);
        top = fmaxf(top, last);
        if (LSE) {
            add_terms<N>(ms, x, top, c);
            ms.s += fast_exp2(__builtin_fmaf(last, c, -base_of(ms.m)));
        }
    } else {
        // Whole rounds, the next on its way, without a condition on any load
        // (it would be waited for at once); a thread that has nothing in the last
        // round loads the last vector, and takes it out.
        const int whole = n_whole / (U * T);
        MaxSum total = ms;
        float bm = -INFINITY;
        int left = per, b = 0;
        auto load = [&](uint4* v, int p) {
#pragma unroll
            for (int u = 0; u < U; u++) v[u] = load_whole_vec<DT, true>(z, ((int64_t)p * U + u) * T * 16, tid * 16);
        };
        auto look = [&](const float* x, int p) {
#pragma unroll
            for (int e = 0; e < N; e++) bm = fmaxf(bm, x[e]);
            if (LSE) add_terms<N>(ms, x, fmaxf(top, bm), c);
            if (--left == 0 || p + 1 == rounds) {
                batch_max[b++ * T + tid] = bm;
                top = fmaxf(top, bm);
                bm = -INFINITY;
                left = per;
            }
        };
        auto widen = [&](const uint4* v, float* x) {
#pragma unroll
            for (int u = 0; u < U; u++) R::widen(v[u], x + u * E);
        };
        uint4 other[U];
        float x[N];
        last = load_last<DT>(z, V, n_whole, tid);
        load(raw, 0);
        for (int p = 0, end = kRun;; end += kRun) {
            for (const int stop = min(whole - 1, end); p < stop; p++) {
                widen(raw, x);
                load(raw, p + 1);
                look(x, p);
            }
            if (p == whole - 1) break;
            fold(total, ms);
        }
        widen(raw, x);
#pragma unroll
        for (int u = 0; u < U; u++)
            other[u] = load_whole_vec<DT, true>(z, (int64_t)min((whole * U + u) * T + tid, n_whole - 1) * 16, 0);
        look(x, whole - 1);
        if (whole < rounds) {
#pragma unroll
            for (int u = 0; u < U; u++)
                if ((whole * U + u) * T + tid >= n_whole) other[u] = make_uint4(R::kEmpty, R::kEmpty, R::kEmpty, R::kEmpty);
            widen(other, x);
            look(x, whole);
        }
        top = fmaxf(top, last);
        if (LSE) {
            add_terms<1>(ms, &last, top, c);
            if (whole > kRun) {
                fold(total, ms);
                ms = total;
            }
        }
    }
    // One wave bisects the threads' maxima, without a barrier; another finishes
    // the log-sum-exp meanwhile.
    constexpr int W = T / 64;
    const int wave = tid >> 6, lane = tid & 63;
    tops[tid] = top;
    if (LSE) {
        ms = team_max_sum<64>(ms);
        if (lane == 0) sh[wave] = ms;
    }
    __syncthreads();
    const bool by_tops = K <= min(T, n_whole) * 3 / 4;
    if (wave == 0) {
        float v[W], least = INFINITY, most = -INFINITY;
#pragma unroll
        for (int i = 0; i < W; i++) {
            v[i] = tops[i * 64 + lane];
            least = fminf(least, v[i]);
            most = fmaxf(most, v[i]);
        }
        least = -team_reduce<64, OpMax>(-least);
        most = team_reduce<64, OpMax>(most);
        uint32_t found = 0;
        if (by_tops)
            found = bound_of([&](const float* b, int* n) {
#pragma unroll
                for (int k = 0; k < 3; k++) {
                    n[k] = 0;
#pragma unroll
                    for (int i = 0; i < W; i++) n[k] += __popcll(__ballot(v[i] >= b[k]));
                }
            }, K, K / 8, least, most);
        if (lane == 0) {
            sh_bound = found;
            sh_most = most;
        }
    }
    if (LSE && wave == W - 1) {
        ms = team_max_sum<W>(sh[lane & (W - 1)]);
        // (in binary64: neither the sum nor the product rounds in binary32)
        float lse = (float)(((double)base_of(ms.m) + (double)log2f(ms.s)) * 0.6931471805599453);
        if (out_of_range(ms)) {
            // nothing but -inf, or a maximum so large that the terms vanish or
            // the products with c overflow: subtracted first
            float most = -INFINITY;
            for (int i = 0; i < W; i++) most = fmaxf(most, tops[i * 64 + lane]);
            most = team_reduce<64, OpMax>(most);
            lse = -INFINITY;
            if (most != -INFINITY) {
                ms = {-INFINITY, 0.0f};
                for (int j = lane; j < n_vec; j += 64) {
                    float y[E];
                    R::widen(load_row_vec<DT, false>(z, j, V), y);
#pragma unroll
                    for (int e = 0; e < E; e++) y[e] -= most;
                    add_terms<E>(ms, y, 0.0f, c);
                }
                lse = most / a.temp + logf(team_max_sum<64>(ms).s);
            }
        }
        if (lane == 0) static_cast<float*>(a.lse.p[w])[r] = lse;
    }
    __syncthreads();
    uint32_t bound = sh_bound;
    if (ONE && !by_tops) {
        int turn = 0;
        bound = bound_of([&](const float* b, int* n) {
            uint32_t mine[3] = {last >= b[0], last >= b[1], last >= b[2]};
#pragma unroll
            for (int u = 0; u < U; u++) {
                float x[E];
                R::widen(raw[u], x);
#pragma unroll
                for (int e = 0; e < E; e++)
#pragma unroll
                    for (int k = 0; k < 3; k++) mine[k] += x[e] >= b[k];
                forget_derived(raw[u]);
            }
#pragma unroll
            for (int k = 0; k < 3; k++) {
                const float all = team_reduce<64, OpSum>((float)mine[k]);
                if (lane == 0) counts[turn][k][wave] = (uint32_t)all;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 3; k++) {
                n[k] = 0;
#pragma unroll
                for (int i = 0; i < W; i++) n[k] += (int)counts[turn][k][i];
            }
            turn ^= 1;
        }, K, K / 8, -INFINITY, sh_most);
    }

    // what reaches the bound (0: NaN as well)
    const float at_least = key_value(bound);
    auto take1 = [&](float y, int col) {
        if ((y >= at_least || bound == 0) && col < V) {
            const uint32_t at = atomicAdd(&n_cand, 1u);
            if (at < kCands) cand[at] = full_key(y, col);
        }
    };
    auto take = [&](const uint4& v, int j) {
        float y[E];
        R::widen(v, y);
#pragma unroll
        for (int e = 0; e < E; e++) take1(y[e], j * E + e);
    };
    bool many = false;
    if (ONE) {
        if (top >= at_least || bound == 0) {
#pragma unroll
            for (int u = 0; u < U; u++)
                if (u * T + tid < n_whole) take(raw[u], u * T + tid);
            if (tid < V - n_whole * E) take1(last, n_whole * E + tid);
        }
    } else {
        // a list of the batches, then their vectors one per thread
        for (int b = 0; b * per < rounds; b++)
            if (batch_max[b * T + tid] >= at_least || bound == 0) {
                const uint32_t at = atomicAdd(&n_again, 1u);
                if (at < kMostBatches) batches[at] = (uint16_t)(b * T + tid);
            }
        __syncthreads();
        const int again = (int)n_again, size = per * U;
        many = again > kMostBatches;
        if (!many)
            for (int64_t i = tid; i < (int64_t)again * size; i += T) {
                const int b = batches[i / size], q = (int)(i % size);
                const int j = (b / T * size + q) * T + b % T;
                if (j < n_whole) take(load_whole_vec<DT, false>(z, (int64_t)j * 16, 0), j);
            }
        if (tid < V - n_whole * E) take1(last, n_whole * E + tid);
    }
    __syncthreads();
    int n = (int)n_cand;
    if (many || n < K || n > kCands) {
        // (fewer than K: NaN below every number hid from the maxima)
        const uint64_t key = select_by_digits<DT, T>(z, V, K, hist, &sh_key);
        if (tid == 0) n_cand = 0;
        __syncthreads();
        for (int j = tid; j < n_vec; j += T) {
            float y[E];
            R::widen(load_row_vec<DT, false>(z, j, V), y);
            for (int e = 0; e < E; e++)
                if (j * E + e < V && full_key(y[e], j * E + e) >= key) {
                    const uint32_t at = atomicAdd(&n_cand, 1u);
                    if (at < kCands) cand[at] = full_key(y[e], j * E + e);
                }
        }
        __syncthreads();
        n = K;                                         // keys differ: exactly K reach the K-th
    }
    auto give = [&](int k, uint64_t key) {
        out_i[k] = (int32_t)~(uint32_t)key;
        out_v[k] = R::narrow1(key_value((uint32_t)(key >> 32)));
    };
    if (n > kCount) {
        sort_keys<T>(cand, n);
        for (int k = tid; k < K; k += T) give(k, cand[k]);
        return;
    }
    // H threads count the keys above one
    int H = 1;
    while (H < 64 && 2 * H * n <= T) H *= 2;
    for (int k0 = 0; k0 < n; k0 += T / H) {
        const int k = k0 + tid / H;
        const uint64_t mine = k < n ? cand[k] : 0;
        int rank = 0;
#pragma unroll 4
        for (int j = tid & (H - 1); j < n; j += H) rank += cand[j] > mine;
        for (int o = 1; o < H; o *= 2) rank += __shfl_xor(rank, o);
        if (k < n && rank < K && (tid & (H - 1)) == 0) give(rank, mine);
    }
}

template <ga_dtype DT, int T, int U, bool ONE> ga_status launch_top(const TopArgs& a, hipStream_t s) {
    // what the kernel takes for granted, whichever rule below chose it: a row
    // in rounds has a whole one (its loads are not masked), one that stays fits
    constexpr int E = RowVec<DT>::kElems;
    if (ONE ? ceil_div(a.V, E) > T * U : a.V / E < T * U)
        return fail(GA_ENOTSUP, "ga_top_logits: rows of %lld do not fit the kernel of %d threads", (long long)a.V, T);
    // (a launch takes fewer than 2^32 work-items along x)
    const int64_t n = a.rows.start[GA_MAX_WORKERS], wide = std::min<int64_t>(n, 1 << 20);
    const dim3 grid((unsigned)wide, (unsigned)ceil_div(n, wide));
    if (a.has_lse) top_kernel<DT, T, U, ONE, true><<<grid, T, 0, s>>>(a);
    else top_kernel<DT, T, U, ONE, false><<<grid, T, 0, s>>>(a);
    return check_launch("ga_top_logits");
}

template <ga_dtype DT> ga_status launch_rows(const TopArgs& a, hipStream_t s) {
    // Few threads where a row is short: it then waits for few others at its
    // barriers, and more rows fit a CU. The rule does not look at how many rows
    // there are. Measured, K = 16 (bf16 but where it says):
    //   65536 rows of 1000: 64 threads 104 us, 256 threads 219
    //   32768 rows of 4000: 256 threads 113 us, 512 threads 339 (an earlier build)
    //   16384 rows of 8000: 256 threads 73 us, 512 threads 143
    //   8192 rows of 16000: in rounds by 512 threads 74 us, held 83; 9000: 76 and 79;
    //     of 8000 f32: 70 and 62 (half the elements wait in as many registers)
    //   8192 rows of 32000: 512 threads 104 us, 1024 threads 169; 2048 of 32000,
    //     K = 380: 76 and 99; 2048 of 131072, K = 128: 112 and 109, K = 300: 150 and 134
    // Three quarters of the threads' maxima can bound the K-th, so more than
    // 384 slots take 1024 threads (and from 600 on, digits: see above). A row in rounds has a whole one: n > 512 * 2,
    // and n > 1024 * 2.
    const int64_t n = ceil_div(a.V, RowVec<DT>::kElems);
    if (n <= 64 * 2) return launch_top<DT, 64, 2, true>(a, s);
    if (n <= 256 * 2) return launch_top<DT, 256, 2, true>(a, s);
    if (n <= 256 * 4) return launch_top<DT, 256, 4, true>(a, s);
    if (a.K <= 384 && (DT == GA_BF16 || n > 512 * 4)) return launch_top<DT, 512, 2, false>(a, s);
    if (n <= 512 * 4) return launch_top<DT, 512, 4, true>(a, s);
    return launch_top<DT, 1024, 2, false>(a, s);
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
    if (!valid_temp(temp)) return fail(GA_EINVAL, "%s: temp must be positive and finite, and log2(e) / temp too", what);
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
    return dt == GA_BF16 ? launch_rows<GA_BF16>(a, st) : launch_rows<GA_F32>(a, st);
}
