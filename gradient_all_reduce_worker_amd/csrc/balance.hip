// balance.hip -- a router's balance loss over the rows of all workers, the
// tokens that every expert got, and the gradient (ga_loss.h).
//
// The loads f need the chosen experts alone (4 K bytes per row); with f known
// a row's loss term s and its gradient need that row's logits alone. So the
// indices are counted first, in a few dozen partial counts, and the logits are
// read once; a workgroup that reads them adds the partial counts up for itself.
// A batch of a few rows is counted and read by one workgroup, in one launch.
//
// Bound: one read and one write of the logits, behind a chain of three launches
// (counts 6 us, rows, the last sum 4). The row kernels' registers (81 for 256
// bf16, 92 for 160 f32) allow two workgroups per CU, and each of them reads all
// partial counts of its group: as many bytes as its own rows, with 256 experts
// and 128 rows. 131072 rows of 256 bf16: 41 us,
// of which the rows take 30 to 33, 4.2 TB/s (a copy of that size 6.5); 524288 rows:
// 120 us, 4.6 TB/s; 65536 rows of 160 f32 in 16 groups: 22 us for the rows, 3.8 TB/s;
// 64 rows of 8 in one launch: 6 us.
// Not kept: the last row workgroup adding up the losses in place of the last
// launch: what it has to read must leave the other XCDs' caches first, and that
// writes all of their lines back (131072 rows of 256 bf16: 41 -> 88 us).
#include "loss.hpp"

namespace ga {
namespace {

constexpr int kCountThreads = 1024;   // (8 workers, 131072 rows: 1024 threads 43.9 us in all, 512 44.3, 256 46.1)
constexpr int kCopies = 4;            // of the counts in LDS, against bank conflicts
constexpr int kRowThreads = 512;
constexpr int kSumThreads = 1024;
constexpr int kMaxUnitBlocks = 1 << 20;

// The rows cut into units of work: worker w's rows into segments of seg_len
// rows (its groups; one segment, or none, where all rows are one group), a segment into
// per_seg slices of `slice` rows. Units are numbered segment by segment;
// first[w] is worker w's first segment.
struct Units {
    int32_t first[GA_MAX_WORKERS + 1];
    int32_t per_seg, one_group;
    int64_t seg_len, slice, n;
};

struct Unit {
    int w;                            // worker
    int64_t group, lo, hi;            // rows [lo, hi) of the worker
};

__device__ __forceinline__ Unit unit_of(const Units& u, const RowMap& rows, int64_t i) {
    Unit r;
    const uint32_t seg = (uint32_t)i / (uint32_t)u.per_seg;
    int lo = 0, hi = rows.P;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((uint32_t)u.first[mid] <= seg) lo = mid;
        else hi = mid;
    }
    r.w = lo;
    const int64_t s0 = (int64_t)(seg - (uint32_t)u.first[lo]) * u.seg_len;
    const int64_t end = min(s0 + u.seg_len, (int64_t)(rows.start[lo + 1] - rows.start[lo]));
    r.lo = s0 + (int64_t)((uint32_t)i - seg * (uint32_t)u.per_seg) * u.slice;
    r.hi = min(r.lo + u.slice, end);
    r.group = u.one_group ? 0 : (int64_t)seg;
    return r;
}

struct BalanceArgs {
    PtrTable logits, idx, mask, grad;
    RowMap rows;
    int32_t E, K, has_mask, has_grad;
    int64_t ld, ldg, groups;
    float scale;
    int32_t slices;                   // partial counts of a group
    int32_t* counts;                  // [groups][E]
    int32_t* n_part;                  // [groups][slices]: rows that count
    int32_t* e_part;                  // [groups][slices][E]: their experts
    int32_t* live;                    // groups with a row that counts (several groups and a mask), or null
    double* part;                     // loss of every row unit
    float* out;
};

// Counts the experts that the rows of u name into hist, and returns the number
// of rows that count that this thread saw.
__device__ __forceinline__ int count_rows(const BalanceArgs& a, const Unit& u, int32_t* hist, int threads) {
    if (u.lo >= u.hi) return 0;
    const int32_t* idx = static_cast<const int32_t*>(a.idx.p[u.w]) + u.lo * a.K;
    const uint8_t* m = static_cast<const uint8_t*>(a.mask.p[u.w]) + u.lo;
    const uint32_t K = (uint32_t)a.K, rows = (uint32_t)(u.hi - u.lo), slots = rows * K;
    const int E = a.E;
    auto count = [&](int e, bool on) {
        if (on && e >= 0 && e < E) atomicAdd(&hist[e], 1);
    };
    // four consecutive slots per load
    constexpr int U = 4;
    for (uint32_t s0 = 4 * threadIdx.x; s0 < slots; s0 += 4 * U * threads) {
        uint4 v[U];
#pragma unroll
        for (int i = 0; i < U; i++) {
            const uint32_t s = s0 + 4 * i * threads;
            v[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (s + 4 <= slots) {
                const u32x4_e4 r = *(const __attribute__((address_space(1))) u32x4_e4*)(idx + s);
                v[i] = make_uint4(r.x, r.y, r.z, r.w);
            } else if (s < slots) {
                v[i].x = idx[s];
                if (s + 1 < slots) v[i].y = idx[s + 1];
                if (s + 2 < slots) v[i].z = idx[s + 2];
            }
        }
#pragma unroll
        for (int i = 0; i < U; i++) {
            const uint32_t s = s0 + 4 * i * threads;
            const int e[4] = {(int)v[i].x, (int)v[i].y, (int)v[i].z, (int)v[i].w};
            uint32_t r = a.has_mask ? s / K : 0, k = s - r * K;
            bool on = !a.has_mask || (r < rows && m[r] != 0);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                count(e[q], on);
                if (a.has_mask && ++k == K) {
                    k = 0;
                    on = ++r < rows && m[r] != 0;
                }
            }
        }
    }
    if (!a.has_mask) return threadIdx.x == 0 ? (int)rows : 0;
    int n = 0;
    for (uint32_t r = threadIdx.x; r < rows; r += threads) n += m[r] != 0;
    return n;
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// The partial counts of a unit.
__global__ __launch_bounds__(kCountThreads) void balance_count_kernel(BalanceArgs a, Units units) {
    extern __shared__ int32_t hist[];                  // kCopies of E
    __shared__ int32_t n_rows;
    const int E = a.E;
    for (int64_t i = blockIdx.x; i < units.n; i += gridDim.x) {
        const Unit u = unit_of(units, a.rows, i);
        for (int e = threadIdx.x; e < kCopies * E; e += kCountThreads) hist[e] = 0;
        if (threadIdx.x == 0) n_rows = 0;
        __syncthreads();
        const int n = wave_sum(count_rows(a, u, hist + (threadIdx.x >> 6) % kCopies * E, kCountThreads));
        if ((threadIdx.x & 63) == 0) atomicAdd(&n_rows, n);
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += kCountThreads) {
            int32_t c = 0;
#pragma unroll
            for (int k = 0; k < kCopies; k++) c += hist[k * E + e];
            a.e_part[i * E + e] = c;
        }
        if (threadIdx.x == 0) a.n_part[i] = n_rows;
        __syncthreads();
    }
}

// Groups that hold a row that counts.
__global__ __launch_bounds__(kSumThreads) void balance_live_kernel(const int32_t* n_part, int64_t groups, int slices,
                                                                   int32_t* live) {
    __shared__ int32_t sum;
    if (threadIdx.x == 0) sum = 0;
    __syncthreads();
    int c = 0;
    for (int64_t g = threadIdx.x; g < groups; g += kSumThreads) {
        int any = 0;
        for (int s = 0; s < slices; s++) any |= n_part[g * slices + s];
        c += any != 0;
    }
    c = wave_sum(c);
    if ((threadIdx.x & 63) == 0) atomicAdd(&sum, c);
    __syncthreads();
    if (threadIdx.x == 0) *live = sum;
}

__device__ __forceinline__ void write_loss(float* out, float scale, double sum, double live) {
    out[0] = (float)sum;
    out[1] = (float)live;
    out[2] = live > 0.0 ? (float)((double)scale * sum / live) : 0.0f;
}

// W consecutive elements of a row as one access; W divides E, so every access
// is whole.
template <ga_dtype DT, int W> struct Piece;
template <> struct Piece<GA_F32, 4> {
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(4)));
    __device__ static __forceinline__ void widen(raw r, float* f) {
#pragma unroll
        for (int k = 0; k < 4; k++) f[k] = __uint_as_float(r[k]);
    }
    __device__ static __forceinline__ raw narrow(const float* f) {
        return raw{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};
template <> struct Piece<GA_F32, 1> {
    typedef float raw;
    __device__ static __forceinline__ void widen(raw r, float* f) { f[0] = r; }
    __device__ static __forceinline__ raw narrow(const float* f) { return f[0]; }
};
template <int N> struct PieceBf16 {                    // N pairs
    typedef uint32_t raw __attribute__((ext_vector_type(N), aligned(2)));
    __device__ static __forceinline__ void widen(raw r, float* f) {
#pragma unroll
        for (int k = 0; k < N; k++) {
            f[2 * k] = bf16_lo(r[k]);
            f[2 * k + 1] = bf16_hi(r[k]);
        }
    }
    __device__ static __forceinline__ raw narrow(const float* f) {
        raw r;
#pragma unroll
        for (int k = 0; k < N; k++) r[k] = RowVec<GA_BF16>::narrow2(f[2 * k], f[2 * k + 1]);
        return r;
    }
};
template <> struct Piece<GA_BF16, 8> : PieceBf16<4> {};
template <> struct Piece<GA_BF16, 4> : PieceBf16<2> {};
template <> struct Piece<GA_BF16, 1> {
    typedef uint16_t raw;
    __device__ static __forceinline__ void widen(raw r, float* f) { f[0] = RowVec<GA_BF16>::value(r); }
    __device__ static __forceinline__ raw narrow(const float* f) { return RowVec<GA_BF16>::narrow1(f[0]); }
};

// What the rows of a group share.
struct Group {
    const int32_t* count;             // LDS: rows per expert
    int32_t n;                        // rows that count
    double live;                      // groups that hold one
};

// Rows of one worker by teams of L lanes, NV pieces of W elements per lane:
// lane l holds pieces l, l + L, .. of a row, and the loads f of those columns.
// AHEAD of a team's rows are on their way (2 where a lane holds 16 elements of
// a row: 47.1 us, with 4 48.1).
template <ga_dtype DT, int W, int L, int NV, bool SIGMOID> struct Rows {
    using R = RowVec<DT>;
    using Pc = Piece<DT, W>;
    typedef __attribute__((address_space(1))) typename Pc::raw g_raw;
    static constexpr int kTeams = kRowThreads / L;
    static constexpr int AHEAD = NV * W <= 8 ? 4 : 2;

    typename Pc::raw raw[AHEAD][NV];
    bool is_on[AHEAD];
    int l, n_pieces;

    __device__ __forceinline__ explicit Rows(int E) : l(threadIdx.x % L), n_pieces(E / W) {}

    __device__ __forceinline__ void fetch(const BalanceArgs& a, const Unit& u, int64_t r, int h) {
        const typename R::elem* x = static_cast<const typename R::elem*>(a.logits.p[u.w]);
        const uint8_t* mask = static_cast<const uint8_t*>(a.mask.p[u.w]);
        is_on[h] = r < u.hi && !(a.has_mask && mask[r] == 0);
        if (!is_on[h]) return;
#pragma unroll
        for (int v = 0; v < NV; v++)
            if (l + v * L < n_pieces)
                raw[h][v] = __builtin_nontemporal_load((const g_raw*)(x + r * a.ld + (l + v * L) * W));
    }
    // the team's first rows
    __device__ __forceinline__ void start(const BalanceArgs& a, const Unit& u) {
#pragma unroll
        for (int h = 0; h < AHEAD; h++) fetch(a, u, u.lo + threadIdx.x / L + h * kTeams, h);
    }

    // The sum of the rows' terms s (in lane 0 of the team), and their gradients.
    __device__ __forceinline__ double run(const BalanceArgs& a, const Unit& u, const Group& gr) {
        typename R::elem* g = static_cast<typename R::elem*>(a.grad.p[u.w]);
        const double per_slot = gr.n > 0 ? (double)a.E / ((double)a.K * (double)gr.n) : 0.0;
        const float coef = gr.n > 0 ? (float)((double)a.scale / (gr.live * (double)gr.n)) : 0.0f;
        float f[NV][W];
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int k = 0; k < W; k++)
                f[v][k] = l + v * L < n_pieces ? (float)(per_slot * (double)gr.count[(l + v * L) * W + k]) : 0.0f;
        double acc = 0.0;
        const int64_t first = u.lo + threadIdx.x / L;
        for (int64_t r0 = first; r0 < u.hi; r0 += AHEAD * kTeams) {
#pragma unroll
            for (int h = 0; h < AHEAD; h++) {
                const int64_t r = r0 + h * kTeams;
                if (r >= u.hi) break;
                const bool on = is_on[h];
                float p[NV][W], slope[NV][W];
#pragma unroll
                for (int v = 0; v < NV; v++) {
                    Pc::widen(raw[h][v], p[v]);
                    if (l + v * L >= n_pieces)
#pragma unroll
                        for (int k = 0; k < W; k++) p[v][k] = -INFINITY;
                }
                fetch(a, u, r + AHEAD * kTeams, h);
                float sum = 0.0f, dot = 0.0f;
                if (SIGMOID) {
                    // p holds a = sigmoid(x); a (1 - a) comes from exp(-|x|),
                    // so that neither end overflows or cancels
#pragma unroll
                    for (int v = 0; v < NV; v++)
#pragma unroll
                        for (int k = 0; k < W; k++) {
                            const float y = p[v][k];
                            const float t = fast_exp2(fabsf(y) * -kLog2e);
                            const float big = __builtin_amdgcn_rcpf(1.0f + t), small = t * big;
                            p[v][k] = y < 0.0f ? small : big;
                            slope[v][k] = small * big;
                            sum += p[v][k];
                            dot = __builtin_fmaf(f[v][k], p[v][k], dot);
                        }
                } else {
                    // p holds exp(x - max)
                    float m = -INFINITY;
#pragma unroll
                    for (int v = 0; v < NV; v++)
#pragma unroll
                        for (int k = 0; k < W; k++) m = fmaxf(m, p[v][k]);
                    m = base_of(team_reduce<L, OpMax>(m));
#pragma unroll
                    for (int v = 0; v < NV; v++)
#pragma unroll
                        for (int k = 0; k < W; k++) {
                            p[v][k] = fast_exp2((p[v][k] - m) * kLog2e);
                            sum += p[v][k];
                            dot = __builtin_fmaf(f[v][k], p[v][k], dot);
                        }
                }
                sum = team_reduce<L, OpSum>(sum);
                dot = team_reduce<L, OpSum>(dot);
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const float s = dot * inv;
                if (l == 0 && on) acc += (double)s;
                if (a.has_grad) {
                    const float ci = coef * inv;
#pragma unroll
                    for (int v = 0; v < NV; v++) {
#pragma unroll
                        for (int k = 0; k < W; k++)
                            p[v][k] = on ? ci * (SIGMOID ? slope[v][k] : p[v][k]) * (f[v][k] - s) : 0.0f;
                        if (l + v * L < n_pieces)
                            __builtin_nontemporal_store(Pc::narrow(p[v]), (g_raw*)(g + r * a.ldg + (l + v * L) * W));
                    }
                }
                __builtin_amdgcn_sched_barrier(0);     // one row's values at a time
            }
        }
        return acc;
    }
};

// One workgroup per unit.
template <ga_dtype DT, int W, int L, int NV, bool SIGMOID>
__global__ __launch_bounds__(kRowThreads) void balance_rows_kernel(BalanceArgs a, Units units) {
    __shared__ int32_t count[GA_MAX_EXPERTS];
    __shared__ int32_t n_rows;
    __shared__ double sh[kRowThreads / 64];
    const int64_t i = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (i >= units.n) return;
    const int E = a.E;
    const Unit u = unit_of(units, a.rows, i);
    Rows<DT, W, L, NV, SIGMOID> rows(E);
    rows.start(a, u);                                  // on their way while the counts are added up
    for (int e = threadIdx.x; e < E; e += kRowThreads) count[e] = 0;
    if (threadIdx.x == 0) n_rows = 0;
    __syncthreads();
    // columns (four at a time) side by side, the slices shared out among the rest
    const int32_t* part = a.e_part + u.group * a.slices * E;
    const int step = E % 4 == 0 ? 4 : 1;
    int wide = 16;
    while (wide * step < E && wide < kRowThreads) wide *= 2;
    for (int e = threadIdx.x % wide * step; e < E; e += wide * step) {
        uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll 8
        for (int s = threadIdx.x / wide; s < a.slices; s += kRowThreads / wide) {
            const int32_t* p = part + (int64_t)s * E + e;
            if (step == 4) {
                const u32x4_e4 v = *(const __attribute__((address_space(1))) u32x4_e4*)p;
                c[0] += v.x;
                c[1] += v.y;
                c[2] += v.z;
                c[3] += v.w;
            } else {
                c[0] += *p;
            }
        }
        for (int k = 0; k < step; k++) atomicAdd(&count[e + k], (int32_t)c[k]);
    }
    int n = 0;
    for (int s = threadIdx.x; s < a.slices; s += kRowThreads) n += a.n_part[u.group * a.slices + s];
    n = wave_sum(n);
    if ((threadIdx.x & 63) == 0) atomicAdd(&n_rows, n);
    __syncthreads();
    if (units.one_group ? i == 0 : (uint32_t)i % (uint32_t)units.per_seg == 0)
        for (int e = threadIdx.x; e < E; e += kRowThreads) a.counts[u.group * E + e] = count[e];
    n = n_rows;
    const double live = a.live ? (double)*a.live : a.groups == 1 ? (n > 0 ? 1.0 : 0.0) : (double)a.groups;
    const double acc = group_sum_f64<kRowThreads>(rows.run(a, u, {count, n, live}), sh);
    if (threadIdx.x == 0) a.part[i] = n > 0 ? acc / (double)n : 0.0;
}

// One workgroup does everything: few rows, one group.
template <ga_dtype DT, int L, int NV, bool SIGMOID>
__global__ __launch_bounds__(kRowThreads) void balance_alone_kernel(BalanceArgs a, Units units) {
    __shared__ int32_t count[GA_MAX_EXPERTS];
    __shared__ int32_t n_rows;
    __shared__ double sh[kRowThreads / 64];
    const int E = a.E;
    for (int e = threadIdx.x; e < E; e += kRowThreads) count[e] = 0;
    if (threadIdx.x == 0) n_rows = 0;
    __syncthreads();
    int n = 0;
    for (int64_t i = 0; i < units.n; i++) n += count_rows(a, unit_of(units, a.rows, i), count, kRowThreads);
    n = wave_sum(n);
    if ((threadIdx.x & 63) == 0) atomicAdd(&n_rows, n);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRowThreads) a.counts[e] = count[e];
    n = n_rows;
    const double live = n > 0 ? 1.0 : 0.0;
    double acc = 0.0;
    for (int64_t i = 0; i < units.n; i++) {
        const Unit u = unit_of(units, a.rows, i);
        Rows<DT, 1, L, NV, SIGMOID> rows(E);
        rows.start(a, u);
        acc += rows.run(a, u, {count, n, live});
    }
    acc = group_sum_f64<kRowThreads>(acc, sh);
    if (threadIdx.x == 0) write_loss(a.out, a.scale, n > 0 ? acc / (double)n : 0.0, live);
}

// live: as in BalanceArgs.
__global__ __launch_bounds__(kSumThreads) void balance_final_kernel(const double* part, int64_t n_units,
                                                                    const int32_t* n_part, int slices, int64_t groups,
                                                                    const int32_t* live, float scale, float* out) {
    __shared__ double sh[kSumThreads / 64];
    double v = 0.0;
    int n = 0;
    for (int64_t i = threadIdx.x; i < n_units; i += kSumThreads) v += part[i];
    if (!live && groups == 1)
        for (int i = threadIdx.x; i < slices; i += kSumThreads) n |= n_part[i];
    const int any = __syncthreads_or(n);
    v = group_sum_f64<kSumThreads>(v, sh);
    if (threadIdx.x == 0)
        write_loss(out, scale, v, live ? (double)*live : groups == 1 ? (any ? 1.0 : 0.0) : (double)groups);
}

// ------------------------------------------------------------------ host
// 64 partial counts: every row workgroup reads them all (131072 rows of 256
// bf16: 64 units 42.1 us, 16 43.2, 32 41.8, 128 45.6; 65536 of 160 f32, masked, in
// groups: 31.9, 34.7, 32.1 and 32.2). 1024 row units, two rounds of the 512 that
// the registers allow at a time, their partial counts read while the first rows
// are on their way (of 256 bf16: 1024 units 42.1 us, 512 41.4, 2048 51.0; of 160
// f32: 31.9, 35.0 and 32.0).
constexpr int64_t kCountUnits = 64, kCountSlice = 256;
constexpr int64_t kRowUnits = 1024, kRowSlice = 64;

// Units of about n_rows / target rows each, at least `least`.
Units make_units(const int64_t* tokens, int32_t P, int64_t group_len, int64_t target, int64_t least) {
    Units u;
    int64_t rows = 0, longest = 1, segs = 0;
    for (int i = 0; i < P; i++) {
        rows += tokens[i];
        longest = std::max(longest, tokens[i]);
    }
    u.one_group = group_len == 0;
    u.seg_len = group_len ? std::min(group_len, longest) : longest;
    for (int i = 0; i < P; i++) {
        u.first[i] = (int32_t)segs;
        segs += ceil_div(tokens[i], u.seg_len);        // none of a worker without rows
    }
    for (int i = P; i <= GA_MAX_WORKERS; i++) u.first[i] = (int32_t)segs;
    u.slice = std::max(least, ceil_div(rows, target));
    u.per_seg = (int32_t)ceil_div(u.seg_len, u.slice);
    u.n = segs * u.per_seg;
    return u;
}

bool sizes_ok(const int64_t* tokens, int32_t P, int64_t group_len) {
    if (!tokens || P < 1 || P > GA_MAX_WORKERS || group_len < 0) return false;
    int64_t sum = 0;
    for (int i = 0; i < P; i++)
        if (tokens[i] < 0 || tokens[i] > INT32_MAX || (sum += tokens[i]) > INT32_MAX) return false;
    return true;
}

// Workspace: the loss of every row unit, the rows and the experts of every
// counting unit, `live`.
struct Layout {
    Units count, row;
    int64_t groups, n_off, live_off, e_off, bytes;
    int32_t slices;
};

Layout make_layout(const int64_t* tokens, int32_t P, int64_t E, int64_t group_len) {
    Layout l;
    l.count = make_units(tokens, P, group_len, kCountUnits, kCountSlice);
    l.row = make_units(tokens, P, group_len, kRowUnits, kRowSlice);
    l.groups = group_len ? l.count.first[GA_MAX_WORKERS] : 1;
    l.slices = (int32_t)(group_len ? l.count.per_seg : l.count.n);
    l.n_off = 8 * l.row.n;
    l.live_off = l.n_off + 4 * l.count.n;
    l.e_off = l.live_off + 4;
    l.bytes = l.e_off + 4 * l.count.n * E;
    return l;
}

// Elements of a piece, lanes of a team, pieces of a lane. Teams of few lanes
// have few steps to their sums, and several pieces of a lane share those: 16
// lanes, which cover whole lines, instead of as many as a row has pieces
// (131072 rows of 256 bf16: 41 and 44 us; 65536 of 160 f32: 29 and 38). Rows
// whose length no wide piece divides, and batches of a few rows, go element by
// element.
struct Team {
    int w, lanes, pieces;
};
Team team_of(int E, int w) {
    const int n = E / w;
    int lanes = w == 1 ? 8 : 1;
    while (lanes < 16 && lanes < n) lanes *= 2;
    if (w == 1) {
        if (n > 16) lanes = 64;
        int pieces = 1;
        while (lanes * pieces < n) pieces *= 2;
        return {w, lanes, pieces};
    }
    if (n <= 64) return {w, lanes, (int)ceil_div(n, lanes)};
    return {w, 64, n <= 128 ? 2 : 4};
}

// Widest pieces first; 8 bf16 elements only where teams of 4 would not leave
// fewer lanes idle (65536 rows of 160: 26.6 us by 4, 29.4 by 8; of 256: 43.3
// and 41.5).
Team team_for(int E, ga_dtype dt) {
    if (E % 4 != 0) return team_of(E, 1);
    const Team t4 = team_of(E, 4);
    if (dt == GA_F32 || E % 8 != 0) return t4;
    const Team t8 = team_of(E, 8);
    return t4.lanes * t4.pieces * 4 < t8.lanes * t8.pieces * 8 ? t4 : t8;
}

// What a launch needs beside the kernel it is of.
struct Launch {
    Units units;
    ga_score score;
    bool alone;
    hipStream_t stream;
};

template <ga_dtype DT, int W, int L, int NV> ga_status launch_team(const BalanceArgs& a, const Launch& l) {
    // what a team takes for granted, whichever rule chose it: whole pieces,
    // which cover a row
    if (a.E % W != 0 || a.E > W * L * NV)
        return fail(GA_ENOTSUP, "ga_balance_loss: rows of %d do not fit teams of %d lanes", a.E, L);
    if constexpr (W == 1)
        if (l.alone) {
            if (l.score == GA_SCORE_SIGMOID)
                balance_alone_kernel<DT, L, NV, true><<<1, kRowThreads, 0, l.stream>>>(a, l.units);
            else
                balance_alone_kernel<DT, L, NV, false><<<1, kRowThreads, 0, l.stream>>>(a, l.units);
            return check_launch("ga_balance_loss");
        }
    // (a launch takes fewer than 2^32 work-items along x)
    const int64_t wide = std::min<int64_t>(l.units.n, kMaxUnitBlocks);
    const dim3 grid((unsigned)wide, (unsigned)ceil_div(l.units.n, wide));
    if (l.score == GA_SCORE_SIGMOID)
        balance_rows_kernel<DT, W, L, NV, true><<<grid, kRowThreads, 0, l.stream>>>(a, l.units);
    else
        balance_rows_kernel<DT, W, L, NV, false><<<grid, kRowThreads, 0, l.stream>>>(a, l.units);
    return check_launch("ga_balance_loss");
}

template <ga_dtype DT, int W> ga_status launch_wide(const BalanceArgs& a, const Team& t, const Launch& l) {
    switch (t.lanes * 8 + t.pieces) {
        case 1 * 8 + 1: return launch_team<DT, W, 1, 1>(a, l);
        case 2 * 8 + 1: return launch_team<DT, W, 2, 1>(a, l);
        case 4 * 8 + 1: return launch_team<DT, W, 4, 1>(a, l);
        case 8 * 8 + 1: return launch_team<DT, W, 8, 1>(a, l);
        case 16 * 8 + 1: return launch_team<DT, W, 16, 1>(a, l);
        case 16 * 8 + 2: return launch_team<DT, W, 16, 2>(a, l);
        case 16 * 8 + 3: return launch_team<DT, W, 16, 3>(a, l);
        case 16 * 8 + 4: return launch_team<DT, W, 16, 4>(a, l);
        case 64 * 8 + 2: return launch_team<DT, W, 64, 2>(a, l);
        default: return launch_team<DT, W, 64, W < 8 ? 4 : 2>(a, l);       // E <= GA_MAX_EXPERTS
    }
}

template <ga_dtype DT> ga_status launch_single(const BalanceArgs& a, const Team& t, const Launch& l) {
    switch (t.lanes * t.pieces) {
        case 8: return launch_team<DT, 1, 8, 1>(a, l);
        case 16: return launch_team<DT, 1, 16, 1>(a, l);
        case 64: return launch_team<DT, 1, 64, 1>(a, l);
        case 128: return launch_team<DT, 1, 64, 2>(a, l);
        case 256: return launch_team<DT, 1, 64, 4>(a, l);
        case 512: return launch_team<DT, 1, 64, 8>(a, l);
        default: return launch_team<DT, 1, 64, 16>(a, l);
    }
}

ga_status launch_rows(const BalanceArgs& a, ga_dtype dt, const Team& t, const Launch& l) {
    if (dt == GA_BF16) {
        if (t.w == 8) return launch_wide<GA_BF16, 8>(a, t, l);
        if (t.w == 4) return launch_wide<GA_BF16, 4>(a, t, l);
        return launch_single<GA_BF16>(a, t, l);
    }
    if (t.w == 4) return launch_wide<GA_F32, 4>(a, t, l);
    return launch_single<GA_F32>(a, t, l);
}

}  // namespace
}  // namespace ga

using namespace ga;

extern "C" int64_t ga_balance_groups(const int64_t* tokens, int32_t P, int64_t group_len) {
    if (!sizes_ok(tokens, P, group_len)) return 0;
    if (!group_len) return 1;
    int64_t n = 0;
    for (int i = 0; i < P; i++) n += ceil_div(tokens[i], group_len);
    return n;
}

extern "C" size_t ga_balance_loss_ws_bytes(const int64_t* tokens, int32_t P, int32_t E, int64_t group_len) {
    if (!sizes_ok(tokens, P, group_len) || E < 1 || E > GA_MAX_EXPERTS) return 0;
    return (size_t)make_layout(tokens, P, E, group_len).bytes;
}

extern "C" ga_status ga_balance_loss(const void* const* logits, const int64_t* tokens, int32_t P, int32_t E,
                                     int64_t ld, ga_dtype dt, const int32_t* const* idx, int32_t K,
                                     const uint8_t* const* mask, ga_score score, int64_t group_len,
                                     float scale, void* const* grad, int64_t ldg, int32_t* d_counts,
                                     float* d_loss, void* d_ws, size_t ws_bytes, void* stream) {
    const char* what = "ga_balance_loss";
    BalanceArgs a = {};
    if (ga_status s = make_rows(tokens, P, &a.rows, what)) return s;
    if (!valid_dtype(dt)) return fail(GA_EINVAL, "%s: bad dtype", what);
    if (score != GA_SCORE_SOFTMAX && score != GA_SCORE_SIGMOID) return fail(GA_EINVAL, "%s: bad score", what);
    if (E < 1 || E > GA_MAX_EXPERTS) return fail(GA_EINVAL, "%s: E = %d outside [1, %d]", what, E, GA_MAX_EXPERTS);
    if (K < 1 || K > GA_TOP_MAX) return fail(GA_EINVAL, "%s: K = %d outside [1, %d]", what, K, GA_TOP_MAX);
    if (group_len < 0) return fail(GA_EINVAL, "%s: negative group_len", what);
    if (!valid_scalar(scale)) return fail(GA_EINVAL, "%s: scale must be finite", what);
    const int64_t n_rows = a.rows.start[GA_MAX_WORKERS];
    if (n_rows * K > INT32_MAX) return fail(GA_EINVAL, "%s: 2^31 slots or more", what);
    const Layout lay = make_layout(tokens, P, E, group_len);
    if (!d_loss || !aligned(d_loss, 4) || (lay.groups > 0 && !d_counts) || !aligned(d_counts, 4))
        return fail(GA_EINVAL, "%s: null or misaligned d_loss or d_counts", what);
    if (!d_ws || !aligned(d_ws, 8) || ws_bytes < (size_t)lay.bytes)
        return fail(GA_EINVAL, "%s: workspace null, misaligned or too small", what);
    Regions reg;
    const bool same = grad && logits && in_place(logits, grad, tokens, P);
    if (same && ldg != ld) return fail(GA_EINVAL, "%s: a gradient in place needs the logits' row stride", what);
    ga_status s;
    if ((s = check_rows(logits, tokens, P, E, ld, elem_size(dt), same, "logits", what, &a.logits, &reg))) return s;
    if ((s = check_rows((const void* const*)idx, tokens, P, K, K, 4, false, "idx", what, &a.idx, &reg))) return s;
    if (mask && (s = check_rows((const void* const*)mask, tokens, P, 1, 1, 1, false, "mask", what, &a.mask, &reg))) return s;
    if (same) a.grad = a.logits;
    else if (grad && (s = check_rows(grad, tokens, P, E, ldg, elem_size(dt), true, "grad", what, &a.grad, &reg))) return s;
    reg.add(d_counts, 4 * lay.groups * E, true);
    reg.add(d_loss, 12, true);
    reg.add(d_ws, lay.bytes, true);
    if (reg.clash()) return fail(GA_EINVAL, "%s: an output overlaps another buffer", what);

    char* ws = static_cast<char*>(d_ws);
    a.E = E;
    a.K = K;
    a.has_mask = mask != nullptr;
    a.has_grad = grad != nullptr;
    a.ld = ld;
    a.ldg = ldg;
    a.groups = lay.groups;
    a.scale = scale;
    a.counts = d_counts;
    a.out = d_loss;
    a.slices = lay.slices;
    a.part = reinterpret_cast<double*>(ws);
    a.n_part = reinterpret_cast<int32_t*>(ws + lay.n_off);
    a.e_part = reinterpret_cast<int32_t*>(ws + lay.e_off);
    a.live = mask && lay.groups > 1 ? reinterpret_cast<int32_t*>(ws + lay.live_off) : nullptr;
    hipStream_t st = static_cast<hipStream_t>(stream);
    // one launch for up to three units of rows, which its workgroup takes one
    // after another, and four rounds of the teams' rows (us on the GPU, and by
    // three launches; f32, E = 8: 64 rows 5.1 and 10.3, 128 7.4 and 10.7, 200 in
    // four units 11.3 and 10.8; workers of one row: 3 9.5 and 11.2, 4 11.9 and
    // 11.3, 8 21.6 and 11.8, 64 169 and 13; bf16, E = 256: 32 rows 7.9 and 11.6,
    // 3 workers of 10 rows 12.6 and 12.2)
    Team team = team_of(E, 1);
    int64_t n_units = 0;
    for (int i = 0; i < P; i++) n_units += ceil_div(tokens[i], lay.row.slice);
    const bool alone = lay.groups == 1 && n_units <= 3 && n_rows <= 4 * kRowThreads / team.lanes;
    if (!alone) team = team_for(E, dt);
    if (lay.groups > 0) {
        if (!alone) {
            balance_count_kernel<<<(int)std::min<int64_t>(lay.count.n, kMaxUnitBlocks), kCountThreads,
                                   4 * (size_t)kCopies * E, st>>>(a, lay.count);
            if ((s = check_launch(what))) return s;
        }
        if (a.live) {
            balance_live_kernel<<<1, kSumThreads, 0, st>>>(a.n_part, lay.groups, lay.slices, a.live);
            if ((s = check_launch(what))) return s;
        }
        if ((s = launch_rows(a, dt, team, {lay.row, score, alone, st}))) return s;
        if (alone) return GA_OK;
    }
    balance_final_kernel<<<1, kSumThreads, 0, st>>>(a.part, lay.groups > 0 ? lay.row.n : 0, a.n_part, lay.slices,
                                                   lay.groups, a.live, scale, d_loss);
    return check_launch(what);
}
