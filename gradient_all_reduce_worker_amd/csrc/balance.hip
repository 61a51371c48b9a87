// balance.hip -- a router's balance loss over the rows of all workers, the
// tokens that every expert got, and the gradient (ga_loss.h).
//
// The loads f need the chosen experts alone (4 K bytes per row); with f known
// a row's loss term s and its gradient need that row's logits alone. So the
// indices are counted first, and the logits are read once.
#include "loss.hpp"

namespace ga {
namespace {

constexpr int kReduceCols = 64;       // experts of a workgroup that adds counts
constexpr int kReduceThreads = 1024;
constexpr int kMaxUnitBlocks = 1 << 20;

// The rows cut into units of work: worker w's rows into segments of seg_len
// rows (its groups; one segment where all rows are one group), a segment into
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
    const int32_t seg = (int32_t)(i / u.per_seg);
    int lo = 0, hi = rows.P;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (u.first[mid] <= seg) lo = mid;
        else hi = mid;
    }
    r.w = lo;
    const int64_t s0 = (int64_t)(seg - u.first[lo]) * u.seg_len;
    const int64_t end = min(s0 + u.seg_len, (int64_t)(rows.start[lo + 1] - rows.start[lo]));
    r.lo = s0 + (i % u.per_seg) * u.slice;
    r.hi = min(r.lo + u.slice, end);
    r.group = u.one_group ? 0 : seg;
    return r;
}

struct BalanceArgs {
    PtrTable logits, idx, mask, grad;
    RowMap rows;
    int32_t E, K, has_mask, has_grad;
    int64_t ld, ldg, groups;
    float scale;
    int32_t* counts;                  // [groups][E]
    int32_t* n;                       // [groups]: rows that count
    int32_t* live;                    // groups with n > 0 (several groups and a mask), or null
    double* part;                     // loss of every unit
};

// Experts named by the slots of a unit's rows, and the rows that count:
// out[unit][E + 1], or counts and n themselves where a unit is a whole group.
__global__ __launch_bounds__(kThreads) void balance_count_kernel(PtrTable idx, PtrTable mask, int has_mask,
                                                                 RowMap rows, Units units, int E, int K,
                                                                 int32_t* out, int32_t* counts, int32_t* n) {
    __shared__ int32_t hist[GA_MAX_EXPERTS + 1];
    for (int64_t i = blockIdx.x; i < units.n; i += gridDim.x) {
        const Unit u = unit_of(units, rows, i);
        for (int e = threadIdx.x; e <= E; e += kThreads) hist[e] = 0;
        __syncthreads();
        const int32_t* x = static_cast<const int32_t*>(idx.p[u.w]);
        const uint8_t* m = static_cast<const uint8_t*>(mask.p[u.w]);
        const int64_t end = u.hi * K;
        for (int64_t s = u.lo * K + threadIdx.x; s < end; s += kThreads) {
            const int e = x[s];
            if (e >= 0 && e < E && (!has_mask || m[s / K])) atomicAdd(&hist[e], 1);
        }
        if (has_mask) {
            int c = 0;
            for (int64_t r = u.lo + threadIdx.x; r < u.hi; r += kThreads) c += m[r] != 0;
            atomicAdd(&hist[E], c);
        } else if (threadIdx.x == 0 && u.hi > u.lo) {
            hist[E] = (int32_t)(u.hi - u.lo);
        }
        __syncthreads();
        if (out) {
            for (int e = threadIdx.x; e <= E; e += kThreads) out[i * (E + 1) + e] = hist[e];
        } else {
            for (int e = threadIdx.x; e < E; e += kThreads) counts[u.group * E + e] = hist[e];
            if (threadIdx.x == 0) n[u.group] = hist[E];
        }
        __syncthreads();
    }
}

// counts and n of every group from its units' (integers: any order).
__global__ __launch_bounds__(kReduceThreads) void balance_reduce_kernel(const int32_t* part, int64_t per_group,
                                                                        int64_t groups, int E, int32_t* counts,
                                                                        int32_t* n) {
    constexpr int kRows = kReduceThreads / kReduceCols;
    __shared__ int32_t sh[kRows][kReduceCols];
    const int col = threadIdx.x % kReduceCols, part_row = threadIdx.x / kReduceCols;
    const int e = blockIdx.y * kReduceCols + col;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        int32_t v = 0;
        if (e <= E)
            for (int64_t i = part_row; i < per_group; i += kRows) v += part[(g * per_group + i) * (E + 1) + e];
        sh[part_row][col] = v;
        __syncthreads();
        if (part_row == 0 && e <= E) {
            for (int k = 1; k < kRows; k++) v += sh[k][col];
            if (e < E) counts[g * E + e] = v;
            else n[g] = v;
        }
        __syncthreads();
    }
}

// Groups that hold a row that counts.
__global__ __launch_bounds__(kReduceThreads) void balance_live_kernel(const int32_t* n, int64_t groups, int32_t* live) {
    __shared__ int32_t sum;
    if (threadIdx.x == 0) sum = 0;
    __syncthreads();
    int32_t c = 0;
    for (int64_t g = threadIdx.x; g < groups; g += kReduceThreads) c += n[g] > 0;
    atomicAdd(&sum, c);
    __syncthreads();
    if (threadIdx.x == 0) *live = sum;
}

__device__ __forceinline__ double live_groups(const BalanceArgs& a) {
    if (a.live) return (double)*a.live;
    return a.groups == 1 ? (a.n[0] > 0 ? 1.0 : 0.0) : (double)a.groups;
}

// A team of L lanes per row, NV vectors per lane: lane l holds vectors
// l, l + L, .. of the row, and the loads f of those columns.
template <ga_dtype DT, int L, int NV, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void balance_rows_kernel(BalanceArgs a, Units units) {
    using R = RowVec<DT>;
    constexpr int VE = R::kElems;
    constexpr int kTeams = kThreads / L;
    __shared__ double sh[kThreads / 64];
    const int l = threadIdx.x % L, team = threadIdx.x / L;
    const int E = a.E;
    const double live = live_groups(a);
    for (int64_t i = blockIdx.x; i < units.n; i += gridDim.x) {
        const Unit u = unit_of(units, a.rows, i);
        const int32_t n = u.lo < u.hi ? a.n[u.group] : 0;
        float f[NV][VE];
        const double per_slot = n > 0 ? (double)E / ((double)a.K * (double)n) : 0.0;
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int k = 0; k < VE; k++) {
                const int e = (l + v * L) * VE + k;
                f[v][k] = e < E && n > 0 ? (float)(per_slot * (double)a.counts[u.group * E + e]) : 0.0f;
            }
        const float coef = n > 0 ? (float)((double)a.scale / (live * (double)n)) : 0.0f;
        const typename R::elem* x = static_cast<const typename R::elem*>(a.logits.p[u.w]);
        typename R::elem* g = static_cast<typename R::elem*>(a.grad.p[u.w]);
        const uint8_t* mask = static_cast<const uint8_t*>(a.mask.p[u.w]);
        double acc = 0.0;
        for (int64_t r = u.lo + team; r < u.hi; r += kTeams) {
            float p[NV][VE];
            if (a.has_mask && mask[r] == 0) {
                if (a.has_grad)
#pragma unroll
                    for (int v = 0; v < NV; v++) {
#pragma unroll
                        for (int k = 0; k < VE; k++) p[v][k] = 0.0f;
                        if ((l + v * L) * VE < E) store_row_vec<DT>(g + r * a.ldg, l + v * L, E, p[v]);
                    }
                continue;
            }
#pragma unroll
            for (int v = 0; v < NV; v++) {
                const uint4 raw = (l + v * L) * VE < E ? load_row_vec<DT, true>(x + r * a.ld, l + v * L, E)
                                                       : make_uint4(R::kEmpty, R::kEmpty, R::kEmpty, R::kEmpty);
                R::widen(raw, p[v]);
            }
            float sum = 0.0f, dot = 0.0f;
            float slope[NV][VE];
            if (SIGMOID) {
                // p holds a = sigmoid(x); a (1 - a) comes from exp(-|x|), so
                // that neither end overflows or cancels
#pragma unroll
                for (int v = 0; v < NV; v++)
#pragma unroll
                    for (int k = 0; k < VE; k++) {
                        const float x = p[v][k];
                        const float t = fast_exp2(fabsf(x) * -kLog2e);
                        const float big = __builtin_amdgcn_rcpf(1.0f + t), small = t * big;
                        p[v][k] = x < 0.0f ? small : big;
                        slope[v][k] = small * big;
                        sum += p[v][k];
                        dot += f[v][k] * p[v][k];
                    }
            } else {
                // p holds exp(x - max)
                float m = -INFINITY;
#pragma unroll
                for (int v = 0; v < NV; v++)
#pragma unroll
                    for (int k = 0; k < VE; k++) m = fmaxf(m, p[v][k]);
                m = base_of(team_reduce<L, OpMax>(m));
#pragma unroll
                for (int v = 0; v < NV; v++)
#pragma unroll
                    for (int k = 0; k < VE; k++) {
                        p[v][k] = fast_exp2((p[v][k] - m) * kLog2e);
                        sum += p[v][k];
                        dot += f[v][k] * p[v][k];
                    }
            }
            sum = team_reduce<L, OpSum>(sum);
            dot = team_reduce<L, OpSum>(dot);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const float s = dot * inv;
            if (l == 0) acc += (double)s;
            if (a.has_grad) {
                const float ci = coef * inv;
#pragma unroll
                for (int v = 0; v < NV; v++) {
#pragma unroll
                    for (int k = 0; k < VE; k++) {
                        p[v][k] = ci * (SIGMOID ? slope[v][k] : p[v][k]) * (f[v][k] - s);
                    }
                    if ((l + v * L) * VE < E) store_row_vec<DT>(g + r * a.ldg, l + v * L, E, p[v]);
                }
            }
        }
        acc = group_sum_f64<kThreads>(acc, sh);
        if (threadIdx.x == 0) a.part[i] = n > 0 ? acc / (double)n : 0.0;
    }
}

__global__ __launch_bounds__(kReduceThreads) void balance_final_kernel(BalanceArgs a, int64_t n_units, float* out) {
    __shared__ double sh[kReduceThreads / 64];
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n_units; i += kReduceThreads) v += a.part[i];
    v = group_sum_f64<kReduceThreads>(v, sh);
    if (threadIdx.x == 0) {
        const double live = live_groups(a);
        out[0] = (float)v;
        out[1] = (float)live;
        out[2] = live > 0.0 ? (float)((double)a.scale * v / live) : 0.0f;
    }
}

// ------------------------------------------------------------------ host
constexpr int64_t kCountUnits = 256, kCountSlice = 512;
constexpr int64_t kRowUnits = 2048, kRowSlice = 64;

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
        segs += group_len ? ceil_div(tokens[i], u.seg_len) : 1;
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

// Workspace: the loss of every row unit, n and `live`, the counts of every
// counting unit.
struct Layout {
    Units count, row;
    int64_t groups, n_off, hist_off, bytes;
    bool direct;                      // a counting unit is a whole group
};

Layout make_layout(const int64_t* tokens, int32_t P, int64_t E, int64_t group_len) {
    Layout l;
    l.count = make_units(tokens, P, group_len, kCountUnits, kCountSlice);
    l.row = make_units(tokens, P, group_len, kRowUnits, kRowSlice);
    l.groups = group_len ? l.count.first[GA_MAX_WORKERS] : 1;
    l.direct = l.count.n == l.groups && l.groups > 0;
    l.n_off = 8 * l.row.n;
    l.hist_off = l.n_off + 8 * ceil_div(4 * (l.groups + 1), 8);
    l.bytes = l.hist_off + (l.direct ? 0 : 4 * l.count.n * (E + 1));
    return l;
}

template <ga_dtype DT, int L, int NV>
void launch_team(const BalanceArgs& a, const Units& u, ga_score score, hipStream_t s) {
    const int blocks = (int)std::min<int64_t>(u.n, kMaxUnitBlocks);
    if (score == GA_SCORE_SIGMOID) balance_rows_kernel<DT, L, NV, true><<<blocks, kThreads, 0, s>>>(a, u);
    else balance_rows_kernel<DT, L, NV, false><<<blocks, kThreads, 0, s>>>(a, u);
}

template <ga_dtype DT>
void launch_rows(const BalanceArgs& a, const Units& u, ga_score score, hipStream_t s) {
    const int64_t nv = ceil_div(a.E, RowVec<DT>::kElems);
    if (nv <= 1) launch_team<DT, 1, 1>(a, u, score, s);
    else if (nv <= 2) launch_team<DT, 2, 1>(a, u, score, s);
    else if (nv <= 4) launch_team<DT, 4, 1>(a, u, score, s);
    else if (nv <= 8) launch_team<DT, 8, 1>(a, u, score, s);
    else if (nv <= 16) launch_team<DT, 16, 1>(a, u, score, s);
    else if (nv <= 32) launch_team<DT, 16, 2>(a, u, score, s);
    else if (nv <= 48) launch_team<DT, 16, 3>(a, u, score, s);
    else if (nv <= 64) launch_team<DT, 16, 4>(a, u, score, s);
    else if (nv <= 128) launch_team<DT, 64, 2>(a, u, score, s);
    else launch_team<DT, 64, 4>(a, u, score, s);
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
    a.part = reinterpret_cast<double*>(ws);
    a.n = reinterpret_cast<int32_t*>(ws + lay.n_off);
    a.live = mask && lay.groups > 1 ? a.n + lay.groups : nullptr;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (lay.groups > 0) {
        int32_t* hist = lay.direct ? nullptr : reinterpret_cast<int32_t*>(ws + lay.hist_off);
        balance_count_kernel<<<(int)std::min<int64_t>(lay.count.n, kMaxUnitBlocks), kThreads, 0, st>>>(
            a.idx, a.mask, a.has_mask, a.rows, lay.count, E, K, hist, d_counts, a.n);
        if ((s = check_launch(what))) return s;
        if (!lay.direct) {
            const dim3 grid((unsigned)std::min<int64_t>(lay.groups, 4096), (unsigned)ceil_div(E + 1, kReduceCols));
            balance_reduce_kernel<<<grid, kReduceThreads, 0, st>>>(hist, lay.count.n / lay.groups, lay.groups, E,
                                                                 d_counts, a.n);
            if ((s = check_launch(what))) return s;
        }
        if (a.live) {
            balance_live_kernel<<<1, kReduceThreads, 0, st>>>(a.n, lay.groups, a.live);
            if ((s = check_launch(what))) return s;
        }
        if (dt == GA_BF16) launch_rows<GA_BF16>(a, lay.row, score, st);
        else launch_rows<GA_F32>(a, lay.row, score, st);
        if ((s = check_launch(what))) return s;
    }
    balance_final_kernel<<<1, kReduceThreads, 0, st>>>(a, lay.groups > 0 ? lay.row.n : 0, d_loss);
    return check_launch(what);
}
