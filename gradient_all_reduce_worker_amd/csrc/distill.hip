// distill.hip -- distillation from a teacher's top logits: the forward
// divergence of the student's softmax from the teacher's known slots, with
// its gradient, over the rows of all workers (ga_loss.h gives the formulas).
//
// A row needs the maximum and the sum of exp over its V logits before a first
// gradient value can be written: it is read once into registers (up to 360 KB
// of a CU's 512), and its gradient is made from those. The weights' sum W over
// all workers comes first where there are weights; the loss is summed last.
//
// Bound: one read and one write of the logits, exp twice per element on the
// way. 4096 rows of 131072 bf16: 385 us, 5.0 TB/s (a copy gets 6.5); about 1000
// rows of 50003 f32: 90 us, 4.9; 32768 rows of 8192 f32: 395 us, 5.4; the loss alone, 2048
// rows of 65536 bf16: 47 us, 5.7 of 7 TB/s that a read gets. The rest is the time
// in which a workgroup waits for its row's sum: its loads are over, its stores
// have not begun, and the registers allow one to four others on the CU. Rows
// that do not stay in registers (the loss alone, and above 90000 f32 or 180000
// bf16) are loaded under conditions, four vectors at a time, none while the
// last are looked at; with a gradient they are read twice (1024 rows of 131072
// f32: 231 us, 151936: 283). 8 rows of 32768: 12 us in two launches, latency.
// Not kept: workgroups that take row after row and load the next one while the
// last is stored (4096 rows of 65536 bf16: 207 -> 225 us); plain stores (8192 rows of
// 16384 bf16: 202 -> 223 us); plain loads (226; 48 instead of 54 where
// the logits fit the Infinity Cache and were just written).
#include "loss.hpp"

namespace ga {
namespace {

constexpr int kWeightGroups = 64;     // partial sums of the weights
constexpr int kSumRows = 8192;        // rows of a workgroup that sums their losses
constexpr int kSumThreads = 1024;

struct DistillArgs {
    PtrTable logits, idx, vals, lse, weight, grad, row_loss;
    RowMap rows;
    int32_t K;
    int64_t V, ld, ldg;
    float temp, scale;
    int32_t vals_bf16, has_lse, has_weight, has_row_loss;
    double* part;                     // kWeightGroups sums of weights, then every row's w l
};

static_assert(sizeof(DistillArgs) + sizeof(int) <= 4096, "a launch's arguments");

__device__ __forceinline__ float weight_of(float w) { return w > 0.0f ? w : 0.0f; }

// Every step-th weight from `first`, in binary64.
__device__ __forceinline__ double weights_of(const PtrTable& weight, const RowMap& rows, int64_t first, int64_t step) {
    double v = 0.0;
    for (int w = 0; w < rows.P; w++) {
        const int n = rows.start[w + 1] - rows.start[w];
        const float* x = static_cast<const float*>(weight.p[w]);
        for (int64_t r = first; r < n; r += step) v += (double)weight_of(x[r]);
    }
    return v;
}

__global__ __launch_bounds__(kThreads) void distill_weights_kernel(PtrTable weight, RowMap rows, double* out) {
    __shared__ double sh[kThreads / 64];
    double v = weights_of(weight, rows, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
    v = group_sum_f64<kThreads>(v, sh);
    if (threadIdx.x == 0) out[blockIdx.x] = v;
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

struct Temp {
    float inv, c;                     // 1 / temp, log2(e) / temp
    __device__ __forceinline__ explicit Temp(float t) : inv(uniform(1.0f / t)), c(uniform(kLog2e / t)) {}
};

// The teacher's slots of a row in LDS.
struct Slots {
    float* q;                         // logit, then probability
    float* z;                         // the student's logit in that column
    int* col;                         // the column; -1: empty
};

template <ga_dtype DT>
__device__ __forceinline__ void put_slot(const DistillArgs& a, const Slots& s, const void* z, int k, int i, float t) {
    using R = RowVec<DT>;
    const bool on = i >= 0 && i < a.V;
    s.col[k] = on ? i : -1;
    s.z[k] = on ? R::value(static_cast<const typename R::elem*>(z)[i]) : 0.0f;
    s.q[k] = on ? t : -INFINITY;
}

// One wave turns the slots' logits into probabilities; their sum. (Without the
// teacher's own lse the largest is subtracted before the temperature divides,
// so that the ends of the type do not overflow.)
__device__ __forceinline__ float teacher_softmax(const Slots& s, int K, float inv_temp, bool has_lse, float L, int lane) {
    float m = -INFINITY;
    for (int k = lane; k < K; k += 64) m = fmaxf(m, s.q[k]);
    m = base_of(team_reduce<64, OpMax>(m));
    if (!has_lse) {
        L = 0.0f;
        for (int k = lane; k < K; k += 64) L += expf((s.q[k] - m) * inv_temp);
        L = logf(team_reduce<64, OpSum>(L));
    }
    float mass = 0.0f;
    for (int k = lane; k < K; k += 64) {
        const float t = s.q[k];
        const float q = t == -INFINITY ? 0.0f : expf((has_lse ? t * inv_temp : (t - m) * inv_temp) - L);
        s.q[k] = q;
        mass += q;
    }
    return team_reduce<64, OpSum>(mass);
}

// A thread's part of a row's maximum (*top) and sum, `shift` taken from every
// logit first. U vectors are in flight.
template <ga_dtype DT, int T, int U, bool STREAM>
__device__ __forceinline__ MaxSum row_max_sum(const void* z, int64_t V, float shift, float c, float* top, int tid) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    const int n_vec = (int)((V + E - 1) / E);
    MaxSum v = {-INFINITY, 0.0f}, total = v;
    float m = -INFINITY;
    for (int j0 = tid, p = 1; j0 < n_vec; j0 += U * T, p++) {
        uint4 u[U];
#pragma unroll
        for (int i = 0; i < U; i++)
            u[i] = j0 + i * T < n_vec ? load_row_vec<DT, STREAM>(z, j0 + i * T, V)
                                      : make_uint4(R::kEmpty, R::kEmpty, R::kEmpty, R::kEmpty);
        float x[U * E];
#pragma unroll
        for (int i = 0; i < U; i++) R::widen(u[i], x + i * E);
#pragma unroll
        for (int e = 0; e < U * E; e++) {
            x[e] -= shift;
            m = fmaxf(m, x[e]);
        }
        add_terms<U * E>(v, x, m, c);
        if ((p & (kRun - 1)) == 0) fold(total, v);
    }
    *top = m;
    if (n_vec > kRun * U * T) {
        fold(total, v);
        v = total;
    }
    return v;
}

// One row of a worker, the same for the whole workgroup.
template <ga_dtype DT> struct Row {
    typedef typename RowVec<DT>::elem elem;
    const elem* z;
    elem* g;                          // null: no gradient
    const int32_t* col;
    const uint16_t* v16;
    const float* v32;
    const float* lse;
    float* row_loss;                  // null: not wanted
    float weight;
    int64_t row;                      // of all workers' rows

    __device__ __forceinline__ Row(const DistillArgs& a, int64_t n, bool grad) : row(n) {
        const int w = worker_of(a.rows, (int32_t)n);
        const int64_t r = n - a.rows.start[w];
        z = static_cast<const elem*>(a.logits.p[w]) + r * a.ld;
        g = grad ? static_cast<elem*>(a.grad.p[w]) + r * a.ldg : nullptr;
        col = static_cast<const int32_t*>(a.idx.p[w]) + r * a.K;
        v16 = static_cast<const uint16_t*>(a.vals.p[w]) + r * a.K;
        v32 = static_cast<const float*>(a.vals.p[w]) + r * a.K;
        lse = static_cast<const float*>(a.lse.p[w]) + r;
        row_loss = a.has_row_loss ? static_cast<float*>(a.row_loss.p[w]) + r : nullptr;
        weight = a.has_weight ? weight_of(static_cast<const float*>(a.weight.p[w])[r]) : 1.0f;
    }
    __device__ __forceinline__ float val(const DistillArgs& a, int k) const {
        return a.vals_bf16 ? RowVec<GA_BF16>::value(v16[k]) : v32[k];
    }
};

// A row that does not count.
template <ga_dtype DT, int T> __device__ __forceinline__ void skip_row(const DistillArgs& a, const Row<DT>& r, int tid) {
    constexpr int E = RowVec<DT>::kElems;
    const float zero[E] = {};
    if (r.g)
        for (int j = tid; (int64_t)j * E < a.V; j += T) store_row_vec<DT>(r.g, j, a.V, zero);
    if (tid == 0) {
        a.part[kWeightGroups + r.row] = 0.0;
        if (r.row_loss) *r.row_loss = 0.0f;
    }
}

// What the gradient of a row is made from: a term of its softmax is
// ca exp2((x - shift) c - b), and a slot takes cg q off.
struct Coef {
    float c, b, shift, ca, cg;
    bool empty;                       // nothing but -inf
    __device__ __forceinline__ float term(float x) const { return ca * fast_exp2(__builtin_fmaf(x - shift, c, -b)); }
    // with shift = 0
    __device__ __forceinline__ float plain_term(float x) const { return ca * fast_exp2(__builtin_fmaf(x, c, -b)); }
};

// A thread's part of the maximum and sum of a row held in registers: N
// vectors, of which the first NV are whole rounds, and one element.
template <ga_dtype DT, int T, int NV, int N>
__device__ __forceinline__ MaxSum held_max_sum(uint4* raw, float last, int n_whole, float c, float* top) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    float m = last;
#pragma unroll
    for (int i = 0; i < N; i++) {
        float x[E];
        R::widen(raw[i], x);
#pragma unroll
        for (int e = 0; e < E; e++) m = fmaxf(m, x[e]);
        forget_derived(raw[i]);
    }
    *top = m;
    MaxSum v;
    v.m = scaled_max(-INFINITY, m, c);
    const float b = base_of(v.m);
    v.s = fast_exp2(__builtin_fmaf(last, c, -b));
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (i >= NV && i * T >= n_whole) continue;
        float x[E];
        R::widen(raw[i], x);
#pragma unroll
        for (int e = 0; e < E; e++) v.s += fast_exp2(__builtin_fmaf(x[e], c, -b));
        forget_derived(raw[i]);
    }
    return v;
}

template <ga_dtype DT, int T, int NV>
__device__ __forceinline__ uint4 load_held(const void* z, int i, int n_whole, int tid) {
    constexpr uint32_t e = RowVec<DT>::kEmpty;
    uint4 r = {e, e, e, e};
    if (i < NV || i * T + tid < n_whole) r = load_whole_vec<DT, true>(z, i * T * 16, tid * 16);
    return r;
}

// The row's sum from its threads' (holds a barrier, after which the slots can
// be read), its loss, and what its gradient is made from. W: the weights' sum.
template <ga_dtype DT, int T>
__device__ __forceinline__ Coef finish_row(const DistillArgs& a, const Temp& temp, const Row<DT>& r, const Slots& slot,
                                           MaxSum v, float top, const float* mass, double W, MaxSum* sh, float* sh_f,
                                           int tid) {
    Coef k;
    const float c = temp.c;
    v = group_max_sum<T>(v, sh);
    // A maximum so large that the terms vanish or the products with c overflow:
    // it is taken from all logits first, and the row is read anew.
    float shift = 0.0f;
    if (out_of_range(v)) {
        top = group_max<T>(top, sh_f);
        if (top != -INFINITY) {
            shift = top;
            v = group_max_sum<T>(row_max_sum<DT, T, 1, false>(r.z, a.V, shift, c, &top, tid), sh);
        }
    }
    const float b = base_of(v.m);
    k.empty = v.s == 0.0f;
    if (tid < 64) {
        // q log q is summed with -q log p slot by slot, so that a student near
        // its teacher does not lose its small difference
        const float ln_s = logf(v.s);
        float l = 0.0f, far = 0.0f;   // far: terms whose (x - shift) c overflows, times temp / 4
        for (int i = tid; i < a.K; i += 64)
            if (slot.q[i] > 0.0f && !k.empty) {
                const float z = slot.z[i], ln_q = logf(slot.q[i]);
                const float lp = __builtin_fmaf(z - shift, c, -b) * kLn2;
                if (lp == -INFINITY && z != -INFINITY)
                    far += slot.q[i] * (0.25f * a.temp * (ln_q + ln_s + b * kLn2) + (0.25f * shift - 0.25f * z));
                else
                    l += slot.q[i] * (ln_q - (lp - ln_s));
            }
        l = team_reduce<64, OpSum>(l);
        if (__any(far != 0.0f)) far = team_reduce<64, OpSum>(far);
        if (tid == 0) {
            // (temp^2 may lie outside binary32 where the loss does not)
            const double loss = (double)a.temp * ((double)a.temp * (double)l + 4.0 * (double)far);
            a.part[kWeightGroups + r.row] = (double)r.weight * loss;
            if (r.row_loss) *r.row_loss = (float)loss;
        }
    }
    k.c = c;
    k.b = b;
    k.shift = shift;
    k.cg = (float)((double)a.scale * (double)a.temp * (double)r.weight / W);
    k.ca = k.empty ? 0.0f : k.cg * *mass / v.s;
    return k;
}

// The gradient in one vector.
template <ga_dtype DT> __device__ __forceinline__ uint4 grad_vec(const Coef& k, const uint4& raw) {
    using R = RowVec<DT>;
    float x[R::kElems];
    R::widen(raw, x);
#pragma unroll
    for (int e = 0; e < R::kElems; e++) x[e] = k.plain_term(x[e]);
    return R::narrow(x);
}

// The gradient of a row that is read again.
template <ga_dtype DT, int T> __device__ __forceinline__ void grad_again(const DistillArgs& a, const Row<DT>& r, const Coef& k, int tid) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    for (int j = tid; (int64_t)j * E < a.V; j += T) {
        float x[E];
        R::widen(load_row_vec<DT, true>(r.z, j, a.V), x);
#pragma unroll
        for (int e = 0; e < E; e++) x[e] = k.term(x[e]);
        store_row_vec<DT>(r.g, j, a.V, x);
    }
}

// The columns of the slots, over what the row's own gradient left there: the
// sum of a column's slots is taken off once.
template <ga_dtype DT, int T>
__device__ __forceinline__ void grad_slots(const DistillArgs& a, const Row<DT>& r, const Slots& slot, const Coef& c, int tid) {
    const int K = a.K;
    // H threads look through the slots for those of slot k's column
    int H = 1;
    while (H < 64 && 2 * H * K <= T) H *= 2;
    for (int k0 = 0; k0 < K; k0 += T / H) {
        const int k = k0 + tid / H;
        const int i = k < K ? slot.col[k] : -1;
        float sum = 0.0f;
        int before = 0;
        for (int j = tid & (H - 1); j < K; j += H) {
            const bool same = slot.col[j] == i;
            sum += same ? slot.q[j] : 0.0f;
            before |= same && j < k;
        }
        for (int o = 1; o < H; o *= 2) {
            sum += __shfl_xor(sum, o);
            before |= __shfl_xor(before, o);
        }
        if (i >= 0 && !before && (tid & (H - 1)) == 0) r.g[i] = RowVec<DT>::narrow1(c.term(slot.z[k]) - c.cg * sum);
    }
}

// HOLD: the row is read once and stays in registers, as NV vectors per thread
//   that every thread has (whole vector i T + t in thread t), up to kMore that
//   only some have, and element t of the V % E behind the whole vectors. NV is
//   known when the kernel is compiled, so those vectors need no masks, and all
//   are asked for before the first is looked at.
// else: the row is read once for its sum, and again for the gradient.
constexpr int kMore = 2;

// One workgroup of T threads per row.
template <ga_dtype DT, int T, bool HOLD, int NV, bool GRAD>
__global__ __launch_bounds__(T) void distill_kernel(DistillArgs a, int n_weights) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    constexpr int N = NV + kMore;
    extern __shared__ float lds[];
    const Slots slot = {lds, lds + a.K, reinterpret_cast<int*>(lds + 2 * a.K)};
    __shared__ MaxSum sh[T / 64];
    __shared__ float sh_f[T / 64];
    __shared__ float s_mass;
    const int tid = threadIdx.x, lane = tid & 63;
    const int32_t n_rows = a.rows.start[GA_MAX_WORKERS];
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= n_rows) return;
    const Row<DT> r(a, row, GRAD);
    if (r.weight == 0.0f) return skip_row<DT, T>(a, r, tid);
    const Temp temp(a.temp);
    const int n_whole = (int)(a.V / E), K = a.K;

    // loads come back in the order they are asked for: the slots first, then
    // the row, then the student's logits in the slots' columns
    int col = -1;
    float val = 0.0f;
    if (tid < K) {
        col = r.col[tid];
        val = r.val(a, tid);
    }
    const float lse = a.has_lse ? *r.lse : 0.0f;
    uint4 raw[N];
    float last = -INFINITY;
    if (HOLD) {
#pragma unroll
        for (int i = 0; i < N; i++) raw[i] = load_held<DT, T, NV>(r.z, i, n_whole, tid);
        if (n_whole * E + tid < a.V) last = R::value(r.z[n_whole * E + tid]);
    }
    if (tid < K) put_slot<DT>(a, slot, r.z, tid, col, val);
    for (int k = tid + T; k < K; k += T) put_slot<DT>(a, slot, r.z, k, r.col[k], r.val(a, k));
    if (K > 64) __syncthreads();                       // slots of other waves
    if (tid < 64) {
        const float mass = teacher_softmax(slot, K, temp.inv, a.has_lse, lse, lane);
        if (lane == 0) s_mass = mass;
    }
    float top;
    const MaxSum v = HOLD ? held_max_sum<DT, T, NV, N>(raw, last, n_whole, temp.c, &top)
                          : row_max_sum<DT, T, 4, !GRAD>(r.z, a.V, 0.0f, temp.c, &top, tid);
    if (T == 64) __syncthreads();                      // the slots (a wider group has a barrier below)
    double W = (double)n_rows;
    if (GRAD && a.has_weight) W = wave_sum_f64(lane < n_weights ? a.part[lane] : 0.0);
    const Coef k = finish_row<DT, T>(a, temp, r, slot, v, top, &s_mass, W, sh, sh_f, tid);
    if (!GRAD) return;
    if (HOLD && k.shift == 0.0f) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            if (i >= NV && i * T >= n_whole) continue;
            const uint4 u = grad_vec<DT>(k, raw[i]);
            if (i < NV || i * T + tid < n_whole) store_whole_vec<DT>(r.g, i * T * 16, tid * 16, u);
        }
        if (n_whole * E + tid < a.V) r.g[n_whole * E + tid] = R::narrow1(k.plain_term(last));
    } else {
        grad_again<DT, T>(a, r, k, tid);
    }
    __syncthreads();                                   // the slots' columns are written over
    if (!k.empty) grad_slots<DT, T>(a, r, slot, k, tid);
}

// Sums of kSumRows rows' losses, for many rows.
__global__ __launch_bounds__(kSumThreads) void distill_sum_kernel(const double* rows, int64_t n, double* out) {
    __shared__ double sh[kSumThreads / 64];
    double v = 0.0;
    const int64_t end = min(((int64_t)blockIdx.x + 1) * kSumRows, n);
    for (int64_t i = (int64_t)blockIdx.x * kSumRows + threadIdx.x; i < end; i += kSumThreads) v += rows[i];
    v = group_sum_f64<kSumThreads>(v, sh);
    if (threadIdx.x == 0) out[blockIdx.x] = v;
}

// The loss from the rows' sums and the weights' sum: that of n_weights
// workgroups' sums, or n_rows without weights.
__device__ __forceinline__ void write_loss(const double* sums, int64_t n, double W, float scale, float* out,
                                           double* sh) {
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kSumThreads) v += sums[i];
    v = group_sum_f64<kSumThreads>(v, sh);
    if (threadIdx.x == 0) {
        out[0] = (float)v;
        out[1] = (float)W;
        out[2] = W > 0.0 ? (float)((double)scale * v / W) : 0.0f;
    }
}
__global__ __launch_bounds__(kSumThreads) void distill_final_kernel(const double* sums, int64_t n,
                                                                    const double* weights, int n_weights,
                                                                    double n_rows, float scale, float* out) {
    __shared__ double sh[kSumThreads / 64];
    const int lane = threadIdx.x & 63;
    const double W = n_weights ? wave_sum_f64(lane < n_weights ? weights[lane] : 0.0) : n_rows;
    write_loss(sums, n, W, scale, out, sh);
}
// ..., or that of the weights themselves.
__global__ __launch_bounds__(kSumThreads) void distill_final_weights_kernel(const double* sums, int64_t n,
                                                                            PtrTable weight, RowMap rows, float scale,
                                                                            float* out) {
    __shared__ double sh[kSumThreads / 64];
    const double W = group_sum_f64<kSumThreads>(weights_of(weight, rows, threadIdx.x, kSumThreads), sh);
    write_loss(sums, n, W, scale, out, sh);
}

// What a launch needs beside the kernel it is of.
struct Launch {
    dim3 grid;
    int n_weights;
    hipStream_t stream;
};

template <ga_dtype DT, int T, bool HOLD, int NV, bool GRAD>
ga_status launch(const DistillArgs& a, const Launch& l) {
    // what a kernel that holds the row takes for granted, whichever rule below
    // chose it: NV whole rounds, whose loads are not masked, and no more than
    // kMore besides
    const int64_t n_whole = a.V / RowVec<DT>::kElems;
    if (HOLD && (n_whole < NV * T || n_whole > (NV + kMore) * T))
        return fail(GA_ENOTSUP, "ga_distill_loss: rows of %lld do not fit the kernel of %d threads and %d rounds",
                    (long long)a.V, T, NV);
    distill_kernel<DT, T, HOLD, NV, GRAD><<<l.grid, T, 12 * (size_t)a.K, l.stream>>>(a, l.n_weights);
    return check_launch("ga_distill_loss");
}

// The row kernel with the most whole rounds of T vectors that a row of
// n_whole vectors has, MIN to NV; kMore rounds hold the rest.
template <ga_dtype DT, int T, int MIN, int NV>
ga_status launch_hold(const DistillArgs& a, const Launch& l, int64_t n_whole) {
    if constexpr (NV > MIN)
        if (n_whole < (int64_t)NV * T) return launch_hold<DT, T, MIN, NV - kMore>(a, l, n_whole);
    return launch<DT, T, true, NV, true>(a, l);
}

template <ga_dtype DT>
ga_status launch_rows(const DistillArgs& a, bool grad, const Launch& l) {
    // Few threads where a row is short: more rows are on their way at a time, and
    // few waves wait for the one with the slots. The rule does not look at how
    // many rows there are. Measured, bf16:
    //   the loss alone, 65536 rows of 1000: 64 threads 60 us, 256 threads 167;
    //     16384 rows of 8192: 51 and 61; 4096 rows of 32768: 50 and 50
    //     (512 threads 49; 65536 rows of 1000: 330)
    //   65536 rows of 1000: 64 threads 78 us, 128 threads 143, 256 threads 236
    //   32768 rows of 2500: 128 threads 83 us, 64 threads 80, 256 threads 122; 8 rows of
    //     4000: 12.5, 13.4 and 13.4; 32768 rows of 6000: 128 threads 186, 256 threads 177
    //   16384 rows of 8192: 256 threads 110 us, 512 threads 124 to 131; 4096 rows of
    //     32768: 110 and 106; f32, 4096 rows of 16384: 101 and 104
    //   2048 rows of 65536: 512 threads 104 us, 1024 threads 110
    //   2048 rows of 131072: held by 1024 threads 212 us, read twice 228; 1024 rows of
    //     160000: 137 and 145; 16 KB more per row no longer fit the registers
    const int64_t n = a.V / RowVec<DT>::kElems;
    if (!grad) {
        if (n <= 64 * 16) return launch<DT, 64, false, 0, false>(a, l);
        return launch<DT, 256, false, 0, false>(a, l);
    }
    if (n < 64 * 4) return launch_hold<DT, 64, 0, 2>(a, l, n);
    if (n < 128 * 5) return launch_hold<DT, 128, 2, 4>(a, l, n);
    if (n < 256 * 18) return launch_hold<DT, 256, 2, 16>(a, l, n);
    if (n < 512 * 18) return launch_hold<DT, 512, 8, 16>(a, l, n);
    if (n < 1024 * 22) return launch_hold<DT, 1024, 8, 20>(a, l, n);
    return launch<DT, 1024, false, 0, true>(a, l);
}

}  // namespace
}  // namespace ga

using namespace ga;

extern "C" size_t ga_distill_loss_ws_bytes(int64_t rows) {
    if (rows <= 0 || rows > INT32_MAX) return 0;
    return sizeof(double) * (size_t)(kWeightGroups + rows + (rows > 2 * kSumRows ? ceil_div(rows, kSumRows) : 0));
}

extern "C" ga_status ga_distill_loss(const void* const* logits, const int64_t* tokens, int32_t P, int64_t V,
                                     int64_t ld, ga_dtype dt, const int32_t* const* idx,
                                     const void* const* vals, ga_dtype vals_dt, const float* const* lse,
                                     int32_t K, const float* const* weight, float temp, float scale,
                                     void* const* grad, int64_t ldg, float* const* row_loss, float* d_loss,
                                     void* d_ws, size_t ws_bytes, void* stream) {
    const char* what = "ga_distill_loss";
    DistillArgs a = {};
    if (ga_status s = make_rows(tokens, P, &a.rows, what)) return s;
    if (!valid_dtype(dt) || !valid_dtype(vals_dt)) return fail(GA_EINVAL, "%s: bad dtype", what);
    if (V < 1 || V > INT32_MAX) return fail(GA_EINVAL, "%s: V = %lld outside [1, 2^31)", what, (long long)V);
    if (K < 1 || K > GA_TOP_MAX) return fail(GA_EINVAL, "%s: K = %d outside [1, %d]", what, K, GA_TOP_MAX);
    if (!valid_temp(temp)) return fail(GA_EINVAL, "%s: temp must be positive and finite, and log2(e) / temp too", what);
    if (!valid_scalar(scale)) return fail(GA_EINVAL, "%s: scale must be finite", what);
    if (!d_loss || !aligned(d_loss, 4)) return fail(GA_EINVAL, "%s: null or misaligned d_loss", what);
    const int64_t n_rows = a.rows.start[GA_MAX_WORKERS];
    if (n_rows > 0 && (!d_ws || !aligned(d_ws, 8) || ws_bytes < ga_distill_loss_ws_bytes(n_rows)))
        return fail(GA_EINVAL, "%s: workspace null, misaligned or too small", what);

    Regions reg;
    const bool same = grad && logits && in_place(logits, grad, tokens, P);
    if (same && ldg != ld) return fail(GA_EINVAL, "%s: a gradient in place needs the logits' row stride", what);
    ga_status s;
    if ((s = check_rows(logits, tokens, P, V, ld, elem_size(dt), same, "logits", what, &a.logits, &reg))) return s;
    if ((s = check_rows((const void* const*)idx, tokens, P, K, K, 4, false, "idx", what, &a.idx, &reg))) return s;
    if ((s = check_rows(vals, tokens, P, K, K, elem_size(vals_dt), false, "vals", what, &a.vals, &reg))) return s;
    if (lse && (s = check_rows((const void* const*)lse, tokens, P, 1, 1, 4, false, "lse", what, &a.lse, &reg))) return s;
    if (weight && (s = check_rows((const void* const*)weight, tokens, P, 1, 1, 4, false, "weight", what, &a.weight, &reg)))
        return s;
    if (same) a.grad = a.logits;
    else if (grad && (s = check_rows(grad, tokens, P, V, ldg, elem_size(dt), true, "grad", what, &a.grad, &reg))) return s;
    if (row_loss && (s = check_rows((const void* const*)row_loss, tokens, P, 1, 1, 4, true, "row_loss", what, &a.row_loss, &reg)))
        return s;
    reg.add(d_loss, 12, true);
    if (n_rows > 0) reg.add(d_ws, (int64_t)ga_distill_loss_ws_bytes(n_rows), true);
    if (reg.clash()) return fail(GA_EINVAL, "%s: an output overlaps another buffer", what);

    hipStream_t st = static_cast<hipStream_t>(stream);
    a.K = K;
    a.V = V;
    a.ld = ld;
    a.ldg = ldg;
    a.temp = temp;
    a.scale = scale;
    a.vals_bf16 = vals_dt == GA_BF16;
    a.has_lse = lse != nullptr;
    a.has_weight = weight != nullptr;
    a.has_row_loss = row_loss != nullptr;
    a.part = static_cast<double*>(d_ws);
    int n_weights = 0;
    const double* sums = a.part + kWeightGroups;
    int64_t n_sums = n_rows;
    if (n_rows > 0) {
        // the gradient needs their sum in every workgroup; the loss alone, once
        if (weight && (grad || n_rows > 2 * kSumRows)) {
            n_weights = (int)std::min<int64_t>(ceil_div(n_rows, kThreads), kWeightGroups);
            distill_weights_kernel<<<n_weights, kThreads, 0, st>>>(a.weight, a.rows, a.part);
            if ((s = check_launch(what))) return s;
        }
        // (a launch takes fewer than 2^32 work-items along x)
        const int64_t wide = std::min<int64_t>(n_rows, 1 << 20);
        const Launch l = {dim3((unsigned)wide, (unsigned)ceil_div(n_rows, wide)), n_weights, st};
        s = dt == GA_BF16 ? launch_rows<GA_BF16>(a, grad != nullptr, l) : launch_rows<GA_F32>(a, grad != nullptr, l);
        if (s) return s;
        if (n_rows > 2 * kSumRows) {
            n_sums = ceil_div(n_rows, kSumRows);
            distill_sum_kernel<<<(unsigned)n_sums, kSumThreads, 0, st>>>(sums, n_rows, a.part + kWeightGroups + n_rows);
            sums += n_rows;
            if ((s = check_launch(what))) return s;
        }
    }
    if (weight && !n_weights)
        distill_final_weights_kernel<<<1, kSumThreads, 0, st>>>(sums, n_sums, a.weight, a.rows, scale, d_loss);
    else
        distill_final_kernel<<<1, kSumThreads, 0, st>>>(sums, n_sums, a.part, n_weights, (double)n_rows, scale, d_loss);
    return check_launch(what);
}
