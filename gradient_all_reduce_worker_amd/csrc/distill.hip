// distill.hip -- distillation from a teacher's top logits: the forward
// divergence of the student's softmax from the teacher's known slots, with
// its gradient, over the rows of all workers (ga_loss.h gives the formulas).
//
// A row needs the maximum and the sum of exp over its V logits before a first
// gradient value can be written. The weights' sum W over all workers comes
// first where there are weights; the loss is summed last.
#include "loss.hpp"

namespace ga {
namespace {

constexpr int kMaxGroups = 8192;      // workgroups of the row kernel; each walks its rows
constexpr int kWeightGroups = 64;     // partial sums of the weights
constexpr int kSumThreads = 1024;

struct DistillArgs {
    PtrTable logits, idx, vals, lse, weight, grad, row_loss;
    RowMap rows;
    int32_t K;
    int64_t V, ld, ldg;
    float temp, scale;
    int32_t vals_bf16, has_lse, has_weight, has_row_loss;
    double* part;                     // num of every workgroup, then kWeightGroups sums of weights
};

__device__ __forceinline__ float weight_of(float w) { return w > 0.0f ? w : 0.0f; }

// Sums of the weights of every kWeightGroups-th run of rows, in binary64.
__global__ __launch_bounds__(kThreads) void distill_weights_kernel(PtrTable weight, RowMap rows,
                                                                   double* out) {
    __shared__ double sh[kThreads / 64];
    double v = 0.0;
    for (int w = 0; w < rows.P; w++) {
        const int n = rows.start[w + 1] - rows.start[w];
        const float* x = static_cast<const float*>(weight.p[w]);
        for (int64_t r = (int64_t)blockIdx.x * kThreads + threadIdx.x; r < n; r += (int64_t)gridDim.x * kThreads)
            v += (double)weight_of(x[r]);
    }
    v = group_sum_f64<kThreads>(v, sh);
    if (threadIdx.x == 0) out[blockIdx.x] = v;
}

// One workgroup of T threads per row.
template <ga_dtype DT, int T, bool GRAD>
__global__ __launch_bounds__(T) void distill_kernel(DistillArgs a, int n_weights) {
    using R = RowVec<DT>;
    constexpr int E = R::kElems;
    extern __shared__ float slots[];                   // K teacher probabilities, student logits, columns
    float* q = slots;
    float* zs = slots + a.K;
    int* col = reinterpret_cast<int*>(slots + 2 * a.K);
    __shared__ MaxSum sh[T / 64];
    __shared__ float s_mass;
    const int tid = threadIdx.x, lane = tid & 63;
    const int32_t n_rows = a.rows.start[GA_MAX_WORKERS];
    const float inv_temp = 1.0f / a.temp, c = kLog2e / a.temp;
    const int64_t n_vec = (a.V + E - 1) / E;

    double W = (double)n_rows;
    if (a.has_weight) W = wave_sum_f64(lane < n_weights ? a.part[kMaxGroups + lane] : 0.0);
    double num = 0.0;

    for (int32_t row = blockIdx.x; row < n_rows; row += gridDim.x) {
        const int w = worker_of(a.rows, row);
        const int64_t r = row - a.rows.start[w];
        const void* z = static_cast<const typename R::elem*>(a.logits.p[w]) + r * a.ld;
        typename R::elem* g = GRAD ? static_cast<typename R::elem*>(a.grad.p[w]) + r * a.ldg : nullptr;
        const float wt = a.has_weight ? weight_of(static_cast<const float*>(a.weight.p[w])[r]) : 1.0f;
        if (wt == 0.0f) {
            if (GRAD) {
                const float zero[E] = {};
                for (int64_t v = tid; v < n_vec; v += T) store_row_vec<DT>(g, v, a.V, zero);
            }
            if (tid == 0 && a.has_row_loss) static_cast<float*>(a.row_loss.p[w])[r] = 0.0f;
            continue;
        }
        __syncthreads();                               // the slots of the row before are done with

        // the teacher's slots, in the first wave
        if (tid < 64) {
            const int32_t* ip = static_cast<const int32_t*>(a.idx.p[w]) + r * a.K;
            float mt = -INFINITY;
            for (int k = lane; k < a.K; k += 64) {
                int i = ip[k];
                const bool on = i >= 0 && i < a.V;
                const float t = (a.vals_bf16 ? RowVec<GA_BF16>::value(static_cast<const uint16_t*>(a.vals.p[w])[r * a.K + k])
                                             : static_cast<const float*>(a.vals.p[w])[r * a.K + k]) * inv_temp;
                i = on ? i : -1;
                col[k] = i;
                zs[k] = on ? R::value(static_cast<const typename R::elem*>(z)[i]) : 0.0f;
                q[k] = on ? t : -INFINITY;             // the logit for now
                mt = fmaxf(mt, q[k]);
            }
            mt = base_of(team_reduce<64, OpMax>(mt));
            float L = 0.0f;
            if (a.has_lse) L = static_cast<const float*>(a.lse.p[w])[r];
            else {
                float s = 0.0f;
                for (int k = lane; k < a.K; k += 64) s += expf(q[k] - mt);
                L = logf(team_reduce<64, OpSum>(s));
            }
            float mass = 0.0f;
            for (int k = lane; k < a.K; k += 64) {
                const float lq = a.has_lse ? q[k] - L : (q[k] - mt) - L;
                const float p = q[k] == -INFINITY ? 0.0f : expf(lq);
                q[k] = p;
                mass += p;
            }
            mass = team_reduce<64, OpSum>(mass);
            if (lane == 0) s_mass = mass;
        }

        // the row's maximum and sum of exponentials
        MaxSum v = {-INFINITY, 0.0f};
        for (int64_t j = tid; j < n_vec; j += T) {
            float x[E];
            R::widen(load_row_vec<DT, false>(z, j, a.V), x);
            float m = x[0];
#pragma unroll
            for (int e = 1; e < E; e++) m = fmaxf(m, x[e]);
            m = fmaxf(m, v.m);
            const float b = base_of(m);
            float s = v.s * fast_exp2((v.m - b) * c);
#pragma unroll
            for (int e = 0; e < E; e++) s += fast_exp2((x[e] - b) * c);
            v.m = m;
            v.s = s;
        }
        if (T == 64) __syncthreads();                  // the slots (a wider group has a barrier below)
        v = group_max_sum<T>(v, c, sh);
        const float b = base_of(v.m);
        const bool empty = v.s == 0.0f;

        if (tid < 64) {
            // q log q is summed with -q log p slot by slot, so that a student
            // near its teacher does not lose its small difference
            const float ln_s = logf(v.s);
            float l = 0.0f;
            for (int k = lane; k < a.K; k += 64)
                if (q[k] > 0.0f && !empty) l += q[k] * (logf(q[k]) - ((zs[k] - b) * inv_temp - ln_s));
            l = a.temp * a.temp * team_reduce<64, OpSum>(l);
            if (lane == 0) {
                num += (double)wt * (double)l;
                if (a.has_row_loss) static_cast<float*>(a.row_loss.p[w])[r] = l;
            }
        }
        if (GRAD) {
            const float cg = W > 0.0 ? (float)((double)a.scale * (double)a.temp * (double)wt / W) : 0.0f;
            const float ca = empty ? 0.0f : cg * s_mass / v.s;
            for (int64_t j = tid; j < n_vec; j += T) {
                float x[E];
                R::widen(load_row_vec<DT, true>(z, j, a.V), x);
#pragma unroll
                for (int e = 0; e < E; e++) x[e] = ca * fast_exp2((x[e] - b) * c);
                store_row_vec<DT>(g, j, a.V, x);
            }
            __syncthreads();                           // the slots' columns are written over
            if (!empty)
                for (int k = tid; k < a.K; k += T) {
                    const int i = col[k];
                    if (i < 0) continue;
                    float sum = 0.0f;
                    bool first = true;
                    for (int j = 0; j < a.K; j++) {
                        const bool same = col[j] == i;
                        sum += same ? q[j] : 0.0f;
                        first = first && !(same && j < k);
                    }
                    if (first) g[i] = R::narrow1(ca * fast_exp2((zs[k] - b) * c) - cg * sum);
                }
        }
    }
    if (tid == 0) a.part[blockIdx.x] = num;
}

__global__ __launch_bounds__(kSumThreads) void distill_final_kernel(const double* part, int n, int n_weights,
                                                                    double rows, float scale, float* out) {
    __shared__ double sh[kSumThreads / 64];
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kSumThreads) v += part[i];
    v = group_sum_f64<kSumThreads>(v, sh);
    const int lane = threadIdx.x & 63;
    const double W = n_weights ? wave_sum_f64(lane < n_weights ? part[kMaxGroups + lane] : 0.0) : rows;
    if (threadIdx.x == 0) {
        out[0] = (float)v;
        out[1] = (float)W;
        out[2] = W > 0.0 ? (float)((double)scale * v / W) : 0.0f;
    }
}

template <ga_dtype DT, int T>
void launch_rows(const DistillArgs& a, bool grad, int blocks, int n_weights, hipStream_t s) {
    const size_t lds = 12 * (size_t)a.K;
    if (grad) distill_kernel<DT, T, true><<<blocks, T, lds, s>>>(a, n_weights);
    else distill_kernel<DT, T, false><<<blocks, T, lds, s>>>(a, n_weights);
}

}  // namespace
}  // namespace ga

using namespace ga;

extern "C" size_t ga_distill_loss_ws_bytes(int64_t rows) {
    return rows > 0 ? sizeof(double) * (kMaxGroups + kWeightGroups) : 0;
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
    if (!(temp > 0.0f) || !valid_scalar(temp) || !valid_scalar(1.0f / temp))
        return fail(GA_EINVAL, "%s: temp must be a positive normal number", what);
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
    const int blocks = (int)std::min<int64_t>(n_rows, kMaxGroups);
    int n_weights = 0;
    if (n_rows > 0) {
        if (weight) {
            n_weights = (int)std::min<int64_t>(ceil_div(n_rows, kThreads), kWeightGroups);
            distill_weights_kernel<<<n_weights, kThreads, 0, st>>>(a.weight, a.rows, a.part + kMaxGroups);
            if ((s = check_launch(what))) return s;
        }
        if (dt == GA_BF16) launch_rows<GA_BF16, 256>(a, grad != nullptr, blocks, n_weights, st);
        else launch_rows<GA_F32, 256>(a, grad != nullptr, blocks, n_weights, st);
        if ((s = check_launch(what))) return s;
    }
    distill_final_kernel<<<1, kSumThreads, 0, st>>>(a.part, blocks, n_weights, (double)n_rows, scale, d_loss);
    return check_launch(what);
}
