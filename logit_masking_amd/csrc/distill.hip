// distill.hip -- gfx950 kernels of the loss against a teacher's recorded top
// logits, and its gradient, over masked rows of a student's logits.
//
//   k_distill_topk   one workgroup per row
#include <math.h>

#include <algorithm>

#include "cg_internal.hpp"

namespace cg {

namespace {

constexpr int kThreads = 1024;
constexpr int kNumWaves = kThreads / 64;
static_assert(CG_MAX_TOP <= kThreads, "one thread per teacher entry");

// A saved normaliser L is rounded to |L| 2^-24, and q by as much: one above
// this (logits at a type's lowest value, say) is not used, the row is summed
// again.
constexpr float kSavedMax = 1024.f;

struct DistillArgs {
    const void *logits;
    int64_t stride;
    const uint64_t *mask;
    int wpr, V;
    const int32_t *t_ids;
    const float *t_logits;
    int k;
    float tau;
    const float *lse_in;  // the rows' normalisers, or NULL: computed here
    float *loss, *lse;    // NULL: not written
    const float *weight;
    void *grad;
    int64_t grad_stride;
};

template <int DT>
__device__ __forceinline__ float load_x(const void *p, size_t i) {
    if (DT == 0) return ((const float *)p)[i];
    return __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16);
}
template <int DT>
__device__ __forceinline__ void store_x(void *p, size_t i, float v) {
    if (DT == 0) {
        ((float *)p)[i] = v;
    } else {
        // round to nearest even; a NaN keeps a set mantissa bit
        const uint32_t u = __float_as_uint(v);
        ((uint16_t *)p)[i] =
            v != v ? (uint16_t)((u >> 16) | 0x40u) : (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
    }
}

template <class T, class F>
__device__ T block_reduce(T v, T *slots, F op) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = op(v, __shfl_xor(v, d));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slots[0];
    for (int w = 1; w < kNumWaves; w++) v = op(v, slots[w]);
    return v;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_distill_topk(DistillArgs a) {
    __shared__ double dslots[kNumWaves];
    __shared__ float fslots[kNumWaves];
    __shared__ float p_of[CG_MAX_TOP];
    __shared__ int id_of[CG_MAX_TOP];
    const int r = blockIdx.x, t = threadIdx.x;
    const char *x = (const char *)a.logits + (size_t)r * (size_t)a.stride * (DT == 0 ? 4 : 2);
    const uint64_t *mask = a.mask ? a.mask + (size_t)r * a.wpr : nullptr;
    auto fmax_op = [](float p, float q) { return fmaxf(p, q); };
    auto sum_op = [](double p, double q) { return p + q; };
    auto logit = [&](int i) -> float {  // -inf: not a candidate
        return !mask || ((mask[i >> 6] >> (i & 63)) & 1) ? load_x<DT>(x, i) : -INFINITY;
    };
    const float kk = (float)(1.4426950408889634 / (double)a.tau);

    // the normaliser: L = m / tau + ln sum 2^((x - m) kk), kept apart as m and
    // log2 of the sum; a saved one stands for a sum of 1 at m = 0
    double L, ln_sum = 0.0;
    float base = 0.f, l2s;
    const float saved = a.lse_in ? a.lse_in[r] : INFINITY;
    if (fabsf(saved) <= kSavedMax) {
        L = (double)saved;
        l2s = (float)(L * 1.4426950408889634);
    } else {
        float m = -INFINITY, s = 0.f;
        for (int i = t; i < a.V; i += kThreads) {
            const float v = logit(i);
            if (v > m) {
                s *= exp2f((m - v) * kk);
                m = v;
            }
            if (v != -INFINITY) s += v == m ? 1.f : exp2f((v - m) * kk);
        }
        const float best = block_reduce(m, fslots, fmax_op);
        double part = m == best ? (double)s : (double)s * exp2((double)(m - best) * (double)kk);
        if (s == 0.f) part = 0.0;
        const double sum = block_reduce(part, dslots, sum_op);
        ln_sum = log(sum);
        L = (double)best / (double)a.tau + ln_sum;
        base = best;
        l2s = (float)log2(sum);
    }

    // the teacher's distribution over the entries the student can take
    int id = -1;
    float s_id = -INFINITY, tl = -INFINITY;
    if (t < a.k) {
        id = a.t_ids[(size_t)r * a.k + t];
        if (id >= 0 && id < a.V) {
            s_id = logit(id);
            if (s_id != -INFINITY) tl = a.t_logits[(size_t)r * a.k + t];
        }
    }
    const float tmax = block_reduce(tl, fslots, fmax_op);
    const bool some = tmax > -INFINITY;
    const double e = tl > -INFINITY ? exp(((double)tl - (double)tmax) / (double)a.tau) : 0.0;
    const double esum = block_reduce(e, dslots, sum_op);
    const double p = some ? e / esum : 0.0;
    if (a.loss) {
        const double term = p > 0.0 ? p * ((((double)tl - (double)tmax) - ((double)s_id - (double)base)) / (double)a.tau -
                                         log(esum) + ln_sum)
                                  : 0.0;
        const double loss = block_reduce(term, dslots, sum_op);
        if (t == 0) a.loss[r] = (float)((double)a.tau * (double)a.tau * loss);
    }
    if (a.lse && t == 0) a.lse[r] = (float)L;
    if (!a.grad) return;

    // d loss / d x_v = tau (q_v - p_v), q_v = 2^((x - base) kk - l2s)
    char *g = (char *)a.grad + (size_t)r * (size_t)a.grad_stride * (DT == 0 ? 4 : 2);
    const double scale = some ? (double)a.weight[r] * (double)a.tau : 0.0;
    const float fs = (float)scale;
    for (int i = t; i < a.V; i += kThreads) {
        const float v = logit(i);
        store_x<DT>(g, i, v == -INFINITY || !some ? 0.f : exp2f(fmaf(v - base, kk, -l2s)) * fs);
    }
    if (t < a.k) {
        id_of[t] = p > 0.0 ? id : -1;
        p_of[t] = (float)p;
    }
    __syncthreads();  // and the row's stores are done before the entries' are written over them
    if (t < a.k && p > 0.0) {
        double sum = 0.0;
        for (int j = 0; j < a.k; j++) sum += id_of[j] == id ? (double)p_of[j] : 0.0;
        const double q = exp2(((double)s_id - (double)base) / (double)a.tau * 1.4426950408889634 - (double)l2s);
        store_x<DT>(g, id, (float)((q - sum) * scale));
    }
}

}  // namespace

}  // namespace cg

using namespace cg;

static int distill_arg_error(const char *msg) {
    set_error("distill_topk: %s", msg);
    return CG_E_ARG;
}

static int distill_launch(const DistillArgs &a, int32_t dtype, int32_t rows, void *stream) {
    if (dtype != 0 && dtype != 1) return distill_arg_error("dtype must be 0 (float32) or 1 (bfloat16)");
    if (rows < 0 || a.V < 1 || a.V > CG_MAX_ROW_VOCAB) return distill_arg_error("bad rows / vocab");
    if (a.k < 1 || a.k > CG_MAX_TOP) return distill_arg_error("k out of range");
    if (!(a.tau > 0.f) || a.tau > 1e30f) return distill_arg_error("temperature must be positive and finite");
    if (a.stride < a.V) return distill_arg_error("row_stride < vocab");
    if (a.mask && a.wpr < (a.V + 63) / 64) return distill_arg_error("words_per_row < ceil(vocab / 64)");
    if (a.grad && a.grad_stride < a.V) return distill_arg_error("grad_stride < vocab");
    if (rows == 0) return CG_OK;
    if (!a.logits || !a.t_ids || !a.t_logits || (a.grad && !a.weight)) return distill_arg_error("NULL device pointer");
    if (dtype == 0)
        hipLaunchKernelGGL((k_distill_topk<0>), dim3(rows), dim3(kThreads), 0, (hipStream_t)stream, a);
    else
        hipLaunchKernelGGL((k_distill_topk<1>), dim3(rows), dim3(kThreads), 0, (hipStream_t)stream, a);
    return launch_status("distill_topk");
}

extern "C" {

int cg_distill_topk(const void *d_logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                    const uint64_t *d_mask, int32_t words_per_row, const int32_t *d_teacher_ids,
                    const float *d_teacher_logits, int32_t k, float temperature, float *d_out_loss, float *d_out_lse,
                    const float *d_weight, void *d_out_grad, int64_t grad_stride, void *stream) {
    if (rows > 0 && !d_out_loss) return distill_arg_error("NULL device pointer");
    const DistillArgs a{d_logits, row_stride, d_mask,     words_per_row, vocab,    d_teacher_ids, d_teacher_logits, k,
                        temperature, nullptr, d_out_loss, d_out_lse,     d_weight, d_out_grad,    grad_stride};
    return distill_launch(a, dtype, rows, stream);
}

int cg_distill_topk_grad(const void *d_logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                         const uint64_t *d_mask, int32_t words_per_row, const int32_t *d_teacher_ids,
                         const float *d_teacher_logits, int32_t k, float temperature, const float *d_lse,
                         const float *d_weight, void *d_out_grad, int64_t grad_stride, void *stream) {
    if (rows > 0 && (!d_lse || !d_out_grad)) return distill_arg_error("NULL device pointer");
    const DistillArgs a{d_logits, row_stride, d_mask,  words_per_row, vocab,    d_teacher_ids, d_teacher_logits, k,
                        temperature, d_lse,   nullptr, nullptr,       d_weight, d_out_grad,    grad_stride};
    return distill_launch(a, dtype, rows, stream);
}

}  // extern "C"
