// distill.hip -- gfx950 kernels of the loss against a teacher's recorded top
// logits, and its gradient, over masked rows of a student's logits.
//
//   k_distill_topk   one workgroup per row; the gradient alone: some per row
//
// loss = tau^2 sum p (ln p - ln q) needs the student's normaliser, one running
// maximum and sum over the row, and k logits; its gradient is tau w (q - p):
// another pass of one exponential a logit, and the teacher's k places
// afterwards.  All of it is bound by memory: 1024 rows of 256000 bf16 are
// summed at 5.65 TB/s, both directions of 2048 x 128256 take 242 us for 1.08
// GB (4.5 TB/s; a copy of that size moves 5.0), the gradient alone of 700 x
// 50021 f32 73 us for 281 MB, whose rows start off a line (62 for 50176).
#include <math.h>

#include <algorithm>

#include "cg_internal.hpp"
#include "row_select.hpp"

namespace cg {

namespace {

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
    int span;  // pieces of a row that one workgroup writes the gradient of
};

// ---- single elements ----------------------------------------------------------
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

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// Reduces N numbers a thread over the workgroup.
template <int WAVES, int N, class T, class F>
__device__ void block_reduce(T (&v)[N], T *slots, F op) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
#pragma unroll
        for (int n = 0; n < N; n++) v[n] = op(v[n], __shfl_xor(v[n], d));
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int n = 0; n < N; n++) slots[n * WAVES + (threadIdx.x >> 6)] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; n++) v[n] = slots[n * WAVES + (threadIdx.x & (WAVES - 1))];
#pragma unroll
    for (int d = WAVES / 2; d; d >>= 1) {
#pragma unroll
        for (int n = 0; n < N; n++) v[n] = op(v[n], __shfl_xor(v[n], d));
    }
}

// ---- the row in 16-byte pieces ------------------------------------------------
// Piece q of the row lies on a 16-byte boundary: a row that starts past one by
// `skew` elements is read from the boundary, what lies before its start is
// never used.
constexpr int kBufWord3 = 0x00020000;  // raw buffer, 32-bit data format

template <int DT>
struct Pieces {
    static constexpr int kN = DT == 0 ? 4 : 8;  // elements of a piece
    static constexpr int kEs = DT == 0 ? 4 : 2;
    static constexpr uint32_t kAll = (1u << kN) - 1u;
    __amdgpu_buffer_rsrc_t rx, rm;
    char *out;  // the gradient's row
    int V, skew;
    bool masked;

    __device__ __forceinline__ Pieces(const char *row, const uint64_t *mask, char *grad, int vocab)
        : out(grad), V(vocab), masked(mask != nullptr) {
        skew = (int)(((uintptr_t)row & 15) / kEs);
        rx = __builtin_amdgcn_make_buffer_rsrc((void *)(row - skew * kEs), (short)0, ((V + skew) * kEs + 3) & ~3, kBufWord3);
        rm = __builtin_amdgcn_make_buffer_rsrc((void *)mask, (short)0, mask ? (vocab + 63) / 64 * 8 : 0, kBufWord3);
    }
    __device__ __forceinline__ int count() const { return (V + skew + kN - 1) / kN; }
    __device__ __forceinline__ int first(int q) const { return q * kN - skew; }  // id of its first element

    // The mask's bits around piece q as they lie, then those of its elements
    // that are in the row and allowed.
    __device__ __forceinline__ uint32_t ask_mask(int q) const {
        if (!masked) return 0xFFFFu;
        const int at = first(q) >> 3;
        uint32_t b = __builtin_amdgcn_raw_buffer_load_b8(rm, at, 0, 0);
        if (skew) b |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rm, at + 1, 0, 0) << 8;
        return b;
    }
    __device__ __forceinline__ uint32_t usable(int q, uint32_t raw) const {
        const int f = first(q), left = V - f;
        uint32_t b = (masked ? raw >> (f & 7) : raw) & kAll;
        if (f < 0) b &= kAll << -f;
        return left >= kN ? b : left <= 0 ? 0u : b & ((1u << left) - 1u);
    }
    // A piece without a usable element asks past the buffer's end, which reads
    // nothing; without a branch, so that loads stay in flight together.
    // ONCE: nothing reads it again (the cache policy's non-temporal bit).
    template <bool ONCE>
    __device__ __forceinline__ uint4 ask(int q, uint32_t use) const {
        return __builtin_bit_cast(
            uint4, __builtin_amdgcn_raw_buffer_load_b128(rx, use ? q * 16 : 0x7FFFFFF0, 0, ONCE ? 2 : 0));
    }
    // -inf in place of what is not usable (bfloat16: lut holds the pair
    // selects of a byte).
    __device__ __forceinline__ uint4 select(uint4 v, uint32_t use, const uint4 *lut) const {
        if (DT == 1) {
            const uint4 s = lut[use];
            v.x = (v.x & s.x) | (~s.x & 0xFF80FF80u);
            v.y = (v.y & s.y) | (~s.y & 0xFF80FF80u);
            v.z = (v.z & s.z) | (~s.z & 0xFF80FF80u);
            v.w = (v.w & s.w) | (~s.w & 0xFF80FF80u);
        } else {
            v.x = use & 1 ? v.x : 0xFF800000u;
            v.y = use & 2 ? v.y : 0xFF800000u;
            v.z = use & 4 ? v.z : 0xFF800000u;
            v.w = use & 8 ? v.w : 0xFF800000u;
        }
        return v;
    }
    static __device__ __forceinline__ void floats(uint4 v, float (&x)[kN]) {
        const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < kN; j++)
            x[j] = __uint_as_float(DT == 0 ? d[j] : (j & 1) ? d[j / 2] & 0xFFFF0000u : d[j / 2] << 16);
    }

    // Writes piece q of the gradient: the elements that are in the row.
    __device__ __forceinline__ void put(int q, const float (&g)[kN]) const {
        const int f = first(q);
        uint32_t d[4];
        if (DT == 0) {
#pragma unroll
            for (int j = 0; j < 4; j++) d[j] = __float_as_uint(g[j]);
        } else {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
            for (int j = 0; j < 4; j++)  // to nearest, ties to even
                d[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){g[2 * j], g[2 * j + 1]}, bf16x2));
        }
        if (f >= 0 && f + kN <= V) {
            // 16 bytes at any element's address: the gradient's rows need not lie as the logits' do (by
            // elements, both directions of 1024 x 128256 bf16 take 250 us, so 142; 137 on boundaries)
            typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
            typedef u32x4 u32x4_any __attribute__((aligned(2)));
            __builtin_nontemporal_store((u32x4_any){d[0], d[1], d[2], d[3]}, (u32x4_any *)(out + (size_t)f * kEs));
        } else {
#pragma unroll
            for (int j = 0; j < kN; j++) {
                if (f + j < 0 || f + j >= V) continue;
                if (DT == 0) ((uint32_t *)out)[f + j] = d[j];
                else ((uint16_t *)out)[f + j] = (uint16_t)(d[j / 2] >> (16 * (j & 1)));
            }
        }
    }
};

// Running maximum and sum of 2^((x - m) kk) of a thread's elements.  (The
// difference first: x kk alone overflows at a type's lowest value.)
struct Running {
    float m, s;
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], float kk) {
        float top = x[0];
#pragma unroll
        for (int j = 1; j < N; j++) top = fmaxf(top, x[j]);
        if (top > m) {
            s *= exp2_fast((m - top) * kk);
            m = top;
        }
        const float base = m == -INFINITY ? 0.f : m;  // only -inf so far
        float part = exp2_fast((x[0] - base) * kk);
#pragma unroll
        for (int j = 1; j < N; j++) part += exp2_fast((x[j] - base) * kk);
        s += part;
    }
};

// The gradient from an element: scale 2^((x - base) kk - l2s), 0 for -inf.
struct Slope {
    float kk, base, l2s, scale;
    bool plain;  // -inf comes out as 0 by itself: no NaN, no infinity among the above
    template <int N>
    __device__ __forceinline__ void operator()(const float (&x)[N], float (&g)[N]) const {
#pragma unroll
        for (int j = 0; j < N; j++) g[j] = exp2_fast(fmaf(x[j] - base, kk, -l2s)) * scale;
        if (!plain) {
#pragma unroll
            for (int j = 0; j < N; j++) g[j] = x[j] == -INFINITY ? 0.f : g[j];
        }
    }
};

// One row a workgroup.  HELD: pieces a thread holds in registers between the
// sum and the gradient (0: the row is read again for it).  ONCE: the sum's
// read is the only one and large beside the caches.
template <int DT, int THREADS, int HELD, bool ONCE>
__global__ __launch_bounds__(THREADS) void k_distill_topk(DistillArgs a) {
    typedef Pieces<DT> P;
    constexpr int kWaves = THREADS / 64, kN = P::kN;
    constexpr int kEntries = (CG_MAX_TOP + THREADS - 1) / THREADS;  // teacher entries a thread
    constexpr int kAhead = 4;                                      // pieces a thread asks for together
    __shared__ double dslots[2 * kWaves];
    __shared__ float fslots[2 * kWaves];
    __shared__ float p_of[CG_MAX_TOP];
    __shared__ int id_of[CG_MAX_TOP];
    __shared__ uint4 lut[DT == 1 ? 256 : 1];
    const int r = blockIdx.x, t = threadIdx.x;
    const char *x = (const char *)a.logits + (size_t)r * (size_t)a.stride * P::kEs;
    const uint64_t *mask = a.mask ? a.mask + (size_t)r * a.wpr : nullptr;
    char *g = a.grad ? (char *)a.grad + (size_t)r * (size_t)a.grad_stride * P::kEs : nullptr;
    const P row(x, mask, g, a.V);
    const int n_pieces = row.count();
    const int from = HELD ? 0 : blockIdx.y * a.span, upto = HELD ? n_pieces : min(n_pieces, from + a.span);
    auto fmax_op = [](float p, float q) { return fmaxf(p, q); };
    auto sum_op = [](double p, double q) { return p + q; };
    const float kk = (float)(1.4426950408889634 / (double)a.tau);

    // the teacher's entries, asked for before the row: three reads one after the other
    int id[kEntries];
    float s_id[kEntries], tl[kEntries];
    double p[kEntries];
    float tmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < kEntries; i++) {
        const int e = t + i * THREADS;
        id[i] = -1;
        s_id[i] = tl[i] = -INFINITY;
        if (e < a.k) {
            id[i] = a.t_ids[(size_t)r * a.k + e];
            if (id[i] >= 0 && id[i] < a.V) {
                if (!mask || ((mask[id[i] >> 6] >> (id[i] & 63)) & 1)) s_id[i] = load_x<DT>(x, id[i]);
                if (s_id[i] != -INFINITY) tl[i] = a.t_logits[(size_t)r * a.k + e];
            }
        }
        tmax = fmaxf(tmax, tl[i]);
    }
    if (DT == 1) {
        for (int v = t; v < 256; v += THREADS) {
            uint32_t m[4];
#pragma unroll
            for (int p = 0; p < 4; p++)
                m[p] = ((v >> (2 * p)) & 1 ? 0x0000FFFFu : 0u) | ((v >> (2 * p + 1)) & 1 ? 0xFFFF0000u : 0u);
            lut[v] = make_uint4(m[0], m[1], m[2], m[3]);
        }
        __syncthreads();
    }

    // the normaliser: L = m / tau + ln sum 2^((x - m) kk), kept apart as m and
    // log2 of the sum; a saved one stands for a sum of 1 at m = 0
    const float saved = a.lse_in ? a.lse_in[r] : INFINITY;
    const bool is_saved = HELD == 0 && fabsf(saved) <= kSavedMax;
    double L = (double)saved, ln_sum = 0.0;
    float base = 0.f, l2s = (float)(L * 1.4426950408889634);
    uint4 d[HELD ? HELD : 1];
    Running run{-INFINITY, 0.f};
    if (!is_saved) {
        if (HELD) {
            uint32_t use[HELD ? HELD : 1], bytes[(HELD + 3) / 4 + 1];  // four pieces' bits a word
#pragma unroll
            for (int i = 0; i < HELD; i++) use[i] = row.ask_mask(t + i * THREADS);
#pragma unroll
            for (int i = 0; i < HELD; i++) {
                const uint32_t b = row.usable(t + i * THREADS, use[i]);
                d[i] = row.template ask<ONCE>(t + i * THREADS, b);
                bytes[i / 4] = (i % 4 ? bytes[i / 4] : 0u) | b << (8 * (i % 4));
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < HELD; i++) {
                const uint32_t b = (bytes[i / 4] >> (8 * (i % 4))) & 0xFFu;
                if (__any(b != P::kAll)) d[i] = row.select(d[i], b, lut);
                if (__any(b != 0)) {
                    float v[kN];
                    P::floats(d[i], v);
                    run.add(v, kk);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            for (int q0 = t; q0 < n_pieces; q0 += kAhead * THREADS) {
                uint32_t use[kAhead];
                uint4 v4[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; i++) use[i] = row.ask_mask(q0 + i * THREADS);
#pragma unroll
                for (int i = 0; i < kAhead; i++) {
                    use[i] = row.usable(q0 + i * THREADS, use[i]);
                    v4[i] = row.template ask<ONCE>(q0 + i * THREADS, use[i]);
                }
#pragma unroll
                for (int i = 0; i < kAhead; i++) {
                    if (!__any(use[i] != 0)) continue;
                    if (__any(use[i] != P::kAll)) v4[i] = row.select(v4[i], use[i], lut);
                    float v[kN];
                    P::floats(v4[i], v);
                    run.add(v, kk);
                }
            }
        }
    }

    // both maxima, then both sums: the row's, and that of the teacher's
    // distribution over the entries the student can take
    float most[2] = {run.m, tmax};
    block_reduce<kWaves>(most, fslots, fmax_op);
    tmax = most[1];
    const bool some = tmax > -INFINITY;
    // (a thread that saw only -inf, or a NaN beside nothing else, has no maximum to scale from)
    double sum[2] = {run.m == most[0] ? (double)run.s : run.s == 0.f ? 0.0 : (double)run.s * exp_falling(((double)run.m - (double)most[0]) / (double)a.tau),
                     0.0};
#pragma unroll
    for (int i = 0; i < kEntries; i++) {
        p[i] = tl[i] > -INFINITY ? exp_falling(((double)tl[i] - (double)tmax) / (double)a.tau) : 0.0;
        sum[1] += p[i];
    }
    block_reduce<kWaves>(sum, dslots, sum_op);
    const double esum = sum[1], ln_esum = log_of(esum);
    if (!is_saved) {
        ln_sum = log_of(sum[0]);
        L = (double)most[0] / (double)a.tau + ln_sum;
        base = most[0];
        l2s = (float)(ln_sum * 1.4426950408889634);
    }
    double loss = 0.0;
#pragma unroll
    for (int i = 0; i < kEntries; i++) {
        p[i] = some ? p[i] / esum : 0.0;
        if (a.loss && p[i] > 0.0)
            loss += p[i] * ((((double)tl[i] - (double)tmax) - ((double)s_id[i] - (double)base)) / (double)a.tau - ln_esum +
                            ln_sum);
    }
    if (a.loss) {
        double whole[1] = {loss};
        block_reduce<kWaves>(whole, dslots, sum_op);
        if (t == 0) a.loss[r] = (float)((double)a.tau * (double)a.tau * whole[0]);
    }
    if (a.lse && t == 0) a.lse[r] = (float)L;
    if (!g) return;

    // d loss / d x_v = tau (q_v - p_v): first the q everywhere
    const double scale = some ? (double)a.weight[r] * (double)a.tau : 0.0;
    Slope slope{kk, base, l2s, (float)scale, false};
    slope.plain = fabsf(base) < INFINITY && fabsf(l2s) < INFINITY && fabsf(slope.scale) < INFINITY;
    auto zeros = [&](int q) {
        float z[kN];
#pragma unroll
        for (int j = 0; j < kN; j++) z[j] = 0.f;
        row.put(q, z);
    };
    if (!some) {  // nothing recorded, or nothing allowed
        for (int q = from + t; q < upto; q += THREADS) zeros(q);
        return;
    }
    if (HELD) {
#pragma unroll
        for (int i = 0; i < HELD; i++) {
            const int q = t + i * THREADS;
            if (q < n_pieces) {
                float v[kN], o[kN];
                P::floats(d[i], v);
                slope(v, o);
                row.put(q, o);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    } else {
        for (int q0 = from + t; q0 < upto; q0 += kAhead * THREADS) {
            uint32_t use[kAhead];
            uint4 v4[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; i++) use[i] = row.ask_mask(q0 + i * THREADS);
#pragma unroll
            for (int i = 0; i < kAhead; i++) {
                use[i] = row.usable(q0 + i * THREADS, use[i]);
                v4[i] = row.template ask<true>(q0 + i * THREADS, use[i]);
            }
#pragma unroll
            for (int i = 0; i < kAhead; i++) {
                const int q = q0 + i * THREADS;
                if (q >= upto) continue;
                if (!__any(use[i] != 0)) {
                    zeros(q);
                    continue;
                }
                if (__any(use[i] != P::kAll)) v4[i] = row.select(v4[i], use[i], lut);
                float v[kN], o[kN];
                P::floats(v4[i], v);
                slope(v, o);
                row.put(q, o);
            }
        }
    }
    // then the entries' places here, over what was just written
#pragma unroll
    for (int i = 0; i < kEntries; i++) {
        const int e = t + i * THREADS;
        if (e < a.k) {
            id_of[e] = p[i] > 0.0 ? id[i] : -1;
            p_of[e] = (float)p[i];
        }
    }
    __syncthreads();  // the row's stores are done as well
#pragma unroll
    for (int i = 0; i < kEntries; i++) {
        const int piece = (id[i] + row.skew) / kN;
        if (p[i] > 0.0 && piece >= from && piece < upto) {
            double own = 0.0;
            for (int j = 0; j < a.k; j++) own += id_of[j] == id[i] ? (double)p_of[j] : 0.0;
            const double y = ((double)s_id[i] - (double)base) / (double)a.tau - (is_saved ? L : ln_sum);
            const double q = y == y ? exp_falling(y) : y;
            store_x<DT>(g, id[i], (float)((q - own) * scale));
        }
    }
}

// Which variant: both directions over up to kRowsHeld rows hold them in
// registers while they fit (a row per CU: what counts is the time of one, and
// a second read would add its latency); all else is read in 512 threads a
// row, four rows a CU, where one row's sums and stores hide behind the
// others' reads and the second read comes mostly from the memory-side cache
// (2048 rows of 128256 bf16, both: 247 us, held 282; 512 of them 64, held 73;
// 256 of them 39, held 35; 24 rows of 32000 f32: held 13.4 us, read twice 17).
// A row that is read once, with more beside it than the L2s hold, is read
// non-temporally: 1024 x 256000, the loss, 101 -> 94 us.
constexpr int kRowsHeld = 256;
constexpr size_t kOnceBytes = size_t(32) << 20;  // a single read above this does not stay in the caches

// The gradient from saved normalisers needs no sum of the row, so that several
// workgroups share one until there are two a CU, each with a load in flight a
// thread at least: 24 rows of 32000 f32 15.9 -> 10.9 us, 64 of 50021 22.2 ->
// 12.5, 200 of 50021 26.1 -> 24.8; up to eight a CU take 1024 of 128256 bf16
// from 114.4 to 116.6.  Not in place, where one would overwrite logits that
// another still looks up for the teacher's ids.
constexpr int kGradGroups = 512, kGradPieces = 4 * 512;

template <int DT>
void launch_rows(DistillArgs a, int rows, hipStream_t st) {
    constexpr int kN = Pieces<DT>::kN;
    const int pieces = (a.V + kN - 1 + kN - 1) / kN;  // with the largest skew
    int parts = 1;
    if (a.lse_in && (const void *)a.grad != a.logits)
        parts = std::max(1, std::min((kGradGroups + rows - 1) / rows, (pieces + kGradPieces - 1) / kGradPieces));
    a.span = (pieces + parts - 1) / parts;
    const dim3 grid(rows, parts);
    const bool both = a.grad && !a.lse_in;
    if (both && rows <= kRowsHeld && pieces <= 16 * 1024) {
        if (pieces <= 4 * 1024) hipLaunchKernelGGL((k_distill_topk<DT, 1024, 4, false>), grid, dim3(1024), 0, st, a);
        else if (pieces <= 8 * 1024) hipLaunchKernelGGL((k_distill_topk<DT, 1024, 8, false>), grid, dim3(1024), 0, st, a);
        else hipLaunchKernelGGL((k_distill_topk<DT, 1024, 16, false>), grid, dim3(1024), 0, st, a);
    } else if (!both && (size_t)rows * (size_t)a.V * Pieces<DT>::kEs > kOnceBytes) {
        hipLaunchKernelGGL((k_distill_topk<DT, 512, 0, true>), grid, dim3(512), 0, st, a);
    } else {
        hipLaunchKernelGGL((k_distill_topk<DT, 512, 0, false>), grid, dim3(512), 0, st, a);
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
    // (log2 e / tau has to be a float32)
    if (!(a.tau >= 1e-30f) || a.tau > 1e30f) return distill_arg_error("temperature must lie in 1e-30 .. 1e30");
    if (a.stride < a.V) return distill_arg_error("row_stride < vocab");
    if (a.mask && a.wpr < (a.V + 63) / 64) return distill_arg_error("words_per_row < ceil(vocab / 64)");
    if (a.grad && a.grad_stride < a.V) return distill_arg_error("grad_stride < vocab");
    if (rows == 0) return CG_OK;
    if (!a.logits || !a.t_ids || !a.t_logits || (a.grad && !a.weight)) return distill_arg_error("NULL device pointer");
    if (dtype == 0) launch_rows<0>(a, rows, (hipStream_t)stream);
    else launch_rows<1>(a, rows, (hipStream_t)stream);
    return launch_status("distill_topk");
}

extern "C" {

int cg_distill_topk(const void *d_logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                    const uint64_t *d_mask, int32_t words_per_row, const int32_t *d_teacher_ids,
                    const float *d_teacher_logits, int32_t k, float temperature, float *d_out_loss, float *d_out_lse,
                    const float *d_weight, void *d_out_grad, int64_t grad_stride, void *stream) {
    if (rows > 0 && !d_out_loss) return distill_arg_error("NULL device pointer");
    const DistillArgs a{d_logits, row_stride, d_mask,     words_per_row, vocab,    d_teacher_ids, d_teacher_logits, k,
                        temperature, nullptr, d_out_loss, d_out_lse,     d_weight, d_out_grad,    grad_stride, 0};
    return distill_launch(a, dtype, rows, stream);
}

int cg_distill_topk_grad(const void *d_logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                         const uint64_t *d_mask, int32_t words_per_row, const int32_t *d_teacher_ids,
                         const float *d_teacher_logits, int32_t k, float temperature, const float *d_lse,
                         const float *d_weight, void *d_out_grad, int64_t grad_stride, void *stream) {
    if (rows > 0 && (!d_lse || !d_out_grad)) return distill_arg_error("NULL device pointer");
    const DistillArgs a{d_logits, row_stride, d_mask,  words_per_row, vocab,    d_teacher_ids, d_teacher_logits, k,
                        temperature, d_lse,   nullptr, nullptr,       d_weight, d_out_grad,    grad_stride, 0};
    return distill_launch(a, dtype, rows, stream);
}

}  // extern "C"
