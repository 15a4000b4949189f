// row_select.hpp -- order statistics of one masked row of logits, by one
// workgroup: the search that the filtered sampler and the top-logits kernel
// share.
//
// A row's candidates are the ids whose mask bit is set and whose logit is
// neither -inf nor NaN, ordered by falling logit, equal logits by rising id
// (the two zeros are one value).  Logits are compared through 32-bit keys
// that rise with the value.  A place in that order -- "rank k", "where the
// mass reaches M" -- is found digit by digit from the key's top: a pass over
// the row counts, and sums the weights of, the candidates of each value of
// the next 8 bits among those that share the digits found so far.  Counts
// are integers and weights are summed as integers of 2^-40 (the largest
// weight is 1 and a row has at most 2^22 ids, so a sum stays under 2^62):
// the order in which the LDS atomics land changes nothing.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace cg {

constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;

// A value that is alike in every lane, as a scalar: what branches on it then
// branches for the whole wave, and holds no vector register.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ bool uniform(bool v) { return __builtin_amdgcn_readfirstlane((int)v) != 0; }
__device__ __forceinline__ float uniform(float v) { return __int_as_float(uniform(__float_as_int(v))); }
__device__ __forceinline__ double uniform(double v) {
    const long long u = __double_as_longlong(v);
    return __longlong_as_double(((long long)uniform((int)(u >> 32)) << 32) | (unsigned)uniform((int)u));
}

// Keys rise with the float's value; 0 stands for "not a candidate" (below the
// key of the lowest finite float).
__device__ __forceinline__ uint32_t key_of_bits(uint32_t b) {
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint32_t candidate_key(float x) {
    x += 0.f;  // -0 becomes +0
    return x > -INFINITY ? key_of_bits(__float_as_uint(x)) : 0u;  // false for NaN too
}

// One row; DT 0: float32, 1: bfloat16.
template <int DT>
struct RowView {
    const void *x;
    const uint64_t *mask;  // NULL: every id allowed
    int V;
    __device__ __forceinline__ uint32_t key(int i) const {
        if (mask && !((mask[i >> 6] >> (i & 63)) & 1)) return 0u;
        if (DT == 0) return candidate_key(((const float *)x)[i]);
        return candidate_key(__uint_as_float((uint32_t)((const uint16_t *)x)[i] << 16));
    }
};

// e^y for y <= 0 (and a little above) to 2^-42 of itself; 0 for NaN.  y = n ln 2
// + r with |r| <= ln 2 / 2 (ln 2 in two parts, so that r is exact), e^r by its
// power series to r^10 / 10! (the next term is under 2^-42), times 2^n.  A mass
// of 2^18 such weights moves by 2^-42 of itself: the chance that this moves a
// draw over a border between 10^5 candidates is 10^-7.
//
// Its constants are put into scalar registers where they are used: kept in
// vector registers over the kernels' loops they are 30 of a thread's 128.
__device__ __forceinline__ double scalar(double c) {
    asm volatile("" : "+s"(c));
    return c;
}
__device__ __forceinline__ double exp_falling(double y) {
    y = fmax(y, -2000.0);  // under every double; NaN comes out of this as -2000
    const double n = rint(y * scalar(1.4426950408889634074));
    double r = fma(-n, scalar(6.93147180369123816490e-01), y);
    r = fma(-n, scalar(1.90821492927058770002e-10), r);
    double p = scalar(1.0 / 3628800.0);
    p = fma(p, r, scalar(1.0 / 362880.0));
    p = fma(p, r, scalar(1.0 / 40320.0));
    p = fma(p, r, scalar(1.0 / 5040.0));
    p = fma(p, r, scalar(1.0 / 720.0));
    p = fma(p, r, scalar(1.0 / 120.0));
    p = fma(p, r, scalar(1.0 / 24.0));
    p = fma(p, r, scalar(1.0 / 6.0));
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)n);
}

// ln s to within a few units of a double's last place; -inf for 0, NaN for
// NaN.  s = 2^e f with f in [sqrt(1/2), sqrt(2)), and with z = (f - 1) / (f + 1)
// ln f = 2 (z + z^3 / 3 + z^5 / 5 + ...): |z| < 0.172, so the term after
// z^21 / 21 is under 2^-57.
__device__ __forceinline__ double log_of(double s) {
    if (s == 0.0) return -INFINITY;
    double f = __builtin_amdgcn_frexp_mant(s);  // [1/2, 1)
    int e = __builtin_amdgcn_frexp_exp(s);
    if (f < 0.70710678118654752) {
        f *= 2.0;
        e--;
    }
    const double z = (f - 1.0) / (f + 1.0), y = z * z;
    double p = scalar(1.0 / 21.0);
    p = fma(p, y, scalar(1.0 / 19.0));
    p = fma(p, y, scalar(1.0 / 17.0));
    p = fma(p, y, scalar(1.0 / 15.0));
    p = fma(p, y, scalar(1.0 / 13.0));
    p = fma(p, y, scalar(1.0 / 11.0));
    p = fma(p, y, scalar(1.0 / 9.0));
    p = fma(p, y, scalar(1.0 / 7.0));
    p = fma(p, y, scalar(1.0 / 5.0));
    p = fma(p, y, scalar(1.0 / 3.0));
    p = fma(p * y, z, z);
    return fma((double)e, scalar(0.693147180559945309), 2.0 * p);
}

// Weight of a candidate under temperature: 1 at the maximum.  +inf counts as
// 1e300, so that at a maximum of +inf it weighs 1 and all else 0.
struct Weight {
    double m, inv_t;  // largest logit; 1 / T (1 for greedy rows)
    __device__ __forceinline__ Weight() {}
    __device__ __forceinline__ Weight(float largest, double inv) {
        m = fmin((double)largest, 1e300);
        inv_t = m < 1e300 ? inv : fmax(inv, 1e-200);
    }
    __device__ __forceinline__ double exponent(float x) const { return (fmin((double)x, 1e300) - m) * inv_t; }
    __device__ __forceinline__ double operator()(float x) const { return exp_falling(exponent(x)); }
    __device__ __forceinline__ float largest() const { return (float)m; }  // (1e300 is +inf again)
};
constexpr double kMassUnit = 0x1p40;
__device__ __forceinline__ uint64_t fixed_mass(double w) { return __double2ull_rn(w * kMassUnit); }

// A place in the order: the candidates before it and their mass, the value
// there, how many candidates share it.
struct Place {
    uint32_t key;
    uint32_t count;       // candidates of this value
    uint32_t above;       // candidates of larger values
    uint64_t mass_above;  // and their mass
};

struct SelectShared {
    uint32_t cnt[256];
    uint64_t mass[256];
    Place place;
    uint32_t wave[kRowWaves];
    uint64_t wave_mass[kRowWaves];
    int found;
};

__device__ __forceinline__ uint64_t shfl_up_u64(uint64_t v, int d) {
    const uint32_t lo = __shfl_up((uint32_t)v, d), hi = __shfl_up((uint32_t)(v >> 32), d);
    return ((uint64_t)hi << 32) | lo;
}

// The largest key of the row (0: no candidate).
template <int DT>
__device__ uint32_t row_max_key(const RowView<DT> &row, SelectShared &sh) {
    uint32_t best = 0;
    for (int i = threadIdx.x; i < row.V; i += kRowThreads) best = max(best, row.key(i));
#pragma unroll
    for (int d = 32; d; d >>= 1) best = max(best, (uint32_t)__shfl_xor((int)best, d));
    if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = best;
    __syncthreads();
    best = 0;
#pragma unroll 1
    for (int w = 0; w < kRowWaves; w++) best = max(best, sh.wave[w]);
    __syncthreads();
    return uniform(best);
}

// Mass and number of the candidates of keys >= least.
template <int DT>
__device__ uint64_t row_mass(const RowView<DT> &row, const Weight &weight, uint32_t least, SelectShared &sh) {
    uint64_t s = 0;
    for (int i = threadIdx.x; i < row.V; i += kRowThreads) {
        const uint32_t k = row.key(i);
        if (k && k >= least) s += fixed_mass(weight(value_of_key(k)));
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint32_t lo = __shfl_xor((uint32_t)s, d), hi = __shfl_xor((uint32_t)(s >> 32), d);
        s += ((uint64_t)hi << 32) | lo;
    }
    if ((threadIdx.x & 63) == 0) sh.wave_mass[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0;
#pragma unroll 1
    for (int w = 0; w < kRowWaves; w++) s += sh.wave_mass[w];
    __syncthreads();
    return (uint64_t)uniform((uint32_t)(s >> 32)) << 32 | uniform((uint32_t)s);
}

// The place of the candidate of rank `rank` (BY_MASS false) or of the first
// one whose mass, with everything before it, is more than `mass` (true); the
// last candidate if there is no such one.  The row has a candidate.
template <int DT, bool BY_MASS>
__device__ Place row_find(const RowView<DT> &row, const Weight &weight, uint32_t rank, uint64_t mass,
                          SelectShared &sh) {
    uint32_t prefix = 0, above = 0, count = 0;
    uint64_t mass_above = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) {
            sh.cnt[threadIdx.x] = 0;
            sh.mass[threadIdx.x] = 0;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < row.V; i += kRowThreads) {
            const uint32_t k = row.key(i);
            if (!k || (shift < 24 && (k >> (shift + 8)) != prefix)) continue;
            // lanes that hold the first lane's value count together: a run of one
            // value would queue at one address
            const uint32_t d = (k >> shift) & 255u, k0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)k);
            const uint64_t same = __ballot(k == k0);
            const uint64_t m = fixed_mass(weight(value_of_key(k)));
            const uint32_t n = __popcll(same);
            if (k != k0 || (threadIdx.x & 63) == (uint32_t)__builtin_ctzll(same)) {
                const uint32_t c = k == k0 ? n : 1u;
                atomicAdd(&sh.cnt[d], c);
                atomicAdd((unsigned long long *)&sh.mass[d], (unsigned long long)(m * c));
            }
        }
        __syncthreads();
        if (threadIdx.x < 64) {  // lane l: the digits 255 - 4l downwards
            const int lane = threadIdx.x;
            uint32_t c = 0;
            uint64_t m = 0;
            for (int j = 0; j < 4; j++) {
                c += sh.cnt[255 - 4 * lane - j];
                m += sh.mass[255 - 4 * lane - j];
            }
            uint32_t ci = c;
            uint64_t mi = m;
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t oc = __shfl_up(ci, d);
                const uint64_t om = shfl_up_u64(mi, d);
                if (lane >= d) {
                    ci += oc;
                    mi += om;
                }
            }
            uint32_t ca = above + ci - c;
            uint64_t ma = mass_above + mi - m;
            // the lane whose digits hold the place; failing that the last one with a candidate
            const uint64_t hit = __ballot(BY_MASS ? ma + m > mass : ca + c > rank);
            const uint64_t some = __ballot(c != 0);
            const uint64_t hold = hit & some;
            const int at = hold ? __builtin_ctzll(hold) : 63 - __builtin_clzll(some);
            if (lane == at) {
                Place p{};
                for (int j = 0; j < 4; j++) {
                    const int d = 255 - 4 * lane - j;
                    const uint32_t dc = sh.cnt[d];
                    const uint64_t dm = sh.mass[d];
                    if (dc) {
                        p = Place{(prefix << 8) | (uint32_t)d, dc, ca, ma};
                        if (BY_MASS ? ma + dm > mass : ca + dc > rank) break;
                    }
                    ca += dc;
                    ma += dm;
                }
                sh.place = p;
            }
        }
        __syncthreads();
        prefix = uniform(sh.place.key);
        above = uniform(sh.place.above);
        mass_above = (uint64_t)uniform((uint32_t)(sh.place.mass_above >> 32)) << 32 | uniform((uint32_t)sh.place.mass_above);
        count = uniform(sh.place.count);
        __syncthreads();
    }
    return Place{prefix, count, above, mass_above};
}

// The id of the n-th candidate (from 0) of key `key`, in rising id order; the
// row has more than n of them.
template <int DT>
__device__ int row_nth(const RowView<DT> &row, uint32_t key, uint32_t n, SelectShared &sh) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t before = 0;
    if (threadIdx.x == 0) sh.found = -1;
    __syncthreads();
    for (int base = 0; base < row.V; base += kRowThreads) {
        const int i = base + threadIdx.x;
        const uint64_t hits = __ballot(i < row.V && row.key(i) == key);
        if (lane == 0) sh.wave[wave] = __popcll(hits);
        __syncthreads();
        uint32_t mine = before;
#pragma unroll 1
        for (int w = 0; w < kRowWaves; w++) {
            if (w < wave) mine += sh.wave[w];
            before += uniform(sh.wave[w]);
        }
        mine += __popcll(hits & ((1ull << lane) - 1));
        if (((hits >> lane) & 1) && mine == n) sh.found = i;
        __syncthreads();
        if (before > n) break;  // uniform: every thread has the same sums
    }
    return uniform(sh.found);
}

}  // namespace cg
