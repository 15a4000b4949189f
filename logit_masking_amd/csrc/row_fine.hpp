// row_fine.hpp -- the order of one masked row of float32 logits, by one
// workgroup.
//
// The counts of row_hist.hpp by the logits' upper 16 bits place every rank
// within its bin.  What is exact comes from a window: the candidates of whole
// bins, at most kWindow of them, gathered and sorted.  A filter that needs the
// row's mass, or what lies above a window that does not start at the top, has
// one pass over the row take one exponential per candidate, into the sum and
// into cells, one for each of the 1024 bins from the largest candidate's on:
// their running sums say in which bin a mass is reached, and what lies above
// every later window.  Beyond the cells (eight powers of two from the largest
// logit) a mass is looked for around where the bins' middle values put it, the
// mass above a window summed with it, and further on where that was wrong.  All comes out as ranks: top-k, top-p and min-p each keep the
// ranks below some number.
//
// 64 rows of 32000, the slowest of which cuts by min-p past its 1024th rank:
// 46 us.  Of these the read and the counts take 3, the pass with the
// exponentials 11 (about 45 instructions each for 32 logits a thread), a
// window 8 to 10: 3 to 4 to choose it, by one wave's searches, 3 to gather, 3
// to sort it and sum its weights.  Before the cells every window's own pass
// took the exponentials above it again: 57 us.
#pragma once
#include "row_hist.hpp"

namespace cg {

constexpr int kFinePieceIds = 4 * kRowThreads;  // ids of one 16-byte load of every thread
constexpr uint32_t kWindow = 1024;              // candidates of a window: one a thread
constexpr uint32_t kNegInf = 0xFF800000u;
constexpr uint32_t kLowest32 = 0xFF7FFFFFu;   // the lowest value's bits; only -inf's are larger here
constexpr uint32_t kLeastKey = 0x00800000u;  // of the type's lowest value

// The row: NP pieces a thread in registers; with SPANS, longer rows in spans
// of NP, read again by every pass.  SUM: each thread also keeps the maximum
// of its candidates and the sum of e^(x - maximum), in float32.
template <int NP, bool SPANS, bool SUM>
struct FineRow {
    static constexpr int kSpan = NP * kFinePieceIds;
    static constexpr bool kExact = false;  // a position is a bin of 2^16 values
    // A bin by its middle, no larger than the largest candidate.
    static __device__ __forceinline__ float bin_value(uint32_t bits, float most) {
        return bits == (uint32_t)kInfIdx ? INFINITY : fminf(__uint_as_float(bits << 16 | 0x8000u), most);
    }
    __amdgpu_buffer_rsrc_t rx, rm;
    const float *x;
    const uint64_t *mask;
    int V, skew;
    uint32_t d[NP][4];
    float run_max = -INFINITY, run_sum = 0.f;

    __device__ void init(const void *logits, const uint64_t *m, int vocab) {
        x = (const float *)logits;
        mask = m;
        V = vocab;
        skew = (int)(((uintptr_t)logits & 15) >> 2);
        rx = __builtin_amdgcn_make_buffer_rsrc((void *)(x - skew), (short)0, (V + skew) * 4, kBufWord3);
        rm = __builtin_amdgcn_make_buffer_rsrc((void *)m, (short)0, m ? (vocab + 63) / 64 * 8 : 0, kBufWord3);
    }
    __device__ int spans() const { return SPANS ? (V + skew + kSpan - 1) / kSpan : 1; }
    __device__ int first_id(int span, int p) const {
        return span * kSpan + p * kFinePieceIds + (int)threadIdx.x * 4 - skew;
    }
    __device__ __forceinline__ uint32_t usable(int span, int p, uint32_t raw) const {
        const int f = first_id(span, p), left = V - f;
        uint32_t b = (mask ? raw >> (f & 7) : raw) & 0xFu;
        if (f < 0) b &= 0xFu << -f;
        return left >= 4 ? b : left <= 0 ? 0u : b & ((1u << left) - 1u);
    }
    // Reads a span: what is no candidate (masked, -inf, NaN) as -inf, zeros as +0.
    __device__ __forceinline__ void ask_mask(int span, uint32_t (&raw)[NP]) const {
#pragma unroll
        for (int p = 0; p < NP; p++) {
            raw[p] = 0xFFFFu;
            if (mask) {
                const int at = first_id(span, p) >> 3;
                raw[p] = __builtin_amdgcn_raw_buffer_load_b8(rm, at, 0, 0);
                if (skew) raw[p] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rm, at + 1, 0, 0) << 8;
            }
        }
    }
    static constexpr int kWords = (NP + 7) / 8;
    __device__ __forceinline__ void ask(int span, const uint32_t (&raw)[NP], uint32_t (&bits)[kWords]) {
#pragma unroll
        for (int p = 0; p < NP; p++) {
            const uint32_t b = usable(span, p, raw[p]);
            bits[p / 8] = (p % 8 ? bits[p / 8] : 0u) | b << (4 * (p % 8));
            const uint4 v = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                                          rx, b ? (first_id(span, p) + skew) * 4 : 0x7FFFFFF0, 0, 0));
            d[p][0] = v.x; d[p][1] = v.y; d[p][2] = v.z; d[p][3] = v.w;
        }
    }
    __device__ __forceinline__ void select(int p, const uint32_t (&bits)[kWords]) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float v = __uint_as_float(d[p][j]) + 0.f;
            d[p][j] = ((bits[p / 8] >> (4 * (p % 8) + j)) & 1) && v > -INFINITY ? __float_as_uint(v) : kNegInf;
        }
    }
    __device__ __forceinline__ void load(int span) {
        uint32_t raw[NP], bits[kWords];
        ask_mask(span, raw);
        ask(span, raw, bits);
#pragma unroll
        for (int p = 0; p < NP; p++) select(p, bits);
    }
    __device__ __forceinline__ void add(const float (&v)[4]) {
        const float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
        constexpr float kLog2e = 1.4426950408889634f;
        if (top > run_max) {
            run_sum *= __builtin_amdgcn_exp2f((run_max - top) * kLog2e);
            run_max = top;
        }
        const float base = run_max == -INFINITY ? 0.f : run_max;  // only -inf so far
#pragma unroll
        for (int j = 0; j < 4; j++) run_sum += __builtin_amdgcn_exp2f((v[j] - base) * kLog2e);
    }

    // Reads and counts the row and finds its largest key.
    template <class F>
    __device__ __forceinline__ void read_and_count(HistShared &sh, F while_waiting) {
        char *h = (char *)sh.h;
        const uint32_t none = (uint32_t)((char *)&sh.dummy[threadIdx.x & 63] - h);
        float top = -INFINITY;
        bool any = false;
        const int n_spans = spans();
        for (int span = 0; span < n_spans; span++) {
            uint32_t raw[NP], bits[kWords];
            ask_mask(span, raw);
            if (span == 0) while_waiting();
            ask(span, raw, bits);
            if (span == 0) __syncthreads();  // the counts are cleared
#pragma unroll
            for (int p = 0; p < NP; p++) {
                select(p, bits);
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t w = d[p][j];
                    v[j] = __uint_as_float(w);
                    atomicAdd((uint32_t *)(h + (w < kLowest32 ? (w >> 14) & 0x1FFFCu : none)), (int)w < 0 ? 0x10000u : 1u);
                }
                top = fmaxf(fmaxf(top, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
                if (SUM) add(v);
                __builtin_amdgcn_sched_barrier(0);
            }
            uint32_t some = 0;
#pragma unroll
            for (int i = 0; i < kWords; i++) some |= bits[i];
            any = any || some != 0;
        }
#pragma unroll
        for (int s = 32; s; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
        if (__any(any) && (threadIdx.x & 63) == 0) sh.any = 1;
        if ((threadIdx.x & 63) == 0 && top > -INFINITY) atomicMax(&sh.top_key, key_of_bits(__float_as_uint(top)));
    }
    // Whether the row holds the type's lowest value.  Every thread calls it.
    __device__ __forceinline__ bool has_lowest(HistShared &sh) {
        bool has = false;
        each([&](float x, int) { has = has || __float_as_uint(x) == kLowest32; });
        __syncthreads();
        if (threadIdx.x == 0) sh.any = 0;
        __syncthreads();
        if (__any(has) && (threadIdx.x & 63) == 0) sh.any = 1;
        __syncthreads();
        return sh.any != 0;
    }
    // f(x, first id) for every four elements; what is no candidate is -inf.
    template <class F>
    __device__ __forceinline__ void each_four(F f) {
        const int n_spans = spans();
        for (int span = 0; span < n_spans; span++) {
            if (SPANS) load(span);
            int first = first_id(span, 0);
            asm volatile("" : "+v"(first));  // a caller's loop keeps nothing worked out from the ids
#pragma unroll
            for (int p = 0; p < NP; p++) {
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t w = d[p][j];
                    asm volatile("" : "+v"(w));  // (nor from the logits)
                    x[j] = __uint_as_float(w);
                }
                f(x, first + p * kFinePieceIds);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // f(x, id) for every element.
    template <class F>
    __device__ __forceinline__ void each(F f) {
        each_four([&](const float (&x)[4], int first) {
#pragma unroll
            for (int j = 0; j < 4; j++) f(x[j], first + j);
        });
    }
};

// The smallest and the largest value of a bin.  Position 32767 is both zeros'
// and holds what is nearer to them than a bin's width, on both sides; the
// infinite one's bounds are infinite; the last one's lowest value is not
// counted.
__device__ __forceinline__ float bin_low(uint32_t pos) {
    return pos == kLowest ? value_of_key(kLeastKey + 1) : pos == 32767u ? value_of_key(0x7FFF0000u) : pos < 128u ? INFINITY : value_of_key((65535u - pos) << 16);
}
__device__ __forceinline__ float bin_high(uint32_t pos) {
    return pos < 128u ? INFINITY : value_of_key((65535u - pos) << 16 | 0xFFFFu);
}
// The position of a key.
__device__ __forceinline__ uint32_t key_pos(uint32_t key) {
    const uint32_t pos = 65535u - (key >> 16);
    return pos == 32768u ? 32767u : pos;
}

struct FineShared {
    uint64_t list[kWindow];  // complement of the key, then the id: rising is the order
    double mass[kWindow];    // inclusive sums over the list
    double wave[kRowWaves];
    uint32_t lo, hi, above;  // the window chosen: positions, candidates before it
    uint32_t n, key, before, end;
    double value[2];
    int hit;
    bool fits;
};

// Sorts list[0, n) rising; n <= kWindow, every thread calls it.  Steps within
// 128 entries stay in one wave, whose LDS accesses keep their order.
__device__ __forceinline__ void sort_rising(uint64_t *list, uint32_t n) {
    uint32_t size_all = 2;
    while (size_all < n) size_all <<= 1;
    for (uint32_t i = n + threadIdx.x; i < size_all; i += kRowThreads) list[i] = ~0ull;
    __syncthreads();
    for (uint32_t size = 2; size <= size_all; size <<= 1) {
        for (uint32_t step = size >> 1; step; step >>= 1) {
            const uint32_t t = threadIdx.x;
            if (t < size_all / 2) {
                const uint32_t lo = 2 * t - (t & (step - 1)), hi = lo + step;
                const uint64_t a = list[lo], b = list[hi];
                if (((lo & size) == 0) == (a > b)) {
                    list[lo] = b;
                    list[hi] = a;
                }
            }
            if (step > 64 || (step == 1 && size >= 128)) __syncthreads();
            else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
    __syncthreads();
}

// The draw among the ranks that the filters keep.  One loop with one pass over
// the row in it: each stage asks for a rank, a mass, the end of the weights
// from some value on, or the whole mass, which the window answers if it holds
// the place, and a pass brings if not.
template <class ROW>
struct FineDraw {
    HistOrder<ROW> &order;
    FineShared &fs;

    __device__ __forceinline__ double block_sum(double v) {
        v = wave_scan(v);
        if ((threadIdx.x & 63) == 63) fs.wave[threadIdx.x >> 6] = v;
        __syncthreads();
        v = fs.wave[threadIdx.x & (kRowWaves - 1)];
        v += __shfl_xor(v, 1);
        v += __shfl_xor(v, 2);
        v += __shfl_xor(v, 4);
        v += __shfl_xor(v, 8);
        __syncthreads();
        return uniform(v);
    }

    // Sorts the list by the bins' own counts: each entry goes to its bin's
    // stretch, then to its place among the few there.  Windows of more bins
    // than fit, or with many candidates in one bin, take the general sort (55
    // steps for 1024 entries: 9 us).
    __device__ __forceinline__ void sort_window(uint32_t lo, uint32_t hi, uint32_t n) {
        constexpr uint32_t kBins = sizeof(fs.mass) / 4;  // two a thread
        if (hi - lo >= kBins || n > kRowThreads) {
            sort_rising(fs.list, n);
            return;
        }
        uint32_t *const end = (uint32_t *)fs.mass;
        const uint32_t t = threadIdx.x;
        __syncthreads();
        const uint64_t e = t < n ? fs.list[t] : 0;
        uint32_t c[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t pos = lo + 2 * t + i;
            c[i] = pos <= hi ? bin_count(pos) : 0u;
        }
        const uint32_t sum = (uint32_t)wave_scan((int)(c[0] + c[1]));
        constexpr uint32_t kCrowd = 0x80000000u;
        const uint32_t crowd = __any(c[0] > 192 || c[1] > 192) ? kCrowd : 0u;
        if ((t & 63) == 63) order.sh.w_cnt[t >> 6] = sum | crowd;
        __syncthreads();
        uint32_t before = (t & 63) < kRowWaves ? order.sh.w_cnt[t & 15] : 0u;
        if (__any((before & kCrowd) != 0)) {  // alike in every wave
            sort_rising(fs.list, n);
            return;
        }
        before = (uint32_t)lane_int(wave_scan((t & 63) < (t >> 6) ? (int)before : 0), 63);
        const uint32_t start = before + sum - c[0] - c[1];
        end[2 * t] = start;
        end[2 * t + 1] = start + c[0];
        __syncthreads();
        const uint32_t bin = t < n ? key_pos(~(uint32_t)(e >> 32)) - lo : 0u;
        if (t < n) fs.list[atomicAdd(&end[bin], 1u)] = e;
        __syncthreads();
        uint32_t at = 0;
        if (t < n) {
            at = bin ? end[bin - 1] : 0u;
#pragma unroll 4
            for (uint32_t i = at, last = end[bin]; i < last; i++) at += fs.list[i] < e;
        }
        __syncthreads();
        if (t < n) fs.list[at] = e;
        __syncthreads();
    }
    // Candidates of one position.
    __device__ __forceinline__ uint32_t bin_count(uint32_t pos) const {
        const uint32_t i = pos_bits(pos) & 0x7FFFu;
        uint32_t cp, cn;
        cleaned((int)i, order.sh.h[i], cp, cn);
        return pos < 32768u ? cp : cn;
    }

    // Chooses a window of whole bins that holds the ranks from `start` up to
    // `end` (a bin's end; `first` and `last` their bins): from the top if that
    // fits, else around them, with 128 ranks before them and `beyond` behind
    // if there is room and `sure` is not set.  Wave 0; the result goes to fs.
    __device__ __forceinline__ void choose(uint32_t start, uint32_t end, uint32_t first, uint32_t last, uint32_t beyond, bool sure) {
        uint32_t a = key_pos(order.sh.top_key), before = 0;
        if (end > kWindow) {
            a = first;
            before = start;
            if (!sure) {
                const HistPlace p = order.find_rank(start > 128 ? start - 128 : 0);
                if (end - p.above <= kWindow) {
                    a = p.pos;
                    before = p.above;
                }
            }
        }
        const bool fits = end - before <= kWindow;
        if (fits && beyond) {
            const HistPlace p = order.find_rank(end - 1 + beyond);
            if (p.pos > last && p.above + p.count - before <= kWindow) last = p.pos;
        }
        if (threadIdx.x == 0) {
            fs.lo = a;
            fs.hi = last;
            fs.above = before;
            fs.fits = fits;
            fs.n = 0;
        }
    }

    // The least key whose weight is at least `least` (weights rise with the
    // key): 64 points of the range at a time.  One wave.
    __device__ __forceinline__ uint32_t least_key(double least) const {
        uint32_t a = kLeastKey - 1, b = key_of_bits(__float_as_uint(order.weight.largest()));  // not at a, but at b
        while (b - a > 1) {
            const uint32_t step = (b - a + 63) / 64, at = min(a + ((threadIdx.x & 63) + 1) * step, b);
            const int l = __builtin_ctzll(__ballot(order.weight(value_of_key(at)) >= least));  // lane 63 is at b
            b = min(a + (uint32_t)(l + 1) * step, b);
            a += (uint32_t)l * step;
        }
        return b;
    }

    // The list's index of the pick and the kept mass; -1 for a row that a
    // window does not take.
    __device__ __forceinline__ int draw(bool greedy, int k, float p, float mp, float u, double &mass) {
        enum { kTopK, kMinP, kTotal, kTopP, kPick, kLast };  // stages
        const uint32_t t = threadIdx.x;
        if (order.searches()) {
            const uint32_t c = order.total_count();
            if (t == 0) fs.n = c;
        }
        __syncthreads();
        const uint32_t count = uniform(fs.n);
        __syncthreads();
        // the window: positions lo .. hi hold the n listed candidates, `above` and mass_above lie before
        uint32_t lo = 0, hi = 0, above = 0, n = 0;
        double mass_above = 0.0;
        // the ranks kept so far and their mass (< 0: not known yet), and what top-p is a share of
        uint32_t kept = count;
        double base = -1.0, scale = 1.0, guess = -1.0;
        mass = -1.0;
        uint32_t from = 0, to = 65535u, key = 0, c_before = 0, c_end = 0;
        bool masses = false, valued = false;  // the bins have theirs; the window's bounds too
        double total = -1.0;                  // the whole row's mass; from then on the cells hold theirs
        const uint32_t top = key_pos(uniform(order.sh.top_key));
        double *const cells = order.sh.cells;
        int tries = 0, stage = greedy ? kTotal : k > 0 && (uint32_t)k < count ? kTopK : kMinP;
        if (!greedy && p <= 0.f) {
            kept = 1;
            mass = 1.0;
            stage = kLast;
        }
        for (;;) {
            if (stage == kMinP && key == 0) {
                if (!(mp > 0.f)) {
                    stage = kTotal;
                } else {
                    if (t < 64) {
                        const uint32_t v = least_key(fmin((double)mp, 1.0)), pos = key_pos(v);
                        const uint32_t e = order.count_to(pos), b = pos ? order.count_to(pos - 1) : 0u;
                        if (t == 0) {
                            fs.key = v;
                            fs.before = b;
                            fs.end = e;
                        }
                    }
                    __syncthreads();
                    key = uniform(fs.key);
                    c_before = uniform(fs.before);
                    c_end = uniform(fs.end);
                    if (c_before >= kept) stage = kTotal;  // it keeps them all
                }
            }
            if (stage == kTotal && (greedy ? false : base >= 0.0 || (mass >= 0.0 && !(p < 1.f)))) stage = kTopP;
            if (stage == kTotal && n && n == count) total = uniform(fs.mass[n - 1]);  // (every answer is in the window)
            if (stage == kTotal && total >= 0.0) {
                base = total;
                if (mass < 0.0) mass = total;
                stage = kTopP;
            }
            if (stage == kTopP && (!(p < 1.f) || mass < (double)p * base)) stage = kPick;
            if (stage == kLast && kept == 0) return -1;
            const bool by_mass = stage == kTopP || stage == kPick;
            const uint32_t rank = stage == kTopK ? (uint32_t)k - 1 : kept - 1;
            const double target = stage == kTopP ? (double)p * base : u > 0.f ? fmin((double)u, 1.0 - 0x1p-53) * mass : 0.0;
            auto reached = [&](double m) { return stage == kTopP ? m >= target : m > target; };
            bool have = false;
            int i = 0;
            // from the window
            if (stage == kTopK || stage == kLast) {
                have = n && above <= rank && rank < above + n;
                i = (int)(rank - above);
            } else if (stage == kMinP) {
                if (n && (above == 0 || above < c_before) && c_end <= above + n) {
                    __syncthreads();
                    if (t == 0) fs.hit = 0;
                    __syncthreads();
                    if (t < n && ~(uint32_t)(fs.list[t] >> 32) >= key && (t + 1 == n || ~(uint32_t)(fs.list[t + 1] >> 32) < key))
                        fs.hit = (int)t;
                    __syncthreads();
                    have = true;
                    i = uniform(fs.hit);
                }
            } else if (by_mass && n) {
                const double end = mass_above + uniform(fs.mass[n - 1]);
                if (lo > 0 && reached(mass_above)) {
                    to = min(to, lo - 1);
                    guess = valued ? uniform(fs.value[0]) * (target / mass_above) : target / scale;
                } else if (!reached(end) && above + n < count) {
                    from = max(from, hi + 1);
                    guess = valued ? uniform(fs.value[1]) + (target - end) / scale : target / scale;
                } else {
                    // the first that reaches it, else the last with weight
                    __syncthreads();
                    if (t == 0) fs.hit = 0;
                    __syncthreads();
                    if (t < n) {
                        const double m1 = fs.mass[t], m0 = t ? fs.mass[t - 1] : 0.0;
                        if (reached(end) ? reached(mass_above + m1) && (t == 0 || !reached(mass_above + m0))
                                         : m1 > m0 && !(fs.mass[n - 1] > m1))
                            fs.hit = (int)t;
                    }
                    __syncthreads();
                    have = true;
                    i = uniform(fs.hit);
                }
            }
            // from the row
            if (!have) {
                if (++tries > 24) return -1;  // (the bounds of the search keep it far from this)
                // what is listed, x_lo .. x_hi; what is summed, above x_sum; the whole mass: nothing is listed
                float x_hi = -INFINITY, x_lo = INFINITY, x_sum = -INFINITY;
                // The mass of few candidates (a constrained row's): a window of them all, no exponentials
                // beforehand.  64 rows of 128256 with 450 each 70 -> 56 us, 256 of 32000 with 480 40 -> 31, one of
                // 400 ids 22 either way; 800 of 4000 23 -> 25.5 (their sort), hence half a window.
                const bool list_all = stage == kTotal && !greedy && count <= kWindow / 2 && n == 0;
                bool sum_all = stage == kTotal && !list_all;
                const bool in_cells = by_mass && total >= 0.0 && reached(uniform(cells[kRowThreads - 1]));
                if (by_mass && !in_cells && !masses) {
                    order.add_masses();
                    masses = true;
                    if (total >= 0.0) {
                        if (order.searches()) {
                            const double m = order.total_mass();
                            if (t == 0) fs.value[0] = m;
                        }
                        __syncthreads();
                        scale = total / uniform(fs.value[0]);
                        __syncthreads();
                    }
                }
                if (!sum_all) {
                    if (!(guess >= 0.0)) guess = target / scale;
                    __syncthreads();
                    if (in_cells) {
                        if (reached(cells[t]) && !(t && reached(cells[t - 1]))) fs.hit = (int)t;
                        __syncthreads();
                    }
                    if (t < 64) {
                        if (list_all) {
                            const HistPlace q = order.find_rank(count - 1);
                            choose(0, count, top, q.pos, 0, true);
                        } else if (stage == kMinP) {
                            const HistPlace q = order.find_rank(c_end > c_before ? c_end - 1 : c_before - 1);
                            const HistPlace q0 = q.above < c_before ? q : order.find_rank(c_before ? c_before - 1 : 0);
                            choose(q0.above, q.above + q.count, q0.pos, q.pos, 0, true);
                        } else {
                            HistPlace q;
                            if (in_cells) {
                                const uint32_t pos = min(max(top + (uint32_t)fs.hit, from), to);
                                q.pos = pos;
                                q.above = pos ? order.count_to(pos - 1) : 0u;
                                q.count = uniform(bin_count(pos));
                                if (!q.count) q = order.find_rank(q.above);  // (a bound of the search, not a cell)
                            } else if (by_mass) {
                                q = stage == kTopP ? order.template find<2>(0, guess) : order.template find<1>(0, guess);
                                if (q.pos < from) q = order.find_rank(order.count_to(from - 1));
                                else if (q.pos > to) q = order.find_rank(order.count_to(to) - 1);
                            } else {
                                q = order.find_rank(rank);
                            }
                            choose(q.above, q.above + q.count, q.pos, q.pos, by_mass && !in_cells ? 64 + (q.above + q.count) / 8 : 0,
                                   !by_mass || in_cells);
                        }
                    }
                    __syncthreads();
                    if (!uniform(fs.fits)) return -1;
                    lo = uniform(fs.lo);
                    hi = uniform(fs.hi);
                    above = uniform(fs.above);
                    x_hi = bin_high(lo);
                    x_lo = bin_low(hi);
                    sum_all = above && total < 0.0;
                    if (!sum_all) x_sum = x_hi;
                }
                const bool to_cells = sum_all && !greedy, sums = sum_all || (above && lo - top > kRowThreads);
                if (to_cells) {
                    cells[t] = 0.0;
                    __syncthreads();
                }
                double s = 0.0;
                order.row.each_four([&](const float (&x)[4], int first) {
                    if (sums) {
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            if (!(x[j] > x_sum)) continue;
                            const double w = order.weight(x[j]);
                            s += w;
                            if (to_cells) {
                                // in units of 2^-41, so that the order of the sums is all one
                                const uint32_t cell = key_pos(key_of_bits(__float_as_uint(x[j]))) - top;
                                if (cell < kRowThreads)
                                    atomicAdd((unsigned long long *)&cells[cell],
                                              (unsigned long long)(__double_as_longlong(w + 2048.0) - __double_as_longlong(2048.0)));
                            }
                        }
                    }
                    if (!sum_all) {
                        // one addition to the list's length a wave: its answer takes 100 instructions' time
                        uint64_t in[4];
                        uint32_t found = 0;
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            in[j] = __ballot(x[j] >= x_lo && x[j] <= x_hi);
                            found += (uint32_t)__popcll(in[j]);
                        }
                        if (found) {
                            uint32_t at = 0;
                            if ((t & 63) == 0) at = atomicAdd(&fs.n, found);
                            at = uniform(at);
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                const uint32_t slot = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(in[j] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in[j], 0u));
                                if (x[j] >= x_lo && x[j] <= x_hi && slot < kWindow)
                                    fs.list[slot] = (uint64_t)~key_of_bits(__float_as_uint(x[j])) << 32 | (uint32_t)(first + j);
                                at += (uint32_t)__popcll(in[j]);
                            }
                        }
                    }
                });
                s = block_sum(s);
                if (to_cells) {
                    total = s;
                    const double m = wave_scan((double)(uint64_t)__double_as_longlong(cells[t]) * 0x1p-41);
                    if ((t & 63) == 63) fs.wave[t >> 6] = m;
                    __syncthreads();
                    double before = 0.0;
#pragma unroll 1
                    for (uint32_t v = 0; v < t >> 6; v++) before += fs.wave[v];
                    cells[t] = before + m;
                    n = 0;  // (a window may have been chosen, but was not listed)
                    __syncthreads();
                    continue;
                }
                if (greedy && stage == kTotal) {
                    mass = s;
                    kept = 1;
                    stage = kLast;
                    continue;
                }
                mass_above = above && lo - top <= kRowThreads ? uniform(cells[lo - top - 1]) : s;
                n = min(uniform(fs.n), kWindow);
                sort_window(lo, hi, n);
                const double w = t < n ? order.weight(value_of_key(~(uint32_t)(fs.list[t] >> 32))) : 0.0;
                const double m = wave_scan(w);
                if ((t & 63) == 63) fs.wave[t >> 6] = m;
                __syncthreads();
                double before = 0.0;
#pragma unroll 1
                for (uint32_t v = 0; v < t >> 6; v++) before += fs.wave[v];
                fs.mass[t] = before + m;
                valued = by_mass && !in_cells;
                if (valued && t < 64) {  // the bounds' mass by the bins, for another try
                    const double m0 = lo ? order.mass_to(lo - 1) : 0.0, m1 = order.mass_to(hi);
                    if (t == 0) {
                        fs.value[0] = m0;
                        fs.value[1] = m1;
                    }
                }
                __syncthreads();
                continue;
            }
            // the stage's answer, and the next stage
            const uint32_t end = above + (uint32_t)i + 1;
            const double m_end = mass_above + uniform(fs.mass[i]);
            if (stage == kTopK) {
                kept = (uint32_t)k;
                base = mass = m_end;
                stage = kMinP;
            } else if (stage == kMinP || stage == kTopP) {
                if (end < kept) {
                    kept = end;
                    mass = m_end;
                }
                stage = stage == kMinP ? kTotal : kPick;
            } else if (stage == kPick && end > kept) {
                stage = kLast;
            } else {
                return i;
            }
            tries = 0;
            from = 0;
            to = 65535u;
            guess = -1.0;
        }
    }
};

// Launches KERNEL<8, SPANS>: rows of up to 8 pieces (3: the largest skew) stay
// in registers (64 rows of 32000 without filters 36.6 us, in spans 41.6),
// longer ones keep nothing between passes and are read in spans of 8.  16
// pieces, 64 of a thread's 128 registers, left the searches too few: top 50 of
// 600 rows of 60000 took 126 us so, 99 in spans, top 20 of 256 rows of 50021
// 33 and 28 us; spans of 16 took up to three times as long as spans of 8.
#define CG_LAUNCH_FINE(KERNEL, V, BATCH, STREAM, ARGS)                                              \
    do {                                                                                            \
        const dim3 grid_(BATCH), block_(kRowThreads);                                               \
        if ((V) + 3 <= 8 * kFinePieceIds)                                                           \
            hipLaunchKernelGGL((KERNEL<8, false>), grid_, block_, 0, STREAM, ARGS);                 \
        else hipLaunchKernelGGL((KERNEL<8, true>), grid_, block_, 0, STREAM, ARGS);                 \
    } while (0)

}  // namespace cg
