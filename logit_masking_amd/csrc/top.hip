// top.hip -- gfx950 kernel of a masked row's k largest logits and its
// log-normaliser: what a teacher records at every position, and the top
// log-probabilities of a reply.
//
//   k_top_counts   bfloat16 rows, one workgroup each (row_hist.hpp)
//   k_top_fine     float32 rows, one workgroup each (row_fine.hpp)
#include <algorithm>

#include "cg_internal.hpp"
#include "row_fine.hpp"

namespace cg {

namespace {

struct TopArgs {
    const void *logits;
    int64_t stride;
    const uint64_t *mask;
    int wpr, V, k;
    int32_t *ids;
    float *top, *lse;
};

// Sorts list[0, n) falling; n a power of two, every thread calls it.
__device__ void sort_falling(uint64_t *list, int n) {
    for (int size = 2; size <= n; size <<= 1) {
        for (int step = size >> 1; step; step >>= 1) {
            __syncthreads();
            for (int t = threadIdx.x; t < n / 2; t += kRowThreads) {
                const int lo = 2 * t - (t & (step - 1)), hi = lo + step;
                const uint64_t a = list[lo], b = list[hi];
                const bool falling = (lo & size) == 0;
                if (falling ? a < b : a > b) {
                    list[lo] = b;
                    list[hi] = a;
                }
            }
        }
    }
    __syncthreads();
}

// The whole row digit by digit (row_select.hpp), for rows that the counts do
// not take (row_hist.hpp), and float32 rows with more candidates in the k-th
// one's bin than the list takes.
struct DigitsShared {
    SelectShared select;
    uint64_t list[CG_MAX_TOP];  // key in the high half, the id's complement in the low: one order
    uint32_t n_list;
};
template <int DT>
__device__ void top_by_digits(const TopArgs &a, int r, DigitsShared &ds) {
    SelectShared &sh = ds.select;
    uint64_t *list = ds.list;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    RowView<DT> row{(const char *)a.logits + (size_t)r * (size_t)a.stride * (DT == 0 ? 4 : 2),
                    a.mask ? a.mask + (size_t)r * a.wpr : nullptr, a.V};
    int n_pow = 1;
    while (n_pow < a.k) n_pow <<= 1;
    for (int i = threadIdx.x; i < n_pow; i += kRowThreads) list[i] = 0;
    if (threadIdx.x == 0) ds.n_list = 0;
    const uint32_t best = row_max_key(row, sh);
    uint64_t mass = 0;
    if (best) {
        const Weight weight(value_of_key(best), 1.0);
        mass = row_mass(row, weight, 0u, sh);
        const Place q = row_find<DT, false>(row, weight, (uint32_t)a.k - 1, 0, sh);
        const uint32_t ties = min(q.count, (uint32_t)a.k - q.above);
        // larger keys in any order, the ties by rising id until enough
        uint32_t before = 0;
        for (int base = 0; base < row.V; base += kRowThreads) {
            const int i = base + threadIdx.x;
            const uint32_t key = i < row.V ? row.key(i) : 0u;
            if (key > q.key) list[atomicAdd(&ds.n_list, 1u)] = ((uint64_t)key << 32) | (uint32_t)~i;
            const uint64_t hits = __ballot(key == q.key);
            if (lane == 0) sh.wave[wave] = __popcll(hits);
            __syncthreads();
            uint32_t mine = before;
#pragma unroll 1
            for (int w = 0; w < kRowWaves; w++) {
                if (w < wave) mine += sh.wave[w];
                before += uniform(sh.wave[w]);
            }
            mine += __popcll(hits & ((1ull << lane) - 1));
            if (key == q.key && mine < ties) list[q.above + mine] = ((uint64_t)key << 32) | (uint32_t)~i;
            __syncthreads();
        }
        sort_falling(list, n_pow);
        if (threadIdx.x == 0) a.lse[r] = (float)(weight.m + log_of((double)mass / kMassUnit));
    } else if (threadIdx.x == 0) {
        a.lse[r] = -INFINITY;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.k; i += kRowThreads) {
        const uint64_t e = list[i];
        a.ids[(size_t)r * a.k + i] = e ? (int32_t)~(uint32_t)e : -1;
        a.top[(size_t)r * a.k + i] = e ? value_of_key((uint32_t)(e >> 32)) : -INFINITY;
    }
}

// Room of the candidates' list: k and the ties of the k-th.
constexpr uint32_t kListRoom = 2048;
static_assert(CG_MAX_TOP < kListRoom && kListRoom * 8 <= sizeof(uint32_t) * kHistDwords, "the list lies over the counts");

// Writes the first k of the n listed candidates in rising order of their
// entries (position, id).
template <class VALUE>
__device__ void write_top(uint64_t *list, uint32_t n, const TopArgs &a, int r, VALUE value) {
    int32_t *ids = a.ids + (size_t)r * a.k;
    float *top = a.top + (size_t)r * a.k;
    auto put = [&](uint32_t rank, uint64_t e) {
        if (rank < (uint32_t)a.k) {
            ids[rank] = (int32_t)(uint32_t)e;
            top[rank] = value((uint32_t)(e >> 32));
        }
    };
    if (n <= 512) {
        // each entry's rank is the number of smaller ones: no barrier, every
        // read a broadcast (sorting 512 takes 45 barriers)
        if (threadIdx.x < n) {
            const uint64_t e = list[threadIdx.x];
            uint32_t rank = 0;
#pragma unroll 8
            for (uint32_t i = 0; i < n; i++) rank += list[i] < e;
            put(rank, e);
        }
    } else {
        int n_pow = 1024;
        while ((uint32_t)n_pow < n) n_pow <<= 1;
        for (uint32_t i = threadIdx.x; i < n; i += kRowThreads) list[i] = ~list[i];
        for (uint32_t i = n + threadIdx.x; i < (uint32_t)n_pow; i += kRowThreads) list[i] = 0;
        sort_falling(list, n_pow);
        for (uint32_t i = threadIdx.x; i < min(n, (uint32_t)a.k); i += kRowThreads) put(i, ~list[i]);
    }
    for (uint32_t i = n + threadIdx.x; i < (uint32_t)a.k; i += kRowThreads) {
        ids[i] = -1;
        top[i] = -INFINITY;
    }
}

// bfloat16 rows: one read, the k-th value from the counts (row_hist.hpp),
// then the candidates down to it from the registers.  The normaliser is the
// counts' too: an exponential a value, not a logit.
//
// 1024 rows of 151936, four after the other on a CU: 130 us, 33 a row: 14 for
// the loads and counts (279 MB in all: 5 TB/s meanwhile), then 4 for
// the blocks' totals, 1 for the k-th's place, 4 to list and 1 to order the 64,
// and the waves' differences; the memory is idle in the second half (see
// k_filter_counts).  4 rows of 128256, where only a row's time counts: 20 us.
template <int NP, bool SPANS, bool ONCE>
__global__ __launch_bounds__(kRowThreads) void k_top_counts(TopArgs a) {
    __shared__ HistShared sh;
    const int r = blockIdx.x;
    HistRow<NP, SPANS, ONCE> row;
    row.init((const uint16_t *)a.logits + (size_t)r * (size_t)a.stride, a.mask ? a.mask + (size_t)r * a.wpr : nullptr,
             a.wpr, a.V);
    typedef HistOrder<HistRow<NP, SPANS, ONCE>> Order;
    Order order(sh, row);
    uint64_t *list = (uint64_t *)sh.h;
    uint32_t n = 0;
    const auto found = order.template build<true>(1.0);
    if (found == Order::kCounted) {
        if (order.searches()) {
            const HistPlace q = order.find_rank((uint32_t)a.k - 1);
            const double mass = order.total_mass();
            if (threadIdx.x == 0) {
                sh.place = q;
                sh.n_list = 0;
                a.lse[r] = (float)(order.weight.m + log_of(mass));
            }
        }
        __syncthreads();
        HistPlace q;
        q.pos = uniform(sh.place.pos);
        q.above = uniform(sh.place.above);
        q.count = uniform(sh.place.count);
        if (q.above + q.count < (uint32_t)a.k && row.has_lowest(sh)) {
            top_by_digits<1>(a, r, *(DigitsShared *)sh.h);
            return;
        }
        // every tie of the last value when they fit, else only the larger
        // candidates here and as many ties as are wanted by their ids
        const bool all = q.above + q.count <= kListRoom;
        const int n_spans = row.spans();
        for (int s = 0; s < n_spans; s++) {
            const int span = (row.span_at + (s ? 1 : 0)) % n_spans;  // the one in the registers first
            if (s) row.load(span, sh.lut);
            if (all || q.pos) row.collect(all ? q.pos : q.pos - 1, list, kListRoom, sh);
        }
        if (all) {
            n = q.above + q.count;
        } else {
            n = min(q.above + q.count, (uint32_t)a.k);
            row.first_of(q.pos, n - q.above, list + q.above, sh);
        }
    } else if (found == Order::kByDigits) {
        __syncthreads();
        top_by_digits<1>(a, r, *(DigitsShared *)sh.h);
        return;
    } else if (threadIdx.x == 0) {
        a.lse[r] = -INFINITY;
    }
    __syncthreads();
    write_top(list, n, a, r, [](uint32_t pos) { return bits_value(pos_bits(pos)); });
}

// float32 rows: the k-th one's bin from the counts (row_fine.hpp), then the
// candidates down to its end.  The normaliser is summed while the row is
// counted, in float32 a thread (32 to 128 terms of one exponential each, under
// a running maximum) and in 64 bits over the threads.  48 rows of 50021: 21 us,
// a row's latency: the loads, the counts and the sums 10.
template <int NP, bool SPANS>
__global__ __launch_bounds__(kRowThreads) void k_top_fine(TopArgs a) {
    __shared__ HistShared sh;
    __shared__ double sums[kRowWaves];
    const int r = blockIdx.x;
    FineRow<NP, SPANS, true> row;
    row.init((const float *)a.logits + (size_t)r * (size_t)a.stride, a.mask ? a.mask + (size_t)r * a.wpr : nullptr, a.V);
    typedef HistOrder<FineRow<NP, SPANS, true>> Order;
    Order order(sh, row);
    uint64_t *list = (uint64_t *)sh.h;
    uint32_t n = 0;
    const auto found = order.template build<false>(1.0);
    if (found == Order::kCounted) {
        const double part = row.run_sum ? (double)row.run_sum * exp_falling((double)row.run_max - order.weight.m) : 0.0;
        const double whole = wave_scan(part);
        if ((threadIdx.x & 63) == 63) sums[threadIdx.x >> 6] = whole;
        if (order.searches()) {
            const HistPlace q = order.find_rank((uint32_t)a.k - 1);
            if (threadIdx.x == 0) {
                sh.place = q;
                sh.n_list = 0;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            double s = 0.0;
            for (int w = 0; w < kRowWaves; w++) s += sums[w];
            a.lse[r] = order.weight.largest() < INFINITY ? (float)(order.weight.m + log_of(s)) : INFINITY;
        }
        HistPlace q;
        q.pos = uniform(sh.place.pos);
        q.above = uniform(sh.place.above);
        q.count = uniform(sh.place.count);
        n = q.above + q.count;
        if (n > kListRoom || (n < (uint32_t)a.k && row.has_lowest(sh))) {
            __syncthreads();
            top_by_digits<0>(a, r, *(DigitsShared *)sh.h);
            return;
        }
        const float x_lo = bin_low(q.pos);
        row.each([&](float x, int id) {
            if (x >= x_lo)
                list[atomicAdd(&sh.n_list, 1u)] = (uint64_t)~key_of_bits(__float_as_uint(x)) << 32 | (uint32_t)id;
        });
    } else if (found == Order::kByDigits) {
        __syncthreads();
        top_by_digits<0>(a, r, *(DigitsShared *)sh.h);
        return;
    } else if (threadIdx.x == 0) {
        a.lse[r] = -INFINITY;
    }
    __syncthreads();
    write_top(list, n, a, r, [](uint32_t key) { return value_of_key(~key); });
}

}  // namespace

}  // namespace cg

using namespace cg;

static int top_arg_error(const char *msg) {
    set_error("top_logits: %s", msg);
    return CG_E_ARG;
}

extern "C" {

size_t cg_top_workspace_bytes(int32_t batch, int32_t vocab, int32_t k) {
    (void)batch;
    (void)vocab;
    (void)k;
    return 0;
}

int cg_top_logits(const void *d_logits, int32_t dtype, int32_t batch, int32_t vocab, int64_t row_stride,
                  const uint64_t *d_mask, int32_t words_per_row, int32_t k, void *d_workspace, int32_t *d_out_ids,
                  float *d_out_logits, float *d_out_lse, void *stream) {
    if (dtype != 0 && dtype != 1) return top_arg_error("dtype must be 0 (float32) or 1 (bfloat16)");
    if (batch < 0 || vocab < 1 || vocab > CG_MAX_ROW_VOCAB) return top_arg_error("bad batch / vocab");
    if (k < 1 || k > CG_MAX_TOP) return top_arg_error("k out of range");
    if (row_stride < vocab) return top_arg_error("row_stride < vocab");
    if (d_mask && words_per_row < (vocab + 63) / 64) return top_arg_error("words_per_row < ceil(vocab / 64)");
    if (batch == 0) return CG_OK;
    if (!d_logits || !d_out_ids || !d_out_logits || !d_out_lse) return top_arg_error("NULL device pointer");
    (void)d_workspace;
    const TopArgs a{d_logits, row_stride, d_mask, words_per_row, vocab, k, d_out_ids, d_out_logits, d_out_lse};
    if (dtype == 0) {
        CG_LAUNCH_FINE(k_top_fine, vocab, batch, (hipStream_t)stream, a);
    } else {
        CG_LAUNCH_ROWS(k_top_counts, vocab, batch, (hipStream_t)stream, a);
    }
    return launch_status("top_logits");
}

}  // extern "C"
