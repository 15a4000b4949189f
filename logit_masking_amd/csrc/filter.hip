// filter.hip -- gfx950 kernel of the filtered draw: temperature, top-k,
// top-p and min-p over a masked row, then the inverse of the cumulative
// weight at a given uniform number ("Constrained decoding", "The guarantee":
// sampling runs after masking, so no sampling strategy can escape it).
//
//   k_filter_counts   bfloat16 rows, one workgroup each (row_hist.hpp)
//   k_filter_fine     float32 rows, one workgroup each (row_fine.hpp)
//
// All filters keep a prefix of the row's order, so each needs one place in it:
// the rank k, the first rank up to which the weights reach top_p of their sum,
// the last weight that reaches min_p; and the draw the first rank up to which
// they pass u of the kept sum.  Nothing is sorted but a window of float32
// candidates, and the kept set is never written: a row is read once and its id
// and log-probability go out.
#include <algorithm>

#include "cg_internal.hpp"
#include "row_fine.hpp"

namespace cg {

namespace {

struct FilterArgs {
    const void *logits;
    int64_t stride;
    const uint64_t *mask;
    int wpr, V;
    const float *temp;
    const int32_t *top_k;
    const float *top_p, *min_p, *uniform;
    int32_t *ids;
    float *logprob;
};

// Under a temperature above this the lowest value of a type weighs something
// beside others: such rows are searched by digits (row_hist.hpp).
constexpr float kEvenT = 1e30f;

// Every filter keeps a prefix of the row's order (row_select.hpp), so the
// kept set is a place: all candidates of larger keys than `key`, and the
// first `ties` of those equal to it.
struct Cut {
    uint32_t key, ties;
};
// The whole draw digit by digit (row_select.hpp), for rows that the counts and
// windows do not take: one value over and over, a bin of float32 logits with
// more candidates than a window, nothing but a type's lowest value.
template <int DT>
__device__ void filter_by_digits(const FilterArgs &a, int r, SelectShared &sh) {
    RowView<DT> row{(const char *)a.logits + (size_t)r * (size_t)a.stride * (DT == 0 ? 4 : 2),
                    a.mask ? a.mask + (size_t)r * a.wpr : nullptr, a.V};
    const float T = uniform(a.temp[r]);
    const bool greedy = !(T > 0.f);
    const uint32_t best = row_max_key(row, sh);
    if (best == 0) {
        if (threadIdx.x == 0) {
            a.ids[r] = -1;
            a.logprob[r] = 0.f;
        }
        return;
    }
    const Weight weight(value_of_key(best), greedy ? 1.0 : 1.0 / (double)T);
    const int k = a.top_k ? uniform(a.top_k[r]) : 0;
    const float p = a.top_p ? uniform(a.top_p[r]) : 1.f;
    const float mp = a.min_p ? uniform(a.min_p[r]) : 0.f;

    Cut cut{0, 0};  // below every candidate: all kept
    uint64_t mass;
    uint32_t pick_key = best, pick_n = 0;
    if (greedy) {
        mass = row_mass(row, weight, 0u, sh);
    } else {
        if (k > 0 && k < a.V) {
            const Place q = row_find<DT, false>(row, weight, (uint32_t)k - 1, 0, sh);
            const uint32_t ties = min(q.count, (uint32_t)k - q.above);
            cut = Cut{q.key, ties};
            mass = q.mass_above + ties * fixed_mass(weight(value_of_key(q.key)));
        } else {
            mass = row_mass(row, weight, 0u, sh);
        }
        if (p < 1.f) {
            // rank j stays while the mass before it is under p * mass: the
            // last one kept is the first whose own end reaches it
            const uint64_t goal = p > 0.f ? (uint64_t)ceil((double)p * (double)mass) : 0;
            if (goal == 0) {
                cut = Cut{best, 1};
                mass = fixed_mass(1.0);
            } else {
                const Place q = row_find<DT, true>(row, weight, 0, goal - 1, sh);
                const uint64_t f = fixed_mass(weight(value_of_key(q.key)));
                uint32_t ties = q.count;
                if (f) ties = (uint32_t)min((uint64_t)ties, (goal - q.mass_above + f - 1) / f);
                const Cut c{q.key, max(ties, 1u)};
                if (c.key > cut.key || (c.key == cut.key && c.ties < cut.ties)) {
                    cut = c;
                    mass = q.mass_above + c.ties * f;
                }
            }
        }
        if (mp > 0.f) {
            // the least key whose weight reaches min_p (weights rise with the key)
            uint32_t lo = key_of_bits(0xFF7FFFFFu), hi = best;
            const double least = fmin((double)mp, 1.0);
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2;
                if (weight(value_of_key(mid)) >= least) hi = mid;
                else lo = mid + 1;
            }
            if (lo > cut.key) {
                cut = Cut{lo, 0xFFFFFFFFu};
                mass = row_mass(row, weight, lo, sh);
            }
        }
        const double u = (double)a.uniform[r];
        const uint64_t at = u > 0.0 ? (uint64_t)fmin(u * (double)mass, (double)(mass - 1)) : 0;
        const Place q = row_find<DT, true>(row, weight, 0, at, sh);
        const uint64_t f = fixed_mass(weight(value_of_key(q.key)));
        uint32_t n = q.count;
        if (q.key == cut.key) n = min(n, cut.ties);
        pick_key = q.key;
        pick_n = f && at > q.mass_above ? (uint32_t)min((uint64_t)(n - 1), (at - q.mass_above) / f) : 0;
    }
    const int id = row_nth(row, pick_key, pick_n, sh);
    if (threadIdx.x == 0) {
        const double y = weight.exponent(value_of_key(pick_key));
        a.ids[r] = id;
        a.logprob[r] = (float)(y - log_of((double)mass / kMassUnit));
    }
}

// The place of the draw at u among what the filters keep, the pick being the
// n-th candidate there, and the kept mass.
template <class ROW>
__device__ __forceinline__ HistPlace draw(HistOrder<ROW> &order, int k, float p, float mp, float u, double &mass,
                                          uint32_t &n) {
    const int lane = threadIdx.x & 63;
    const uint32_t top = order.top_pos();
    uint32_t cut = 0xFFFFFFFFu, ties = 0;  // the last kept position, and how many of it stay
    if (k > 0 && (uint32_t)k < order.total_count()) {
        const HistPlace q = order.template find<0>((uint32_t)k - 1, 0.0);
        cut = q.pos;
        ties = (uint32_t)k - q.above;
        mass = q.mass_above + ties * q.w;
    }
    if (p <= 0.f) {
        cut = top;
        ties = 1;
        mass = 1.0;
    } else if (p < 1.f) {
        // rank j stays while the mass before it is under p * mass: the last
        // one kept is the first whose own end reaches it
        const double goal = (double)p * mass;
        const HistPlace q = order.template find<2>(0, goal);
        const uint32_t keep = min(q.count, (uint32_t)fmin(fmax(ceil((goal - q.mass_above) / q.w), 1.0), 4294967040.0));
        if (q.pos < cut || (q.pos == cut && keep < ties)) {
            cut = q.pos;
            ties = keep;
            mass = q.mass_above + ties * q.w;
        }
    }
    if (mp > 0.f) {
        // the last position whose weight reaches min_p (weights fall with the
        // position): 64 points of the range at a time
        const double least = fmin((double)mp, 1.0);
        uint32_t lo = top, hi = 32768u + (uint32_t)kInfIdx;  // holds at lo, not at hi (-inf)
        while (hi - lo > 1) {
            const uint32_t step = (hi - lo + 63) / 64, at = min(lo + (uint32_t)lane * step, hi);
            const uint64_t ok = __ballot(at < hi && order.weight(bits_value(pos_bits(at))) >= least);
            const int l = 63 - __builtin_clzll(ok);  // lane 0 holds
            lo = lo + (uint32_t)l * step;
            hi = min(lo + step, hi);
        }
        if (lo < cut) {
            cut = lo;
            ties = 0xFFFFFFFFu;
            mass = order.mass_to(lo);
        }
    }
    const double at = u > 0.f ? fmin((double)u, 1.0 - 0x1p-53) * mass : 0.0;
    HistPlace q = order.template find<1>(0, at);
    uint32_t left = q.count;
    if (q.pos >= cut) {
        if (q.pos > cut) q = order.template find<1>(0, mass * (1.0 - 0x1p-50));
        left = min(q.count, ties);
    }
    const double j = floor((at - q.mass_above) / q.w);
    n = j > 0.0 ? min((uint32_t)fmin(j, 4294967040.0), left - 1) : 0u;
    return q;
}

// bfloat16 rows: one read, the filters on the counts of the row's values
// (row_hist.hpp).
//
// 256 rows of 128256 under a grammar's mask, one per CU: 33 us, of which the
// loads and counts take 14 (62 MB: 4.4 TB/s meanwhile; an addition in LDS a
// logit), finding the blocks in use 2, their masses 2, the searches by one
// wave 3, the id 5, launch and end 4.  512 rows of 256000 in two spans:
// 104 us, 24 of each row's 48 for the loads and counts, at 5.5 TB/s.  A workgroup holds 143 of
// a CU's 160 KB of LDS, so that a row's searches have no other row's loads
// beside them; counts that leave room for two would hold a row's 65536 values
// in fewer than 16 bits each.
template <int NP, bool SPANS, bool ONCE>
__global__ __launch_bounds__(kRowThreads) void k_filter_counts(FilterArgs a) {
    __shared__ HistShared sh;
    const int r = blockIdx.x;
    HistRow<NP, SPANS, ONCE> row;
    row.init((const uint16_t *)a.logits + (size_t)r * (size_t)a.stride, a.mask ? a.mask + (size_t)r * a.wpr : nullptr,
             a.wpr, a.V);
    const float T = uniform(a.temp[r]);
    const int k = a.top_k ? uniform(a.top_k[r]) : 0;
    const float p = a.top_p ? uniform(a.top_p[r]) : 1.f;
    const float mp = a.min_p ? uniform(a.min_p[r]) : 0.f;
    const float u = uniform(a.uniform[r]);
    const bool greedy = !(T > 0.f);
    typedef HistOrder<HistRow<NP, SPANS, ONCE>> Order;
    Order order(sh, row);
    const auto found = T > kEvenT ? Order::kByDigits : order.template build<true>(greedy ? 1.0 : 1.0 / (double)T);
    if (found == Order::kByDigits) {
        __syncthreads();
        filter_by_digits<1>(a, r, *(SelectShared *)sh.h);
        return;
    }
    if (found == Order::kNone) {
        if (threadIdx.x == 0) {
            a.ids[r] = -1;
            a.logprob[r] = 0.f;
        }
        return;
    }
    if (order.searches()) {
        double mass = order.total_mass();
        uint32_t n = 0;
        const HistPlace q = greedy ? order.template find<0>(0, 0.0) : draw(order, k, p, mp, u, mass, n);
        if (threadIdx.x == 0) {
            sh.place = q;
            sh.n = n;
            sh.mass = mass;
        }
    }
    __syncthreads();
    const uint32_t pos = uniform(sh.place.pos), count = uniform(sh.place.count), n = uniform(sh.n);
    const double mass = uniform(sh.mass);
    const int id = row.nth(pos, count, n, sh);
    if (threadIdx.x == 0) {
        const double y = order.weight.exponent(bits_value(pos_bits(pos)));
        a.ids[r] = id;
        a.logprob[r] = (float)(y - log_of(mass));
    }
}

// float32 rows: the filters as ranks (row_fine.hpp, with its times).  One row
// of 32000 takes 20 us, 64 of them, whose slowest counts, 45 to 51.
template <int NP, bool SPANS>
__global__ __launch_bounds__(kRowThreads) void k_filter_fine(FilterArgs a) {
    __shared__ HistShared sh;
    __shared__ FineShared fs;
    const int r = blockIdx.x;
    FineRow<NP, SPANS, false> row;
    row.init((const float *)a.logits + (size_t)r * (size_t)a.stride, a.mask ? a.mask + (size_t)r * a.wpr : nullptr, a.V);
    const float T = uniform(a.temp[r]);
    const int k = a.top_k ? uniform(a.top_k[r]) : 0;
    const float p = a.top_p ? uniform(a.top_p[r]) : 1.f;
    const float mp = a.min_p ? uniform(a.min_p[r]) : 0.f;
    const float u = uniform(a.uniform[r]);
    const bool greedy = !(T > 0.f);
    typedef HistOrder<FineRow<NP, SPANS, false>> Order;
    Order order(sh, row);
    const auto found = T > kEvenT ? Order::kByDigits : order.template build<false>(greedy ? 1.0 : 1.0 / (double)T);
    if (found == Order::kNone) {
        if (threadIdx.x == 0) {
            a.ids[r] = -1;
            a.logprob[r] = 0.f;
        }
        return;
    }
    int i = -1;
    double mass = 0.0;
    if (found == Order::kCounted) {
        FineDraw<FineRow<NP, SPANS, false>> fine{order, fs};
        i = fine.draw(greedy, k, p, mp, u, mass);
    }
    if (i < 0) {
        __syncthreads();
        filter_by_digits<0>(a, r, *(SelectShared *)sh.h);
        return;
    }
    if (threadIdx.x == 0) {
        const uint64_t e = fs.list[i];
        const double y = order.weight.exponent(value_of_key(~(uint32_t)(e >> 32)));
        a.ids[r] = (int32_t)(uint32_t)e;
        a.logprob[r] = (float)(y - log_of(mass));
    }
}

}  // namespace

}  // namespace cg

using namespace cg;

static int filter_arg_error(const char *msg) {
    set_error("filter_sample: %s", msg);
    return CG_E_ARG;
}

extern "C" {

size_t cg_filter_workspace_bytes(int32_t batch, int32_t vocab) {
    (void)batch;
    (void)vocab;
    return 0;
}

int cg_filter_sample(const void *d_logits, int32_t dtype, int32_t batch, int32_t vocab, int64_t row_stride,
                     const uint64_t *d_mask, int32_t words_per_row, const float *d_temperature,
                     const int32_t *d_top_k, const float *d_top_p, const float *d_min_p, const float *d_uniform,
                     void *d_workspace, int32_t *d_out_ids, float *d_out_logprob, void *stream) {
    if (dtype != 0 && dtype != 1) return filter_arg_error("dtype must be 0 (float32) or 1 (bfloat16)");
    if (batch < 0 || vocab < 1 || vocab > CG_MAX_ROW_VOCAB) return filter_arg_error("bad batch / vocab");
    if (row_stride < vocab) return filter_arg_error("row_stride < vocab");
    if (d_mask && words_per_row < (vocab + 63) / 64) return filter_arg_error("words_per_row < ceil(vocab / 64)");
    if (batch == 0) return CG_OK;
    if (!d_logits || !d_temperature || !d_uniform || !d_out_ids || !d_out_logprob)
        return filter_arg_error("NULL device pointer");
    (void)d_workspace;
    const FilterArgs a{d_logits, row_stride, d_mask, words_per_row, vocab, d_temperature,
                       d_top_k,  d_top_p,    d_min_p, d_uniform,    d_out_ids, d_out_logprob};
    if (dtype == 0) {
        CG_LAUNCH_FINE(k_filter_fine, vocab, batch, (hipStream_t)stream, a);
    } else {
        CG_LAUNCH_ROWS(k_filter_counts, vocab, batch, (hipStream_t)stream, a);
    }
    return launch_status("filter_sample");
}

}  // extern "C"
