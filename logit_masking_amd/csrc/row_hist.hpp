// row_hist.hpp -- the order of one masked row of bfloat16 logits, by one
// workgroup in one read of the row.
//
// A bfloat16 has 65536 values, so a row is known up to the ids by how often
// each value occurs, and the weight of a value's candidates is their count
// times one exponential: no weight is summed per logit, every sum is exact
// to the last bits of a double, and its order is fixed.  The row is read
// once into registers (16 bytes a lane and load) while its values are
// counted in LDS; what follows looks at the counts, and at the registers
// again for the ids.
//
// Counts are 16 bits, 128 KB of LDS: dword i holds the counts of the value
// with bits i in its low half and of its negative in the high one.  A count
// can only overflow in a row of 65536 candidates or more; the carry breaks
// the sum of all counts, which is checked, and such a row is counted again
// in 32 bits, one sign at a time (`wide`; -0 with the positives).
//
// Order positions run from the largest value down: position p < 32768 is the
// value of bits 32767 - p, the others the negatives, magnitude rising.  The
// two zeros (positions 32767 and 32768) are one value, kept at 32767.  A
// block is 64 positions in a row, one per lane.
#pragma once
#include "row_select.hpp"

namespace cg {

constexpr int kHistDwords = 32768;
constexpr int kPieceIds = 8 * kRowThreads;  // ids of one 16-byte load of every thread
constexpr int kMaxPieces = 16;              // pieces a thread holds at most; shorter rows are launched with enough
constexpr int kNegInfPair = (int)0xFF80FF80;
constexpr int kInfIdx = 0x7F80;             // bits of +inf; larger ones are NaN
constexpr int kBufWord3 = 0x00020000;       // raw buffer, 32-bit data format

struct HistShared {
    uint32_t h[kHistDwords];
    uint32_t dummy[64];  // where lanes count what is no candidate
    uint4 lut[256];      // mask byte -> half of ones per allowed id of four pairs
    uint32_t blk_cnt[1024];
    double blk_mass[1024];
    uint32_t w_cnt[kRowWaves];
    double w_mass[kRowWaves];
    uint32_t counted;    // sum of every count, the dummies' included
    uint32_t top_pos;    // smallest order position with a candidate
    uint32_t n_list;
    int found;
};

// ---- 64-lane inclusive scan (DPP: rows of 16, then row broadcasts) ----------
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or0(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or0(double v) {
    const long long u = __double_as_longlong(v);
    const int lo = dpp_or0<CTRL, ROWS>((int)u), hi = dpp_or0<CTRL, ROWS>((int)(u >> 32));
    return __longlong_as_double(((long long)hi << 32) | (unsigned)lo);
}
template <class T>
__device__ __forceinline__ T wave_scan(T v) {
    v += dpp_or0<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v += dpp_or0<0x112, 0xF>(v);
    v += dpp_or0<0x114, 0xF>(v);
    v += dpp_or0<0x118, 0xF>(v);
    v += dpp_or0<0x142, 0xA>(v);  // lane 15 of rows 0, 2 into rows 1, 3
    v += dpp_or0<0x143, 0xC>(v);  // lane 31 into rows 2, 3
    return v;
}
// The value of the lane before (0 for lane 0): a wave shift by one.
template <class T>
__device__ __forceinline__ T from_left(T v) {
    return dpp_or0<0x138, 0xF>(v);
}
__device__ __forceinline__ int lane_int(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ double lane_double(double v, int l) {
    const long long u = __double_as_longlong(v);
    const int lo = __builtin_amdgcn_readlane((int)u, l), hi = __builtin_amdgcn_readlane((int)(u >> 32), l);
    return __longlong_as_double(((long long)hi << 32) | (unsigned)lo);
}

__device__ __forceinline__ uint32_t pos_bits(uint32_t pos) {
    return pos < 32768u ? 32767u - pos : pos;  // negatives: 0x8000 | magnitude
}
__device__ __forceinline__ float bits_value(uint32_t b) { return __uint_as_float(b << 16); }

// A place in the order: the position, its candidates, those before it, their mass.
struct HistPlace {
    uint32_t pos, count, above;
    double mass_above, w;
};

// The row: NP pieces a thread held in registers; rows longer than NP pieces
// are taken in spans of NP.  Every load is 16 bytes from a 16-byte boundary:
// a row that starts past one by `skew` ids is taken from the boundary, the
// ids before its own start never allowed.
template <int NP>
struct HistRow {
    static constexpr int kSpan = NP * kPieceIds;
    __amdgpu_buffer_rsrc_t rx, rm;
    const uint16_t *x;
    const uint64_t *mask;
    int V, skew;
    uint32_t d[NP][4];
    int span_at;  // the span in the registers

    __device__ void init(const void *logits, const uint64_t *m, int wpr, int vocab) {
        x = (const uint16_t *)logits;
        mask = m;
        V = vocab;
        skew = (int)(((uintptr_t)logits & 15) >> 1);
        rx = __builtin_amdgcn_make_buffer_rsrc((void *)(x - skew), (short)0, ((V + skew) * 2 + 3) & ~3, kBufWord3);
        rm = __builtin_amdgcn_make_buffer_rsrc((void *)m, (short)0, m ? (vocab + 63) / 64 * 8 : 0, kBufWord3);
    }
    __device__ int spans() const { return NP < kMaxPieces ? 1 : (V + skew + kSpan - 1) / kSpan; }
    __device__ int first_id(int span, int p) const {
        return span * kSpan + p * kPieceIds + (int)threadIdx.x * 8 - skew;
    }

    // Bit j: id first + j is in the row and allowed.
    __device__ __forceinline__ uint32_t allowed8(uint32_t byte, int first) const {
        const int left = V - first;
        if (first < 0) byte &= 0xFFu << -first;
        return left >= 8 ? byte : left <= 0 ? 0u : byte & ((1u << left) - 1u);
    }

    // Reads a span, what is not allowed as -inf.  The mask's bytes come first:
    // a lane whose 8 ids are all masked asks past the buffer's end, which
    // reads nothing (a constrained row's mask is mostly zeros).  while_waiting
    // runs once the mask's loads are in flight.
    template <class F>
    __device__ __forceinline__ void load(int span, const uint4 *lut, F while_waiting) {
        span_at = span;
        const int base = span * kSpan;
        uint32_t mb[NP];
#pragma unroll
        for (int p = 0; p < NP; p++) {
            mb[p] = 0xFFu;
            if (mask) {
                const int q = (base + p * kPieceIds) / 8 + (int)threadIdx.x;
                mb[p] = __builtin_amdgcn_raw_buffer_load_b8(rm, q, 0, 0);
                if (skew) mb[p] = (mb[p] << 8) | __builtin_amdgcn_raw_buffer_load_b8(rm, q - 1, 0, 0);
            }
        }
        while_waiting();
#pragma unroll
        for (int p = 0; p < NP; p++) {
            const int first = first_id(span, p);
            mb[p] = allowed8(mask && skew ? (mb[p] >> (8 - skew)) & 0xFFu : mb[p], first);
            const uint4 v = __builtin_bit_cast(
                uint4, __builtin_amdgcn_raw_buffer_load_b128(rx, mb[p] ? (first + skew) * 2 : 0x7FFFFFF0, 0, 0));
            d[p][0] = v.x; d[p][1] = v.y; d[p][2] = v.z; d[p][3] = v.w;
        }
#pragma unroll
        for (int p = 0; p < NP; p++) {
            if (mask || skew || base + (p + 1) * kPieceIds > V) {  // uniform
                const uint4 s = lut[mb[p]];
                d[p][0] = (d[p][0] & s.x) | (~s.x & kNegInfPair);
                d[p][1] = (d[p][1] & s.y) | (~s.y & kNegInfPair);
                d[p][2] = (d[p][2] & s.z) | (~s.z & kNegInfPair);
                d[p][3] = (d[p][3] & s.w) | (~s.w & kNegInfPair);
            }
        }
    }

    // Counts the registers' values.  -inf and negative NaNs go to the lane's
    // own dummy (a run of one value would queue at one address).
    __device__ __forceinline__ void count(HistShared &sh) {
        char *h = (char *)sh.h;
        const uint32_t none = (uint32_t)((char *)&sh.dummy[threadIdx.x & 63] - h);
#pragma unroll
        for (int p = 0; p < NP; p++) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t w = d[p][j];
                const uint32_t a0 = (w << 2) & 0x1FFFCu, a1 = (w >> 14) & 0x1FFFCu;
                atomicAdd((uint32_t *)(h + ((uint16_t)w < 0xFF80u ? a0 : none)), (w & 0x8000u) ? 0x10000u : 1u);
                atomicAdd((uint32_t *)(h + (w < 0xFF800000u ? a1 : none)), (int)w < 0 ? 0x10000u : 1u);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Appends every candidate of position <= last to the list as (position,
    // id), any order.  Its length (sh.n_list, zeroed by the caller) may pass
    // `room`: what does not fit is dropped.
    __device__ __forceinline__ void collect(uint32_t last, uint64_t *list, uint32_t room, HistShared &sh) {
        typedef short s16x2 __attribute__((ext_vector_type(2)));
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        // positive down to bits b: as signed 16-bit numbers, at least b;
        // negatives too: as unsigned ones, at most the last's bits (zeros:
        // the negative one's).  Positive NaNs pass here and fail below.
        const bool pos = last < 32767u;
        const uint32_t b = last == 32767u ? 0x8000u : pos_bits(last);
#pragma unroll
        for (int p = 0; p < NP; p++) {
            bool hit;
            if (pos) {  // uniform
                s16x2 m = __builtin_elementwise_max(__builtin_bit_cast(s16x2, d[p][0]), __builtin_bit_cast(s16x2, d[p][1]));
                m = __builtin_elementwise_max(m, __builtin_elementwise_max(__builtin_bit_cast(s16x2, d[p][2]),
                                                                           __builtin_bit_cast(s16x2, d[p][3])));
                hit = max((int)m.x, (int)m.y) >= (int)b;
            } else {
                u16x2 m = __builtin_elementwise_min(__builtin_bit_cast(u16x2, d[p][0]), __builtin_bit_cast(u16x2, d[p][1]));
                m = __builtin_elementwise_min(m, __builtin_elementwise_min(__builtin_bit_cast(u16x2, d[p][2]),
                                                                           __builtin_bit_cast(u16x2, d[p][3])));
                hit = min((uint32_t)m.x, (uint32_t)m.y) <= b;
            }
            if (hit) {
                uint64_t lo = d[p][0] | ((uint64_t)d[p][1] << 32), hi = d[p][2] | ((uint64_t)d[p][3] << 32);
                const int first = first_id(span_at, p);
#pragma unroll 1
                for (int j = 0; j < 8; j++) {
                    const uint32_t v = (uint32_t)lo & 0xFFFFu;
                    lo = (lo >> 16) | (hi << 48);
                    hi >>= 16;
                    const uint32_t at = v == 0x8000u ? 32767u : v < 0x8000u ? 32767u - v : v;
                    if (at <= last && (v <= (uint32_t)kInfIdx || v >= 0x8000u)) {
                        const uint32_t slot = atomicAdd(&sh.n_list, 1u);
                        if (slot < room) list[slot] = ((uint64_t)at << 32) | (uint32_t)(first + j);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Calls take(rank, id) for the first `upto` candidates of position pos by
    // rising id, reading the row again 1024 ids at a time.
    template <class F>
    __device__ void walk(uint32_t pos, uint32_t upto, HistShared &sh, F take) const {
        const uint32_t bits = pos_bits(pos), same = bits == 0 ? 0x7FFFu : 0xFFFFu;  // the two zeros
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        uint32_t before = 0;
        __syncthreads();
        for (int base = 0; base < V && before < upto; base += kRowThreads) {  // uniform
            const int i = base + (int)threadIdx.x;
            const bool hit = i < V && (!mask || ((mask[i >> 6] >> (i & 63)) & 1)) && ((x[i] ^ bits) & same) == 0;
            const uint64_t hits = __ballot(hit);
            if (lane == 0) sh.w_cnt[wave] = __popcll(hits);
            __syncthreads();
            uint32_t mine = before;
            for (int w = 0; w < kRowWaves; w++) {
                const uint32_t c = sh.w_cnt[w];
                mine += w < wave ? c : 0;
                before += c;
            }
            mine += __popcll(hits & ((1ull << lane) - 1));
            if (hit && mine < upto) take(mine, i);
            __syncthreads();
        }
    }
    // The first `upto` candidates of position pos, listed in order.
    __device__ void first_of(uint32_t pos, uint32_t upto, uint64_t *list, HistShared &sh) const {
        walk(pos, upto, sh, [&](uint32_t rank, int id) { list[rank] = ((uint64_t)pos << 32) | (uint32_t)id; });
    }

    // The id of the n-th (from 0) of the row's `count` candidates of position
    // pos, by rising id.
    __device__ int nth(uint32_t pos, uint32_t count, uint32_t n, HistShared &sh) {
        const uint32_t bits = pos_bits(pos);
        const uint32_t same = bits == 0 ? 0x7FFF7FFFu : 0xFFFFFFFFu;  // the two zeros
        const uint32_t want = bits | (bits << 16);
        uint32_t *list = sh.blk_cnt;  // no longer needed
        // match bits of a piece
        auto match = [&](int p) -> uint32_t {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t y = (d[p][j] ^ want) & same;
                m |= ((y & 0xFFFFu) == 0 ? 1u : 0u) << (2 * j);
                m |= ((y >> 16) == 0 ? 1u : 0u) << (2 * j + 1);
            }
            return m;
        };
        if (count <= 512) {
            // few: list their ids in any order, the n-th is the one with n smaller ones
            __syncthreads();
            if (threadIdx.x == 0) sh.n_list = 0;
            __syncthreads();
            const int n_spans = spans();
            for (int s = 0; s < n_spans; s++) {
                const int span = (span_at + (s ? 1 : 0)) % n_spans;  // the one in the registers first
                if (s) load(span, sh.lut, [] {});
#pragma unroll
                for (int p = 0; p < NP; p++) {
                    uint32_t m = match(p);
                    while (m) {
                        const int j = __builtin_ctz(m);
                        m &= m - 1;
                        list[atomicAdd(&sh.n_list, 1u)] = first_id(span, p) + j;
                    }
                }
                __syncthreads();
                if (sh.n_list >= count) break;  // uniform
            }
            if (threadIdx.x < count) {
                const uint32_t id = list[threadIdx.x];
                uint32_t smaller = 0;
                for (uint32_t i = 0; i < count; i++) smaller += list[i] < id;
                if (smaller == n) sh.found = (int)id;
            }
            __syncthreads();
            return sh.found;
        }
        // many: walk the row again
        if (threadIdx.x == 0) sh.found = -1;
        walk(pos, n + 1, sh, [&](uint32_t rank, int id) {
            if (rank == n) sh.found = id;
        });
        return sh.found;
    }
};

// The counted row: totals by block, and the searches.  Every wave runs the
// searches alike, so no result is handed over.
template <int NP>
struct HistOrder {
    HistShared &sh;
    HistRow<NP> &row;
    Weight weight;
    int wide;  // -1: h holds both signs in 16 bits; 0 / 1: that sign in 32 bits
    // lane w < 16: candidates and mass before, and up to the end of, the 64 blocks of w
    uint32_t w_above, w_incl;
    double w_mass_above, w_mass_incl;

    __device__ __forceinline__ HistOrder(HistShared &s, HistRow<NP> &r) : sh(s), row(r) {}

    static __device__ __forceinline__ void clear(HistShared &sh) {
        uint4 *h = (uint4 *)sh.h;
#pragma unroll
        for (int i = 0; i < kHistDwords / 4 / kRowThreads; i++) h[threadIdx.x + i * kRowThreads] = make_uint4(0, 0, 0, 0);
    }

    // Counts of dword i, cleaned: no NaN, both zeros in the positive one.
    __device__ __forceinline__ void cleaned(int i, uint32_t c, uint32_t &pos, uint32_t &neg) const {
        pos = wide < 0 ? c & 0xFFFFu : wide == 0 ? c : 0u;
        neg = wide < 0 ? c >> 16 : wide == 1 ? c : 0u;
        if (i > kInfIdx) pos = 0;
        if (i == 0) {
            pos += neg;
            neg = 0;
        }
    }
    // Candidates of order position b * 64 + lane.
    __device__ __forceinline__ uint32_t bin(int b) const {
        const int lane = threadIdx.x & 63;
        const int i = b >= 512 ? (b - 512) * 64 + lane : (511 - b) * 64 + 63 - lane;
        uint32_t pos, neg;
        cleaned(i, sh.h[i], pos, neg);
        return b >= 512 ? neg : pos;
    }

    // Reads, counts and orders the row under weights 1 / T.  False: no candidate.
    __device__ bool build(double inv_t) {
        const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
        wide = -1;
        row.load(0, sh.lut, [&] {
            clear(sh);
            if (t < 64) sh.dummy[t] = 0;
            if (t < 256) {
                uint32_t m[4];
#pragma unroll
                for (int p = 0; p < 4; p++)
                    m[p] = ((t >> (2 * p)) & 1 ? 0x0000FFFFu : 0u) | ((t >> (2 * p + 1)) & 1 ? 0xFFFF0000u : 0u);
                sh.lut[t] = make_uint4(m[0], m[1], m[2], m[3]);
            }
            sh.blk_cnt[t] = 0;
            sh.blk_mass[t] = 0.0;
            if (t == 0) {
                sh.counted = 0;
                sh.top_pos = 0xFFFFFFFFu;
            }
            __syncthreads();
        });
        row.count(sh);
        const int n_spans = row.spans();
        for (int s = 1; s < n_spans; s++) {
            row.load(s, sh.lut, [] {});
            row.count(sh);
        }
        __syncthreads();
        uint32_t pg, ng;
        survey(pg, ng, true);
        __syncthreads();
        if (sh.counted != (uint32_t)n_spans * (uint32_t)HistRow<NP>::kSpan) {
            // a count overflowed
            if (t == 0) sh.top_pos = 0xFFFFFFFFu;
            for (int sign = 0; sign < 2; sign++) {
                recount(sign);
                survey(pg, ng, false);
                __syncthreads();
                top_pos_ = sh.top_pos;
                if (top_pos_ != 0xFFFFFFFFu) {
                    weight = Weight{(double)bits_value(pos_bits(top_pos_)), inv_t};
                    total(pg, ng);
                }
            }
        } else {
            top_pos_ = sh.top_pos;
            if (top_pos_ == 0xFFFFFFFFu) return false;
            weight = Weight{(double)bits_value(pos_bits(top_pos_)), inv_t};
            total(pg, ng);
        }
        __syncthreads();
        if (top_pos_ == 0xFFFFFFFFu) return false;
        // inclusive sums over each wave's 64 blocks, then over the waves
        const int b = wave * 64 + lane;
        const uint32_t c = (uint32_t)wave_scan((int)sh.blk_cnt[b]);
        const double m = wave_scan(sh.blk_mass[b]);
        sh.blk_cnt[b] = c;
        sh.blk_mass[b] = m;
        if (lane == 63) {
            sh.w_cnt[wave] = c;
            sh.w_mass[wave] = m;
        }
        __syncthreads();
        const uint32_t wc = lane < kRowWaves ? sh.w_cnt[lane] : 0u;
        const double wm = lane < kRowWaves ? sh.w_mass[lane] : 0.0;
        w_incl = (uint32_t)wave_scan((int)wc);
        w_mass_incl = wave_scan(wm);
        w_above = w_incl - wc;
        w_mass_above = from_left(w_mass_incl);
        return true;
    }
    // (These read other lanes: every lane calls them.)
    __device__ uint32_t top_pos() const { return top_pos_; }
    __device__ double total_mass() const { return lane_double(w_mass_incl, kRowWaves - 1); }
    __device__ uint32_t total_count() const { return (uint32_t)lane_int((int)w_incl, kRowWaves - 1); }

    // The first position up to whose end there are more than `rank`
    // candidates (HOW 0), more than `mass` (1), at least `mass` (2); the last
    // one with a candidate (0) or with weight (1, 2) if there is none.
    template <int HOW>
    __device__ HistPlace find(uint32_t rank, double mass) {
        const int lane = threadIdx.x & 63;
        auto reached = [&](uint32_t c, double m) { return HOW == 0 ? c > rank : HOW == 1 ? m > mass : m >= mass; };
        auto some = [&](uint32_t c, double m) { return HOW == 0 ? c != 0 : m > 0.0; };
        auto pick = [&](bool hit, bool full) {  // the first hit, else the last that is not empty
            const uint64_t h = __ballot(hit && full), f = __ballot(full);
            return h ? __builtin_ctzll(h) : f ? 63 - __builtin_clzll(f) : 0;
        };
        const int W = pick(reached(w_incl, w_mass_incl),
                           lane < kRowWaves && some(w_incl - w_above, w_mass_incl - w_mass_above));
        const uint32_t wc = (uint32_t)lane_int((int)w_above, W);
        const double wm = lane_double(w_mass_above, W);
        const uint32_t bc = sh.blk_cnt[W * 64 + lane];
        const double bm = sh.blk_mass[W * 64 + lane];
        const uint32_t bc0 = (uint32_t)from_left((int)bc);
        const double bm0 = from_left(bm);
        const int B = pick(reached(wc + bc, wm + bm), some(bc - bc0, bm - bm0));
        const int b = W * 64 + B;
        const uint32_t c_above = wc + (uint32_t)lane_int((int)bc0, B);
        const double m_above = wm + lane_double(bm0, B);
        hold(b);
        const uint32_t c = bin(b);
        const double w = c ? weight(bits_value(pos_bits(b * 64 + lane))) : 0.0;
        const uint32_t ci = (uint32_t)wave_scan((int)c);
        const double mi = wave_scan((double)c * w);
        const int L = pick(reached(c_above + ci, m_above + mi), some(c, (double)c * w));
        HistPlace q;
        q.pos = b * 64 + L;
        q.count = (uint32_t)lane_int((int)c, L);
        q.above = c_above + (uint32_t)lane_int((int)(ci - c), L);
        q.mass_above = m_above + (L ? lane_double(mi, L - 1) : 0.0);
        q.w = lane_double(w, L);
        return q;
    }

    // Mass of the positions up to pos, its own included.
    __device__ double mass_to(uint32_t pos) {
        const int b = pos >> 6, W = b >> 6, lane = threadIdx.x & 63;
        const double above = lane_double(w_mass_above, W) + ((b & 63) ? sh.blk_mass[b - 1] : 0.0);
        hold(b);
        const uint32_t c = bin(b);
        const double mi = wave_scan(c ? (double)c * weight(bits_value(pos_bits(b * 64 + lane))) : 0.0);
        return above + lane_double(mi, pos & 63);
    }

  private:
    uint32_t top_pos_;

    // Which of the wave's 32 groups of 64 dwords (wave + 16 i) hold positive
    // and negative candidates; the smallest position with one and, where
    // asked, the sum of all counts go to LDS.
    __device__ void survey(uint32_t &pg, uint32_t &ng, bool sum_up) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        uint32_t sum = 0, top = 0xFFFFFFFFu;
        pg = ng = 0;
#pragma unroll 8
        for (int i = 0; i < 32; i++) {
            const int g = wave + 16 * i;
            const uint32_t c = sh.h[g * 64 + lane];
            sum += (c & 0xFFFFu) + (c >> 16);
            uint32_t pos, neg;
            cleaned(g * 64 + lane, c, pos, neg);
            const uint64_t mp = __ballot(pos != 0), mn = __ballot(neg != 0);
            if (mp) {
                pg |= 1u << i;
                top = min(top, (uint32_t)((511 - g) * 64 + __builtin_clzll(mp)));
            }
            if (mn) {
                ng |= 1u << i;
                top = min(top, (uint32_t)(32768 + g * 64 + __builtin_ctzll(mn)));
            }
        }
        if (sum_up) {
            if (wave == 0) sum += (sh.dummy[lane] & 0xFFFFu) + (sh.dummy[lane] >> 16);
            sum = (uint32_t)wave_scan((int)sum);
            if (lane == 63) atomicAdd(&sh.counted, sum);
        }
        if (lane == 0) atomicMin(&sh.top_pos, top);
    }

    // Totals of the blocks of the surveyed groups.
    __device__ void total(uint32_t pg, uint32_t ng) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        uint32_t any = pg | ng;
        while (any) {
            const int i = __builtin_ctz(any);
            any &= any - 1;
            const int g = wave + 16 * i;
            uint32_t pos, neg;
            cleaned(g * 64 + lane, sh.h[g * 64 + lane], pos, neg);
            if ((pg >> i) & 1) put(511 - g, pos, bits_value(g * 64 + lane));
            if ((ng >> i) & 1) put(512 + g, neg, bits_value(0x8000 + g * 64 + lane));
        }
    }
    __device__ __forceinline__ void put(int b, uint32_t c, float value) {
        const uint32_t cs = (uint32_t)wave_scan((int)c);
        const double ms = wave_scan(c ? (double)c * weight(value) : 0.0);
        if ((threadIdx.x & 63) == 63) {
            sh.blk_cnt[b] = cs;
            sh.blk_mass[b] = ms;
        }
    }

    // Block b's counts in h (a row counted one sign at a time holds one).
    __device__ __forceinline__ void hold(int b) {
        if (wide >= 0 && wide != (b >= 512)) recount(b >= 512);  // uniform
    }
    __device__ void recount(int sign) {
        __syncthreads();
        clear(sh);
        __syncthreads();
        wide = sign;
        for (int i = threadIdx.x; i < row.V; i += kRowThreads) {
            if (row.mask && !((row.mask[i >> 6] >> (i & 63)) & 1)) continue;
            const uint32_t v = row.x[i];
            if (v >= 0xFF80u || (v > 0x8000u) != (sign != 0)) continue;
            atomicAdd(&sh.h[v & 0x7FFFu], 1u);
        }
        __syncthreads();
    }
};

}  // namespace cg
