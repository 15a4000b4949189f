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
// the sum of all counts, which is checked, and such a row is left to the
// search by digits (row_select.hpp).  The type's lowest value, which many
// programs write where a logit is masked, is not counted: it weighs nothing
// beside any other candidate; a row that has nothing else, or of which it is
// asked for, goes the same way.
//
// Order positions run from the largest value down: position p < 32768 is the
// value of bits 32767 - p, the others the negatives, magnitude rising.  The
// two zeros (positions 32767 and 32768) are one value, kept at 32767.  A
// block is 256 positions in a row, four per lane.
#pragma once
#include "row_select.hpp"

namespace cg {

constexpr int kHistDwords = 32768, kHistBlocks = 256;
constexpr int kPieceIds = 8 * kRowThreads;  // ids of one 16-byte load of every thread
constexpr int kNegInfPair = (int)0xFF80FF80;
constexpr int kInfIdx = 0x7F80;             // bits of +inf; larger ones are NaN
constexpr uint32_t kLowest = 0xFF7Fu;       // bits of the lowest value; larger ones are -inf and NaN
constexpr int kBufWord3 = 0x00020000;       // raw buffer, 32-bit data format

// A place in the order: the position, its candidates, those before it, their mass.
struct HistPlace {
    uint32_t pos, count, above;
    double mass_above, w;
};

struct HistShared {
    uint32_t h[kHistDwords];
    uint32_t dummy[64];  // where lanes count what is no candidate
    union {
        struct {
            uint4 lut[256];              // mask byte -> half of ones per allowed id of four pairs
            uint32_t list[kRowThreads];  // candidates of a value by piece and wave
        };
        double cells[kRowThreads];  // (rows of float32: row_fine.hpp)
    };
    uint32_t blk_cnt[kHistBlocks];
    double blk_mass[kHistBlocks];
    uint32_t counted;    // sum of every count, the dummies' included
    uint32_t any;        // the row has an allowed id
    uint32_t top_block;  // first block with a candidate
    uint32_t top_key;    // key of the largest candidate (rows of float32)
    uint32_t n_blocks;   // blocks with a candidate, listed in any order
    uint16_t blocks[kHistBlocks];
    uint32_t n_list;
    uint32_t w_cnt[kRowWaves];
    int found;
    HistPlace place;     // what the searching wave found
    uint32_t n;
    double mass;
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

// sum + the two 16-bit halves of c
__device__ __forceinline__ uint32_t add_halves(uint32_t c, uint32_t sum) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_udot2(__builtin_bit_cast(u16x2, c), (u16x2){1, 1}, sum, false);
}

__device__ __forceinline__ uint32_t pos_bits(uint32_t pos) {
    return pos < 32768u ? 32767u - pos : pos;  // negatives: 0x8000 | magnitude
}
__device__ __forceinline__ float bits_value(uint32_t b) { return __uint_as_float(b << 16); }

// The row: NP pieces a thread held in registers; with SPANS, longer rows are
// taken in spans of NP.  With ONCE the loads are non-temporal.  Every load is 16 bytes from a 16-byte boundary:
// a row that starts past one by `skew` ids is taken from the boundary, the
// ids before its own start never allowed.
template <int NP, bool SPANS, bool ONCE>
struct HistRow {
    static constexpr int kSpan = NP * kPieceIds;
    static constexpr bool kExact = true;  // a position is one value
    static __device__ __forceinline__ float bin_value(uint32_t bits, float) { return bits_value(bits); }
    __amdgpu_buffer_rsrc_t rx, rm;
    const uint16_t *x;
    const uint64_t *mask;
    int V, skew;
    uint32_t d[NP][4];
    int span_at;    // the span in the registers
    uint32_t live;  // bit p: the wave's piece p has an allowed id

    __device__ void init(const void *logits, const uint64_t *m, int wpr, int vocab) {
        x = (const uint16_t *)logits;
        mask = m;
        V = vocab;
        skew = (int)(((uintptr_t)logits & 15) >> 1);
        rx = __builtin_amdgcn_make_buffer_rsrc((void *)(x - skew), (short)0, ((V + skew) * 2 + 3) & ~3, kBufWord3);
        rm = __builtin_amdgcn_make_buffer_rsrc((void *)m, (short)0, m ? (vocab + 63) / 64 * 8 : 0, kBufWord3);
    }
    __device__ int spans() const { return SPANS ? (V + skew + kSpan - 1) / kSpan : 1; }
    __device__ int first_id(int span, int p) const {
        return span * kSpan + p * kPieceIds + (int)threadIdx.x * 8 - skew;
    }

    // Bit j: id first + j is in the row and allowed.
    __device__ __forceinline__ uint32_t allowed8(uint32_t byte, int first) const {
        const int left = V - first;
        if (first < 0) byte &= 0xFFu << -first;
        return left >= 8 ? byte : left <= 0 ? 0u : byte & ((1u << left) - 1u);
    }

    // The mask bytes of a span's pieces as they lie (8 bits, or 16 that hold a skewed row's 8).
    __device__ __forceinline__ void ask_mask(int span, uint32_t (&raw)[NP]) const {
#pragma unroll
        for (int p = 0; p < NP; p++) {
            raw[p] = 0xFFFFu;
            if (mask) {
                const int q = (span * kSpan + p * kPieceIds) / 8 + (int)threadIdx.x;
                raw[p] = __builtin_amdgcn_raw_buffer_load_b8(rm, q, 0, 0);
                if (skew) raw[p] = (raw[p] << 8) | __builtin_amdgcn_raw_buffer_load_b8(rm, q - 1, 0, 0);
            }
        }
    }
    __device__ __forceinline__ uint32_t usable(int span, int p, uint32_t raw) const {
        return allowed8(skew ? (raw >> (8 - skew)) & 0xFFu : raw & 0xFFu, first_id(span, p));
    }
    // Asks for a piece.  A lane whose 8 ids are all masked asks past the
    // buffer's end, which reads nothing (a constrained row's mask is mostly
    // zeros); without a branch, so that the loads stay in flight together.
    __device__ __forceinline__ void ask(int span, int p, bool any) {
        const uint4 v = __builtin_bit_cast(
            uint4, __builtin_amdgcn_raw_buffer_load_b128(rx, any ? (first_id(span, p) + skew) * 2 : 0x7FFFFFF0, 0, ONCE ? 2 : 0));
        d[p][0] = v.x; d[p][1] = v.y; d[p][2] = v.z; d[p][3] = v.w;
    }
    // Piece p's ids that are not allowed become -inf (bytes: piece p's in
    // byte p % 4 of word p / 4).
    static constexpr int kWords = (NP + 3) / 4;
    __device__ __forceinline__ void select(int span, int p, const uint32_t (&bytes)[kWords], const uint4 *lut) {
        if (mask || skew || span * kSpan + (p + 1) * kPieceIds > V) {  // uniform
            const uint4 s = lut[(bytes[p / 4] >> (8 * (p % 4))) & 0xFFu];
            d[p][0] = (d[p][0] & s.x) | (~s.x & kNegInfPair);
            d[p][1] = (d[p][1] & s.y) | (~s.y & kNegInfPair);
            d[p][2] = (d[p][2] & s.z) | (~s.z & kNegInfPair);
            d[p][3] = (d[p][3] & s.w) | (~s.w & kNegInfPair);
        }
    }
    static __device__ __forceinline__ uint32_t bit_if_any(bool v, int p) { return (__ballot(v) ? 1u : 0u) << p; }

    // Asks for the pieces from `from` on and notes which may be used.
    __device__ __forceinline__ void ask_rest(int span, int from, const uint32_t (&raw)[NP], uint32_t (&bytes)[kWords]) {
        live = 0;
#pragma unroll
        for (int p = 0; p < NP; p++) {
            const uint32_t b = usable(span, p, raw[p]);
            bytes[p / 4] = (p % 4 ? bytes[p / 4] : 0u) | b << (8 * (p % 4));
            live |= bit_if_any(b != 0, p);
            if (p >= from) ask(span, p, b != 0);
        }
    }

    // Reads a span.
    __device__ __forceinline__ void load(int span, const uint4 *lut) {
        uint32_t raw[NP], bytes[kWords];
        span_at = span;
        ask_mask(span, raw);
        ask_rest(span, 0, raw, bytes);
#pragma unroll
        for (int p = 0; p < NP; p++)
            if ((live >> p) & 1) select(span, p, bytes, lut);
    }

    // Reads and counts the whole row.  The first quarter of the first span is
    // asked for before the mask is known, so that memory is busy meanwhile;
    // while_waiting runs then.  Of a longer row each piece is asked for as soon
    // as the one before it in its registers is counted.  The last span stays
    // in the registers.
    template <class F>
    __device__ __forceinline__ void read_and_count(HistShared &sh, F while_waiting) {
        constexpr int kEager = NP / 4;
        uint32_t raw[NP], bytes[kWords], dead = 0;
        const int n_spans = spans();
        ask_mask(0, raw);
#pragma unroll
        for (int p = 0; p < kEager; p++) ask(0, p, true);
        while_waiting();
        ask_rest(0, kEager, raw, bytes);
        __syncthreads();  // the counts are cleared
        for (span_at = 0;; span_at++) {
            const bool more = span_at + 1 < n_spans;  // uniform
            uint32_t live_next = 0, bytes_next[kWords];
            if (more) ask_mask(span_at + 1, raw);
#pragma unroll
            for (int p = 0; p < NP; p++) {
                if ((live >> p) & 1) {
                    select(span_at, p, bytes, sh.lut);
                    count(p, sh);
                } else {
                    dead++;
                }
                if (more) {
                    const uint32_t b = usable(span_at + 1, p, raw[p]);
                    bytes_next[p / 4] = (p % 4 ? bytes_next[p / 4] : 0u) | b << (8 * (p % 4));
                    live_next |= bit_if_any(b != 0, p);
                    ask(span_at + 1, p, b != 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (!more) break;
            live = live_next;
#pragma unroll
            for (int i = 0; i < kWords; i++) bytes[i] = bytes_next[i];
        }
        if ((threadIdx.x & 63) == 0) {
            if (dead) atomicAdd(&sh.counted, dead * 512u);  // of one wave
            if (dead < (uint32_t)(NP * n_spans)) sh.any = 1;
        }
    }

    // Counts a piece.  The lowest value, -inf and negative NaNs go to the
    // lane's own dummy (a run of one value would queue at one address).
    __device__ __forceinline__ void count(int p, HistShared &sh) {
        char *h = (char *)sh.h;
        const uint32_t none = (uint32_t)((char *)&sh.dummy[threadIdx.x & 63] - h);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t w = d[p][j];
            const uint32_t a0 = (w << 2) & 0x1FFFCu, a1 = (w >> 14) & 0x1FFFCu;
            atomicAdd((uint32_t *)(h + ((uint16_t)w < kLowest ? a0 : none)), (w & 0x8000u) ? 0x10000u : 1u);
            atomicAdd((uint32_t *)(h + (w < kLowest << 16 ? a1 : none)), (int)w < 0 ? 0x10000u : 1u);
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
            if (!((live >> p) & 1)) continue;
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

    // Whether the row holds the type's lowest value.  Every thread calls it.
    __device__ __forceinline__ bool has_lowest(HistShared &sh) {
        const uint32_t want = kLowest | kLowest << 16;
        bool has = false;
        const int n_spans = spans();
        for (int s = 0; s < n_spans; s++) {
            if (SPANS && s) load(s - 1, sh.lut);
#pragma unroll
            for (int p = 0; p < NP; p++) {
                if (!((live >> p) & 1)) continue;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t y = d[p][j] ^ want;
                    has = has || (uint16_t)y == 0 || y < 0x10000u;
                }
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) sh.any = 0;
        __syncthreads();
        if (__any(has) && (threadIdx.x & 63) == 0) sh.any = 1;
        __syncthreads();
        return uniform(sh.any) != 0;
    }

    // Lists the first `upto` candidates of position pos by rising id, reading
    // the row again 1024 ids at a time (more of one value than the list takes).
    __device__ void first_of(uint32_t pos, uint32_t upto, uint64_t *list, HistShared &sh) const {
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
#pragma unroll 1
            for (int w = 0; w < kRowWaves; w++) {
                const uint32_t c = uniform(sh.w_cnt[w]);
                mine += w < wave ? c : 0;
                before += c;
            }
            mine += __popcll(hits & ((1ull << lane) - 1));
            if (hit && mine < upto) list[mine] = (uint64_t)pos << 32 | (uint32_t)i;
            __syncthreads();
        }
    }
    // Whether the two halves of each of a piece's words are the value.
    struct Match {
        uint32_t want, same;  // the value's bits twice; what of them counts (the two zeros)
        __device__ __forceinline__ explicit Match(uint32_t pos) {
            const uint32_t bits = pos_bits(pos);
            want = bits | bits << 16;
            same = bits == 0 ? 0x7FFF7FFFu : 0xFFFFFFFFu;
        }
        __device__ __forceinline__ uint32_t rest(uint32_t w) const { return (w ^ want) & same; }
        static __device__ __forceinline__ bool low(uint32_t rest) { return (uint16_t)rest == 0; }
        static __device__ __forceinline__ bool high(uint32_t rest) { return rest < 0x10000u; }
        // Bit j: id j of a piece is the value.
        static __device__ __forceinline__ uint32_t bits(uint32_t y0, uint32_t y1, uint32_t y2, uint32_t y3) {
            return (low(y0) ? 1u : 0u) | (high(y0) ? 2u : 0u) | (low(y1) ? 4u : 0u) | (high(y1) ? 8u : 0u) |
                   (low(y2) ? 16u : 0u) | (high(y2) ? 32u : 0u) | (low(y3) ? 64u : 0u) | (high(y3) ? 128u : 0u);
        }
    };

    // The id of the n-th (from 0) of the row's `count` candidates of position
    // pos, by rising id: counted by piece and wave, which is the ids' order,
    // then the one wave that holds it looks closer.  A longer row's last span
    // is in the registers: its ids are the largest, the other spans are read
    // again only if the n-th is not among them.
    __device__ __forceinline__ int nth(uint32_t pos, uint32_t count, uint32_t n, HistShared &sh) {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        const Match match(pos);
        const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6)), n_spans = spans();
        uint32_t *const cnt = sh.list;  // by piece, then wave
        static_assert(NP * kRowWaves <= kRowThreads, "the counts fit");
        uint32_t before = 0;  // in the spans looked at
        for (int s = 0; s < n_spans; s++) {
            if (SPANS && s) load(s - 1, sh.lut);
            // ids of a piece that differ, two pieces a register, then summed over the wave
            uint32_t other[(NP + 1) / 2];
#pragma unroll
            for (int p = 0; p < NP; p++) {
                uint32_t o = 8;
                if ((live >> p) & 1) {
                    u16x2 m = (u16x2){0, 0};
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        m += __builtin_elementwise_min(__builtin_bit_cast(u16x2, match.rest(d[p][j])), (u16x2){1, 1});
                    o = add_halves(__builtin_bit_cast(uint32_t, m), 0);
                }
                other[p / 2] = p % 2 ? other[p / 2] | o << 16 : o;
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < (NP + 1) / 2; i++) other[i] = (uint32_t)wave_scan((int)other[i]);  // the last lane has the sum
            __syncthreads();  // (the counts' last readers)
            if (lane == 63) {
#pragma unroll
                for (int p = 0; p < NP; p++) cnt[p * kRowWaves + wave] = 512u - ((other[p / 2] >> (16 * (p % 2))) & 0xFFFFu);
            }
            __syncthreads();
            // every wave: where the n-th is
            constexpr int kEach = (NP * kRowWaves + 63) / 64;
            uint32_t c[kEach], sum = 0;
#pragma unroll
            for (int i = 0; i < kEach; i++) {
                c[i] = lane * kEach + i < NP * kRowWaves ? cnt[lane * kEach + i] : 0u;
                sum += c[i];
            }
            const uint32_t incl = (uint32_t)wave_scan((int)sum);
            const uint32_t all = (uint32_t)lane_int((int)incl, 63);
            uint32_t skip = before;
            if (SPANS && s == 0 && n_spans > 1) {  // the last span
                skip = count - all;
                if (n < skip) continue;
            }
            if (n < skip + all) {
                const uint32_t left = n - skip;
                const int L = __builtin_ctzll(__ballot(incl > left));
                uint32_t at = 0, first = incl - sum, run = first;
                bool done = false;
#pragma unroll
                for (int i = 0; i < kEach; i++) {
                    const bool is = !done && run + c[i] > left;
                    at = is ? (uint32_t)(lane * kEach + i) : at;
                    first = is ? run : first;
                    done = done || is;
                    run += c[i];
                }
                const int where = lane_int((int)at, L);
                uint32_t rest = left - (uint32_t)lane_int((int)first, L);
                if (where % kRowWaves == wave) {
                    const int piece = where / kRowWaves;
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int p = 0; p < NP; p++)
                        if (p == piece) {  // uniform
#pragma unroll
                            for (int j = 0; j < 4; j++) w[j] = match.rest(d[p][j]);
                        }
                    uint32_t bits = match.bits(w[0], w[1], w[2], w[3]);
                    const uint32_t mine = __popc(bits), upto = (uint32_t)wave_scan((int)mine);
                    if (upto > rest && upto - mine <= rest) {
                        for (uint32_t i = rest - (upto - mine); i; i--) bits &= bits - 1;
                        sh.found = first_id(span_at, piece) + __builtin_ctz(bits);
                    }
                }
                break;
            }
            before += all;
        }
        __syncthreads();
        return uniform(sh.found);
    }
};

__device__ __forceinline__ void clear_counts(HistShared &sh) {
    uint4 *h = (uint4 *)sh.h;
#pragma unroll
    for (int i = 0; i < kHistDwords / 4 / kRowThreads; i++) h[threadIdx.x + i * kRowThreads] = make_uint4(0, 0, 0, 0);
}

// What dword i counts, without NaN, both zeros as the positive one.
__device__ __forceinline__ void cleaned(int i, uint32_t c, uint32_t &pos, uint32_t &neg) {
    pos = i > kInfIdx ? 0u : c & 0xFFFFu;
    neg = c >> 16;
    if (i == 0) {
        pos += neg;
        neg = 0;
    }
}
// Candidates of the lane's four order positions of a block, b * 256 + 4 lane + j.
__device__ __forceinline__ void bins(const HistShared &sh, int b, uint32_t (&c)[4]) {
    const int lane = threadIdx.x & 63;
    const bool neg = b >= kHistBlocks / 2;  // uniform
    const int q = neg ? (b - kHistBlocks / 2) * 64 + lane : (kHistBlocks / 2 - 1 - b) * 64 + 63 - lane;
    const uint4 v = ((const uint4 *)sh.h)[q];
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint32_t cp, cn;
        const int at = neg ? j : 3 - j;
        cleaned(q * 4 + at, neg ? d[j] : d[3 - j], cp, cn);
        c[j] = neg ? cn : cp;
    }
}
// Weights of those positions; what stands where there is no candidate is
// finite and of no meaning.  Four positions of bfloat16 values in a row are
// equally far apart, so their weights are a geometric progression: two
// exponentials, while a step is small (the first may lie three steps above
// the largest candidate) and none of them is infinite.
template <class ROW>
__device__ __forceinline__ void bin_weights(const Weight &weight, int b, const uint32_t (&c)[4], double (&w)[4]) {
    const uint32_t pos = b * 256 + 4 * (threadIdx.x & 63);
    if constexpr (ROW::kExact) {
        const double y0 = weight.exponent(bits_value(pos_bits(pos))), y1 = weight.exponent(bits_value(pos_bits(pos + 1)));
        const double step = y1 - y0;
        if (b > 0 && b < kHistBlocks - 1 && __all(step >= -1.0 && step <= 0.0)) {
            const double ratio = exp_falling(step);
            w[0] = exp_falling(fmin(y0, 3.0));
            w[1] = w[0] * ratio;
            w[2] = w[1] * ratio;
            w[3] = w[2] * ratio;
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        w[j] = weight(c[j] ? ROW::bin_value(pos_bits(pos + j), weight.largest()) : weight.largest());
        __builtin_amdgcn_sched_barrier(0);  // one at a time: four at once take the registers that hold the row
    }
}

// Lists the blocks that hold candidates and notes the first; where asked,
// sums all counts.  A wave takes 256 dwords at a time, 4 a lane: a block of
// positives and one of negatives.
__device__ __forceinline__ void survey(HistShared &sh, bool sum_up) {
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const uint4 *h4 = (const uint4 *)sh.h;
    uint32_t sum = 0;
#pragma unroll
    for (int part = 0; part < 4; part++) {
        uint4 c[2];
#pragma unroll
        for (int i = 0; i < 2; i++) c[i] = h4[(wave + 16 * (2 * part + i)) * 64 + lane];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int g = wave + 16 * (2 * part + i);
            const uint32_t all = c[i].x | c[i].y | c[i].z | c[i].w;
            if (__ballot(all != 0) == 0) continue;  // most are empty
            if (sum_up) {
                sum = add_halves(c[i].x, add_halves(c[i].y, sum));
                sum = add_halves(c[i].z, add_halves(c[i].w, sum));
            }
            uint32_t pos = all & 0xFFFFu, neg = all >> 16;
            if (g == 0 || g == kHistDwords / 256 - 1) {  // zeros and NaNs
                pos = neg = 0;
                const uint32_t v[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t cp, cn;
                    cleaned(g * 256 + lane * 4 + j, v[j], cp, cn);
                    pos |= cp;
                    neg |= cn;
                }
            }
            const bool has_pos = __ballot(pos != 0) != 0, has_neg = __ballot(neg != 0) != 0;
            if (lane < 2 && (lane ? has_neg : has_pos)) {
                const int b = lane ? kHistBlocks / 2 + g : kHistBlocks / 2 - 1 - g;
                sh.blocks[atomicAdd(&sh.n_blocks, 1u)] = (uint16_t)b;
                atomicMin(&sh.top_block, (uint32_t)b);
            }
        }
    }
    if (sum_up) {
        if (wave == 0) sum = add_halves(sh.dummy[lane], sum);
        sum = (uint32_t)wave_scan((int)sum);
        if (lane == 63) atomicAdd(&sh.counted, sum);
    }
}

// Totals of the listed blocks, a block a wave: candidates, and with MASS their weights.
template <class ROW, bool MASS>
__device__ __forceinline__ void total(HistShared &sh, const Weight &weight) {
    const int wave = uniform((int)(threadIdx.x >> 6)), n = uniform((int)sh.n_blocks);
    for (int e = wave; e < n; e += kRowWaves) {
        const int b = uniform((int)sh.blocks[e]);
        uint32_t c[4];
        bins(sh, b, c);
        const int s = wave_scan((int)(c[0] + c[1] + c[2] + c[3]));
        if ((threadIdx.x & 63) == 63) sh.blk_cnt[b] = (uint32_t)s;
        if (MASS) {
            double w[4];
            bin_weights<ROW>(weight, b, c, w);
            const double m =
                wave_scan(((double)c[0] * w[0] + (double)c[1] * w[1]) + ((double)c[2] * w[2] + (double)c[3] * w[3]));
            if ((threadIdx.x & 63) == 63) sh.blk_mass[b] = m;
        }
    }
}

// The largest candidate's position, from the first block.
__device__ __forceinline__ uint32_t top_position(const HistShared &sh) {
    const int b = uniform((int)sh.top_block);
    uint32_t c[4];
    bins(sh, b, c);
    const int first = c[0] ? 0 : c[1] ? 1 : c[2] ? 2 : 3;
    const int lane = __builtin_ctzll(__ballot((c[0] | c[1] | c[2] | c[3]) != 0));
    return b * 256 + lane * 4 + lane_int(first, lane);
}

// The counted row: totals by block, and the searches, which one wave runs
// (a workgroup's worth of waves running them alike costs their instructions
// sixteen times: 5 us of 35 at 256 rows of 128256).
template <class ROW>
struct HistOrder {
    HistShared &sh;
    ROW &row;
    Weight weight;
    // Candidates and mass up to the end of the lane's blocks 4 lane + j.
    uint32_t incl;
    double mass_incl;
    __device__ __forceinline__ void blocks(uint32_t (&bc)[4], double (&bm)[4]) const {
        const int lane = threadIdx.x & 63;
        const uint4 c = ((const uint4 *)sh.blk_cnt)[lane];
        bc[0] = c.x; bc[1] = c.y; bc[2] = c.z; bc[3] = c.w;
#pragma unroll
        for (int j = 0; j < 4; j++) bm[j] = sh.blk_mass[4 * lane + j];
    }

    __device__ __forceinline__ HistOrder(HistShared &s, ROW &r) : sh(s), row(r) {}

    // Reads, counts and orders the row under weights 1 / T.
    enum Found { kNone, kCounted, kByDigits };  // no candidate; all well; not a row for counts
    template <bool MASS>
    __device__ __forceinline__ Found build(double inv_t) {
        const int t = threadIdx.x;
        row.read_and_count(sh, [&] {
            clear_counts(sh);
            if (t < 64) sh.dummy[t] = 0;
            if (t < 256) {
                uint32_t m[4];
#pragma unroll
                for (int p = 0; p < 4; p++)
                    m[p] = ((t >> (2 * p)) & 1 ? 0x0000FFFFu : 0u) | ((t >> (2 * p + 1)) & 1 ? 0xFFFF0000u : 0u);
                sh.lut[t] = make_uint4(m[0], m[1], m[2], m[3]);
            }
            if (t < kHistBlocks) {
                sh.blk_cnt[t] = 0;
                sh.blk_mass[t] = 0.0;
            }
            if (t == 0) {
                sh.counted = 0;
                sh.any = 0;
                sh.n_blocks = 0;
                sh.top_block = 0xFFFFFFFFu;
                sh.top_key = 0;
            }
        });
        __syncthreads();
        const bool check = row.V > 65535;  // a count may have overflowed
        survey(sh, check);
        __syncthreads();
        if (check && uniform(sh.counted) != (uint32_t)row.spans() * (uint32_t)ROW::kSpan) return kByDigits;
        if (uniform(sh.top_block) == 0xFFFFFFFFu) return uniform(sh.any) ? kByDigits : kNone;
        if constexpr (ROW::kExact) {
            top_pos_ = top_position(sh);
            weight = Weight(bits_value(pos_bits(top_pos_)), uniform(inv_t));
        } else {
            weight = Weight(uniform(value_of_key(sh.top_key)), uniform(inv_t));
        }
        total<ROW, MASS>(sh, weight);
        __syncthreads();
        if (searches()) {
            uint32_t bc[4];
            double bm[4];
            blocks(bc, bm);
            incl = (uint32_t)wave_scan((int)(bc[0] + bc[1] + bc[2] + bc[3]));
            mass_incl = MASS ? wave_scan((bm[0] + bm[1]) + (bm[2] + bm[3])) : 0.0;
        }
        return kCounted;
    }
    // The masses of a row built without them; every wave calls it.
    __device__ __forceinline__ void add_masses() {
        total<ROW, true>(sh, weight);
        __syncthreads();
        if (searches()) {
            uint32_t bc[4];
            double bm[4];
            blocks(bc, bm);
            mass_incl = wave_scan((bm[0] + bm[1]) + (bm[2] + bm[3]));
        }
    }
    // (These read other lanes: every lane calls them.)
    __device__ bool searches() const { return threadIdx.x < 64; }
    __device__ uint32_t top_pos() const { return top_pos_; }
    __device__ double total_mass() const { return lane_double(mass_incl, 63); }
    __device__ uint32_t total_count() const { return (uint32_t)lane_int((int)incl, 63); }

    // Of four items a lane, in lane order: the first up to whose end there
    // are more than `rank` candidates (HOW 0), more than `mass` (1), at least
    // `mass` (2); the last one with a candidate (0) or with weight (1, 2) if
    // there is none.  c, m: an item's own; ci, mi: the lane's inclusive sums;
    // c0, m0: what lies before all.  Returns its number, the sums before it
    // in c0, m0.
    template <int HOW>
    __device__ __forceinline__ int pick(const uint32_t (&c)[4], const double (&m)[4], uint32_t ci, double mi, uint32_t rank,
                                        double mass, uint32_t &c0, double &m0) const {
        auto reached = [&](uint32_t cs, double ms) { return HOW == 0 ? cs > rank : HOW == 1 ? ms > mass : ms >= mass; };
        auto some = [&](uint32_t cs, double ms) { return HOW == 0 ? cs != 0 : ms > 0.0; };
        const bool full = some(c[0] | c[1] | c[2] | c[3], (m[0] + m[1]) + (m[2] + m[3]));
        const uint64_t f = __ballot(full), h = __ballot(full && reached(c0 + ci, m0 + mi));
        const int L = h ? __builtin_ctzll(h) : f ? 63 - __builtin_clzll(f) : 0;
        // every lane looks at its own four as if it were the one
        uint32_t cb = c0 + ci - (c[0] + c[1] + c[2] + c[3]);
        double mb = m0 + from_left(mi);
        int at = 0;
        bool done = false;
        uint32_t c_at = cb;
        double m_at = mb;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (!done && some(c[j], m[j])) {
                at = j;
                c_at = cb;
                m_at = mb;
                done = reached(cb + c[j], mb + m[j]);
            }
            cb += c[j];
            mb += m[j];
        }
        c0 = (uint32_t)lane_int((int)c_at, L);
        m0 = lane_double(m_at, L);
        return 4 * L + lane_int(at, L);
    }

    // The place of the first position up to whose end ... (see pick).
    template <int HOW>
    __device__ __forceinline__ HistPlace find(uint32_t rank, double mass) {
        HistPlace q;
        q.above = 0;
        q.mass_above = 0.0;
        uint32_t c[4];
        double w[4], m[4];
        blocks(c, m);
        const int b = pick<HOW>(c, m, incl, mass_incl, rank, mass, q.above, q.mass_above);
        bins(sh, b, c);
        bin_weights<ROW>(weight, b, c, w);
#pragma unroll
        for (int j = 0; j < 4; j++) m[j] = (double)c[j] * w[j];
        const uint32_t ci = (uint32_t)wave_scan((int)(c[0] + c[1] + c[2] + c[3]));
        const double mi = wave_scan((m[0] + m[1]) + (m[2] + m[3]));
        const int i = pick<HOW>(c, m, ci, mi, rank, mass, q.above, q.mass_above);
        const int j = i & 3;
        q.pos = b * 256 + i;
        q.count = (uint32_t)lane_int((int)(j == 0 ? c[0] : j == 1 ? c[1] : j == 2 ? c[2] : c[3]), i >> 2);
        q.w = lane_double(j == 0 ? w[0] : j == 1 ? w[1] : j == 2 ? w[2] : w[3], i >> 2);
        return q;
    }

    // Candidates of the positions up to pos, its own included.
    __device__ __forceinline__ uint32_t count_to(uint32_t pos) {
        const int b = pos >> 8, lane = threadIdx.x & 63, at = (int)(pos & 255u);
        uint32_t before = (uint32_t)from_left((int)incl), n = 0, c[4];
        double m[4];
        blocks(c, m);
#pragma unroll
        for (int j = 0; j < 3; j++) before += j < (b & 3) ? c[j] : 0u;
        before = (uint32_t)lane_int((int)before, b >> 2);
        bins(sh, b, c);
#pragma unroll
        for (int j = 0; j < 4; j++) n += 4 * lane + j <= at ? c[j] : 0u;
        return before + (uint32_t)lane_int(wave_scan((int)n), 63);
    }
    // The same by rank without masses.
    __device__ __forceinline__ HistPlace find_rank(uint32_t rank) {
        const int lane = threadIdx.x & 63;
        HistPlace q;
        q.mass_above = q.w = 0.0;
        uint32_t c[4];
        const uint4 v = ((const uint4 *)sh.blk_cnt)[lane];
        c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
        uint32_t before = 0, in = incl;
#pragma unroll
        for (int step = 0; step < 2; step++) {
            const uint32_t own = c[0] + c[1] + c[2] + c[3];
            const uint64_t f = __ballot(own != 0), h = __ballot(own != 0 && before + in > rank);
            const int L = h ? __builtin_ctzll(h) : f ? 63 - __builtin_clzll(f) : 0;
            // every lane looks at its own four as if it were the one: the
            // first that reaches the rank, else the last with a candidate
            uint32_t sum = before + in - own, at = 0, sum_at = sum, c_at = 0;
            bool done = false;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bool is = !done && c[j] != 0;
                at = is ? j : at;
                sum_at = is ? sum : sum_at;
                c_at = is ? c[j] : c_at;
                sum += c[j];
                done = done || (is && sum > rank);
            }
            before = (uint32_t)lane_int((int)sum_at, L);
            q.count = (uint32_t)lane_int((int)c_at, L);
            const int i = 4 * L + lane_int((int)at, L);
            if (step == 0) {
                q.pos = (uint32_t)i;
                        bins(sh, i, c);
                in = (uint32_t)wave_scan((int)(c[0] + c[1] + c[2] + c[3]));
            } else {
                q.pos = q.pos * 256 + i;
            }
        }
        q.above = before;
        return q;
    }

    // Mass of the positions up to pos, its own included.
    __device__ __forceinline__ double mass_to(uint32_t pos) {
        const int b = pos >> 8, lane = threadIdx.x & 63, at = (int)(pos & 255u);
        double before = from_left(mass_incl), m = 0.0, w[4];
        uint32_t c[4];
        blocks(c, w);
#pragma unroll
        for (int j = 0; j < 3; j++) before += j < (b & 3) ? w[j] : 0.0;
        before = lane_double(before, b >> 2);
        bins(sh, b, c);
        bin_weights<ROW>(weight, b, c, w);
#pragma unroll
        for (int j = 0; j < 4; j++) m += 4 * lane + j <= at ? (double)c[j] * w[j] : 0.0;
        return before + lane_double(wave_scan(m), 63);
    }

  private:
    uint32_t top_pos_;
};

// Launches KERNEL<NP, SPANS, ONCE> with as many pieces as rows of V ids need
// (7: the largest skew).  20 pieces are 80 of a thread's 128 registers; beyond
// that, spans of 16.  ONCE for rows that are read once and do not fit the
// caches together: above 32 MB, all L2s' size, such loads take top 64 of
// 1024 x 151936 from 135.7 to 129.5 us and the draw of 256 x 128256 from 33.1
// to 32.6; rows that the L2s still hold are slower so (top 20 of 128 x 128256
// 22.5 -> 24.3 us), and so are spans, which are read again (64 x 256000
// 35.7 -> 39.9).
constexpr size_t kOnceBytes = size_t(32) << 20;
#define CG_LAUNCH_PIECES(KERNEL, NP, ONCE, GRID, STREAM, ARGS)                                                \
    do {                                                                                                      \
        if (ONCE) hipLaunchKernelGGL((KERNEL<NP, false, true>), GRID, dim3(kRowThreads), 0, STREAM, ARGS);    \
        else hipLaunchKernelGGL((KERNEL<NP, false, false>), GRID, dim3(kRowThreads), 0, STREAM, ARGS);        \
    } while (0)
#define CG_LAUNCH_ROWS(KERNEL, V, BATCH, STREAM, ARGS)                                                        \
    do {                                                                                                      \
        const int pieces_ = ((V) + 7 + kPieceIds - 1) / kPieceIds;                                            \
        const bool once_ = (size_t)(BATCH) * (size_t)(V) * 2 > kOnceBytes;                                    \
        const dim3 grid_(BATCH);                                                                              \
        if (pieces_ <= 4) CG_LAUNCH_PIECES(KERNEL, 4, once_, grid_, STREAM, ARGS);                            \
        else if (pieces_ <= 8) CG_LAUNCH_PIECES(KERNEL, 8, once_, grid_, STREAM, ARGS);                       \
        else if (pieces_ <= 16) CG_LAUNCH_PIECES(KERNEL, 16, once_, grid_, STREAM, ARGS);                     \
        else if (pieces_ <= 20) CG_LAUNCH_PIECES(KERNEL, 20, once_, grid_, STREAM, ARGS);                     \
        else hipLaunchKernelGGL((KERNEL<16, true, false>), grid_, dim3(kRowThreads), 0, STREAM, ARGS);        \
    } while (0)

}  // namespace cg
