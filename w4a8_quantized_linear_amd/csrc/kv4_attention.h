// Device-side pieces that the attention kernels over the 4-bit key/value cache
// share: the nibble operands, the queries' scaling, the pages a tile of columns
// sees, and where its result goes.  The mathematics is stated in
// kv4_few_rows.hip.
#pragma once

#include "kv4_layout.h"
#include "quant_common.h"

namespace cider {

constexpr float kLog2e = 1.4426950408889634f;

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Maximum of a value and the one 32 (16) lanes away (v_permlane32_swap: no LDS
// round trip, unlike a shuffle).  The second operand is made another value in
// the compiler's eyes: given one value twice it takes both results for equal.
__device__ __forceinline__ float max_lane32(float v)
{
    unsigned u = __builtin_bit_cast(unsigned, v), w = u;
    asm("" : "+v"(w));
    const auto r = __builtin_amdgcn_permlane32_swap(u, w, false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
}
__device__ __forceinline__ float max_lane16(float v)
{
    unsigned u = __builtin_bit_cast(unsigned, v), w = u;
    asm("" : "+v"(w));
    const auto r = __builtin_amdgcn_permlane16_swap(u, w, false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
}

// Maximum over the wavefront, in every lane.
template <int CTRL>
__device__ __forceinline__ float max_dpp(float v)
{
    const int u = __builtin_bit_cast(int, v);
    return __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(u, u, CTRL, 0xF, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v)
{
    v = max_dpp<0xB1>(v);   // quad_perm [1,0,3,2]
    v = max_dpp<0x4E>(v);   // quad_perm [2,3,0,1]
    v = max_dpp<0x141>(v);  // row_half_mirror
    v = max_dpp<0x140>(v);  // row_mirror
    return max_lane32(max_lane16(v));
}

// Maxima of two 16-bit halves at once: over a row of 16 lanes, with the row next to
// it, with the other half of the wavefront.
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b)
{
    typedef unsigned short halves __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(halves, a), __builtin_bit_cast(halves, b)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t max_halves_dpp(uint32_t v)
{
    return max_halves(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t max_halves_row(uint32_t v)
{
    v = max_halves_dpp<0xB1>(v);
    v = max_halves_dpp<0x4E>(v);
    v = max_halves_dpp<0x141>(v);
    return max_halves_dpp<0x140>(v);
}
__device__ __forceinline__ uint32_t max_halves_lane16(uint32_t u)
{
    uint32_t w = u;
    asm("" : "+v"(w));
    const auto r = __builtin_amdgcn_permlane16_swap(u, w, false, false);
    return max_halves(r[0], r[1]);
}
__device__ __forceinline__ uint32_t max_halves_lane32(uint32_t u)
{
    uint32_t w = u;
    asm("" : "+v"(w));
    const auto r = __builtin_amdgcn_permlane32_swap(u, w, false, false);
    return max_halves(r[0], r[1]);
}

// Lane N's value in each row of 16 lanes: a broadcast that the instruction
// which uses it does itself (DPP).
template <int N>
__device__ __forceinline__ float row_lane(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x150 + N, 0xF, 0xF, true));
}
// The same for a constant after unrolling.
__device__ __forceinline__ float row_value(float v, int n)
{
    switch (n) {
    case 0: return row_lane<0>(v);
    case 1: return row_lane<1>(v);
    case 2: return row_lane<2>(v);
    case 3: return row_lane<3>(v);
    case 4: return row_lane<4>(v);
    case 5: return row_lane<5>(v);
    case 6: return row_lane<6>(v);
    case 7: return row_lane<7>(v);
    case 8: return row_lane<8>(v);
    case 9: return row_lane<9>(v);
    case 10: return row_lane<10>(v);
    case 11: return row_lane<11>(v);
    case 12: return row_lane<12>(v);
    case 13: return row_lane<13>(v);
    case 14: return row_lane<14>(v);
    default: return row_lane<15>(v);
    }
}
// A scale of K as the factor of its scores; NaN where it is infinite: the sums that it
// meets are finite, and one below 0 would make the score minus infinity, the token hidden.
__device__ __forceinline__ float key_factor(float scale, float factor) { return __builtin_fmaf(scale, 0.0f, scale * factor); }
// x times the value of lane n of the row.
__device__ __forceinline__ float scaled(float x, float scales, int n) { return row_value(scales, n) * x; }

// What a launch adds to the call's arguments.
struct Kv4Launch {
    int cols;          // columns of a tile
    int tiles;         // column tiles of the longest sequence
    int splits;        // workgroups that a tile's pages may be dealt to
    int pages;         // pages of one of them (splits > 1)
    int waves;         // wavefronts of a few-row workgroup, 4 or 8
    bool once;         // few rows: pages are read by one tile and are more than the last-level cache keeps
    float *part;       // splits > 1: [rows * q_heads][splits][head_dim] outputs, not yet divided by their sums,
                       // times 2^-sum_bits(pages),
    float *part_stat;  // [rows * q_heads][splits][2]: maximum in units of log2, sum
    // With shared prefixes: the first front_groups workgroups are for the runs' shared pages
    // (tiles and splits of their own, front_pages pages a split), the others for what each
    // sequence has behind them.  All leave parts, of one sum_bits(sum_pages): those of
    // shared pages in the first front_splits of `slots`.  The last split has all that is
    // left of a tile's pages.
    Kv4Runs runs;
    unsigned front_groups;
    int front_tiles, front_splits, front_pages, slots, sum_pages;
};

// All: what a launch without shared prefixes does.  Shared: the other, a workgroup's
// part of it told by its Tile.
enum class Pages { All, Shared };

__device__ __forceinline__ float ldexp_f(float x, int e) { return __builtin_amdgcn_ldexpf(x, e); }
__device__ __forceinline__ f32x4 ldexp_f(f32x4 x, int e)
{
    return f32x4{ldexp_f(x.x, e), ldexp_f(x.y, e), ldexp_f(x.z, e), ldexp_f(x.w, e)};
}

// A sum of weights over so many pages is below 2^sum_bits (a weight below 2^3): sums
// of values are kept this much smaller, or those of many large ones would not be
// finite.
__device__ __forceinline__ int sum_bits(int pages) { return 9 + 32 - __builtin_clz(pages | 1); }

// 1 / l of a sum of weights (0, or about 1 and more), 2^-23 off at most; 0 where
// nothing was seen.
__device__ __forceinline__ float reciprocal(float l) { return l == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(l); }

// The 8 nibbles of a dword as fp16 operands u 2^-24, in the order 0 4 1 5 2 6
// 3 7; elements 2, 3, 6, 7 of the result (nibbles 1, 5, 3, 7) are 16 times as
// large.
__device__ __forceinline__ uint4 nibble_halves(uint32_t w)
{
    const uint32_t hi = w >> 8;
    return uint4{w & 0x000F000Fu, w & 0x00F000F0u, hi & 0x000F000Fu, hi & 0x00F000F0u};
}

// -8 2^-24 and -128 2^-24: the codes' offset in the same order.
constexpr uint32_t kOffset = 0x80088008u, kOffset16 = 0x80808080u;

// A lane's share of a query row: N chunks of 8 values.  For finite values the
// magnitudes order as their bit patterns; a chunk with NaN or infinity (no
// scale is taken from those: they would push other columns' values out of
// fp16) is looked at value by value.
template <int DT, int N>
__device__ __forceinline__ float query_top(const uint4 (&w)[N])
{
    constexpr uint32_t kInf = DT == DT_BF16 ? 0x7F80u : 0x7C00u;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t m = chunk_absmax_bits(w[i]);
        top = m > top ? m : top;
    }
    if (top >= kInf) {
        top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t m = (e & 1 ? u[e / 2] >> 16 : u[e / 2]) & 0x7FFFu;
                top = m < kInf && m > top ? m : top;
            }
        }
    }
    return widen_bits<DT>(top);
}
template <int N>
__device__ __forceinline__ float query_top(const uint4 (&w)[N], int dtype)
{
    return dtype == DT_BF16 ? query_top<DT_BF16>(w) : query_top<DT_F16>(w);
}

// 8 query values times 2^shift as an operand against nibble_halves: in the
// order 0 4 1 5 2 6 3 7, those of the odd nibbles divided by 16.
template <int DT>
__device__ __forceinline__ half8 query_operand(uint4 w, int shift)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // values e and e + 4
        const int by = e & 1 ? shift - 4 : shift;
        const uint32_t lo = e & 1 ? u[e / 2] >> 16 : u[e / 2], hi = e & 1 ? u[e / 2 + 2] >> 16 : u[e / 2 + 2];
        o[e] = pack2<OUT_F16>(ldexp_f(widen_bits<DT>(lo), by), ldexp_f(widen_bits<DT>(hi), by));
    }
    return __builtin_bit_cast(half8, uint4{o[0], o[1], o[2], o[3]});
}
template <int N>
__device__ __forceinline__ void query_operands(const uint4 (&w)[N], int dtype, int shift, half8 (&op)[N])
{
    if (dtype == DT_BF16) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            op[i] = query_operand<DT_BF16>(w[i], shift);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            op[i] = query_operand<DT_F16>(w[i], shift);
    }
}

// The sum of an operand's values, the divided ones counted in full.
__device__ __forceinline__ float operand_sum(half8 op, float sum)
{
    const half2_t one = {(_Float16)1, (_Float16)1}, sixteen = {(_Float16)16, (_Float16)16};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        sum = __builtin_amdgcn_fdot2(half2_t{op[2 * e], op[2 * e + 1]}, e & 1 ? sixteen : one, sum, false);
    return sum;
}

// Exponents of V's scales.  Weights go to the matrix cores in fp16, times V's
// scale and a power of two that puts the largest s_v that the column has seen
// just under fp16's end; its outputs are in those units.  The exponent is the
// column's own: a token that the column does not see (behind its window, in front
// of its row) must not move it, or a large value there would flush the column's
// weights.  Powers of two are exact, so a column's result has the same bits
// whatever its neighbours see.  Most often all columns of a wavefront have seen
// scales of one exponent, and the power of two goes into the scales, once a page;
// where they stand apart every weight takes its column's difference.
constexpr int kNoScale = -200;  // nothing seen; below the exponent of every fp32 number
constexpr int kExpBias = 512;   // makes 16-bit halves of exponents
// Where columns stand apart the scales are taken 2^kMiddle up and the columns are
// kept within kSpread, so that every product is a normal number: one that sees
// values 2^kSpread below another's of its wavefront loses bits.
constexpr int kMiddle = 60, kSpread = 180;

__device__ __forceinline__ int scale_exponent(float s)
{
    return s > 0.0f && s < __builtin_inff() ? __builtin_amdgcn_frexp_expf(s) : kNoScale;
}

// One group's exponents, the same in every lane; a column's own (2^own is above
// every finite s_v that it has seen) is kept by the kernel.
struct ScaleExponents {
    int all;    // what the scales are taken to
    int reach;  // the least of own, as a power of two that is a number: scales below 2^reach move nothing
    bool same;  // every lane's own is `all`

    __device__ __forceinline__ void set(int top)
    {
        all = reach = top < -149 ? -149 : top;
        same = true;
    }
    // A page's scales are below 2^top where the lane's column sees them; returns the
    // column's new exponent.  valid: there is such a column.  LANES: 16, or 32.
    template <int LANES>
    __device__ __forceinline__ int raise(int own, int top, bool valid)
    {
        const int now = top > own ? top : own;
        uint32_t u = valid ? (uint32_t)(now + kExpBias) << 16 | (uint32_t)(kExpBias - now) : 0u;
        u = max_halves_row(u);
        if constexpr (LANES == 32)
            u = max_halves_lane16(u);
        u = __builtin_amdgcn_readfirstlane(u);
        const int hi = u ? (int)(u >> 16) - kExpBias : all, lo = u ? kExpBias - (int)(u & 0xFFFFu) : hi;
        set(hi);
        if (lo != hi) {
            all = hi - kMiddle;
            reach = lo < -149 ? -149 : lo;
            same = false;
        }
        return !valid ? hi : (now > kNoScale && now < hi - kSpread ? hi - kSpread : now);
    }
};
// The power of two that a column's weights are short of when they are worked out
// for all; a column that has seen no scale has no weights.
__device__ __forceinline__ int scale_shift(int all, int own) { return own == kNoScale ? 0 : all - own; }

// Masks.  A lane's tokens lie at offsets STRIDE (e / 4) + e % 4 from its first
// one, which rises with e: those in front of an offset are the low bits of a
// word, so a page's mask takes a few operations, not some for every token.
template <int STRIDE>
__device__ __forceinline__ uint32_t tokens_below(int offset)
{
    const int u = offset < 0 ? 0 : (offset > kPageTokens ? kPageTokens : offset);
    const int n = 4 * (u / STRIDE) + (u % STRIDE < 4 ? u % STRIDE : 4);
    return n >= 32 ? ~0u : (1u << n) - 1u;
}
// The tokens that a column at position p sees, the lane's first at position at.
template <int STRIDE>
__device__ __forceinline__ uint32_t tokens_seen(int p, int at, int window, int sinks)
{
    uint32_t seen = tokens_below<STRIDE>(p + 1 - at);
    if (window > 0)
        seen &= ~tokens_below<STRIDE>(p - window + 1 - at) | tokens_below<STRIDE>(sinks - at);
    return seen;
}
__device__ __forceinline__ uint32_t seen_bits(uint32_t seen, int e) { return (uint32_t)((int32_t)(seen << (31 - e)) >> 31); }
// A score, or minus infinity where bit e of the mask is 0.
__device__ __forceinline__ float seen_score(float s, uint32_t seen, int e)
{
    const uint32_t keep = seen_bits(seen, e);
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, s) & keep) | (0xFF800000u & ~keep));
}
// The largest, by halves, of what 16 N tokens have (a row of lanes holds 16), 0
// for those whose bit is 0: it goes round the row, the lane's bits with it.  A loop,
// not 16 copies: it is taken rarely, and its mere length would cost the code around
// it 5 % (registers, instruction fetches).
template <int N>
__device__ __forceinline__ uint32_t seen_largest(const uint32_t (&halves)[N], uint32_t seen, int lane)
{
    uint32_t top = 0, s[N], bits[N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
        s[t] = halves[t];
        bits[t] = (seen >> 16 * t & 0xFFFFu) * 0x10001u >> lane % 16;
    }
#pragma unroll 1
    for (int n = 0; n < 4; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < N; ++t) {
                top = max_halves(top, s[t] & seen_bits(bits[t], i));
                s[t] = (uint32_t)__builtin_amdgcn_mov_dpp((int)s[t], 0x12F, 0xF, 0xF, true);
            }
#pragma unroll
        for (int t = 0; t < N; ++t)
            bits[t] >>= 4;
    }
    return top;
}
// The exponent in a half; 0 there is none.
__device__ __forceinline__ int half_exponent(uint32_t halves, int g)
{
    const int e = (int)(halves >> 16 * g & 0xFFFFu);
    return e ? e - kExpBias : kNoScale;
}

// The pages that a tile of columns sees: [0, sink_pages) and [first, end).
struct PageRange {
    int sink_pages, first, count;
    int lead;  // pages before the first one that lies inside every column's window
    __device__ __forceinline__ int at(int i) const { return i < sink_pages ? i : first + i - sink_pages; }
    // From there on, the ones before it last: what every column sees comes first.
    __device__ __forceinline__ int at_turned(int i) const
    {
        i += lead;
        return at(i < count ? i : i - count);
    }
};

// Columns at positions p_lo .. p_hi; count 0 where p_hi < 0.
__device__ __forceinline__ PageRange pages_seen(int p_lo, int p_hi, int window, int sinks)
{
    PageRange r = {0, 0, 0, 0};
    if (p_hi < 0)
        return r;
    const int end = p_hi / kPageTokens + 1;
    const int from = window > 0 && p_lo - window + 1 > 0 ? p_lo - window + 1 : 0;
    r.first = from / kPageTokens;
    const int kept = window > 0 ? (sinks < p_hi + 1 ? sinks : p_hi + 1) : 0;
    const int kept_pages = (kept + kPageTokens - 1) / kPageTokens;
    r.sink_pages = kept_pages < r.first ? kept_pages : r.first;
    r.count = r.sink_pages + end - r.first;
    if (window > 0 && p_hi >= window) {
        const int lead = r.sink_pages + (p_hi - window) / kPageTokens + 1 - r.first;
        r.lead = lead < r.count ? lead : 0;
    }
    return r;
}

// A run of sequences that share their first pages; pages 0 where there is none, or the
// device's numbers are not sound.
struct Run {
    int first, end, row0, n, pages;  // its sequences first .. end - 1, its rows
};
__device__ __forceinline__ Run run_of(const Kv4Args &a, const Kv4Runs &r, int g)
{
    Run run = {r.group_start[g], r.group_start[g + 1], 0, 0, 0};
    if (run.first < 0 || run.end <= run.first || run.end > a.batch)
        return run;
    run.row0 = a.row_start[run.first];
    const int last = a.row_start[run.end];
    if (run.row0 < 0 || last < run.row0 || last > a.rows || last - run.row0 > r.max_rows)
        return run;
    run.n = last - run.row0;
    const int pages = r.shared_len[g] / kPageTokens;
    run.pages = pages < 0 ? 0 : (pages > r.max_pages ? r.max_pages : pages);
    return run;
}

// The pages that a sequence's rows leave to its run: 0 for a sequence of no run, or one
// whose rows do not all stand behind the shared pages.
__device__ __forceinline__ int shared_pages(const Kv4Args &a, const Kv4Runs &r, int b, const Kv4Sequence &s)
{
    int lo = 0, hi = r.groups;  // the last group that starts at b or before
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (r.group_start[mid] <= b)
            lo = mid;
        else
            hi = mid;
    }
    if (b < r.group_start[lo] || b >= r.group_start[lo + 1])
        return 0;
    const Run run = run_of(a, r, lo);
    const bool in = s.row0 >= run.row0 && s.row0 + s.n <= run.row0 + run.n;
    return in && s.kv - s.n >= run.pages * kPageTokens ? run.pages : 0;
}

// A tile of COLS columns of one (sequence, kv head): columns are the pairs
// (row, query head of the group), c = row * G + g.  Over shared pages (front): of one
// (run, kv head), all of whose rows see all tokens.
struct Tile {
    Kv4Sequence seq;
    int b;                 // whose page table
    int h, G, tile, cols;  // cols: columns of the sequence
    int p_lo, p_hi;        // positions of the tile's first and last column
    bool front;
    int shared;            // pages in front of the range, left to the sequence's run
    PageRange range;
};

template <int COLS, Pages PAGES>
__device__ __forceinline__ bool tile_of(const Kv4AttentionArgs &a, const Kv4Launch &n, int b, int h, int tile, bool front, Tile &t)
{
    t.h = h;
    t.G = a.q_heads / a.kv.kv_heads;
    t.tile = tile;
    t.b = b;
    t.shared = 0;
    t.front = PAGES == Pages::Shared && front;
    if (t.front) {
        const Run run = run_of(a.kv, n.runs, b);
        if (run.pages == 0)
            return false;
        // the first whose rows stand behind the shared pages: a padded slot's table may
        // name anything
        for (t.b = run.first;; ++t.b) {
            if (t.b == run.end)
                return false;
            const Kv4Sequence s = kv4_sequence(a.kv, t.b);
            if (s.n > 0 && s.kv - s.n >= run.pages * kPageTokens)
                break;
        }
        t.seq.row0 = run.row0;
        t.seq.n = run.n;
        t.seq.kv = run.pages * kPageTokens;
    } else {
        t.seq = kv4_sequence(a.kv, b);
    }
    t.cols = t.seq.n * t.G;
    if ((int64_t)tile * COLS >= t.cols)
        return false;
    const int first = t.seq.kv - t.seq.n;
    const int last = t.cols - tile * COLS < COLS ? t.cols - 1 : tile * COLS + COLS - 1;
    t.p_lo = t.front ? t.seq.kv - 1 : first + tile * COLS / t.G;
    t.p_hi = t.front ? t.seq.kv - 1 : first + last / t.G;
    t.range = pages_seen(t.p_lo, t.p_hi, a.window, a.sinks);
    if (PAGES == Pages::Shared && !t.front) {  // window 0: the range is [0, count)
        t.shared = shared_pages(a.kv, n.runs, b, t.seq);
        t.range.first += t.shared;
        t.range.count -= t.shared;
    }
    return true;
}

// The position of a row of the tile's sequence.
template <Pages PAGES>
__device__ __forceinline__ int position_of(const Tile &t, int row)
{
    return PAGES == Pages::Shared && t.front ? t.p_hi : t.seq.kv - t.seq.n + row;
}

// What a workgroup has: a tile of a kv head of a sequence, or of a run (front), and which
// of its chunks.  Heads go fastest, then sequences, splits and tiles.
struct Work {
    bool front;
    int head, b, split, tile;
};
template <Pages PAGES>
__host__ __device__ __forceinline__ int splits_of(const Kv4Launch &n, bool front)
{
    return PAGES == Pages::Shared && front ? n.front_splits : n.splits;
}
// False past the launch's last workgroup: a grid of more than kMostX is rounded up to
// whole rows of those, and a launch for shared pages alone (tiles 0) has none behind the
// front's.
template <Pages PAGES>
__host__ __device__ __forceinline__ bool work_of(const Kv4AttentionArgs &a, const Kv4Launch &n, unsigned id, Work &w)
{
    w.front = PAGES == Pages::Shared && id < n.front_groups;
    if (PAGES == Pages::Shared && !w.front)
        id -= n.front_groups;
    w.head = (int)(id % (unsigned)a.kv.kv_heads);
    id /= (unsigned)a.kv.kv_heads;
    const unsigned batch = (unsigned)(w.front ? n.runs.groups : a.kv.batch), splits = (unsigned)splits_of<PAGES>(n, w.front);
    w.b = (int)(id % batch);
    id /= batch;
    w.split = (int)(id % splits);
    w.tile = (int)(id / splits);
    return w.front || w.tile < n.tiles;
}
// How many chunks of how many pages a tile's pages are dealt to.
template <Pages PAGES>
__device__ __forceinline__ bool chunk_of(const Kv4Launch &n, const Tile &t, int split, int &begin, int &end)
{
    const int splits = splits_of<PAGES>(n, t.front), pages = PAGES == Pages::Shared && t.front ? n.front_pages : n.pages;
    begin = splits > 1 ? split * pages : 0;
    if (split > 0 && begin >= t.range.count)
        return false;
    const bool rest = PAGES == Pages::All ? splits < 2 : split == splits - 1;
    end = !rest && begin + pages < t.range.count ? begin + pages : t.range.count;
    return true;
}

// Whether a tile's results are parts.  (With shared prefixes all are, but for a tile that
// sees no page, rows in front of their sequence: it has its zeros at once.)
template <Pages PAGES>
__device__ __forceinline__ bool in_parts(const Kv4Launch &n, const Tile &t)
{
    return PAGES == Pages::All ? n.splits > 1 && t.range.count > n.pages : t.range.count > 0;
}
template <Pages PAGES>
__device__ __forceinline__ int64_t part_of(const Kv4Launch &n, const Tile &t, int64_t pair, int split)
{
    return PAGES == Pages::All ? pair * n.splits + split : pair * n.slots + (t.front ? 0 : n.front_splits) + split;
}

// The tile's first position is its newest token that all columns may see (false: their
// windows share none): the columns' exponents start of V's scales there, so that a page
// which only some of them see finds them alike.  Of a tile that sees pages; 0 where
// there is none.
__device__ __forceinline__ bool tile_has_first(const Kv4AttentionArgs &a, const Tile &t)
{
    return t.p_lo >= 0 && (a.window == 0 || t.p_lo > t.p_hi - a.window || t.p_lo < a.sinks);
}
template <int D, int GS>
__device__ __forceinline__ void first_scales(const Kv4AttentionArgs &a, const Tile &t, const int32_t *table, float (&s)[D / GS])
{
    // loaded in any case, from memory that is there, and taken or not: nothing waits
    const int token = t.p_lo > 0 ? t.p_lo : 0, number = table[token / kPageTokens];
    const bool there = (unsigned)number < (unsigned)a.kv.num_pages;
    const uint8_t *block = a.kv.cache + ((int64_t)(there ? number : 0) * a.kv.kv_heads + t.h) * kv4_block_bytes(D, GS);
    // one address for all lanes: constant to the launch, so that a scalar load serves
    typedef const __attribute__((address_space(4))) float scalar_float;
    const scalar_float *v = (const scalar_float *)reinterpret_cast<const float *>(block + kv4_scale_offset(D)) +
                            D / GS * kPageTokens + token % kPageTokens;
    const bool taken = there && tile_has_first(a, t);
#pragma unroll
    for (int g = 0; g < D / GS; ++g)
        s[g] = taken ? v[g * kPageTokens] : 0.0f;
}

// Whether some column of the tile sees a token.
__device__ __forceinline__ bool tile_sees(const Kv4AttentionArgs &a, const Tile &t, int token)
{
    return token <= t.p_hi && (a.window == 0 || token > t.p_lo - a.window || token < a.sinks);
}

// Whether every one does.
__device__ __forceinline__ bool tile_shares(const Kv4AttentionArgs &a, const Tile &t, int token)
{
    return token <= t.p_lo && (a.window == 0 || token > t.p_hi - a.window || token < a.sinks);
}

// Where column `col` of a tile's result goes: 16-bit outputs, or one split's
// part of them.
__device__ __forceinline__ int64_t pair_of(const Kv4AttentionArgs &a, const Tile &t, int col)
{
    return (int64_t)(t.seq.row0 + col / t.G) * a.q_heads + t.h * t.G + col % t.G;
}
__device__ __forceinline__ uint16_t *output_of(const Kv4AttentionArgs &a, const Tile &t, int col)
{
    return a.y + (int64_t)(t.seq.row0 + col / t.G) * a.ldy + (int64_t)(t.h * t.G + col % t.G) * a.kv.head_dim;
}

__device__ __forceinline__ uint32_t pack_out(float a, float b, int dtype)
{
    return dtype == DT_BF16 ? pack2<OUT_BF16>(a, b) : pack2<OUT_F16>(a, b);
}

// The kernels, one launch each: tiles of 16 columns (few rows), of 128 or 256.
constexpr int kFewCols = 16;
hipError_t launch_kv4_few_rows(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream);
hipError_t launch_kv4_many_rows(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream);
// With shared prefixes: front_groups 0, or tiles 0, for one of the two alone.
hipError_t launch_kv4_few_rows_shared(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream);
hipError_t launch_kv4_many_rows_shared(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream);

}  // namespace cider
