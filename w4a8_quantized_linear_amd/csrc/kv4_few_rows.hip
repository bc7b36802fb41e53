// Causal attention over the 4-bit key/value cache (include/cider.h,
// cider_kv4_attention) for few rows per sequence: decoding steps and drafts.
//
// Mathematics.  For a row at position p and tokens t it sees,
//   S[t] = scale * sum_d q[d] s_k[t,g(d)] (u_k[t,d] - 8)
//   y[d] = sum_t e^(S[t] - m) s_v[t,g(d)] (u_v[t,d] - 8) / sum_t e^(S[t] - m)
// in one pass over the tokens with the running maximum m.  The codes u are
// never turned into values: a nibble put into the low bits of a half is the
// fp16 number u 2^-24 (the next nibble up: 16 u 2^-24, whose partner operand
// is divided by 16), exact in the matrix cores, which keep fp16 denormals and
// sum in fp32.  So one AND per two codes (and half a shift) makes an operand;
// the offset -8 enters as the score product's initial accumulator
// (-8 sum_d q[d] per group) and, for V, as one more matrix product whose left
// operand is the constant -8 2^-24; the scales multiply the fp32 scores and
// the softmax weights.
//
// Rounding.  q is scaled per row by a power of two to a largest magnitude in
// [2^13, 2^14) and held in fp16: exact unless an element is below 2^-23 of the
// row's largest, then off by at most 2^-34 of it (operands of the odd nibbles are
// stored divided by 16).  The weights e^(S - m) s_v are fp32 rounded once to fp16
// after scaling by a power of two that puts the largest s_v that the column has
// seen into [2^13, 2^14), of several rows into [2^11, 2^15): 11 significant bits down
// to 2^-27 (2^-25) of the largest possible weight, 2^-23 (2^-21) for the tokens of
// odd nibbles.  What the column does not see has no part in that power of two
// (ScaleExponents).  That error is as large as an fp16
// output's own rounding (and far below a bf16 one's), so for fp16 outputs the
// weights go in as two halves, hi + lo, 22 bits: twice the products of V and some
// operations a weight, which cost little where the cache's bytes bound the call and
// 6 % elsewhere (batch of 64 over up to 8192 tokens: 72.5 us without, 77.5 with),
// and take the error against 64 bits from 2.9e-4 to 2.0e-4, the output's rounding
// alone.  Scores, maxima, sums and outputs are fp32.
//
// Shape.  Columns are the 16 (row, query head) pairs c = r * G + g of one kv
// head, tokens the rows of S^T = K Q^T (v_mfma_f32_16x16x32_f16), so lane
// (j, c) ends with the scores of tokens 4 j + i of column c in its registers
// and they are, rounded and packed, the right operand of O^T += V^T P^T: no
// transpose, no LDS for either product.  A wavefront takes whole 64-token pages
// (every 4th or 8th of the workgroup's), loads the next page's codes as soon as
// it has used this one's, and the wavefronts' maxima, sums and outputs meet in
// LDS at the end.
//
// What bounds it.  A page's 8 to 10 KB feed 16 columns, so with enough pages
// the bytes do: 64 sequences of up to 8192 tokens (341 MB) in 70 us, 4.9 TB/s;
// one of 131072 (143 MB) in 28, 5.1; 256 of 4096 in 200, 6.1, the rate at
// which a plain reading kernel streams here.  A call of few pages is a chain of
// loads (lengths, page number, page: 0.8 us each) and the parts' meeting, 6.6 us
// for one sequence of 1001; with 2 to 3 tiles a head and pages in the caches
// (16 sequences of up to 3001, 35 columns: 13.7 us) the vector instructions of
// a page, 1.2 us for two wavefronts on a SIMD.
#include <type_traits>

#include "kv4_attention.h"

namespace cider {
namespace {

constexpr int kCols = kFewCols;

// Which columns a workgroup has.  One: every sequence has one row at most, so all
// columns see the same tokens and the exponents of V's scales are one for all of
// them.  Alike: of several rows, which have met scales of one exponent so far.  Apart:
// of several rows, each column with its own.
enum class Columns { One, Alike, Apart };

// With several rows the exponent of V's scales may lie kLag below a column's largest
// before it is moved: else one page in twenty that not all of a tile's rows see would
// move it for some of them alone.  (It starts of a token that all see: 16 x 5 rows with
// a window of 1000 11.9 us without, 8.5 with.)  kTop: scales go into the weights
// 2^(kTop - exponent) times as large, which stay below 2^15 (fp16 holds 2^16).
template <Columns KIND>
constexpr int kLag = KIND == Columns::One ? 0 : 3;
template <Columns KIND>
constexpr int kTop = KIND == Columns::One ? 14 : 12;

// Maximum and sum over the 4 lanes (j = 0 .. 3) of a column.
__device__ __forceinline__ float column_max(float v) { return max_lane32(max_lane16(v)); }
__device__ __forceinline__ float column_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// One page's codes as the lanes use them, and its scales: lane (j, n) holds
// those of token 16 (n / 4) + 4 j + n % 4, so each row of 16 lanes has the
// scales of its own 16 tokens and takes them by broadcast.  K and V are loaded
// apart: the next page's K as soon as the scores have used this one's, its V
// after the outputs have, so one page's registers serve and other wavefronts
// cover what is left of the latency.
template <int D, int GS>
struct PageData {
    uint32_t k[4][D / 32];
    uint4 v[2][D / 64];
    float ks[D / GS], vs[D / GS];
};

__device__ __forceinline__ int scale_token(int lane) { return 16 * (lane / 4 % 4) + 4 * (lane / 16) + lane % 4; }

// ONCE: a kv head's columns are one tile, so each page is read once, and the
// pages are more than half the 256 MB last-level cache: they go past the caches (batch of 64 over up to 8192 tokens 78.2 -> 72.5 us, 256 of
// 4096 215 -> 200, 6.1 TB/s; with 3 and more tiles it costs 3 - 12 %, as it does
// for a small cache that was read a moment ago, 64 sequences of 1024: 18.4 ->
// 20.3).
template <typename T, bool ONCE>
__device__ __forceinline__ T load_codes(const uint8_t *p)
{
    typedef uint32_t words __attribute__((ext_vector_type(sizeof(T) / 4)));
    const words *w = reinterpret_cast<const words *>(p);
    if constexpr (ONCE)
        return __builtin_bit_cast(T, __builtin_nontemporal_load(w));
    else
        return __builtin_bit_cast(T, *w);
}

template <int D, int GS, bool ONCE>
__device__ __forceinline__ void load_k(PageData<D, GS> &p, const uint8_t *block, int lane)
{
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const uint8_t *at = block + 16 * t * (D / 2);
        const uint32_t off = lane % 16 * (D / 2) + lane / 16 * (D / 8);
        if constexpr (D == 128) {
            const uint4 w = load_codes<uint4, ONCE>(at + off);
            p.k[t][0] = w.x;
            p.k[t][1] = w.y;
            p.k[t][2] = w.z;
            p.k[t][3] = w.w;
        } else {
            const uint2 w = load_codes<uint2, ONCE>(at + off);
            p.k[t][0] = w.x;
            p.k[t][1] = w.y;
        }
    }
    const float *s = reinterpret_cast<const float *>(block + kv4_scale_offset(D));
#pragma unroll
    for (int g = 0; g < D / GS; ++g)
        p.ks[g] = s[g * kPageTokens + (uint32_t)scale_token(lane)];
}

template <int D, int GS, bool ONCE>
__device__ __forceinline__ void load_v(PageData<D, GS> &p, const uint8_t *block, int lane)
{
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
            p.v[b][g] = load_codes<uint4, ONCE>(block + kv4_v_offset(D) + (b * (D / 64) + g) * 1024 + (uint32_t)lane * 16);
    const float *s = reinterpret_cast<const float *>(block + kv4_scale_offset(D));
#pragma unroll
    for (int g = 0; g < D / GS; ++g)
        p.vs[g] = s[(D / GS + g) * kPageTokens + (uint32_t)scale_token(lane)];
}

__device__ __forceinline__ half8 halves(uint32_t w) { return __builtin_bit_cast(half8, nibble_halves(w)); }

// Running state of a wavefront's columns.
template <int D, int GS>
struct State {
    f32x4 acc[D / 16], off[D / 64];
    float m, l;  // m in units of log2
    ScaleExponents exps[D / GS];  // of V's scales; where columns stand apart (not same) each has
    int *own;                     // its own, a group's 16 apart
    template <Columns KIND>
    __device__ __forceinline__ int exponent(int g) const
    {
        return KIND != Columns::Apart || exps[g].same ? exps[g].all : own[16 * g];
    }
    half8 q[D / 32];
    float zero[D / GS];
    float k_factor, q_factor;  // of the scores, to units of log2: on K's scales; the row's, a power of two
};

// Scores of a page, short of the row's factor: s[t][e] is token 16 t + 4 j + e of
// the lane's column.
template <int D, int GS>
__device__ __forceinline__ void page_scores(const State<D, GS> &st, const PageData<D, GS> &pg, float (&s)[4][4])
{
    constexpr int NG = D / GS;
    float ks[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g)
        ks[g] = pg.ks[g] * st.k_factor;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f32x4 r = {st.zero[g], st.zero[g], st.zero[g], st.zero[g]};
#pragma unroll
            for (int m = g * GS / 32; m < (g + 1) * GS / 32; ++m)
                r = __builtin_amdgcn_mfma_f32_16x16x32_f16(halves(pg.k[t][m]), st.q[m], r, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[t][e] = g == 0 ? scaled(r[e], ks[g], 4 * t + e)
                                 : __builtin_fmaf(row_value(ks[g], 4 * t + e), r[e], s[t][e]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // all 4 tiles' operands at once would not fit the registers
    }
}

__device__ __forceinline__ float largest(const float (&s)[4][4])
{
    float top = s[0][0];
#pragma unroll
    for (int n = 1; n < 16; ++n)
        top = __builtin_fmaxf(top, s[n / 4][n % 4]);
    return top;
}

// The outputs' products of tokens 32 B .. 32 B + 31 and elements 64 y .. 64 y + 63.
template <int D, int GS, int PARTS>
__device__ __forceinline__ void output_products(State<D, GS> &st, uint4 codes, int y, const uint32_t (&w)[PARTS][4])
{
    const half8 offset = __builtin_bit_cast(half8, uint4{kOffset, kOffset16, kOffset, kOffset16});
    half8 weights[PARTS];
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
        weights[i] = __builtin_bit_cast(half8, uint4{w[i][0], w[i][1], w[i][2], w[i][3]});
    const uint32_t u[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const half8 code = halves(u[x]);
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
            st.acc[4 * y + x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(code, weights[i], st.acc[4 * y + x], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
        st.off[y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(offset, weights[i], st.off[y], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
}

// Two weights rounded to fp16, as one part or as hi + lo.
template <int PARTS>
__device__ __forceinline__ void round_weights(float x, float y, int e, uint32_t (&w)[PARTS][4])
{
    if constexpr (PARTS == 2)  // kept from being computed twice, by the subtraction below too
        asm("" : "+v"(x), "+v"(y));
    w[0][e] = pack2<OUT_F16>(x, y);
    if constexpr (PARTS == 2) {
        const half2_t hi = __builtin_bit_cast(half2_t, w[0][e]);
        w[1][e] = pack2<OUT_F16>(x - (float)hi.x, y - (float)hi.y);
    }
}

// Their weights, and the outputs.  top: the largest score; seen: bit 4 t + e
// set where the lane's column sees the token (read where the page is not whole);
// whole: every column sees every token; held, common: some column of the tile,
// or every one, sees the token of the lane's scales; valid: the lane has a column.
// False, and the state is spoilt, where columns that were alike no longer are.
template <int D, int GS, bool FINE, Columns KIND>
__device__ __forceinline__ bool page_outputs(State<D, GS> &st, const PageData<D, GS> &pg, int lane,
                                             float (&s)[4][4], float top, bool whole, uint32_t seen,
                                             bool held, bool common, bool valid)
{
    constexpr int NG = D / GS, NT = D / 16, PARTS = FINE ? 2 : 1, LAG = kLag<KIND>;
    const float inf = __builtin_inff();
    // V's scales; the columns' exponents move up first
    float vs[NG];
    bool above = false, alike = true, apart = false;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        vs[g] = held ? pg.vs[g] : 0.0f;
        above |= vs[g] >= ldexp_f(1.0f, st.exps[g].reach + LAG) && vs[g] < inf;
    }
    if (__any(above)) {
        uint32_t e = 0;  // exponents of the lane's token, a half each
#pragma unroll
        for (int g = 0; g < NG; ++g)
            e |= (uint32_t)(scale_exponent(vs[g]) + kExpBias) << 16 * g;
        auto largest = [](uint32_t u) {
            return (uint32_t)__builtin_amdgcn_readfirstlane(max_halves_lane32(max_halves_lane16(max_halves_row(u))));
        };
        const uint32_t most = largest(e);
        const uint32_t all = KIND == Columns::One || whole ? most : largest(common ? e : 0u);
        auto rescale = [&](int g, float f) {
#pragma unroll
            for (int x = g * GS / 16; x < (g + 1) * GS / 16; ++x)
                st.acc[x] *= f;
#pragma unroll
            for (int y = g * GS / 64; y < (g + 1) * GS / 64; ++y)
                st.off[y] *= f;
        };
        // up to the largest that every column sees
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int top = half_exponent(all, g), was = st.exps[g].all;
            if (KIND == Columns::Apart && !st.exps[g].same) {
                alike = false;
            } else {
                const int now = top > was + LAG ? top : was;
                rescale(g, ldexp_f(1.0f, was - now));
                st.exps[g].set(now);
                alike &= half_exponent(most, g) <= now + LAG;
            }
        }
        if (KIND == Columns::Apart && !alike) {  // then to what each does
            const uint32_t own = max_halves_lane32(max_halves_lane16(seen_largest({e}, seen, lane)));
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int top = half_exponent(all, g), e = half_exponent(own, g), was = st.template exponent<KIND>(g);
                const int next = top > was + LAG ? top : was;
                const int then = st.exps[g].template raise<16>(was, e > next + LAG ? e : next, valid);
                st.own[16 * g] = then;
                rescale(g, ldexp_f(1.0f, was - then));
            }
        }
    }
    // the 16 times larger codes belong to tokens 1 and 3 of each 4
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        vs[g] = ldexp_f(vs[g], kTop<KIND> - st.exps[g].all - (lane & 1 ? 4 : 0));
        apart |= KIND == Columns::Apart && !st.exps[g].same;
    }
    const float m_new = __builtin_fmaxf(st.m, column_max(top) * st.q_factor);
    const float m_sub = m_new == -inf ? 0.0f : m_new;
    if (__any(m_new > st.m)) {
        const float f = __builtin_amdgcn_exp2f(st.m - m_sub);
        st.l *= f;
#pragma unroll
        for (int x = 0; x < NT; ++x)
            st.acc[x] *= f;
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
            st.off[g] *= f;
        st.m = m_new;
    }
#pragma unroll
    for (int n = 0; n < 16; ++n) {
        float &x = s[n / 4][n % 4];
        x = __builtin_amdgcn_exp2f(__builtin_fmaf(x, st.q_factor, -m_sub));
        st.l += x;
    }
    uint32_t w[NG][2][PARTS][4];
    auto weigh = [&](auto is_apart) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int by = is_apart() ? scale_shift(st.exps[g].all, st.template exponent<KIND>(g)) : 0;
#pragma unroll
            for (int B = 0; B < 2; ++B)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = s[2 * B][e], y = s[2 * B + 1][e];
                    if constexpr (is_apart()) {
                        x = ldexp_f(x, by);
                        y = ldexp_f(y, by);
                    }
                    round_weights<PARTS>(scaled(x, vs[g], 8 * B + e), scaled(y, vs[g], 8 * B + 4 + e), e, w[g][B]);
                }
        }
    };
    if (apart)
        weigh(std::true_type{});
    else
        weigh(std::false_type{});
    // a hidden token's weight is 0, and times a scale that is not finite it would
    // not stay so
    bool odd = false;
#pragma unroll
    for (int g = 0; g < NG; ++g)
        odd |= !(__builtin_fabsf(vs[g]) < inf);
    if (!whole && __any(odd)) {
#pragma unroll
        for (int B = 0; B < 2; ++B)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t keep = ((seen >> (8 * B + e)) & 1u ? 0xFFFFu : 0u) |
                                      ((seen >> (8 * B + 4 + e)) & 1u ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int i = 0; i < PARTS; ++i)
                        w[g][B][i][e] &= keep;
            }
    }
#pragma unroll
    for (int B = 0; B < 2; ++B)
#pragma unroll
        for (int y = 0; y < D / 64; ++y)
            output_products<D, GS, PARTS>(st, pg.v[B][y], y, w[y * 64 / GS][B]);
    return KIND != Columns::Alike || alike;
}

// A wavefront's pages, every WAVES-th of begin .. end - 1 from its own number on, and
// its part of the outputs (element stride 1, columns D + 4 apart), maxima and sums.
// False where columns that were alike no longer are: nothing is written then.
template <int D, int GS, int WAVES, bool FINE, bool ONCE, Columns KIND>
__device__ __forceinline__ bool wave_pages(const Kv4AttentionArgs &a, const Kv4Launch &n, const Tile &t, int b, int begin,
                                           int end, int wave, const int lane, int *own, float (*part)[D + 4],
                                           float *part_m, float *part_l)
{
    constexpr int NM = D / 32;   // score products per 16 tokens
    constexpr int NG = D / GS;   // scales per token
    constexpr int NT = D / 16;   // output tiles
    constexpr bool LATE = KIND == Columns::Apart;  // K's next page: registers first
    const int c = lane % 16, j = lane / 16;
    const int col = t.tile * kCols + c;
    const bool valid = col < t.cols;
    const int row = valid ? col / t.G : 0;
    const int p = valid ? t.seq.kv - t.seq.n + row : -1;

    // q is asked for first and used last: the first page's codes are on their
    // way while it is scaled
    uint4 qw[NM];
    {
        const uint16_t *q = a.q + (int64_t)(t.seq.row0 + row) * a.ldq +
                            (int64_t)(t.h * t.G + (valid ? col % t.G : 0)) * D + 8 * j;
#pragma unroll
        for (int m = 0; m < NM; ++m)
            qw[m] = *reinterpret_cast<const uint4 *>(q + 32 * m);
    }
    const int32_t *table = a.kv.pages + (int64_t)b * a.kv.max_pages;
    const uint8_t *heads = a.kv.cache + (int64_t)t.h * kv4_block_bytes(D, GS);
    const int64_t page_bytes = (int64_t)a.kv.kv_heads * kv4_block_bytes(D, GS);
    // a page number outside the cache is never followed: page 0 is loaded in
    // its place and its tokens are left out
    auto block_of = [&](int number) {
        return heads + ((unsigned)number < (unsigned)a.kv.num_pages ? number : 0) * page_bytes;
    };
    // page numbers are read two pages ahead
    PageData<D, GS> pg;
    int i = begin + wave, n0 = -1, n1 = -1;
    float first[NG] = {};
    if (i < end) {
        n0 = table[t.range.at(i)];
        if constexpr (KIND != Columns::One)
            first_scales<D, GS>(a, t, table, first);
        load_k<D, GS, ONCE>(pg, block_of(n0), lane);
        load_v<D, GS, ONCE>(pg, block_of(n0), lane);
    }
    if (i + WAVES < end)
        n1 = table[t.range.at(i + WAVES)];

    State<D, GS> st;
    st.own = own + c;
    {
#pragma unroll
        for (int m = 0; m < NM; ++m)
            qw[m] = valid ? qw[m] : uint4{0, 0, 0, 0};
        const float top = column_max(query_top(qw, a.q_dtype));
        const int shift = 14 - __builtin_amdgcn_frexp_expf(top);
        // the row's factor is a power of two, exact: with a rounded product the maximum
        // of large scores would lie below one of them by more than fp32's exponents.
        // 2^12 of the operands' 2^24 go to K's scales, which keeps it a number for any q
        st.k_factor = ldexp_f(a.scale * kLog2e, 12);
        st.q_factor = ldexp_f(1.0f, 12 - shift);
        query_operands(qw, a.q_dtype, shift, st.q);
#pragma unroll
        for (int g = 0; g < NG; ++g)
            st.zero[g] = 0.0f;
#pragma unroll
        for (int m = 0; m < NM; ++m)
            st.zero[m * 32 / GS] = operand_sum(st.q[m], st.zero[m * 32 / GS]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            st.zero[g] = column_sum(st.zero[g]) * -0x1p-21f;
            const int e = __builtin_amdgcn_readfirstlane(scale_exponent(first[g]));
            st.exps[g].set(KIND == Columns::One ? kNoScale : e);
        }
#pragma unroll
        for (int x = 0; x < NT; ++x)
            st.acc[x] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
            st.off[g] = f32x4{0, 0, 0, 0};
        st.m = -__builtin_inff();
        st.l = 0.0f;
    }

    bool alike = true;
    for (; alike && i < end; i += WAVES) {
        int n2 = -1;
        if (i + 2 * WAVES < end)
            n2 = table[t.range.at(i + 2 * WAVES)];
        // past the last page this one is loaded again (from the caches): a load
        // under a branch would cost its registers twice
        const uint8_t *ahead = block_of(i + WAVES < end ? n1 : n0);
        const bool there = (unsigned)n0 < (unsigned)a.kv.num_pages;
        const int t0 = t.range.at(i) * kPageTokens;
        const bool whole = there && t0 + kPageTokens - 1 <= t.p_lo &&
                           (a.window == 0 || t0 > t.p_hi - a.window || t0 + kPageTokens <= a.sinks);
        float s[4][4];
        page_scores<D, GS>(st, pg, s);
        if constexpr (!LATE)
            load_k<D, GS, ONCE>(pg, ahead, lane);
        uint32_t seen = 0xFFFFu;
        float top = largest(s);
        if (!whole) {
            seen = there ? tokens_seen<16>(p, t0 + 4 * j, a.window, a.sinks) : 0u;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                s[e / 4][e % 4] = seen_score(s[e / 4][e % 4], seen, e);
            top = largest(s);
        }
        const bool held = whole || (there && tile_sees(a, t, t0 + scale_token(lane)));
        const bool common = whole || tile_shares(a, t, t0 + scale_token(lane));
        alike = page_outputs<D, GS, FINE, KIND>(st, pg, lane, s, top, whole, seen, held, common, valid && p >= 0);
        if constexpr (LATE)
            load_k<D, GS, ONCE>(pg, ahead, lane);
        load_v<D, GS, ONCE>(pg, ahead, lane);
        n0 = n1;
        n1 = n2;
    }

    if (KIND == Columns::Alike && !alike)
        return false;
    // lane (j, c) holds elements 16 x + 4 j .. + 3 of column c
    st.l = column_sum(st.l);
    const int less = sum_bits(n.splits > 1 ? n.pages : t.range.count);
#pragma unroll
    for (int x = 0; x < NT; ++x)
        *reinterpret_cast<f32x4 *>(&part[c][16 * x + 4 * j]) =
            ldexp_f(st.acc[x] + st.off[x / 4], st.template exponent<KIND>(x * 16 / GS) + 24 - kTop<KIND> - less);
    if (j == 0) {
        part_m[c] = st.m;
        part_l[c] = st.l;
    }
    return true;
}

// ONE: one row a sequence at most.  Of several rows a wavefront whose columns no longer
// are alike (a page that only some of them see has far larger values than all before
// it) begins again with a copy of its loop that keeps them apart: what that takes stays
// out of the way of the others (512 rows of a prompt 17.9 us, 19.6 with both in one
// loop; a batch of 64 over up to 8192 tokens, one row each, 71 and 98).  Pages read
// past the caches want the registers of 2 wavefronts a SIMD rather than a third
// (64 x 2 rows over 4000 tokens 56.0 us, 57.6 with 3), others the third.
template <int D, int GS, int WAVES, bool FINE, bool ONCE, bool ONE>
__global__ __launch_bounds__(64 * WAVES, WAVES > 4 ? WAVES / 4 : (ONE || !ONCE ? 3 : 2)) void kv4_few_rows_kernel(Kv4AttentionArgs a, Kv4Launch n)
{
    __shared__ __align__(16) float part[WAVES][kCols][D + 4];
    __shared__ float part_m[WAVES][kCols], part_l[WAVES][kCols];
    __shared__ int own[ONE ? 1 : WAVES][D / GS][kCols];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // heads fastest, then sequences, splits and tiles
    unsigned id = kv4_workgroup();
    const int head = (int)(id % (unsigned)a.kv.kv_heads);
    id /= (unsigned)a.kv.kv_heads;
    const int b = (int)(id % (unsigned)a.kv.batch);
    id /= (unsigned)a.kv.batch;
    const int split = (int)(id % (unsigned)n.splits), tile = (int)(id / (unsigned)n.splits);
    Tile t;
    if (!tile_of<kCols>(a, b, head, tile, t))
        return;
    const int begin = n.splits > 1 ? split * n.pages : 0;
    if (split > 0 && begin >= t.range.count)
        return;
    const int end = n.splits > 1 && begin + n.pages < t.range.count ? begin + n.pages : t.range.count;

    int lane = threadIdx.x & 63;
    if constexpr (ONE) {
        wave_pages<D, GS, WAVES, FINE, ONCE, Columns::One>(a, n, t, b, begin, end, wave, lane, nullptr, part[wave], part_m[wave],
                                                           part_l[wave]);
    } else if (!wave_pages<D, GS, WAVES, FINE, ONCE, Columns::Alike>(a, n, t, b, begin, end, wave, lane, nullptr, part[wave],
                                                                     part_m[wave], part_l[wave])) {
        asm volatile("" : "+v"(lane));  // nothing of the first way kept
        wave_pages<D, GS, WAVES, FINE, ONCE, Columns::Apart>(a, n, t, b, begin, end, wave, lane, own[wave][0], part[wave],
                                                             part_m[wave], part_l[wave]);
    }
    __syncthreads();
    constexpr int PER = kCols * D / (64 * WAVES);  // elements per thread
    const int oc = threadIdx.x / (D / PER), d0 = threadIdx.x % (D / PER) * PER;
    const int ocol = t.tile * kCols + oc;
    if (ocol >= t.cols)
        return;
    float m = -__builtin_inff(), l = 0.0f, o[PER] = {};
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        m = __builtin_fmaxf(m, part_m[w][oc]);
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        if (part_l[w][oc] == 0.0f)  // saw nothing
            continue;
        const float f = __builtin_amdgcn_exp2f(part_m[w][oc] - m);
        l += part_l[w][oc] * f;
#pragma unroll
        for (int e = 0; e < PER; ++e)
            o[e] += part[w][oc][d0 + e] * f;
    }
    if (n.splits > 1 && t.range.count > n.pages) {
        const int64_t at = pair_of(a, t, ocol) * n.splits + split;
#pragma unroll
        for (int e = 0; e < PER; ++e)
            n.part[at * D + d0 + e] = o[e];
        if (d0 == 0) {
            n.part_stat[2 * at] = m;
            n.part_stat[2 * at + 1] = l;
        }
        return;
    }
    const float inv = ldexp_f(reciprocal(l), sum_bits(n.splits > 1 ? n.pages : t.range.count));
    uint32_t w[PER / 2];
#pragma unroll
    for (int e = 0; e < PER; e += 2)
        w[e / 2] = pack_out(o[e] * inv, o[e + 1] * inv, a.y_dtype);
    uint16_t *y = output_of(a, t, ocol) + d0;
    if constexpr (PER == 8)
        *reinterpret_cast<uint4 *>(y) = uint4{w[0], w[1], w[2], w[3]};
    else if constexpr (PER == 4)
        *reinterpret_cast<uint2 *>(y) = uint2{w[0], w[1]};
    else
        *reinterpret_cast<uint32_t *>(y) = w[0];
}

}  // namespace

template <int WAVES, bool FINE, bool ONCE, bool ONE>
static hipError_t launch(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    const unsigned grid = (unsigned)n.tiles * (unsigned)n.splits * (unsigned)a.kv.kv_heads *
                          (unsigned)a.kv.batch;
    if (a.kv.head_dim == 64)
        return kv4_launch(kv4_few_rows_kernel<64, 64, WAVES, FINE, ONCE, ONE>, grid, 64 * WAVES, stream, a, n);
    if (a.kv.group_size == 64)
        return kv4_launch(kv4_few_rows_kernel<128, 64, WAVES, FINE, ONCE, ONE>, grid, 64 * WAVES, stream, a, n);
    return kv4_launch(kv4_few_rows_kernel<128, 128, WAVES, FINE, ONCE, ONE>, grid, 64 * WAVES, stream, a, n);
}

template <int WAVES, bool FINE, bool ONCE>
static hipError_t launch(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    return a.kv.max_rows == 1 ? launch<WAVES, FINE, ONCE, true>(a, n, stream) : launch<WAVES, FINE, ONCE, false>(a, n, stream);
}

template <int WAVES>
static hipError_t launch(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    if (a.y_dtype == DT_F16)
        return n.once ? launch<WAVES, true, true>(a, n, stream) : launch<WAVES, true, false>(a, n, stream);
    return n.once ? launch<WAVES, false, true>(a, n, stream) : launch<WAVES, false, false>(a, n, stream);
}

hipError_t launch_kv4_few_rows(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    return n.waves == 8 ? launch<8>(a, n, stream) : launch<4>(a, n, stream);
}

}  // namespace cider
