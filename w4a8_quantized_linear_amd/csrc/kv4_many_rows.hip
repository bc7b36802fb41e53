// Causal attention over the 4-bit key/value cache (include/cider.h,
// cider_kv4_attention) for many rows per sequence: prompts and chunks of them.
//
// The mathematics is that of kv4_few_rows.hip.  Here every page serves many
// columns, so what counts is vector work per (column, token): a workgroup of 4
// or 8 wavefronts (128 or 256 columns) shares each page's unpacking.  A thread
// turns its share of the codes into fp16 operands (u - 8) 2^-24 (the odd
// nibbles 16 times as large, their partners divided by 16; exact) and writes
// them to LDS in the order in which the matrix instructions take them; a
// wavefront has 32 columns and computes
//   S^T = K Q^T  and  O^T += V^T P^T   (v_mfma_f32_32x32x16_f16)
// reading 1 KB fragments that are consecutive over the lanes.  Lane (h, c)
// holds the scores of tokens 8 i + 4 h .. + 3 of column c, which V's code
// order makes the right operand's own tokens, so the weights go from the
// softmax to the second product in registers.
//
// Two LDS buffers each for K and V, one barrier a page: while the weights of
// page i are worked out the scores of page i + 1 are multiplied, and between
// the products of page i's outputs those scores are scaled and K of page i + 2
// and V of page i + 1, loaded at the step's start, are unpacked.
//
// Rounding.  q is scaled by a power of two and held in fp16: exact unless an element
// is below 2^-17 of its row's largest, then off by at most 2^-28 of it.  One power
// for the whole tile (its largest magnitude to [2^13, 2^14)), so that the scores'
// factor goes into K's scales once a page, where all rows are within kReach bits of
// one another; else each row's own, which meets the products' sums.  The weights are
// rounded once to fp16, 11 significant bits down to 2^-25 of the largest, 2^-21 for
// the tokens of odd nibbles, by an exponent that only tokens the column sees have a
// part in: the error against 64 bits is 2.9e-4 with fp16 outputs, 2.1e-4 of it the
// output's rounding.  (Two halves, as for few rows, would double the second product,
// which is not hidden here.)
//
// What bounds it: the vector units.  A wavefront takes about 365 vector
// instructions a page (D 128 in groups of 64), which cost 4.4 cycles of its SIMD
// each (8.3 an exponential) while products run, 1730 in all, next to 32 products of
// 32 cycles: two wavefronts of a SIMD, 240 pages each on average, 830 thousand
// cycles or about 390 us for 2048 rows over 16384 tokens.  Counters for that call:
// of a wavefront's life the vector units work 65 %, the matrix cores 38 %, either
// 80 %; the rest is the page's barrier and results waited for.  So the work was
// moved, not only cut: scaling under the outputs' products, loads and unpacking
// between products, exponentials a step early (a tenth of the call with the 256
// columns).
// Measured: 2048 rows over 16384 tokens 603 us, 855 TFLOP/s (groups of 128: 539,
// 956); 4 ragged prompts of up to 4096 rows, groups of 128, 231 us, 776; 8000
// rows with a window of 1024 217 us, 581 (18 pages a tile do not hide a tile's
// beginning and end, 9 us of 60).
#include "kv4_attention.h"

namespace cider {
namespace {

constexpr int kWaveCols = 32;  // one matrix operand
constexpr uint32_t kRsrcWord3 = 0x00020000;  // raw 32-bit buffer

// The running maximum may lie kSlack (in units of log2) below the true one before
// it is moved, and the exponent of V's scales kLag: the outputs are rescaled in few
// pages instead of nearly all (with 32 columns some column has a new maximum in
// most pages).  A column's moves are its own, whatever its neighbours see.  kTop
// leaves fp16 the room: weights times V's scale stay below 2^(kTop + kSlack + kLag),
// 61147.  (A kLag of 2 sends a batch's first tiles, whose columns share few tokens, the
// long way: 8 prompts of 64 rows 20.1 us, 11.1 with 3.)
constexpr float kSlack = 1.9f;
constexpr int kLag = 3;
constexpr int kTop = 11;
constexpr int kReach = 7;
constexpr int kLeastExp = -126;  // of scales that are not normal numbers

// One page's K and V in LDS.  They are used one step apart (the scores of page
// i + 1 are computed while page i's weights are), so each has its own pair of
// buffers.
template <int D, int GS>
struct PageK {
    uint4 code[2][D / 16][64];  // [32-token tile][16-element step][lane]
    float scale[kPageTokens];   // of the scores, to units of log2: the last group's times k_factor
    float ratio[kPageTokens];   // groups of 64 in 128: the first group's scale over the last one's
};  // scales stand at scale_slot(token)
template <int D, int GS>
struct PageV {
    uint4 code[2][2][D / 32][64];     // [32-token tile][16-token step][32-element tile][lane]
    float scale[D / GS][kPageTokens];
    int exp[D / GS];                  // V's scales are 2^(kTop - exp) times as large
    int base[D / GS];                 // the exponent that tokens of all columns have led to
};

// Scales by token.  Lane (h, c) needs those of the 16 tokens 8 i + 4 h + f of a
// tile; each row of 16 lanes holds them one a lane, and the multiplications
// take them by a broadcast within the row (DPP), so a tile's scales cost one
// 4-byte LDS read instead of four 16-byte ones.
__device__ __forceinline__ int scale_slot(int t) { return t / 32 * 32 + t / 4 % 2 * 16 + t / 8 % 4 * 4 + t % 4; }
// A thread's share of a page on its way: ND dwords of K and of V.
template <int ND>
struct Share {
    uint32_t k[ND], v[ND];
    float k_scale[2], v_scale;  // by token: wavefront 0 K's groups, wavefront 1 + g V's group g
};

// Loads of a block go through a buffer descriptor made from its address: one
// offset register for all pages and no vector arithmetic for a page's address.
template <int N>
__device__ __forceinline__ void load_dwords(uint32_t (&w)[N], __amdgpu_buffer_rsrc_t block, uint32_t off, uint32_t base)
{
    if constexpr (N == 4) {
        const uint4 x = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(block, off, base, 0));
        w[0] = x.x;
        w[1] = x.y;
        w[2] = x.z;
        w[3] = x.w;
    } else if constexpr (N == 1) {
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_raw_buffer_load_b32(block, off, base, 0));
    } else {
        const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(block, off, base, 0));
        w[0] = x.x;
        w[1] = x.y;
    }
}

// (u - 8) 2^-24 of 8 nibbles, the odd ones 16 times as large.
__device__ __forceinline__ uint4 code_halves(uint32_t w)
{
    const uint4 u = nibble_halves(w);
    const half2_t one = __builtin_bit_cast(half2_t, kOffset), sixteen = __builtin_bit_cast(half2_t, kOffset16);
    return uint4{__builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, u.x) + one),
                 __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, u.y) + sixteen),
                 __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, u.z) + one),
                 __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, u.w) + sixteen)};
}

__device__ __forceinline__ f32x16 mfma(uint4 x, half8 y, f32x16 z)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, x), y, z, 0, 0, 0);
}

template <int D, int GS, int COLS>
struct Lds {
    PageK<D, GS> page_k[2];
    PageV<D, GS> page_v[2];
    float tile_top[COLS / kWaveCols], tile_low[COLS / kWaveCols];  // of the rows' largest magnitudes
    int own[D / GS][COLS];  // where columns stand apart: the exponents of V's scales
    int stand_apart[2];     // by a page's number: some wavefront's columns do
};

// One tile's share of pages.  Its rows' queries are of about one size, V's scales
// are taken to the exponent that tokens of all its columns have led to, and the powers
// of two of both are staged with the page's scales.  Where that is not enough (tokens
// that only some columns see have scales 2^kLag times larger, rows 2^kReach apart) the
// columns stand apart: every score takes its row's factor and every weight its
// column's difference, 32 instructions a group and page more.  APART does that.
// Without it the workgroup, all wavefronts together, leaves off there and returns
// false.
template <int D, int GS, int COLS, Pages PAGES, bool APART>
__device__ __forceinline__ bool many_rows_tile(const Kv4AttentionArgs &a, const Kv4Launch &n, Lds<D, GS, COLS> &lds,
                                               const Tile &t, int split, int begin, int end, const int tid)
{
    constexpr int NG = D / GS;   // scales per token
    constexpr int NK = D / 16;   // score products per 32 tokens
    constexpr int NT = D / 32;   // output tiles
    constexpr int WAVES = COLS / kWaveCols, TEAMS = WAVES / 4;
    constexpr int ND = D / 32 / TEAMS;  // dwords of K and of V that a thread unpacks
    static_assert(TEAMS == 1 || TEAMS == 2, "teams of 256 threads take a page's code runs");
    PageK<D, GS>(&page_k)[2] = lds.page_k;
    PageV<D, GS>(&page_v)[2] = lds.page_v;

    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane % 32, h = lane / 32;
    const float inf = __builtin_inff();
    const int col0 = t.tile * COLS + wave * kWaveCols;
    const int col = col0 + c;
    const bool valid = col < t.cols;
    const int row = valid ? col / t.G : 0;
    const int p = valid ? position_of<PAGES>(t, row) : -1;
    // positions of the wavefront's columns (hi below lo: it has none)
    const int w_lo = position_of<PAGES>(t, col0 / t.G);
    const int w_last = col0 + kWaveCols <= t.cols ? col0 + kWaveCols - 1 : t.cols - 1;
    const int w_hi = col0 < t.cols ? position_of<PAGES>(t, w_last / t.G) : -1;

    // q is asked for first and used last: the first pages' codes are on their
    // way while it is scaled
    uint4 qw[NK];
    {
        const uint16_t *at = a.q + (int64_t)(t.seq.row0 + row) * a.ldq +
                             (int64_t)(t.h * t.G + (valid ? col % t.G : 0)) * D + 8 * h;
#pragma unroll
        for (int k = 0; k < NK; ++k)
            qw[k] = *reinterpret_cast<const uint4 *>(at + 16 * k);
    }
    const int32_t *table = a.kv.pages + (int64_t)t.b * a.kv.max_pages;
    const uint8_t *heads = a.kv.cache + (int64_t)t.h * kv4_block_bytes(D, GS);
    const uint32_t page_bytes = (uint32_t)a.kv.kv_heads * kv4_block_bytes(D, GS);
    // a page number outside the cache is never followed: page 0 is loaded in
    // its place and its tokens are left out
    auto block_of = [&](int number) {
        const uint32_t in = (unsigned)number < (unsigned)a.kv.num_pages ? (uint32_t)number : 0u;
        return __builtin_amdgcn_make_buffer_rsrc((void *)(heads + (uint64_t)in * page_bytes), (short)0,
                                                 kv4_block_bytes(D, GS), kRsrcWord3);
    };
    const uint32_t code_off = tid % 256 * (D / 8) + tid / 256 * 4 * ND, scale_off = lane * 4;
    auto fetch_k = [&](Share<ND> &s, __amdgpu_buffer_rsrc_t block) {
        load_dwords(s.k, block, code_off, 0);
#pragma unroll
        for (int g = 0; g < NG; ++g)
            s.k_scale[g] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                block, scale_off, kv4_scale_offset(D) + 4 * kPageTokens * g, 0));
    };
    auto fetch_v = [&](Share<ND> &s, __amdgpu_buffer_rsrc_t block) {
        load_dwords(s.v, block, code_off, kv4_v_offset(D));
        s.v_scale = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
            block, scale_off, kv4_scale_offset(D) + 4 * kPageTokens * (NG + (wave == 2 && NG == 2 ? 1 : 0)), 0));
    };
    // page numbers: of page i + 1 (V) and i + 2 (K); read one step ahead
    Share<ND> share, share1;
    const int last_page = end - 1;
    auto number_of = [&](int i) { return table[(uint32_t)t.range.at_turned(i < last_page ? i : last_page)]; };
    f32x16 r[2];
    int n0 = -1, n1 = -1, n2 = -1;
    if (begin < end) {
        n0 = number_of(begin);
        n1 = number_of(begin + 1);
        n2 = number_of(begin + 2);
        fetch_k(share, block_of(n0));
        fetch_v(share, block_of(n0));
        fetch_k(share1, block_of(n1));
    }
    __amdgpu_buffer_rsrc_t v_block = block_of(n1);  // of page i + 1

    half8 q[NK];
    float k_factor, q_factor = 1.0f;  // of the scores, to units of log2: on K's scales, on the row
    {
#pragma unroll
        for (int k = 0; k < NK; ++k)
            qw[k] = p >= 0 ? qw[k] : uint4{0, 0, 0, 0};
        float top = max_lane32(query_top(qw, a.q_dtype));
        if constexpr (APART) {
            k_factor = ldexp_f(a.scale * kLog2e, 12);
            const int shift = 14 - __builtin_amdgcn_frexp_expf(top);
            q_factor = ldexp_f(1.0f, 12 - shift);
            query_operands(qw, a.q_dtype, shift, q);
        } else {
            float low = -wave_max(top == 0.0f ? -inf : -top);
            top = wave_max(top);
            if (lane == 0) {
                lds.tile_top[wave] = top;
                lds.tile_low[wave] = low;
            }
            if (tid < 2)
                lds.stand_apart[tid] = 0;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                top = __builtin_fmaxf(top, lds.tile_top[w]);
                low = __builtin_fminf(low, lds.tile_low[w]);
            }
            const int e = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(top));
            if (low < ldexp_f(1.0f, e - kReach) || e > 64)
                return false;
            const int shift = 14 - e;
            k_factor = ldexp_f(a.scale * kLog2e, 24 - shift);
            query_operands(qw, a.q_dtype, shift, q);
        }
    }

    f32x16 acc[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x)
        acc[x] = f32x16{};
    float m_run = -inf, l_run = 0.0f;
    int v_exp[NG];             // of the outputs so far,
    ScaleExponents exps[NG];   // where columns stand apart these and lds.own
    const int own_at = wave * kWaveCols + c;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if constexpr (APART) {
            exps[g].set(kNoScale);
            lds.own[g][own_at] = kNoScale;
        } else {
            v_exp[g] = kLeastExp;
        }
    }
    // of the wavefront that writes V's scales: 2^(v_exp_run + kLag) is above those that
    // every column of the tile saw so far, up to 2^kMostStaged, past which small ones
    // would not stay normal numbers
    constexpr int kMostStaged = 60, kPast = 4096;  // added where some column sees larger ones
    int v_exp_run = kLeastExp;
    if (wave >= 1 && wave <= NG && begin < end) {
        float first[NG];
        first_scales<D, GS>(a, t, table, first);
        const float v = first[NG == 2 ? wave - 1 : 0];
        const int e = (__builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v > 0.0f && v < inf ? v : 0.0f)) >> 23) + kLeastExp;
        v_exp_run = e < kMostStaged ? e : kMostStaged;
    }

    // where a thread's operands go, and where a lane finds its own: K's slots
    // are exchanged by j so that the 8 lanes of one write cycle (2 tokens, 4 j)
    // hit different banks
    const int slot = 16 * h + lane % 16;  // of the lane's own scale in a tile's
    const int kt = tid % 256 / 4, kj = tid % 4, km = tid / 256 * ND;
    const int k_to = ((kj % 2) * 32 + kt % 32) ^ (2 * kj);
    const int k_from[2] = {lane ^ (2 * h), lane ^ (4 + 2 * h)};
    const int unit = D == 128 ? tid % 256 : tid % 256 / 2;
    const int vx = (D == 128 ? 0 : 2 * (tid % 2)) + tid / 256 * ND;
    const int vc = unit % 16, vj = unit / 16 % 4, vg = unit / 64 % (D / 64), vb = unit / (64 * (D / 64));
    auto stage_k_dword = [&](PageK<D, GS> &to, const Share<ND> &s, int m) {
        to.code[kt / 32][2 * (km + m) + kj / 2][k_to] = code_halves(s.k[m]);
    };
    auto stage_k_scales = [&](PageK<D, GS> &to, const Share<ND> &s) {
        if (wave != 0)
            return;
        if (NG == 1) {
            to.scale[scale_slot(lane)] = key_factor(s.k_scale[0], k_factor);
        } else {
            // s[0] r0 + s[1] r1 as (s[0] / s[1] r0 + r1) s[1], the first product done on
            // the way; s[1] is kept off 0 (its codes then stand for 0) and the ratio under
            // 2^120, which r0, below 2, leaves finite
            const float low = __builtin_fmaxf(s.k_scale[0] * (s.k_scale[1] == 0.0f ? 0x1p-60f : 0x1p-120f), 0x1p-149f);
            const float last = s.k_scale[1] < low ? low : s.k_scale[1];  // NaN stays
            to.scale[scale_slot(lane)] = key_factor(last, k_factor);
            // (a division without its last bits: 2^-22)
            const float rest = __builtin_amdgcn_rcpf(__builtin_amdgcn_frexp_mantf(last));
            to.ratio[scale_slot(lane)] = ldexp_f(s.k_scale[0] * rest, -__builtin_amdgcn_frexp_expf(last));
        }
    };
    auto stage_v_dword = [&](PageV<D, GS> &to, const Share<ND> &s, int e) {
        const int x = vx + e;
        to.code[vb][vj / 2][2 * vg + x / 2][(vj % 2) * 32 + 16 * (x % 2) + vc] = code_halves(s.v[e]);
    };
    // the first tokens in some column's window, and in every one's
    const int held_from = a.window > 0 ? t.p_lo - a.window + 1 : 0;
    const int shared_from = a.window > 0 ? t.p_hi - a.window + 1 : 0;
    // number, t0: the page's
    auto stage_v_scales = [&](PageV<D, GS> &to, const Share<ND> &s, int number, int t0) {
        if (wave >= 1 && wave <= NG) {
            const int token = t0 + lane;
            const bool held = (unsigned)number < (unsigned)a.kv.num_pages && token <= t.p_hi &&
                              (token >= held_from || token < a.sinks);
            const bool shared = token <= t.p_lo && (token >= shared_from || token < a.sinks);
            const float v = held ? s.v_scale : 0.0f;
            // the upper halves of the largest that some column sees, and that all do
            const uint32_t u = __builtin_bit_cast(uint32_t, v < inf ? v : 0.0f);
            const uint32_t top = __builtin_amdgcn_readfirstlane(
                max_halves_lane32(max_halves_lane16(max_halves_row((u & 0xFFFF0000u) | (shared ? u >> 16 : 0u)))));
            const int most = (int)(top >> 23) + kLeastExp, all = (int)((top & 0xFFFFu) >> 7) + kLeastExp;
            if (all > v_exp_run + kLag)
                v_exp_run = all < kMostStaged ? all : kMostStaged;
            const bool past = most > v_exp_run + kLag;
            const int exp = !past ? v_exp_run : (most < kMostStaged ? most : kMostStaged);
            // the 16 times larger codes belong to tokens 1 and 3 of each 4
            to.scale[wave - 1][scale_slot(lane)] = ldexp_f(v, kTop - exp - (lane & 1 ? 4 : 0));
            if (lane == 0) {
                to.exp[wave - 1] = past ? exp + kPast : exp;
                to.base[wave - 1] = v_exp_run;
            }
        }
    };
    // the K operands of step s of a page: steps go through both tiles' first
    // group, then both tiles' second
    constexpr int SG = GS / 16;  // steps of a group
    auto k_tile = [](int s) { return s / SG % 2; };
    auto k_step = [](int s) { return s / (2 * SG) * SG + s % SG; };

    if (begin < end) {
#pragma unroll
        for (int m = 0; m < ND; ++m) {
            stage_k_dword(page_k[0], share, m);
            stage_v_dword(page_v[0], share, m);
            stage_k_dword(page_k[1], share1, m);
        }
        stage_k_scales(page_k[0], share);
        stage_v_scales(page_v[0], share, n0, t.range.at_turned(begin) * kPageTokens);
        stage_k_scales(page_k[1], share1);
    }
    __syncthreads();
    // scores of the page in turn less the running maximum, and the lane's largest
    float x[2][16], top = 0.0f;
    if (begin < end) {
#pragma unroll
        for (int s = 0; s < 2 * NK; ++s) {
            const int tt = k_tile(s), k = k_step(s);
            if (k == 0)
                r[tt] = f32x16{};
            else if (k % SG == 0) {
                const float ratio = page_k[0].ratio[32 * tt + slot];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    r[tt][e] = scaled(r[tt][e], ratio, e);
            }
            r[tt] = mfma(page_k[0].code[tt][k][k_from[k % 2]], q[k], r[tt]);
        }
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const float ks = page_k[0].scale[32 * tt + slot];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                x[tt][e] = scaled(APART ? r[tt][e] * q_factor : r[tt][e], ks, e);
                top = e + tt == 0 ? x[tt][e] : __builtin_fmaxf(top, x[tt][e]);
            }
        }
    }
    __syncthreads();  // the first step unpacks the third page's K to where the first one's was
    int t1 = t.range.at_turned(begin) * kPageTokens;  // the next page's first token
    int stop = 0;  // columns stand apart: known a page later, when the word has come from LDS
    for (int i = begin; i < end; ++i) {
        if (!APART && stop)
            return false;
        const PageV<D, GS> &pv = page_v[(i - begin) & 1];
        const PageK<D, GS> &pk = page_k[(i - begin + 1) & 1];
        int n3 = -1;
        const int t0 = t1;
        t1 = t.range.at_turned(i + 1 < end ? i + 1 : i) * kPageTokens;

        // Operands come from LDS kAhead steps before they are used: the first of
        // K's before the softmax begins, of V's in its last steps.
        constexpr int kSteps = 2 * NK, kAhead = 2;  // score products, and as many of the outputs
        static_assert(kSteps == 4 * NT, "");
        uint4 kf[kAhead + 1], vf[kAhead + 1];
        auto read_k = [&](int s) {
            if (s < kSteps)
                kf[s % (kAhead + 1)] = pk.code[k_tile(s)][k_step(s)][k_from[k_step(s) % 2]];
        };
        auto read_v = [&](int s) {
            if (s < kSteps)
                vf[s % (kAhead + 1)] = pv.code[s / (2 * NT)][s / NT % 2][s % NT][lane];
        };
        const int stood_apart = lds.stand_apart[(i - begin + 1) & 1];  // in the page before
        float vs[2][NG];  // V's scales and the page's exponents
        int vs_exp[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            vs_exp[g] = pv.exp[g];
            vs[0][g] = pv.scale[g][slot];
            vs[1][g] = pv.scale[g][32 + slot];
        }

#pragma unroll
        for (int s = 0; s < kAhead; ++s)
            read_k(s);
        const float m_old = m_run == -inf ? 0.0f : m_run;  // what x is less by
        const bool whole = t0 + kPageTokens - 1 <= w_lo && (unsigned)n0 < (unsigned)a.kv.num_pages &&
                           (a.window == 0 || t0 > w_hi - a.window || t0 + kPageTokens <= a.sinks);
        uint32_t seen = ~0u;
        if (!whole) {
            seen = (unsigned)n0 < (unsigned)a.kv.num_pages ? tokens_seen<8>(p, t0 + 4 * h, a.window, a.sinks) : 0u;
#pragma unroll
            for (int e = 0; e < 32; ++e)
                x[e / 16][e % 16] = seen_score(x[e / 16][e % 16], seen, e);
            top = x[0][0];
#pragma unroll
            for (int e = 1; e < 32; ++e)
                top = __builtin_fmaxf(top, x[e / 16][e % 16]);
        }
        if (__any(top > (m_run == -inf ? -inf : kSlack))) {
            top = max_lane32(top);
            const float up = top > kSlack || m_run == -inf ? top : 0.0f;  // of the column's own maximum
            if (up != -inf) {
                const float f = m_run == -inf ? 0.0f : __builtin_amdgcn_exp2f(-up);
                m_run = m_old + up;
                l_run *= f;
#pragma unroll
                for (int y = 0; y < NT; ++y)
                    acc[y] *= f;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    x[e / 16][e % 16] -= up;
            }
        }
        stop = __builtin_amdgcn_readfirstlane(stood_apart);
        int by[NG];  // what a column's weights are short of
        if constexpr (!APART) {
            // the exponents move with what every column sees
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int e = __builtin_amdgcn_readfirstlane(vs_exp[g]);
                if (e != v_exp[g]) {
                    if (e > kPast / 2)
                        lds.stand_apart[(i - begin) & 1] = 1;
                    const float f = ldexp_f(1.0f, v_exp[g] - e);
#pragma unroll
                    for (int y = g * GS / 32; y < (g + 1) * GS / 32; ++y)
                        acc[y] *= f;
                    v_exp[g] = e;
                }
            }
        } else {
            bool look = false;  // else the page is within the lag of every column's
            int base[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                vs_exp[g] = __builtin_amdgcn_readfirstlane(vs_exp[g]);
                base[g] = __builtin_amdgcn_readfirstlane(pv.base[g]);
                look |= vs_exp[g] > kPast / 2 || base[g] > exps[g].reach;
                vs_exp[g] -= vs_exp[g] > kPast / 2 ? kPast : 0;
            }
            if (look) {
                uint32_t e[2] = {0, 0};  // exponents of the lane's two tokens, a half for a group
#pragma unroll
                for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const float v = ldexp_f(vs[tt][g], vs_exp[g] - kTop + (lane & 1 ? 4 : 0));  // as it is
                        e[tt] |= (uint32_t)(scale_exponent(v) + kExpBias) << 16 * g;
                    }
                const uint32_t largest = max_halves_lane32(seen_largest(e, seen, lane));
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const int was = lds.own[g][own_at], top = half_exponent(largest, g);
                    const int next = base[g] > was ? base[g] : was;
                    const int now = exps[g].template raise<32>(was, top > next + kLag ? top : next, p >= 0);
                    lds.own[g][own_at] = now;
                    const float f = ldexp_f(1.0f, was - now);
#pragma unroll
                    for (int y = g * GS / 32; y < (g + 1) * GS / 32; ++y)
                        acc[y] *= f;
                }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                by[g] = scale_shift(exps[g].all, lds.own[g][own_at]);
                vs[0][g] = ldexp_f(vs[0][g], vs_exp[g] - exps[g].all);
                vs[1][g] = ldexp_f(vs[1][g], vs_exp[g] - exps[g].all);
            }
        }

        // The weights of page i, one pair of tokens a step, each step with one
        // score product of page i + 1 in front of it: the matrix core works
        // while the vector unit does.  The
        // barriers keep the compiler from gathering the products.  (Past
        // the last page the products take what lies in the buffer; unused.)
        uint32_t w[2][NG][2][4];
        bool masked = false;
        float ks[2];  // K's scales of page i + 1
        {
            float ratio[2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                ks[tt] = pk.scale[32 * tt + slot];
                if (NG == 2)
                    ratio[tt] = pk.ratio[32 * tt + slot];
            }
            // a hidden token's weight is 0, and times a scale that is not finite
            // it would not stay so
            if (!whole) {
                bool odd = false;
#pragma unroll
                for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        odd |= !(__builtin_fabsf(vs[tt][g]) < inf);
                masked = __any(odd);
            }
            // exponentials are taken a step before their use, which waits for them else
            constexpr int kPairs = 16 / kSteps;
            auto power = [&](int pair) {
                if (pair < 16) {
                    float &lo = x[pair / 8][4 * (pair / 4 % 2) + pair % 4];
                    float &hi = x[pair / 8][8 + 4 * (pair / 4 % 2) + pair % 4];
                    lo = __builtin_amdgcn_exp2f(lo);
                    hi = __builtin_amdgcn_exp2f(hi);
                }
            };
#pragma unroll
            for (int pair = 0; pair < kPairs; ++pair)
                power(pair);
            float sum[2] = {0.0f, 0.0f};
            r[0] = f32x16{};
            r[1] = f32x16{};
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                r[k_tile(s)] = mfma(kf[s % (kAhead + 1)], q[k_step(s)], r[k_tile(s)]);
                read_k(s + kAhead);
                if (s == 0) {  // what is unpacked in this step's second half
                    n3 = number_of(i + 3);
                    fetch_v(share, v_block);
                    v_block = block_of(n2);
                    fetch_k(share, v_block);
                }
                if (s >= kSteps - kAhead)
                    read_v(s - (kSteps - kAhead));
                // pairs of tokens of this step: one of 16 steps, two of 8
#pragma unroll
                for (int pair = s * 16 / kSteps; pair < (s + 1) * 16 / kSteps; ++pair) {
                    const int tt = pair / 8, y = pair / 4 % 2, e = pair % 4;
                    const float lo = x[tt][4 * y + e], hi = x[tt][8 + 4 * y + e];
                    power(pair + kPairs);
                    sum[0] += lo;
                    sum[1] += hi;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        w[tt][g][y][e] = pack2<OUT_F16>(scaled(APART ? ldexp_f(lo, by[g]) : lo, vs[tt][g], 4 * y + e),
                                                        scaled(APART ? ldexp_f(hi, by[g]) : hi, vs[tt][g], 8 + 4 * y + e));
                }
                // between a tile's groups its products are scaled, a quarter a step
                if (NG == 2 && s >= SG && s < 3 * SG) {
                    f32x16 &to = r[s / SG - 1];
#pragma unroll
                    for (int e = 4 * (s % SG); e < 4 * (s % SG) + 4; ++e)
                        to[e] = scaled(to[e], ratio[s / SG - 1], e);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            l_run += sum[0] + sum[1];
        }
        if (masked) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const int tt = e / 8, y = e / 4 % 2, f = e % 4;
                    w[tt][g][y][f] &= ((seen >> (16 * tt + 4 * y + f)) & 1u ? 0xFFFFu : 0u) |
                                      ((seen >> (16 * tt + 8 + 4 * y + f)) & 1u ? 0xFFFF0000u : 0u);
                }
        }

        // The outputs of page i, with vector work of what comes next between
        // them: the scaling of page i + 1's scores and their maximum, the
        // unpacking of K of page i + 2 and V of page i + 1.
        {
            const float m_sub = m_run == -inf ? 0.0f : m_run;
            PageK<D, GS> &to_k = page_k[(i - begin) & 1];
            PageV<D, GS> &to_v = page_v[(i - begin + 1) & 1];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int tt = s / (2 * NT), y = s / NT % 2, z = s % NT;
                const uint32_t(&o)[4] = w[tt][z * 32 / GS][y];
                acc[z] = mfma(vf[s % (kAhead + 1)], __builtin_bit_cast(half8, uint4{o[0], o[1], o[2], o[3]}), acc[z]);
                read_v(s + kAhead);
#pragma unroll
                for (int e = s * 32 / kSteps; e < (s + 1) * 32 / kSteps; ++e) {
                    const float s = APART ? r[e / 16][e % 16] * q_factor : r[e / 16][e % 16];
                    // (fused both ways, which makes them agree to the last bit)
                    x[e / 16][e % 16] = __builtin_fmaf(row_value(ks[e / 16], e % 16), s, -m_sub);
                    top = e == 0 ? x[0][0] : __builtin_fmaxf(top, x[e / 16][e % 16]);
                }
                constexpr int EVERY = kSteps / (2 * ND);
                if (s % EVERY == EVERY - 1) {
                    if (s / EVERY < ND)
                        stage_k_dword(to_k, share, s / EVERY);
                    else
                        stage_v_dword(to_v, share, s / EVERY - ND);
                }
                if (s == kSteps / 2) {  // a chain of a few operations in one wavefront each
                    stage_v_scales(to_v, share, n1, t1);
                    stage_k_scales(to_k, share);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        n0 = n1;
        n1 = n2;
        n2 = n3;
        __syncthreads();
    }

    if (!APART && begin < end && (stop || __builtin_amdgcn_readfirstlane(lds.stand_apart[(end - begin - 1) & 1])))
        return false;

    // lane (h, c) holds elements 32 x + 8 i + 4 h .. + 3 of column c
    l_run += __shfl_xor(l_run, 32);
    if (!valid)
        return true;
    auto exp_of = [&](int g) { return APART ? lds.own[g][own_at] : v_exp[g]; };
    // taken to their units last: a power of two by itself would not be finite for the
    // largest
    auto result = [&](int x, int i, float f, int e) {
        return ldexp_f(f32x4{acc[x][4 * i], acc[x][4 * i + 1], acc[x][4 * i + 2], acc[x][4 * i + 3]} * f,
                       exp_of(x * 32 / GS) + 24 - kTop - e);
    };
    if (in_parts<PAGES>(n, t)) {
        const int64_t at = part_of<PAGES>(n, t, pair_of(a, t, col), split);
        const int less = sum_bits(PAGES == Pages::All ? n.pages : n.sum_pages);
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f32x4 *>(n.part + at * D + 32 * x + 8 * i + 4 * h) = result(x, i, 1.0f, less);
        if (h == 0) {
            n.part_stat[2 * at] = m_run;
            n.part_stat[2 * at + 1] = l_run;
        }
        return true;
    }
    const float inv = reciprocal(l_run);
    uint16_t *y = output_of(a, t, col) + 4 * h;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 o = result(x, i, inv, 0);
            *reinterpret_cast<uint2 *>(y + 32 * x + 8 * i) =
                uint2{pack_out(o.x, o.y, a.y_dtype), pack_out(o.z, o.w, a.y_dtype)};
        }
    return true;
}

template <int D, int GS, int COLS, Pages PAGES>
__global__ __launch_bounds__(COLS * 2, 2) void kv4_many_rows_kernel(Kv4AttentionArgs a, Kv4Launch n)
{
    __shared__ Lds<D, GS, COLS> lds;
    // heads fastest (one kv head's pages stay in one XCD's L2), then sequences,
    // splits and tiles, the last tiles, which see most, first.  Sequences are
    // dealt in another order for every tile: in one fixed order a batch of 4
    // falls into step with the 4 shader engines that an XCD fills in turn, and
    // the longest sequence lands on one of them (ragged prompts up to 4096 rows:
    // 617 us against 232)
    Work work;
    if (!work_of<PAGES>(a, n, kv4_workgroup(), work))
        return;
    const unsigned batch = (unsigned)(work.front ? n.runs.groups : a.kv.batch);
    const int split = work.split, tile = (work.front ? n.front_tiles : n.tiles) - 1 - work.tile;
    const int b = (int)(((unsigned)work.b + (unsigned)tile) % batch);
    Tile t;
    if (!tile_of<COLS, PAGES>(a, n, b, work.head, tile, work.front, t))
        return;
    int begin, end;
    if (!chunk_of<PAGES>(n, t, split, begin, end))
        return;

    // a tile whose columns share no token goes the long way at once
    int tid = threadIdx.x;
    if (tile_has_first(a, t) && many_rows_tile<D, GS, COLS, PAGES, false>(a, n, lds, t, split, begin, end, tid))
        return;
    // From the beginning, nothing of the first way kept: whatever both had in common
    // would cost that one its registers (2048 rows over 16384 tokens 603 us; with a
    // block for such pages in its loop 4 % more, with a copy of the loop in place four
    // times as much).
    __syncthreads();
    asm volatile("" : "+v"(tid));
    many_rows_tile<D, GS, COLS, PAGES, true>(a, n, lds, t, split, begin, end, tid);
}

}  // namespace

template <int COLS, Pages PAGES>
static hipError_t launch(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    const unsigned grid = (PAGES == Pages::Shared ? n.front_groups : 0u) +
                          (unsigned)n.tiles * (unsigned)n.splits * (unsigned)a.kv.kv_heads * (unsigned)a.kv.batch;
    if (a.kv.head_dim == 64)
        return kv4_launch(kv4_many_rows_kernel<64, 64, COLS, PAGES>, grid, COLS * 2, stream, a, n);
    if (a.kv.group_size == 64)
        return kv4_launch(kv4_many_rows_kernel<128, 64, COLS, PAGES>, grid, COLS * 2, stream, a, n);
    return kv4_launch(kv4_many_rows_kernel<128, 128, COLS, PAGES>, grid, COLS * 2, stream, a, n);
}

hipError_t launch_kv4_many_rows(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    return n.cols == 256 ? launch<256, Pages::All>(a, n, stream) : launch<128, Pages::All>(a, n, stream);
}
hipError_t launch_kv4_many_rows_shared(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    return n.cols == 256 ? launch<256, Pages::Shared>(a, n, stream) : launch<128, Pages::Shared>(a, n, stream);
}

}  // namespace cider
