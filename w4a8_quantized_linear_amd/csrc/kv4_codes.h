// What writing to the 4-bit key/value cache and reading it back share: which tokens a
// workgroup has, the int4 codes of a chunk, and the change between V's two orders.
// kv4_cache.hip states the formulas.
#pragma once

#include <type_traits>

#include "kv4_layout.h"
#include "quant_common.h"

namespace cider {

constexpr int kThreads = 256;
constexpr int kSpan = 32;  // token positions of a workgroup

// The 16-bit rows pass through once: non-temporal (a batch's caches read back
// 50.8 -> 34.1 us, 6.5 TB/s), so the cache's pages keep the L2.
__device__ __forceinline__ uint4 nt_load(const uint16_t *p)
{
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p)));
}
__device__ __forceinline__ void nt_store(uint16_t *p, uint4 v)
{
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4 *>(p));
}

// Which 32 positions, head and sequence a workgroup has.  base may be below 0
// (rows in front of the sequence's first token).
struct Place {
    int b, h, base;
    int lo, hi;     // positions of the call's rows within [base, base + 32), lo < hi
    int64_t shift;  // row of position p is p + shift
};

__device__ __forceinline__ bool place_of(const Kv4Args &a, int spans, Place &w)
{
    unsigned id = kv4_workgroup();
    w.h = (int)(id % (unsigned)a.kv_heads);
    id /= (unsigned)a.kv_heads;
    const int span = (int)(id % (unsigned)spans);
    w.b = (int)(id / (unsigned)spans);
    if (w.b >= a.batch)
        return false;
    const Kv4Sequence s = kv4_sequence(a, w.b);
    const int first = s.kv - s.n;
    w.base = (first & ~(kSpan - 1)) + span * kSpan;  // rounds down below 0 too
    w.lo = first > w.base ? first : w.base;
    w.hi = s.kv < w.base + kSpan ? s.kv : w.base + kSpan;
    w.shift = (int64_t)s.row0 - first;
    return w.lo < w.hi;
}

// The block of a place's page; null where there is no such page.
template <int D, int GS>
__device__ __forceinline__ uint8_t *block_of(const Kv4Args &a, const Place &w)
{
    if (w.hi <= 0)
        return nullptr;
    const int page = a.pages[(int64_t)w.b * a.max_pages + w.base / kPageTokens];
    if ((unsigned)page >= (unsigned)a.num_pages)
        return nullptr;
    return a.cache + ((int64_t)page * a.kv_heads + w.h) * kv4_block_bytes(D, GS);
}

// Largest of v over aligned runs of L lanes (8 or 16), within rows of 16 by DPP.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp_u(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
    return o > v ? o : v;
}
template <int L>
__device__ __forceinline__ uint32_t run_max(uint32_t v)
{
    v = max_dpp_u<0xB1>(v);   // quad_perm [1,0,3,2]
    v = max_dpp_u<0x4E>(v);   // quad_perm [2,3,0,1]
    v = max_dpp_u<0x141>(v);  // row_half_mirror
    if constexpr (L == 16)
        v = max_dpp_u<0x140>(v);  // row_mirror
    return v;
}

// a / 7 correctly rounded, a the magnitude of a 16-bit value: the product with
// 1/7 and one correction by its exact remainder (right for every fp16 and, by
// their mantissas, every bf16 value whose remainder does not underflow; the
// others, 0 and infinity divide).
__device__ __forceinline__ float seventh(float a)
{
    constexpr float kInv = 1.0f / 7.0f;
    if (!(a >= 0x1p-90f && a < __builtin_inff()))
        return a / quant_divisor<4>();
    const float q = a * kInv;
    return __builtin_fmaf(__builtin_fmaf(-7.0f, q, a), kInv, q);
}

// The int4 codes of 8 values, packed: quantize_chunk's, by fewer operations.
// r = rint(x * rs) by adding and taking off 1.5 2^23, d = x * rs - r its
// distance, and the nibbles u = r + 8 are put together as whole numbers in
// fp32 (at most 16 bits, exact).  x * rs, exact inside the fused operations, is
// within 2^-19 of the correctly rounded quotient x / s (|x / s| <= 7.5, rs, the
// hardware's 1 / s, off by at most 2^-23 of itself), so where d stays 2^-14 away
// from a half the rounding is the quotient's; a chunk with a value nearer to
// one, or of a group whose scale is not a normal number (0, NaN and infinity
// too), divides.
__device__ __forceinline__ bool int4_codes(const float (&x)[8], float s, float rs, uint32_t &codes)
{
    constexpr float kMagic = 12582912.0f;
    float r[8], far = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        r[e] = __builtin_fmaf(x[e], rs, kMagic) - kMagic;
        far = __builtin_fmaxf(far, __builtin_fabsf(__builtin_fmaf(x[e], rs, -r[e])));
    }
    uint32_t half[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float *q = r + 4 * i;
        const float lo = __builtin_fmaf(q[1], 16.0f, q[0]), hi = __builtin_fmaf(q[3], 16.0f, q[2]);
        half[i] = (uint32_t)(__builtin_fmaf(hi, 256.0f, lo) + 34952.0f);  // 0x8888: 8 to each nibble
    }
    codes = half[0] | half[1] << 16;
    return !(tiny_scale(s) || !(s < __builtin_inff()) || !(far < 0.5f - 0x1p-14f));
}
template <int DT>
__device__ __forceinline__ uint32_t int4_codes(uint4 v, float s, float rs)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = widen_bits<DT>(e & 1 ? w[e / 2] >> 16 : w[e / 2]);
    uint32_t codes;
    return int4_codes(x, s, rs, codes) ? codes : quantize_chunk_div<4, DT>(v, s).x;
}
// Of fp32 values.
__device__ __forceinline__ uint32_t int4_codes(const float (&x)[8], float s, float rs)
{
    uint32_t codes;
    if (int4_codes(x, s, rs, codes))
        return codes;
    int q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        q[e] = code_of<4>(x[e] / s, s);
    return pack_codes<4>(q).x;
}

// Where a lane's chunks (8 elements each) are: chunk column and, per register,
// token of the span.  D 128: 16 columns, i = lane / 16, b the register; D 64: 8
// columns, b = lane / 32, i = lane / 8 % 4.
template <int D>
__device__ __forceinline__ int token_of(int lane, int j, int reg)
{
    return D == 128 ? 16 * reg + 4 * j + lane / 16 : lane / 32 * 16 + 4 * j + lane / 8 % 4;
}

// Exchanges between registers and lane halves (rows of 16): the first's upper
// half (odd rows) against the second's lower half (even rows).  The second
// operand is made another value in the compiler's eyes: given one value twice
// it takes both results for equal.
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b)
{
    asm("" : "+v"(b));
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b)
{
    asm("" : "+v"(b));
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// V's codes between orders, the same steps in reverse order both ways.  Tokens:
// w[b] holds a chunk's 8 elements of the lane's token.  Dwords: w holds, per
// element, the wavefront's 8 tokens; the lane's dwords lie together at
// dword_of.
//   halves  elements 0 - 3 and 4 - 7 of the two b   <->  lane bit 5
//   pairs   within them                             <->  lane bit 4
//   nibbles of a pair                               <->  the register (D 128) or lane bit 3 (D 64)
// and, D 128, two dwords that are neighbours in the cache (x, x + 1; lanes l and
// l ^ 2) into one lane.
constexpr uint32_t kLowHalves = 0x05040100u, kHighHalves = 0x07060302u;  // byte selectors of v_perm
constexpr uint32_t kEvenBytes = 0x06020400u, kOddBytes = 0x07030501u;
constexpr uint32_t kLowNibbles = 0x0F0F0F0Fu;

template <int D>
__device__ __forceinline__ int dword_of(int lane, int j)
{
    if constexpr (D == 128) {
        const int c8 = lane % 16, c = c8 % 2 * 8 + lane / 32 * 4 + lane / 16 % 2 * 2 + c8 / 2 % 2;
        return ((c8 / 8 * 4 + j) * 16 + c) * 4 + c8 / 4 % 2 * 2;
    } else {
        const int c8 = lane % 8, c = c8 % 2 * 8 + lane / 32 * 4 + lane / 16 % 2 * 2 + lane / 8 % 2;
        return (j * 16 + c) * 4 + c8 / 2;
    }
}

__device__ __forceinline__ void neighbours(uint32_t (&w)[2], int lane)
{
    const bool odd = lane & 2;
    const uint32_t got = dpp<0x4E>(odd ? w[0] : w[1]);  // quad_perm [2,3,0,1]
    w[0] = odd ? got : w[0];
    w[1] = odd ? w[1] : got;
}
__device__ __forceinline__ void nibbles(uint32_t (&w)[2])
{
    const uint32_t a = w[0], b = w[1];
    w[0] = (a & kLowNibbles) | ((b << 4) & ~kLowNibbles);
    w[1] = ((a >> 4) & kLowNibbles) | (b & ~kLowNibbles);
}
__device__ __forceinline__ void select(uint32_t (&w)[2], uint32_t first, uint32_t second)
{
    const uint32_t a = w[0], b = w[1];
    w[0] = __builtin_amdgcn_perm(b, a, first);
    w[1] = __builtin_amdgcn_perm(b, a, second);
}
__device__ __forceinline__ void nibbles(uint32_t (&w)[1], int lane)
{
    const uint32_t a = w[0], b = dpp<0x128>(a);  // row_ror:8, the lane 8 away
    w[0] = lane & 8 ? ((b >> 4) & kLowNibbles) | (a & ~kLowNibbles)
                    : (a & kLowNibbles) | ((b << 4) & ~kLowNibbles);
}
__device__ __forceinline__ void pairs(uint32_t (&w)[1], int lane)
{
    uint32_t a = w[0], b = a;
    swap16(a, b);
    w[0] = __builtin_amdgcn_perm(b, a, lane & 16 ? kOddBytes : kEvenBytes);
}
__device__ __forceinline__ void half_words(uint32_t (&w)[1], int lane)
{
    uint32_t a = w[0], b = a;
    swap32(a, b);
    w[0] = __builtin_amdgcn_perm(b, a, lane & 32 ? kHighHalves : kLowHalves);
}
__device__ __forceinline__ void tokens_to_dwords(uint32_t (&w)[2], int lane)
{
    select(w, kLowHalves, kHighHalves);
    swap32(w[0], w[1]);
    select(w, kEvenBytes, kOddBytes);
    swap16(w[0], w[1]);
    nibbles(w);
    neighbours(w, lane);
}
__device__ __forceinline__ void dwords_to_tokens(uint32_t (&w)[2], int lane)
{
    neighbours(w, lane);
    nibbles(w);
    swap16(w[0], w[1]);
    select(w, kEvenBytes, kOddBytes);
    swap32(w[0], w[1]);
    select(w, kLowHalves, kHighHalves);
}
__device__ __forceinline__ void tokens_to_dwords(uint32_t (&w)[1], int lane)
{
    half_words(w, lane);
    pairs(w, lane);
    nibbles(w, lane);
}
__device__ __forceinline__ void dwords_to_tokens(uint32_t (&w)[1], int lane)
{
    nibbles(w, lane);
    pairs(w, lane);
    half_words(w, lane);
}
template <int N>
__device__ __forceinline__ void load_dwords(uint32_t (&w)[N], const uint32_t *at)
{
    if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(at);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *at;
    }
}

// Positions that a sequence's max_rows rows may lie across, in spans of 32.
inline int spans_of(const Kv4Args &a) { return (int)(((int64_t)a.max_rows + 2 * kSpan - 2) / kSpan); }

// Calls f<D, GS, DT>() for the batch's geometry.
template <typename F>
hipError_t with_geometry(const Kv4Args &a, int dtype, F f)
{
    using std::integral_constant;
    auto typed = [&](auto D, auto GS) {
        return dtype == DT_BF16 ? f(D, GS, integral_constant<int, DT_BF16>{})
                                : f(D, GS, integral_constant<int, DT_F16>{});
    };
    if (a.head_dim == 64)
        return typed(integral_constant<int, 64>{}, integral_constant<int, 64>{});
    if (a.group_size == 64)
        return typed(integral_constant<int, 128>{}, integral_constant<int, 64>{});
    return typed(integral_constant<int, 128>{}, integral_constant<int, 128>{});
}

}  // namespace cider
