// Writing the 4-bit key/value cache and reading it back.
//
//   s = absmax / 7, q = clamp(rint(x / s), -8, 7), u = q + 8   (append)
//   x^ = s * (u - 8)                                           (read)
// per group of GS consecutive elements of a head (Cider README, ossradar.top
// repo page, "Quantization" table: symmetric INT4 with zero-point 8), with the
// quantizers' own arithmetic (quant_common.h), so the codes are those
// cider_quantize_weight gives the same rows.
//
// One workgroup per (sequence, head, 32 consecutive token positions): the 32
// tokens are what shares a dword of V codes, so every dword of the cache has
// one writer in a call and a partly filled one is read, patched and written
// back without atomics.  Both directions move 16 bytes per lane on the 16-bit
// side (a head of a row is one contiguous run) and dwords on the cache side.
// Wavefront j has the 8 tokens 16 b + 4 j + i that share dwords of V, so V's
// codes change between token-major and element-major order in registers, by
// exchanges across the wavefront: 14 operations for 128 dwords, no LDS.
//
// What bounds them: bytes.  The append of 6 ragged prompts of up to 4096 rows
// (8 heads of 128, 70 MB) takes 22.1 us, 3.2 TB/s, of 65536 rows 4.3 TB/s, where
// its arithmetic (56 % of the vector units' time) still shows next to a plain
// copy's 4.85; the read of 8 sequences of up to 8192 (223 MB, three quarters of
// it written) 33.5 us, 6.6 TB/s.  One token is the launch and three loads in a
// row (lengths, then row and page number, then the codes that share its words):
// append 4.7 us, read 2.7.
#include <type_traits>

#include "kv4_layout.h"
#include "quant_common.h"

namespace cider {
namespace {

constexpr int kThreads = 256;
constexpr int kSpan = 32;  // token positions of a workgroup

// The 16-bit rows pass through once: non-temporal (a batch's caches read back
// 50.8 -> 34.1 us, 6.5 TB/s), so the cache's pages keep the L2.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
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
template <int DT>
__device__ __forceinline__ uint32_t int4_codes(uint4 v, float s, float rs)
{
    constexpr float kMagic = 12582912.0f;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float r[8], far = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = widen_bits<DT>(e & 1 ? w[e / 2] >> 16 : w[e / 2]);
        r[e] = __builtin_fmaf(x, rs, kMagic) - kMagic;
        far = __builtin_fmaxf(far, __builtin_fabsf(__builtin_fmaf(x, rs, -r[e])));
    }
    if (tiny_scale(s) || !(s < __builtin_inff()) || !(far < 0.5f - 0x1p-14f))
        return quantize_chunk_div<4, DT>(v, s).x;
    uint32_t half[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float *q = r + 4 * i;
        const float lo = __builtin_fmaf(q[1], 16.0f, q[0]), hi = __builtin_fmaf(q[3], 16.0f, q[2]);
        half[i] = (uint32_t)(__builtin_fmaf(hi, 256.0f, lo) + 34952.0f);  // 0x8888: 8 to each nibble
    }
    return half[0] | half[1] << 16;
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

template <int D, int GS, int DT>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(Kv4Args a, const uint16_t *k,
                                                              const uint16_t *v, int64_t ldk,
                                                              int64_t ldv, int spans)
{
    constexpr int CH = D / 8;   // 8-value chunks of a token
    constexpr int PT = D / 64;  // chunks of K and of V, and V dwords, per thread
    Place w;
    if (!place_of(a, spans, w))
        return;
    const int lane = threadIdx.x % 64, c8 = lane % CH;
    const int j = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    uint32_t mask = 0;  // of a V dword's tokens, those of this call
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int p = w.base + e / 4 * 16 + 4 * j + e % 4;
        mask |= (p >= w.lo && p < w.hi ? 15u : 0u) << (4 * e);
    }
    if (mask == 0)
        return;
    uint4 kx[PT], vx[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int p = w.base + token_of<D>(lane, j, i);
        kx[i] = vx[i] = uint4{0, 0, 0, 0};
        if (p >= w.lo && p < w.hi) {
            kx[i] = nt_load(k + (p + w.shift) * ldk + w.h * D + c8 * 8);
            vx[i] = nt_load(v + (p + w.shift) * ldv + w.h * D + c8 * 8);
        }
    }
    uint8_t *block = block_of<D, GS>(a, w);
    if (!block)
        return;
    const int half = (w.base / kSpan) & 1;  // which 32 tokens of the page
    float *kscale = reinterpret_cast<float *>(block + kv4_scale_offset(D));
    float *vscale = kscale + kPageTokens * (D / GS);
    uint32_t *kcode = reinterpret_cast<uint32_t *>(block);
    uint32_t *vout = reinterpret_cast<uint32_t *>(block + kv4_v_offset(D)) + half * 4 * D + dword_of<D>(lane, j);
    uint32_t old[PT] = {};  // what a partly filled dword keeps
    if (mask != ~0u)
        load_dwords(old, vout);
    uint32_t vcode[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int t = token_of<D>(lane, j, i), p = w.base + t, token = half * kSpan + t;
        const float ks = seventh(widen_bits<DT>(run_max<GS / 8>(chunk_absmax_bits(kx[i]))));
        const float vs = seventh(widen_bits<DT>(run_max<GS / 8>(chunk_absmax_bits(vx[i]))));
        const uint32_t kq = int4_codes<DT>(kx[i], ks, __builtin_amdgcn_rcpf(ks));
        vcode[i] = int4_codes<DT>(vx[i], vs, __builtin_amdgcn_rcpf(vs));
        if (p >= w.lo && p < w.hi) {
            kcode[token * CH + (c8 % 4) * (D / 32) + c8 / 4] = kq;
            if (c8 % (GS / 8) == 0) {
                kscale[c8 / (GS / 8) * kPageTokens + token] = ks;
                vscale[c8 / (GS / 8) * kPageTokens + token] = vs;
            }
        }
    }
    tokens_to_dwords(vcode, lane);
#pragma unroll
    for (int i = 0; i < PT; ++i)
        vcode[i] = (old[i] & ~mask) | (vcode[i] & mask);
    if constexpr (PT == 2)
        *reinterpret_cast<uint2 *>(vout) = uint2{vcode[0], vcode[1]};
    else
        *vout = vcode[0];
}

// 8 codes (nibble e: value e) as 16-bit values scaled by s.
template <int DT>
__device__ __forceinline__ uint4 values_of(uint32_t codes, float s)
{
    constexpr int OUT = DT == DT_BF16 ? OUT_BF16 : OUT_F16;
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o[j] = pack2<OUT>(s * (float)((int)((codes >> (8 * j)) & 15u) - 8),
                          s * (float)((int)((codes >> (8 * j + 4)) & 15u) - 8));
    return uint4{o[0], o[1], o[2], o[3]};
}

template <int D, int GS, int DT>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4Args a, uint16_t *k, uint16_t *v,
                                                            int64_t ldk, int64_t ldv, int spans)
{
    constexpr int CH = D / 8, PT = D / 64;
    Place w;
    if (!place_of(a, spans, w))
        return;
    const uint8_t *block = block_of<D, GS>(a, w);
    const int lane = threadIdx.x % 64, c8 = lane % CH;
    const int j = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const int half = (w.base / kSpan) & 1;
    const uint32_t *kcode = reinterpret_cast<const uint32_t *>(block);
    const float *kscale = reinterpret_cast<const float *>(block + kv4_scale_offset(D));
    const float *vscale = kscale + kPageTokens * (D / GS);
    uint32_t vcode[PT] = {};
    if (block)
        load_dwords(vcode, reinterpret_cast<const uint32_t *>(block + kv4_v_offset(D)) + half * 4 * D +
                               dword_of<D>(lane, j));
    dwords_to_tokens(vcode, lane);
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int t = token_of<D>(lane, j, i), p = w.base + t, token = half * kSpan + t;
        if (p < w.lo || p >= w.hi)
            continue;
        uint4 kv = {0, 0, 0, 0}, vv = {0, 0, 0, 0};
        if (p >= 0 && block) {
            const int s = c8 / (GS / 8) * kPageTokens + token;
            kv = values_of<DT>(kcode[token * CH + (c8 % 4) * (D / 32) + c8 / 4], kscale[s]);
            vv = values_of<DT>(vcode[i], vscale[s]);
        }
        nt_store(k + (p + w.shift) * ldk + w.h * D + c8 * 8, kv);
        nt_store(v + (p + w.shift) * ldv + w.h * D + c8 * 8, vv);
    }
}

// Positions that a sequence's max_rows rows may lie across, in spans of 32.
int spans_of(const Kv4Args &a) { return (int)(((int64_t)a.max_rows + 2 * kSpan - 2) / kSpan); }

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

}  // namespace

hipError_t launch_kv4_append(const Kv4Args &a, const uint16_t *k, const uint16_t *v, int dtype,
                             int64_t ldk, int64_t ldv, hipStream_t stream)
{
    const int spans = spans_of(a);
    const unsigned grid = (unsigned)spans * (unsigned)a.kv_heads * (unsigned)a.batch;
    return with_geometry(a, dtype, [&](auto D, auto GS, auto DT) {
        return kv4_launch(kv4_append_kernel<D(), GS(), DT()>, grid, kThreads, stream, a, k, v, ldk, ldv, spans);
    });
}

hipError_t launch_kv4_read(const Kv4Args &a, uint16_t *k, uint16_t *v, int dtype, int64_t ldk,
                           int64_t ldv, hipStream_t stream)
{
    const int spans = spans_of(a);
    const unsigned grid = (unsigned)spans * (unsigned)a.kv_heads * (unsigned)a.batch;
    return with_geometry(a, dtype, [&](auto D, auto GS, auto DT) {
        return kv4_launch(kv4_read_kernel<D(), GS(), DT()>, grid, kThreads, stream, a, k, v, ldk, ldv, spans);
    });
}

}  // namespace cider
