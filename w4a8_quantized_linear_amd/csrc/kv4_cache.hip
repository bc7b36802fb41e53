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
// side (a head of a row is one contiguous run) and dwords on the cache side;
// V's codes cross from token-major to element-major through LDS.
#include <type_traits>

#include "kv4_layout.h"
#include "quant_common.h"

namespace cider {
namespace {

constexpr int kThreads = 256;
constexpr int kSpan = 32;  // token positions of a workgroup

// Which 32 positions, head and sequence a workgroup has.  base may be below 0
// (rows in front of the sequence's first token).
struct Place {
    int b, h, base;
    int lo, hi;     // positions of the call's rows within [base, base + 32), lo < hi
    int64_t shift;  // row of position p is p + shift
    uint8_t *block; // null: no such page
};

template <int D, int GS>
__device__ __forceinline__ bool place_of(const Kv4Args &a, int spans, Place &w)
{
    const unsigned id = blockIdx.x;
    const int span = (int)(id % (unsigned)spans);
    const unsigned bh = id / (unsigned)spans;
    w.h = (int)(bh % (unsigned)a.kv_heads);
    w.b = (int)(bh / (unsigned)a.kv_heads);
    const Kv4Sequence s = kv4_sequence(a, w.b);
    const int first = s.kv - s.n;
    w.base = (first & ~(kSpan - 1)) + span * kSpan;  // rounds down below 0 too
    w.lo = first > w.base ? first : w.base;
    w.hi = s.kv < w.base + kSpan ? s.kv : w.base + kSpan;
    w.shift = (int64_t)s.row0 - first;
    w.block = nullptr;
    if (w.lo >= w.hi)
        return false;
    if (w.hi > 0) {
        const int page = a.pages[(int64_t)w.b * a.max_pages + w.base / kPageTokens];
        if ((unsigned)page < (unsigned)a.num_pages)
            w.block = a.cache + ((int64_t)page * a.kv_heads + w.h) * kv4_block_bytes(D, GS);
    }
    return true;
}

// Largest of v over aligned runs of L lanes (8 or 16).
template <int L>
__device__ __forceinline__ uint32_t run_max(uint32_t v)
{
#pragma unroll
    for (int d = 1; d < L; d *= 2) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, d);
        v = o > v ? o : v;
    }
    return v;
}

template <int D, int GS, int DT>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(Kv4Args a, const uint16_t *k,
                                                              const uint16_t *v, int64_t ldk,
                                                              int64_t ldv, int spans)
{
    constexpr int CH = D / 8;                     // 8-value chunks of a token
    constexpr int PT = kSpan * CH / kThreads;     // chunks per thread
    constexpr int WT = 4 * D / kThreads;          // V dwords per thread
    __shared__ uint32_t vcode[kSpan][CH];
    Place w;
    if (!place_of<D, GS>(a, spans, w) || !w.block)
        return;
    const int tid = threadIdx.x;
    const int half = (w.base / kSpan) & 1;  // which 32 tokens of the page
    float *kscale = reinterpret_cast<float *>(w.block + kv4_scale_offset(D));
    float *vscale = kscale + kPageTokens * (D / GS);
    uint32_t *kcode = reinterpret_cast<uint32_t *>(w.block);
    uint4 kx[PT], vx[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int c8 = (tid + i * kThreads) % CH, p = w.base + (tid + i * kThreads) / CH;
        kx[i] = vx[i] = uint4{0, 0, 0, 0};
        if (p >= w.lo && p < w.hi) {
            kx[i] = *reinterpret_cast<const uint4 *>(k + (p + w.shift) * ldk + w.h * D + c8 * 8);
            vx[i] = *reinterpret_cast<const uint4 *>(v + (p + w.shift) * ldv + w.h * D + c8 * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int c8 = (tid + i * kThreads) % CH, t = (tid + i * kThreads) / CH, p = w.base + t;
        const int token = half * kSpan + t;
        const float ks = widen_bits<DT>(run_max<GS / 8>(chunk_absmax_bits(kx[i]))) / quant_divisor<4>();
        const float vs = widen_bits<DT>(run_max<GS / 8>(chunk_absmax_bits(vx[i]))) / quant_divisor<4>();
        const uint32_t kq = quantize_chunk<4, DT>(kx[i], ks, 1.0f / ks).x;
        vcode[t][c8] = quantize_chunk<4, DT>(vx[i], vs, 1.0f / vs).x;
        if (p >= w.lo && p < w.hi) {
            kcode[token * CH + (c8 % 4) * (D / 32) + c8 / 4] = kq;
            if (c8 % (GS / 8) == 0) {
                kscale[c8 / (GS / 8) * kPageTokens + token] = ks;
                vscale[c8 / (GS / 8) * kPageTokens + token] = vs;
            }
        }
    }
    __syncthreads();
    uint32_t *vout = reinterpret_cast<uint32_t *>(w.block + kv4_v_offset(D)) + half * 4 * D;
#pragma unroll
    for (int i = 0; i < WT; ++i) {
        const int n = tid + i * kThreads;
        const int x = n & 3, c = (n >> 2) & 15, j = (n >> 6) & 3, d = (n >> 8) * 64 + x * 16 + c;
        uint32_t word = 0, mask = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = (e >> 2) * 16 + 4 * j + (e & 3), p = w.base + t;
            word |= ((vcode[t][d >> 3] >> (4 * (d & 7))) & 15u) << (4 * e);
            mask |= (p >= w.lo && p < w.hi ? 15u : 0u) << (4 * e);
        }
        if (mask == ~0u)
            vout[n] = word;
        else if (mask)
            vout[n] = (vout[n] & ~mask) | (word & mask);
    }
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
    constexpr int CH = D / 8;
    constexpr int PT = kSpan * CH / kThreads;
    constexpr int WT = 4 * D / kThreads;
    __shared__ uint32_t vword[4 * D];
    Place w;
    if (!place_of<D, GS>(a, spans, w))
        return;
    const int tid = threadIdx.x;
    const int half = (w.base / kSpan) & 1;
    if (w.block) {
        const uint32_t *vin = reinterpret_cast<const uint32_t *>(w.block + kv4_v_offset(D)) + half * 4 * D;
#pragma unroll
        for (int i = 0; i < WT; ++i)
            vword[tid + i * kThreads] = vin[tid + i * kThreads];
    }
    __syncthreads();
    const float *kscale = reinterpret_cast<const float *>(w.block + kv4_scale_offset(D));
    const float *vscale = kscale + kPageTokens * (D / GS);
    const uint32_t *kcode = reinterpret_cast<const uint32_t *>(w.block);
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int c8 = (tid + i * kThreads) % CH, t = (tid + i * kThreads) / CH, p = w.base + t;
        const int token = half * kSpan + t;
        if (p < w.lo || p >= w.hi)
            continue;
        uint4 kv = {0, 0, 0, 0}, vv = {0, 0, 0, 0};
        if (p >= 0 && w.block) {
            const int s = c8 / (GS / 8) * kPageTokens + token;
            kv = values_of<DT>(kcode[token * CH + (c8 % 4) * (D / 32) + c8 / 4], kscale[s]);
            const int shift = 4 * ((t >> 4) * 4 + (t & 3)), j = (t >> 2) & 3;
            uint32_t codes = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = c8 * 8 + e;
                const int n = (((d >> 6) * 4 + j) * 16 + (d & 15)) * 4 + ((d >> 4) & 3);
                codes |= ((vword[n] >> shift) & 15u) << (4 * e);
            }
            vv = values_of<DT>(codes, vscale[s]);
        }
        *reinterpret_cast<uint4 *>(k + (p + w.shift) * ldk + w.h * D + c8 * 8) = kv;
        *reinterpret_cast<uint4 *>(v + (p + w.shift) * ldv + w.h * D + c8 * 8) = vv;
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
        kv4_append_kernel<D(), GS(), DT()><<<grid, kThreads, 0, stream>>>(a, k, v, ldk, ldv, spans);
        return hipGetLastError();
    });
}

hipError_t launch_kv4_read(const Kv4Args &a, uint16_t *k, uint16_t *v, int dtype, int64_t ldk,
                           int64_t ldv, hipStream_t stream)
{
    const int spans = spans_of(a);
    const unsigned grid = (unsigned)spans * (unsigned)a.kv_heads * (unsigned)a.batch;
    return with_geometry(a, dtype, [&](auto D, auto GS, auto DT) {
        kv4_read_kernel<D(), GS(), DT()><<<grid, kThreads, 0, stream>>>(a, k, v, ldk, ldv, spans);
        return hipGetLastError();
    });
}

}  // namespace cider
