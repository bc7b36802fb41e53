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
#include "kv4_codes.h"

namespace cider {
namespace {

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
