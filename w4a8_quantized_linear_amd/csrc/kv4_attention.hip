// Causal attention over the 4-bit key/value cache (include/cider.h,
// cider_kv4_attention): grouped query heads, a sliding window with a few first
// tokens kept, any number of rows per sequence.
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
// row's largest, then off by at most 2^-38 of it.  The weights e^(S - m) s_v
// are fp32 rounded once to fp16 after scaling by a power of two that puts the
// largest s_v seen into [2^13, 2^14): 11 significant bits down to 2^-28 of the
// largest possible weight, and sums of many weights average the error below
// that of the 16-bit output.  Scores, maxima, sums and outputs are fp32.
//
// Shape.  Columns are the 16 (row, query head) pairs c = r * G + g of one kv
// head, tokens the rows of S^T = K Q^T (v_mfma_f32_16x16x32_f16), so lane
// (j, c) ends with the scores of tokens 4 j + i of column c in its registers
// and they are, rounded and packed, the right operand of O^T += V^T P^T: no
// transpose, no LDS for either product.  A wavefront takes whole 64-token pages
// (every 4th of the workgroup's), loads the next page while it computes, and
// the 4 wavefronts' maxima, sums and outputs meet in LDS at the end.
#include "kv4_layout.h"
#include "quant_common.h"

namespace cider {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kCols = 16;
constexpr float kLog2e = 1.4426950408889634f;

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The 8 nibbles of a dword as fp16 operands, in the order 0 4 1 5 2 6 3 7;
// elements 2, 3, 6, 7 of the result (nibbles 1, 5, 3, 7) are 16 times as large.
__device__ __forceinline__ half8 codes_as_halves(uint32_t w)
{
    const uint32_t hi = w >> 8;
    return __builtin_bit_cast(
        half8, uint4{w & 0x000F000Fu, w & 0x00F000F0u, hi & 0x000F000Fu, hi & 0x00F000F0u});
}

// -8 2^-24 and -128 2^-24 in the same order.
__device__ __forceinline__ half8 offset_halves()
{
    return __builtin_bit_cast(half8, uint4{0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u});
}

__device__ __forceinline__ float ldexp_f(float x, int e) { return __builtin_amdgcn_ldexpf(x, e); }

// Maximum and sum over the 4 lanes (j = 0 .. 3) of a column.
__device__ __forceinline__ float column_max(float v)
{
    v = __builtin_fmaxf(v, __shfl_xor(v, 16));
    return __builtin_fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float column_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// The pages that a tile of columns sees: [0, sink_pages) and [first, end).
struct PageRange {
    int sink_pages, first, count;
    __device__ __forceinline__ int at(int i) const { return i < sink_pages ? i : first + i - sink_pages; }
};

// Columns at positions p_lo .. p_hi (p_hi >= 0).
__device__ __forceinline__ PageRange pages_seen(int p_lo, int p_hi, int window, int sinks)
{
    PageRange r;
    const int end = p_hi / kPageTokens + 1;
    const int from = window > 0 && p_lo - window + 1 > 0 ? p_lo - window + 1 : 0;
    r.first = from / kPageTokens;
    const int kept = window > 0 ? (sinks < p_hi + 1 ? sinks : p_hi + 1) : 0;
    const int kept_pages = (int)(((unsigned)kept + kPageTokens - 1) / kPageTokens);
    r.sink_pages = kept_pages < r.first ? kept_pages : r.first;
    r.count = r.sink_pages + end - r.first;
    return r;
}

// One page of codes as the lanes use them, and its scales by token (lane = token).
template <int D, int GS>
struct PageData {
    uint32_t k[4][D / 32];
    uint4 v[2][D / 64];
    float ks[D / GS], vs[D / GS];
};

template <int D, int GS>
__device__ __forceinline__ void load_page(PageData<D, GS> &p, const uint8_t *block, int lane)
{
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const uint8_t *at = block + (16 * t + lane % 16) * (D / 2) + lane / 16 * (D / 8);
        if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(at);
            p.k[t][0] = w.x;
            p.k[t][1] = w.y;
            p.k[t][2] = w.z;
            p.k[t][3] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(at);
            p.k[t][0] = w.x;
            p.k[t][1] = w.y;
        }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
            p.v[b][g] = *reinterpret_cast<const uint4 *>(block + kv4_v_offset(D) +
                                                         (b * (D / 64) + g) * 1024 + lane * 16);
    const float *s = reinterpret_cast<const float *>(block + kv4_scale_offset(D));
#pragma unroll
    for (int g = 0; g < D / GS; ++g) {
        p.ks[g] = s[g * kPageTokens + lane];
        p.vs[g] = s[(D / GS + g) * kPageTokens + lane];
    }
}

template <int D, int GS>
__global__ __launch_bounds__(kThreads) void kv4_attention_kernel(Kv4AttentionArgs a, int tiles)
{
    constexpr int NM = D / 32;   // score products per 16 tokens
    constexpr int NG = D / GS;   // scales per token
    constexpr int NT = D / 16;   // output tiles
    __shared__ __align__(16) float scales[kWaves][2][NG][kPageTokens];
    __shared__ __align__(16) float part[kWaves][kCols][D + 4];
    __shared__ float part_m[kWaves][kCols], part_l[kWaves][kCols];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane % 16, j = lane / 16;
    const int G = a.q_heads / a.kv.kv_heads;
    const unsigned id = blockIdx.x;
    const int tile = (int)(id % (unsigned)tiles);
    const unsigned bh = id / (unsigned)tiles;
    const int h = (int)(bh % (unsigned)a.kv.kv_heads), b = (int)(bh / (unsigned)a.kv.kv_heads);
    const Kv4Sequence seq = kv4_sequence(a.kv, b);
    const int cols = seq.n * G;  // < 2^31: rows * q_heads is
    if (tile >= (cols + kCols - 1) / kCols)
        return;
    const int col = tile * kCols + c;
    const bool valid = col < cols;
    const int row = valid ? col / G : 0;
    const int head = h * G + (valid ? col % G : 0);
    const int first = seq.kv - seq.n;  // position of row 0
    const int p = valid ? first + row : -1;
    const int last_col = (tile + 1) * kCols <= cols ? tile * kCols + kCols - 1 : cols - 1;
    const int p_lo = first + tile * kCols / G, p_hi = first + last_col / G;

    // q: scaled to a largest magnitude in [2^13, 2^14) and put in operand order
    half8 qop[NM];
    float zero[NG], qmul;
    {
        float x[NM][8], top = 0.0f;
        const uint16_t *q = a.q + (int64_t)(seq.row0 + row) * a.ldq + (int64_t)head * D + 8 * j;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            uint4 w = *reinterpret_cast<const uint4 *>(q + 32 * m);
            if (!valid)
                w = uint4{0, 0, 0, 0};
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t bits = e & 1 ? u[e / 2] >> 16 : u[e / 2];
                x[m][e] = a.q_dtype == DT_BF16 ? widen_bits<DT_BF16>(bits) : widen_bits<DT_F16>(bits);
                top = __builtin_fmaxf(top, __builtin_fabsf(x[m][e]));
            }
        }
        top = column_max(top);
        const int shift = 14 - __builtin_amdgcn_frexp_expf(top);
        qmul = ldexp_f(a.scale * kLog2e, 24 - shift);
#pragma unroll
        for (int g = 0; g < NG; ++g)
            zero[g] = 0.0f;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // operand order 0 4 1 5 2 6 3 7
                const int n = e / 2 + 4 * (e & 1);
                const bool sixteenth = (e >> 1) & 1;
                const _Float16 v = (_Float16)ldexp_f(x[m][n], sixteenth ? shift - 4 : shift);
                qop[m][e] = v;
                sum += sixteenth ? 16.0f * (float)v : (float)v;
            }
            zero[m * 32 / GS] += sum;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)
            zero[g] = column_sum(zero[g]) * -0x1p-21f;
    }

    f32x4 acc[NT], off[D / 64];
#pragma unroll
    for (int x = 0; x < NT; ++x)
        acc[x] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
        off[g] = f32x4{0, 0, 0, 0};
    float m_run = -__builtin_inff(), l_run = 0.0f;
    int v_exp[NG];  // 2^v_exp is above every finite s_v seen
#pragma unroll
    for (int g = 0; g < NG; ++g)
        v_exp[g] = -100;

    if (p_hi >= 0) {
        const PageRange range = pages_seen(p_lo, p_hi, a.window, a.sinks);
        const int32_t *table = a.kv.pages + (int64_t)b * a.kv.max_pages;
        const uint8_t *heads = a.kv.cache + (int64_t)h * kv4_block_bytes(D, GS);
        const int64_t page_bytes = (int64_t)a.kv.kv_heads * kv4_block_bytes(D, GS);
        const float inf = __builtin_inff();
        PageData<D, GS> cur, next;
        int i = wave, page = 0, page_next = 0;
        // a page number outside the cache is never followed: page 0 is loaded
        // in its place and its tokens are left out
        auto fetch = [&](PageData<D, GS> &d, int n) {
            const int number = table[range.at(n)];
            const bool there = (unsigned)number < (unsigned)a.kv.num_pages;
            load_page<D, GS>(d, heads + (there ? number : 0) * page_bytes, lane);
            return there ? range.at(n) : -1;
        };
        if (i < range.count)
            page = fetch(cur, i);
        for (; i < range.count; i += kWaves) {
            if (i + kWaves < range.count)
                page_next = fetch(next, i + kWaves);
            if (page >= 0) {
                const int t0 = page * kPageTokens;
                // scales by token into LDS; weights' exponents move up first
                const bool written = t0 + lane <= p_hi;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float s = written ? cur.vs[g] : 0.0f;
                    if (__any(s >= ldexp_f(1.0f, v_exp[g]) && s < inf)) {
                        float top = s < inf ? s : 0.0f;
#pragma unroll
                        for (int d = 1; d < 64; d *= 2)
                            top = __builtin_fmaxf(top, __shfl_xor(top, d));
                        const int e = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(top));
                        const float f = ldexp_f(1.0f, v_exp[g] - e);
                        v_exp[g] = e;
#pragma unroll
                        for (int x = g * GS / 16; x < (g + 1) * GS / 16; ++x)
                            acc[x] *= f;
#pragma unroll
                        for (int y = g * GS / 64; y < (g + 1) * GS / 64; ++y)
                            off[y] *= f;
                    }
                    scales[wave][0][g][lane] = cur.ks[g];
                    // the 16 times larger codes belong to tokens 1 and 3 of each 4
                    scales[wave][1][g][lane] = ldexp_f(s, 14 - v_exp[g] - (lane & 1 ? 4 : 0));
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();

                float s[4][4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f32x4 sum;
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        f32x4 r = {zero[g], zero[g], zero[g], zero[g]};
#pragma unroll
                        for (int m = g * GS / 32; m < (g + 1) * GS / 32; ++m)
                            r = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_as_halves(cur.k[t][m]),
                                                                       qop[m], r, 0, 0, 0);
                        const f32x4 ks = *reinterpret_cast<const f32x4 *>(&scales[wave][0][g][16 * t + 4 * j]);
                        sum = g == 0 ? r * ks : sum + r * ks;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[t][e] = sum[e];
                }
                uint32_t seen = 0xFFFFu;
                const bool all_seen = t0 + kPageTokens - 1 <= p_lo &&
                                      (a.window == 0 || t0 > p_hi - a.window || t0 + kPageTokens <= a.sinks);
                if (!all_seen) {
                    seen = 0;
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        const int t = t0 + 16 * (n / 4) + 4 * j + n % 4;
                        const bool see = t <= p && (a.window == 0 || t > p - a.window || t < a.sinks);
                        seen |= (uint32_t)see << n;
                        s[n / 4][n % 4] = see ? s[n / 4][n % 4] : -inf;
                    }
                }
                float top = s[0][0];
#pragma unroll
                for (int n = 1; n < 16; ++n)
                    top = __builtin_fmaxf(top, s[n / 4][n % 4]);
                const float m_new = __builtin_fmaxf(m_run, column_max(top));
                const float m_sub = m_new == -inf ? 0.0f : m_new;
                if (__any(m_new > m_run)) {
                    const float f = __builtin_amdgcn_exp2f((m_run - m_sub) * qmul);
                    l_run *= f;
#pragma unroll
                    for (int x = 0; x < NT; ++x)
                        acc[x] *= f;
#pragma unroll
                    for (int g = 0; g < D / 64; ++g)
                        off[g] *= f;
                    m_run = m_new;
                }
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    float &x = s[n / 4][n % 4];
                    x = __builtin_amdgcn_exp2f((x - m_sub) * qmul);
                    l_run += x;
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
#pragma unroll
                    for (int B = 0; B < 2; ++B) {
                        const f32x4 lo = *reinterpret_cast<const f32x4 *>(&scales[wave][1][g][32 * B + 4 * j]);
                        const f32x4 hi = *reinterpret_cast<const f32x4 *>(&scales[wave][1][g][32 * B + 16 + 4 * j]);
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = s[2 * B][e] * lo[e], y = s[2 * B + 1][e] * hi[e];
                            if (!all_seen) {  // a masked token's scale may be anything
                                x = (seen >> (8 * B + e)) & 1u ? x : 0.0f;
                                y = (seen >> (8 * B + 4 + e)) & 1u ? y : 0.0f;
                            }
                            w[e] = pack2<OUT_F16>(x, y);
                        }
                        const half8 pop = __builtin_bit_cast(half8, uint4{w[0], w[1], w[2], w[3]});
#pragma unroll
                        for (int y = g * GS / 64; y < (g + 1) * GS / 64; ++y) {
                            const uint32_t u[4] = {cur.v[B][y].x, cur.v[B][y].y, cur.v[B][y].z, cur.v[B][y].w};
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                acc[4 * y + x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                    codes_as_halves(u[x]), pop, acc[4 * y + x], 0, 0, 0);
                            off[y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(offset_halves(), pop, off[y], 0, 0, 0);
                        }
                    }
                }
            }
            cur = next;
            page = page_next;
        }
    }

    // the wavefronts' parts: lane (j, c) holds elements 16 x + 4 j .. + 3 of column c
    l_run = column_sum(l_run);
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        const f32x4 o = (acc[x] + off[x / 4]) * ldexp_f(1.0f, v_exp[x * 16 / GS] + 10);
        *reinterpret_cast<f32x4 *>(&part[wave][c][16 * x + 4 * j]) = o;
    }
    if (j == 0) {
        // in units of log2, so that parts compare without the column's qmul
        part_m[wave][c] = m_run == -__builtin_inff() ? m_run : m_run * qmul;
        part_l[wave][c] = l_run;
    }
    __syncthreads();
    constexpr int PER = D / 16;  // elements per thread
    const int oc = threadIdx.x / 16, d0 = threadIdx.x % 16 * PER;
    const int ocol = tile * kCols + oc;
    if (ocol >= cols)
        return;
    float m = -__builtin_inff(), l = 0.0f, o[PER] = {};
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        m = __builtin_fmaxf(m, part_m[w][oc]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (part_l[w][oc] == 0.0f)  // saw nothing
            continue;
        const float f = __builtin_amdgcn_exp2f(part_m[w][oc] - m);
        l += part_l[w][oc] * f;
#pragma unroll
        for (int e = 0; e < PER; ++e)
            o[e] += part[w][oc][d0 + e] * f;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t w[PER / 2];
#pragma unroll
    for (int e = 0; e < PER; e += 2)
        w[e / 2] = a.y_dtype == DT_BF16 ? pack2<OUT_BF16>(o[e] * inv, o[e + 1] * inv)
                                        : pack2<OUT_F16>(o[e] * inv, o[e + 1] * inv);
    uint16_t *y = a.y + (int64_t)(seq.row0 + ocol / G) * a.ldy + (int64_t)(h * G + ocol % G) * D + d0;
    if constexpr (PER == 8)
        *reinterpret_cast<uint4 *>(y) = uint4{w[0], w[1], w[2], w[3]};
    else
        *reinterpret_cast<uint2 *>(y) = uint2{w[0], w[1]};
}

}  // namespace

hipError_t launch_kv4_attention(const Kv4AttentionArgs &a, hipStream_t stream)
{
    const int G = a.q_heads / a.kv.kv_heads;
    const int tiles = (int)(((int64_t)a.kv.max_rows * G + kCols - 1) / kCols);
    const unsigned grid = (unsigned)tiles * (unsigned)a.kv.kv_heads * (unsigned)a.kv.batch;
    if (a.kv.head_dim == 64)
        kv4_attention_kernel<64, 64><<<grid, kThreads, 0, stream>>>(a, tiles);
    else if (a.kv.group_size == 64)
        kv4_attention_kernel<128, 64><<<grid, kThreads, 0, stream>>>(a, tiles);
    else
        kv4_attention_kernel<128, 128><<<grid, kThreads, 0, stream>>>(a, tiles);
    return hipGetLastError();
}

}  // namespace cider
