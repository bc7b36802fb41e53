// Norm and rotation of a step's queries and keys, and the keys' and values' way
// into the 4-bit cache, in one pass (include/cider.h, cider_kv4_append_rotated).
//
// Mathematics.  A head x [D] of a row, with weights w and r = 1 / sqrt(mean x^2 +
// eps), is n_d = x_d r w_d (without weights n = x).  Its first rot_dim elements form
// pairs (a, b), the i-th (i, i + rot_dim / 2) or (2 i, 2 i + 1), and turn by the
// table's (c, s) of the row's position on the pair's axis:
//   a' = a c - b s,   b' = b c + a s.
// q' is rounded to 16 bits once.  k' is worked out in 64 bits, rounded to fp32 once
// and quantized as kv4_cache.hip states: near the border between two codes 32 bits
// would choose the code by the order of their operations.  64-bit operations cost
// what 32-bit ones do here (4 cycles a wavefront), and k is a sixth of the values.
//
// Shape.  One workgroup per (sequence, 32 positions, kv head), as the append: it
// has that head's k and v and the group's query heads.  D / 16 lanes a head, each
// with two chunks of 8 elements that are one another's partners (chunks l and l +
// rot_dim / 16), so no value of a pair crosses lanes; a wavefront has 8 tokens, and
// a lane's 8 pairs of (c, s) stay in registers for k and all query heads.  Of up to 8
// tokens the first wavefront has the keys and the others share the query heads out (64
// single rows, G 4: 6.4 us, 9.4 with each token's heads one after the other).  v goes
// its own way, by the lanes that kv4_codes.h's exchanges want.
//
// What bounds it.  Bytes: 13400 rows of 32 + 2 x 8 heads of 128 (bf16, norms) move 296
// MB in 62 us, 4.8 TB/s, a copy's rate; the vector units work half that time.  Query
// heads are loaded one ahead (none: 1.5 us more; four: 5 % more, fewer wavefronts).  5000
// rows of 28 + 2 x 4 heads of 64, 3 axes (40 MB), take 16.7: one round of wavefronts, each
// a chain of loads, the table's entries one by one, and 64-bit operations, which with
// heads of 64 both halves of a wavefront do for the same 8 keys.  Dealing the query heads
// to more workgroups made both slower (the pairs' entries loaded again).  One row: 4.2,
// the launch and three loads in a row.
#include "kv4_codes.h"

namespace cider {
namespace {

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v)
{
    const uint2 u = __builtin_bit_cast(uint2, v);
    const uint2 w = {(uint32_t)__builtin_amdgcn_update_dpp((int)u.x, (int)u.x, CTRL, 0xF, 0xF, false),
                     (uint32_t)__builtin_amdgcn_update_dpp((int)u.y, (int)u.y, CTRL, 0xF, 0xF, false)};
    return v + __builtin_bit_cast(double, w);
}

// Over the 4 or 8 lanes of a head; every lane has the result.
template <int L>
__device__ __forceinline__ double head_sum(double v)
{
    v = dpp_add<0xB1>(v);  // quad_perm [1,0,3,2]
    v = dpp_add<0x4E>(v);  // quad_perm [2,3,0,1]
    return L == 8 ? dpp_add<0x141>(v) : v;  // row_half_mirror
}
template <int L>
__device__ __forceinline__ uint32_t head_max(uint32_t v)
{
    v = max_dpp_u<0xB1>(v);
    v = max_dpp_u<0x4E>(v);
    return L == 8 ? max_dpp_u<0x141>(v) : v;
}

// 1 / sqrt(v) of a normal number: the hardware's (2^-23 at the least) and two steps,
// each of which squares the error.  Of infinity 0, which the steps would make NaN.
__device__ __forceinline__ double inverse_root(double v)
{
    double r = __builtin_amdgcn_rsq(v);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r = __builtin_fma(r * 0.5, __builtin_fma(-v * r, r, 1.0), r);
    return v == __builtin_inf() ? 0.0 : r;
}

// A lane's part of every head: where its two chunks are, and its pairs' turns.
struct Share {
    int chunk[2];
    bool turns;
    float2 cs[8];
};

// (The squares are summed in 64 bits: those of large bf16 values leave fp32.)
template <int L, typename T>
__device__ __forceinline__ void norm(T (&x)[2][8], const float (&w)[2][8], float eps)
{
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum = __builtin_fma((double)x[c][e], (double)x[c][e], sum);
    const T r = (T)inverse_root(head_sum<L>(sum) * (1.0 / (16 * L)) + (double)eps);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[c][e] = x[c][e] * r * (T)w[c][e];
}

template <typename T>
__device__ __forceinline__ void turn(T &a, T &b, float2 cs)
{
    const T c = cs.x, s = cs.y, was = a;
    a = a * c - b * s;
    b = b * c + was * s;
}

template <bool INTERLEAVED, typename T>
__device__ __forceinline__ void turn(T (&x)[2][8], const Share &t)
{
    if (!t.turns)
        return;
    if constexpr (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            turn(x[e / 4][e % 4 * 2], x[e / 4][e % 4 * 2 + 1], t.cs[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            turn(x[0][e], x[1][e], t.cs[e]);
    }
}

template <int DT, typename T>
__device__ __forceinline__ void widen(const uint4 (&w)[2], T (&x)[2][8])
{
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[c][e] = widen_bits<DT>(e & 1 ? u[e / 2] >> 16 : u[e / 2]);
    }
}

__device__ __forceinline__ void load_weights(const float *w, const Share &t, float (&x)[2][8])
{
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float4 v = *reinterpret_cast<const float4 *>(w + 8 * t.chunk[c] + 4 * e);
            x[c][4 * e] = v.x;
            x[c][4 * e + 1] = v.y;
            x[c][4 * e + 2] = v.z;
            x[c][4 * e + 3] = v.w;
        }
}

// The table's entries of the lane's pairs for the token at position p, row `row`.
template <bool INTERLEAVED>
__device__ __forceinline__ void load_turns(const Kv4Rotation &r, int rows, int p, int64_t row, Share &t)
{
    if (!t.turns)
        return;
    const int pairs = r.rot_dim / 2;
    // first pair of the lane's first four and last four
    const int at[2] = {INTERLEAVED ? 4 * t.chunk[0] : 8 * t.chunk[0],
                       INTERLEAVED ? 4 * t.chunk[1] : 8 * t.chunk[0] + 4};
    const int most = r.table_len - 1;
    auto entry = [&](int position) {
        const int q = position < 0 ? 0 : (position > most ? most : position);
        return r.table + (int64_t)q * pairs;
    };
    if (r.axes == 1) {
        const float2 *from = entry(r.positions ? r.positions[row] : p);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 v = *reinterpret_cast<const float4 *>(from + at[h] + 2 * e);
                t.cs[4 * h + 2 * e] = float2{v.x, v.y};
                t.cs[4 * h + 2 * e + 1] = float2{v.z, v.w};
            }
        return;
    }
    const float2 *from[kMostAxes];
#pragma unroll
    for (int x = 0; x < kMostAxes; ++x)
        from[x] = entry(r.positions[(int64_t)(x < r.axes ? x : 0) * rows + row]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int pair = at[e / 4] + e % 4;
        const int x = (int)((pair < 32 ? r.pair_axis_low : r.pair_axis_high) >> 2 * (pair % 32)) & 3;
        const float2 *f = x & 1 ? (x & 2 ? from[3] : from[1]) : (x & 2 ? from[2] : from[0]);
        t.cs[e] = f[pair];
    }
}

// The keys of 8 tokens of a wavefront (D 64: the lower half of it).
template <int D, int GS, int DT, bool INTERLEAVED>
__device__ __forceinline__ void put_key(const Kv4Rotation &r, const uint4 (&raw)[2], const Share &t, const float (&w)[2][8],
                                        uint8_t *block, int token, bool store, int l)
{
    constexpr int L = D / 16, NG = D / GS;
    double x[2][8];
    widen<DT>(raw, x);
    if (r.k_weight)
        norm<L>(x, w, r.eps);
    turn<INTERLEAVED>(x, t);
    // the largest magnitudes by their bits, NaN among them: a maximum of numbers leaves NaN
    // out, and a key without a number would come to be one of zeros
    float f[2][8], scale[NG];
    uint32_t top[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g)
        top[g] = 0;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[c][e] = (float)x[c][e];
            const uint32_t u = __builtin_bit_cast(uint32_t, f[c][e]) & 0x7FFFFFFFu;
            m = u > m ? u : m;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)
            top[g] = t.chunk[c] / (GS / 8) == g && m > top[g] ? m : top[g];
    }
#pragma unroll
    for (int g = 0; g < NG; ++g)
        scale[g] = __builtin_bit_cast(float, head_max<L>(top[g])) / quant_divisor<4>();
    uint32_t *kcode = reinterpret_cast<uint32_t *>(block);
    float *kscale = reinterpret_cast<float *>(block + kv4_scale_offset(D));
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float s = NG == 2 && t.chunk[c] / (GS / 8) ? scale[NG - 1] : scale[0];
        const uint32_t code = int4_codes(f[c], s, __builtin_amdgcn_rcpf(s));
        if (store)
            kcode[token * (D / 8) + t.chunk[c] % 4 * (D / 32) + t.chunk[c] / 4] = code;
    }
    if (store && l == 0) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
            kscale[g * kPageTokens + token] = scale[g];
    }
}

// A head of q.
template <int D, int DT, bool INTERLEAVED>
__device__ __forceinline__ void put_query(const Kv4Rotation &r, const uint4 (&raw)[2], const Share &t,
                                          const float (&w)[2][8], uint16_t *to, bool there)
{
    constexpr int OUT = DT == DT_BF16 ? OUT_BF16 : OUT_F16;
    float x[2][8];
    widen<DT>(raw, x);
    if (r.q_weight)
        norm<D / 16>(x, w, r.eps);
    turn<INTERLEAVED>(x, t);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint4 o;
        o.x = pack2<OUT>(x[c][0], x[c][1]);
        o.y = pack2<OUT>(x[c][2], x[c][3]);
        o.z = pack2<OUT>(x[c][4], x[c][5]);
        o.w = pack2<OUT>(x[c][6], x[c][7]);
        *reinterpret_cast<uint4 *>(to + 8 * t.chunk[c]) = there ? o : uint4{0, 0, 0, 0};
    }
}

template <int D, int GS, int DT, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void kv4_rotate_kernel(Kv4Args a, Kv4Rotation r, Kv4Rows io, int spans)
{
    constexpr int CH = D / 8, PT = D / 64, L = D / 16;
    constexpr int HEADS = 8 / L;  // query heads that a wavefront works on at once
    Place w;
    if (!place_of(a, spans, w))
        return;
    const int lane = threadIdx.x % 64;
    const int j = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const int half = (w.base / kSpan) & 1;  // which 32 tokens of the page
    uint8_t *block = block_of<D, GS>(a, w);

    // v: the wavefront's tokens are 16 b + 4 j + i
    uint32_t mask = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int p = w.base + e / 4 * 16 + 4 * j + e % 4;
        mask |= (p >= w.lo && p < w.hi ? 15u : 0u) << (4 * e);
    }
    const int c8 = lane % CH;
    uint4 vx[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int p = w.base + token_of<D>(lane, j, i);
        vx[i] = uint4{0, 0, 0, 0};
        if (p >= w.lo && p < w.hi)
            vx[i] = nt_load(io.v + (p + w.shift) * io.ldv + w.h * D + c8 * 8);
    }

    // q and k.  Many tokens: the wavefront has 8 of them, each with its key and then its
    // query heads.  Up to 8 in all: the first wavefront has their keys, the others share
    // their query heads out.
    const int l = lane % L, G = io.q_heads / a.kv_heads;
    const bool few = w.hi - w.lo <= 8;
    const int sub = few ? 0 : lane / (8 * L);
    Share s;
    s.turns = l < r.rot_dim / 16;
    s.chunk[0] = s.turns ? l : 2 * l;  // rot_dim / 8 + 2 (l - rot_dim / 16)
    s.chunk[1] = s.turns ? l + r.rot_dim / 16 : 2 * l + 1;
    auto load = [&](uint4 (&x)[2], const uint16_t *head) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
            x[c] = nt_load(head + 8 * s.chunk[c]);
    };
    float weight[2][8];
    uint4 x[2];
    auto key = [&](int p, bool mine) {
        const int64_t row = (mine ? p : w.lo) + w.shift;
        load(x, io.k + row * io.ldk + w.h * D);
        load_turns<INTERLEAVED>(r, a.rows, p, row, s);
        if (r.k_weight)
            load_weights(r.k_weight, s, weight);
        if (block)
            put_key<D, GS, DT, INTERLEAVED>(r, x, s, weight, block, half * kSpan + p - w.base, mine && p >= 0 && sub == 0, l);
        if (r.q_weight)
            load_weights(r.q_weight, s, weight);
    };
    if (!few) {
        if (w.base + 8 * j < w.hi && w.base + 8 * j + 8 > w.lo) {
            const int p = w.base + 8 * j + lane / L % 8;
            const bool mine = p >= w.lo && p < w.hi;
            const int64_t row = (mine ? p : w.lo) + w.shift;
            const uint16_t *from = io.q + row * io.ldq + w.h * G * D;
            uint16_t *to = io.q_out + row * io.ldo + w.h * G * D;
            uint4 next[2] = {};  // the next head, one ahead; the first before the key
            if (G > 0)
                load(next, from + (sub < G ? sub : G - 1) * D);
            key(p, mine);
            for (int g0 = 0; g0 < G; g0 += HEADS) {
                const int g = g0 + sub, after = g + HEADS < G ? g + HEADS : G - 1;
                x[0] = next[0];
                x[1] = next[1];
                if (g0 + HEADS < G)
                    load(next, from + after * D);
                if (mine && g < G)
                    put_query<D, DT, INTERLEAVED>(r, x, s, weight, to + g * D, p >= 0);
            }
        }
    } else if (j == 0) {
        const int p = w.lo + lane / L;
        key(p, p < w.hi);
    } else {
        if (r.q_weight)
            load_weights(r.q_weight, s, weight);
        const int count = (w.hi - w.lo) * G;
        for (int i0 = (j - 1) * (64 / L); i0 < count; i0 += 3 * (64 / L)) {
            const int i = i0 + lane / L, at = i < count ? i : i0;
            const int p = w.lo + at / G, head = w.h * G + at % G;
            const int64_t row = p + w.shift;
            load(x, io.q + row * io.ldq + head * D);
            load_turns<INTERLEAVED>(r, a.rows, p, row, s);
            if (i < count)
                put_query<D, DT, INTERLEAVED>(r, x, s, weight, io.q_out + row * io.ldo + head * D, p >= 0);
        }
    }

    if (mask == 0 || !block)
        return;
    float *vscale = reinterpret_cast<float *>(block + kv4_scale_offset(D)) + kPageTokens * (D / GS);
    uint32_t *vout = reinterpret_cast<uint32_t *>(block + kv4_v_offset(D)) + half * 4 * D + dword_of<D>(lane, j);
    uint32_t old[PT] = {};  // what a partly filled dword keeps
    if (mask != ~0u)
        load_dwords(old, vout);
    uint32_t vcode[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int t = token_of<D>(lane, j, i), p = w.base + t;
        const float s = seventh(widen_bits<DT>(run_max<GS / 8>(chunk_absmax_bits(vx[i]))));
        vcode[i] = int4_codes<DT>(vx[i], s, __builtin_amdgcn_rcpf(s));
        if (p >= w.lo && p < w.hi && c8 % (GS / 8) == 0)
            vscale[c8 / (GS / 8) * kPageTokens + half * kSpan + t] = s;
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

}  // namespace

hipError_t launch_kv4_append_rotated(const Kv4Args &a, const Kv4Rotation &r, const Kv4Rows &io, int dtype,
                                     hipStream_t stream)
{
    const int spans = spans_of(a);
    const unsigned grid = (unsigned)spans * (unsigned)a.kv_heads * (unsigned)a.batch;
    return with_geometry(a, dtype, [&](auto D, auto GS, auto DT) {
        auto *kernel = r.interleaved ? kv4_rotate_kernel<D(), GS(), DT(), true> : kv4_rotate_kernel<D(), GS(), DT(), false>;
        return kv4_launch(kernel, grid, kThreads, stream, a, r, io, spans);
    });
}

}  // namespace cider
