// Low-rank adapters beside a projection (include/cider.h, cider_lora_add):
//   t[r, j] = sum_k A[slot, j, k] x[r, k]
//   y[r, n] = y_in[r, n] + scale[slot] sum_j B[slot, n, j] t[r, s(n) R + j]
// for rows r of segments that each have a slot, s(n) the slice of output n, R the
// rank.  Two launches: `down` leaves t, in parts over the inputs k, in the workspace,
// `up` adds the parts, multiplies by B and adds y_in.
//
// Shape.  Both are products on the matrix cores (v_mfma_f32_16x16x32) with the
// adapter's rows as the left operand and tokens as columns, operands loaded as they
// lie in memory: 8 consecutive inputs of a row are a lane's 16 bytes.  No LDS but for
// joining a workgroup's 4 wavefronts, which take a quarter of the inputs each.
// A lane of `up` takes the rows of B in the order that leaves it 16 consecutive
// outputs of one token, so y_in and y move 16 bytes a lane and a whole line a token.
//
// Rounding.  t is fp32; times the scale it goes to the second product as two 16-bit
// numbers, high and low, one behind the other along the summed axis with B's row
// repeated: 16 bits (bf16) or 22 (fp16, after a power of two of the token that keeps
// it in range) of t, and for ranks up to 16 no more products than t rounded once
// would take.  Sums are fp32, y is rounded once.
#include "kv4_layout.h"
#include "quant_common.h"

namespace cider {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bhalf8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ f32x4 mfma(uint4 x, uint4 y, f32x4 z)
{
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bhalf8, x), __builtin_bit_cast(bhalf8, y), z, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, x), __builtin_bit_cast(half8, y), z, 0, 0, 0);
}

// What a launch adds to the call's arguments.
struct Launch {
    int tiles;   // of 16 TT rows, of the longest segment
    int blocks;  // down: of 16 NT rows of A; up: of `per` 64-output blocks a wavefront
    int splits;  // parts of t
    int chunk;   // down: inputs of a wavefront, a multiple of 64
    int per;
    float *t;    // [splits][rows][slices * rank]
};

// A tile of a segment's rows; n 0: nothing to do.
struct Rows {
    int first, n, slot;
};
__device__ __forceinline__ Rows rows_of(const LoraArgs &a, int segment, int tile, int size)
{
    const int from = a.seg_start[segment], to = a.seg_start[segment + 1];
    Rows r = {from + tile * size, 0, a.slot[segment]};
    if (from < 0 || to < from || to > a.rows || to - from > a.max_rows)
        return r;
    const int left = to - from - tile * size;
    r.n = left < 0 ? 0 : (left < size ? left : size);
    return r;
}

template <int DT, int TT, int NT>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs a, Launch l)
{
    constexpr int U = TT + NT <= 2 ? 8 : (TT + NT <= 4 ? 4 : 2);  // steps of 32 inputs loaded at once
    __shared__ f32x4 part[4][TT * NT][64];
    unsigned id = kv4_workgroup();
    const int block = (int)(id % (unsigned)l.blocks);
    id /= (unsigned)l.blocks;
    const int split = (int)(id % (unsigned)l.splits);
    id /= (unsigned)l.splits;
    const int tile = (int)(id % (unsigned)l.tiles), segment = (int)(id / (unsigned)l.tiles);
    if (segment >= a.segments)
        return;
    const Rows r = rows_of(a, segment, tile, 16 * TT);
    if (r.n == 0 || (unsigned)r.slot >= (unsigned)a.slots)
        return;
    const int lane = threadIdx.x & 63, c = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int width = a.slices * a.rank;  // rows of A
    const uint16_t *x[TT], *w[NT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const int row = 16 * i + c < r.n ? 16 * i + c : r.n - 1;
        x[i] = a.x + (int64_t)(r.first + row) * a.ldx + 8 * q;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int j = (block * NT + i) * 16 + c;
        w[i] = a.a + ((int64_t)r.slot * width + (j < width ? j : width - 1)) * a.inputs + 8 * q;
    }
    const int k0 = (split * 4 + wave) * l.chunk, k1 = k0 + l.chunk < a.inputs ? k0 + l.chunk : a.inputs;
    f32x4 acc[TT][NT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            acc[i][j] = f32x4{0, 0, 0, 0};
    struct Steps {
        uint4 x[U][TT], w[U][NT];
    };
    auto load = [&](Steps &s, int k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = k + 32 * u < k1 ? k + 32 * u : k1 - 32;  // past the end: again what is there
#pragma unroll
            for (int i = 0; i < TT; ++i)
                s.x[u][i] = *reinterpret_cast<const uint4 *>(x[i] + at);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                s.w[u][i] = *reinterpret_cast<const uint4 *>(w[i] + at);
        }
    };
    auto multiply = [&](const Steps &s, int k) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k + 32 * u < k1) {
#pragma unroll
                for (int i = 0; i < TT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[i][j] = mfma<DT>(s.w[u][j], s.x[u][i], acc[i][j]);
            }
    };
    if (k0 < k1) {
        Steps one, two;
        load(one, k0);
        for (int k = k0; k < k1; k += 64 * U) {
            if (k + 32 * U < k1)
                load(two, k + 32 * U);
            multiply(one, k);
            if (k + 64 * U < k1)
                load(one, k + 64 * U);
            multiply(two, k + 32 * U);
        }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            part[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    // lane (q, c) has rows 4 q .. 4 q + 3 of a block of A for token c
#pragma unroll
    for (int n = 0; n < TT * NT; n += 4) {
        const int at = n + wave;
        if (at >= TT * NT)
            break;
        const f32x4 sum = (part[0][at][lane] + part[1][at][lane]) + (part[2][at][lane] + part[3][at][lane]);
        const int row = at / NT * 16 + c, j = (block * NT + at % NT) * 16 + 4 * q;
        if (row < r.n && j < width)
            *reinterpret_cast<f32x4 *>(l.t + ((int64_t)split * a.rows + r.first + row) * width + j) = sum;
    }
}

// STEPS: products of 32 along 2 R numbers, the high halves of t and then the low ones.
template <int DT, int TT, int STEPS>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a, Launch l)
{
    constexpr int OUT = DT == DT_BF16 ? OUT_BF16 : OUT_F16;
    unsigned id = kv4_workgroup();
    const int lane = threadIdx.x & 63, c = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int group = (int)(id % (unsigned)l.blocks);
    id /= (unsigned)l.blocks;
    const int tile = (int)(id % (unsigned)l.tiles), segment = (int)(id / (unsigned)l.tiles);
    if (segment >= a.segments)
        return;
    const Rows r = rows_of(a, segment, tile, 16 * TT);
    const bool adapted = (unsigned)r.slot < (unsigned)a.slots;
    if (r.n == 0 || (!adapted && a.y == a.y_in))
        return;
    const int outputs = a.ends[a.slices - 1], R = a.rank, width = a.slices * R;
    int row[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
        row[i] = r.first + (16 * i + c < r.n ? 16 * i + c : r.n - 1);

    // which 8 numbers of t, and of a row of B, each step's operand of the lane has
    int at[STEPS];
    bool low[STEPS], some[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int k = 32 * s + 8 * q;
        some[s] = k < 2 * R;
        low[s] = k >= R;
        at[s] = !some[s] ? 0 : (low[s] ? k - R : k);
    }
    const float scale = !adapted ? 0.0f : (a.scale ? a.scale[r.slot] : 1.0f);
    uint4 t[TT][STEPS];
    int exponent[TT] = {};
    auto load_t = [&](int slice) {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            float v[STEPS][8], top = 0.0f;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const float *from = l.t + (int64_t)row[i] * width + slice * R + at[s];
                f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
                for (int p = 0; p < l.splits; ++p) {
                    lo += *reinterpret_cast<const f32x4 *>(from + (int64_t)p * a.rows * width);
                    hi += *reinterpret_cast<const f32x4 *>(from + (int64_t)p * a.rows * width + 4);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[s][e] = (e < 4 ? lo[e] : hi[e - 4]) * scale;
                    top = __builtin_fmaxf(top, __builtin_fabsf(v[s][e]));
                }
            }
            exponent[i] = 0;
            if constexpr (DT == DT_F16) {  // the token's largest to [2^13, 2^14)
                top = __builtin_fmaxf(top, __shfl_xor(top, 16));
                top = __builtin_fmaxf(top, __shfl_xor(top, 32));
                exponent[i] = top > 0.0f && top < __builtin_inff() ? __builtin_amdgcn_frexp_expf(top) - 14 : 0;
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float u[2];
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const float x = __builtin_amdgcn_ldexpf(v[s][2 * e + f], -exponent[i]);
                        u[f] = low[s] ? x - widen_bits<DT>(out_bits<OUT>(x)) : x;
                    }
                    o[e] = some[s] ? pack2<OUT>(u[0], u[1]) : 0u;
                }
                t[i][s] = uint4{o[0], o[1], o[2], o[3]};
            }
        }
    };

    const int first = (group * 4 + wave) * l.per * 64;
    int slice = -1;
    for (int n0 = first; n0 < first + l.per * 64 && n0 < outputs; n0 += 64) {
        f32x4 acc[TT][4];
        uint4 in[TT][2];
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                in[i][h] = *reinterpret_cast<const uint4 *>(a.y_in + (int64_t)row[i] * a.ldy_in + n0 + 16 * q + 8 * h);
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = f32x4{0, 0, 0, 0};
        if (adapted) {
            uint4 b[4][STEPS];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + c / 4 * 16 + 4 * j + c % 4;
                const uint16_t *from = a.b + ((int64_t)r.slot * outputs + n) * R;
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
                    b[j][s] = *reinterpret_cast<const uint4 *>(from + at[s]);
            }
            int now = 0;
            while (n0 >= a.ends[now])
                ++now;
            if (now != slice) {
                slice = now;
                load_t(slice);
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < TT; ++i)
                        acc[i][j] = mfma<DT>(b[j][s], t[i][s], acc[i][j]);
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (16 * i + c >= r.n)
                continue;
            uint16_t *to = a.y + (int64_t)row[i] * a.ldy + n0 + 16 * q;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t u[4] = {in[i][h].x, in[i][h].y, in[i][h].z, in[i][h].w};
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int m = 8 * h + 2 * e;
                    const float d0 = __builtin_amdgcn_ldexpf(acc[i][m / 4][m % 4], exponent[i]);
                    const float d1 = __builtin_amdgcn_ldexpf(acc[i][m / 4][m % 4 + 1], exponent[i]);
                    o[e] = adapted ? pack2<OUT>(widen_bits<DT>(u[e]) + d0, widen_bits<DT>(u[e] >> 16) + d1) : u[e];
                }
                *reinterpret_cast<uint4 *>(to + 8 * h) = uint4{o[0], o[1], o[2], o[3]};
            }
        }
    }
}

constexpr int kMaxSplits = 16;

// Rows of A that a workgroup of `down` has, in blocks of 16.
int down_blocks(const LoraArgs &a)
{
    const int all = (a.slices * a.rank + 15) / 16;
    return all >= 8 ? 8 : (all >= 4 && all != 6 ? 4 : all);
}

Launch plan_down(const LoraArgs &a)
{
    Launch l{};
    const int size = a.max_rows > 16 ? 32 : 16, nt = down_blocks(a);
    l.tiles = (int)(((int64_t)a.max_rows + size - 1) / size);
    l.blocks = (a.slices * a.rank + 16 * nt - 1) / (16 * nt);
    // parts: workgroups for the compute units, wavefronts of 128 inputs and more
    const int64_t units = (int64_t)a.segments * l.tiles * l.blocks;
    int64_t splits = 1024 / units;
    const int64_t most = a.inputs / 512 < kMaxSplits ? a.inputs / 512 : kMaxSplits;
    splits = splits > most ? most : splits;
    l.splits = splits < 1 ? 1 : (int)splits;
    return l;
}

size_t part_bytes(const LoraArgs &a) { return (size_t)a.rows * a.slices * a.rank * sizeof(float); }

template <int DT, int TT>
hipError_t launch_down(const LoraArgs &a, const Launch &l, hipStream_t stream)
{
    const unsigned grid = (unsigned)a.segments * (unsigned)l.tiles * (unsigned)l.blocks * (unsigned)l.splits;
    switch (down_blocks(a)) {
    case 1: return kv4_launch(lora_down_kernel<DT, TT, 1>, grid, 256, stream, a, l);
    case 2: return kv4_launch(lora_down_kernel<DT, TT, 2>, grid, 256, stream, a, l);
    case 3: return kv4_launch(lora_down_kernel<DT, TT, 3>, grid, 256, stream, a, l);
    case 4: return kv4_launch(lora_down_kernel<DT, TT, 4>, grid, 256, stream, a, l);
    case 6: return kv4_launch(lora_down_kernel<DT, TT, 6>, grid, 256, stream, a, l);
    default: return kv4_launch(lora_down_kernel<DT, TT, 8>, grid, 256, stream, a, l);
    }
}

template <int DT, int TT>
hipError_t launch_up(const LoraArgs &a, Launch l, hipStream_t stream)
{
    l.tiles = (int)(((int64_t)a.max_rows + 16 * TT - 1) / (16 * TT));
    const int64_t all = a.ends[a.slices - 1] / 64, units = (int64_t)a.segments * l.tiles;
    int64_t per = all * units / 4096;
    per = per < 1 ? 1 : (per > 8 ? 8 : per);
    l.per = (int)per;
    l.blocks = (int)((all + 4 * per - 1) / (4 * per));
    const unsigned grid = (unsigned)a.segments * (unsigned)l.tiles * (unsigned)l.blocks;
    if (a.rank <= 16)
        return kv4_launch(lora_up_kernel<DT, TT, 1>, grid, 256, stream, a, l);
    if (a.rank <= 32)
        return kv4_launch(lora_up_kernel<DT, TT, 2>, grid, 256, stream, a, l);
    if (a.rank <= 64 || TT > 2)
        return kv4_launch(lora_up_kernel<DT, TT, 4>, grid, 256, stream, a, l);
    return kv4_launch(lora_up_kernel<DT, (TT > 2 ? 2 : TT), 8>, grid, 256, stream, a, l);
}

template <int DT>
hipError_t launch(const LoraArgs &a, const Launch &l, hipStream_t stream)
{
    const hipError_t e = a.max_rows > 16 ? launch_down<DT, 2>(a, l, stream) : launch_down<DT, 1>(a, l, stream);
    if (e != hipSuccess)
        return e;
    if (a.max_rows <= 16)
        return launch_up<DT, 1>(a, l, stream);
    return a.max_rows <= 32 || a.rank > 64 ? launch_up<DT, 2>(a, l, stream) : launch_up<DT, 4>(a, l, stream);
}

}  // namespace

size_t lora_least_workspace(const LoraArgs &a) { return part_bytes(a); }

size_t lora_workspace(const LoraArgs &a) { return part_bytes(a) * plan_down(a).splits; }

hipError_t launch_lora_add(const LoraArgs &a, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    Launch l = plan_down(a);
    const size_t room = workspace_bytes / part_bytes(a);
    l.splits = (size_t)l.splits > room ? (int)room : l.splits;
    const int steps = a.inputs / 64;
    l.chunk = (steps + 4 * l.splits - 1) / (4 * l.splits) * 64;
    l.splits = (steps * 64 + 4 * l.chunk - 1) / (4 * l.chunk);
    l.t = static_cast<float *>(workspace);
    return a.dtype == DT_BF16 ? launch<DT_BF16>(a, l, stream) : launch<DT_F16>(a, l, stream);
}

}  // namespace cider
