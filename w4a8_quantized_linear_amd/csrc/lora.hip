// Low-rank adapters beside a projection (include/cider.h, cider_lora_add):
//   t[r, j] = sum_k A[slot, j, k] x[r, k]
//   y[r, n] = y_in[r, n] + scale[slot] sum_j B[slot, n, j] t[r, s(n) R + j]
// for rows r of segments that each have a slot, s(n) the slice of output n, R the
// rank.  `down` leaves t, in parts over the inputs k, in the workspace; `up` adds the
// parts, multiplies by B and adds y_in; `step` does both for few rows.
//
// Shape.  Both products run on the matrix cores (v_mfma_f32_16x16x32) with the adapter's
// rows as the left operand and tokens as columns, 8 consecutive numbers of a row a lane's
// operand.  The operands' lanes go from row to row, which the load path takes four times
// as long as lanes that go along rows, so that what is long (x, A, B past rank 32) comes
// by rows and through LDS, and y leaves by whole lines.
//
// Rounding.  t is fp32; times the scale it goes to the second product as two 16-bit
// numbers, high and low, one behind the other along the summed axis with B's row
// repeated: 16 bits (bf16) or 22 (fp16, after a power of two of the token and slice that
// keeps t in range; of numbers below 2^-16 of the largest there, what is above 2^-38 of
// that), and for ranks up to 16 no more products than t rounded once would take.  Sums
// are fp32, y is rounded once: against 64 bits outputs are off by that rounding alone
// (fp16 2.1e-4, bf16 1.6e-3).
//
// What bounds it.  Many rows: bytes.  8400 rows of 4096 inputs beside 6144 outputs (bf16,
// rank 16): `down` 21.9 us, 14 at 5 TB/s, a wavefront's few loads in
// flight against their latency; `up` 48.7, where a copy by the same pattern takes 45 and
// one at 5 TB/s 41.  2000 rows beside 24576 outputs (fp16, rank 64): 13.0 and 50.5, the
// latter 39 as a copy.  Few rows: latency, one chain of loads (the segment, then x and A, or B
// and y) and a barrier each: 1 row beside 4096 outputs 6.8 us, 64 with 24 adapters beside
// 6144 9.6.
#include "kv4_layout.h"
#include "quant_common.h"

namespace cider {
namespace {

typedef __bf16 bhalf8 __attribute__((ext_vector_type(8)));

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 x, u32x4 y, f32x4 z)
{
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bhalf8, x), __builtin_bit_cast(bhalf8, y), z, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, x), __builtin_bit_cast(half8, y), z, 0, 0, 0);
}

// Lanes of a wavefront have written to LDS what others read.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// What a launch adds to the call's arguments.
struct Launch {
    int tiles;   // of 16 TT rows, of the longest segment
    int blocks;  // down: of 16 NT rows of A; up: of a workgroup's outputs, in all slices
    int splits;  // parts of t
    int chunk;   // down: inputs of a wavefront, a multiple of 64
    int per;     // up: blocks of outputs of a wavefront
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

// The products of 16 TT rows of x with 16 NT rows of A, the j-th of the slot's `width`
// and those behind it, over the inputs k0 .. k1 - 1, by one wavefront.  Both go through
// its LDS: memory is read by consecutive lanes, 8 and more to a row, where the operands'
// lanes go from row to row, which the load path takes a quarter as fast (8400 rows of
// 4096 inputs 36 us by the operands' lanes, 24 so).  KS: times 64 inputs loaded at once.
// Lane (q, c) ends with rows 4 q .. 4 q + 3 of a block of A for token c.
template <int TT, int NT, int KS>
constexpr int kStageWords = 16 * (TT + NT) * 8 * KS;
template <int DT, int TT, int NT, int KS>
__device__ __forceinline__ void multiply_rows(const LoraArgs &a, const Rows &r, int j0, int width, int k0, int k1, int lane,
                                              u32x4 *stage, f32x4 (&acc)[TT][NT])
{
    constexpr int CHUNKS = 8 * KS, LOADS = kStageWords<TT, NT, KS> / 64;
    if (k0 >= k1)
        return;
    const int c = lane % 16, q = lane / 16;
    // the lane's i-th word is chunk (64 i + lane) % CHUNKS of row (64 i + lane) / CHUNKS
    const uint16_t *from[LOADS];
    const int chunk = lane % CHUNKS;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = (64 * i + lane) / CHUNKS;
        if (row < 16 * TT) {
            from[i] = a.x + (int64_t)(r.first + (row < r.n ? row : r.n - 1)) * a.ldx;
        } else {
            const int j = j0 + row - 16 * TT;
            from[i] = a.a + ((int64_t)r.slot * width + (j < width ? j : width - 1)) * a.inputs;
        }
    }
    u32x4 word[LOADS];
    auto load = [&](int k) {
        const int at = k + 8 * chunk < k1 ? k + 8 * chunk : k1 - 8;  // past the end: anything that is there
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            word[i] = *reinterpret_cast<const u32x4 *>(from[i] + at);
    };
    load(k0);
    for (int k = k0; k < k1; k += 64 * KS) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int row = (64 * i + lane) / CHUNKS;
            stage[row * CHUNKS + (chunk ^ row % 8)] = word[i];
        }
        wave_fence();
        if (k + 64 * KS < k1)
            load(k + 64 * KS);
#pragma unroll
        for (int s = 0; s < 2 * KS; ++s)
            if (k + 32 * s < k1) {
                u32x4 x[TT];
                const int at = (4 * s + q) ^ c % 8;
#pragma unroll
                for (int i = 0; i < TT; ++i)
                    x[i] = stage[(16 * i + c) * CHUNKS + at];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const u32x4 w = stage[(16 * (TT + j) + c) * CHUNKS + at];
#pragma unroll
                    for (int i = 0; i < TT; ++i)
                        acc[i][j] = mfma<DT>(w, x[i], acc[i][j]);
                }
            }
        wave_fence();
    }
}

// A workgroup has 16 TT rows of x and 16 NT rows of A, each of its wavefronts a quarter
// of the split's inputs.
template <int DT, int TT, int NT>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs a, Launch l)
{
    constexpr int KS = TT + NT <= 2 ? 4 : (TT + NT <= 4 ? 2 : 1);
    constexpr int STAGE = kStageWords<TT, NT, KS>, PART = TT * NT * 64;  // of a wavefront
    __shared__ u32x4 lds[4][STAGE > PART ? STAGE : PART];
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
    const int k0 = (split * 4 + wave) * l.chunk, k1 = k0 + l.chunk < a.inputs ? k0 + l.chunk : a.inputs;
    f32x4 acc[TT][NT] = {};
    multiply_rows<DT, TT, NT, KS>(a, r, block * NT * 16, width, k0, k1, lane, lds[wave], acc);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            lds[wave][(i * NT + j) * 64 + lane] = __builtin_bit_cast(u32x4, acc[i][j]);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < TT * NT; n += 4) {
        const int at = n + wave;
        if (at >= TT * NT)
            break;
        auto part = [&](int w) { return __builtin_bit_cast(f32x4, lds[w][at * 64 + lane]); };
        const f32x4 sum = (part(0) + part(1)) + (part(2) + part(3));
        const int row = at / NT * 16 + c, j = (block * NT + at % NT) * 16 + 4 * q;
        if (row < r.n && j < width)
            *reinterpret_cast<f32x4 *>(l.t + ((int64_t)split * a.rows + r.first + row) * width + j) = sum;
    }
}

// Of a token whose largest |t| has these bits: 2^-exponent takes it to [2^13, 2^14).
// Not below -100: what is smaller yet, times fp16 numbers, is nothing to an fp16 output,
// and 2^exponent stays a normal number.  Of a token with an infinite t every output is
// infinite or NaN; there the exponent is the greatest, and its other numbers stay finite.
__device__ __forceinline__ int token_exponent(uint32_t top)
{
    const float x = __builtin_bit_cast(float, top);
    const int e = x > 0.0f ? (x < __builtin_inff() ? __builtin_amdgcn_frexp_expf(x) : 128) - 14 : 0;
    return e < -100 ? -100 : e;
}

// Two numbers of t, times 2^by, as high and low halves.  High is within the type's finite
// numbers, so that of infinity low is infinite and not infinity less itself, and of what
// bf16 would round to infinity low is the rest.
template <int OUT>
__device__ __forceinline__ void halves(float x, float y, int by, uint32_t &high, uint32_t &low)
{
    constexpr int DT = OUT == OUT_BF16 ? DT_BF16 : DT_F16;
    constexpr float kEnd = OUT == OUT_BF16 ? 0x1.FEp127f : 65504.0f;
    x = __builtin_amdgcn_ldexpf(x, by);
    y = __builtin_amdgcn_ldexpf(y, by);
    high = pack2<OUT>(__builtin_amdgcn_fmed3f(x, -kEnd, kEnd), __builtin_amdgcn_fmed3f(y, -kEnd, kEnd));
    low = pack2<OUT>(x - widen_bits<DT>(high), y - widen_bits<DT>(high >> 16));
}

// What the lane next to it has.
__device__ __forceinline__ uint32_t neighbour(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xF, 0xF, false);  // quad_perm [1,0,3,2]
}

constexpr int kBlock = 64;  // outputs

// A workgroup's slice and its outputs there, `span` at most: begin .. end - 1.
struct Outputs {
    int slice, begin, end;
};
__device__ __forceinline__ Outputs outputs_of(const LoraArgs &a, int group, int span)
{
    Outputs o = {0, group * span, 0};
    int from = 0;
    for (; o.begin >= a.ends[o.slice] - from; ++o.slice) {
        o.begin -= (a.ends[o.slice] - from + span - 1) / span * span;
        from = a.ends[o.slice];
    }
    o.begin += from;
    o.end = o.begin + span < a.ends[o.slice] ? o.begin + span : a.ends[o.slice];
    return o;
}

// A wavefront's blocks of 64 outputs for 16 TT rows.  STEPS: products of 32 along 2 R
// numbers, the high halves of t and then the low ones, which are in LDS as operands; NB:
// blocks of 16 outputs whose rows of B are in registers at once.  The rows of B are taken
// in the order that leaves a lane 8 consecutive outputs of 32, and neighbouring lanes
// exchange theirs, so that y is written by whole lines.
template <int DT, int TT, int NB, int STEPS>
struct Block {
    const LoraArgs &a;
    const Rows r;
    const bool adapted;
    const int c, q;
    u32x4 in[TT][2], b[NB][STEPS];

    __device__ __forceinline__ Block(const LoraArgs &a, const Rows &r, bool adapted, int lane)
        : a(a), r(r), adapted(adapted), c(lane % 16), q(lane / 16)
    {
    }
    __device__ __forceinline__ void load_b(int n0, int pass)
    {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int at = NB * pass + j, n = n0 + at / 2 * 32 + c / 4 * 8 + at % 2 * 4 + c % 4, R = a.rank;
            const uint16_t *from = a.b + ((int64_t)r.slot * a.ends[a.slices - 1] + n) * R;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int k = 32 * s + 8 * q;
                b[j][s] = *reinterpret_cast<const u32x4 *>(from + (k < R ? k : (k < 2 * R ? k - R : 0)));
            }
        }
    }
    __device__ __forceinline__ void load_in(u32x4 (&in)[TT][2], int n0) const
    {
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int token = 16 * i + c < r.n ? 16 * i + c : r.n - 1;
                in[i][h] = *reinterpret_cast<const u32x4 *>(a.y_in + (int64_t)(r.first + token) * a.ldy_in + n0 + 32 * h + 8 * q);
            }
    }
    __device__ __forceinline__ void load(int n0)
    {
        load_in(in, n0);
        if (adapted)
            load_b(n0, 0);
    }
    __device__ __forceinline__ void products(const u32x4 (&half)[4 * STEPS][16 * TT], f32x4 (&acc)[4], int i, int pass)
    {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const u32x4 t = half[4 * s + q][16 * i + c];
#pragma unroll
            for (int j = 0; j < NB; ++j)
                acc[NB * pass + j] = mfma<DT>(b[j][s], t, acc[NB * pass + j]);
        }
    }
    // top: of the tokens that i counts
    __device__ __forceinline__ void put(const uint32_t *top, const f32x4 (&acc)[4], int i, int n0)
    {
        constexpr int OUT = DT == DT_BF16 ? OUT_BF16 : OUT_F16;
        const float f = DT == DT_F16 && adapted ? __builtin_amdgcn_ldexpf(1.0f, token_exponent(top[16 * i + c])) : 1.0f;
        const bool odd = c & 1;
        uint32_t o[2][4];  // of 32 outputs each, 8 of the lane's token
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t u = in[i][h][e];
                const f32x4 d = acc[2 * h + e / 2];
                o[h][e] = adapted ? pack2<OUT>(__builtin_fmaf(d[2 * (e % 2)], f, widen_bits<DT>(u)),
                                               __builtin_fmaf(d[2 * (e % 2) + 1], f, widen_bits<DT>(u >> 16)))
                                  : u;
            }
        // the even token's 64 outputs by both lanes, then the odd one's
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t other = neighbour(odd ? o[0][e] : o[1][e]);
            o[0][e] = odd ? other : o[0][e];
            o[1][e] = odd ? o[1][e] : other;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int token = 16 * i + (c & ~1) + h;
            if (token < r.n)
                *reinterpret_cast<u32x4 *>(a.y + (int64_t)(r.first + token) * a.ldy + n0 + 32 * (c & 1) + 8 * q) =
                    u32x4{o[h][0], o[h][1], o[h][2], o[h][3]};
        }
    }
    __device__ __forceinline__ void run(const u32x4 (&half)[4 * STEPS][16 * TT], const uint32_t (&top)[16 * TT], int n0)
    {
        if constexpr (NB == 4) {
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                f32x4 acc[4] = {};
                if (adapted)
                    products(half, acc, i, 0);
                put(top, acc, i, n0);
                __builtin_amdgcn_sched_barrier(0);  // one 16 tokens' registers
            }
        } else {
            f32x4 acc[TT][4] = {};
            if (adapted) {
#pragma unroll
                for (int pass = 0; pass < 4 / NB; ++pass) {
                    if (pass > 0)
                        load_b(n0, pass);
#pragma unroll
                    for (int i = 0; i < TT; ++i)
                        products(half, acc[i], i, pass);
                }
            }
#pragma unroll
            for (int i = 0; i < TT; ++i)
                put(top, acc[i], i, n0);
        }
    }
};

// Adds t's parts for a workgroup's T rows and one slice and leaves their halves in LDS,
// as operands, and the bits of their largest magnitudes (fp16).  Ends in a barrier.
template <int DT, int T, int STEPS>
__device__ __forceinline__ void halves_of(const LoraArgs &a, const Launch &l, const Rows &r, int slice, u32x4 (&half)[4 * STEPS][T],
                                          uint32_t (&top)[T])
{
    constexpr int OUT = DT == DT_BF16 ? OUT_BF16 : OUT_F16;
    constexpr int ITEMS = (T * STEPS * 2 + 255) / 256;  // of 8 numbers of t, a thread
    const float scale = a.scale ? a.scale[r.slot] : 1.0f;
    const int R = a.rank, width = a.slices * R, chunks = R / 8;
    float v[ITEMS][8];
    if (DT == DT_F16 && threadIdx.x < T)
        top[threadIdx.x] = 0;
    if constexpr (DT == DT_F16)
        __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int item = i * 256 + (int)threadIdx.x, token = item / chunks, chunk = item % chunks;
        f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
        if (token < r.n) {
            const float *from = l.t + (int64_t)(r.first + token) * width + slice * R + 8 * chunk;
#pragma unroll 4
            for (int p = 0; p < l.splits; ++p) {
                lo += *reinterpret_cast<const f32x4 *>(from + (int64_t)p * a.rows * width);
                hi += *reinterpret_cast<const f32x4 *>(from + (int64_t)p * a.rows * width + 4);
            }
        }
        float most = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[i][e] = (e < 4 ? lo[e] : hi[e - 4]) * scale;
            most = __builtin_fmaxf(most, __builtin_fabsf(v[i][e]));
        }
        if (DT == DT_F16 && token < T)
            atomicMax(&top[token], __builtin_bit_cast(uint32_t, most));
    }
    if constexpr (DT == DT_F16)
        __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int item = i * 256 + (int)threadIdx.x, token = item / chunks, chunk = item % chunks;
        if (token >= T)
            break;
        uint32_t high[4], low[4];
        const int by = DT == DT_F16 ? -token_exponent(top[token]) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            halves<OUT>(v[i][2 * e], v[i][2 * e + 1], by, high[e], low[e]);
        half[chunk][token] = u32x4{high[0], high[1], high[2], high[3]};
        half[chunks + chunk][token] = u32x4{low[0], low[1], low[2], low[3]};
    }
    for (int i = 2 * chunks * T + threadIdx.x; i < 4 * STEPS * T; i += 256)
        half[i / T][i % T] = u32x4{0, 0, 0, 0};
    __syncthreads();
}

// A workgroup has 16 TT rows and l.per blocks of 64 outputs of one slice for each of
// its wavefronts.
template <int DT, int TT, int NB, int STEPS>
__global__ __launch_bounds__(256, STEPS <= 2 ? 4 : (STEPS == 4 ? 3 : 1)) void lora_up_kernel(LoraArgs a, Launch l)
{
    constexpr int T = 16 * TT;
    __shared__ u32x4 half[4 * STEPS][T];
    __shared__ uint32_t top[T];
    unsigned id = kv4_workgroup();
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int group = (int)(id % (unsigned)l.blocks);
    id /= (unsigned)l.blocks;
    const int tile = (int)(id % (unsigned)l.tiles), segment = (int)(id / (unsigned)l.tiles);
    if (segment >= a.segments)
        return;
    const Rows r = rows_of(a, segment, tile, T);
    const bool adapted = (unsigned)r.slot < (unsigned)a.slots;
    if (r.n == 0 || (!adapted && a.y == a.y_in))
        return;
    const Outputs o = outputs_of(a, group, 4 * l.per * kBlock);
    const int begin = o.begin + wave * kBlock;
    // what comes from memory first of all
    Block<DT, TT, NB, STEPS> block(a, r, adapted, lane);
    if (begin < o.end)
        block.load(begin);
    if (adapted)
        halves_of<DT, T, STEPS>(a, l, r, o.slice, half, top);
    for (int n0 = begin; n0 < o.end; n0 += 4 * kBlock) {
        if (n0 > begin)
            block.load(n0);
        block.run(half, top, n0);
    }
}

// The same for ranks whose rows of B are a line and more: there the operands' lanes, which
// go from row to row, take the load path four times as long as consecutive ones, for every
// wavefront anew.  So the workgroup's wavefronts have rows of their own, 16 TT each, and the
// blocks in common: a block's rows of B come by consecutive lanes, through LDS, two blocks
// by turns, with one barrier a block.
template <int DT, int TT, int STEPS>
__global__ __launch_bounds__(256, 2) void lora_up_rows_kernel(LoraArgs a, Launch l)
{
    constexpr int T = 64 * TT, WORDS = kBlock * 2 * STEPS, LOADS = WORDS / 256;  // of a block of B, 16 bytes
    constexpr int HALVES = 4 * STEPS * T;
    __shared__ u32x4 lds[HALVES > 2 * WORDS ? HALVES : 2 * WORDS];
    __shared__ uint32_t top[T];
    unsigned id = kv4_workgroup();
    const int lane = threadIdx.x & 63, c = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int group = (int)(id % (unsigned)l.blocks);
    id /= (unsigned)l.blocks;
    const int tile = (int)(id % (unsigned)l.tiles), segment = (int)(id / (unsigned)l.tiles);
    if (segment >= a.segments)
        return;
    const Rows r = rows_of(a, segment, tile, T);
    const bool adapted = (unsigned)r.slot < (unsigned)a.slots;
    if (r.n == 0 || (!adapted && a.y == a.y_in))
        return;
    const Outputs o = outputs_of(a, group, l.per * kBlock);
    const int t0 = 16 * TT * wave, left = r.n - t0;
    const bool some = left > 0;  // the wavefront has rows
    const Rows mine = {some ? r.first + t0 : r.first, some ? (left < 16 * TT ? left : 16 * TT) : 1, r.slot};
    Block<DT, TT, 4, STEPS> block(a, mine, adapted, lane);
    const int per_row = a.rank / 8, words = kBlock * per_row;
    u32x4 word[LOADS], next[TT][2];
    auto load_b = [&](int n0) {
        const u32x4 *from = reinterpret_cast<const u32x4 *>(a.b + ((int64_t)r.slot * a.ends[a.slices - 1] + n0) * a.rank);
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            word[i] = from[256 * i + (int)threadIdx.x < words ? 256 * i + (int)threadIdx.x : 0];
    };
    // words of a row exchanged so that 8 rows' words of one place are in other banks
    auto slot_of = [&](int row, int at) { return row * 2 * STEPS + (at ^ (row % 8 & (2 * STEPS - 1))); };
    block.load_in(block.in, o.begin);
    u32x4 t[TT][STEPS];
    if (adapted) {
        load_b(o.begin);
        u32x4(&half)[4 * STEPS][T] = reinterpret_cast<u32x4(&)[4 * STEPS][T]>(lds);
        halves_of<DT, T, STEPS>(a, l, r, o.slice, half, top);
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
                t[i][s] = half[4 * s + q][t0 + 16 * i + c];
        __syncthreads();  // the blocks of B take its place
    }
    int turn = 0;
    for (int n0 = o.begin; n0 < o.end; n0 += kBlock) {
        u32x4 *own = lds + turn * WORDS;
        turn ^= 1;
        if (adapted) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int at = 256 * i + (int)threadIdx.x;
                if (at < words)
                    own[slot_of(at / per_row, at % per_row)] = word[i];
            }
            __syncthreads();
        }
        if (n0 + kBlock < o.end) {
            if (adapted)
                load_b(n0 + kBlock);
            block.load_in(next, n0 + kBlock);
        }
        f32x4 acc[TT][4] = {};
        if (adapted) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int k = 4 * s + q;
                    const u32x4 b = own[slot_of(j / 2 * 32 + c / 4 * 8 + j % 2 * 4 + c % 4,
                                                k < per_row ? k : (k < 2 * per_row ? k - per_row : 0))];
#pragma unroll
                    for (int i = 0; i < TT; ++i)
                        acc[i][j] = mfma<DT>(b, t[i][s], acc[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (some)
                block.put(top + t0, acc[i], i, n0);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                block.in[i][h] = next[i][h];
        }
    }
}

// Both products in one launch, for few rows and ranks up to 16: a workgroup of 16
// wavefronts has 1024 l.per outputs of one slice and works out t for them by itself, a
// sixteenth of the inputs a wavefront.  What it takes is A read again by every workgroup,
// what it saves a launch, t's way through memory and the wait for it.
template <int DT>
__global__ __launch_bounds__(1024) void lora_step_kernel(LoraArgs a, Launch l)
{
    constexpr int OUT = DT == DT_BF16 ? OUT_BF16 : OUT_F16, WAVES = 16, KS = 2;
    constexpr int STAGE = kStageWords<1, 1, KS>;
    __shared__ u32x4 lds[WAVES * STAGE];
    __shared__ u32x4 half[4][16];
    __shared__ uint32_t top[16];
    unsigned id = kv4_workgroup();
    const int lane = threadIdx.x & 63, c = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int group = (int)(id % (unsigned)l.blocks), segment = (int)(id / (unsigned)l.blocks);
    if (segment >= a.segments)
        return;
    const Rows r = rows_of(a, segment, 0, 16);
    const bool adapted = (unsigned)r.slot < (unsigned)a.slots;
    if (r.n == 0 || (!adapted && a.y == a.y_in))
        return;
    const Outputs o = outputs_of(a, group, WAVES * l.per * kBlock);
    const int begin = o.begin + wave * kBlock, R = a.rank;
    Block<DT, 1, 4, 1> block(a, r, adapted, lane);
    if (begin < o.end)
        block.load(begin);
    if (adapted) {
        const float scale = a.scale ? a.scale[r.slot] : 1.0f;
        const int k0 = wave * l.chunk, k1 = k0 + l.chunk < a.inputs ? k0 + l.chunk : a.inputs;
        f32x4 acc[1][1] = {};
        multiply_rows<DT, 1, 1, KS>(a, r, o.slice * R, a.slices * R, k0, k1, lane, lds + wave * STAGE, acc);
        __syncthreads();
        lds[threadIdx.x] = __builtin_bit_cast(u32x4, acc[0][0]);
        __syncthreads();
        if (wave == 0) {
            f32x4 t = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
                t += __builtin_bit_cast(f32x4, lds[64 * w + lane]);
            const bool there = 4 * q < R;  // of R numbers
            float most = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[e] = there ? t[e] * scale : 0.0f;
                most = __builtin_fmaxf(most, __builtin_fabsf(t[e]));
            }
            most = __builtin_fmaxf(most, __shfl_xor(most, 16));
            most = __builtin_fmaxf(most, __shfl_xor(most, 32));
            if (q == 0)
                top[c] = __builtin_bit_cast(uint32_t, most);
            const int by = DT == DT_F16 ? -token_exponent(__builtin_bit_cast(uint32_t, most)) : 0;
            uint32_t high[2], low[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                halves<OUT>(t[2 * e], t[2 * e + 1], by, high[e], low[e]);
            // numbers 4 q .. 4 q + 3 of the high halves' R, and of the low ones' behind them;
            // R 8: zeros to the operand's end
            uint2 *to = reinterpret_cast<uint2 *>(&half[0][0]);
            auto put = [&](int k, uint2 v) { to[(k / 8 * 16 + c) * 2 + k / 4 % 2] = v; };
            put(there ? 4 * q : 4 * q + R, uint2{high[0], high[1]});
            put(there ? 4 * q + R : 4 * q + 2 * R, uint2{low[0], low[1]});
        }
        __syncthreads();
    }
    for (int n0 = begin; n0 < o.end; n0 += WAVES * kBlock) {
        if (n0 > begin)
            block.load(n0);
        block.run(half, top, n0);
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
    int64_t splits = (size > 16 ? 2048 : 1024) / units;
    const int64_t many = size > 16 ? 4 : kMaxSplits, most = a.inputs / 1024 < many ? a.inputs / 1024 : many;
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

template <int DT, int TT, int NB, int STEPS>
hipError_t launch_up(const LoraArgs &a, Launch l, hipStream_t stream)
{
    l.tiles = (int)(((int64_t)a.max_rows + 16 * TT - 1) / (16 * TT));
    // blocks of outputs of a wavefront: as leave the wavefronts that are resident at once
    // (64 rows beside 6144 outputs 13.2 us with one, 11.8 with two; 2000 beside 24576 at rank
    // 64 74 us with three, 70.7 with four, 76.8 with six), up to two at low ranks, whose t
    // costs little to set up again (8400 rows beside 6144 74.2 with four, 73.3 with two)
    const int64_t all = a.ends[a.slices - 1] / kBlock, units = (int64_t)a.segments * l.tiles;
    constexpr int64_t kResident = (STEPS > 2 ? 3 : 4) * 1024, kMost = STEPS == 1 ? 2 : 4;
    int64_t per = (all * units + kResident - 1) / kResident;
    per = per < 1 ? 1 : (per > kMost ? kMost : per);
    l.per = (int)per;
    l.blocks = 0;
    for (int i = 0, from = 0; i < a.slices; from = a.ends[i++])
        l.blocks += (a.ends[i] - from + 4 * kBlock * l.per - 1) / (4 * kBlock * l.per);
    const unsigned grid = (unsigned)a.segments * (unsigned)l.tiles * (unsigned)l.blocks;
    return kv4_launch(lora_up_kernel<DT, TT, NB, STEPS>, grid, 256, stream, a, l);
}

template <int DT, int TT, int STEPS>
hipError_t launch_up_rows(const LoraArgs &a, Launch l, hipStream_t stream)
{
    l.tiles = (int)(((int64_t)a.max_rows + 64 * TT - 1) / (64 * TT));
    const int64_t all = a.ends[a.slices - 1] / kBlock, units = (int64_t)a.segments * l.tiles;
    // as many workgroups as are resident: 3 a compute unit (2000 rows beside 24576 outputs at
    // rank 64 63.8 us, 71.6 with 1024, 66.1 with 512)
    constexpr int64_t kHeld = 768;
    int64_t per = (all * units + kHeld - 1) / kHeld;
    per = per < 1 ? 1 : (per > 16 ? 16 : per);
    l.per = (int)per;
    l.blocks = 0;
    for (int i = 0, from = 0; i < a.slices; from = a.ends[i++])
        l.blocks += (a.ends[i] - from + kBlock * l.per - 1) / (kBlock * l.per);
    const unsigned grid = (unsigned)a.segments * (unsigned)l.tiles * (unsigned)l.blocks;
    return kv4_launch(lora_up_rows_kernel<DT, TT, STEPS>, grid, 256, stream, a, l);
}

template <int DT, int TT>
hipError_t launch_up(const LoraArgs &a, const Launch &l, hipStream_t stream)
{
    if (a.rank <= 16)
        return launch_up<DT, TT, 4, 1>(a, l, stream);
    if (a.rank <= 32)
        return launch_up<DT, TT, 4, 2>(a, l, stream);
    if (a.rank <= 64)
        return TT > 1 ? launch_up_rows<DT, 2, 4>(a, l, stream) : launch_up<DT, 1, 4, 4>(a, l, stream);
    return TT > 1 ? launch_up_rows<DT, 1, 8>(a, l, stream) : launch_up<DT, 1, 2, 8>(a, l, stream);
}

// Workgroups that share a segment's outputs out.
int step_groups(const LoraArgs &a, int per)
{
    int n = 0;
    for (int i = 0, from = 0; i < a.slices; from = a.ends[i++])
        n += (a.ends[i] - from + 16 * per * kBlock - 1) / (16 * per * kBlock);
    return n;
}

// Blocks of outputs of a wavefront with which one launch does both, 0: two launches.
// One, while all its workgroups run at once, one a compute unit, and a wavefront's share
// of the inputs is short.  In a graph, rank 16, one launch against two: 1 row of 4096
// inputs beside 4096 outputs 6.8 / 7.4 us (from the host 7.0 / 9.4), 6144 in three slices
// 7.0 / 8.6, 32 rows with as many adapters 8.7 / 9.6, 64 of them with two blocks 9.7 /
// 11.4 (with one 14.4), 200 beside 4096 with four 10.8 / 14.2; 8 beside 24576 8.9 / 8.4
// (from the host the launch decides).  Inputs, 1 row, beside 4096 | 6144 outputs: 6144
// 8.0 / 7.7 | 8.1 / 9.1 (from the host 8.1 / 9.5 | 8.3 / 9.6), 7168 9.0 / 8.0 | 9.1 / 9.4
// (9.1 / 9.4 | 9.2 / 9.8), 8192 9.2 / 7.7 | 9.2 / 8.9 (9.2 / 9.4 | 9.3 / 9.5), 12288 11.5 /
// 8.1 | 11.6 / 9.3.  So up to 8192 a host gains by one launch and a graph loses for few
// outputs; 6144 is between (most it loses there, 16 segments of 8 rows beside 4096 in a
// graph, 9.9 / 8.3; from the host 9.5 / 9.1).
int in_one(const LoraArgs &a)
{
    if (a.max_rows > 16 || a.rank > 16 || a.inputs > 6144)
        return 0;
    for (int per = 1; per <= 4; per *= 2)
        if ((int64_t)a.segments * step_groups(a, per) <= 256)
            return per;
    return 0;
}

template <int DT>
hipError_t launch(const LoraArgs &a, Launch l, hipStream_t stream)
{
    if (const int per = in_one(a)) {
        l.per = per;
        l.chunk = (a.inputs / 64 + 15) / 16 * 64;
        l.blocks = step_groups(a, per);
        return kv4_launch(lora_step_kernel<DT>, (unsigned)a.segments * (unsigned)l.blocks, 1024, stream, a, l);
    }
    const hipError_t e = a.max_rows > 16 ? launch_down<DT, 2>(a, l, stream) : launch_down<DT, 1>(a, l, stream);
    if (e != hipSuccess)
        return e;
    return a.max_rows > 16 ? launch_up<DT, 4>(a, l, stream) : launch_up<DT, 1>(a, l, stream);
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
