// Layout of the 4-bit key/value cache: where the codes and scales of a token
// are in a block (one head of one 64-token page), and how a sequence's rows
// map to positions.  include/cider.h states the same layout for users.
//
// Both code orders are chosen for the attention's matrix instructions, whose
// operands are 8 consecutive values of the summed axis per lane: a dword of 8
// nibbles is one such operand.  Lane l = 16 j + c of a wavefront reads
//   K   16 tokens c, dwords (t, j, 0 .. D/32 - 1): contiguous per lane, the
//       whole wavefront one contiguous run of 16 * D/2 bytes;
//   V   dwords (B, g, j, c, 0 .. 3): 16 bytes per lane, 1 KB per wavefront;
//       a dword's 8 tokens are the ones whose scores lane (j, c) already holds
//       after the score product (rows 4 j .. 4 j + 3 of two 16-token tiles).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cider_kernels.h"

namespace cider {

// Registers of a lane: operands and results of the matrix instructions, 16 bytes of
// memory (uint4 in arrays that a loop fills went to scratch).
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kPageTokens = 64;

__host__ __device__ constexpr int kv4_scale_bytes(int D, int GS) { return 4 * kPageTokens * (D / GS); }
__host__ __device__ constexpr int kv4_block_bytes(int D, int GS)
{
    return kPageTokens * D + 2 * kv4_scale_bytes(D, GS);
}
__host__ __device__ constexpr int kv4_v_offset(int D) { return kPageTokens * D / 2; }
__host__ __device__ constexpr int kv4_scale_offset(int D) { return kPageTokens * D; }

// Workgroups are counted over x and y: a launch holds less than 2^32 threads along
// x, 2^23 workgroups of 512, and calls with wide bounds have more.
constexpr unsigned kMostX = 1u << 22;
__device__ __forceinline__ unsigned kv4_workgroup() { return blockIdx.y * kMostX + blockIdx.x; }

// Launches a kernel on that many workgroups at least (those past `grid` are to
// return) and returns the launch's own status.  (The triple-bracket
// form stores the configuration first and takes it back: 0.23 us of the 2.4 that
// a launch costs the host, which is what bounds the smallest calls.)
template <typename... P, typename... A>
inline hipError_t kv4_launch(void (*kernel)(P...), unsigned grid, unsigned threads, hipStream_t stream, A... args)
{
    return [&](P... p) {
        void *at[] = {&p...};
        const hipError_t e =
            hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(grid < kMostX ? grid : kMostX, (grid + kMostX - 1) / kMostX),
                            dim3(threads), at, 0, stream);
        if (e != hipSuccess)
            (void)hipGetLastError();  // returned, and not left for another call to find
        return e;
    }(args...);
}

// Rows of one sequence in a call: its first row, their count (0 where the row
// range is not inside the call's) and the tokens in the cache, clipped to the
// batch's bounds.
struct Kv4Sequence {
    int row0, n, kv;
};

__device__ __forceinline__ Kv4Sequence kv4_sequence(const Kv4Args &a, int b)
{
    Kv4Sequence s;
    s.row0 = a.row_start[b];
    const int end = a.row_start[b + 1];
    s.kv = a.kv_len[b];
    s.kv = s.kv < 0 ? 0 : (s.kv > a.max_kv_len ? a.max_kv_len : s.kv);
    const bool inside = s.row0 >= 0 && end >= s.row0 && end <= a.rows;
    s.n = inside ? end - s.row0 : 0;
    if (s.n > a.max_rows)
        s.n = 0;
    return s;
}

}  // namespace cider
