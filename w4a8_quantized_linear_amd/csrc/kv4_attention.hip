// The attention call over the 4-bit key/value cache: which kernel takes it,
// how a long cache is dealt to several workgroups, and the joining of their
// parts.
//
// Splitting.  The kernels give a workgroup one tile of columns of one kv head
// and some of the pages that the tile sees.  With few sequences and rows that
// leaves compute units idle, so a tile's pages are cut into equal chunks, one
// workgroup each; a chunk's unscaled outputs (fp32), maximum and sum go to the
// workspace, and a second small launch joins them in chunk order:
//   m = max m_i, y = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i.
// Chunk boundaries depend on the sizes of the call alone, not on timing.
#include "kv4_attention.h"

namespace cider {
namespace {

constexpr int kJoinWaves = 4;

// One workgroup per (row, query head); its wavefronts take every 4th part.
template <int D, int COLS>
__global__ __launch_bounds__(64 * kJoinWaves) void kv4_join_kernel(Kv4AttentionArgs a, Kv4Launch n)
{
    constexpr int PER = D / 64;
    __shared__ float part[kJoinWaves][D], part_l[kJoinWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cols = a.kv.max_rows * (a.q_heads / a.kv.kv_heads);
    const int col = (int)(blockIdx.x % (unsigned)cols);
    const unsigned bh = blockIdx.x / (unsigned)cols;
    Tile t;
    if (!tile_of<COLS>(a, (int)(bh / (unsigned)a.kv.kv_heads), (int)(bh % (unsigned)a.kv.kv_heads), col / COLS, t) ||
        col >= t.cols || t.range.count <= n.pages)
        return;
    const int parts = (t.range.count + n.pages - 1) / n.pages;
    const int64_t at = pair_of(a, t, col) * n.splits;
    float m = -__builtin_inff();
    for (int i = lane; i < parts; i += 64)
        m = __builtin_fmaxf(m, n.part_stat[2 * (at + i)]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        m = __builtin_fmaxf(m, __shfl_xor(m, d));
    float l = 0.0f, o[PER] = {};
    for (int i = wave; i < parts; i += kJoinWaves) {
        const float li = n.part_stat[2 * (at + i) + 1];
        const float f = li == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(n.part_stat[2 * (at + i)] - m);
        l += li * f;
#pragma unroll
        for (int e = 0; e < PER; ++e)
            o[e] += n.part[(at + i) * D + PER * lane + e] * f;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e)
        part[wave][PER * lane + e] = o[e];
    if (lane == 0)
        part_l[wave] = l;
    __syncthreads();
    if (wave != 0)
        return;
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w)
        l += part_l[w];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *y = output_of(a, t, col) + PER * lane;
    float r[PER] = {};
#pragma unroll
    for (int e = 0; e < PER; ++e) {
#pragma unroll
        for (int w = 0; w < kJoinWaves; ++w)
            r[e] += part[w][PER * lane + e];
        r[e] *= inv;
    }
    if constexpr (PER == 2)
        *reinterpret_cast<uint32_t *>(y) = pack_out(r[0], r[1], a.y_dtype);
    else
        y[0] = (uint16_t)pack_out(r[0], 0.0f, a.y_dtype);
}

// Columns of a (sequence, kv head) at most.
int64_t most_columns(const Kv4AttentionArgs &a) { return (int64_t)a.kv.max_rows * (a.q_heads / a.kv.kv_heads); }

int64_t tiles_of(const Kv4AttentionArgs &a, int cols) { return (most_columns(a) + cols - 1) / cols; }

// Pages that a tile of `cols` columns sees at most.
int64_t most_pages(const Kv4AttentionArgs &a, int cols)
{
    const int64_t all = ((int64_t)a.kv.max_kv_len + kPageTokens - 1) / kPageTokens;
    if (a.window == 0)
        return all;
    const int64_t rows = cols / (a.q_heads / a.kv.kv_heads) + 2;
    const int64_t seen = ((int64_t)a.window + rows + 2 * kPageTokens) / kPageTokens +
                         ((int64_t)a.sinks + kPageTokens - 1) / kPageTokens;
    return seen < all ? seen : all;
}

// Columns of the tiles of the kernel that takes the call.
int tile_cols(const Kv4AttentionArgs &a) { return most_columns(a) > 48 ? kManyCols : kFewCols; }

Kv4Launch plan(const Kv4AttentionArgs &a)
{
    Kv4Launch n{};
    const int cols = tile_cols(a);
    n.tiles = (int)tiles_of(a, cols);
    n.splits = 1;
    const int64_t pages = most_pages(a, cols);
    const int64_t units = n.tiles * (int64_t)a.kv.kv_heads * a.kv.batch;
    // chunks of at least kMinPages pages, as many as give kWanted workgroups
    const int64_t kMinPages = 16, kWanted = cols == kManyCols ? 512 : 2048;
    if (pages > kMinPages && units < kWanted) {
        int64_t splits = (kWanted + units - 1) / units;
        const int64_t most = (pages + kMinPages - 1) / kMinPages;
        splits = splits < most ? splits : most;
        n.pages = (int)((pages + splits - 1) / splits);
        n.splits = (int)((pages + n.pages - 1) / n.pages);
    }
    return n;
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

size_t part_bytes(const Kv4AttentionArgs &a, const Kv4Launch &n)
{
    return round256((size_t)a.kv.rows * a.q_heads * n.splits * a.kv.head_dim * sizeof(float));
}

size_t bytes_of(const Kv4AttentionArgs &a, const Kv4Launch &n)
{
    return n.splits < 2 ? 0
                        : part_bytes(a, n) + round256((size_t)a.kv.rows * a.q_heads * n.splits * 2 * sizeof(float));
}

template <int D>
void launch_join(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    const unsigned grid = (unsigned)most_columns(a) * (unsigned)a.kv.kv_heads * (unsigned)a.kv.batch;
    if (tile_cols(a) == kManyCols)
        kv4_join_kernel<D, kManyCols><<<grid, 64 * kJoinWaves, 0, stream>>>(a, n);
    else
        kv4_join_kernel<D, kFewCols><<<grid, 64 * kJoinWaves, 0, stream>>>(a, n);
}

}  // namespace

size_t kv4_attention_workspace(const Kv4AttentionArgs &a) { return bytes_of(a, plan(a)); }

hipError_t launch_kv4_attention(const Kv4AttentionArgs &a, void *workspace, size_t workspace_bytes,
                                hipStream_t stream)
{
    Kv4Launch n = plan(a);
    while (n.splits > 1 && (!workspace || bytes_of(a, n) > workspace_bytes)) {
        // fewer, longer chunks until the parts fit
        n.pages = n.pages * 2;
        n.splits = (n.splits + 1) / 2;
    }
    if (n.splits > 1) {
        n.part = static_cast<float *>(workspace);
        n.part_stat = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + part_bytes(a, n));
    }
    const hipError_t e = tile_cols(a) == kManyCols ? launch_kv4_many_rows(a, n, stream)
                                                   : launch_kv4_few_rows(a, n, stream);
    if (e != hipSuccess || n.splits < 2)
        return e;
    if (a.kv.head_dim == 64)
        launch_join<64>(a, n, stream);
    else
        launch_join<128>(a, n, stream);
    return hipGetLastError();
}

}  // namespace cider
