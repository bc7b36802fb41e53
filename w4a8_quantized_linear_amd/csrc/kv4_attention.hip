// The attention call over the 4-bit key/value cache: which kernel takes it,
// how a long cache is dealt to several workgroups, and the joining of their
// parts.
//
// Splitting.  The kernels give a workgroup one tile of columns of one kv head
// and some of the pages that the tile sees.  With few sequences and rows that
// leaves compute units idle, so a tile's pages are cut into equal chunks, one
// workgroup each; a chunk's unscaled outputs (fp32, small by a power of two so that
// sums of many large values are finite), maximum and sum go to the workspace, and a
// second small launch joins them in chunk order:
//   m = max m_i, y = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i.
// Chunk boundaries depend on the sizes of the call alone, not on timing.
//
// Shared prefixes.  Sequences of a run hold the same first pages, and all rows of the
// run see all of their tokens.  So some workgroups take the run's rows as columns over
// the shared pages, without any mask, others each sequence's over the pages behind, and
// the same join puts the parts of both together.  Both are one launch where both have
// tiles of as many columns (two launches, 64 sequences behind 8192 tokens: 44 us, one:
// 36).  What bounds it: with 16 columns a tile the vector instructions of a page, about
// 500 a wavefront (32 us for 21000 tile pages, 75 % of them issue); for the prompts of 16
// questions over 65536 tokens the many-row kernel's own bounds (1.1 PFLOP/s).
#include "kv4_attention.h"

namespace cider {
namespace {

constexpr int kMaxSplits = 256;

// The (row, query head) pair of a number, and the parts it has (0: none, its
// workgroup wrote the output itself or the pair is not there).  With shared
// prefixes (SHARED) the first `front` are over the shared pages.
template <int COLS, bool SHARED>
__device__ __forceinline__ int parts_of(const Kv4AttentionArgs &a, const Kv4Launch &n, int64_t id, Tile &t, int &col, int &front)
{
    constexpr Pages PAGES = SHARED ? Pages::Shared : Pages::All;
    const int64_t cols = (int64_t)a.kv.max_rows * (a.q_heads / a.kv.kv_heads);
    col = (int)(id % cols);
    front = 0;
    const int64_t bh = id / cols;
    const bool mine = bh < (int64_t)a.kv.kv_heads * a.kv.batch &&
                      tile_of<COLS, PAGES>(a, n, (int)(bh / a.kv.kv_heads), (int)(bh % a.kv.kv_heads), col / COLS, false, t) &&
                      col < t.cols && in_parts<PAGES>(n, t);
    if (!mine)
        return 0;
    const int parts = (t.range.count + n.pages - 1) / n.pages;
    if constexpr (!SHARED)
        return parts;
    front = (t.shared + n.front_pages - 1) / n.front_pages;
    front = front < n.front_splits ? front : n.front_splits;
    return front + (parts < n.splits ? parts : n.splits);
}

// Where a pair's part is among its own.
template <bool SHARED>
__device__ __forceinline__ int slot_of(const Kv4Launch &n, int i, int front)
{
    return SHARED && i >= front ? n.front_splits + i - front : i;
}
template <bool SHARED>
__device__ __forceinline__ int64_t slots_of(const Kv4Launch &n) { return SHARED ? n.slots : n.splits; }
template <bool SHARED>
__device__ __forceinline__ int part_bits(const Kv4Launch &n) { return sum_bits(SHARED ? n.sum_pages : n.pages); }

__device__ __forceinline__ void write_joined(const Kv4AttentionArgs &a, const Tile &t, int col, int d4, f32x4 o)
{
    *reinterpret_cast<uint2 *>(output_of(a, t, col) + 4 * d4) =
        uint2{pack_out(o.x, o.y, a.y_dtype), pack_out(o.z, o.w, a.y_dtype)};
}

// At most PARTS parts: D / 4 lanes a pair, each with 4 elements of every part.
// All loads are on their way at once: a chain of two (lengths, then statistics
// and parts), 2.9 us for 32 pairs of 4 parts, 4.6 for 2048, the launch included.
template <int D, int COLS, int PARTS, bool SHARED>
__global__ __launch_bounds__(256) void kv4_join_few_kernel(Kv4AttentionArgs a, Kv4Launch n)
{
    constexpr int LANES = D / 4;
    Tile t;
    int col, front;
    const int parts = parts_of<COLS, SHARED>(a, n, (int64_t)kv4_workgroup() * (256 / LANES) + (int)threadIdx.x / LANES, t,
                                             col, front);
    if (parts == 0)
        return;
    const int d4 = (int)threadIdx.x % LANES;
    const int64_t at = pair_of(a, t, col) * slots_of<SHARED>(n);
    const float2 *stat = reinterpret_cast<const float2 *>(n.part_stat) + at;
    const f32x4 *part = reinterpret_cast<const f32x4 *>(n.part) + at * LANES + d4;
    float2 ml[PARTS];  // maximum, sum
    f32x4 v[PARTS];
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        const int slot = slot_of<SHARED>(n, i < parts ? i : 0, front);
        ml[i] = stat[slot];
        v[i] = part[slot * LANES];
    }
    float m = ml[0].x, l = 0.0f;
#pragma unroll
    for (int i = 1; i < PARTS; ++i)
        m = __builtin_fmaxf(m, ml[i].x);
    // only what is not there or saw nothing (sum 0) stays out: NaN in a part is the
    // result's NaN though its factor be 0
    float f[PARTS];
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        f[i] = i < parts && ml[i].y != 0.0f ? __builtin_amdgcn_exp2f(ml[i].x - m) : 0.0f;
        l += ml[i].y * f[i];
    }
    const float inv = ldexp_f(reciprocal(l), part_bits<SHARED>(n));
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
        o += v[i] * (f[i] * inv);
    write_joined(a, t, col, d4, o);
}

// Up to 256 parts: a workgroup per pair.  A part's factor is computed once, by
// the lane of its number; then groups of D / 4 lanes add up the parts, 16 bytes a
// lane.  A chain of three loads (lengths, statistics, parts): 4.6 us for 32 pairs
// of 64 parts, the launch included.
template <int D, int COLS, bool SHARED>
__global__ __launch_bounds__(256) void kv4_join_many_kernel(Kv4AttentionArgs a, Kv4Launch n)
{
    constexpr int GROUPS = 256 / (D / 4);
    __shared__ float factor[kMaxSplits];
    __shared__ f32x4 sums[GROUPS][D / 4];
    __shared__ float wave_m[4], wave_l[4];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = (int)threadIdx.x;
    Tile t;
    int col, front;
    const int parts = parts_of<COLS, SHARED>(a, n, kv4_workgroup(), t, col, front);
    if (parts == 0)
        return;
    const int64_t at = pair_of(a, t, col) * slots_of<SHARED>(n);
    float m = -__builtin_inff(), l = 0.0f;
    if (lane < parts) {
        const int64_t slot = at + slot_of<SHARED>(n, lane, front);
        m = n.part_stat[2 * slot];
        l = n.part_stat[2 * slot + 1];
    }
    float top = wave_max(m);
    if (lane % 64 == 0)
        wave_m[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w)
        top = __builtin_fmaxf(top, wave_m[w]);
    const float f = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m - top);  // l 0: saw nothing
    l *= f;
    factor[lane] = f;
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        l += __shfl_xor(l, d);
    if (lane % 64 == 0)
        wave_l[wave] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        l += wave_l[w];
    const float inv = ldexp_f(reciprocal(l), part_bits<SHARED>(n));
    const int g = lane / (D / 4), d4 = lane % (D / 4);
    f32x4 o = {0, 0, 0, 0};
    const f32x4 *part = reinterpret_cast<const f32x4 *>(n.part) + at * (D / 4) + d4;
#pragma unroll 4
    for (int i = g; i < parts; i += GROUPS)
        o += part[(int64_t)slot_of<SHARED>(n, i, front) * (D / 4)] * (factor[i] * inv);
    sums[g][d4] = o;
    __syncthreads();
    if (g != 0)
        return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i)
        o += sums[i][d4];
    write_joined(a, t, col, d4, o);
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

// Tiles of `cols` columns over all heads and sequences.
int64_t units_of(const Kv4AttentionArgs &a, int cols)
{
    return tiles_of(a, cols) * (int64_t)a.kv.kv_heads * a.kv.batch;
}

// Pages that a tile sees on average: a prompt's rows see what lies before them.
double mean_pages(const Kv4AttentionArgs &a, int cols)
{
    if (a.flat)
        return (double)most_pages(a, cols);
    const double mean = (a.kv.max_kv_len - 0.5 * a.kv.max_rows) / kPageTokens + 0.5, most = (double)most_pages(a, cols);
    return mean < most ? mean : most;
}

// Times in us, fitted to calls of 64 to 4096 rows over 256 to 16384 tokens, 2 to 8
// kv heads, G 1 to 7.  Over 68 of them the many-row one is 29 % below to 16 % above
// what is measured, the few-row one 36 % below to 49 % above, far off mostly where the
// other kernel is far ahead or behind: the choice by them is within 3 % of the best
// in 59, within 15 % in all.
//
// The few-row kernel: a tile costs its beginning and its pages.
double few_rows_time(const Kv4AttentionArgs &a)
{
    return 8 + (a.kv.head_dim == 64 ? 0.57 : 1.0) * (double)units_of(a, kFewCols) *
                   (0.0068 + 0.00104 * mean_pages(a, kFewCols));
}

// The other one, 128 columns, a tile's pages in `splits` chunks: beginnings, of
// which 512 run at a time; then the longest chunk, 1.85 us a page of 128 elements
// for a workgroup alone on its compute unit and 2.1 for one of two, or all pages
// at 2.4 us with 512 at work and what the longest tile has over the mean; then
// the parts' way through memory and the second launch.
double many_rows_time(const Kv4AttentionArgs &a, int64_t splits)
{
    const double units = (double)units_of(a, 128), pages = (double)most_pages(a, 128), mean = mean_pages(a, 128);
    const double rounds = units * splits / 512;
    const double longest = (rounds > 0.5 ? 2.1 : 1.85) * pages / splits;
    const double all = units * mean * 2.4 / 512 + 1.8 * (pages - mean) / splits;
    const double join = splits < 2 ? 0 : 4 + units * 128 * splits * a.kv.head_dim * 8 / 5e6;
    return 3 + 5 * (rounds > 1 ? rounds : 1) + (a.kv.head_dim == 64 ? 0.7 : 1.0) * (longest > all ? longest : all) + join;
}

// Chunks of a tile of 128 columns: as many as make the call shortest, of 4 pages
// and more; as many as run at once, or a half, a quarter of that, which fills the
// compute units evenly.  (4096 rows, 448 tiles of 64 pages: whole 96
// us, halved 125; 512 rows over 4096, 128 tiles of 64: whole 125, in four 70; 128
// over 16384, 32 of 256: 8 chunks 75, 16 73.)
int64_t many_rows_splits(const Kv4AttentionArgs &a)
{
    const int64_t units = units_of(a, 128), pages = most_pages(a, 128);
    int64_t best = 1, most = 512 / units;
    most = most < pages / 4 ? most : pages / 4;
    most = most < kMaxSplits ? most : kMaxSplits;
    for (int64_t s = most; s >= 2; s /= 2)
        if (many_rows_time(a, s) < many_rows_time(a, best))
            best = s;
    return best;
}

// Columns of the tiles.  Up to 64 columns take the few-row kernel: it is bound by
// the pages' bytes there.  Past that the kernel that the estimates above prefer
// (prompts of 1 x 512 / 2 x 512 / 4 x 512 rows, 8 kv heads of 128, G 4: 19 / 30 /
// 52 us against 26 / 28 / 33; of 2 x 1024 and 4 x 1024, 2 heads of 64, G 7: 23 /
// 39 against 31 / 34; 2048 rows with a window of 256: 56 against 32).
// One long sequence takes 256 columns, one workgroup a compute unit: half the
// unpacking per column (2048 rows over 16384 tokens 631 -> 595 us, 4096 of 4096
// 205 -> 200), but coarser where tiles end at different times (ragged prompts 229
// -> 246, 8000 rows with a window of 1024 212 -> 235).  Of several sequences the
// launch knows only the longest's bounds: equal ones mostly gain (2 x 2048 rows over
// 8192 tokens 581 -> 557, 4 x 1024 623 -> 589, but 2 x 4096 of 4096 335 -> 342),
// ragged ones lose more.
int columns_of(const Kv4AttentionArgs &a)
{
    if (a.tiles)
        return a.tiles;
    if (most_columns(a) <= 64 || few_rows_time(a) <= many_rows_time(a, many_rows_splits(a)))
        return kFewCols;
    const int64_t units = units_of(a, 256);
    return a.kv.batch == 1 && a.window == 0 && units >= 128 && units <= 512 && most_pages(a, 256) >= 64 ? 256 : 128;
}

Kv4Launch plan(const Kv4AttentionArgs &a)
{
    Kv4Launch n{};
    n.cols = columns_of(a);
    n.tiles = (int)tiles_of(a, n.cols);
    n.splits = 1;
    n.waves = 4;
    const int64_t pages = most_pages(a, n.cols), units = units_of(a, n.cols);
    if (n.cols == kFewCols) {
        n.once = n.tiles == 1 &&
                 units * pages * kv4_block_bytes(a.kv.head_dim, a.kv.group_size) >= int64_t(128) << 20;
        // One workgroup per tile, or chunks and a second launch.  Measured (bf16,
        // equal lengths; units = tiles of all heads and sequences): a page of 128
        // elements takes a workgroup of 8 wavefronts 0.27 us; splitting costs 4 us
        // and 1.9 ns for every page of all tiles on top.  8 / 64 units: 16 pages
        // 9.6 / 10.0 us whole, 9.2 / 10.3 split; 64 pages 20.6 / 21.5 against 9.4 /
        // 16.2; 256 units of 64 pages 31.7 against 36.3.  Past kWhole pages a
        // ragged batch's longest sequence would be waited for.
        constexpr int64_t kWhole = 80;
        if (pages <= kWhole && pages * a.kv.head_dim * (2700 - 19 * (units < 1000 ? units : 1000)) <= 4 * 128 * 10000) {
            // from two workgroups a compute unit on, more wavefronts in each only
            // wait for one another (512 units of 16 pages: 21.9 us with 8, 16.4 with 4)
            n.waves = units < 512 ? 8 : 4;
            return n;
        }
        // Chunks that make about two workgroups a compute unit, of 4 pages (one a
        // wavefront) to kLongest: below that a chunk's fixed cost shows (one
        // sequence of 131072 tokens: 34 us in chunks of 32 pages, 42 of 8), above
        // it the longest sequence of a ragged batch does.
        constexpr int64_t kWanted = 512, kShortest = 4, kLongest = 32;
        int64_t chunk = (units * pages / kWanted + 3) / 4 * 4;
        chunk = chunk < kShortest ? kShortest : (chunk > kLongest ? kLongest : chunk);
        const int64_t least = (pages + kMaxSplits - 1) / kMaxSplits;
        chunk = chunk < least ? least : chunk;
        n.pages = (int)chunk;
    } else {
        // 256 columns: one workgroup a compute unit, chunks of 16 pages and more
        const int64_t most = 256 / units < pages / 16 ? 256 / units : pages / 16;
        const int64_t splits = n.cols == 128 ? many_rows_splits(a) : (most < kMaxSplits ? most : kMaxSplits);
        if (splits < 2)
            return n;
        n.pages = (int)((pages + splits - 1) / splits);
    }
    n.splits = (int)((pages + n.pages - 1) / n.pages);
    if (units * n.splits >= int64_t(1) << 31)  // a launch counts workgroups in 32 bits
        n.splits = 1;
    return n;
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

size_t part_bytes(const Kv4AttentionArgs &a, int slots)
{
    return round256((size_t)a.kv.rows * a.q_heads * slots * a.kv.head_dim * sizeof(float));
}

size_t bytes_of(const Kv4AttentionArgs &a, int slots)
{
    return part_bytes(a, slots) + round256((size_t)a.kv.rows * a.q_heads * slots * 2 * sizeof(float));
}

void use_workspace(const Kv4AttentionArgs &a, Kv4Launch &n, int slots, void *workspace)
{
    n.part = static_cast<float *>(workspace);
    n.part_stat = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + part_bytes(a, slots));
}

template <int D, int COLS, bool SHARED>
hipError_t launch_join(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    const unsigned pairs = (unsigned)most_columns(a) * (unsigned)a.kv.kv_heads * (unsigned)a.kv.batch;
    const int parts = SHARED ? n.slots : n.splits;
    constexpr unsigned PAIRS = 256 / (D / 4);
    // 5 to 16 parts: a workgroup per pair while there are few pairs (256 of 16
    // parts: the call 16.3 us, 17.0 by lanes; 4096 of 16 and 8192 of 8: 75 and 125
    // us, 71 and 114 by lanes)
    if (parts <= 4)
        return kv4_launch(kv4_join_few_kernel<D, COLS, 4, SHARED>, (pairs + PAIRS - 1) / PAIRS, 256, stream, a, n);
    if (parts <= 16 && pairs >= 2048)
        return kv4_launch(kv4_join_few_kernel<D, COLS, 16, SHARED>, (pairs + PAIRS - 1) / PAIRS, 256, stream, a, n);
    return kv4_launch(kv4_join_many_kernel<D, COLS, SHARED>, pairs, 256, stream, a, n);
}

template <int D, bool SHARED>
hipError_t launch_join(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    if (n.cols == kFewCols)
        return launch_join<D, kFewCols, SHARED>(a, n, stream);
    return n.cols == 128 ? launch_join<D, 128, SHARED>(a, n, stream) : launch_join<D, 256, SHARED>(a, n, stream);
}

template <bool SHARED>
hipError_t launch_join(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    return a.kv.head_dim == 64 ? launch_join<64, SHARED>(a, n, stream) : launch_join<128, SHARED>(a, n, stream);
}

// The workgroups over shared pages (front) and over those behind them (own), each
// planned as a call of its own: the runs as sequences of max_pages pages, and the
// sequences with what the longest has behind the longest prefix.  A sequence that has
// more (it is in no run, its run shares less) gives it to its last split.
struct SharedPlan {
    Kv4Launch front, own;
};

SharedPlan plan_shared(const Kv4AttentionArgs &a, const Kv4Runs &r)
{
    const int all = (a.kv.max_kv_len + kPageTokens - 1) / kPageTokens;
    Kv4AttentionArgs f = a;
    f.kv.batch = r.groups;
    f.kv.max_rows = r.max_rows;
    f.kv.max_kv_len = r.max_pages * kPageTokens;
    f.flat = true;
    Kv4AttentionArgs o = a;
    o.kv.max_kv_len -= r.max_pages * kPageTokens;
    const int least = a.kv.max_rows < a.kv.max_kv_len ? a.kv.max_rows : a.kv.max_kv_len;
    o.kv.max_kv_len = o.kv.max_kv_len < least ? least : o.kv.max_kv_len;
    SharedPlan p = {plan(f), plan(o)};
    // Tiles of 16 columns: there is a join in any case, so that chunks are as long as
    // leaves 768 workgroups of 4 wavefronts, which the compute units hold at once, of both
    // kinds together (64 sequences behind 8192 tokens: 36.1 us with 768, 38.6 with 1024,
    // 42.2 with 2048; 30 with drafts behind 3 prefixes: 27.1, 28.6, 30.9).
    constexpr int kHeld = 768;
    auto few_pages = [](const Kv4AttentionArgs &x, const Kv4Launch &n) {
        return n.cols == kFewCols ? units_of(x, kFewCols) * most_pages(x, kFewCols) : int64_t(0);
    };
    const int64_t chunk = (few_pages(f, p.front) + few_pages(o, p.own) + 4 * kHeld - 1) / (4 * kHeld) * 4;
    auto deal = [&](const Kv4AttentionArgs &x, Kv4Launch &n) {
        const int64_t pages = most_pages(x, n.cols) > 0 ? most_pages(x, n.cols) : 1;
        if (n.cols == kFewCols)
            n.pages = (int)(chunk < 4 ? 4 : (chunk < 32 ? chunk : 32));  // (0: no tile of 16 sees a page)
        else if (n.splits < 2)
            n.pages = (int)pages;
        // a join takes kMaxSplits, and a launch counts workgroups in 32 bits
        const int64_t room = (int64_t(1) << 30) / units_of(x, n.cols), most = room < kMaxSplits / 2 ? (room < 1 ? 1 : room) : kMaxSplits / 2;
        if ((pages + n.pages - 1) / n.pages > most)
            n.pages = (int)((pages + most - 1) / most);
        n.splits = (int)((pages + n.pages - 1) / n.pages);
    };
    deal(f, p.front);
    deal(o, p.own);
    for (Kv4Launch *n : {&p.front, &p.own}) {
        n->runs = r;
        n->slots = p.front.splits + p.own.splits;
        n->sum_pages = all > r.max_pages ? all : r.max_pages;
        n->front_groups = (unsigned)p.front.tiles * (unsigned)p.front.splits * (unsigned)a.kv.kv_heads * (unsigned)r.groups;
        n->front_tiles = p.front.tiles;
        n->front_splits = p.front.splits;
        n->front_pages = p.front.pages;
    }
    return p;
}

hipError_t launch_pages(const Kv4AttentionArgs &a, const Kv4Launch &n, hipStream_t stream)
{
    return n.cols == kFewCols ? launch_kv4_few_rows_shared(a, n, stream) : launch_kv4_many_rows_shared(a, n, stream);
}

}  // namespace

size_t kv4_attention_workspace(const Kv4AttentionArgs &a)
{
    const Kv4Launch n = plan(a);
    return n.splits < 2 ? 0 : bytes_of(a, n.splits);
}

hipError_t launch_kv4_attention(const Kv4AttentionArgs &a, void *workspace, size_t workspace_bytes,
                                hipStream_t stream)
{
    Kv4Launch n = plan(a);
    while (n.splits > 1 && (!workspace || bytes_of(a, n.splits) > workspace_bytes)) {
        // fewer, longer chunks until the parts fit
        n.pages = n.pages * 2;
        n.splits = (n.splits + 1) / 2;
    }
    if (n.splits > 1)
        use_workspace(a, n, n.splits, workspace);
    const hipError_t e = n.cols == kFewCols ? launch_kv4_few_rows(a, n, stream) : launch_kv4_many_rows(a, n, stream);
    if (e != hipSuccess || n.splits < 2)
        return e;
    return launch_join<false>(a, n, stream);
}

size_t kv4_shared_workspace(const Kv4AttentionArgs &a, const Kv4Runs &r) { return bytes_of(a, plan_shared(a, r).own.slots); }

hipError_t launch_kv4_attention_shared(const Kv4AttentionArgs &a, const Kv4Runs &r, void *workspace, hipStream_t stream)
{
    SharedPlan p = plan_shared(a, r);
    for (Kv4Launch *n : {&p.front, &p.own})
        use_workspace(a, *n, n->slots, workspace);
    hipError_t e = hipSuccess;
    const Kv4Launch own = p.own;
    if (p.front.cols != p.own.cols) {
        p.front.tiles = 0;
        e = launch_pages(a, p.front, stream);
        p.own.front_groups = 0;
    }
    if (e == hipSuccess)
        e = launch_pages(a, p.own, stream);
    return e == hipSuccess ? launch_join<true>(a, own, stream) : e;
}

}  // namespace cider
