// C ABI of the fused quantized linear layer (declared in include/cider.h).
//
// Host side only: argument checks (all before the first HIP call), the
// device check, the choice between the matrix-vector and the matrix-core
// kernel (Cider README, ossradar.top repo page, "Quick Start": seq_len > 1 ->
// INT8 GEMM, seq_len == 1 -> INT8 MV kernel), and the launches on the
// caller's stream.  No allocation, no synchronization.
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "cider.h"
#include "cider_kernels.h"
#include "kv4_layout.h"

namespace {

constexpr int64_t kMaxK = 133144;       // K * 127^2 < 2^31
constexpr int64_t kGemvMaxBytes = 65536;  // M * K int8 codes held in LDS (kernel limit)
constexpr int64_t kMaxOperandBytes = int64_t(1) << 31;
constexpr int64_t kDecodeMaxK = 32768;  // decode kernel: 16 activation chunks per thread, x [K] in LDS

std::atomic<int> g_path{0};
std::atomic<int> g_kv4_tiles{0};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// Bytes of the split product's partial sums (4-byte words per tile and
// split), and those plus the tile counters.
size_t split_part_bytes(const cider::SplitPlan &p)
{
    return round256((size_t)(p.tiles * p.splits * p.tile_elems) * 4u);
}
size_t split_bytes(const cider::SplitPlan &p)
{
    return split_part_bytes(p) + round256((size_t)p.tiles * sizeof(uint32_t));
}

// 1: usable gfx950 device current; 0: not.  Cached per device id.
int device_usable()
{
    const char *force = std::getenv("CIDER_FORCE_UNAVAILABLE");
    if (force && force[0] == '1')
        return 0;
    int count = 0;
    if (hipGetDeviceCount(&count) != hipSuccess || count <= 0) {
        (void)hipGetLastError();
        return 0;
    }
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return 0;
    }
    static std::atomic<int> cache[64];  // 0 unknown, 1 usable, 2 not usable
    if (dev < 64) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c)
            return c == 1;
    }
    hipDeviceProp_t prop;
    int ok = 0;
    if (hipGetDeviceProperties(&prop, dev) == hipSuccess)
        ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    else
        (void)hipGetLastError();
    if (dev < 64)
        cache[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok;
}

cider_status from_hip(hipError_t e) { return e == hipSuccess ? CIDER_OK : CIDER_ERR_HIP; }

// Workspace of cider_linear_ex_noalloc: a device array of fixed size, one per
// GPU, kept for the life of the process.  Host code never passes the array's
// name to a kernel or a copy (on the host it is only a stand-in for the
// symbol); it uses the device address hipGetSymbolAddress returns for the
// current device, looked up once per device.
__device__ __align__(256) uint8_t scratch[CIDER_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::atomic<void *> g_scratch_ptr[kMaxDevices];
std::mutex g_scratch_mutex;

// The current device's scratch address, or nullptr when it cannot be had.
void *scratch_address()
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        return nullptr;
    }
    void *p = g_scratch_ptr[dev].load(std::memory_order_acquire);
    if (p)
        return p;
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    p = g_scratch_ptr[dev].load(std::memory_order_relaxed);
    if (p)
        return p;
    void *addr = nullptr;
    if (hipGetSymbolAddress(&addr, HIP_SYMBOL(scratch)) != hipSuccess || !addr) {
        (void)hipGetLastError();
        return nullptr;
    }
    g_scratch_ptr[dev].store(addr, std::memory_order_release);
    return addr;
}

// Shape / mode checks shared by the product calls.
cider_status check_shape(int64_t M, int64_t N, int64_t K, int bits, int group_size)
{
    if (M < 0 || N < 0 || K <= 0)
        return CIDER_ERR_INVALID_ARG;
    if (bits != 8 && bits != 4)
        return CIDER_ERR_INVALID_ARG;
    if (group_size != 0 && group_size != 64 && group_size != 128)
        return CIDER_ERR_INVALID_ARG;
    if (K % 64 != 0 || K > kMaxK || N % 64 != 0)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    if (group_size && K % group_size != 0)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    // The kernels address operands with 32-bit byte offsets (one tile past
    // the end included): each operand stays below 2 GiB.
    if ((M + 256) * K >= kMaxOperandBytes || (N + 256) * K >= kMaxOperandBytes)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    return CIDER_OK;
}

enum Path { PATH_AUTO = 0, PATH_GEMV = 1, PATH_GEMM = 2 };

// Which kernel serves M tokens of K features; CIDER_ERR_UNSUPPORTED_SHAPE
// when the matrix-vector kernel is forced outside its range.  Automatic: the
// matrix-vector kernel (one pass over the weights, each token's dot products
// on the vector ALUs) where it measured faster than the matrix-core products
// on the operator shapes (N=10240 K=2560 and N=2560 K=10240, every mode,
// whole layer): where the few-token matrix-core kernel takes the product, up
// to 3 tokens per channel and 2 per group (per channel int8, M = 3 / 4:
// 8.9 / 10.8 us against 10.2 / 10.1; per group int8 gs64, M = 2 / 3: 11.3 /
// 15.6 against 15.0 / 15.1); elsewhere up to 8 int8-weight or 4 int4-weight
// tokens.
cider_status pick_path(int64_t M, int64_t N, int64_t K, int bits, int group_size, cider::OutKind kind,
                       int *path)
{
    const int forced = g_path.load(std::memory_order_relaxed);
    const bool gemv_ok = M <= 8 && M * K <= kGemvMaxBytes;
    cider::ProductArgs fa{};
    fa.M = M;
    fa.N = N;
    fa.K = K;
    fa.bits = bits;
    fa.group_size = group_size;
    fa.out_kind = kind;
    const int64_t gemv_max = cider::few_supported(fa) ? (group_size ? 2 : 3) : (bits == 4 ? 4 : 8);
    const bool gemv_auto = gemv_ok && M <= gemv_max;
    if (forced == PATH_GEMV) {
        if (!gemv_ok)
            return CIDER_ERR_UNSUPPORTED_SHAPE;
        *path = PATH_GEMV;
    } else if (forced == PATH_GEMM) {
        *path = PATH_GEMM;
    } else {
        *path = gemv_auto ? PATH_GEMV : PATH_GEMM;
    }
    return CIDER_OK;
}

cider_status run_product(const int8_t *xq, const float *s_tok, const void *wq, const float *s_w,
                         int64_t M, int64_t N, int64_t K, int bits, int group_size,
                         cider::OutKind kind, void *out, void *stream)
{
    cider_status st = check_shape(M, N, K, bits, group_size);
    if (st != CIDER_OK)
        return st;
    if (M == 0 || N == 0)
        return CIDER_OK;
    const bool scaled = kind != cider::OUT_I32;
    if (!xq || !wq || !out || (scaled && (!s_tok || !s_w)))
        return CIDER_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(wq) || !aligned16(out) || (scaled && !aligned16(s_w)))
        return CIDER_ERR_MISALIGNED;
    int path = PATH_GEMM;
    st = pick_path(M, N, K, bits, group_size, kind, &path);
    if (st != CIDER_OK)
        return st;
    if (!device_usable())
        return CIDER_ERR_NO_DEVICE;
    cider::ProductArgs a{};
    a.xq = xq;
    a.s_tok = s_tok;
    a.wq = wq;
    a.s_w = s_w;
    a.M = M;
    a.N = N;
    a.K = K;
    a.bits = bits;
    a.group_size = group_size;
    a.out_kind = kind;
    a.out = out;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return from_hip(path == PATH_GEMV ? cider::launch_gemv(a, s) : cider::launch_gemm(a, s));
}

bool dtype_ok(int d) { return d == CIDER_DTYPE_F16 || d == CIDER_DTYPE_BF16; }

cider::OutKind out_kind_of(int y_dtype)
{
    return y_dtype == CIDER_DTYPE_BF16 ? cider::OUT_BF16 : cider::OUT_F16;
}

// The whole layer.  static_ws: ignore ws / ws_bytes and use the current
// device's scratch array instead (after every argument and device check).
cider_status run_linear(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                        const float *smooth, const void *wq, const float *s_w, int64_t N, int bits,
                        int group_size, int y_dtype, void *ws, size_t ws_bytes, void *y,
                        void *stream, bool static_ws = false)
{
    cider_status st = check_shape(M, N, K, bits, group_size);
    if (st != CIDER_OK)
        return st;
    if (ldx < K || !dtype_ok(x_dtype) || !dtype_ok(y_dtype))
        return CIDER_ERR_INVALID_ARG;
    if (M == 0 || N == 0)
        return CIDER_OK;
    if (!x || !wq || !s_w || !y)
        return CIDER_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(wq) || !aligned16(s_w) || !aligned16(y) || ldx % 8 != 0 ||
        (smooth && !aligned16(smooth)))
        return CIDER_ERR_MISALIGNED;
    int path = PATH_GEMM;
    st = pick_path(M, N, K, bits, group_size, out_kind_of(y_dtype), &path);
    if (st != CIDER_OK)
        return st;
    // Calls in the matrix-vector kernel's earlier automatic range (up to 8
    // int8-weight or 4 int4-weight tokens) may come without a workspace:
    // those keep that kernel, which needs none.
    if (path == PATH_GEMM && !static_ws && (!ws || ws_bytes < cider_linear_workspace_bytes(M, K)) &&
        g_path.load(std::memory_order_relaxed) == PATH_AUTO && M <= (bits == 4 ? 4 : 8) &&
        M * K <= kGemvMaxBytes)
        path = PATH_GEMV;
    // fp16 tokens without smoothing on the matrix-vector path: quantized inside
    // the matrix-vector kernel, whose buffer descriptor spans the tokens with
    // 32-bit byte offsets; a row stride that puts the last token 2 GiB or more
    // past the first goes through the quantize kernel (64-bit row addresses)
    const bool fused = path == PATH_GEMV && x_dtype == CIDER_DTYPE_F16 && !smooth &&
                       ((M - 1) * ldx + K) * 2 < (int64_t(1) << 31);
    if (!fused) {
        if (static_ws) {
            if (cider_linear_workspace_bytes(M, K) > CIDER_NOALLOC_SCRATCH_BYTES)
                return CIDER_ERR_SCRATCH_LIMIT;
        } else {
            if (!ws || ws_bytes < cider_linear_workspace_bytes(M, K))
                return CIDER_ERR_WORKSPACE;
            if (!aligned16(ws))
                return CIDER_ERR_MISALIGNED;
        }
    }
    if (!device_usable())
        return CIDER_ERR_NO_DEVICE;
    if (static_ws && !fused) {
        ws = scratch_address();
        if (!ws)
            return CIDER_ERR_HIP;
        ws_bytes = CIDER_NOALLOC_SCRATCH_BYTES;
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (fused)
        return from_hip(cider::launch_gemv_fused(static_cast<const uint16_t *>(x), M, K, ldx, wq, s_w,
                                                 N, bits, group_size, y, nullptr, nullptr,
                                                 out_kind_of(y_dtype), s));
    int8_t *xq = static_cast<int8_t *>(ws);
    float *s_tok = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + round256((size_t)(M * K)));
    // Split K when the plan asks for it and the workspace has room for the
    // partial sums and tile counters (the quantize launch clears the counters).
    cider::SplitPlan plan{1, 0, 0};
    void *part = nullptr;
    uint32_t *cnt = nullptr;
    if (path == PATH_GEMM) {
        plan = cider::plan_split(M, N, K, bits, group_size);
        if (plan.splits > 1 && ws_bytes >= cider_linear_workspace_bytes(M, K) + split_bytes(plan)) {
            part = static_cast<uint8_t *>(ws) + cider_linear_workspace_bytes(M, K);
            cnt = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(part) + split_part_bytes(plan));
        } else {
            plan.splits = 1;
        }
    }
    hipError_t e = cider::launch_quantize_rows(static_cast<const uint16_t *>(x), x_dtype, M, K, ldx,
                                               smooth, 8, xq, s_tok, s, cnt,
                                               cnt ? (int)plan.tiles : 0);
    if (e != hipSuccess)
        return CIDER_ERR_HIP;
    cider::ProductArgs a{};
    a.xq = xq;
    a.s_tok = s_tok;
    a.wq = wq;
    a.s_w = s_w;
    a.M = M;
    a.N = N;
    a.K = K;
    a.bits = bits;
    a.group_size = group_size;
    a.out_kind = out_kind_of(y_dtype);
    a.out = y;
    if (plan.splits > 1)
        return from_hip(cider::launch_gemm_split(a, plan, part, cnt, s));
    return from_hip(path == PATH_GEMV ? cider::launch_gemv(a, s) : cider::launch_gemm(a, s));
}

cider_status run_quantize_weight(const void *w_f16, int w_dtype, int64_t N, int64_t K, int bits,
                                 int group_size, double clip_percentile, void *wq, float *s_w,
                                 void *stream)
{
    if (N < 0 || K <= 0 || (bits != 8 && bits != 4) || !dtype_ok(w_dtype))
        return CIDER_ERR_INVALID_ARG;
    if (group_size != 0 && group_size != 64 && group_size != 128)
        return CIDER_ERR_INVALID_ARG;
    if (!(clip_percentile > 0.0 && clip_percentile <= 100.0))  // NaN fails too
        return CIDER_ERR_INVALID_ARG;
    if (K % 64 != 0 || K > kMaxK || (group_size && K % group_size != 0))
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    if (N == 0)
        return CIDER_OK;
    if (!w_f16 || !wq || !s_w)
        return CIDER_ERR_INVALID_ARG;
    if (!aligned16(w_f16) || !aligned16(wq) || (reinterpret_cast<uintptr_t>(s_w) & 3u))
        return CIDER_ERR_MISALIGNED;
    if (!device_usable())
        return CIDER_ERR_NO_DEVICE;
    const int64_t len = group_size ? group_size : K;
    const int64_t rows = N * (K / len);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint16_t *w = static_cast<const uint16_t *>(w_f16);
    if (clip_percentile == 100.0)
        return from_hip(cider::launch_quantize_rows(w, w_dtype, rows, len, len, nullptr, bits, wq,
                                                    s_w, s));
    // fractional rank h = (len - 1) * (p / 100) in fp64, as numpy.percentile
    const double h = (double)(len - 1) * (clip_percentile / 100.0);
    const double j = std::floor(h);
    const int64_t r0 = (int64_t)j;
    const int64_t r1 = r0 + 1 < len ? r0 + 1 : len - 1;
    return from_hip(cider::launch_clip_quantize_rows(w, w_dtype, rows, len, r0, r1, h - j, bits, wq,
                                                     s_w, s));
}

constexpr int64_t kMaxHeads = 65536;
constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxTokens = int64_t(1) << 30;  // positions, and positions - window, fit an int

// Geometry shared by every key/value cache call.
cider_status check_kv4_geometry(int64_t num_pages, int64_t kv_heads, int64_t head_dim, int group_size)
{
    if (num_pages < 1 || kv_heads < 1 || head_dim < 1 || (group_size != 64 && group_size != 128))
        return CIDER_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || head_dim % group_size != 0 || kv_heads > kMaxHeads ||
        num_pages > kMaxInt)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    return CIDER_OK;
}

// Sizes of a batch (no pointer is looked at).
cider_status check_kv4_sizes(const cider_kv4_batch *b)
{
    if (!b)
        return CIDER_ERR_INVALID_ARG;
    cider_status st = check_kv4_geometry(b->num_pages, b->kv_heads, b->head_dim, b->group_size);
    if (st != CIDER_OK)
        return st;
    if (b->batch < 0 || b->rows < 0 || b->max_rows < 0 || b->max_kv_len < 0 || b->max_pages < 0)
        return CIDER_ERR_INVALID_ARG;
    if (b->batch > kMaxInt || b->rows > kMaxTokens || b->max_rows > kMaxTokens ||
        b->max_pages > kMaxTokens / cider::kPageTokens)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    if (b->max_kv_len > b->max_pages * cider::kPageTokens)
        return CIDER_ERR_INVALID_ARG;
    return CIDER_OK;
}

bool kv4_empty(const cider_kv4_batch *b) { return b->batch == 0 || b->rows == 0 || b->max_rows == 0; }

cider_status check_kv4_pointers(const cider_kv4_batch *b)
{
    if (!b->cache || !b->row_start || !b->kv_len || (b->max_pages && !b->pages))
        return CIDER_ERR_INVALID_ARG;
    const uintptr_t words = reinterpret_cast<uintptr_t>(b->row_start) |
                            reinterpret_cast<uintptr_t>(b->kv_len) | reinterpret_cast<uintptr_t>(b->pages);
    if (!aligned16(b->cache) || (words & 3u))
        return CIDER_ERR_MISALIGNED;
    return CIDER_OK;
}

cider::Kv4Args kv4_args(const cider_kv4_batch *b)
{
    cider::Kv4Args a{};
    a.cache = static_cast<uint8_t *>(b->cache);
    a.pages = b->pages;
    a.row_start = b->row_start;
    a.kv_len = b->kv_len;
    a.batch = (int)b->batch;
    a.rows = (int)b->rows;
    a.max_rows = (int)(b->max_rows < b->rows ? b->max_rows : b->rows);
    a.max_kv_len = (int)b->max_kv_len;
    a.max_pages = (int)b->max_pages;
    a.num_pages = (int)b->num_pages;
    a.kv_heads = (int)b->kv_heads;
    a.head_dim = (int)b->head_dim;
    a.group_size = b->group_size;
    return a;
}

// Checks of the append and read calls; *run says whether anything is to be done.
cider_status check_kv4_rows(const cider_kv4_batch *b, const void *k, const void *v, int dtype,
                            int64_t ldk, int64_t ldv, bool *run)
{
    *run = false;
    cider_status st = check_kv4_sizes(b);
    if (st != CIDER_OK)
        return st;
    const int64_t width = b->kv_heads * b->head_dim;
    if (!dtype_ok(dtype) || ldk < width || ldv < width)
        return CIDER_ERR_INVALID_ARG;
    // one workgroup per head and 32-token block that a sequence may touch
    const int64_t heads = b->batch * b->kv_heads;
    if (heads > kMaxInt || (heads > 0 && b->max_rows / 32 + 2 > kMaxInt / heads))
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    if (kv4_empty(b))
        return CIDER_OK;
    if (!k || !v)
        return CIDER_ERR_INVALID_ARG;
    st = check_kv4_pointers(b);
    if (st != CIDER_OK)
        return st;
    if (!aligned16(k) || !aligned16(v) || ldk % 8 != 0 || ldv % 8 != 0)
        return CIDER_ERR_MISALIGNED;
    if (!device_usable())
        return CIDER_ERR_NO_DEVICE;
    *run = true;
    return CIDER_OK;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sizes, scalars and the host array of a rotation (no device pointer is followed; in an
// empty call none is looked at, as a tensor without elements has none).
cider_status check_rotation(const cider_rotation *r, int64_t head_dim, bool empty)
{
    if (!r || r->rot_dim < 0)
        return CIDER_ERR_INVALID_ARG;
    if (r->rot_dim % 16 != 0 || r->rot_dim > head_dim)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    if ((r->q_weight || r->k_weight) && !(r->eps > 0.0f && std::isfinite(r->eps)))  // NaN fails too
        return CIDER_ERR_INVALID_ARG;
    if (r->rot_dim == 0)
        return CIDER_OK;
    if (r->table_len < 1 || r->axes < 1 || (!r->cos_sin && !empty))
        return CIDER_ERR_INVALID_ARG;
    if (r->table_len > kMaxTokens || r->axes > cider::kMostAxes)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    if (r->axes > 1) {
        if ((!r->positions && !empty) || !r->pair_axis)
            return CIDER_ERR_INVALID_ARG;
        for (int64_t i = 0; i < r->rot_dim / 2; ++i)
            if (r->pair_axis[i] >= r->axes)
                return CIDER_ERR_INVALID_ARG;
    }
    return CIDER_OK;
}

cider::Kv4Rotation rotation_args(const cider_rotation *r)
{
    cider::Kv4Rotation a{};
    a.q_weight = r->q_weight;
    a.k_weight = r->k_weight;
    a.eps = r->eps;
    a.rot_dim = (int)r->rot_dim;
    if (r->rot_dim == 0)
        return a;
    a.table = reinterpret_cast<const float2 *>(r->cos_sin);
    a.positions = r->positions;
    a.table_len = (int)r->table_len;
    a.axes = (int)r->axes;
    a.interleaved = r->interleaved != 0;
    for (int64_t i = 0; r->axes > 1 && i < r->rot_dim / 2; ++i)
        (i < 32 ? a.pair_axis_low : a.pair_axis_high) |= (uint64_t)r->pair_axis[i] << 2 * (i % 32);
    return a;
}

// Sizes and scalars of the attention call.
cider_status check_kv4_attention(const cider_kv4_batch *b, int64_t q_heads, int64_t window, int64_t sinks)
{
    cider_status st = check_kv4_sizes(b);
    if (st != CIDER_OK)
        return st;
    if (q_heads < 1 || window < 0 || sinks < 0)
        return CIDER_ERR_INVALID_ARG;
    if (q_heads % b->kv_heads != 0 || q_heads > kMaxHeads || b->rows * q_heads > kMaxTokens)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    // launches count workgroups in 32 bits: at most one per (row, query head) pair of the longest sequence
    const int64_t pairs = (b->max_rows < b->rows ? b->max_rows : b->rows) * (q_heads / b->kv_heads);
    const int64_t heads = b->batch * b->kv_heads;
    if (heads > kMaxInt || (heads > 0 && pairs > kMaxInt / heads))
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    return CIDER_OK;
}

// Sizes of the runs of a call; *none: there is nothing to share, which makes the call an
// ordinary one.
cider_status check_kv4_runs(const cider_kv4_batch *b, const cider_kv4_runs *r, int64_t q_heads, bool *none)
{
    if (!r || r->groups < 0 || r->max_rows < 0 || r->max_shared_len < 0 ||
        r->max_shared_len > b->max_pages * cider::kPageTokens)
        return CIDER_ERR_INVALID_ARG;
    if (r->groups > kMaxInt || r->max_rows > kMaxTokens)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    *none = r->groups == 0 || r->max_rows == 0 || r->max_shared_len < cider::kPageTokens;
    // workgroups, as for the batch
    const int64_t pairs = (r->max_rows < b->rows ? r->max_rows : b->rows) * (q_heads / b->kv_heads);
    const int64_t heads = r->groups * b->kv_heads;
    if (!*none && (heads > kMaxInt || pairs > kMaxInt / heads))
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    return CIDER_OK;
}

cider::Kv4Runs kv4_runs_args(const cider_kv4_batch *b, const cider_kv4_runs *r)
{
    cider::Kv4Runs a{};
    a.group_start = r->group_start;
    a.shared_len = r->shared_len;
    a.groups = (int)r->groups;
    a.max_rows = (int)(r->max_rows < b->rows ? r->max_rows : b->rows);
    a.max_pages = (int)(r->max_shared_len / cider::kPageTokens);
    return a;
}

cider::Kv4AttentionArgs kv4_attention_args(const cider_kv4_batch *b, int64_t q_heads, int64_t window,
                                           int64_t sinks)
{
    cider::Kv4AttentionArgs a{};
    a.kv = kv4_args(b);
    a.q_heads = (int)q_heads;
    a.tiles = g_kv4_tiles.load(std::memory_order_relaxed);
    a.window = (int)(window < kMaxTokens ? window : 0);  // a window past every length hides nothing
    a.sinks = (int)(sinks < kMaxTokens ? sinks : kMaxTokens);
    return a;
}

// Sizes of an adapter call (no pointer is looked at).
cider_status check_lora(const cider_lora *l, int64_t segments, int64_t rows, int64_t max_rows)
{
    if (!l || l->slots < 1 || l->rank < 1 || l->in_features < 1 || l->slices < 1 || segments < 0 || rows < 0 ||
        max_rows < 0)
        return CIDER_ERR_INVALID_ARG;
    constexpr int64_t kMaxWidth = int64_t(1) << 24;
    if (l->slots > kMaxInt || l->rank % 8 != 0 || l->rank > 128 || l->in_features % 64 != 0 ||
        l->in_features >= kMaxWidth || l->slices > CIDER_LORA_MAX_SLICES || segments > kMaxInt || rows > kMaxTokens ||
        max_rows > kMaxTokens)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    int64_t end = 0;
    for (int64_t i = 0; i < l->slices; ++i) {
        if (l->slice_end[i] <= end)
            return CIDER_ERR_INVALID_ARG;
        end = l->slice_end[i];
        if (end % 64 != 0 || end >= kMaxWidth)
            return CIDER_ERR_UNSUPPORTED_SHAPE;
    }
    // launches count workgroups in 32 bits
    const int64_t tiles = ((max_rows < rows ? max_rows : rows) + 15) / 16, per = end / 64 + l->slices * l->rank;
    if (segments > 0 && tiles > 0 && (tiles > kMaxInt / segments || per > kMaxInt / (segments * tiles)))
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    return CIDER_OK;
}

bool lora_empty(int64_t segments, int64_t rows, int64_t max_rows) { return segments == 0 || rows == 0 || max_rows == 0; }

cider::LoraArgs lora_args(const cider_lora *l, int64_t segments, int64_t rows, int64_t max_rows)
{
    cider::LoraArgs a{};
    a.a = static_cast<const uint16_t *>(l->a);
    a.b = static_cast<const uint16_t *>(l->b);
    a.scale = l->scale;
    a.segments = (int)segments;
    a.rows = (int)rows;
    a.max_rows = (int)(max_rows < rows ? max_rows : rows);
    a.slots = (int)l->slots;
    a.rank = (int)l->rank;
    a.inputs = (int)l->in_features;
    a.slices = (int)l->slices;
    for (int i = 0; i < a.slices; ++i)
        a.ends[i] = (int)l->slice_end[i];
    return a;
}

// Either attention call; runs: null for the ordinary one.
cider_status run_kv4_attention(const cider_kv4_batch *b, const cider_kv4_runs *runs, const void *q, int q_dtype,
                               int64_t ldq, int64_t q_heads, float scale, int64_t window, int64_t sinks,
                               void *workspace, size_t workspace_bytes, void *y, int y_dtype, int64_t ldy,
                               void *stream)
{
    cider_status st = check_kv4_attention(b, q_heads, window, sinks);
    if (st != CIDER_OK)
        return st;
    bool none = true;
    if (runs && (st = check_kv4_runs(b, runs, q_heads, &none)) != CIDER_OK)
        return st;
    const int64_t width = q_heads * b->head_dim;
    if (!dtype_ok(q_dtype) || !dtype_ok(y_dtype) || ldq < width || ldy < width ||
        !(scale > 0.0f && std::isfinite(scale)))  // NaN fails too
        return CIDER_ERR_INVALID_ARG;
    if (kv4_empty(b))
        return CIDER_OK;
    if (!q || !y || (!none && (!runs->group_start || !runs->shared_len)))
        return CIDER_ERR_INVALID_ARG;
    st = check_kv4_pointers(b);
    if (st != CIDER_OK)
        return st;
    if (!aligned16(q) || !aligned16(y) || ldq % 8 != 0 || ldy % 8 != 0 || !aligned16(workspace) ||
        (!none && (!aligned4(runs->group_start) || !aligned4(runs->shared_len))))
        return CIDER_ERR_MISALIGNED;
    cider::Kv4AttentionArgs a = kv4_attention_args(b, q_heads, window, sinks);
    if (!none && (!workspace || workspace_bytes < cider::kv4_shared_workspace(a, kv4_runs_args(b, runs))))
        return CIDER_ERR_WORKSPACE;
    if (!device_usable())
        return CIDER_ERR_NO_DEVICE;
    a.q = static_cast<const uint16_t *>(q);
    a.y = static_cast<uint16_t *>(y);
    a.ldq = ldq;
    a.ldy = ldy;
    a.q_dtype = q_dtype;
    a.y_dtype = y_dtype;
    a.scale = scale;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return from_hip(none ? cider::launch_kv4_attention(a, workspace, workspace_bytes, s)
                         : cider::launch_kv4_attention_shared(a, kv4_runs_args(b, runs), workspace, s));
}

}  // namespace

extern "C" {

int cider_is_available(void) { return device_usable(); }

const char *cider_status_str(int status)
{
    switch (status) {
    case CIDER_OK: return "ok";
    case CIDER_ERR_INVALID_ARG: return "invalid argument";
    case CIDER_ERR_UNSUPPORTED_SHAPE: return "shape outside the supported envelope";
    case CIDER_ERR_MISALIGNED: return "pointer or stride not 16-byte aligned";
    case CIDER_ERR_NO_DEVICE: return "no usable gfx950 device";
    case CIDER_ERR_HIP: return "HIP runtime error at launch";
    case CIDER_ERR_WORKSPACE: return "workspace missing or too small";
    case CIDER_ERR_SCRATCH_LIMIT: return "call needs more than the static scratch array holds";
    default: return "unknown status";
    }
}

cider_status cider_quantize_weight(const void *w_f16, int64_t N, int64_t K, int bits,
                                   int group_size, void *wq, float *s_w, void *stream)
{
    return run_quantize_weight(w_f16, CIDER_DTYPE_F16, N, K, bits, group_size, 100.0, wq, s_w,
                               stream);
}

cider_status cider_quantize_weight_clipped(const void *w_f16, int64_t N, int64_t K, int bits,
                                           int group_size, double clip_percentile, void *wq,
                                           float *s_w, void *stream)
{
    return run_quantize_weight(w_f16, CIDER_DTYPE_F16, N, K, bits, group_size, clip_percentile, wq,
                               s_w, stream);
}

cider_status cider_quantize_weight_ex(const void *w, int w_dtype, int64_t N, int64_t K, int bits,
                                      int group_size, double clip_percentile, void *wq, float *s_w,
                                      void *stream)
{
    return run_quantize_weight(w, w_dtype, N, K, bits, group_size, clip_percentile, wq, s_w,
                               stream);
}

cider_status cider_smooth_fold_weight(const void *w, int w_dtype, int64_t N, int64_t K,
                                      const float *smooth, void *w_out, void *stream)
{
    if (N < 0 || K <= 0 || !dtype_ok(w_dtype))
        return CIDER_ERR_INVALID_ARG;
    if (K % 8 != 0)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    if (N == 0)
        return CIDER_OK;
    if (!w || !smooth || !w_out)
        return CIDER_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(smooth) || !aligned16(w_out))
        return CIDER_ERR_MISALIGNED;
    if (!device_usable())
        return CIDER_ERR_NO_DEVICE;
    return from_hip(cider::launch_smooth_fold(static_cast<const uint16_t *>(w), w_dtype, N, K, smooth,
                                              static_cast<uint16_t *>(w_out),
                                              static_cast<hipStream_t>(stream)));
}

cider_status cider_quantize_act_ex(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                                   const float *smooth, int8_t *xq, float *s_tok, void *stream)
{
    if (M < 0 || K <= 0 || ldx < K || !dtype_ok(x_dtype))
        return CIDER_ERR_INVALID_ARG;
    if (K % 64 != 0 || K > kMaxK)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    if (M == 0)
        return CIDER_OK;
    if (!x || !xq || !s_tok)
        return CIDER_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || ldx % 8 != 0 ||
        (reinterpret_cast<uintptr_t>(s_tok) & 3u) || (smooth && !aligned16(smooth)))
        return CIDER_ERR_MISALIGNED;
    if (!device_usable())
        return CIDER_ERR_NO_DEVICE;
    return from_hip(cider::launch_quantize_rows(static_cast<const uint16_t *>(x), x_dtype, M, K, ldx,
                                                smooth, 8, xq, s_tok,
                                                static_cast<hipStream_t>(stream)));
}

cider_status cider_quantize_act(const void *x_f16, int64_t M, int64_t K, int64_t ldx,
                                int8_t *xq, float *s_tok, void *stream)
{
    return cider_quantize_act_ex(x_f16, CIDER_DTYPE_F16, M, K, ldx, nullptr, xq, s_tok, stream);
}

cider_status cider_w8a8_gemm(const int8_t *xq, const float *s_tok, const int8_t *wq,
                             const float *s_w, int64_t M, int64_t N, int64_t K, int group_size,
                             void *y_f16, void *stream)
{
    return run_product(xq, s_tok, wq, s_w, M, N, K, 8, group_size, cider::OUT_F16, y_f16, stream);
}

cider_status cider_w4a8_gemm(const int8_t *xq, const float *s_tok, const uint8_t *wq4,
                             const float *s_w, int64_t M, int64_t N, int64_t K, int group_size,
                             void *y_f16, void *stream)
{
    return run_product(xq, s_tok, wq4, s_w, M, N, K, 4, group_size, cider::OUT_F16, y_f16, stream);
}

cider_status cider_gemm_ex(const int8_t *xq, const float *s_tok, const void *wq, const float *s_w,
                           int64_t M, int64_t N, int64_t K, int bits, int group_size, int y_dtype,
                           void *y, void *stream)
{
    if (!dtype_ok(y_dtype))
        return CIDER_ERR_INVALID_ARG;
    return run_product(xq, s_tok, wq, s_w, M, N, K, bits, group_size, out_kind_of(y_dtype), y,
                       stream);
}

cider_status cider_w8a8_gemm_i32(const int8_t *xq, const int8_t *wq, int64_t M, int64_t N,
                                 int64_t K, int group_size, int32_t *acc, void *stream)
{
    return run_product(xq, nullptr, wq, nullptr, M, N, K, 8, group_size, cider::OUT_I32, acc,
                       stream);
}

cider_status cider_w4a8_gemm_i32(const int8_t *xq, const uint8_t *wq4, int64_t M, int64_t N,
                                 int64_t K, int group_size, int32_t *acc, void *stream)
{
    return run_product(xq, nullptr, wq4, nullptr, M, N, K, 4, group_size, cider::OUT_I32, acc,
                       stream);
}

size_t cider_linear_workspace_bytes(int64_t M, int64_t K)
{
    if (M <= 0 || K <= 0)
        return 0;
    return round256((size_t)(M * K)) + round256((size_t)M * sizeof(float));
}

size_t cider_linear_workspace_bytes_ex(int64_t M, int64_t N, int64_t K, int bits, int group_size)
{
    const size_t base = cider_linear_workspace_bytes(M, K);
    int path = PATH_GEMM;
    if (check_shape(M, N, K, bits, group_size) != CIDER_OK || M <= 0 || N <= 0 ||
        pick_path(M, N, K, bits, group_size, cider::OUT_F16, &path) != CIDER_OK || path != PATH_GEMM)
        return base;
    const cider::SplitPlan p = cider::plan_split(M, N, K, bits, group_size);
    return p.splits < 2 ? base : base + split_bytes(p);
}

cider_status cider_w8a8_linear(const void *x_f16, int64_t M, int64_t K, int64_t ldx,
                               const int8_t *wq, const float *s_w, int64_t N, int group_size,
                               void *workspace, size_t workspace_bytes, void *y_f16, void *stream)
{
    return run_linear(x_f16, CIDER_DTYPE_F16, M, K, ldx, nullptr, wq, s_w, N, 8, group_size,
                      CIDER_DTYPE_F16, workspace, workspace_bytes, y_f16, stream);
}

cider_status cider_w4a8_linear(const void *x_f16, int64_t M, int64_t K, int64_t ldx,
                               const uint8_t *wq4, const float *s_w, int64_t N, int group_size,
                               void *workspace, size_t workspace_bytes, void *y_f16, void *stream)
{
    return run_linear(x_f16, CIDER_DTYPE_F16, M, K, ldx, nullptr, wq4, s_w, N, 4, group_size,
                      CIDER_DTYPE_F16, workspace, workspace_bytes, y_f16, stream);
}

cider_status cider_linear_ex(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                             const float *smooth, const void *wq, const float *s_w, int64_t N,
                             int bits, int group_size, int y_dtype, void *workspace,
                             size_t workspace_bytes, void *y, void *stream)
{
    return run_linear(x, x_dtype, M, K, ldx, smooth, wq, s_w, N, bits, group_size, y_dtype,
                      workspace, workspace_bytes, y, stream);
}

cider_status cider_linear_ex_noalloc(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                                     const float *smooth, const void *wq, const float *s_w,
                                     int64_t N, int bits, int group_size, int y_dtype, void *y,
                                     void *stream)
{
    return run_linear(x, x_dtype, M, K, ldx, smooth, wq, s_w, N, bits, group_size, y_dtype,
                      nullptr, 0, y, stream, true);
}

cider_status cider_decode_linear(const void *x_f16, int64_t K, const void *wq, const float *s_w,
                                 int64_t N, int bits, int group_size, int y_dtype, void *y,
                                 void *stream)
{
    if (N < 0 || K <= 0 || (bits != 8 && bits != 4) || !dtype_ok(y_dtype))
        return CIDER_ERR_INVALID_ARG;
    if (group_size != 0 && group_size != 64 && group_size != 128)
        return CIDER_ERR_INVALID_ARG;
    if (K % 64 != 0 || K > kDecodeMaxK ||
        (group_size && K % group_size != 0))
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    if (N == 0)
        return CIDER_OK;
    if (!x_f16 || !wq || !s_w || !y)
        return CIDER_ERR_INVALID_ARG;
    if (!aligned16(x_f16) || !aligned16(wq) || (reinterpret_cast<uintptr_t>(s_w) & 3u) ||
        (reinterpret_cast<uintptr_t>(y) & 1u))
        return CIDER_ERR_MISALIGNED;
    if (!device_usable())
        return CIDER_ERR_NO_DEVICE;
    return from_hip(cider::launch_decode(static_cast<const uint16_t *>(x_f16), K, wq, s_w, N, bits,
                                         group_size, out_kind_of(y_dtype), y,
                                         static_cast<hipStream_t>(stream)));
}

size_t cider_lora_workspace_bytes(const cider_lora *lora, int64_t segments, int64_t rows,
                                  int64_t max_rows)
{
    if (check_lora(lora, segments, rows, max_rows) != CIDER_OK || lora_empty(segments, rows, max_rows))
        return 0;
    return cider::lora_workspace(lora_args(lora, segments, rows, max_rows));
}

cider_status cider_lora_add(const cider_lora *lora, const int32_t *seg_start, const int32_t *slot,
                            int64_t segments, int64_t rows, int64_t max_rows, const void *x,
                            int dtype, int64_t ldx, const void *y_in, int64_t ldy_in,
                            void *workspace, size_t workspace_bytes, void *y, int64_t ldy,
                            void *stream)
{
    const cider_status st = check_lora(lora, segments, rows, max_rows);
    if (st != CIDER_OK)
        return st;
    const int64_t outputs = lora->slice_end[lora->slices - 1];
    if (!dtype_ok(dtype) || ldx < lora->in_features || ldy_in < outputs || ldy < outputs)
        return CIDER_ERR_INVALID_ARG;
    if (lora_empty(segments, rows, max_rows))
        return CIDER_OK;
    if (!lora->a || !lora->b || !seg_start || !slot || !x || !y_in || !y)
        return CIDER_ERR_INVALID_ARG;
    if (!aligned16(lora->a) || !aligned16(lora->b) || !aligned4(lora->scale) || !aligned4(seg_start) ||
        !aligned4(slot) || !aligned16(x) || !aligned16(y_in) || !aligned16(y) || !aligned16(workspace) ||
        ldx % 8 != 0 || ldy_in % 8 != 0 || ldy % 8 != 0)
        return CIDER_ERR_MISALIGNED;
    if (y == y_in && ldy != ldy_in)
        return CIDER_ERR_INVALID_ARG;
    cider::LoraArgs a = lora_args(lora, segments, rows, max_rows);
    if (!workspace || workspace_bytes < cider::lora_least_workspace(a))
        return CIDER_ERR_WORKSPACE;
    if (!device_usable())
        return CIDER_ERR_NO_DEVICE;
    a.seg_start = seg_start;
    a.slot = slot;
    a.x = static_cast<const uint16_t *>(x);
    a.y_in = static_cast<const uint16_t *>(y_in);
    a.y = static_cast<uint16_t *>(y);
    a.ldx = ldx;
    a.ldy_in = ldy_in;
    a.ldy = ldy;
    a.dtype = dtype;
    return from_hip(cider::launch_lora_add(a, workspace, workspace_bytes, static_cast<hipStream_t>(stream)));
}

size_t cider_kv4_cache_bytes(int64_t num_pages, int64_t kv_heads, int64_t head_dim, int group_size)
{
    if (check_kv4_geometry(num_pages, kv_heads, head_dim, group_size) != CIDER_OK)
        return 0;
    return (size_t)num_pages * (size_t)kv_heads * cider::kv4_block_bytes((int)head_dim, group_size);
}

cider_status cider_kv4_append(const cider_kv4_batch *b, const void *k, const void *v, int dtype,
                              int64_t ldk, int64_t ldv, void *stream)
{
    bool run = false;
    const cider_status st = check_kv4_rows(b, k, v, dtype, ldk, ldv, &run);
    if (!run)
        return st;
    return from_hip(cider::launch_kv4_append(kv4_args(b), static_cast<const uint16_t *>(k),
                                             static_cast<const uint16_t *>(v), dtype, ldk, ldv,
                                             static_cast<hipStream_t>(stream)));
}

cider_status cider_kv4_append_rotated(const cider_kv4_batch *b, const cider_rotation *rotation,
                                      const void *q, const void *k, const void *v, int dtype,
                                      int64_t ldq, int64_t ldk, int64_t ldv, int64_t q_heads,
                                      void *q_out, int64_t ldq_out, void *stream)
{
    cider_status st = check_kv4_sizes(b);
    if (st != CIDER_OK)
        return st;
    st = check_rotation(rotation, b->head_dim, kv4_empty(b));
    if (st != CIDER_OK)
        return st;
    if (q_heads < 0)
        return CIDER_ERR_INVALID_ARG;
    if (q_heads % b->kv_heads != 0 || q_heads > kMaxHeads)
        return CIDER_ERR_UNSUPPORTED_SHAPE;
    const int64_t width = q_heads * b->head_dim;
    if (width && (ldq < width || ldq_out < width))
        return CIDER_ERR_INVALID_ARG;
    if (!kv4_empty(b) && width) {
        if (!q || !q_out)
            return CIDER_ERR_INVALID_ARG;
        if (!aligned16(q) || !aligned16(q_out) || ldq % 8 != 0 || ldq_out % 8 != 0)
            return CIDER_ERR_MISALIGNED;
        if (q == q_out && ldq != ldq_out)
            return CIDER_ERR_INVALID_ARG;
    }
    if (!kv4_empty(b) && (!aligned16(rotation->q_weight) || !aligned16(rotation->k_weight) ||
                          (rotation->rot_dim && (!aligned16(rotation->cos_sin) || !aligned4(rotation->positions)))))
        return CIDER_ERR_MISALIGNED;
    bool run = false;
    st = check_kv4_rows(b, k, v, dtype, ldk, ldv, &run);
    if (!run)
        return st;
    cider::Kv4Rows io{};
    io.q = static_cast<const uint16_t *>(q);
    io.k = static_cast<const uint16_t *>(k);
    io.v = static_cast<const uint16_t *>(v);
    io.q_out = static_cast<uint16_t *>(q_out);
    io.ldq = ldq;
    io.ldk = ldk;
    io.ldv = ldv;
    io.ldo = ldq_out;
    io.q_heads = (int)q_heads;
    return from_hip(cider::launch_kv4_append_rotated(kv4_args(b), rotation_args(rotation), io, dtype,
                                                     static_cast<hipStream_t>(stream)));
}

cider_status cider_kv4_read(const cider_kv4_batch *b, void *k, void *v, int dtype, int64_t ldk,
                            int64_t ldv, void *stream)
{
    bool run = false;
    const cider_status st = check_kv4_rows(b, k, v, dtype, ldk, ldv, &run);
    if (!run)
        return st;
    return from_hip(cider::launch_kv4_read(kv4_args(b), static_cast<uint16_t *>(k),
                                           static_cast<uint16_t *>(v), dtype, ldk, ldv,
                                           static_cast<hipStream_t>(stream)));
}

cider_status cider_kv4_attention(const cider_kv4_batch *b, const void *q, int q_dtype, int64_t ldq,
                                 int64_t q_heads, float scale, int64_t window, int64_t sinks,
                                 void *workspace, size_t workspace_bytes, void *y, int y_dtype,
                                 int64_t ldy, void *stream)
{
    return run_kv4_attention(b, nullptr, q, q_dtype, ldq, q_heads, scale, window, sinks, workspace,
                             workspace_bytes, y, y_dtype, ldy, stream);
}

size_t cider_kv4_attention_workspace_bytes(const cider_kv4_batch *b, int64_t q_heads,
                                           int64_t window, int64_t sinks)
{
    if (check_kv4_attention(b, q_heads, window, sinks) != CIDER_OK || kv4_empty(b))
        return 0;
    return cider::kv4_attention_workspace(kv4_attention_args(b, q_heads, window, sinks));
}

cider_status cider_kv4_attention_shared(const cider_kv4_batch *b, const cider_kv4_runs *runs,
                                        const void *q, int q_dtype, int64_t ldq, int64_t q_heads,
                                        float scale, void *workspace, size_t workspace_bytes,
                                        void *y, int y_dtype, int64_t ldy, void *stream)
{
    if (!runs)
        return CIDER_ERR_INVALID_ARG;
    return run_kv4_attention(b, runs, q, q_dtype, ldq, q_heads, scale, 0, 0, workspace, workspace_bytes, y,
                             y_dtype, ldy, stream);
}

size_t cider_kv4_attention_shared_workspace_bytes(const cider_kv4_batch *b,
                                                  const cider_kv4_runs *runs, int64_t q_heads)
{
    bool none = true;
    if (check_kv4_attention(b, q_heads, 0, 0) != CIDER_OK || check_kv4_runs(b, runs, q_heads, &none) != CIDER_OK ||
        kv4_empty(b))
        return 0;
    const cider::Kv4AttentionArgs a = kv4_attention_args(b, q_heads, 0, 0);
    return none ? cider::kv4_attention_workspace(a) : cider::kv4_shared_workspace(a, kv4_runs_args(b, runs));
}

int cider_kv4_set_tiles(int columns)
{
    if (columns != 0 && columns != 16 && columns != 128 && columns != 256)
        return -1;
    return g_kv4_tiles.exchange(columns);
}

int cider_set_path(int path)
{
    if (path < 0 || path > 2)
        return -1;
    return g_path.exchange(path);
}

}  // extern "C"
