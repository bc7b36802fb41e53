// The launches of an attention call over shared prefixes, on the host: the library's own sources compiled for the host
// alone, with a runtime that writes down what is launched instead of launching it.  For each launch over pages, every
// workgroup of its grid, the surplus that a wide grid is rounded up to among them, is asked what it has; those that have
// something must be as many as the plan deals out, each once, within the plan's tiles and the workspace's slots.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "kv4_attention.h"

namespace {
struct Launched {
    unsigned x, y, threads;
    cider::Kv4AttentionArgs a;
    cider::Kv4Launch n;
};
std::vector<Launched> launched;
}  // namespace

extern "C" {
hipError_t hipLaunchKernel(const void *, dim3 grid, dim3 block, void **args, size_t, hipStream_t)
{
    launched.push_back({grid.x, grid.y, block.x, *static_cast<cider::Kv4AttentionArgs *>(args[0]),
                        *static_cast<cider::Kv4Launch *>(args[1])});
    return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3 *, dim3 *, size_t *, hipStream_t *) { return hipSuccess; }
void **__hipRegisterFatBinary(const void *) { return nullptr; }
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *, char *, const char *, unsigned, void *, void *, void *, void *, int *) {}
void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}
}

// batch rows max_rows max_kv_len kv_heads q_heads head_dim groups run_rows max_shared_len tiles
int main(int argc, char **argv)
{
    if (argc != 12)
        return 2;
    auto arg = [&](int i) { return atoi(argv[i]); };
    cider::Kv4AttentionArgs a{};
    a.kv.batch = arg(1);
    a.kv.rows = arg(2);
    a.kv.max_rows = arg(3);
    a.kv.max_kv_len = arg(4);
    a.kv.max_pages = (a.kv.max_kv_len + 63) / 64;
    a.kv.num_pages = 1;
    a.kv.kv_heads = arg(5);
    a.q_heads = arg(6);
    a.kv.head_dim = arg(7);
    a.kv.group_size = 64;
    a.tiles = arg(11);
    cider::Kv4Runs r{};
    r.groups = arg(8);
    r.max_rows = arg(9);
    r.max_pages = arg(10) / cider::kPageTokens;
    if (cider::launch_kv4_attention_shared(a, r, reinterpret_cast<void *>(256), nullptr) != hipSuccess)
        return 3;
    launched.pop_back();  // the join
    int wrong = 0;
    for (const Launched &l : launched) {
        const unsigned long long grid = (unsigned long long)l.x * l.y;
        const unsigned own = (unsigned)l.n.tiles * l.n.splits * l.a.kv.kv_heads * l.a.kv.batch;
        const unsigned front = (unsigned)l.n.front_tiles * l.n.front_splits * l.a.kv.kv_heads * l.n.runs.groups;
        unsigned long long busy = 0, outside = 0;
        std::vector<bool> seen[2] = {std::vector<bool>(own), std::vector<bool>(l.n.front_groups ? front : 0)};
        for (unsigned long long id = 0; id < grid; ++id) {
            cider::Work w;
            if (!cider::work_of<cider::Pages::Shared>(l.a, l.n, (unsigned)id, w))
                continue;
            ++busy;
            const int splits = w.front ? l.n.front_splits : l.n.splits, batch = w.front ? l.n.runs.groups : l.a.kv.batch;
            const int tiles = w.front ? l.n.front_tiles : l.n.tiles, slot = w.split + (w.front ? 0 : l.n.front_splits);
            const bool in = w.head >= 0 && w.head < l.a.kv.kv_heads && w.b >= 0 && w.b < batch && w.split >= 0 &&
                            w.split < splits && slot < l.n.slots && w.tile >= 0 && w.tile < tiles;
            std::vector<bool> &taken = seen[w.front];
            const size_t at = in ? ((size_t)(w.tile * (size_t)splits + w.split) * batch + w.b) * l.a.kv.kv_heads + w.head : 0;
            if (!in || at >= taken.size() || taken[at])
                ++outside;
            else
                taken[at] = true;
        }
        const unsigned long long planned = (unsigned long long)l.n.front_groups + own;
        wrong += busy != planned || outside || (l.n.front_groups && l.n.front_groups != front) || grid < planned;
        printf("columns %d grid %llu planned %llu busy %llu outside %llu front %u splits %d + %d of %d slots\n", l.n.cols, grid,
               planned, busy, outside, l.n.front_groups, l.n.front_splits, l.n.splits, l.n.slots);
    }
    return wrong != 0;
}
