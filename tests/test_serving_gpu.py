"""What stands around the cache's attention, run together as a server does: adapters beside the products, norm and
rotation into the cache, attention over shared prefixes; prompts, then steps from a graph."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests import rotate_reference as rr
from tests.test_kv4_gpu import i32
from tests.test_kv4_rotate_gpu import table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.mark.parametrize("args", [["--rotate"], ["--adapters", "2"], ["--shared", "70"],
                                  ["--rotate", "--adapters", "3", "--shared", "130", "--prompt", "300"]])
def test_attention_block(args):
    from examples import attention_block
    gu.announce("attention block " + " ".join(args))
    r = attention_block.main(["--batch", "3", "--prompt", "150", "--steps", "8"] + args)
    assert r["finite"]
    # as without them: what 4 bits of keys and values cost
    assert 0.02 < r["error"] < 0.3


def test_steps_against_64_bits():
    """Two steps of 5 sequences, three of them behind one prefix, two adapters: every operator's output is checked
    against 64 bits on what the one before it left."""
    import torch
    r = np.random.default_rng(3)
    D, gs, H, G, K, dtype = 128, 64, 2, 3, 256, 0
    HQ, width = H * G, (H * G + 2 * H) * D
    lens, shared, B = [200, 190, 215, 0, 70], 128, 5
    half = lambda *shape: ref.to_f64(ref.to_bits(r.standard_normal(shape), 0), 0)  # noqa: E731
    dev = lambda x: gu.bits_to_dev(ref.to_bits(x, 0))  # noqa: E731
    a, b = half(2, 3 * 16, K) / 16, half(2, width, 16) / 4
    lora = cider.cider_lora(dev(a), dev(b), None, 2, 16, K, [HQ * D, (HQ + H) * D, width])
    a, b = (ref.to_f64(ref.to_bits(t, 0), 0) for t in (a, b))
    w = r.uniform(0.5, 1.5, D).astype(np.float32)
    turn = rr.Rotation(table_of(300, D), q_weight=w, k_weight=w)
    dw, dt = torch.from_numpy(w).cuda(), torch.from_numpy(turn.table).cuda()
    rotation = cider.cider_rotation(dt, 300, D, q_weight=dw, k_weight=dw)
    # the cache before the first step: sequences 0 - 2 share two pages
    table = np.arange(20).reshape(5, 4).astype(np.int32)
    table[1:3, :2] = table[0, :2]
    cache = ref.Cache(np.full((20, H, ref.block_bytes(D, gs)), 0xFF, np.uint8), D, gs)
    k, v = ([half(n, H, D) for n in lens] for _ in range(2))
    for t in (k, v):
        t[1][:shared], t[2][:shared] = t[0][:shared], t[0][:shared]
    ref.fill(cache, table, lens, k, v)
    dcache, pages = torch.from_numpy(cache.data.copy()).cuda(), i32(table)
    slots, starts = [0, 1, 0, -1, 1], np.arange(B + 1)
    kv, row_start, slot = i32(lens), i32(starts), i32(slots)
    runs = cider.cider_kv4_runs(i32([0, 3]), i32([shared]), 1, 3, shared)
    batch = cider.cider_kv4_batch(dcache, pages, row_start, kv, B, B, 1, 256, 4, 20, H, D, gs)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    qkv, y = (torch.zeros((B, n), dtype=torch.int16, device="cuda") for n in (width, HQ * D))
    x, base = torch.zeros((B, K), dtype=torch.int16, device="cuda"), torch.zeros((B, width), dtype=torch.int16, device="cuda")

    def step():
        cider.cider_lora_add(lora, row_start, slot, B, B, 1, x, 0, K, base, width, ws, ws.numel(), qkv, width)
        cider.cider_kv4_append_rotated(batch, rotation, qkv, qkv[:, HQ * D:], qkv[:, (HQ + H) * D:], 0, width, width, width,
                                       HQ, q, HQ * D)
        cider.cider_kv4_attention_shared(batch, runs, q, 0, HQ * D, HQ, 0.0883, ws, ws.numel(), y, 0, HQ * D)

    q = torch.zeros((B, HQ * D), dtype=torch.int16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    kv += 1
    step()  # eager once, on zeros; the graph's replays append to the same places
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    kv -= 1
    for n in range(2):
        xs, bs = half(B, K), half(B, width)
        x.copy_(dev(xs))
        base.copy_(dev(bs))
        kv += 1
        lens = [t + 1 for t in lens]
        graph.replay()
        torch.cuda.synchronize()
        rows = ref.to_f64(gu.bits_to_host(qkv), 0)
        for i, s in enumerate(slots):
            want = bs[i].copy()
            if s >= 0:
                for j, (lo, hi) in enumerate(((0, HQ * D), (HQ * D, (HQ + H) * D), ((HQ + H) * D, width))):
                    want[lo:hi] += b[s, lo:hi] @ (a[s, 16 * j:16 * j + 16] @ xs[i])
            # halves' rounding and fp32 sums of a few units: far below the output's step
            assert (np.abs(rows[i] - want) <= 2.0 ** -14 + rr.half_step(0, want) * 1.01).all()
        heads = rows.reshape(B, -1, D)
        rr.put_keys(cache, table, lens, [1] * B, heads[:, HQ:HQ + H], heads[:, HQ + H:], turn, gs)
        assert np.array_equal(gu.to_host(dcache), cache.data)
        qs = ref.to_f64(gu.bits_to_host(q), 0).reshape(B, HQ, D)
        got = ref.to_f64(gu.bits_to_host(y), 0).reshape(B, HQ, D)
        for i in range(B):
            want, bound = turn.apply(heads[i, :HQ], w, i, lens[i] - 1)
            assert (np.abs(qs[i] - want) <= bound + rr.half_step(0, np.abs(want) + bound)).all()
            want, bound = ref.attention(cache, table[i], lens[i], qs[i:i + 1], G, 0.0883, 0, 0)
            assert (np.abs(got[i] - want[0]) <= bound[0] + rr.half_step(0, np.abs(want[0]) + bound[0])).all()
