"""Rotation into the cache and adapters with so many sequences, heads and segments, most of them without rows, that a
launch has more than 2^22 workgroups and is rounded up to whole rows of those: each kernel, with its results."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests import rotate_reference as rr
from tests.test_kv4_gpu import Setup, i32
from tests.test_kv4_rotate_gpu import heads, on_device, rotation_of
from tests.test_lora_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert cider.cider_is_available(), "libcider.so reports no usable gfx950 device"
    yield


@pytest.fixture(autouse=True)
def _announce(request):
    gu.announce(request.node.nodeid)
    yield


@pytest.mark.parametrize("max_rows,batch", [(1, 70000), (40, 30000)])
def test_rotation(max_rows, batch):
    """Two sequences with rows, the first and the last; 64 heads."""
    import torch
    H, D = 64, 64
    n = min(max_rows, 35)
    s = Setup([n + 70, 67], [n, 1], H, D, 64, seed=11)
    s.to_device()
    q, k, v = heads(s, 1, 0)
    t = rotation_of(s, (64, False, 1, True), 5)
    starts = np.full(batch + 1, n + 1, np.int32)
    starts[0], starts[1:batch] = 0, n
    kv = np.zeros(batch, np.int32)
    kv[0], kv[-1] = s.lens
    table = torch.full((batch, s.max_pages), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    table[0], table[-1] = i32(s.table[0]), i32(s.table[1])
    rows = max(max_rows, n + 1)  # as many as the bound says
    b = cider.cider_kv4_batch(s.dcache, table, i32(starts), i32(kv), batch, rows, max_rows, s.max_pages * 64, s.max_pages,
                              s.num_pages, H, D, 64)
    pad = lambda x: np.concatenate([ref.to_bits(x, 0).reshape(s.rows, -1), np.full((rows - s.rows, H * D), 0x7E00, np.uint16)])  # noqa: E731
    data = [gu.bits_to_dev(pad(x)) for x in (q, k, v)]
    out = torch.full((rows, H * D), 99, dtype=torch.int16, device="cuda")
    cider.cider_kv4_append_rotated(b, on_device(t, rows), *data, 0, H * D, H * D, H * D, H, out, H * D)
    want = ref.Cache(s.cache.data.copy(), D, 64)
    rr.put_keys(want, s.table, s.lens, s.n, k, v, t, 64)
    assert np.array_equal(gu.to_host(s.dcache), want.data)
    got = gu.bits_to_host(out).reshape(rows, H, D)
    assert (got[s.rows:] == 99).all()
    for row in range(s.rows):
        y, bound = t.apply(q[row], t.q_weight, row, 70 + row if row < n else 66)
        e = np.abs(ref.to_f64(got[row], 0) - y)
        assert (e <= bound + rr.half_step(0, np.abs(y) + bound)).all()


@pytest.mark.parametrize("segments,rank,ends", [
    (100000, 16, [8192, 24576]),               # the product with B, rows of B in registers
    (200000, 64, [24576]),                     # and in common
    (300000, 128, list(range(64, 513, 64))),   # the product with A
])
def test_adapters(segments, rank, ends):
    """Four segments with rows, the last among them; bounded to 40 rows each."""
    counts, slots = np.zeros(segments, np.int64), np.full(segments, -1)
    counts[[0, 7, segments // 2, segments - 1]] = 3, 2, 34, 1
    slots[[0, 7, segments // 2, segments - 1]] = 1, -1, 0, 3
    c = Case(counts, slots, rank, 64, ends, 1, seed=41)
    c.check(c.run(max_rows=40))
