"""cider_kv4_attention_shared with bounds so wide that its launches have more than 2^22 workgroups, most of which have
nothing to do: shared pages in a launch of their own beside tiles of many columns, and both parts in one.  The launches'
arithmetic is checked on the host first (tests/test_kv4_shared_launches_cpu.py)."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests.test_kv4_gpu import compare, i32, reference
from tests.test_kv4_shared_gpu import setup_of

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


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("max_rows,batch", [(512, 5), (1, 600)])
def test_wide_bounds(max_rows, batch, dtype):
    """1100 runs bounded to 262144 shared tokens, most of them empty; the last sequence has 40 pages of its own."""
    import torch
    H, HQ, D, groups, pages = 8, 32, 64, 1100, 4688
    many = max_rows > 1
    lens, rows = [200, 190, 350, 330, 2600], [1, 3, 2, 1, 4] if many else [1] * 5
    s = setup_of(lens, rows, H, D, 64, [0, 2, 4], [128, 320], dtype, seed=31 + many)
    s.to_device()
    table = torch.full((batch, pages), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    table[:5, :s.max_pages] = i32(s.table)
    starts = np.full(batch + 1, s.rows, np.int32)
    starts[:6] = s.row_start
    kv = np.zeros(batch, np.int32)
    kv[:5] = s.lens
    b = cider.cider_kv4_batch(s.dcache, table, i32(starts), i32(kv), batch, s.rows, max_rows, 300000, pages, s.num_pages,
                              H, D, 64)
    first = np.full(groups + 1, 4, np.int32)
    first[:2] = 0, 2
    runs = cider.cider_kv4_runs(i32(first), i32([128, 320] + [262144] * (groups - 2)), groups, 16, 262144)
    q = ref.to_bits(s.rng.standard_normal((s.rows, HQ, D)) * 2, dtype)
    qd = gu.bits_to_dev(q.reshape(s.rows, -1))
    y = torch.full((s.rows, HQ * D), 99, dtype=torch.int16, device="cuda")
    need = cider.cider_kv4_attention_shared_workspace_bytes(b, runs, HQ)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    gu.sync()
    cider.cider_kv4_attention_shared(b, runs, qd, dtype, HQ * D, HQ, 0.125, ws, need, y, dtype, HQ * D)
    gu.sync()
    assert (ws[need:] == 0xFF).all()
    compare(s, gu.bits_to_host(y).reshape(s.rows, HQ, D), reference(s, q, dtype, HQ, 0.125), dtype)
