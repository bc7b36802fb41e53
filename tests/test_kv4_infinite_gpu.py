"""Attention over caches whose keys or values have infinite scales (an infinite key or value was appended): a row that may
see such a token has no finite output where the formula has none, whatever the signs, and other rows have theirs as if
the token were not there.  Both attentions, every tile."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests.test_kv4_gpu import GEOMETRY, TILES, i32, reference
from tests.test_kv4_shared_gpu import attend, runs_of, setup_of

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
    cider.cider_kv4_set_tiles(0)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("D,gs", GEOMETRY)
@pytest.mark.parametrize("group", [0, -1])
@pytest.mark.parametrize("token", [70, 215])
@pytest.mark.parametrize("which", ["key", "value"])
def test_an_infinite_scale_is_not_hidden(which, token, group, D, gs, tiles):
    """Token 70 is in a shared page, 215 behind them; rows of the first sequence stand at 190 .. 229."""
    cider.cider_kv4_set_tiles(tiles)
    s = setup_of([230, 200, 130], [40, 3, 2], 1, D, gs, [0, 2], [128], 0, seed=6)
    q = ref.to_bits(s.rng.standard_normal((s.rows, 4, D)) * 2, 0)
    want = reference(s, q, 0, 4, 0.1)
    at = 64 * D + (256 * (D // gs) if which == "value" else 0) + 4 * (group % (D // gs) * 64 + token % 64)
    s.cache.data[s.table[0, token // 64], 0, at:at + 4] = np.array([np.inf], np.float32).view(np.uint8)
    batch = s.to_device()
    outs = [attend(s, batch, runs_of(s, [0, 2], [128]), q, 0, 0, 4, 0.1),
            attend(s, batch, runs_of(s, [], []), q, 0, 0, 4, 0.1)]
    # the group's codes of a value: those of 0 have no product with infinity, the others an infinite one
    elements = slice(group % (D // gs) * gs, (group % (D // gs) + 1) * gs)
    for got in outs:
        g = ref.to_f64(got, 0)
        for b in range(3):
            for i in range(s.n[b]):
                sees = token <= s.lens[b] - s.n[b] + i and (b == 0 or b == 1 and token == 70)
                y, mine = want[b][0][i], g[s.row_start[b] + i]
                bad = np.zeros(D, bool)
                if sees:
                    bad[slice(None) if which == "key" else elements] = True
                    assert not np.isfinite(mine[:, bad]).any()
                    if which == "key":
                        assert np.isnan(mine).all()
                fine = ~bad
                bound = want[b][1][i]
                err = np.abs(mine - y)[:, fine]
                assert (err <= (bound + 2.0 ** -11 * (np.abs(y) + bound) + 2.0 ** -25)[:, fine]).all()
