"""cider_kv4_append_rotated with NaN and infinity in keys and queries: what the formula makes of them in 64 bits is what
the cache and q' hold, as a scale that is no number or infinite, and every other group, head and token is as it would be
without them.  Without norm and turn, the append's own bits."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests import rotate_reference as rr
from tests.test_kv4_gpu import GEOMETRY, Setup
from tests.test_kv4_rotate_gpu import heads, rotation_of, run

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


INF, NAN = np.inf, np.nan
# (row, head, element, value) of keys and of queries; elements in either group of a head
SPOILT = [(0, 0, 5, NAN), (2, 1, 40, INF), (3, 0, 63, -INF), (9, 1, 0, NAN), (9, 1, 1, INF), (20, 0, 17, -INF),
          (20, 0, 30, INF), (33, 1, 62, NAN)]


def spoil(x, D):
    """Half of the values in the head's second half; the rows that are spoilt."""
    for i, (row, head, d, value) in enumerate(SPOILT):
        x[row, head, d + (D - 64 if i % 2 else 0)] = value
    return x


def reference(s, t, k, v):
    """The cache by the formula, and which scales of K [page, head, group, token] it makes not finite (their tokens'
    codes are of no value)."""
    want = ref.Cache(s.cache.data.copy(), s.D, s.gs)
    before = want.scales(0).copy()
    with np.errstate(invalid="ignore", over="ignore"):
        rr.put_keys(want, s.table, s.lens, s.n, k, v, t, s.gs)
    after = want.scales(0)
    return want, ~np.isfinite(after) & (after.view(np.uint32) != before.view(np.uint32))


def check_cache(s, want, bad):
    got = ref.Cache(gu.to_host(s.dcache), s.D, s.gs)
    assert bad.any()
    a, b = got.scales(0)[bad], want.scales(0)[bad]
    assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(b)], b[~np.isnan(b)])
    # the codes and scales of the tokens' groups apart, bit for bit
    byte, high = got.places[0]
    data = [x.data.copy() for x in (got, want)]
    for page, head, group, token in zip(*np.nonzero(bad)):
        at = slice(group * s.gs, (group + 1) * s.gs)
        scale = 64 * s.D + 4 * (group * 64 + token)
        for x in data:
            for d in range(s.D)[at]:
                x[page, head, byte[token, d]] &= 0x0F if high[token, d] else 0xF0
            x[page, head, scale:scale + 4] = 0
    assert np.array_equal(data[0], data[1])


def check_queries(s, t, q, dtype, got):
    row = 0
    for b, (kv, n) in enumerate(zip(s.lens, s.n)):
        for i in range(n):
            with np.errstate(invalid="ignore", over="ignore"):
                y, bound = t.apply(q[row], t.q_weight, row, kv - n + i)
                g = ref.to_f64(got[row], dtype)
                fine = np.isfinite(y)
                assert np.array_equal(np.isnan(g), np.isnan(y))
                assert np.array_equal(g[np.isinf(y)], y[np.isinf(y)])
                e = np.abs(g - y)[fine]
                assert (e <= (bound + rr.half_step(dtype, np.abs(y) + bound))[fine]).all()
            row += 1


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("D,gs", GEOMETRY)
@pytest.mark.parametrize("turn", [(64, False, 1, True), (64, True, 1, False), (48, False, 3, True), (32, True, 2, False),
                                  (0, False, 1, True), (0, False, 1, False)])
@pytest.mark.parametrize("rows", [[38], [2, 3, 1, 4, 7, 6, 8, 7]])
def test_by_the_formula(rows, turn, D, gs, dtype):
    """Many rows of a sequence, and few of several."""
    s = Setup([n + 50 * i for i, n in enumerate(rows)], rows, 2, D, gs, seed=D + gs)
    s.to_device()
    q, k, v = heads(s, 2, dtype)
    q, k = spoil(q, D), spoil(k, D)
    t = rotation_of(s, turn, 7)
    want, bad = reference(s, t, k, v)
    got = run(s, t, q, k, v, dtype, 2)
    check_cache(s, want, bad)
    check_queries(s, t, q, dtype, got)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("D,gs", GEOMETRY)
def test_without_norm_and_turn_it_is_the_append(D, gs, dtype):
    """NaN's own bits apart, which no one reads."""
    s = Setup([70, 130], [70, 5], 2, D, gs, seed=3)
    batch = s.to_device()
    q, k, v = heads(s, 1, dtype)
    k, v = spoil(k, D), spoil(v, D)
    dk, dv = (gu.bits_to_dev(ref.to_bits(x, dtype).reshape(s.rows, -1)) for x in (k, v))
    cider.cider_kv4_append(batch, dk, dv, dtype, 2 * D, 2 * D)
    want = ref.Cache(gu.to_host(s.dcache), D, gs)
    s.to_device()
    run(s, rr.Rotation(), q, k, v, dtype, 1)
    got = ref.Cache(gu.to_host(s.dcache), D, gs)
    assert np.array_equal(got.data[:, :, :64 * D], want.data[:, :, :64 * D])
    for which in (0, 1):
        a, b = got.scales(which), want.scales(which)
        none = np.isnan(b)
        assert none.any() and np.array_equal(np.isnan(a), none)
        assert np.array_equal(a[~none].view(np.uint32), b[~none].view(np.uint32))


@pytest.mark.parametrize("norm,value", [(False, NAN), (True, NAN), (True, INF)])
def test_the_attention_meets_it(norm, value):
    """A key with NaN (or, normed, infinity) makes the rows that see its token NaN, and no others."""
    import torch
    s = Setup([40, 30], [40, 30], 1, 128, 64, seed=5)
    batch = s.to_device()
    q, k, v = heads(s, 2, 0)
    k[25, 0, 3] = value
    w = np.ones(128, np.float32) if norm else None
    got = run(s, rr.Rotation(q_weight=w, k_weight=w), q, k, v, 0, 2)
    y = torch.zeros((s.rows, 256), dtype=torch.int16, device="cuda")
    need = cider.cider_kv4_attention_workspace_bytes(batch, 2, 0, 0)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    cider.cider_kv4_attention(s.batch(s.dcache), gu.bits_to_dev(got.reshape(s.rows, -1)), 0, 256, 2, 0.1, 0, 0, ws, need, y,
                              0, 256)
    out = np.isnan(ref.to_f64(gu.bits_to_host(y), 0))
    assert out[25:40].all() and not out[:25].any() and not out[40:].any()
