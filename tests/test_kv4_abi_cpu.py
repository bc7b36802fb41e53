"""The cache calls' argument checks on the host (no kernel is launched: the
library is told that there is no device), and the reference that the GPU tests
compare with, pinned by the layout's own properties."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import kv4_reference as ref

P, BAD, ODD = 0x10000, 0x10008, 0x10002


@pytest.fixture(autouse=True)
def _no_device(monkeypatch):
    monkeypatch.setenv("CIDER_FORCE_UNAVAILABLE", "1")


def _batch(**kw):
    a = dict(cache=P, pages=P, row_start=P, kv_len=P, batch=3, rows=5, max_rows=3, max_kv_len=256, max_pages=4,
             num_pages=9, kv_heads=2, head_dim=128, group_size=64)
    a.update(kw)
    return cider.cider_kv4_batch(*a.values())


def _append(b=None, k=P, v=P, dtype=0, ldk=256, ldv=256, f=None, **kw):
    f = f or cider.cider_kv4_append
    return f(b or _batch(**kw), k, v, dtype, ldk, ldv, stream=0, check=False)


def _attend(q=P, q_dtype=0, ldq=1024, q_heads=8, scale=0.1, window=0, sinks=0, ws=None, nbytes=0, y=P, y_dtype=0,
            ldy=1024, **kw):
    return cider.cider_kv4_attention(_batch(**kw), q, q_dtype, ldq, q_heads, scale, window, sinks, ws, nbytes, y,
                                     y_dtype, ldy, stream=0, check=False)


SHARED = [
    (dict(), cider.CIDER_ERR_NO_DEVICE),
    (dict(head_dim=64), cider.CIDER_ERR_NO_DEVICE),
    (dict(group_size=128), cider.CIDER_ERR_NO_DEVICE),
    (dict(head_dim=64, group_size=128), cider.CIDER_ERR_UNSUPPORTED_SHAPE),
    (dict(head_dim=96), cider.CIDER_ERR_UNSUPPORTED_SHAPE),
    (dict(head_dim=0), cider.CIDER_ERR_INVALID_ARG),
    (dict(group_size=0), cider.CIDER_ERR_INVALID_ARG),
    (dict(group_size=32), cider.CIDER_ERR_INVALID_ARG),
    (dict(kv_heads=0), cider.CIDER_ERR_INVALID_ARG),
    (dict(num_pages=0), cider.CIDER_ERR_INVALID_ARG),
    (dict(num_pages=1 << 31), cider.CIDER_ERR_UNSUPPORTED_SHAPE),
    (dict(batch=-1), cider.CIDER_ERR_INVALID_ARG),
    (dict(rows=-1), cider.CIDER_ERR_INVALID_ARG),
    (dict(max_rows=-1), cider.CIDER_ERR_INVALID_ARG),
    (dict(max_kv_len=-1), cider.CIDER_ERR_INVALID_ARG),
    (dict(max_kv_len=257), cider.CIDER_ERR_INVALID_ARG),
    (dict(max_pages=1 << 25), cider.CIDER_ERR_UNSUPPORTED_SHAPE),
    (dict(rows=(1 << 30) + 1), cider.CIDER_ERR_UNSUPPORTED_SHAPE),
    (dict(batch=1 << 30, max_rows=1 << 20, rows=1 << 20), cider.CIDER_ERR_UNSUPPORTED_SHAPE),
    (dict(cache=None), cider.CIDER_ERR_INVALID_ARG),
    (dict(pages=None), cider.CIDER_ERR_INVALID_ARG),
    (dict(row_start=None), cider.CIDER_ERR_INVALID_ARG),
    (dict(kv_len=None), cider.CIDER_ERR_INVALID_ARG),
    (dict(cache=BAD), cider.CIDER_ERR_MISALIGNED),
    (dict(kv_len=ODD), cider.CIDER_ERR_MISALIGNED),
    (dict(batch=0, cache=None), cider.CIDER_OK),
    (dict(rows=0, cache=None), cider.CIDER_OK),
    (dict(max_rows=0, cache=None), cider.CIDER_OK),
    (dict(max_pages=0, max_kv_len=0, pages=None), cider.CIDER_ERR_NO_DEVICE),
]


@pytest.mark.parametrize("kw,status", SHARED)
def test_batch_checks(kw, status):
    assert _append(**kw) == status
    assert _append(f=cider.cider_kv4_read, **kw) == status
    assert _attend(**kw) == status


def test_append_and_read_checks():
    for f in (cider.cider_kv4_append, cider.cider_kv4_read):
        assert _append(k=None, f=f) == cider.CIDER_ERR_INVALID_ARG
        assert _append(v=None, f=f) == cider.CIDER_ERR_INVALID_ARG
        assert _append(dtype=2, f=f) == cider.CIDER_ERR_INVALID_ARG
        assert _append(ldk=248, f=f) == cider.CIDER_ERR_INVALID_ARG
        assert _append(ldv=248, f=f) == cider.CIDER_ERR_INVALID_ARG
        assert _append(ldk=260, f=f) == cider.CIDER_ERR_MISALIGNED
        assert _append(k=BAD, f=f) == cider.CIDER_ERR_MISALIGNED
        assert _append(v=BAD, f=f) == cider.CIDER_ERR_MISALIGNED
        assert f(None, P, P, 0, 256, 256, stream=0, check=False) == cider.CIDER_ERR_INVALID_ARG


def test_attention_checks():
    inf, nan = float("inf"), float("nan")
    for kw in (dict(q=None), dict(y=None), dict(q_dtype=7), dict(y_dtype=-1), dict(ldq=1016), dict(ldy=1016),
               dict(q_heads=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf), dict(scale=nan),
               dict(window=-1), dict(sinks=-1)):
        assert _attend(**kw) == cider.CIDER_ERR_INVALID_ARG, kw
    for kw in (dict(q_heads=7), dict(q_heads=1 << 17, ldq=1 << 24, ldy=1 << 24),
               dict(rows=1 << 28, max_rows=1 << 28)):
        assert _attend(**kw) == cider.CIDER_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(q=BAD), dict(y=BAD), dict(ldq=1028), dict(ldy=1028), dict(ws=BAD, nbytes=64)):
        assert _attend(**kw) == cider.CIDER_ERR_MISALIGNED, kw
    for kw in (dict(window=1 << 62, sinks=1 << 62), dict(ws=P, nbytes=1 << 30), dict(q_heads=2)):
        assert _attend(**kw) == cider.CIDER_ERR_NO_DEVICE, kw


def test_sizes():
    assert cider.cider_kv4_cache_bytes(3, 8, 128, 64) == 3 * 8 * 9216
    assert cider.cider_kv4_cache_bytes(3, 8, 128, 128) == 3 * 8 * 8704
    assert cider.cider_kv4_cache_bytes(1, 1, 64, 64) == 4608
    assert cider.cider_kv4_cache_bytes(1 << 30, 8, 128, 64) == (1 << 30) * 8 * 9216
    for bad in ((0, 8, 128, 64), (3, 0, 128, 64), (3, 8, 96, 64), (3, 8, 64, 128), (3, 8, 128, 32)):
        assert cider.cider_kv4_cache_bytes(*bad) == 0
    for kw, window in ((dict(group_size=32), 0), (dict(batch=-1), 0), (dict(), -1)):
        assert cider.cider_kv4_attention_workspace_bytes(_batch(**kw), 8, window, 0) == 0
    assert cider.cider_kv4_attention_workspace_bytes(None, 8, 0, 0) == 0


def test_set_tiles():
    assert cider.cider_kv4_set_tiles(128) == 0
    assert cider.cider_kv4_set_tiles(256) == 128
    assert cider.cider_kv4_set_tiles(16) == 256
    for bad in (1, -16, 64, 512):
        assert cider.cider_kv4_set_tiles(bad) == -1
    assert cider.cider_kv4_set_tiles(0) == 16


def test_workspace_follows_the_sizes():
    """Enough for every split of a long cache, nothing for what is never split; more rows never need less per row."""
    one = _batch(batch=1, rows=1, max_rows=1, max_kv_len=131072, max_pages=2048)
    parts = cider.cider_kv4_attention_workspace_bytes(one, 32, 0, 0)
    assert parts % 256 == 0 and 32 * 2 * (128 * 4 + 8) <= parts <= 32 * 256 * (128 * 4 + 8) + 512
    short = _batch(batch=1, rows=1, max_rows=1, max_kv_len=64, max_pages=2048)
    assert cider.cider_kv4_attention_workspace_bytes(short, 32, 0, 0) == 0
    window = cider.cider_kv4_attention_workspace_bytes(one, 32, 128, 4)
    assert window <= parts


@pytest.mark.parametrize("D,gs", [(64, 64), (128, 64), (128, 128)])
def test_reference_layout_is_one_to_one(D, gs):
    """Every nibble of a block's code bytes is one element of one token, and what is put in comes back."""
    t, d = np.meshgrid(np.arange(64), np.arange(D), indexing="ij")
    for place, at in ((ref.k_place, 0), (ref.v_place, 32 * D)):
        byte, high = place(t, d, D)
        nibbles = np.sort((2 * byte + high).ravel())
        assert np.array_equal(nibbles, np.arange(2 * at, 2 * at + 64 * D))
    r = np.random.default_rng(D + gs)
    c = ref.Cache(r.integers(0, 256, (3, 2, ref.block_bytes(D, gs)), dtype=np.uint8), D, gs)
    x = ref.to_f64(ref.to_bits(r.standard_normal((70, 2, D)), 0), 0)
    ref.fill(c, [[2, 0]], [70], [x], [-x])
    u, s = ref.quantize(x, gs)
    want = (np.repeat(s, gs, -1).astype(np.float64) * (u.astype(np.float64) - 8)).transpose(1, 0, 2)
    assert np.array_equal(c.values(0, [2, 0])[0][:, :70], want)
    assert np.array_equal(c.values(1, [2, 0])[0][:, :70], -want)
    d2 = ref.Cache(c.data.copy(), D, gs)
    d2.put(2, 5, 0, u[5], s[5])
    assert np.array_equal(d2.data, c.data)
    assert np.abs(x.transpose(1, 0, 2) - want).max() <= 0.5 * s.max() * (1 + 1e-6)


def test_reference_attention_by_hand():
    """One head, codes that stand for whole numbers: scores and outputs worked out by hand."""
    D, gs = 64, 64
    c = ref.Cache(np.full((1, 1, ref.block_bytes(D, gs)), 0xFF, np.uint8), D, gs)
    k, v = np.zeros((3, 1, D)), np.zeros((3, 1, D))
    k[:, 0, 0] = [7, 7, -7]
    v[:, 0, 1] = [7, 14, 21]
    ref.fill(c, [[0]], [3], [k], [v])
    q = np.zeros((2, 1, D))
    q[:, 0, 0] = np.log(2) / 7
    y, _ = ref.attention(c, [0], 3, q, 1, 1.0, 0, 0)
    assert np.allclose(y[0, 0, 1], 10.5) and np.allclose(y[1, 0, 1], (2 * 7 + 2 * 14 + 0.5 * 21) / 4.5)
    y, _ = ref.attention(c, [0], 3, q, 1, 1.0, 1, 0)
    assert np.allclose(y[:, 0, 1], [14, 21])
    y, _ = ref.attention(c, [0], 3, q, 1, 1.0, 1, 1)
    assert np.allclose(y[1, 0, 1], (2 * 7 + 0.5 * 21) / 2.5)
