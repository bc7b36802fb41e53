"""Argument checks of cider_kv4_attention_shared on the host (no kernel is launched: the library is told that there is
no device), and its workspace."""
import pytest

import w4a8_quantized_linear_amd as cider

P, BAD, ODD = 0x10000, 0x10008, 0x10002
INVALID, SHAPE, MISALIGNED = (cider.CIDER_ERR_INVALID_ARG, cider.CIDER_ERR_UNSUPPORTED_SHAPE,
                              cider.CIDER_ERR_MISALIGNED)
YES, ROOM, OK = cider.CIDER_ERR_NO_DEVICE, cider.CIDER_ERR_WORKSPACE, cider.CIDER_OK


@pytest.fixture(autouse=True)
def _no_device(monkeypatch):
    monkeypatch.setenv("CIDER_FORCE_UNAVAILABLE", "1")


def _batch(**kw):
    a = dict(cache=P, pages=P, row_start=P, kv_len=P, batch=3, rows=5, max_rows=3, max_kv_len=256, max_pages=4,
             num_pages=9, kv_heads=2, head_dim=128, group_size=64)
    a.update(kw)
    return cider.cider_kv4_batch(*a.values())


def _runs(**kw):
    a = dict(group_start=P, shared_len=P, groups=1, max_rows=5, max_shared_len=128)
    a.update(kw)
    return cider.cider_kv4_runs(*a.values())


def _call(runs=None, q=P, q_dtype=0, ldq=1024, q_heads=8, scale=0.1, ws=P, nbytes=1 << 30, y=P, y_dtype=0, ldy=1024, **kw):
    return cider.cider_kv4_attention_shared(_batch(**kw), _runs(**(runs or {})), q, q_dtype, ldq, q_heads, scale, ws,
                                            nbytes, y, y_dtype, ldy, stream=0, check=False)


@pytest.mark.parametrize("runs,status", [
    ({}, YES), (dict(groups=3), YES), (dict(max_rows=1 << 30), YES), (dict(max_shared_len=256), YES),
    (dict(groups=-1), INVALID), (dict(max_rows=-1), INVALID), (dict(max_shared_len=-1), INVALID),
    (dict(max_shared_len=257), INVALID), (dict(groups=1 << 31), SHAPE), (dict(max_rows=(1 << 30) + 1), SHAPE),
    (dict(groups=1 << 30), SHAPE),
    (dict(group_start=None), INVALID), (dict(shared_len=None), INVALID), (dict(group_start=ODD), MISALIGNED),
    (dict(shared_len=ODD), MISALIGNED),
    # nothing to share: the ordinary call
    (dict(groups=0, group_start=None, shared_len=None), YES), (dict(max_rows=0, group_start=None), YES),
    (dict(max_shared_len=63, shared_len=ODD), YES),
])
def test_runs_checks(runs, status):
    assert _call(runs) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(y=None), INVALID), (dict(q_dtype=2), INVALID), (dict(y_dtype=-1), INVALID),
    (dict(ldq=1016), INVALID), (dict(ldy=1016), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q_heads=0), INVALID), (dict(q_heads=7), SHAPE), (dict(head_dim=96), SHAPE), (dict(cache=None), INVALID),
    (dict(pages=None), INVALID), (dict(q=BAD), MISALIGNED), (dict(ldq=1028), MISALIGNED), (dict(ws=BAD), MISALIGNED),
    (dict(ws=None), ROOM), (dict(nbytes=0), ROOM), (dict(ws=None, nbytes=0, runs=dict(groups=0)), YES),
    (dict(batch=0, cache=None), OK), (dict(rows=0, q=None), OK), (dict(max_rows=0, ws=None), OK),
])
def test_call_checks(kw, status):
    assert _call(**kw) == status


def test_null_structs():
    assert cider.cider_kv4_attention_shared(_batch(), None, P, 0, 1024, 8, 0.1, P, 1 << 30, P, 0, 1024, stream=0,
                                            check=False) == INVALID
    assert cider.cider_kv4_attention_shared(None, _runs(), P, 0, 1024, 8, 0.1, P, 1 << 30, P, 0, 1024, stream=0,
                                            check=False) == INVALID
    assert cider.cider_kv4_attention_shared_workspace_bytes(None, _runs(), 8) == 0
    assert cider.cider_kv4_attention_shared_workspace_bytes(_batch(), None, 8) == 0


@pytest.mark.parametrize("kw,runs", [
    ({}, {}), (dict(batch=64, rows=64, max_rows=1, max_kv_len=9216, max_pages=144), dict(max_rows=64, max_shared_len=8192)),
    (dict(batch=16, rows=1024, max_rows=64, max_kv_len=65664, max_pages=1026), dict(max_rows=1024, max_shared_len=65536)),
    (dict(batch=2, rows=2, max_rows=1, max_kv_len=1 << 30, max_pages=1 << 24), dict(max_rows=2, max_shared_len=1 << 29)),
])
def test_workspace(kw, runs):
    """At least a part over shared pages and one behind them for every (row, query head) pair, at most 256; the call
    takes exactly that much and nothing less."""
    b, r = _batch(**kw), _runs(**runs)
    need = cider.cider_kv4_attention_shared_workspace_bytes(b, r, 8)
    pair = 8 * b.rows * (128 + 2) * 4
    assert 2 * pair <= need <= 256 * pair + 512
    call = lambda n: cider.cider_kv4_attention_shared(b, r, P, 0, 1024, 8, 0.1, P, n, P, 0, 1024, stream=0, check=False)  # noqa: E731
    assert call(need) == YES and call(need - 1) == ROOM


def test_workspace_of_nothing_shared_is_the_ordinary_one():
    b = _batch(batch=1, rows=1, max_rows=1, max_kv_len=131072, max_pages=2048)
    want = cider.cider_kv4_attention_workspace_bytes(b, 8, 0, 0)
    assert want and cider.cider_kv4_attention_shared_workspace_bytes(b, _runs(groups=0), 8) == want


@pytest.mark.parametrize("tiles", [0, 16, 128, 256])
@pytest.mark.parametrize("max_rows", [1, 3, 200, 4096])
@pytest.mark.parametrize("max_kv_len", [0, 1, 64, 70000])
def test_bounds_of_every_order(max_kv_len, max_rows, tiles):
    """Prefixes' bounds above and below the lengths', 0 among them: the call is planned, with a workspace."""
    rows = 128441
    kw = dict(batch=15443, rows=rows, max_rows=max_rows, max_kv_len=max_kv_len, max_pages=4417, num_pages=1, kv_heads=1)
    cider.cider_kv4_set_tiles(tiles)
    try:
        for groups, run_rows, shared in ((1000, 1271, 57974), (1, 1 << 30, 64), (15443, 8, 1 << 18), (1, rows, 1 << 18)):
            runs = dict(groups=groups, max_rows=run_rows, max_shared_len=shared)
            nbytes = cider.cider_kv4_attention_shared_workspace_bytes(_batch(**kw), _runs(**runs), 4)
            assert nbytes >= 2 * 4 * 4 * 128 * rows  # a part of both kinds for each head of each row
            assert _call(runs, nbytes=nbytes, q_heads=4, **kw) == YES
            assert _call(runs, nbytes=nbytes - 1, q_heads=4, **kw) == ROOM
    finally:
        cider.cider_kv4_set_tiles(0)
