"""Calls around the 4-bit cache that have no rows: nothing is done and no device pointer looked at (a tensor without
elements has none), while sizes, scalars and host arrays are checked all the same."""
import pytest

import w4a8_quantized_linear_amd as cider

OK, INVALID, SHAPE = cider.CIDER_OK, cider.CIDER_ERR_INVALID_ARG, cider.CIDER_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(autouse=True)
def _no_device(monkeypatch):
    monkeypatch.setenv("CIDER_FORCE_UNAVAILABLE", "1")


EMPTY = [dict(batch=0), dict(rows=0), dict(max_rows=0)]
AXES = dict(axes=2, pair_axis=[0, 1] * 32)


def _batch(**kw):
    b = dict(cache=None, pages=None, row_start=None, kv_len=None, batch=3, rows=5, max_rows=3, max_kv_len=256,
             max_pages=4, num_pages=9, kv_heads=2, head_dim=128, group_size=64)
    b.update(kw)
    return cider.cider_kv4_batch(*b.values())


def _rotated(turn, **kw):
    t = dict(cos_sin=None, table_len=10, rot_dim=128)
    t.update(turn)
    return cider.cider_kv4_append_rotated(_batch(**kw), cider.cider_rotation(**t), None, None, None, 0, 1024, 256, 256, 8,
                                          None, 1024, stream=0, check=False)


@pytest.mark.parametrize("empty", EMPTY)
@pytest.mark.parametrize("turn,status", [
    ({}, OK), (AXES, OK), (dict(positions=0x10002), OK), (dict(cos_sin=0x10004), OK), (dict(q_weight=0x10008), OK),
    (dict(table_len=0), INVALID), (dict(axes=0), INVALID), (dict(axes=5), SHAPE), (dict(rot_dim=8), SHAPE),
    ({**AXES, "pair_axis": None}, INVALID), ({**AXES, "pair_axis": [0, 2] * 32}, INVALID),
    (dict(q_weight=0x10000, eps=0.0), INVALID),
])
def test_rotation(turn, status, empty):
    assert _rotated(turn, **empty) == status


@pytest.mark.parametrize("empty", EMPTY)
def test_the_others(empty):
    b = _batch(**empty)
    for f in (cider.cider_kv4_append, cider.cider_kv4_read):
        assert f(b, None, None, 0, 256, 256, stream=0, check=False) == OK
    runs = cider.cider_kv4_runs(None, None, 1, 5, 128)
    assert cider.cider_kv4_attention_shared(b, runs, None, 0, 1024, 8, 0.1, None, 0, None, 0, 1024, stream=0,
                                            check=False) == OK
    assert cider.cider_kv4_attention(b, None, 0, 1024, 8, 0.1, 0, 0, None, 0, None, 0, 1024, stream=0, check=False) == OK
