"""Argument checks of cider_kv4_append_rotated on the host (no kernel is launched: the library is told that there is no
device), and the reference that the GPU tests compare with, pinned by what a rotation is."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import rotate_reference as rr

P, BAD, ODD = 0x10000, 0x10008, 0x10002
INVALID, SHAPE, MISALIGNED = (cider.CIDER_ERR_INVALID_ARG, cider.CIDER_ERR_UNSUPPORTED_SHAPE,
                              cider.CIDER_ERR_MISALIGNED)
YES = cider.CIDER_ERR_NO_DEVICE


@pytest.fixture(autouse=True)
def _no_device(monkeypatch):
    monkeypatch.setenv("CIDER_FORCE_UNAVAILABLE", "1")


def _call(turn=None, q=P, k=P, v=P, dtype=0, ldq=1024, ldk=256, ldv=256, q_heads=8, q_out=P, ldo=1024, **kw):
    b = dict(cache=P, pages=P, row_start=P, kv_len=P, batch=3, rows=5, max_rows=3, max_kv_len=256, max_pages=4,
             num_pages=9, kv_heads=2, head_dim=128, group_size=64)
    b.update(kw)
    t = dict(cos_sin=P, table_len=10, rot_dim=128)
    t.update(turn or {})
    return cider.cider_kv4_append_rotated(cider.cider_kv4_batch(*b.values()), cider.cider_rotation(**t), q, k, v, dtype,
                                          ldq, ldk, ldv, q_heads, q_out, ldo, stream=0, check=False)


AXES = dict(axes=3, positions=P, pair_axis=[0, 1, 2, 1] * 16)


@pytest.mark.parametrize("turn,status", [
    ({}, YES), (dict(rot_dim=96), YES), (dict(rot_dim=16, interleaved=True), YES),
    (dict(rot_dim=0, cos_sin=None, table_len=0, axes=0), YES),
    (dict(positions=P), YES), (AXES, YES), ({**AXES, "axes": 4}, YES),
    (dict(q_weight=P, k_weight=P), YES), (dict(q_weight=P), YES), (dict(k_weight=P, eps=1e-30), YES),
    (dict(eps=-1.0), YES),  # without weights it is not looked at
    (dict(rot_dim=-16), INVALID), (dict(rot_dim=8), SHAPE), (dict(rot_dim=120), SHAPE), (dict(rot_dim=144), SHAPE),
    (dict(cos_sin=None), INVALID), (dict(table_len=0), INVALID), (dict(table_len=-1), INVALID),
    (dict(table_len=(1 << 30) + 1), SHAPE), (dict(axes=0), INVALID),
    ({**AXES, "axes": 5}, SHAPE), ({**AXES, "axes": 2}, INVALID), ({**AXES, "positions": None}, INVALID),
    ({**AXES, "pair_axis": None}, INVALID),
    (dict(q_weight=P, eps=0.0), INVALID), (dict(k_weight=P, eps=float("nan")), INVALID),
    (dict(k_weight=P, eps=float("inf")), INVALID), (dict(k_weight=P, eps=-1e-6), INVALID),
    (dict(cos_sin=BAD), MISALIGNED), (dict(positions=ODD), MISALIGNED), (dict(q_weight=BAD), MISALIGNED),
    (dict(k_weight=BAD), MISALIGNED),
])
def test_rotation_checks(turn, status):
    assert _call(turn) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), YES), (dict(q_out=P + 4096, ldo=2048), YES), (dict(q_heads=0, q=None, q_out=None, ldq=0, ldo=0), YES), (dict(q_heads=2, ldq=256, ldo=256), YES),
    (dict(q_heads=-2), INVALID), (dict(q_heads=7), SHAPE), (dict(q_heads=1 << 17, ldq=1 << 24, ldo=1 << 24), SHAPE),
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(dtype=2), INVALID), (dict(ldq=1016), INVALID), (dict(ldo=1016), INVALID), (dict(ldo=2048), INVALID), (dict(ldk=248), INVALID),
    (dict(ldv=248), INVALID), (dict(ldq=1028), MISALIGNED), (dict(ldo=1028), MISALIGNED), (dict(ldk=260), MISALIGNED),
    (dict(q=BAD), MISALIGNED), (dict(q_out=BAD), MISALIGNED), (dict(k=BAD), MISALIGNED), (dict(v=BAD), MISALIGNED),
    (dict(cache=None), INVALID), (dict(cache=BAD), MISALIGNED), (dict(head_dim=96), SHAPE), (dict(group_size=32), INVALID),
    (dict(batch=-1), INVALID), (dict(max_kv_len=257), INVALID),
    (dict(batch=0, cache=None, q=None, k=None), cider.CIDER_OK), (dict(rows=0, q=None), cider.CIDER_OK),
    (dict(max_rows=0, v=None), cider.CIDER_OK),
    (dict(head_dim=64, ldq=512, ldo=512, ldk=128, ldv=128, turn=dict(rot_dim=128)), SHAPE),
])
def test_call_checks(kw, status):
    assert _call(**kw) == status


def test_null_structs():
    r = cider.cider_rotation(P, 10, 128)
    assert cider.cider_kv4_append_rotated(None, r, P, P, P, 0, 1024, 256, 256, 8, P, 1024, stream=0, check=False) == INVALID
    b = cider.cider_kv4_batch(P, P, P, P, 3, 5, 3, 256, 4, 9, 2, 128, 64)
    assert cider.cider_kv4_append_rotated(b, None, P, P, P, 0, 1024, 256, 256, 8, P, 1024, stream=0, check=False) == INVALID


def test_pair_axis_has_an_entry_for_each_pair():
    with pytest.raises(ValueError):
        cider.cider_rotation(P, 10, 128, positions=P, axes=2, pair_axis=[0, 1])


def _table(length, pairs):
    angle = np.arange(length)[:, None] * 10000.0 ** (-np.arange(pairs) / pairs)
    return np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 48, 64])
def test_reference_turns_by_differences_of_positions(rot, interleaved):
    """Lengths stay, and the product of a turned q and k depends on how far apart they stand."""
    r = np.random.default_rng(rot)
    q, k = r.standard_normal((2, 1, 64))
    turn = rr.Rotation(_table(60, rot // 2), interleaved)
    at = [turn.apply(q, None, 0, p)[0] @ turn.apply(k, None, 0, p - 7)[0].T for p in (7, 20, 59)]
    assert np.allclose(at, at[0], atol=1e-5)
    assert np.allclose(np.linalg.norm(turn.apply(q, None, 0, 33)[0]), np.linalg.norm(q), rtol=1e-6)
    assert np.array_equal(turn.apply(q, None, 0, 33)[0][:, rot:], q[:, rot:])
    assert np.array_equal(turn.apply(q, None, 0, 0)[0], q)


def test_reference_by_hand():
    table = np.zeros((3, 8, 2), np.float32)
    table[..., 0] = 1
    table[2, 0] = 0, 1                       # a quarter turn of pair 0 at position 2
    x = np.zeros((1, 64))
    x[0, [0, 1, 8, 20]] = 3, 5, 4, 2
    for interleaved, other in ((False, 8), (True, 1)):
        y, _ = rr.Rotation(table, interleaved).apply(x, None, 0, 2)
        assert y[0, 0] == -x[0, other] and y[0, other] == 3 and y[0, 20] == 2
    y, _ = rr.Rotation(table, positions=[[0]], interleaved=True).apply(x, None, 0, 2)
    assert np.array_equal(y, x)
    axis = np.ones(8, int)
    axis[0] = 0
    y, _ = rr.Rotation(table, True, [[2], [1]], axis).apply(x, None, 0, 0)
    assert y[0, 0] == -5 and y[0, 1] == 3
    y, _ = rr.Rotation(table, True, [[9], [1]], axis).apply(x, None, 0, 0)  # past the table: its end
    assert y[0, 0] == -5
    w = np.full(64, 2, np.float32)
    y, _ = rr.Rotation(q_weight=w, eps=10.0).apply(x, w, 0, 0)
    assert np.allclose(y, 2 * x / np.sqrt((9 + 25 + 16 + 4) / 64 + 10))
