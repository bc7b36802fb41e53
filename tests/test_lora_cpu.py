"""Argument checks of cider_lora_add on the host (no kernel is launched: the library is told that there is no device),
and its workspace."""
import pytest

import w4a8_quantized_linear_amd as cider

P, BAD, ODD = 0x10000, 0x10008, 0x10002
INVALID, SHAPE, MISALIGNED = (cider.CIDER_ERR_INVALID_ARG, cider.CIDER_ERR_UNSUPPORTED_SHAPE,
                              cider.CIDER_ERR_MISALIGNED)
YES, ROOM, OK = cider.CIDER_ERR_NO_DEVICE, cider.CIDER_ERR_WORKSPACE, cider.CIDER_OK


@pytest.fixture(autouse=True)
def _no_device(monkeypatch):
    monkeypatch.setenv("CIDER_FORCE_UNAVAILABLE", "1")


def _lora(a=P, b=P, scale=P, slots=4, rank=16, in_features=256, slice_end=(128, 192)):
    return cider.cider_lora(a, b, scale, slots, rank, in_features, slice_end)


def _call(seg_start=P, slot=P, segments=3, rows=20, max_rows=9, x=P, dtype=0, ldx=256, y_in=P, ldy_in=192, ws=P,
          nbytes=1 << 20, y=P, ldy=192, **kw):
    return cider.cider_lora_add(_lora(**kw), seg_start, slot, segments, rows, max_rows, x, dtype, ldx, y_in, ldy_in, ws,
                                nbytes, y, ldy, stream=0, check=False)


@pytest.mark.parametrize("kw,status", [
    ({}, YES), (dict(scale=None), YES), (dict(rank=8), YES), (dict(rank=128), YES), (dict(slice_end=[64]), YES),
    (dict(slice_end=range(64, 513, 64), ldy=512, ldy_in=512), YES), (dict(dtype=1), YES),
    (dict(y=P + 4096, ldy=200), YES), (dict(max_rows=1 << 30), YES),
    (dict(slots=0), INVALID), (dict(rank=0), INVALID), (dict(in_features=0), INVALID), (dict(slice_end=[]), INVALID),
    (dict(slice_end=[128, 128]), INVALID), (dict(slice_end=[128, 64]), INVALID), (dict(slice_end=[0, 64]), INVALID),
    (dict(segments=-1), INVALID), (dict(rows=-1), INVALID), (dict(max_rows=-1), INVALID),
    (dict(slots=1 << 31), SHAPE), (dict(rank=12), SHAPE), (dict(rank=136), SHAPE), (dict(in_features=96), SHAPE),
    (dict(in_features=1 << 24, ldx=1 << 24), SHAPE), (dict(slice_end=[96, 192]), SHAPE),
    (dict(slice_end=[1 << 24], ldy=1 << 24, ldy_in=1 << 24), SHAPE), (dict(slice_end=range(64, 600, 64)), SHAPE),
    (dict(rows=(1 << 30) + 1), SHAPE), (dict(max_rows=(1 << 30) + 1), SHAPE), (dict(segments=1 << 31), SHAPE),
    (dict(segments=1 << 26), SHAPE),
    (dict(dtype=2), INVALID), (dict(ldx=248), INVALID), (dict(ldy=184), INVALID), (dict(ldy_in=184), INVALID),
    (dict(ldy=200), INVALID),  # in place with another stride
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(seg_start=None), INVALID), (dict(slot=None), INVALID),
    (dict(x=None), INVALID), (dict(y_in=None), INVALID), (dict(y=None), INVALID),
    (dict(a=BAD), MISALIGNED), (dict(b=BAD), MISALIGNED), (dict(scale=ODD), MISALIGNED), (dict(x=BAD), MISALIGNED),
    (dict(seg_start=ODD), MISALIGNED), (dict(slot=ODD), MISALIGNED), (dict(y_in=BAD), MISALIGNED),
    (dict(y=BAD), MISALIGNED), (dict(ws=BAD), MISALIGNED), (dict(ldx=260), MISALIGNED), (dict(ldy=196), MISALIGNED),
    (dict(ldy_in=196), MISALIGNED),
    (dict(ws=None), ROOM), (dict(nbytes=20 * 32 * 4 - 1), ROOM), (dict(nbytes=20 * 32 * 4), YES),
    (dict(segments=0, a=None, x=None, ws=None), OK), (dict(rows=0, y=None), OK), (dict(max_rows=0, seg_start=None), OK),
])
def test_checks(kw, status):
    assert _call(**kw) == status


def test_null_struct():
    assert cider.cider_lora_add(None, P, P, 3, 20, 9, P, 0, 256, P, 192, P, 1 << 20, P, 192, stream=0,
                                check=False) == INVALID
    assert cider.cider_lora_workspace_bytes(None, 3, 20, 9) == 0


@pytest.mark.parametrize("segments,rows,max_rows,inputs", [(1, 1, 1, 4096), (64, 64, 1, 4096), (6, 7000, 2048, 4096),
                                                           (1, 1, 1, 64), (3, 20, 9, 256)])
def test_workspace(segments, rows, max_rows, inputs):
    """A whole number of copies of the rows' products with A, up to 16."""
    need = cider.cider_lora_workspace_bytes(_lora(in_features=inputs), segments, rows, max_rows)
    one = rows * 2 * 16 * 4
    assert need % one == 0 and one <= need <= 16 * one
    assert cider.cider_lora_workspace_bytes(_lora(in_features=inputs), segments, 0, max_rows) == 0
    assert cider.cider_lora_workspace_bytes(_lora(rank=4), segments, rows, max_rows) == 0
