"""Where the cache calls' envelope ends (host checks; no kernel is launched)."""
import pytest

import w4a8_quantized_linear_amd as cider

P = 0x10000
YES, NO = cider.CIDER_ERR_NO_DEVICE, cider.CIDER_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(autouse=True)
def _no_device(monkeypatch):
    monkeypatch.setenv("CIDER_FORCE_UNAVAILABLE", "1")


def _batch(batch, rows, kv_heads, pages=4, D=64):
    return cider.cider_kv4_batch(P, P, P, P, batch, rows, rows, 64 * pages, pages, 9, kv_heads, D, 64)


@pytest.mark.parametrize("batch,rows,kv_heads,status", [
    (1024, 65536, 8, YES),          # 2^24 workgroups and more
    (1 << 14, 1 << 9, 1 << 12, YES),   # 18 spans of 2^26 heads
    (1 << 14, 1 << 10, 1 << 12, NO),   # 34
    (1 << 14, 32, 1 << 15, YES),
    (1 << 15, 32, 1 << 15, NO),
])
def test_append_and_read(batch, rows, kv_heads, status):
    b = _batch(batch, rows, kv_heads)
    for f in (cider.cider_kv4_append, cider.cider_kv4_read):
        assert f(b, P, P, 0, kv_heads * 64, kv_heads * 64, stream=0, check=False) == status


@pytest.mark.parametrize("batch,rows,kv_heads,q_heads,pages,status", [
    (4096, 1, 64, 64, 2048, YES),
    (16384, 1, 64, 1024, 544, YES),
    (16384, 2046, 64, 64, 4, YES),
    (16384, 2047, 64, 64, 4, YES),
    (16384, 2048, 64, 64, 4, NO),
    (1 << 20, 1, 2048, 2048, 4, NO),
    (1, (1 << 30) // 64, 1, 64, 4, YES),
    (1, (1 << 30) // 64 + 1, 1, 64, 4, NO),
])
def test_attention(batch, rows, kv_heads, q_heads, pages, status):
    b = _batch(batch, rows, kv_heads, pages)
    ld = q_heads * 64
    assert cider.cider_kv4_attention(b, P, 0, ld, q_heads, 0.1, 0, 0, None, 0, P, 0, ld, stream=0, check=False) == status
    parts = cider.cider_kv4_attention_workspace_bytes(b, q_heads, 0, 0)
    assert parts == 0 if status == NO else parts >= 0
