"""The 4-bit key/value cache on the GPU: append and read bit for bit, and the
attention within a derived bound, against the 64-bit implementation of
tests/kv4_reference.py.  Sizes and masks are those where it can go wrong:
lengths 0, 1 and around pages, rows in front of the sequence, windows and
sinks at page edges, rows that see nothing, garbage (NaN, infinity) wherever a
row may not look, head counts that do not fill a tile, scales far apart, page
numbers outside the cache, blocks past 4 GiB."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref

pytestmark = pytest.mark.gpu

GEOMETRY = [(64, 64), (128, 64), (128, 128)]


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


TILES = [0, 16, 128, 256]   # automatic, and each kernel


def i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Setup:
    """A pool of pages of garbage and the page table of a batch, with more room than it needs."""

    def __init__(self, lens, rows, H, D, gs, seed=0, garbage="bytes", spare=2, table_room=1):
        r = np.random.default_rng([seed, D, gs, H])
        self.lens, self.n, self.H, self.D, self.gs, self.rng = list(lens), list(rows), H, D, gs, r
        need = [-(-kv // 64) for kv in lens]
        self.num_pages = sum(need) + spare
        order = r.permutation(self.num_pages).astype(np.int32)
        self.max_pages = max(max(need), 1) + table_room
        self.table = np.full((len(lens), self.max_pages), 2 ** 31 - 1, np.int32)   # never to be followed
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        shape = (self.num_pages, H, ref.block_bytes(D, gs))
        data = r.integers(0, 256, shape, dtype=np.uint8) if garbage == "bytes" else np.full(shape, 0xFF, np.uint8)
        self.cache = ref.Cache(data, D, gs)
        self.row_start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.rows = int(self.row_start[-1])

    def values(self, dtype, std=1.0):
        """Whole sequences' k and v: 16-bit values as float64."""
        out = []
        for i in range(2):
            x = [self.rng.standard_normal((kv, self.H, self.D)) * std for kv in self.lens]
            out.append([ref.to_f64(ref.to_bits(y, dtype), dtype).reshape(y.shape) for y in x])
        return out

    def to_device(self, max_rows=None, max_kv_len=None):
        import torch
        self.dcache = torch.from_numpy(self.cache.data.copy()).cuda()
        return self.batch(self.dcache, max_rows, max_kv_len)

    def batch(self, dcache, max_rows=None, max_kv_len=None):
        return cider.cider_kv4_batch(
            dcache, i32(self.table), i32(self.row_start), i32(self.lens), len(self.lens), self.rows,
            max(self.n) if max_rows is None else max_rows,
            self.max_pages * 64 if max_kv_len is None else max_kv_len, self.max_pages, self.num_pages,
            self.H, self.D, self.gs)


def rows_of(s, x):
    """The call's rows of whole sequences x, rows in front of a sequence as 7s: float64 [rows, H, D]."""
    out = []
    for b, (kv, n) in enumerate(zip(s.lens, s.n)):
        lead = max(0, n - kv)
        out.append(np.full((lead, s.H, s.D), 7.0))
        out.append(x[b][kv - (n - lead):kv])
    return np.concatenate(out) if out else np.zeros((0, s.H, s.D))


CACHE_CASES = [
    # lengths once the rows are in, rows, kv heads
    ([1], [1], 1), ([64], [1], 3), ([65], [2], 2), ([100], [100], 2), ([33, 0, 200, 64], [1, 1, 70, 64], 2),
    ([5, 31, 32, 96], [9, 31, 32, 33], 1), ([127, 130], [63, 66], 3),
]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("D,gs", GEOMETRY)
@pytest.mark.parametrize("lens,rows,H", CACHE_CASES)
def test_append_and_read_bit_exact(lens, rows, H, D, gs, dtype):
    import torch
    s = Setup(lens, rows, H, D, gs, seed=len(lens))
    k, v = s.values(dtype)
    k[0][-1, 0] = 0                       # a group of zeros
    v[-1][-1:, -1, :gs] = [[0.0, 1.75, -1.75, 0.125] * (gs // 4)]   # ties at scale 0.25
    batch = s.to_device()
    kr, vr = rows_of(s, k), rows_of(s, v)
    # a fused product's rows: queries in front, keys and values behind one another, a stride with room
    ldq = 2 * H * D + 24
    fused = np.zeros((s.rows, ldq), np.uint16)
    fused[:, 8:8 + H * D] = ref.to_bits(kr, dtype).reshape(s.rows, -1)
    fused[:, 8 + H * D:8 + 2 * H * D] = ref.to_bits(vr, dtype).reshape(s.rows, -1)
    d = gu.bits_to_dev(fused)
    cider.cider_kv4_append(batch, d[:, 8:], d[:, 8 + H * D:], dtype, ldq, ldq)
    want = s.cache
    for b, (kv, n) in enumerate(zip(s.lens, s.n)):
        for t in range(max(0, kv - n), kv):
            for which, x in ((0, k), (1, v)):
                want.put(s.table[b, t // 64], t % 64, which, *ref.quantize(x[b][t], gs))
    assert np.array_equal(gu.to_host(s.dcache), want.data)   # every other byte as it was
    ko = torch.full((s.rows, ldq), 99, dtype=torch.int16, device="cuda")
    vo = torch.full((s.rows, H * D), 99, dtype=torch.int16, device="cuda")
    cider.cider_kv4_read(batch, ko[:, 16:], vo, dtype, ldq, H * D)
    got_k, got_v = gu.bits_to_host(ko), gu.bits_to_host(vo)
    assert (got_k[:, :16] == 99).all() and (got_k[:, 16 + H * D:] == 99).all()
    for which, x, got in ((0, k, got_k[:, 16:16 + H * D]), (1, v, got_v)):
        u = [ref.quantize(y, gs) for y in x]
        back = [np.float32(np.repeat(sc, gs, -1)) * (uu.astype(np.float32) - 8) for uu, sc in u]
        rows_want = rows_of(s, back)
        for b, (kv, n) in enumerate(zip(s.lens, s.n)):
            rows_want[s.row_start[b]:s.row_start[b] + max(0, n - kv)] = 0
        assert np.array_equal(got, ref.to_bits(rows_want, dtype).reshape(s.rows, -1))


def test_append_step_by_step_equals_append_at_once():
    D, gs, H, dtype = 128, 64, 2, 0
    at_once = Setup([150], [150], H, D, gs)
    k, v = at_once.values(dtype)
    dk, dv = (gu.bits_to_dev(ref.to_bits(x[0], dtype).reshape(150, -1)) for x in (k, v))
    cider.cider_kv4_append(at_once.to_device(), dk, dv, dtype, H * D, H * D)
    want = gu.to_host(at_once.dcache)
    steps = Setup([150], [150], H, D, gs)
    steps.to_device()
    t = 0
    for n in (1, 1, 5, 30, 27, 1, 64, 21):
        t += n
        one = cider.cider_kv4_batch(steps.dcache, i32(steps.table), i32([0, n]), i32([t]), 1, n, n,
                                    steps.max_pages * 64, steps.max_pages, steps.num_pages, H, D, gs)
        cider.cider_kv4_append(one, dk[t - n:t], dv[t - n:t], dtype, H * D, H * D)
    assert t == 150
    assert np.array_equal(gu.to_host(steps.dcache), want)
    # a token that is appended again (a draft that was not taken) is overwritten
    again = cider.cider_kv4_batch(steps.dcache, i32(steps.table), i32([0, 3]), i32([70]), 1, 3, 3,
                                  steps.max_pages * 64, steps.max_pages, steps.num_pages, H, D, gs)
    cider.cider_kv4_append(again, dk[:3], dv[:3], dtype, H * D, H * D)
    cider.cider_kv4_append(again, dk[67:70], dv[67:70], dtype, H * D, H * D)
    assert np.array_equal(gu.to_host(steps.dcache), want)


@pytest.mark.parametrize("dtype", [0, 1])
def test_scales_of_every_magnitude(dtype):
    """Each finite 16-bit magnitude once as a group's largest value, the group's other values spread below it."""
    r = np.random.default_rng(dtype)
    top = np.arange(0, 0x7F80 if dtype else 0x7C00, dtype=np.uint16)
    D, n = 64, len(top)
    x = ref.to_f64(top, dtype)[:, None] * np.concatenate([[1.0], r.uniform(-1, 1, D - 1)])
    x = ref.to_f64(ref.to_bits(x, dtype), dtype).reshape(n, 1, D)
    s = Setup([n], [n], 1, D, 64, garbage="nan")
    batch = s.to_device()
    rows = gu.bits_to_dev(ref.to_bits(x, dtype).reshape(n, D))
    cider.cider_kv4_append(batch, rows, rows, dtype, D, D)
    u, sc = ref.quantize(x, 64)
    c = ref.Cache(gu.to_host(s.dcache), D, 64)
    pages = list(s.table[0, :-(-n // 64)])
    with np.errstate(over="ignore"):
        want = sc.astype(np.float64) * (u.astype(np.float64) - 8)
    for which in (0, 1):
        v, _ = c.values(which, pages)
        assert np.array_equal(v[0, :n], want.reshape(n, D))


def attend(s, batch, q, q_dtype, y_dtype, HQ, scale, window=0, sinks=0, workspace=True, stream=None):
    """q uint16 patterns [rows, HQ, D]; returns uint16 patterns, rows as they were where nothing is written."""
    import torch
    ldq, ldy = HQ * s.D + 40, HQ * s.D + 8
    wide = np.full((s.rows, ldq), 0x7E00, np.uint16)   # NaN beside the heads
    wide[:, :HQ * s.D] = q.reshape(s.rows, -1)
    qd = gu.bits_to_dev(wide)
    y = torch.full((s.rows, ldy), 99, dtype=torch.int16, device="cuda")
    nbytes = cider.cider_kv4_attention_workspace_bytes(batch, HQ, window, sinks) if workspace else 0
    ws = torch.full((max(nbytes, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    cider.cider_kv4_attention(batch, qd, q_dtype, ldq, HQ, scale, window, sinks, ws if nbytes else None, nbytes,
                              y, y_dtype, ldy, stream)
    got = gu.bits_to_host(y)
    assert (got[:, HQ * s.D:] == 99).all()
    return got[:, :HQ * s.D].reshape(s.rows, HQ, s.D)


def reference(s, q, q_dtype, HQ, scale, window=0, sinks=0):
    """(outputs, bound) of every sequence."""
    q = ref.to_f64(q, q_dtype)
    return [ref.attention(s.cache, s.table[b], kv, q[s.row_start[b]:s.row_start[b] + n], HQ // s.H, scale, window, sinks)
            for b, (kv, n) in enumerate(zip(s.lens, s.n))]


def compare(s, got, want, y_dtype):
    got = ref.to_f64(got, y_dtype)
    step = 2.0 ** -8 if y_dtype == 1 else 2.0 ** -11
    for b, (y, bound) in enumerate(want):
        assert np.isfinite(y).all()
        err = np.abs(got[s.row_start[b]:s.row_start[b] + s.n[b]] - y)
        ok = err <= bound + step * (np.abs(y) + bound) + 2.0 ** -25   # fp16's smallest step
        assert ok.all(), "sequence %d: %d outside, worst %.3g of %.3g" % (
            b, int((~ok).sum()), err[~ok].max(), np.abs(y).max())


def check(s, got, q, q_dtype, y_dtype, HQ, scale, window=0, sinks=0):
    compare(s, got, reference(s, q, q_dtype, HQ, scale, window, sinks), y_dtype)


ATTEND_CASES = [
    # lengths, rows, kv heads, query heads, window, sinks
    ([1], [1], 1, 1, 0, 0),
    ([63, 64, 65], [1, 1, 1], 2, 8, 0, 0),
    ([700], [1], 1, 7, 0, 0),
    ([300, 0, 1, 129], [1, 1, 1, 1], 2, 6, 0, 0),
    ([130, 90, 4], [5, 3, 9], 2, 14, 0, 0),            # the last one's first rows are not there
    ([257], [40], 1, 4, 0, 0),
    ([200], [200], 1, 3, 0, 0),
    ([70], [33], 1, 40, 0, 0),                         # more heads than a tile has columns
    ([500, 64, 3], [1, 1, 1], 2, 2, 1, 0),             # sees itself alone
    ([500, 64, 3], [2, 2, 2], 2, 2, 1, 4),
    ([500, 321], [3, 1], 1, 5, 64, 0),
    ([500, 321], [3, 1], 1, 5, 63, 1),
    ([400, 130], [70, 130], 1, 2, 65, 70),             # sinks past the first page
    ([400], [100], 2, 4, 10, 300),                     # more sinks than a row has tokens
    ([1000], [1], 4, 16, 200, 4),
    ([4096], [1], 1, 8, 0, 0),
]


@pytest.mark.parametrize("D,gs", GEOMETRY)
@pytest.mark.parametrize("lens,rows,H,HQ,window,sinks", ATTEND_CASES)
def test_attention(lens, rows, H, HQ, window, sinks, D, gs):
    """Each kernel, with and without a workspace, against the reference worked out once."""
    dtype = (len(lens) + HQ + D // 64 + gs // 64) % 2
    s = Setup(lens, rows, H, D, gs, seed=HQ, garbage="nan")
    ref.fill(s.cache, s.table, s.lens, *s.values(dtype))
    batch = s.to_device()
    q = ref.to_bits(s.rng.standard_normal((s.rows, HQ, D)) * 2, dtype)
    scale = 1 / np.sqrt(D)
    want = reference(s, q, dtype, HQ, scale, window, sinks)
    for tiles in TILES:
        cider.cider_kv4_set_tiles(tiles)
        for workspace in (True, False):
            compare(s, attend(s, batch, q, dtype, dtype, HQ, scale, window, sinks, workspace), want, dtype)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("q_dtype,y_dtype", [(0, 1), (1, 0)])
def test_attention_types_are_independent(q_dtype, y_dtype, tiles):
    cider.cider_kv4_set_tiles(tiles)
    s = Setup([200, 77], [4, 1], 1, 128, 128, garbage="nan")
    ref.fill(s.cache, s.table, s.lens, *s.values(1))
    q = ref.to_bits(s.rng.standard_normal((s.rows, 4, 128)), q_dtype)
    check(s, attend(s, s.to_device(), q, q_dtype, y_dtype, 4, 0.11), q, q_dtype, y_dtype, 4, 0.11)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("rows", [1, 50])
def test_attention_scores_and_scales_far_apart(rows, tiles):
    """A sharp softmax, values whose scales lie 2^20 apart, the large ones far back, tiny and huge bf16 queries."""
    cider.cider_kv4_set_tiles(tiles)
    s = Setup([400, 150], [rows, 1], 1, 128, 64, garbage="nan")
    k, v = s.values(1)
    for b in range(2):
        v[b][:, :, :64] *= 2.0 ** -18
        v[b][10:13, :, :64] *= 2.0 ** 20
        v[b][100:, :, 64:] *= 2.0 ** 60
        k[b][5] = 0
        v[b][7] = 0
    ref.fill(s.cache, s.table, s.lens, k, v)
    x = s.rng.standard_normal((s.rows, 4, 128)) * 6
    x[-1] *= 2.0 ** -120
    x[0, 1] = 0
    x[0, 2] *= 2.0 ** 10   # every weight but one underflows
    q = ref.to_bits(x, 1)
    check(s, attend(s, s.to_device(), q, 1, 1, 4, 0.0883), q, 1, 1, 4, 0.0883)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("rows", [1, 50])
def test_attention_scores_that_vanish(rows, tiles):
    """Queries and a scale so small that their product with every key is 0 in 32 bits: the mean of what is seen."""
    cider.cider_kv4_set_tiles(tiles)
    s = Setup([400, 150], [rows, 1], 1, 64, 64, garbage="nan")
    ref.fill(s.cache, s.table, s.lens, *s.values(1))
    q = ref.to_bits(s.rng.standard_normal((s.rows, 4, 64)) * 2.0 ** -125, 1)
    check(s, attend(s, s.to_device(), q, 1, 1, 4, 1e-30, 90, 2), q, 1, 1, 4, 1e-30, 90, 2)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("rows", [2, 40])
def test_what_a_row_may_not_see_does_not_reach_it(rows, tiles):
    """NaN and infinite keys and values behind the window and in front of the row, inside pages it does read."""
    cider.cider_kv4_set_tiles(tiles)
    s = Setup([300], [rows], 2, 128, 64, garbage="nan")
    k, v = s.values(0)
    ref.fill(s.cache, s.table, s.lens, k, v)
    clean = s.cache.data.copy()
    for t, bad in ((20, 0x7F800000), (230, 0x7FC00000), (299, 0x7F800000), (190, 0xFFFFFFFF)):
        for at in (64 * 128, 64 * 128 + 512):   # K's and V's scales
            block = s.cache.data[s.table[0, t // 64]]
            for g in range(2):
                block[:, at + 4 * (g * 64 + t % 64):][:, :4] = np.array([bad], np.uint32).view(np.uint8)
    q = ref.to_bits(s.rng.standard_normal((s.rows, 4, 128)), 0)
    batch = s.to_device()
    window, sinks = 50, 6
    got = ref.to_f64(attend(s, batch, q, 0, 0, 4, 0.1, window, sinks), 0)
    s.cache.data = clean
    for i in range(rows):
        see = ref.visible(300 - rows + i, 300, window, sinks)
        hit = any(see[t] for t in (20, 190, 230, 299))
        if hit:
            assert np.isnan(got[i]).all(), i
        else:
            want, bound = ref.attention(s.cache, s.table[0], 300 - rows + i + 1,
                                        ref.to_f64(q[i:i + 1], 0), 2, 0.1, window, sinks)
            assert (np.abs(got[i] - want[0]) <= bound[0] + 2.0 ** -11 * (np.abs(want[0]) + bound[0]) + 2.0 ** -25).all(), i


@pytest.mark.parametrize("tiles", TILES)
def test_a_query_with_nan_spoils_its_own_head_only(tiles):
    cider.cider_kv4_set_tiles(tiles)
    s = Setup([90], [3], 1, 64, 64, garbage="nan")
    ref.fill(s.cache, s.table, s.lens, *s.values(0))
    x = s.rng.standard_normal((3, 5, 64))
    q = ref.to_bits(x, 0)
    bad = q.copy()
    bad[1, 2, 9] = 0x7E00
    good = attend(s, s.to_device(), q, 0, 0, 5, 0.125)
    got = attend(s, s.to_device(), bad, 0, 0, 5, 0.125)
    assert np.isnan(ref.to_f64(got[1, 2], 0)).all()
    got[1, 2] = good[1, 2]
    assert np.array_equal(got, good)


@pytest.mark.parametrize("tiles", TILES)
def test_bounds_of_the_device_arrays(tiles):
    """Lengths, rows and pages outside the batch's bounds are clipped, left out or not followed."""
    cider.cider_kv4_set_tiles(tiles)
    import torch
    D, gs, H, HQ = 128, 64, 1, 2
    s = Setup([130, 100, 64], [2, 2, 2], H, D, gs, garbage="nan", table_room=0)
    ref.fill(s.cache, s.table, s.lens, *s.values(0))
    q = ref.to_bits(s.rng.standard_normal((6, HQ, D)), 0)
    good = attend(s, s.to_device(), q, 0, 0, HQ, 0.1)
    base = s.to_device()

    def call(kv_len=None, row_start=None, table=None, max_rows=2, max_kv_len=192):
        b = cider.cider_kv4_batch(s.dcache, i32(s.table if table is None else table),
                                  i32(s.row_start if row_start is None else row_start),
                                  i32(s.lens if kv_len is None else kv_len), 3, 6, max_rows, max_kv_len,
                                  s.max_pages, s.num_pages, H, D, gs)
        return b, attend(s, b, q, 0, 0, HQ, 0.1)

    _, got = call(kv_len=[2 ** 31 - 1, 100, -5], max_kv_len=130)   # clipped to 130, as it was; and to 0
    assert np.array_equal(got[:4], good[:4]) and (got[4:] == 0).all()
    _, got = call(row_start=[0, 2, 4, 7])                          # the last one's rows run over the end
    assert np.array_equal(got[:4], good[:4]) and (got[4:] == 99).all()
    _, got = call(row_start=[0, 2, -3, 6])
    assert np.array_equal(got[:2], good[:2]) and (got[2:] == 99).all()
    _, got = call(max_rows=1)
    assert (got == 99).all()
    table = s.table.copy()
    table[1, 0] = -1
    b, got = call(table=table)
    assert np.array_equal(got[[0, 1, 4, 5]], good[[0, 1, 4, 5]])
    # sequence 1 without its first 64 tokens: as a window over the others sees it
    t = Setup([100], [2], H, D, gs, table_room=0)
    t.cache, t.table, t.num_pages, t.n = s.cache, s.table[1:2], s.num_pages, [2]
    want = [ref.attention(t.cache, t.table[0], 99 + i, ref.to_f64(q[2 + i:3 + i], 0), HQ, 0.1, 35 + i, 0)
            for i in range(2)]
    for i in range(2):
        y, bound = want[i]
        assert (np.abs(ref.to_f64(got[2 + i], 0) - y[0]) <= bound[0] + 2.0 ** -11 * (np.abs(y[0]) + bound[0]) + 2.0 ** -25).all()
    before = gu.to_host(s.dcache).copy()
    rows = torch.ones((6, H * D), dtype=torch.float16, device="cuda")
    table[:] = 2 ** 30
    b = cider.cider_kv4_batch(s.dcache, i32(table), i32(s.row_start), i32(s.lens), 3, 6, 2, 192, s.max_pages,
                              s.num_pages, H, D, gs)
    cider.cider_kv4_append(b, rows, rows, 0, H * D, H * D)
    assert np.array_equal(gu.to_host(s.dcache), before)
    cider.cider_kv4_read(b, rows, rows, 0, H * D, H * D)
    assert not rows.any().item()
    assert (attend(s, b, q, 0, 0, HQ, 0.1) == 0).all()
    assert base is not None


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("rows", [1, 40])
def test_a_page_that_is_not_there_leaves_no_trace(rows, tiles):
    """Whatever the cache's first page holds (the largest scales here), a page number outside the cache only
    hides its tokens."""
    cider.cider_kv4_set_tiles(tiles)
    s = Setup([300], [rows], 1, 128, 64, garbage="nan")
    ref.fill(s.cache, s.table, s.lens, *s.values(1))
    if s.table[0, 1] == 0 or 0 in s.table[0, 2:5]:   # page 0 is to be one that no token is in
        free = next(n for n in range(s.num_pages) if n not in s.table[0, :5])
        s.cache.data[[0, free]] = s.cache.data[[free, 0]]
        s.table[0][s.table[0] == 0] = free
    s.table[0, 1] = -7
    s.cache.data[0, :, 64 * 128:] = np.tile(np.array([2.0 ** 100], np.float32).view(np.uint8), 256)
    q = ref.to_bits(s.rng.standard_normal((rows, 4, 128)), 1)
    got = ref.to_f64(attend(s, s.to_device(), q, 1, 0, 4, 0.1), 0)
    # the same with the hidden tokens' keys far below all others
    t = ref.Cache(s.cache.data.copy(), 128, 64)
    pages = list(s.table[0, :5])
    k, v = (t.values(i, [n if n >= 0 else pages[0] for n in pages]) for i in (0, 1))
    for i in range(rows):
        see = [u for u in range(300 - rows + i + 1) if u // 64 != 1]
        for h in range(4):
            x = 0.1 * (k[0][0][see] @ ref.to_f64(q[i, h], 1))
            w = np.exp(x - x.max())
            w /= w.sum()
            want, size = w @ v[0][0][see], w @ (np.abs(v[0][0][see]) + 16 * v[1][0][see])
            assert (np.abs(got[i, h] - want) <= 2.0 ** -9 * size + 2.0 ** -11 * np.abs(want)).all(), (i, h)


def test_blocks_past_4_gib():
    import torch
    D, gs, H = 128, 64, 8
    s = Setup([200], [70], H, D, gs, garbage="nan", spare=0)
    k, v = s.values(0)
    ref.fill(s.cache, s.table, s.lens, k, v)
    q = ref.to_bits(s.rng.standard_normal((70, 16, D)), 0)
    want = attend(s, s.to_device(), q, 0, 0, 16, 0.1)
    per_page = H * ref.block_bytes(D, gs)
    far = (1 << 32) // per_page + 5
    big = torch.empty((far + s.num_pages, H, ref.block_bytes(D, gs)), dtype=torch.uint8, device="cuda")
    big[:5] = 0x55
    big[far:].fill_(0xFF)
    s.table[0, :4] += far
    s.num_pages += far
    b = s.batch(big)
    kd, vd = (gu.bits_to_dev(ref.to_bits(x[0], 0).reshape(200, -1)) for x in (k, v))
    whole = cider.cider_kv4_batch(big, i32(s.table), i32([0, 200]), i32([200]), 1, 200, 200, 256, s.max_pages,
                                  s.num_pages, H, D, gs)
    cider.cider_kv4_append(whole, kd, vd, 0, H * D, H * D)
    assert np.array_equal(attend(s, b, q, 0, 0, 16, 0.1), want)
    back = torch.empty((2, 200, H * D), dtype=torch.int16, device="cuda")
    cider.cider_kv4_read(whole, back[0], back[1], 0, H * D, H * D)
    u, sc = ref.quantize(v[0], gs)
    expect = np.repeat(sc, gs, -1) * (u.astype(np.float32) - 8)
    assert np.array_equal(gu.bits_to_host(back[1]), ref.to_bits(expect, 0).reshape(200, -1))
    assert (big[:5] == 0x55).all().item()


@pytest.mark.parametrize("tiles", TILES)
def test_same_bits_every_time_on_another_stream_and_from_a_graph(tiles):
    cider.cider_kv4_set_tiles(tiles)
    import torch
    D, gs, H, HQ = 128, 64, 2, 8
    s = Setup([2000, 900, 0], [1, 1, 1], H, D, gs, garbage="nan")
    ref.fill(s.cache, s.table, s.lens, *s.values(0))
    batch = s.to_device()
    q = ref.to_bits(s.rng.standard_normal((3, HQ, D)), 0)
    want = attend(s, batch, q, 0, 0, HQ, 0.1)
    assert np.array_equal(attend(s, batch, q, 0, 0, HQ, 0.1), want)
    side = torch.cuda.Stream()
    qd = gu.bits_to_dev(q.reshape(3, -1))
    y = torch.zeros((3, HQ * D), dtype=torch.int16, device="cuda")
    k = torch.randn((3, H * D), device="cuda").half()
    nbytes = cider.cider_kv4_attention_workspace_bytes(batch, HQ, 0, 0)
    ws = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    cider.cider_kv4_attention(batch, qd, 0, HQ * D, HQ, 0.1, 0, 0, ws, nbytes, y, 0, HQ * D, stream=side)
    side.synchronize()
    assert np.array_equal(gu.bits_to_host(y).reshape(3, HQ, D), want)
    # a decoding step: append, then attend; lengths move between replays
    lens = i32(s.lens)
    step = cider.cider_kv4_batch(s.dcache, i32(s.table), i32(s.row_start), lens, 3, 3, 1, s.max_pages * 64,
                                 s.max_pages, s.num_pages, H, D, gs)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cider.cider_kv4_append(step, k, k, 0, H * D, H * D)
        cider.cider_kv4_attention(step, qd, 0, HQ * D, HQ, 0.1, 0, 0, ws, nbytes, y, 0, HQ * D)
    for lengths in ([2000, 900, 0], [1999, 897, 0], [1, 64, 0], [2000, 899, 0]):
        lens.copy_(i32(lengths))
        k.normal_()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = gu.bits_to_host(y).copy()
        eager = torch.zeros_like(y)
        cider.cider_kv4_append(step, k, k, 0, H * D, H * D)
        cider.cider_kv4_attention(step, qd, 0, HQ * D, HQ, 0.1, 0, 0, ws, nbytes, eager, 0, HQ * D)
        assert np.array_equal(got, gu.bits_to_host(eager))
        s.cache.data = gu.to_host(s.dcache)
        s.lens = lengths
        check(s, got.reshape(3, HQ, D), q, 0, 0, HQ, 0.1)
