"""The 4-bit key/value cache where its calls meet their limits: the joins of
split caches (every one of them, with pairs of none, one and all parts, and
with NaN in a part), workspaces smaller than asked for, finite values of any
size where a row may not look, values at the ends of bf16's range, scores of any
size, rows of one tile that are far apart, and launches past 2^24 workgroups."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests.test_kv4_gpu import GEOMETRY, TILES, Setup, attend, compare, i32, reference

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


# ---------------------------------------------------------------- joins

# (tiles, sequences, rows of each, kv heads, query heads, bound on the lengths, parts, pairs): the parts and pairs
# choose the join: up to 4 parts, up to 16 with 2048 pairs and more, any number
JOINS = {
    "few columns, 4 parts": (0, 64, 1, 2, 4, 8192, 4, 256),
    "few columns, 10 parts": (0, 64, 1, 2, 32, 20480, 10, 2048),
    "few columns, 8 parts of few pairs": (0, 4, 1, 2, 4, 2048, 8, 16),
    "few columns, 32 parts": (0, 1, 1, 2, 4, 8192, 32, 4),
    "128 columns, up to 4 parts": (128, 1, 64, 1, 2, 1024, (2, 4), 128),
    "128 columns, up to 16 parts": (128, 1, 64, 8, 32, 4096, (5, 16), 2048),
    "128 columns, many parts": (128, 1, 64, 1, 2, 8192, (5, 128), 128),
    "256 columns, 4 parts": (256, 1, 64, 1, 4, 4096, 4, 256),
    "256 columns, 8 parts": (256, 1, 128, 4, 16, 8192, 8, 2048),
    "256 columns, 8 parts of few pairs": (256, 1, 64, 1, 4, 8192, 8, 256),
}


def join_batch(name, D, gs, lens, seed=0):
    """The setup and batch of a join's case; how many parts and pages a part the call takes.  The workspace holds
    4 D + 8 bytes for every row, query head and part, each kind rounded up to 256."""
    tiles, batch, rows, H, HQ, bound, parts, pairs = JOINS[name]
    cider.cider_kv4_set_tiles(tiles)
    lens = (list(lens) + [5] * batch)[:batch]
    s = Setup(lens, [rows] * batch, H, D, gs, seed=seed, garbage="nan")
    pages = bound // 64
    table = np.full((batch, pages), 2 ** 31 - 1, np.int32)
    width = min(pages, s.table.shape[1])
    table[:, :width] = s.table[:, :width]
    s.table, s.max_pages = table, pages
    want = parts if isinstance(parts, tuple) else (parts, parts)

    def batch_of():
        b = s.to_device(max_kv_len=bound)
        n = cider.cider_kv4_attention_workspace_bytes(b, HQ, 0, 0)
        got = n // (s.rows * HQ * (4 * D + 8))
        assert rows * HQ * batch == pairs and want[0] <= got <= want[1], (got, want)
        return b, -(-pages // got)

    return s, batch_of, HQ


@pytest.mark.parametrize("D,gs", [(64, 64), (128, 64)])
@pytest.mark.parametrize("name", JOINS)
def test_joins(name, D, gs):
    """Sequences that end in their first, a middle and the last part, one token into a part, and without tokens."""
    bound, rows = JOINS[name][5], JOINS[name][2]
    lens = [bound] if rows > 1 else [bound // 2 + 1, bound, 0, 1, 64, bound // 4, bound // 4 + 1, bound - 70]
    s, batch_of, HQ = join_batch(name, D, gs, lens)
    dtype = D // 64 % 2
    ref.fill(s.cache, s.table, s.lens, *s.values(dtype))
    b, _ = batch_of()
    x = s.rng.standard_normal((s.rows, HQ, D))
    q = ref.to_bits(x, dtype)
    scale = 1 / np.sqrt(D)
    got = attend(s, b, q, dtype, dtype, HQ, scale)
    if rows == 1:
        compare(s, got, reference(s, q, dtype, HQ, scale), dtype)
        return
    qf = ref.to_f64(q, dtype)
    step = 2.0 ** -8 if dtype == 1 else 2.0 ** -11
    for i in (0, 1, 31, 62, rows - 1):   # (the reference would take minutes for every row)
        y, bound_y = ref.attention(s.cache, s.table[0], s.lens[0] - rows + i + 1, qf[i:i + 1], HQ // s.H, scale, 0, 0)
        err = np.abs(ref.to_f64(got[i:i + 1], dtype) - y)
        assert (err <= bound_y + step * (np.abs(y) + bound_y) + 2.0 ** -25).all(), (i, err.max())


def spoil(s, t, which, bits, heads=slice(None)):
    """Every scale of K (0) or V (1) of token t of sequence 0 becomes the fp32 number of that pattern."""
    D, gs = s.D, s.gs
    block = s.cache.data[s.table[0, t // 64]]
    for g in range(D // gs):
        at = 64 * D + which * 256 * (D // gs) + 4 * (g * 64 + t % 64)
        block[heads, at:at + 4] = np.array([bits], np.uint32).view(np.uint8)


@pytest.mark.parametrize("which", ["K", "V", "V, weight vanishes"])
@pytest.mark.parametrize("name", JOINS)
def test_nan_in_a_part_of_its_own_reaches_the_row(name, which):
    """The newest token alone in its part: NaN keys there leave the part without a maximum, and NaN values count
    even where the part's factor is 0."""
    D, gs = 128, 64
    rows = JOINS[name][2]
    s, batch_of, HQ = join_batch(name, D, gs, [3])   # for the size of a part
    _, pages = batch_of()
    kv = (2 if JOINS[name][5] >= 3 * 64 * pages else 1) * pages * 64 + 1
    s, batch_of, HQ = join_batch(name, D, gs, [kv])
    k, v = s.values(0)
    x = s.rng.standard_normal((s.rows, HQ, D))
    if which == "V, weight vanishes":
        x = np.abs(x) + 0.5
        k[0][0] = 40.0    # the first token takes all the weight
        k[0][-1] = -40.0
    ref.fill(s.cache, s.table, s.lens, k, v)
    q = ref.to_bits(x, 0)
    clean = attend(s, batch_of()[0], q, 0, 0, HQ, 0.1)
    spoil(s, kv - 1, 0 if which == "K" else 1, 0x7FC00000, heads=slice(0, 1))
    got = attend(s, batch_of()[0], q, 0, 0, HQ, 0.1)
    G, last = HQ // s.H, rows - 1
    assert np.isnan(ref.to_f64(got[last, :G], 0)).all()
    got[last, :G] = clean[last, :G]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("name", JOINS)
def test_workspace_smaller_than_asked_for(name):
    """Fewer, longer parts; nothing behind the bytes that were given is written."""
    import torch
    D, gs = 128, 128
    bound, rows = JOINS[name][5], JOINS[name][2]
    s, batch_of, HQ = join_batch(name, D, gs, [min(bound, 3000), 700])
    ref.fill(s.cache, s.table, s.lens, *s.values(1))
    b, _ = batch_of()
    q = ref.to_bits(s.rng.standard_normal((s.rows, HQ, D)), 1)
    few = sorted({0, min(1, s.rows - 1), s.rows - 1})
    qf = ref.to_f64(q, 1)
    want = []
    for i in few:
        at = i if rows == 1 else 0
        kv = s.lens[0] - rows + i + 1 if rows > 1 else s.lens[at]
        want.append(ref.attention(s.cache, s.table[at], kv, qf[i:i + 1], HQ // s.H, 0.09, 0, 0))
    full = cider.cider_kv4_attention_workspace_bytes(b, HQ, 0, 0)
    qd = gu.bits_to_dev(q.reshape(s.rows, -1))
    guard = 1 << 16
    for nbytes in (full, full - 1, full // 2, full // 2 - 256, full // 4, full // 8, 300, 1):
        ws = torch.full((full + guard,), 0xA5, dtype=torch.uint8, device="cuda")
        y = torch.full((s.rows, HQ * D), 99, dtype=torch.int16, device="cuda")
        cider.cider_kv4_attention(b, qd, 1, HQ * D, HQ, 0.09, 0, 0, ws, nbytes, y, 1, HQ * D)
        assert (ws[nbytes:] == 0xA5).all().item(), nbytes
        got = ref.to_f64(gu.bits_to_host(y).reshape(s.rows, HQ, D), 1)
        for i, (w, bound_y) in zip(few, want):
            assert (np.abs(got[i] - w[0]) <= bound_y[0] + 2.0 ** -8 * (np.abs(w[0]) + bound_y[0])).all(), (nbytes, i)


# ---------------------------------------------------------------- what a row may not see

def bits_of(x):
    return int(np.array([x], np.float32).view(np.uint32)[0])


HUGE = [2.0 ** 24, 2.0 ** 40, 2.0 ** 100, 2.0 ** 120, float(np.finfo(np.float32).max)]


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("huge", HUGE)
@pytest.mark.parametrize("rows,window,sinks", [(1, 50, 6), (2, 0, 0), (2, 50, 6), (5, 3, 0), (40, 0, 0), (40, 50, 6),
                                               (100, 64, 70)])
def test_finite_scales_that_a_row_may_not_see_change_nothing(rows, window, sinks, huge, tiles):
    """Scales of any size behind the window, after the sinks and in front of a row, in pages that it does read:
    the row's bits are those of a cache without them."""
    cider.cider_kv4_set_tiles(tiles)
    for dtype, (D, gs) in zip((0, 1, 1), GEOMETRY):
        s = Setup([300], [rows], 2, D, gs, garbage="nan")
        ref.fill(s.cache, s.table, s.lens, *s.values(dtype))
        q = ref.to_bits(s.rng.standard_normal((s.rows, 6, D)), dtype)
        clean = attend(s, s.to_device(), q, dtype, dtype, 6, 0.1, window, sinks)
        plain = s.cache.data.copy()
        for base in {0, rows - 1}:   # everything that the first row, or the last, may not see
            hidden = ~ref.visible(300 - rows + base, 300, window, sinks)
            bad = [t for t in (20, 200, 230, 262, 288, 299) if hidden[t]]
            s.cache.data = plain.copy()
            for t in bad:
                for which in (0, 1):
                    spoil(s, t, which, bits_of(huge))
            got = attend(s, s.to_device(), q, dtype, dtype, 6, 0.1, window, sinks)
            for i in range(rows):
                if not ref.visible(300 - rows + i, 300, window, sinks)[bad].any():
                    assert np.array_equal(got[i], clean[i]), (base, i)


@pytest.mark.parametrize("tiles", TILES)
def test_a_later_token_far_larger(tiles):
    """Two rows, the second token's values 2^40 times the first's: the first row is the first token's values."""
    import torch
    cider.cider_kv4_set_tiles(tiles)
    for D, gs in GEOMETRY:
        s = Setup([2], [2], 1, D, gs, garbage="nan")
        k, v = s.values(1)
        v[0][1] *= 2.0 ** 40
        b = s.to_device()
        kd, vd = (gu.bits_to_dev(ref.to_bits(x[0], 1).reshape(2, -1)) for x in (k, v))
        cider.cider_kv4_append(b, kd, vd, 1, D, D)
        back = torch.empty((2, 2, D), dtype=torch.int16, device="cuda")
        cider.cider_kv4_read(b, back[0], back[1], 1, D, D)
        q = ref.to_bits(s.rng.standard_normal((2, 1, D)), 1)
        got = attend(s, b, q, 1, 1, 1, 0.1)
        assert np.array_equal(got[0, 0], gu.bits_to_host(back[1])[0])


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("window,sinks,power", [(0, 0, 0.7), (5, 0, -0.7), (5, 0, 0.7), (9, 2, -0.5), (0, 0, -0.7)])
def test_every_row_has_values_of_its_own_size(window, sinks, power, tiles):
    """Values that grow or shrink by a power of two every token or two, whole prompts: no row may lose bits to what
    another row of its tile sees.  (A head's halves apart too.)"""
    cider.cider_kv4_set_tiles(tiles)
    for D, gs in GEOMETRY:
        s = Setup([100, 61], [100, 7], 1, D, gs, garbage="nan")
        k, v = s.values(1)
        for x in v:
            x *= 2.0 ** np.floor(power * np.arange(len(x)))[:, None, None]
            x[:, :, :D // 2] *= 2.0 ** np.floor(5 * np.sin(np.arange(len(x))))[:, None, None]
        ref.fill(s.cache, s.table, s.lens, k, v)
        q = ref.to_bits(s.rng.standard_normal((s.rows, 3, D)), 1)
        want = reference(s, q, 1, 3, 0.1, window, sinks)
        got = ref.to_f64(attend(s, s.to_device(), q, 1, 1, 3, 0.1, window, sinks), 1)
        for b, (y, bound) in enumerate(want):
            err = np.abs(got[s.row_start[b]:s.row_start[b] + s.n[b]] - y)
            assert (err <= bound + 2.0 ** -8 * (np.abs(y) + bound)).all(), (D, gs, b)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (40, 4), (100, 0), (100, 70)])
def test_one_larger_token_moves_only_the_rows_that_see_it(window, sinks, tiles):
    """A prompt whose rows see one page by halves or no page together, one token's values 2 to 2^30 times the others':
    rows that see it are within the bound, the others keep their bits."""
    cider.cider_kv4_set_tiles(tiles)
    for dtype, (D, gs) in zip((0, 1, 1), GEOMETRY):
        for token, by in ((0, 4), (0, 2 ** 30), (3, 8), (64, 16), (130, 2), (130, 32), (199, 64), (150, 2 ** 30)):
            by = min(by, 2 ** 12) if dtype == 0 else by
            s = Setup([200], [200], 1, D, gs, garbage="nan")
            k, v = s.values(dtype)
            ref.fill(s.cache, s.table, s.lens, k, v)
            q = ref.to_bits(s.rng.standard_normal((s.rows, 3, D)), dtype)
            clean = attend(s, s.to_device(), q, dtype, dtype, 3, 0.1, window, sinks)
            v[0][token] *= by
            ref.fill(s.cache, s.table, s.lens, k, v)
            got = attend(s, s.to_device(), q, dtype, dtype, 3, 0.1, window, sinks)
            compare(s, got, reference(s, q, dtype, 3, 0.1, window, sinks), dtype)
            for i in range(200):
                if not ref.visible(i, 200, window, sinks)[token]:
                    assert np.array_equal(got[i], clean[i]), (D, gs, token, by, i)


# ---------------------------------------------------------------- the ends of the range

@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("kv,rows,HQ", [(1, 1, 1), (70, 1, 4), (70, 70, 4), (4097, 1, 4), (4100, 8, 40)])
def test_values_at_the_end_of_bf16(kv, rows, HQ, tiles):
    """Values of 1.75 2^126, all alike, beside elements of 0: the outputs are those values and 0 within the
    reference's bound, though a sum of the tokens' would not be finite."""
    cider.cider_kv4_set_tiles(tiles)
    for D, gs in GEOMETRY:
        s = Setup([kv], [rows], 1, D, gs, garbage="nan")
        k, v = s.values(1)
        v[0][:] = 0
        v[0][:, :, ::3] = 1.75 * 2.0 ** 126
        v[0][:, :, ::6] *= -1
        ref.fill(s.cache, s.table, s.lens, k, v)
        q = ref.to_bits(s.rng.standard_normal((s.rows, HQ, D)), 1)
        got = attend(s, s.to_device(), q, 1, 1, HQ, 0.1)
        assert np.isfinite(ref.to_f64(got, 1)).all()
        compare(s, got, reference(s, q, 1, HQ, 0.1), 1)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("rows", [1, 40])
def test_values_at_the_other_end_of_bf16(rows, tiles):
    """Values around 2^-118: their scales are as exact as any, and so are the outputs."""
    cider.cider_kv4_set_tiles(tiles)
    for D, gs in GEOMETRY:
        s = Setup([200], [rows], 1, D, gs, garbage="nan")
        k, v = s.values(1)
        v[0] *= 2.0 ** -118
        ref.fill(s.cache, s.table, s.lens, k, v)
        q = ref.to_bits(s.rng.standard_normal((s.rows, 2, D)), 1)
        (y, bound), = reference(s, q, 1, 2, 0.1)
        err = np.abs(ref.to_f64(attend(s, s.to_device(), q, 1, 1, 2, 0.1), 1) - y)
        # 2^-134: half of bf16's smallest step
        assert (err <= bound + 2.0 ** -8 * (np.abs(y) + bound) + 2.0 ** -134).all()


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("power", [12, 24, 40, 70])
def test_scores_of_any_size(power, rows, tiles):
    """Scores of 2^power and more: where the largest stands out by 2^-12 of itself it takes all the weight."""
    cider.cider_kv4_set_tiles(tiles)
    for D, gs in GEOMETRY:
        s = Setup([200], [rows], 1, D, gs, garbage="nan")
        k, v = s.values(1)
        ref.fill(s.cache, s.table, s.lens, k, v)
        pages = list(s.table[0, :4])
        q = ref.to_bits(s.rng.standard_normal((s.rows, 5, D)) * 2.0 ** power, 1)
        (kk, _), (vv, _) = s.cache.values(0, pages), s.cache.values(1, pages)
        got = ref.to_f64(attend(s, s.to_device(), q, 1, 1, 5, 0.5), 1)
        assert np.isfinite(got).all()
        tried = 0
        for i in range(rows):
            for h in range(5):
                x = 0.5 * (kk[0][:201 - rows + i] @ ref.to_f64(q[i, h], 1))
                top = x.argmax()
                second = np.delete(x, top).max()
                if x[top] - second >= max(2.0 ** -12 * x[top], 40):
                    tried += 1
                    assert (np.abs(got[i, h] - vv[0][top]) <= 2.0 ** -8 * np.abs(vv[0][top]) + 2.0 ** -11).all()
        assert tried >= rows


@pytest.mark.parametrize("tiles", TILES)
def test_rows_of_a_tile_do_not_share_their_queries_size(tiles):
    """Rows that are not there hold anything, 2^100 here; one row that is there holds 2^40; the others are as exact
    as alone."""
    cider.cider_kv4_set_tiles(tiles)
    for D, gs in GEOMETRY:
        s = Setup([30, 120], [40, 30], 2, D, gs, garbage="nan")
        ref.fill(s.cache, s.table, s.lens, *s.values(1))
        x = s.rng.standard_normal((s.rows, 4, D))
        x[:10] *= 2.0 ** 100
        x[50, 1] *= 2.0 ** 40
        x[60:63] *= 2.0 ** -40
        q = ref.to_bits(x, 1)
        want = reference(s, q, 1, 4, 0.1)
        want[1][1][10, 1] = np.inf   # scores of 2^40 are known to 2^22: no bound for that one
        compare(s, attend(s, s.to_device(), q, 1, 1, 4, 0.1), want, 1)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("first", [50, 56, 57, 58, 60, 100])
@pytest.mark.parametrize("up", [1, 2, 3, 4, 5])
def test_values_and_scores_that_grow_from_page_to_page(up, first, tiles):
    """Scales of 2^first, then 2^up times those with scores a little higher, which a running maximum may lag
    behind."""
    cider.cider_kv4_set_tiles(tiles)
    for D, gs in GEOMETRY:
        s = Setup([4 * 64], [50], 1, D, gs, garbage="nan")
        k, v = s.values(1)
        v[0][:] = np.sign(v[0]) * 7 * 2.0 ** first
        v[0][64:] *= 2.0 ** up
        k[0][:64] = 0
        k[0][64:] = 1.94 / (0.1 * D)   # 2.8 in units of log2
        ref.fill(s.cache, s.table, s.lens, k, v)
        q = ref.to_bits(np.ones((s.rows, 3, D)), 1)
        compare(s, attend(s, s.to_device(), q, 1, 1, 3, 0.1), reference(s, q, 1, 3, 0.1), 1)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("rows", [1, 40])
def test_queries_at_the_end_of_bf16(rows, tiles):
    """Queries around 2^122 with keys around 2^-121, next to ordinary ones."""
    cider.cider_kv4_set_tiles(tiles)
    for D, gs in GEOMETRY:
        s = Setup([150, 90], [rows, 1], 1, D, gs, garbage="nan")
        k, v = s.values(1)
        k[0] *= 2.0 ** -121
        ref.fill(s.cache, s.table, s.lens, k, v)
        x = s.rng.standard_normal((s.rows, 2, D))
        x[:rows] *= 2.0 ** 122
        q = ref.to_bits(x, 1)
        compare(s, attend(s, s.to_device(), q, 1, 1, 2, 0.3), reference(s, q, 1, 2, 0.3), 1)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("power", [35, 55])
def test_keys_whose_halves_are_far_apart(power, rows, tiles):
    """K's groups 2^(2 power) apart, queries in either half alone, so that the scores matter."""
    cider.cider_kv4_set_tiles(tiles)
    for big in (0, 1):
        s = Setup([130], [rows], 1, 128, 64, garbage="nan")
        k, v = s.values(1)
        halves = [slice(0, 64), slice(64, 128)]
        k[0][:, :, halves[big]] *= 2.0 ** power
        k[0][:, :, halves[1 - big]] *= 2.0 ** -power
        ref.fill(s.cache, s.table, s.lens, k, v)
        x = s.rng.standard_normal((s.rows, 4, 128))
        x[:, :2, halves[big]] = 0
        x[:, :2, halves[1 - big]] *= 2.0 ** power
        x[:, 2:, halves[1 - big]] = 0
        x[:, 2:, halves[big]] *= 2.0 ** -power
        q = ref.to_bits(x, 1)
        compare(s, attend(s, s.to_device(), q, 1, 1, 4, 0.1), reference(s, q, 1, 4, 0.1), 1)


# ---------------------------------------------------------------- launches past 2^24 workgroups

def test_append_and_read_with_wide_bounds():
    """1024 sequences of up to 65536 rows and 8 heads: 16.8 million workgroups, nearly all without work."""
    import torch
    D, gs, H, batch, bound = 64, 64, 8, 1024, 65536
    s = Setup([70, 3], [2, 3], H, D, gs, garbage="nan")
    k, v = s.values(0)
    starts = np.full(batch + 1, 5, np.int32)
    starts[0] = 0
    starts[1:batch] = 2
    lens = np.zeros(batch, np.int32)
    lens[0], lens[-1] = 70, 3
    table = np.zeros((batch, bound // 64), np.int32)
    table[0, :2], table[-1, :1] = s.table[0, :2], s.table[1, :1]
    d = torch.from_numpy(s.cache.data.copy()).cuda()
    b = cider.cider_kv4_batch(d, i32(table), i32(starts), i32(lens), batch, bound, bound, bound, bound // 64,
                              s.num_pages, H, D, gs)
    kr, vr = (np.concatenate([x[0][68:], x[1]]) for x in (k, v))
    kd, vd = (gu.bits_to_dev(ref.to_bits(x, 0).reshape(5, -1)) for x in (kr, vr))
    cider.cider_kv4_append(b, kd, vd, 0, H * D, H * D)
    for seq, kv, n in ((0, 70, 2), (1, 3, 3)):
        for t in range(kv - n, kv):
            for which, x in ((0, k), (1, v)):
                s.cache.put(s.table[seq, t // 64], t % 64, which, *ref.quantize(x[seq][t], gs))
    assert np.array_equal(gu.to_host(d), s.cache.data)
    out = torch.zeros((2, 5, H * D), dtype=torch.int16, device="cuda")
    cider.cider_kv4_read(b, out[0], out[1], 0, H * D, H * D)
    for x, got in ((kr, out[0]), (vr, out[1])):
        u, sc = ref.quantize(x, gs)
        want = np.repeat(sc, gs, -1) * (u.astype(np.float32) - 8)
        assert np.array_equal(gu.bits_to_host(got), ref.to_bits(want, 0).reshape(5, -1))


@pytest.mark.parametrize("tiles,batch,kv_heads,q_heads,pages,rows", [
    (16, 4096, 64, 64, 2048, 1),      # a split launch of 2^24 workgroups
    (16, 16384, 64, 1024, 544, 1),    # and its join
    (128, 16384, 64, 64, 4, 2046),    # tiles of many columns, whole
])
def test_attention_with_wide_bounds(tiles, batch, kv_heads, q_heads, pages, rows):
    import torch
    cider.cider_kv4_set_tiles(tiles)
    D, gs = 64, 64
    n = min(rows, 3)
    s = Setup([200, 67], [n, 1], kv_heads, D, gs, garbage="nan")
    ref.fill(s.cache, s.table, s.lens, *s.values(0))
    s.to_device()
    starts = np.full(batch + 1, n + 1, np.int32)
    starts[0] = 0
    starts[1:batch] = n
    lens = np.zeros(batch, np.int32)
    lens[0], lens[-1] = s.lens
    table = torch.zeros((batch, pages), dtype=torch.int32, device="cuda")
    table[0, :4], table[-1, :2] = i32(s.table[0, :4]), i32(s.table[1, :2])
    rows = max(rows, n + 1)
    b = cider.cider_kv4_batch(s.dcache, table, i32(starts), i32(lens), batch, rows, rows if n > 1 else 1, pages * 64,
                              pages, s.num_pages, kv_heads, D, gs)
    q = ref.to_bits(s.rng.standard_normal((n + 1, q_heads, D)), 0)
    qd = gu.bits_to_dev(q.reshape(n + 1, -1))
    y = torch.zeros((n + 1, q_heads * D), dtype=torch.int16, device="cuda")
    nbytes = cider.cider_kv4_attention_workspace_bytes(b, q_heads, 0, 0)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    cider.cider_kv4_attention(b, qd, 0, q_heads * D, q_heads, 0.1, 0, 0, ws, nbytes, y, 0, q_heads * D)
    compare(s, gu.bits_to_host(y).reshape(n + 1, q_heads, D), reference(s, q, 0, q_heads, 0.1), 0)
