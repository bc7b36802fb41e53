"""cider_kv4_attention_shared on the GPU against the 64-bit attention of each sequence by itself, within the bound of
the ordinary attention's tests: runs of one and of many sequences, shared lengths around pages, sequences outside any
run, padded slots and rows inside the prefix, lengths and runs that are not sound, parts of very different sizes,
streams, graphs."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests.test_kv4_gpu import GEOMETRY, TILES, Setup, compare, i32, reference

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


def setup_of(lens, rows, H, D, gs, starts, shared, dtype, seed=0, change=None):
    """A batch whose runs' sequences name the same pages for the whole pages of `shared` tokens and hold the same
    tokens there; change(k, v) may spoil the values before they are quantized."""
    s = Setup(lens, rows, H, D, gs, seed=seed, garbage="nan")
    k, v = s.values(dtype)
    if change:
        change(k, v)
    for g, n in enumerate(shared):
        first = starts[g]
        for b in range(first + 1, starts[g + 1]):
            m = min(n // 64 * 64, lens[b], lens[first])
            k[b][:m], v[b][:m] = k[first][:m], v[first][:m]
            s.table[b, :n // 64] = s.table[first, :n // 64]
    ref.fill(s.cache, s.table, s.lens, k, v)
    return s


def runs_of(s, starts, shared, max_rows=None, max_shared=None):
    most = max([sum(s.n[a:b]) for a, b in zip(starts, starts[1:])] + [1]) if max_rows is None else max_rows
    return cider.cider_kv4_runs(i32(starts), i32(shared), len(shared), most,
                                max(list(shared) + [0]) if max_shared is None else max_shared)


def attend(s, batch, runs, q, q_dtype, y_dtype, HQ, scale, workspace=None, stream=None):
    import torch
    ldq, ldy = HQ * s.D + 40, HQ * s.D + 8
    wide = np.full((s.rows, ldq), 0x7E00, np.uint16)   # NaN beside the heads
    wide[:, :HQ * s.D] = q.reshape(s.rows, -1)
    qd = gu.bits_to_dev(wide)
    y = torch.full((s.rows, ldy), 99, dtype=torch.int16, device="cuda")
    need = cider.cider_kv4_attention_shared_workspace_bytes(batch, runs, HQ)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    gu.sync()
    cider.cider_kv4_attention_shared(batch, runs, qd, q_dtype, ldq, HQ, scale, ws, need, y, y_dtype, ldy, stream)
    gu.sync()
    assert workspace is not None or (ws[need:] == 0xFF).all()
    got = gu.bits_to_host(y)
    assert (got[:, HQ * s.D:] == 99).all()
    return got[:, :HQ * s.D].reshape(s.rows, HQ, s.D)


CASES = [
    # lengths, rows, kv heads, query heads, runs' starts, shared tokens
    ([70, 80, 64 + 1], [1, 1, 1], 2, 8, [0, 3], [64]),
    ([200], [1], 1, 7, [0, 1], [190]),                                       # a run of one
    ([300, 0, 290, 257], [1, 1, 1, 1], 2, 4, [0, 4], [256]),                 # a padded slot
    ([150, 140, 129, 131, 500, 66], [4, 3, 2, 4, 5, 1], 1, 6, [1, 4, 5], [128, 320]),  # some in no run
    ([200, 100, 190], [5, 60, 2], 2, 2, [0, 3], [128]),                      # rows inside the prefix
    ([400, 390], [40, 100], 1, 4, [0, 2], [256]),
    ([330, 340, 350, 335], [9, 17, 30, 1], 2, 6, [0, 2, 4], [320, 300]),
    ([100, 90], [1, 2], 1, 3, [0, 2], [63]),                                 # less than a page
    ([1100, 1030, 1090], [1, 1, 1], 4, 16, [0, 3], [1024]),
    ([130, 140, 150], [1, 0, 3], 1, 20, [0, 3], [128]),                      # a sequence without rows
    ([70, 75], [1, 1], 1, 40, [0, 0, 2], [64, 64]),                          # an empty run
]


@pytest.mark.parametrize("D,gs", GEOMETRY)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, D, gs):
    lens, rows, H, HQ, starts, shared = CASES[case]
    dtype = (case + D // 64 + gs // 64) % 2
    s = setup_of(lens, rows, H, D, gs, starts, shared, dtype, seed=case)
    batch = s.to_device()
    q = ref.to_bits(s.rng.standard_normal((s.rows, HQ, D)) * 2, dtype)
    want = reference(s, q, dtype, HQ, 1 / np.sqrt(D))
    for tiles in TILES:
        cider.cider_kv4_set_tiles(tiles)
        compare(s, attend(s, batch, runs_of(s, starts, shared), q, dtype, dtype, HQ, 1 / np.sqrt(D)), want, dtype)


@pytest.mark.parametrize("tiles", TILES)
def test_loose_bounds(tiles):
    """A program that captures a graph passes bounds, not sizes: rows, shared lengths and lengths far below them."""
    cider.cider_kv4_set_tiles(tiles)
    s = setup_of([300, 310, 280, 40], [3, 1, 2, 1], 2, 128, 64, [0, 3], [200], 0, seed=5)
    s.table = np.pad(s.table, ((0, 0), (0, 90)), constant_values=2 ** 31 - 1)
    s.max_pages += 90
    batch = s.to_device(max_rows=6)
    q = ref.to_bits(s.rng.standard_normal((s.rows, 8, 128)), 0)
    want = reference(s, q, 0, 8, 0.1)
    for max_shared in (200, 1000, s.max_pages * 64):
        got = attend(s, batch, runs_of(s, [0, 3], [200], max_rows=7, max_shared=max_shared), q, 0, 0, 8, 0.1)
        compare(s, got, want, 0)
    # shared_len past its bound is the bound; a bound of fewer rows than the run has, nothing is shared
    compare(s, attend(s, batch, runs_of(s, [0, 3], [200], max_shared=130), q, 0, 0, 8, 0.1), want, 0)
    compare(s, attend(s, batch, runs_of(s, [0, 3], [200], max_rows=5, max_shared=200), q, 0, 0, 8, 0.1), want, 0)


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("starts,shared", [
    ([-1, 3], [128]), ([0, 5], [128]), ([2, 1], [128]), ([4, 9], [128]), ([0, 3], [-2 ** 31]), ([0, 3], [0]),
    ([2 ** 31 - 1, -2 ** 31], [128]),
])
def test_runs_that_are_not_sound_share_nothing(starts, shared, tiles):
    cider.cider_kv4_set_tiles(tiles)
    s = setup_of([200, 170, 150, 60], [1, 2, 1, 1], 1, 64, 64, [0, 3], [128], 1, seed=2)
    q = ref.to_bits(s.rng.standard_normal((s.rows, 5, 64)), 1)
    got = attend(s, s.to_device(), runs_of(s, starts, shared, max_rows=5, max_shared=192), q, 1, 1, 5, 0.125)
    compare(s, got, reference(s, q, 1, 5, 0.125), 1)


@pytest.mark.parametrize("tiles", TILES)
def test_a_bound_of_no_tokens(tiles):
    """Lengths bounded to 0: no row is there, whatever the runs say."""
    cider.cider_kv4_set_tiles(tiles)
    s = setup_of([200, 190], [2, 1], 1, 128, 64, [0, 2], [128], 0, seed=9)
    s.to_device()
    q = ref.to_bits(s.rng.standard_normal((s.rows, 4, 128)), 0)
    got = attend(s, s.batch(s.dcache, max_kv_len=0), runs_of(s, [0, 2], [128]), q, 0, 0, 4, 0.1)
    assert not got.any()


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("lens,rows", [
    ([0, 200, 190, 180], [1, 1, 1, 1]), ([0, 0, 190, 180], [1, 0, 2, 1]), ([70, 200, 190, 180], [1, 2, 1, 1]),
    ([200, 190, 180, 0], [1, 1, 1, 1]), ([0, 70, 0, 60], [1, 1, 1, 1]),
])
def test_slots_whose_tables_are_not_the_runs(lens, rows, tiles):
    """A run's slots without its pages: padded ones, one without rows, one in front of the prefix's end, whose tables
    name nothing in the cache or pages of their own."""
    cider.cider_kv4_set_tiles(tiles)
    first = next((b for b in range(4) if lens[b] - rows[b] >= 128), 3)
    s = setup_of(lens, rows, 2, 128, 64, [first, 4], [128], 0, seed=4)
    for b in range(4):
        if lens[b] - rows[b] < 128:
            s.table[b, -(-lens[b] // 64):] = (-1, 2 ** 31 - 1)[b % 2]
    q = ref.to_bits(s.rng.standard_normal((s.rows, 8, 128)), 0)
    got = attend(s, s.to_device(), runs_of(s, [0, 4], [128]), q, 0, 0, 8, 0.1)
    compare(s, got, reference(s, q, 0, 8, 0.1), 0)


def test_rows_that_are_left_out_stay():
    """A sequence with more rows than the bound, inside a run."""
    s = setup_of([200, 190, 210], [2, 9, 1], 1, 128, 64, [0, 3], [128], 0, seed=3)
    q = ref.to_bits(s.rng.standard_normal((s.rows, 4, 128)), 0)
    got = attend(s, s.to_device(max_rows=4), runs_of(s, [0, 3], [128]), q, 0, 0, 4, 0.1)
    want = reference(s, q, 0, 4, 0.1)
    assert (got[2:11] == 99).all()
    for b in (0, 2):
        y, bound = want[b]
        err = np.abs(ref.to_f64(got[s.row_start[b]:s.row_start[b + 1]], 0) - y)
        assert (err <= bound + 2.0 ** -11 * (np.abs(y) + bound) + 2.0 ** -25).all()


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("large", ["prefix", "own"])
@pytest.mark.parametrize("rows", [1, 20])
def test_parts_of_very_different_sizes(rows, large, tiles):
    """Values 2^40 times as large, and scores that leave the other part no weight, in front or behind."""
    cider.cider_kv4_set_tiles(tiles)

    def change(k, v):
        for b in range(2):
            at = slice(0, 192) if large == "prefix" else slice(192, None)
            v[b][at] *= 2.0 ** 40
            k[b][at, :, 64:] *= 2.0 ** 5

    s = setup_of([250, 240], [rows, rows], 1, 128, 64, [0, 2], [192], 1, seed=4, change=change)
    q = ref.to_bits(s.rng.standard_normal((s.rows, 6, 128)) * 3, 1)
    got = attend(s, s.to_device(), runs_of(s, [0, 2], [192]), q, 1, 1, 6, 0.0883)
    compare(s, got, reference(s, q, 1, 6, 0.0883), 1)


@pytest.mark.parametrize("tiles", TILES)
def test_nan_in_a_shared_page_reaches_the_run_and_no_one_else(tiles):
    cider.cider_kv4_set_tiles(tiles)
    s = setup_of([200, 190, 130, 100], [1, 1, 1, 1], 1, 128, 128, [0, 2], [128], 0, seed=6)
    q = ref.to_bits(s.rng.standard_normal((4, 4, 128)), 0)
    want = reference(s, q, 0, 4, 0.1)
    s.cache.data[s.table[0, 1], 0, 64 * 128 + 4 * 5:][:4] = np.array([0x7FC00000], np.uint32).view(np.uint8)
    got = ref.to_f64(attend(s, s.to_device(), runs_of(s, [0, 2], [128]), q, 0, 0, 4, 0.1), 0)
    assert np.isnan(got[:2]).all()
    for b in (2, 3):
        assert (np.abs(got[b] - want[b][0][0]) <= want[b][1][0] + 2.0 ** -10 * np.abs(want[b][0][0]) + 2.0 ** -24).all()


@pytest.mark.parametrize("tiles", TILES)
def test_shared_pages_that_are_not_in_the_cache_are_not_seen(tiles):
    cider.cider_kv4_set_tiles(tiles)
    s = setup_of([300, 290], [2, 1], 1, 64, 64, [0, 2], [256], 0, seed=7)
    whole = s.table.copy()
    s.table[:, 1] = [s.num_pages, -5]
    q = ref.to_bits(s.rng.standard_normal((3, 4, 64)), 0)
    got = attend(s, s.to_device(), runs_of(s, [0, 2], [256]), q, 0, 0, 4, 0.1)
    data = s.cache.data
    s.table = whole  # the reference: scores of minus infinity for that page's tokens
    y = []
    for b, (kv, n) in enumerate(zip(s.lens, s.n)):
        k, v = (s.cache.values(w, list(s.table[b, :-(-kv // 64)]))[0] for w in (0, 1))
        for i in range(n):
            see = np.concatenate([np.arange(64), np.arange(128, kv - n + i + 1)])
            x = 0.1 * np.einsum("hd,td->ht", ref.to_f64(q[s.row_start[b] + i], 0), k[0][see])
            w = np.exp(x - x.max(1, keepdims=True))
            y.append(w / w.sum(1, keepdims=True) @ v[0][see])
    assert np.abs(ref.to_f64(got, 0) - np.array(y)).max() < 4e-3 and data is s.cache.data


def test_types_are_independent_and_another_stream():
    import torch
    s = setup_of([200, 177], [4, 1], 1, 128, 128, [0, 2], [128], 1, seed=8)
    batch = s.to_device()
    for q_dtype, y_dtype in ((0, 1), (1, 0)):
        q = ref.to_bits(s.rng.standard_normal((s.rows, 4, 128)), q_dtype)
        got = attend(s, batch, runs_of(s, [0, 2], [128]), q, q_dtype, y_dtype, 4, 0.11, stream=torch.cuda.Stream())
        compare(s, got, reference(s, q, q_dtype, 4, 0.11), y_dtype)


@pytest.mark.parametrize("tiles", [0, 128])
def test_graphs_that_share_a_workspace(tiles):
    """Two captured calls of other sizes, one workspace, replayed by turns while lengths change, with eager calls between."""
    import torch
    cider.cider_kv4_set_tiles(tiles)
    made = []
    for i, (lens, rows, starts, shared) in enumerate([([300, 310, 330], [1, 1, 1], [0, 3], [256]),
                                                      ([900, 880], [6, 4], [0, 2], [860])]):
        s = setup_of(lens, rows, 2, 128, 64, starts, shared, 0, seed=20 + i)
        s.max_pages = s.table.shape[1]
        batch, runs = s.to_device(), runs_of(s, starts, shared)
        q = ref.to_bits(s.rng.standard_normal((s.rows, 8, 128)), 0)
        made.append((s, batch, runs, q, gu.bits_to_dev(q.reshape(s.rows, -1)),
                     torch.zeros((s.rows, 8 * 128), dtype=torch.int16, device="cuda")))
    need = max(cider.cider_kv4_attention_shared_workspace_bytes(m[1], m[2], 8) for m in made)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    call = lambda m: cider.cider_kv4_attention_shared(m[1], m[2], m[4], 0, 1024, 8, 0.0883, ws, need, m[5], 0, 1024)  # noqa: E731
    graphs = []
    for m in made:
        call(m)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(m)
        graphs.append(g)
    for turn in range(4):
        for m, g in zip(made, graphs):
            s = m[0]
            g.replay()
            got = m[5].clone()
            m[5].zero_()
            call(m)
            assert torch.equal(m[5], got)
            compare(s, gu.bits_to_host(got).reshape(s.rows, 8, 128), reference(s, m[3], 0, 8, 0.0883), 0)
            s.lens[0] -= 7   # the first sequence is cut back, still behind the prefix
            m[1]._tensors[3].copy_(i32(s.lens))
        ws.fill_(turn)
