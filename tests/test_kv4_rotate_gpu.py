"""cider_kv4_append_rotated on the GPU against 64 bits: the cache bit for bit, q within its rounding.  Lengths and rows
in front of a sequence as in the append's tests; every pair layout, part of a head, axes; far positions; norms of tiny
and huge rows; pages that are not there; in place; streams and graphs."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests import rotate_reference as rr
from tests.test_kv4_gpu import CACHE_CASES, GEOMETRY, Setup, i32, rows_of

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


def table_of(length, rot, base=10000.0):
    pairs = rot // 2
    angle = np.arange(length)[:, None] * base ** (-np.arange(pairs) / pairs)
    return np.stack([np.cos(angle), np.sin(angle)], -1).astype(np.float32)


def on_device(t, rows):
    import torch
    f = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    pos = None if t.positions is None else i32(t.positions)
    return cider.cider_rotation(f(t.table), 0 if t.table is None else len(t.table), t.rot, t.interleaved, pos,
                                1 if t.positions is None else len(t.positions), t.pair_axis, f(t.q_weight),
                                f(t.k_weight), t.eps)


def run(s, t, q, k, v, dtype, G, in_place=False, max_rows=None, stream=None):
    """q, k, v float64 [rows, heads, D] of 16-bit values, side by side in rows with room; returns q_out's patterns."""
    import torch
    HQ, W = s.H * G * s.D, s.H * s.D
    ld = HQ + 2 * W + 24
    wide = np.full((s.rows, ld), 0x7E00, np.uint16)
    for at, x in ((8, q), (8 + HQ, k), (8 + HQ + W, v)):
        wide[:, at:at + x[0].size] = ref.to_bits(x, dtype).reshape(s.rows, -1)
    d = gu.bits_to_dev(wide)
    ldo = ld if in_place else HQ + 8
    out = d[:, 8:] if in_place else torch.full((s.rows, ldo), 99, dtype=torch.int16, device="cuda")
    batch = s.batch(s.dcache, max_rows)
    gu.sync()  # the inputs are made on the current stream
    cider.cider_kv4_append_rotated(batch, on_device(t, s.rows), d[:, 8:], d[:, 8 + HQ:], d[:, 8 + HQ + W:], dtype, ld, ld,
                                   ld, s.H * G, out, ldo, stream)
    gu.sync()
    got = gu.bits_to_host(d if in_place else out)
    if in_place:
        wide[:, 8:8 + HQ] = got[:, 8:8 + HQ]
        assert np.array_equal(got, wide)   # k, v and what lies beside them as they were
        return got[:, 8:8 + HQ].reshape(s.rows, -1, s.D)
    assert (got[:, HQ:] == 99).all()
    return got[:, :HQ].reshape(s.rows, -1, s.D)


def check(s, t, q, k, v, dtype, got, skip=()):
    """`skip`: rows of sequences that the call leaves out."""
    want = ref.Cache(s.cache.data.copy(), s.D, s.gs)
    lens = [0 if b in skip else kv for b, kv in enumerate(s.lens)]
    rr.put_keys(want, s.table, lens, s.n, k, v, t, s.gs)
    assert np.array_equal(gu.to_host(s.dcache), want.data)
    row = 0
    for b, (kv, n) in enumerate(zip(s.lens, s.n)):
        for i in range(n):
            if b in skip:
                assert (got[row] == 99).all()
            elif kv - n + i < 0:
                assert not got[row].any()
            else:
                y, bound = t.apply(q[row], t.q_weight, row, kv - n + i)
                e = np.abs(ref.to_f64(got[row], dtype) - y)
                assert (e <= bound + rr.half_step(dtype, np.abs(y) + bound)).all(), (b, i, e.max())
            row += 1


def heads(s, G, dtype, std=1.0):
    """The rows' q, k, v: float64 of 16-bit values."""
    return [ref.to_f64(ref.to_bits(s.rng.standard_normal((s.rows, h, s.D)) * std, dtype), dtype)
            for h in (s.H * G, s.H, s.H)]


TURNS = [
    # rot (of 64ths of the head), interleaved, axes, norm
    (64, False, 1, True), (64, True, 1, False), (48, False, 3, True), (16, True, 2, True), (32, False, 1, False),
    (48, True, 4, False), (0, False, 1, True), (16, False, 1, False),
]


def rotation_of(s, turn, seed=0, length=211):
    rot, interleaved, axes, norm = turn
    rot = rot * s.D // 64 // 16 * 16
    r = np.random.default_rng([seed, rot, axes])
    w = [r.uniform(0.2, 2.0, s.D).astype(np.float32) * r.choice([-1, 1], s.D).astype(np.float32) for _ in range(2)] \
        if norm else (None, None)
    return rr.Rotation(table_of(length, rot) if rot else None, interleaved,
                       r.integers(-3, length + 3, (axes, s.rows)) if axes > 1 else None,
                       r.integers(0, axes, rot // 2) if axes > 1 else None, *w)


@pytest.mark.parametrize("D,gs", GEOMETRY)
@pytest.mark.parametrize("turn", TURNS)
@pytest.mark.parametrize("case", range(len(CACHE_CASES)))
def test_against_64_bits(case, turn, D, gs):
    lens, rows, H = CACHE_CASES[case]
    G, dtype = [1, 4, 3, 2, 7, 5, 8][case], (case + TURNS.index(turn)) % 2
    s = Setup(lens, rows, H, D, gs, seed=case)
    s.to_device()
    q, k, v = heads(s, G, dtype)
    k[0, 0] = 0                            # a head of zeros
    t = rotation_of(s, turn, case)
    check(s, t, q, k, v, dtype, run(s, t, q, k, v, dtype, G, in_place=case % 2 == 1))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("D,gs", GEOMETRY)
def test_without_turning_it_is_the_append(D, gs, dtype):
    """A table of (1, 0) and no weights: the same bits in the cache as cider_kv4_append, and q as it was."""
    s = Setup([70, 130, 3], [70, 5, 4], 2, D, gs, seed=3)
    batch = s.to_device()
    q, k, v = heads(s, 3, dtype, 3.0)
    dk, dv = (gu.bits_to_dev(ref.to_bits(x, dtype).reshape(s.rows, -1)) for x in (k, v))
    cider.cider_kv4_append(batch, dk, dv, dtype, 2 * D, 2 * D)
    want = gu.to_host(s.dcache)
    s.to_device()
    got = run(s, rr.Rotation(np.stack([np.ones((140, D // 2)), np.zeros((140, D // 2))], -1).astype(np.float32)), q, k, v,
              dtype, 3)
    assert np.array_equal(gu.to_host(s.dcache), want)
    there = np.ones(s.rows, bool)
    there[75] = False                       # the row in front of the third sequence
    assert np.array_equal(got[there], ref.to_bits(q, dtype)[there]) and not got[~there].any()


@pytest.mark.parametrize("dtype,top", [(0, 6e4), (1, 3e38), (1, 1e-30), (0, 3e-7)])
def test_norms_of_huge_and_tiny_rows(dtype, top):
    s = Setup([40], [40], 1, 128, 64, seed=9)
    s.to_device()
    q, k, v = heads(s, 2, dtype)
    q, k = (ref.to_f64(ref.to_bits(x / np.abs(x).max(-1, keepdims=True) * top, dtype), dtype) for x in (q, k))
    w = np.linspace(0.5, 1.5, 128).astype(np.float32)
    t = rr.Rotation(table_of(64, 128), q_weight=w, k_weight=w, eps=1e-12)
    check(s, t, q, k, v, dtype, run(s, t, q, k, v, dtype, 2))


@pytest.mark.parametrize("q_weight,k_weight", [(True, False), (False, True)])
def test_norm_of_one_of_them(q_weight, k_weight):
    s = Setup([33, 70], [33, 2], 2, 128, 128, seed=4)
    s.to_device()
    q, k, v = heads(s, 4, 1)
    w = np.linspace(-1, 2, 128).astype(np.float32)
    t = rr.Rotation(table_of(80, 64), True, q_weight=w if q_weight else None, k_weight=w if k_weight else None)
    check(s, t, q, k, v, 1, run(s, t, q, k, v, 1, 4))


def test_far_positions_and_a_long_table():
    """Entries past 2^31 bytes of a table; positions outside it are its ends."""
    import torch
    length, rot = (1 << 31) // 512 + 100, 128
    s = Setup([5], [5], 1, 128, 64, seed=6)
    s.to_device()
    q, k, v = heads(s, 1, 0)
    big = torch.zeros((length, rot // 2, 2), dtype=torch.float32, device="cuda")
    at = [length - 1, length - 60, 3, 2 ** 31 - 1, -2 ** 31]
    small = table_of(4, rot, 3.0)
    for p, e in ((length - 1, 1), (length - 60, 2), (3, 3), (0, 0)):
        big[p] = torch.from_numpy(small[e]).cuda()
    t = rr.Rotation(small, positions=[[1, 2, 3, 1, 0]])
    d = on_device(t, 5)
    pos = i32([at])
    d = cider.cider_rotation(big, length, rot, False, pos)
    rows = [gu.bits_to_dev(ref.to_bits(x, 0).reshape(5, -1)) for x in (q, k, v)]
    out = torch.full((5, 128), 99, dtype=torch.int16, device="cuda")
    cider.cider_kv4_append_rotated(s.batch(s.dcache), d, *rows, 0, 128, 128, 128, 1, out, 128)
    check(s, t, q, k, v, 0, gu.bits_to_host(out).reshape(5, 1, 128))


def test_pages_that_are_not_there_and_sequences_left_out():
    s = Setup([100, 90, 64, 70], [100, 3, 5, 2], 2, 128, 64, seed=7)
    s.table[0, 1] = s.num_pages             # the second page of the first sequence
    s.table[1, 1] = -1
    s.to_device()
    q, k, v = heads(s, 2, 0)
    t = rotation_of(s, (64, False, 1, True))
    got = run(s, t, q, k, v, 0, 2, max_rows=50)   # the first sequence has more rows than the bound
    check(s, t, q, k, v, 0, got, skip=(0,))
    s.to_device()
    check(s, t, q, k, v, 0, run(s, t, q, k, v, 0, 2))


def test_only_keys_and_values():
    s = Setup([50], [20], 3, 64, 64, seed=8)
    s.to_device()
    _, k, v = heads(s, 1, 1)
    t = rotation_of(s, (64, True, 1, True))
    dk, dv = (gu.bits_to_dev(ref.to_bits(x, 1).reshape(20, -1)) for x in (k, v))
    cider.cider_kv4_append_rotated(s.batch(s.dcache), on_device(t, 20), None, dk, dv, 1, 0, 192, 192, 0, None, 0)
    want = ref.Cache(s.cache.data.copy(), 64, 64)
    rr.put_keys(want, s.table, s.lens, s.n, k, v, t, 64)
    assert np.array_equal(gu.to_host(s.dcache), want.data)


def test_step_by_step_and_all_at_once_are_the_same():
    t = rr.Rotation(table_of(200, 128), q_weight=np.ones(128, np.float32), k_weight=np.linspace(0, 1, 128, dtype=np.float32))
    one = Setup([150], [150], 2, 128, 64)
    one.to_device()
    q, k, v = heads(one, 2, 0)
    whole = run(one, t, q, k, v, 0, 2)
    steps = Setup([150], [150], 2, 128, 64)
    steps.to_device()
    lo = 0
    for n in (1, 1, 5, 30, 27, 1, 64, 21):
        part = Setup([lo + n], [n], 2, 128, 64)
        part.table, part.max_pages, part.num_pages = steps.table, steps.max_pages, steps.num_pages
        part.dcache = steps.dcache
        got = run(part, t, *(x[lo:lo + n] for x in (q, k, v)), 0, 2)
        assert np.array_equal(got, whole[lo:lo + n])
        lo += n
    assert np.array_equal(gu.to_host(steps.dcache), gu.to_host(one.dcache))


def test_another_stream():
    import torch
    s = Setup([70], [70], 2, 128, 64, seed=12)
    s.to_device()
    q, k, v = heads(s, 4, 1)
    t = rotation_of(s, (64, False, 3, True))
    stream = torch.cuda.Stream()
    check(s, t, q, k, v, 1, run(s, t, q, k, v, 1, 4, stream=stream))


def test_a_captured_step_follows_the_lengths():
    """One row a sequence, captured once and replayed while the lengths grow; each replay equals an eager call."""
    import torch
    lens = [61, 130, 5]
    s = Setup([x + 6 for x in lens], [1, 1, 1], 2, 128, 64, seed=13)
    q, k, v = heads(s, 4, 0)
    t = rotation_of(s, (64, False, 1, True))
    data = [gu.bits_to_dev(ref.to_bits(x, 0).reshape(3, -1)) for x in (q, k, v)]
    out = torch.zeros((3, 2 * 4 * 128), dtype=torch.int16, device="cuda")
    s.to_device()
    kv = i32(lens)
    turn = on_device(t, 3)

    def batch(cache):
        return cider.cider_kv4_batch(cache, pages, starts, kv, 3, 3, 1, s.max_pages * 64, s.max_pages, s.num_pages, 2, 128, 64)

    pages, starts = i32(s.table), i32([0, 1, 2, 3])
    captured, eager = batch(s.dcache), batch(s.dcache.clone())
    call = lambda b, o: cider.cider_kv4_append_rotated(b, turn, *data, 0, 1024, 256, 256, 8, o, 1024)  # noqa: E731
    call(captured, out)
    call(eager, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(captured, out)
    for step in range(6):
        kv += 1
        graph.replay()
        got = out.clone()
        call(eager, out)
        assert torch.equal(got, out)
        assert torch.equal(captured._tensors[0], eager._tensors[0])
        want, _ = t.apply(q[1], t.q_weight, 1, 130 + step)
        assert np.abs(ref.to_f64(gu.bits_to_host(got)[1].reshape(8, 128), 0) - want).max() < 0.02
