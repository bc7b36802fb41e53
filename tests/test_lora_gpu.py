"""cider_lora_add on the GPU against 64 bits within a derived bound: every rank, one and several slices, one row to many,
inputs that do not fill a workgroup's share, slots that are none or shared, segments that are not sound, values at the
ends of the types, strides, in place, workspaces of any size, streams and graphs; and the whole of a projection with its
adapters against the quantized product."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests.rotate_reference import half_step
from tests.test_kv4_gpu import i32

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


def rounded(x, dtype):
    return ref.to_f64(ref.to_bits(x, dtype), dtype).reshape(np.shape(x))


class Case:
    def __init__(self, rows, slots, rank, inputs, ends, dtype, adapters=4, seed=0, x_std=1.0, a_std=None, b_std=None,
                 scale=True):
        r = np.random.default_rng([seed, rank, inputs, len(rows)])
        self.counts, self.slots, self.R, self.K, self.ends, self.dtype = list(rows), list(slots), rank, inputs, ends, dtype
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
        self.rows, self.N, S = int(self.start[-1]), ends[-1], len(ends)
        self.x = rounded(r.standard_normal((self.rows, inputs)) * x_std, dtype)
        self.a = rounded(r.standard_normal((adapters, S * rank, inputs)) * (a_std or inputs ** -0.5), dtype)
        self.b = rounded(r.standard_normal((adapters, self.N, rank)) * (b_std or rank ** -0.5), dtype)
        self.scale = r.uniform(0.25, 2, adapters).astype(np.float32) if scale else None
        self.y_in = rounded(r.standard_normal((self.rows, self.N)), dtype)

    def reference(self):
        """(y, bound without the output's rounding).

        With T = sum |A||x| and D = sum |B| scale T: t is a sum of `inputs` exact products in fp32, in products of 32
        on the matrix cores, chains of which are added up; any order of the additions is off by at most inputs 2^-24 T,
        and in fact by few of them: 2^-16 T covers 256 roundings in a row (chains here are of 128 steps and less, with
        a few levels on top).  High and low halves leave 2^-17 of t in bf16, 2^-22 in fp16, and of the token's largest
        t below fp16's steps 2^-38.  The second sum has 2 rank products: 2^-17.  The sum with y_in: 2^-24 of both."""
        y, bound = self.y_in.copy(), np.zeros_like(self.y_in)
        for i, slot in enumerate(self.slots):
            if not 0 <= slot < len(self.a):
                continue
            lo, hi = self.start[i], self.start[i + 1]
            f = 1.0 if self.scale is None else np.float64(self.scale[slot])
            first = 0
            for s, end in enumerate(self.ends):
                a, b = self.a[slot, s * self.R:(s + 1) * self.R], self.b[slot, first:end]
                t, size = self.x[lo:hi] @ a.T * f, np.abs(self.x[lo:hi]) @ np.abs(a).T * f
                y[lo:hi, first:end] += t @ b.T
                bound[lo:hi, first:end] = (2.0 ** -16 + 2.0 ** -17) * (size @ np.abs(b).T) + 2.0 ** -17 * (np.abs(t) @ np.abs(b).T) \
                    + 2.0 ** -38 * np.abs(t).max(1, initial=0, keepdims=True) * np.abs(b).sum(1) + 2.0 ** -23 * np.abs(y[lo:hi, first:end])
                first = end
        return y, bound

    def device(self):
        import torch
        w = lambda x: gu.bits_to_dev(ref.to_bits(x, self.dtype))  # noqa: E731
        sc = None if self.scale is None else torch.from_numpy(self.scale).cuda()
        return cider.cider_lora(w(self.a), w(self.b), sc, len(self.a), self.R, self.K, self.ends)

    def run(self, in_place=False, max_rows=None, segments=None, nbytes=None, stream=None):
        """Patterns [rows, N] of y; every stride has room, with NaN beside x and 99 beside y."""
        import torch
        ldx, ldi = self.K + 24, self.N + 16
        ldo = ldi if in_place else self.N + 8
        x = np.full((self.rows, ldx), 0x7FFF, np.uint16)
        x[:, :self.K] = ref.to_bits(self.x, self.dtype)
        y_in = np.full((self.rows, ldi), 99, np.uint16)
        y_in[:, :self.N] = ref.to_bits(self.y_in, self.dtype)
        dx, di = gu.bits_to_dev(x), gu.bits_to_dev(y_in)
        out = di if in_place else torch.full((self.rows, ldo), 99, dtype=torch.int16, device="cuda")
        lora = self.device()
        most = max(self.counts) if max_rows is None else max_rows
        starts, slots = (self.start, self.slots) if segments is None else segments
        need = cider.cider_lora_workspace_bytes(lora, len(slots), self.rows, most) if nbytes is None else nbytes
        ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        gu.sync()
        cider.cider_lora_add(lora, i32(starts), i32(slots), len(slots), self.rows, most, dx, self.dtype, ldx, di, ldi,
                             ws, need, out, ldo, stream)
        gu.sync()
        assert (ws[need:] == 0xFF).all()
        got = gu.bits_to_host(out)
        assert (got[:, self.N:] == 99).all()
        return got[:, :self.N]

    def check(self, got, rows=slice(None)):
        """An infinite input (x_std may take some past fp16's end) has outputs that are no numbers, by the formula too."""
        with np.errstate(invalid="ignore"):
            y, bound = self.reference()
        got = ref.to_f64(got, self.dtype)
        fine = np.isfinite(y)
        assert not np.isfinite(got[rows][~fine[rows]]).any()
        e = np.where(fine, np.abs(np.where(fine, got - np.where(fine, y, 0), 0)), 0)[rows]
        ok = e <= np.where(fine, bound + half_step(self.dtype, np.abs(np.where(fine, y, 0)) + bound), 0)[rows]
        assert ok.all(), "%d of %d outside, worst %.3g" % ((~ok).sum(), ok.size, e[~ok].max())


SHAPES = [
    # rows of segments, slots, rank, inputs, ends
    ([1], [0], 16, 64, [64]),
    ([1], [3], 8, 4096, [128]),
    ([1, 1, 1, 1], [2, -1, 2, 0], 16, 320, [64, 128, 192]),
    ([2, 0, 5, 1], [1, 0, 3, 4], 24, 1088, [128, 192]),
    ([16, 17], [0, 1], 32, 512, [64]),
    ([33, 1, 64, 70], [3, 0, 1, 3], 16, 704, [192, 256, 320]),
    ([130], [2], 64, 1024, [128, 256]),
    ([9, 40], [1, 2], 128, 448, [64, 192]),
    ([5], [1], 128, 256, [128]),
    ([50, 3], [0, 3], 40, 192, [64]),
    ([31], [0], 56, 128, [64, 128, 192, 256, 320, 384, 448, 512]),
    ([100], [1], 104, 640, [64]),
    ([20], [7], 16, 64, [64]),                       # no such slot
    ([300, 299], [0, 1], 16, 2048, [1024]),
]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_against_64_bits(shape, dtype):
    c = Case(*SHAPES[shape], dtype, seed=shape, scale=shape % 3 != 0)
    got = c.run(in_place=shape % 2 == 1)
    c.check(got)
    for i, slot in enumerate(c.slots):   # without an adapter every bit stays
        if not 0 <= slot < 4:
            at = slice(c.start[i], c.start[i + 1])
            assert np.array_equal(got[at], ref.to_bits(c.y_in, dtype)[at])


@pytest.mark.parametrize("rank", range(8, 129, 8))
def test_every_rank(rank):
    for rows in ([3], [20], [70]):
        c = Case(rows, [1], rank, 128, [64, 128], rank // 8 % 2, seed=1)
        c.check(c.run())


@pytest.mark.parametrize("inputs", [64, 128, 192, 512, 576, 2112, 8256])
def test_every_share_of_the_inputs(inputs):
    """And every number of parts that a smaller workspace leaves, down to one."""
    for rows, rank, ends in (([1], 16, [64]), ([40], 32, [64, 128])):
        c = Case(rows, [2], rank, inputs, ends, 0, seed=2)
        one = c.rows * rank * len(ends) * 4
        most = cider.cider_lora_workspace_bytes(c.device(), 1, c.rows, c.rows) // one
        for parts in {1, 2, 3, most}:
            c.check(c.run(nbytes=parts * one + parts % 2 * 4))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rank", [8, 16])
def test_many_segments_of_few_rows(rank, dtype):
    """More than one launch of both products holds at once, and fewer; outputs that end inside a workgroup's."""
    r = np.random.default_rng(rank)
    for segments, ends in ((200, [64]), (90, [1088, 1152]), (40, [1088, 1152])):
        rows = list(r.integers(0, 4, segments))
        c = Case(rows, r.integers(-1, 4, segments), rank, 192, ends, dtype, seed=13)
        c.check(c.run(in_place=dtype == 1))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rank,rows", [(16, 16), (16, 17), (24, 16), (24, 17), (64, 16), (64, 17), (40, 150),
                                       (128, 16), (128, 17), (104, 90)])
def test_workgroups_of_several_blocks(rank, rows, dtype):
    """So many outputs and tiles that a workgroup takes some blocks of outputs in turn, with slices that end inside its
    share and a slot that is none."""
    r = np.random.default_rng(rank)
    counts = [rows] + list(r.integers(1, min(rows, 17) + 1, 29))
    c = Case(counts, r.integers(-1, 4, 30), rank, 64, [64 * 7, 64 * 130, 64 * 131, 64 * 149], dtype, seed=14)
    c.check(c.run(in_place=dtype == 0))


@pytest.mark.parametrize("dtype,x_std,a_std,b_std", [
    (0, 2e4, 1.0, 1e-4), (0, 1e-6, 1e-3, 1e3), (1, 1e15, 1e10, 1e-26), (1, 1e-20, 1e-10, 1e30), (0, 1.0, 100.0, 1e-3),
])
def test_products_far_from_one(dtype, x_std, a_std, b_std):
    """t past fp16's end or below its smallest number."""
    c = Case([3, 20], [0, 1], 16, 512, [64, 128], dtype, seed=3, x_std=x_std, a_std=a_std, b_std=b_std)
    c.check(c.run())


def test_a_row_keeps_to_itself():
    """NaN and infinity in one row's inputs, another's y_in and an adapter that others use not."""
    c = Case([5, 20, 40], [0, 1, 2], 16, 256, [64, 128], 0, seed=4)
    want = c.run()
    c.x[3, 7], c.x[10, 200], c.y_in[30, 5], c.a[1, 3, 9] = np.nan, np.inf, np.nan, np.nan
    got = c.run()
    clean = np.ones(c.rows, bool)
    clean[3] = clean[5:25] = clean[30] = False
    assert np.array_equal(got[clean], want[clean])
    assert np.isnan(ref.to_f64(got[3], 0)).all() and np.isnan(ref.to_f64(got[30, 5], 0))


@pytest.mark.parametrize("max_rows", [12, 100])
def test_segments_that_are_not_sound_are_left_out(max_rows):
    """Rows outside the call, falling starts, more rows than the bound: their rows stay as they were."""
    c = Case([10, 12, 13, 5], [0, 1, 2, 3], 16, 256, [64], 0, seed=5)
    got = c.run(max_rows=max_rows)
    long = c.start[2], c.start[3]
    keep = np.ones(c.rows, bool)
    if max_rows == 12:
        keep[long[0]:long[1]] = False
        assert (got[long[0]:long[1]] == 99).all()
    c.check(got, keep)
    for starts in ([-1, 10, 22, 35, 40], [0, 10, 9, 8, 41], [2 ** 31 - 1, -2 ** 31, 22, 35, 40]):
        got = c.run(segments=(starts, c.slots), max_rows=max_rows)
        sound = np.zeros(c.rows, bool)
        for i in range(4):
            a, b = starts[i], starts[i + 1]
            if 0 <= a <= b <= c.rows and b - a <= max_rows:
                sound[a:b] = True
        assert (got[~sound] == 99).all()
        if starts[2] == 22:
            c.check(got, sound)


@pytest.mark.parametrize("slot", [-1, -2 ** 31, 4, 2 ** 31 - 1])
def test_slots_that_are_none(slot):
    for rows in ([3], [40]):
        for in_place in (False, True):
            c = Case(rows, [slot], 16, 128, [128], 1, seed=6)
            assert np.array_equal(c.run(in_place=in_place), ref.to_bits(c.y_in, 1))


def test_rows_of_no_segment_stay():
    c = Case([4, 6, 5], [0, 1, 2], 16, 128, [64], 0, seed=7)
    got = c.run(segments=([4, 10], [1]), max_rows=6)
    assert (got[:4] == 99).all() and (got[10:] == 99).all()
    c.check(got, slice(4, 10))


def test_addresses_past_4_gib():
    """A slot whose A lies past 2^32 bytes."""
    import torch
    K, R, N = 8192, 128, 64
    slots = (1 << 32) // (R * K * 2) + 2
    c = Case([3], [0], R, K, [N], 1, adapters=1, seed=8)
    big = torch.zeros((slots, R, K), dtype=torch.int16, device="cuda")
    big[-1] = gu.bits_to_dev(ref.to_bits(c.a[0], 1))
    b = torch.zeros((slots, N, R), dtype=torch.int16, device="cuda")
    b[-1] = gu.bits_to_dev(ref.to_bits(c.b[0], 1))
    sc = torch.zeros(slots, device="cuda")
    sc[-1] = float(c.scale[0])
    lora = cider.cider_lora(big, b, sc, slots, R, K, [N])
    need = cider.cider_lora_workspace_bytes(lora, 1, 3, 3)
    ws, y = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.zeros((3, N), dtype=torch.int16, device="cuda")
    cider.cider_lora_add(lora, i32([0, 3]), i32([slots - 1]), 1, 3, 3, gu.bits_to_dev(ref.to_bits(c.x, 1)), 1, K,
                         gu.bits_to_dev(ref.to_bits(c.y_in, 1)), N, ws, need, y, N)
    c.check(gu.bits_to_host(y))


def test_another_stream():
    import torch
    c = Case([33, 1, 4], [1, 2, 1], 16, 512, [128, 192], 1, seed=9)
    c.check(c.run(stream=torch.cuda.Stream()))


def test_graphs_that_share_a_workspace():
    """Two captured calls, replayed by turns while slots and segments change, eager calls between."""
    import torch
    made = []
    for i, (rows, most) in enumerate((([1, 1, 1, 1], 1), ([30, 45], 60))):
        c = Case(rows, [0, 1, 2, 3][:len(rows)], 16, 512, [64, 192], 0, seed=10 + i)
        made.append([c, c.device(), i32(c.start), i32(c.slots), gu.bits_to_dev(ref.to_bits(c.x, 0)),
                     gu.bits_to_dev(ref.to_bits(c.y_in, 0)), torch.zeros((c.rows, c.N), dtype=torch.int16, device="cuda"), most])
    need = max(cider.cider_lora_workspace_bytes(m[1], len(m[0].slots), m[0].rows, m[7]) for m in made)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(m):
        c = m[0]
        cider.cider_lora_add(m[1], m[2], m[3], len(c.slots), c.rows, m[7], m[4], 0, c.K, m[5], c.N, ws, need, m[6], c.N)

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
            g.replay()
            got = m[6].clone()
            m[6].zero_()
            call(m)
            assert torch.equal(got, m[6])
            m[0].check(gu.bits_to_host(got))
            m[0].slots = [(s + 1) % 5 - 1 for s in m[0].slots]
            m[3].copy_(i32(m[0].slots))
        ws.fill_(turn)
        c = made[1][0]
        c.start = np.array([0, 30 - 5 * turn, 75])
        c.counts = [30 - 5 * turn, 45 + 5 * turn]
        made[1][2].copy_(i32(c.start))


def test_beside_the_quantized_product():
    """y = x W^T by cider_linear_ex, then the adapters on top, as a projection of several tenants is served: the sum is
    the product's own output plus the adapters' correction."""
    import torch
    c = Case([1, 20, 1, 7], [0, 1, -1, 2], 16, 512, [256, 384], 0, seed=12)
    w = torch.randn((c.N, c.K), device="cuda").half() / 20
    wq, s_w = torch.empty((c.N, c.K), dtype=torch.int8, device="cuda"), torch.empty(c.N, device="cuda")
    cider.cider_quantize_weight(w, c.N, c.K, 8, 0, wq, s_w)
    x = gu.bits_to_dev(ref.to_bits(c.x, 0))
    y = torch.empty((c.rows, c.N), dtype=torch.int16, device="cuda")
    nbytes = cider.cider_linear_workspace_bytes_ex(c.rows, c.N, c.K, 8, 0)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    cider.cider_linear_ex(x, 0, c.rows, c.K, c.K, None, wq, s_w, c.N, 8, 0, 0, ws, nbytes, y)
    c.y_in = ref.to_f64(gu.bits_to_host(y), 0)
    lora = c.device()
    need = cider.cider_lora_workspace_bytes(lora, 4, c.rows, 20)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    cider.cider_lora_add(lora, i32(c.start), i32(c.slots), 4, c.rows, 20, x, 0, c.K, y, c.N, ws, need, y, c.N)
    c.check(gu.bits_to_host(y))
