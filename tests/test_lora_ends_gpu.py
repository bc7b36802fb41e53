"""cider_lora_add where the product with A is infinite, past bf16's end or of very different sizes within a token, by the
formula in 64 bits: one launch and two, few rows and many, low ranks and high ones."""
import numpy as np
import pytest

import w4a8_quantized_linear_amd as cider
from tests import gpu_util as gu
from tests import kv4_reference as ref
from tests.rotate_reference import half_step
from tests.test_lora_gpu import Case, rounded

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


# rows, rank: in one launch; in two with 16 rows and less a segment, then with more, whose rows of B a wavefront has in
# registers or the workgroup in common
SHAPES = [(3, 16), (2, 8), (5, 24), (4, 128), (40, 16), (20, 32), (70, 64), (33, 128), (30, 40)]


def by_the_formula(c, got):
    """Infinite where the formula is, by its sign, NaN where it is, else within the derived bound."""
    with np.errstate(invalid="ignore"):
        y, bound = c.reference()
        got = ref.to_f64(got, c.dtype)
        fine = np.isfinite(y)
        assert np.array_equal(np.isnan(got), np.isnan(y))
        assert np.array_equal(got[~fine & ~np.isnan(y)], y[~fine & ~np.isnan(y)])
        ok = np.abs(got - y)[fine] <= (bound + half_step(c.dtype, np.abs(y) + bound))[fine]
    assert ok.all()
    return y


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,rank", SHAPES)
def test_an_infinite_input(rows, rank, dtype):
    """Adapter 1 takes the input with one sign for each number of t, so that rows of B of one sign have infinite outputs;
    those of both, NaN; and finite values next to it may be of any size."""
    c = Case([rows, rows], [1, 0], rank, 256, [64, 128], dtype, seed=21)
    c.a[1, :, 7] = np.abs(c.a[1, :, 7]) + 0.125
    c.a[1, :, 9] *= 2.0 ** 10
    c.b[1] = np.abs(c.b[1]) + 0.125
    c.b[1, 20:40] *= -1
    c.b[1, 40:90:2, rank // 2] *= -1
    c.x[0, 7], c.x[rows - 1, 7] = np.inf, -np.inf
    c.x[0, 9] = 2.0 ** 10
    c.a, c.b = rounded(c.a, dtype), rounded(c.b, dtype)
    y = by_the_formula(c, c.run())
    for row in (0, rows - 1):
        assert np.isinf(y[row]).any() and np.isnan(y[row]).any() and not np.isfinite(y[row]).any()
    assert np.isfinite(y[1:rows - 1]).all() and np.isfinite(y[rows:]).all()


@pytest.mark.parametrize("rows,rank", SHAPES)
def test_an_infinite_number_of_t_beside_finite_ones(rows, rank):
    """Of A: one slice's t has an infinite number, the other slice's has none."""
    c = Case([rows], [1], rank, 256, [64, 128], 0, seed=22)
    c.a[1, 1, 5] = np.inf
    c.x[:, 5] = np.where(np.arange(rows) % 2, -0.5, 0.25)
    c.b[1, :, 1] = np.where(np.arange(128) % 3, 0.5, -2.0)
    y = by_the_formula(c, c.run())
    assert np.isinf(y[:, :64]).all() and np.isfinite(y[:, 64:]).all()


@pytest.mark.parametrize("rows,rank", SHAPES)
def test_finite_numbers_of_t_that_bf16_has_no_place_for(rows, rank):
    """t = 2^128 (1 - 2^-10) rounds to infinity in bf16; the outputs are of ordinary size."""
    c = Case([rows], [1], rank, 128, [64], 1, seed=23, scale=False)
    c.x[:], c.a[1] = 0, 0
    c.x[:, 0], c.x[:, 70] = 2.0 ** 128 * (1 - 2.0 ** -8), 2.0 ** 118 * 3
    c.x[1::2] *= -1
    c.a[1, 0, [0, 70]] = 1
    c.b[1, :, 0] = np.where(np.arange(64) % 2, 2.0 ** -126, -(2.0 ** -120))
    assert np.isfinite(by_the_formula(c, c.run())).all()

@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,rank", SHAPES)
def test_numbers_of_t_far_apart(rows, rank, dtype):
    """Within a token and slice the first number of t is about 2^14, the others 1 and less, down to 2^-20, and some
    outputs take those alone: fp16 keeps 22 bits of a number down to 2^-16 of the largest, and of a smaller one what is
    above 2^-38 of that; bf16 16 bits of each."""
    c = Case([rows], [1], rank, 256, [64, 128], dtype, seed=24, scale=False)
    for s in range(2):
        a = c.a[1, s * rank:(s + 1) * rank]
        a *= 2.0 ** np.minimum(-(np.arange(rank) * 30 // rank) + 2, 0)[:, None]
        a[0] *= 2.0 ** 14
    c.a = rounded(c.a, dtype)
    c.b[1, ::2, 0] = 0
    c.y_in[:, ::2] = 0
    assert np.isfinite(by_the_formula(c, c.run())).all()
