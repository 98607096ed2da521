"""The products where an expert's rows split into tiles, where few rows meet
several experts, and the bias gradient on both of its ways.  Bounds as in
test_linear.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_linear import ACTS, DTYPES, as_offsets, check_forward, check_gradient, normal  # noqa: E402


# rows about the tiles' edges: one tile's, one more, odd parts, parts of whole
# steps of 32; enough rows on average for each tile size
TILED = [[257, 511, 0, 513, 769, 1025, 31, 640], [256, 255, 512, 544], [65, 129, 1, 97, 64, 63], [33, 32, 160, 161, 127],
         [2049]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts", TILED)
def test_rows_that_split_into_tiles(gpu_lib, dtype, counts):
    dropped, n, k = 9, 520, 136
    m, e = sum(counts) + dropped, len(counts)
    x, w = normal((m, k), dtype, 1), normal((e, n, k), dtype, 2, k ** -0.5)
    offsets = as_offsets(np.array(counts))
    name = ACTS[m % 5]
    check_forward(gpu_lib, x, w, normal((e, n), dtype, 3), normal((m, n), dtype, 4), offsets, name, True)
    dy, pre = normal((m, n), dtype, 5), normal((m, n), dtype, 6)
    check_gradient(gpu_lib, dy, x, w, pre, offsets, name)


@pytest.mark.parametrize("counts", [[8], [0, 8, 0], [3, 0, 0, 5], [1, 1, 1, 1, 1], [7, 1]])
@pytest.mark.parametrize("n,k", [(200, 512), (33, 51)])
def test_few_rows_of_several_experts(gpu_lib, counts, n, k):
    m, e = sum(counts), len(counts)
    x, w = normal((m, k), torch.bfloat16, 1), normal((e, n, k), torch.bfloat16, 2, k ** -0.5)
    check_forward(gpu_lib, x, w, normal((e, n), torch.bfloat16, 3), None, as_offsets(np.array(counts)), "silu", True)


@pytest.mark.parametrize("counts,n,k", [([30000], 40, 24), ([70000], 40, 24), ([12000, 5, 0, 9000], 33, 17),
                                        ([1000, 0, 700], 1000, 64)])
def test_bias_gradient_beside_the_weight_gradient_and_alone(gpu_lib, counts, n, k):
    m, e = sum(counts), len(counts)
    x, w = normal((m, k), torch.float16, 1), normal((e, n, k), torch.float16, 2, k ** -0.5)
    dy, pre, offsets = normal((m, n), torch.float16, 3), normal((m, n), torch.float16, 4), as_offsets(np.array(counts))
    _, _, db = check_gradient(gpu_lib, dy, x, w, pre, offsets, "silu")
    _, none, alone = gpu_lib.kmeans_linear_grad(dy, x, w, pre=pre, offsets=offsets, activation="silu", need_dx=False,
                                                need_dw=False)
    assert none is None
    # the same partial sums in another order: both within (tiles) 2^-24 of their
    # magnitudes' sum before one rounding each
    magnitude = torch.stack([dy[a:b].double().abs().sum(0) for a, b in
                             zip(offsets.tolist()[:-1], offsets.tolist()[1:])]) * 1.1
    bound = 2 * (m / 16 + e) * 2.0 ** -24 * magnitude + 2 * 2.0 ** -11 * db.double().abs() + 2.0 ** -24
    assert bool(((alone.double() - db.double()).abs() <= bound).all())
