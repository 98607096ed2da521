"""Groups whose two best experts have biases of opposite sign: their sum cancels,
and what decides between two groups is smaller than a last bit of either part.
Compared with float64, in which s + bias and the sums of two are formed as the
operator's definition says; rows that float64 itself cannot tell apart (nearer
than 2^-48 of the parts) are left out."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def scores_of(z, kind):
    z = z.astype(np.float64)
    if kind == "sigmoid":
        return 1 / (1 + np.exp(-z))
    e = np.exp(z - z.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def kept_groups(z, bias, kind, groups, topk_groups):
    """The groups that stay, (n, groups), and how near the last of them is to the first that does not."""
    n, E = z.shape
    c = scores_of(z, kind) + bias.astype(np.float64)
    best = np.sort(c.reshape(n, groups, E // groups), 2)[:, :, -2:]
    total = best[:, :, 1] + best[:, :, 0]
    order = np.argsort(-total, 1, kind="stable")
    kept = np.zeros((n, groups), bool)
    np.put_along_axis(kept, order[:, :topk_groups], True, 1)
    t = np.take_along_axis(total, order, 1)
    return c, kept, t[:, topk_groups - 1] - t[:, topk_groups]


def draw(kind, groups, size, large, n, seed):
    """One expert of a group pinned, the others held back by about as much.  The logits differ from group to group by
    about as much as a float32 of the bias's size can tell, half of that, and a hundredth of it."""
    r = np.random.RandomState(seed)
    base = r.randn(size)
    step = large * 2.0 ** -22 * np.array([1, 0.5, 0.01])[np.arange(n) % 3][:, None, None]
    z = (base + step * r.randn(n, groups, size)).reshape(n, groups * size).astype(np.float32)
    bias = np.full((groups, size), -large, np.float32)
    bias[:, 0] = large
    return z, bias.ravel()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("large", [32.0, 64.0, 1000.0, 1e4, 1e6])
@pytest.mark.parametrize("groups,topk_groups,size", [(2, 1, 2), (8, 3, 4), (5, 2, 6), (32, 8, 8), (8, 4, 128)])
def test_groups_whose_biases_cancel(gpu_lib, kind, large, groups, topk_groups, size):
    n, topk = 600, min(4, topk_groups * size)
    z, bias = draw(kind, groups, size, large, n, groups + size)
    c, kept, gap = kept_groups(z, bias, kind, groups, topk_groups)
    clear = gap > 2.0 ** -48 * large
    assert clear.sum() > n // 3
    ids, _ = gpu_lib.kmeans_gate(torch.from_numpy(z).cuda(), topk, scores=kind, bias=torch.from_numpy(bias).cuda(),
                                 groups=groups, topk_groups=topk_groups)
    c = np.where(np.repeat(kept, size, 1), c, -np.inf)
    want = np.argsort(-c, 1, kind="stable")[:, :topk]
    order = -np.sort(-c, 1)[:, :topk + 1]
    with np.errstate(invalid="ignore"):
        clear &= ~((order[:, :-1] - order[:, 1:]) < 2.0 ** -48 * large).any(1)
    assert clear.sum() > n // 3
    assert np.array_equal(ids.cpu().numpy()[clear], want[clear])


def test_two_groups_of_a_pinned_and_a_discouraged_expert(gpu_lib):
    """In float32 the sums are 1.125 and 1.0625; they are 1.0640 and 1.1230."""
    z = torch.tensor([[0.1282, 0.1282, 0.3763, 0.1201]], device="cuda")
    bias = torch.tensor([1e6, -1e6, 1e6, -1e6], device="cuda")
    ids, _ = gpu_lib.kmeans_gate(z, 2, scores="sigmoid", bias=bias, groups=2, topk_groups=1)
    assert ids.tolist() == [[2, 3]]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_a_group_that_is_pinned_without_end_beside_ordinary_ones(gpu_lib, kind):
    """A bias of infinity is exact in the order; the other groups' sums are ordinary ones."""
    r = np.random.RandomState(3)
    z, bias = r.randn(500, 32).astype(np.float32), (0.1 * r.randn(32)).astype(np.float32)
    bias[9] = np.inf
    c, kept, gap = kept_groups(z, bias, kind, 8, 3)
    clear = gap > 2.0 ** -48
    assert clear.sum() > 490 and kept[:, 2].all()
    ids, _ = gpu_lib.kmeans_gate(torch.from_numpy(z).cuda(), 5, scores=kind, bias=torch.from_numpy(bias).cuda(), groups=8,
                                 topk_groups=3)
    want = np.argsort(-np.where(np.repeat(kept, 4, 1), c, -np.inf), 1, kind="stable")[:, :5]
    assert np.array_equal(ids.cpu().numpy()[clear], want[clear])


def by_definition(z, bias, kind, topk, groups, topk_groups):
    """Token by token in float64; a logit or a bias of -inf closes."""
    s = scores_of(z, kind)
    n, E = z.shape
    size = E // groups
    ids = np.full((n, topk), -1, np.int64)
    for t in range(n):
        c = s[t] + bias.astype(np.float64)
        total = []
        for g in range(groups):
            best = sorted(c[g * size:(g + 1) * size], reverse=True)[:2]
            total.append(best[0] if len(best) < 2 or best[1] == -np.inf else best[0] + best[1])
        for g in sorted(range(groups), key=lambda g: (-total[g], g))[topk_groups:]:
            c[g * size:(g + 1) * size] = -np.inf
        order = sorted((e for e in range(E) if c[e] != -np.inf), key=lambda e: (-c[e], e))[:topk]
        ids[t, :len(order)] = order
    return ids


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", [float(np.finfo(np.float32).min), -3e38, -1.5e38, -1e30, -1e4])
@pytest.mark.parametrize("E,groups", [(32, 8), (30, 5), (256, 8), (96, 32)])
def test_masks_of_the_lowest_value(gpu_lib, kind, E, groups, mask):
    """A large negative bias holds an expert back, it does not close it: whole groups of such ones stay where the
    number of groups asks for them, though their sums pass float32."""
    n, size = 40, E // groups
    r = np.random.RandomState(E)
    z, bias = r.randn(n, E).astype(np.float32), (0.1 * r.randn(E)).astype(np.float32)
    for g in (1, 3, groups - 1):
        bias[g * size:(g + 1) * size] = mask
    bias[2 * size + 1:3 * size] = mask  # one left
    for topk_groups in sorted({1, groups // 2, groups - 3, groups - 2, groups - 1, groups}):
        for topk in (2, min(32, topk_groups * size)):
            ids, _ = gpu_lib.kmeans_gate(torch.from_numpy(z).cuda(), topk, scores=kind, bias=torch.from_numpy(bias).cuda(),
                                         groups=groups, topk_groups=topk_groups)
            want = by_definition(z, bias, kind, topk, groups, topk_groups)
            assert np.array_equal(ids.cpu().numpy(), want), (topk_groups, topk)


@pytest.mark.parametrize("large", [1e4, 1e30, 3e38])
def test_a_group_with_large_biases_does_not_disturb_the_others(gpu_lib, large):
    """Pinned in one group, held back in another: the groups between them are told apart as without those."""
    n, E, groups = 300, 64, 8
    r = np.random.RandomState(5)
    z, bias = r.randn(n, E).astype(np.float32), (0.1 * r.randn(E)).astype(np.float32)
    bias[8:16], bias[40:48] = large, -large
    ids, _ = gpu_lib.kmeans_gate(torch.from_numpy(z).cuda(), 12, scores="sigmoid", bias=torch.from_numpy(bias).cuda(),
                                 groups=groups, topk_groups=3)
    assert np.array_equal(ids.cpu().numpy(), by_definition(z, bias, "sigmoid", 12, groups, 3))
