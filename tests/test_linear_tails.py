"""The activations where their result goes to zero with z: few rows and many,
forward and slope, against float64.

Bounds, fixed before any run, all relative to the value.  z Phi(z) and its slope
take 1 - erf of the formula 7.1.26 of Abramowitz and Stegun (the polynomial's
tail against erfc in float64: at most 0.4% off up to z = -6 and 3.2% up to -12).
exp2's argument reaches 104 for them and 130 for the logistic forms (z = -90, and
z = -9 of the tanh form), so its rounding shifts the power by 130 2^-24 ln 2 or
less, three such roundings by 2^-15.  A result in 8 bits is within 2^-8 of
itself."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_linear import act  # noqa: E402

CASES = [("gelu", -6.0, -1.5, 0.004), ("gelu", -12.0, -6.0, 0.032), ("gelu_tanh", -9.0, -1.5, 0.0),
         ("silu", -80.0, -2.0, 0.0)]


def exact(z, name):
    """The activation of z < 0 without differences of nearly equal values."""
    if name == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return z * torch.sigmoid(2 * u)
    return act(z, name)


@pytest.mark.parametrize("name,lo,hi,formula", CASES)
@pytest.mark.parametrize("m", [8, 2048])
def test_the_negative_tail_keeps_its_bits(gpu_lib, m, name, lo, hi, formula):
    z = torch.linspace(lo, hi, m, device="cuda").bfloat16()
    x, w = torch.zeros(m, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0], w[0, 0] = z, 1
    bound = 2.0 ** -8 + formula + 2.0 ** -15
    y, pre = gpu_lib.kmeans_linear(x, w, activation=name, save_pre=True)
    assert torch.equal(pre[:, 0], z)
    want = exact(z.double(), name)
    assert bool(((y[:, 0].double() - want).abs() <= bound * want.abs()).all())

    # dx[:, 0] = dy[:, 0] * slope, rounded once (dz) and copied by the product
    leaf = z.double().requires_grad_()
    want, = torch.autograd.grad(exact(leaf, name).sum(), leaf)
    dx, _, _ = gpu_lib.kmeans_linear_grad(x.bool().to(x.dtype), x, w, pre=pre, activation=name, need_dw=False,
                                          need_db=False)
    # near the slope's own zero (z = -0.75, -1.28 for SiLU) its terms cancel; here they do not
    assert bool(((dx[:, 0].double() - want).abs() <= bound * want.abs()).all())
