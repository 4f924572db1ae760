"""What the definition of the 8-bit factored product costs in accuracy, in 64 bits.
CPU only."""
import pytest
import torch

from tests import int8_ref as R


def _case(n, m, k, seed):
    g = torch.Generator().manual_seed(seed)

    def ternary(rows, cols):
        sign = 2.0 * torch.randint(0, 2, (rows, cols), generator=g) - 1
        return (sign * (torch.rand(rows, cols, generator=g) < 0.62)).double()
    B, C = ternary(k, m), ternary(k, n)
    D = 0.02 * torch.arange(1, k + 1).float() ** -0.5 * torch.exp(0.2 * torch.randn(k, generator=g))
    return B, C, D, torch.randn(16, n, generator=g)


@pytest.mark.parametrize("n,m,k", [(640, 256, 1920), (2560, 256, 2000)])
def test_rounding_of_the_component_sums(n, m, k):
    """As the header states it: half a step of z for each nonzero of B's row at
    most, z sqrt(nonzeros / 12) as a rule (independent roundings, uniform over a
    step).  16 x 256 results estimate the latter to 1 / sqrt(2 * 4096) = 1.1 %, and
    the sum over a token's own roundings varies by sqrt(0.8 / (0.62 k)) = 2.6 %
    at most, over 16 tokens less: 10 % is four and more of both."""
    B, C, D, x = _case(n, m, k, n)
    q, s = R.rows(x)
    exact = ((q @ C.T) * D.double()) @ B
    h, z = R.components(q, C, D)
    err = (z[:, None] * (h @ B) - exact) / z[:, None]
    nonzeros = B.abs().sum(0)
    # (the components' own rounding to fp32: half a step of values below 32512)
    assert (err.abs() <= 0.5 * nonzeros + k * 32512 * R.U32).all()
    assert (err / (nonzeros / 12).sqrt()).square().mean().sqrt().sub(1).abs() < 0.1
    assert h.abs().max() <= 32512


def test_bits_that_the_bound_leaves_unused():
    """The bound holds for any token, so a usual one's sums are about sqrt(n) below
    it: the largest of |h| stays far below 16 bits, the more so with n."""
    tops = []
    for n in (160, 640, 2560):
        B, C, D, x = _case(n, 8, 1000, 1)
        h, z = R.components(R.rows(x)[0], C, D)
        tops.append(float(h.abs().max()))
    assert tops[0] > tops[1] > tops[2] and tops[2] < 32512 / 8
