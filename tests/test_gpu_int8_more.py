"""More of the 8-bit inference operators: what a change of the factors after their
packing may not reach.  Needs a B200."""
import pytest
import torch

from expanded_rank_matrix_b200 import externd as X
from tests import int8_ref as R
from tests.test_gpu_int8 import _factors, _x

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 2, 40, 700])
def test_factors_changed_after_packing(t):
    """The codes stand for the factors as they were packed: their bound belongs
    to that D."""
    f, B, C, D = _factors(130, 200, 300, 1)
    x = _x(t, 200, torch.float32, 2)
    D = D.clone()
    c, head = X.pack_codes(f), X.pack_codes(X.truncate(X.Factors(f.packed_B, f.packed_C, f.D, f.D,
                                                                 f.m, f.n), 77))
    want, want_head = X.apply_i8(c, x), X.apply_i8(head, x)
    R.check(want, *R.factors(*R.rows(x), B, C, D))
    f.D.mul_(1000.0)
    assert torch.equal(X.apply_i8(c, x), want) and torch.equal(X.apply_i8(head, x), want_head)
    f.packed_B.zero_()
    f.packed_C.zero_()
    assert torch.equal(X.apply_i8(c, x), want) and torch.equal(X.apply_i8(head, x), want_head)
