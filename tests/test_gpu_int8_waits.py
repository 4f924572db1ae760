"""The bounded waits of the 8-bit tensor-core kernels, with a budget so short
that they run out: the call reports it, the kernels leave in order, and the
next call on the same context is exact.  Needs a B200."""
import time

import pytest
import torch

from expanded_rank_matrix_b200 import externd as X
from tests import int8_ref as R
from tests.test_gpu_int8 import _factors, _held, _x

pytestmark = pytest.mark.gpu


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _matmul(x, w, budget):
    t, m = x.q.shape[0], w.q.shape[0]
    y = torch.empty(t, m, device="cuda")
    assert X.load().externd_matmul_i8_ex(
        x.q.data_ptr(), X.I8, x.q.stride(0), x.scale.data_ptr(), w.q.data_ptr(), w.q.stride(0),
        w.scale.data_ptr(), None, t, x.q.shape[1], m, y.data_ptr(), X.F32, m, budget,
        _stream()) == X.OK
    return y


def _apply(c, x, budget):
    t = x.shape[0]
    y = torch.empty(t, c.m, device="cuda")
    assert X.load().externd_ternary_apply_i8_ex(
        c.codes_B.data_ptr(), c.codes_C.data_ptr(), c.D.data_ptr(), c.bound.data_ptr(), c.m, c.n,
        c.k, x.data_ptr(), X.F32, x.shape[1], None, t, y.data_ptr(), X.F32, c.m, budget,
        _stream()) == X.OK
    return y


# few tiles, split over clusters; many, on pairs of CTAs; more than the GPU holds.
# (Inner dimensions long enough that an epilogue waits for its products longer
# than a test of a barrier may pause.)
@pytest.mark.parametrize("t,m,n", [(32, 2560, 40000), (100, 300, 65536), (1024, 2560, 20000),
                                   (3000, 5000, 9999)])
def test_product_waits_run_out(t, m, n):
    x, w = _held(t, n, 1), _held(m, n, 2)
    _matmul(x, w, 1)
    assert X.sync_status() == X.ERR_TIMEOUT
    for budget in (0, 1 << 40):
        y = _matmul(x, w, budget)
        assert X.sync_status() == X.OK
        R.check(y, *R.dense(x.q, x.scale, w.q, w.scale))


@pytest.mark.parametrize("t,m,n,k", [(24, 512, 65536, 384), (100, 384, 512, 65536),
                                     (16, 9728, 2560, 30000), (1024, 2560, 1300, 20000),
                                     (3000, 2560, 700, 20000)])
def test_factors_waits_run_out(t, m, n, k):
    f, B, C, D = _factors(m, n, k, t)
    c, x = X.pack_codes(f), _x(t, n, torch.float32, 1)
    _apply(c, x, 1)
    assert X.sync_status() == X.ERR_TIMEOUT
    for budget in (0, 1 << 40):
        y = _apply(c, x, budget)
        assert X.sync_status() == X.OK
        R.check(y, *R.factors(*R.rows(x), B, C, D))


@pytest.mark.parametrize("budget", [1, 30, 300, 1000, 2000, 4000, 8000, 16000])
def test_waits_run_out_anywhere(budget):
    """Budgets that run out at some wait or other, in some CTAs and not in
    others: nothing hangs, and calls that report no timeout are exact."""
    t, m, n, k = 700, 2560, 2560, 2600
    x, w = _held(t, n, 1), _held(m, n, 2)
    f, B, C, D = _factors(m, n, k, 3)
    c, xf = X.pack_codes(f), _x(t, n, torch.float32, 4)
    xs, ws = _held(40, n, 5), _held(300, n, 6)
    want = _matmul(x, w, 0), _apply(c, xf, 0), _matmul(xs, ws, 0)
    assert X.sync_status() == X.OK
    for r in range(5):
        for i, call in enumerate((lambda: _matmul(x, w, budget), lambda: _apply(c, xf, budget),
                                  lambda: _matmul(xs, ws, budget))):
            t0 = time.perf_counter()
            y = call()
            st = X.sync_status()
            # (the waits of the end have an end of their own, a second: they
            # were answered)
            assert time.perf_counter() - t0 < 0.5
            assert st in (X.OK, X.ERR_TIMEOUT)
            if st == X.OK:
                assert torch.equal(y, want[i])
    assert torch.equal(_matmul(x, w, 0), want[0]) and torch.equal(_apply(c, xf, 0), want[1])
    assert torch.equal(_matmul(xs, ws, 0), want[2]) and X.sync_status() == X.OK
