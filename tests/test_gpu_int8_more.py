"""More of the 8-bit inference operators: what a change of the factors after their
packing may not reach, the memory that a call takes, and whose errors are
whose, the smallest numbers of each type, gradients, and negated views.  Needs a B200."""
import pytest
import torch

from expanded_rank_matrix_b200 import externd as X
from tests import int8_ref as R
from tests.test_gpu_int8 import _factors, _gen, _held, _x

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


def _taken(call):
    """The call's result, and the device memory that it leaves in the library's pool."""
    call()  # (code and torch's own blocks)
    torch.cuda.synchronize()
    assert X.load().externd_release_cache() == X.OK
    before = torch.cuda.mem_get_info()[0]
    y = call()
    torch.cuda.synchronize()
    return y, before - torch.cuda.mem_get_info()[0]


def test_scratch_of_the_longest_ranks():
    """4096 tokens of the largest rank: passes of fewer tokens, and the same
    results over their seams."""
    t, m, n, k = 4096, 9, 40, X.I8_MAX_INNER
    f, B, C, D = _factors(m, n, k, 1)
    c, x = X.pack_codes(f), _x(t, n, torch.float32, 2)
    y, taken = _taken(lambda: X.apply_i8(c, x))
    assert taken <= 300 << 20
    q, s = R.rows(x)
    for i in (0, 510, 766, 1534, 2302, 4092):  # (passes of 768 tokens)
        R.check(y[i:i + 4], *R.factors(q[i:i + 4], s[i:i + 4], B, C, D))


def test_scratch_of_the_longest_rows():
    t, m, n = 8192, 16, X.I8_MAX_INNER
    x, w = _x(t, n, torch.float16, 1), _held(m, n, 2)
    y, taken = _taken(lambda: X.matmul_i8(x, w, out_dtype=torch.float32))
    assert taken <= 300 << 20
    for i in (0, 1790, 1792, 3583, 8188):  # (passes of 1792)
        R.check(y[i:i + 4], *R.dense(*R.rows(x[i:i + 4]), w.q, w.scale))


@pytest.mark.parametrize("block", [1, 32])
def test_decompositions_beside_rows_that_are_not_finite(block):
    """A row that is not finite is no error of a decomposition made after it, and
    is still reported behind one."""
    x = _x(3, 64, torch.float32, 1)
    x[1, 5] = float("nan")
    A = _x(96, 64, torch.float32, 2)
    bad = A.clone()
    bad[0, 0] = float("inf")
    assert X.sync_status() == X.OK
    f = X.decompose(A, 0.5, 0.5, 2, block=block)
    for call in (lambda: X.quantize_rows(x), lambda: X.apply_i8(X.pack_codes(f), x),
                 lambda: X.matmul_i8(x, X.Quantized(*_rows(A)))):
        call()
        g = X.decompose(A, 0.5, 0.5, 2, block=block)
        assert torch.equal(g.D, f.D)
        assert X.sync_status() == X.ERR_NONFINITE and X.sync_status() == X.OK
        call()
        with pytest.raises(X.ExterndError) as e:
            X.decompose(bad, 0.5, 0.5, 2, block=block)
        assert e.value.code == X.ERR_NONFINITE
        assert X.sync_status() == X.ERR_NONFINITE and X.sync_status() == X.OK


def _rows(A):
    r = X.quantize_rows(A)
    return r.q, r.scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [24, 2560, 2561])
def test_subnormal_rows(dtype, n):
    """Rows whose largest magnitude is a subnormal of the type, down to its
    smallest, and rows that mix subnormals with normal numbers."""
    tiny = torch.finfo(dtype).tiny
    step = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}[dtype]
    g = torch.Generator().manual_seed(n)
    rows = [torch.full((n,), step, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)]
    rows[1][n // 2] = -step
    for top in (2, 3, 126, 127, 128, tiny / step - 1, tiny / step, 300 * tiny / step):
        v = torch.randint(-int(top), int(top) + 1, (n,), generator=g).double() * step
        v[n - 1] = top * step
        rows.append(v)
    x = torch.stack(rows).to(dtype)
    assert (x.double().abs().amax(1) > 0).all()
    x = x.cuda()
    r = X.quantize_rows(x)
    q, s = R.rows(x)
    assert torch.equal(r.scale.double(), s) and torch.equal(r.q.double(), q)
    w = _held(40, n, 2)
    R.check(X.matmul_i8(x, w, out_dtype=torch.float32), *R.dense(q, s, w.q, w.scale))
    for i in range(len(rows)):  # (a single row is quantised within the product)
        R.check(X.matmul_i8(x[i:i + 1], w, out_dtype=torch.float32),
                *R.dense(q[i:i + 1], s[i:i + 1], w.q, w.scale))
    assert X.sync_status() == X.OK


def test_no_gradients():
    f, *_ = _factors(20, 32, 30, 1)
    w, c = _held(20, 32, 2), X.pack_codes(f)
    x = _x(3, 32, torch.float32, 3).requires_grad_()
    b = torch.zeros(20, device="cuda", requires_grad=True)
    r = X.quantize_rows(x)
    for y in (r.q, r.scale, X.matmul_i8(x, w, bias=b), X.apply_i8(c, x)):
        assert not y.requires_grad and y.grad_fn is None
    # what does have a gradient keeps its own
    (x.sum() + X.apply_i8(c, x).sum()).backward()
    assert torch.equal(x.grad, torch.ones_like(x)) and b.grad is None
    for make in (X.quantize_rows, X.matmul_i8, X.apply_i8):
        assert "Not differentiable" in make.__doc__


def test_negated_views():
    """Tensors that hold the negatives of their values (the imaginary part of a
    conjugate), in the shapes that need no copy for their layout."""
    z = torch.randn(5, 8, dtype=torch.complex64, generator=_gen(1), device="cuda").conj().imag
    assert z.is_neg()
    for x in (z, z[:, :1], z[:1, :1], torch._neg_view(_x(4, 32, torch.float32, 2))):
        assert x.is_neg()
        n = x.shape[1]
        plain = x + 0.0
        assert not plain.is_neg()
        w, c = _held(6, n, 3), X.pack_codes(_factors(6, n, 9, 4)[0])
        a, b = X.quantize_rows(x), X.quantize_rows(plain)
        assert torch.equal(a.q, b.q) and torch.equal(a.scale, b.scale)
        assert torch.equal(X.matmul_i8(x, w), X.matmul_i8(plain, w))
        assert torch.equal(X.apply_i8(c, x), X.apply_i8(c, plain))
    v = torch._neg_view(_x(1, 6, torch.float32, 5)[0])
    x, w = _x(2, 16, torch.float32, 6), _held(6, 16, 7)
    assert torch.equal(X.matmul_i8(x, w, bias=v), X.matmul_i8(x, w, bias=v + 0.0))
    assert torch.equal(X.matmul_i8(x, X.Quantized(w.q, v)), X.matmul_i8(x, X.Quantized(w.q, v + 0.0)))


@pytest.mark.parametrize("t", [1, 2, 40, 700])
def test_columns_of_a_wider_matrix(t):
    """8-bit operands that are columns of a wider matrix, taken as they are: the
    last row ends with its own 16 bytes, at the end of the storage."""
    n, m, k = 61, 70, 90
    g = _gen(t)
    base = torch.randint(-127, 128, (t, 192), generator=g, device="cuda", dtype=torch.int8)
    wide = torch.randint(-127, 128, (m, 160), generator=g, device="cuda", dtype=torch.int8)
    s, ws = torch.rand(t, generator=g, device="cuda"), torch.rand(m, generator=g, device="cuda")
    x, w = X.Quantized(base[:, 128:128 + n], s), X.Quantized(wide[:, 96:96 + n], ws)
    assert x.q.data_ptr() == base.data_ptr() + 128 and w.q.data_ptr() == wide.data_ptr() + 96
    R.check(X.matmul_i8(x, w), *R.dense(x.q, s, w.q, ws))
    f, B, C, D = _factors(m, n, k, 3)
    R.check(X.apply_i8(X.pack_codes(f), x), *R.factors(x.q.double(), s, B, C, D))
