"""The 8-bit inference operators (quantize_rows, matmul_i8, pack_codes,
apply_i8) against plain 64-bit forms of their formulas.  Needs a B200."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from expanded_rank_matrix_b200 import externd as X
from expanded_rank_matrix_b200 import workloads as W
from tests import int8_ref as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FLOATS = [torch.float32, torch.float16, torch.bfloat16]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _x(t, n, dtype, seed):
    g = _gen(seed)
    x = torch.randn(t, n, generator=g, device="cuda")
    return (x * torch.exp(torch.randn(t, 1, generator=g, device="cuda"))).to(dtype)


def _held(rows, n, seed, lo=-127):
    """Random 8-bit rows in padded storage whose padding holds garbage."""
    g = _gen(seed)
    ld = (n + 15) // 16 * 16
    full = torch.randint(lo, 128, (rows, ld), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(rows, generator=g, device="cuda") * 0.01 + 1e-4
    return X.Quantized(full[:, :n], s)


def _ternary(k, length, seed, density=0.62):
    g = _gen(seed)
    v = torch.randint(0, 2, (k, length), generator=g, device="cuda") * 2 - 1
    return v * (torch.rand(k, length, generator=g, device="cuda") < density)


def _factors(m, n, k, seed, density=0.62):
    B, C = _ternary(k, m, seed, density), _ternary(k, n, seed + 1, density)
    D = 0.02 * torch.randn(k, generator=_gen(seed + 2), device="cuda")
    return X.Factors(R.planes(B), R.planes(C), D, None, m, n), B.double(), C.double(), D


# --- quantising rows ---------------------------------------------------------

@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("shape", [(1, 1), (1, 16), (3, 5), (9, 31), (2, 127), (5, 128), (7, 129),
                                   (300, 64), (33, 1024), (5, 2047), (6, 2049), (64, 2560),
                                   (3, 9729), (1, 20000), (2, 40001)])
def test_quantize_rows(dtype, shape):
    x = _x(*shape, dtype, sum(shape))
    r = X.quantize_rows(x)
    q, s = R.rows(x)
    assert r.q.shape == x.shape and r.q.dtype == torch.int8
    assert torch.equal(r.scale.double(), s)
    assert torch.equal(r.q.double(), q)
    assert X.sync_status() == X.OK


def test_quantize_borders_and_extremes():
    """Halves go to the even neighbour; neighbours of a half to their side;
    subnormal and huge rows keep the definition; a zero row is zero."""
    half = torch.tensor([127.0, 0.5, 1.5, 2.5, 63.5, -0.5, -1.5, -126.5, 0.0])
    up, down = torch.nextafter(half, torch.tensor(1e9)), torch.nextafter(half, torch.tensor(-1e9))
    up[0] = down[0] = 127.0
    rows = [half, up, down, half * 2.0 ** -20, half * 2.0 ** 100, half * 2.0 ** -120,
            half * 2.0 ** -141, half * 2.0 ** -149, torch.zeros(9), -torch.zeros(9),
            half * 2.0 ** 120, half / 3, half * 1.1, half * 2.0 ** -130 * 1.3]
    x = torch.stack(rows).cuda()
    r = X.quantize_rows(x)
    q, s = R.rows(x)
    assert torch.equal(r.scale.double(), s)
    assert torch.equal(r.q.double(), q)
    assert X.sync_status() == X.OK


@pytest.mark.parametrize("seed", range(3))
def test_quantize_every_border(seed):
    """Random scales with every half step of the range and its neighbours."""
    g = _gen(seed)
    s = torch.exp(20 * torch.randn(40, 1, generator=g, device="cuda")).clamp(1e-37, 1e35)
    steps = torch.arange(-126.5, 127.0, 0.5, device="cuda")[None, :]
    mid = s * steps
    big = torch.tensor(1e38, device="cuda")
    x = torch.cat([s * 127, mid, torch.nextafter(mid, big), torch.nextafter(mid, -big)], 1)
    r = X.quantize_rows(x)
    q, sc = R.rows(x)
    assert torch.equal(r.scale.double(), sc)
    assert torch.equal(r.q.double(), q)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("n", [40, 2560, 9729])
def test_quantize_rows_that_are_not_finite(dtype, n):
    x = _x(6, n, dtype, n)
    x[1, n - 1] = float("nan")
    x[3, 0] = float("inf")
    x[4, n // 2] = -float("inf")
    r = X.quantize_rows(x)
    assert X.sync_status() == X.ERR_NONFINITE
    q, s = R.rows(x)
    assert torch.equal(torch.isnan(r.scale), torch.isnan(s).cuda())
    assert torch.equal(r.q.double(), q)
    ok = ~torch.isnan(s)
    assert torch.equal(r.scale.double()[ok], s[ok])
    # the products with such a row are NaN, the others untouched
    w = _held(24, n, 5)
    y = X.matmul_i8(x, w, out_dtype=torch.float32)
    assert X.sync_status() == X.ERR_NONFINITE
    R.check(y, *R.dense(q, s, w.q, w.scale))
    f, B, C, D = _factors(24, n, 30, 7)
    y = X.apply_i8(X.pack_codes(f), x, out_dtype=torch.float32)
    assert X.sync_status() == X.ERR_NONFINITE
    R.check(y, *R.factors(q, s, B, C, D))


@pytest.mark.parametrize("dtype", FLOATS)
def test_quantize_strides(dtype):
    """Row distances, offsets and orders other than the plain one."""
    base = _x(20, 301, dtype, 1)
    for x in (base[:, :256], base[:, 1:258], base[::2, 3:], base[3:4, 5:], base.T, base[:, ::3],
              base[5].expand(4, 301), base.reshape(4, 5, 301), base[7]):
        r = X.quantize_rows(x)
        x2 = x.reshape(-1, x.shape[-1])
        q, s = R.rows(x2)
        assert torch.equal(r.q.double(), q) and torch.equal(r.scale.double(), s)


def test_quantize_leaves_the_padding():
    x = _x(5, 37, torch.float32, 3)
    q = torch.full((6, 48), 77, dtype=torch.int8, device="cuda")
    s = torch.full((6,), 9.0, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert X.load().externd_quantize_rows(x.data_ptr(), X.F32, 37, 5, 37, q.data_ptr(), 48,
                                          s.data_ptr(), st) == X.OK
    rq, rs = R.rows(x)
    assert torch.equal(q[:5, :37].double(), rq) and torch.equal(s[:5].double(), rs)
    assert (q[:5, 37:] == 77).all() and (q[5] == 77).all() and s[5] == 9.0


# --- the 8-bit product -------------------------------------------------------

@pytest.mark.parametrize("t", [1, 2, 7, 8, 9, 16, 17, 32, 33, 48, 64, 65, 128, 200, 257, 600])
@pytest.mark.parametrize("mn", [(1, 1), (16, 64), (33, 127), (130, 129), (257, 1000), (640, 512)])
def test_matmul_quantized(t, mn):
    m, n = mn
    x, w = _held(t, n, t + m), _held(m, n, t + n, lo=-128)
    y = X.matmul_i8(x, w)
    assert y.dtype == torch.float32
    R.check(y, *R.dense(x.q, x.scale, w.q, w.scale))


@pytest.mark.parametrize("tmn", [(1100, 2001, 300), (3000, 1500, 129), (2048, 2560, 640),
                                 (4100, 5000, 64), (40, 9729, 130), (5, 12000, 256),
                                 (600, 20000, 48)])
def test_matmul_many_tiles(tmn):
    """More tiles than the GPU holds at once: whole and ragged ones."""
    t, m, n = tmn
    x, w = _held(t, n, t + m), _held(m, n, t + n)
    bias = torch.randn(m, generator=_gen(4), device="cuda")
    R.check(X.matmul_i8(x, w, bias=bias), *R.dense(x.q, x.scale, w.q, w.scale, bias))


@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("ytype", FLOATS)
@pytest.mark.parametrize("t", [1, 20, 150, 2100])
def test_matmul_types_and_bias(xtype, ytype, t):
    m, n = 270, 333
    x, w = _x(t, n, xtype, t), _held(m, n, 3)
    bias = torch.randn(m, generator=_gen(4), device="cuda")
    q, s = R.rows(x)
    for b in (None, bias):
        y = X.matmul_i8(x, w, bias=b, out_dtype=ytype)
        assert y.dtype == ytype
        R.check(y, *R.dense(q, s, w.q, w.scale, b))
    assert X.matmul_i8(x, w).dtype == xtype


@pytest.mark.parametrize("t", [1, 3, 40, 300, 20000])
def test_matmul_largest_sums(t):
    """The longest inner dimension with every product at its largest: sums of
    both signs next to the ends of 32 bits."""
    n = X.I8_MAX_INNER
    ld = n + 1
    xq = torch.full((t, ld), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((20, ld), -128, dtype=torch.int8, device="cuda")
    wq[1::2] = 127
    x = X.Quantized(xq[:, :n], torch.ones(t, device="cuda"))
    w = X.Quantized(wq[:, :n], torch.ones(20, device="cuda"))
    y = X.matmul_i8(x, w)
    ref = torch.where(torch.arange(20, device="cuda") % 2 == 0, 16384.0 * n, -16256.0 * n)
    assert torch.equal(y, ref.float().expand(t, 20))


@pytest.mark.parametrize("t", [1, 12, 100, 520])
def test_matmul_exact_in_batches(t):
    """A row's result does not depend on the rows beside it."""
    x, w = _held(t, 700, 1), _held(300, 700, 2)
    y = X.matmul_i8(x, w)
    for i in {0, t // 2, t - 1}:
        one = X.matmul_i8(X.Quantized(x.q[i:i + 1], x.scale[i:i + 1]), w)
        assert torch.equal(one[0], y[i])
    assert torch.equal(X.matmul_i8(x, w), y)


def test_matmul_layouts():
    """8-bit operands in orders other than padded rows, batched and broadcast
    activations, an output with rows apart."""
    g = _gen(1)
    wq = torch.randint(-127, 128, (70, 50), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(70, generator=g, device="cuda")
    x = _x(30, 50, torch.float32, 2).reshape(5, 6, 50)
    q, s = R.rows(x.reshape(30, 50))
    ref, bound = R.dense(q, s, wq, ws)
    for wv in (wq, wq.T.contiguous().T, torch.cat([wq, wq], 1)[:, :50], torch.cat([wq, wq], 1)[:, 50:]):
        y = X.matmul_i8(x, X.Quantized(wv, ws))
        assert y.shape == (5, 6, 70)
        R.check(y.reshape(30, 70), ref, bound)
    y = X.matmul_i8(x[0, :1].expand(4, 50), X.Quantized(wq, ws))
    R.check(y, ref[:1].expand(4, 70), bound[:1].expand(4, 70))
    assert X.matmul_i8(x[:0], X.Quantized(wq, ws)).shape == (0, 6, 70)
    w = X.quantize_rows(_x(70, 64, torch.float32, 9))
    xq = X.quantize_rows(_x(3, 64, torch.float32, 8))
    st = torch.cuda.current_stream().cuda_stream
    for rows, t in ((3, xq), ):
        out = torch.full((rows + 1, 90), 5.0, device="cuda")
        assert X.load().externd_matmul_i8(t.q.data_ptr(), X.I8, 64, t.scale.data_ptr(),
                                          w.q.data_ptr(), 64, w.scale.data_ptr(), None, rows, 64,
                                          70, out.data_ptr(), X.F32, 90, st) == X.OK
        R.check(out[:rows, :70], *R.dense(t.q, t.scale, w.q, w.scale))
        assert (out[:, 70:] == 5).all() and (out[rows] == 5).all()


# --- the factored product ----------------------------------------------------

@pytest.mark.parametrize("mnk", [(1, 1, 1), (5, 33, 7), (31, 64, 128), (130, 257, 129),
                                 (300, 100, 515), (129, 1000, 1024)])
def test_pack_codes(mnk):
    m, n, k = mnk
    f, B, C, D = _factors(m, n, k, m + k)
    c = X.pack_codes(f)

    def decode(words, length):
        w = words.to(torch.int64) & 0xFFFFFFFF
        at = torch.arange(words.shape[1] * 16, device="cuda")
        field = (w[:, at // 16] >> (8 * (at % 4) + 6 - 2 * (at // 4 % 4))) & 3
        v = torch.where(field == 3, -1, field)
        assert (v[:, length:] == 0).all()
        return v[:, :length].double()
    assert c.codes_B.shape == (m, X.code_words(k)) and c.codes_C.shape == (k, X.code_words(n))
    assert torch.equal(decode(c.codes_B, k), B.T) and torch.equal(decode(c.codes_C, n), C)
    rho = (D.double().abs() * C.abs().sum(1).sqrt()).amax().float()
    assert float(c.bound) == float(rho)


@pytest.mark.parametrize("t", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 100, 129, 300])
@pytest.mark.parametrize("mnk", [(1, 1, 1), (16, 64, 32), (33, 127, 65), (130, 129, 300),
                                 (257, 640, 1000)])
def test_apply(t, mnk):
    m, n, k = mnk
    f, B, C, D = _factors(m, n, k, t + k)
    c = X.pack_codes(f)
    x = _x(t, n, torch.float32, t)
    q, s = R.rows(x)
    y = X.apply_i8(c, x)
    R.check(y, *R.factors(q, s, B, C, D))
    # given the quantised rows, the same bits
    assert torch.equal(X.apply_i8(c, X.quantize_rows(x)), y)


@pytest.mark.parametrize("tmnk", [(1500, 1300, 257, 2100), (2000, 2560, 128, 1111),
                                  (4096, 300, 400, 5003), (40, 9730, 130, 129),
                                  (700, 129, 1000, 9000)])
def test_apply_many_tiles(tmnk):
    t, m, n, k = tmnk
    f, B, C, D = _factors(m, n, k, t + k)
    x = _x(t, n, torch.float16, t)
    y = X.apply_i8(X.pack_codes(f), x, out_dtype=torch.float32)
    R.check(y, *R.factors(*R.rows(x), B, C, D))


@pytest.mark.parametrize("xtype", FLOATS)
@pytest.mark.parametrize("ytype", FLOATS)
@pytest.mark.parametrize("t", [1, 40, 2100])
def test_apply_types(xtype, ytype, t):
    f, B, C, D = _factors(200, 150, 333, 3)
    x = _x(t, 150, xtype, t)
    y = X.apply_i8(X.pack_codes(f), x, out_dtype=ytype)
    assert y.dtype == ytype
    R.check(y, *R.factors(*R.rows(x), B, C, D))


@pytest.mark.parametrize("t", [1, 3, 70, 30000])
def test_apply_extreme_factors(t):
    """Zero scales, empty components and rows, dense same-sign factors whose
    sums reach the bound, tiny and huge scales, D that is not finite."""
    m, n, k = 140, 256, 192
    x = _x(t, n, torch.float32, 1)
    ones = torch.ones(k, n, device="cuda")
    cases = []
    f, B, C, D = _factors(m, n, k, 5)
    cases.append((B, C, torch.zeros_like(D)))
    cases.append((torch.zeros_like(B), C, D))
    cases.append((B, torch.zeros_like(C), D))
    B2, C2 = B.clone(), C.clone()
    B2[:, ::3] = 0
    C2[::2] = 0
    cases.append((B2, C2, D))
    cases.append((torch.ones_like(B), ones.double(), D.abs()))
    cases.append((B, C, D * 2.0 ** -110))
    cases.append((B, C, D * 2.0 ** 90))
    for i, (b, c, d) in enumerate(cases):
        xi = torch.ones_like(x) * (1 + torch.arange(t, device="cuda")[:, None]) if i == 4 else x
        fac = X.Factors(R.planes(b), R.planes(c), d, None, m, n)
        y = X.apply_i8(X.pack_codes(fac), xi)
        R.check(y, *R.factors(*R.rows(xi), b, c, d))
    for bad in (float("nan"), float("inf"), -float("inf")):
        d = D.clone()
        d[3] = bad
        y = X.apply_i8(X.pack_codes(X.Factors(R.planes(B), R.planes(C), d, None, m, n)), x)
        assert torch.isnan(y).all()
    assert X.sync_status() == X.OK


@pytest.mark.parametrize("t", [1, 3, 20, 300, 6000])
def test_apply_component_ties(t):
    """Component sums that lie exactly between two steps of their scale: a
    component of 65536 ones and tokens of norm 254 make z = 2, so the odd sums
    are ties, which go to the even neighbour."""
    n, k, m = 65536, 200, 70
    C = _ternary(k, n, 1)
    C[0] = 1
    B = _ternary(k, m, 2)
    D = torch.ones(k, device="cuda")
    q = torch.zeros(t, n, dtype=torch.int8, device="cuda")
    at = torch.randint(0, n, (t, 4), generator=_gen(3), device="cuda")
    at = at // 4 * 4 + torch.arange(4, device="cuda")  # four places, never the same
    sign = torch.randint(0, 2, (t, 4), generator=_gen(4), device="cuda") * 2 - 1
    q.scatter_(1, at, (127 * sign).to(torch.int8))
    s = torch.rand(t, generator=_gen(5), device="cuda")
    f = X.Factors(R.planes(B), R.planes(C), D, None, m, n)
    h, z = R.components(q[:50].double(), C.double(), D)
    assert (z == 2).all() and bool((h % 1 == 0).all())
    y = X.apply_i8(X.pack_codes(f), X.Quantized(q, s))
    for i in range(0, t, 1000):
        R.check(y[i:i + 1000], *R.factors(q[i:i + 1000], s[i:i + 1000], B.double(), C.double(), D))


@pytest.mark.parametrize("t", [1, 4, 40, 3000])
def test_apply_largest_ranks(t):
    """The longest inner dimensions with every sum at its largest."""
    n, k, m = 40, X.I8_MAX_INNER, 9
    B, C = torch.ones(k, m, device="cuda"), torch.ones(k, n, device="cuda")
    D = torch.ones(k, device="cuda")
    q = torch.full((t, 48), 127, dtype=torch.int8, device="cuda")[:, :n]
    s = torch.ones(t, device="cuda")
    f = X.Factors(R.planes(B), R.planes(C), D, None, m, n)
    y = X.apply_i8(X.pack_codes(f), X.Quantized(q, s))
    ref, bound = R.factors(q[:1], s[:1], B.double(), C.double(), D)
    R.check(y, ref.expand(t, m), bound.expand(t, m))


@pytest.mark.parametrize("t", [1, 12, 100, 520])
def test_apply_exact_in_batches(t):
    f, *_ = _factors(300, 200, 500, 1)
    c = X.pack_codes(f)
    x = X.quantize_rows(_x(t, 200, torch.float32, 2))
    y = X.apply_i8(c, x)
    for i in {0, t // 2, t - 1}:
        one = X.apply_i8(c, X.Quantized(x.q[i:i + 1], x.scale[i:i + 1]))
        assert torch.equal(one[0], y[i])
    assert torch.equal(X.apply_i8(c, x), y)


@pytest.mark.parametrize("t", [4096, 4097, 9000])
def test_apply_long_prompts(t):
    """More tokens than one pass takes."""
    f, B, C, D = _factors(96, 64, 100, 4)
    x = _x(t, 64, torch.bfloat16, 5)
    y = X.apply_i8(X.pack_codes(f), x, out_dtype=torch.float32)
    R.check(y, *R.factors(*R.rows(x), B, C, D))


@pytest.mark.parametrize("t", [17, 40, 70, 100, 130, 170, 200, 230, 256, 257, 300, 420, 512, 700,
                               900, 1300, 1700])
@pytest.mark.parametrize("mnk", [(2560, 300, 2600), (6000, 1300, 515), (300, 2049, 9000)])
def test_apply_tile_widths(t, mnk):
    """Tiles of every width, one and several of them a pair of CTAs, over few and
    many steps."""
    m, n, k = mnk
    f, B, C, D = _factors(m, n, k, t)
    x = _x(t, n, torch.bfloat16, t + 1)
    y = X.apply_i8(X.pack_codes(f), x, out_dtype=torch.float32)
    R.check(y, *R.factors(*R.rows(x), B, C, D))


@pytest.mark.parametrize("t", [33, 48, 64, 80, 100, 128, 160, 250])
def test_apply_split_over_long_dimensions(t):
    """Many steps of codes through rings of every depth (a ring's depth follows
    the tokens), beside copies on another stream that delay their arrivals."""
    m, n, k = 512, 8192, 384
    f, B, C, D = _factors(m, n, k, t)
    f2, B2, C2, D2 = _factors(k, 512, 8192, t + 1)
    x, x2 = _x(t, n, torch.bfloat16, t), _x(t, 512, torch.bfloat16, t)
    c, c2 = X.pack_codes(f), X.pack_codes(f2)
    R.check(X.apply_i8(c, x, out_dtype=torch.float32), *R.factors(*R.rows(x), B, C, D))
    R.check(X.apply_i8(c2, x2, out_dtype=torch.float32), *R.factors(*R.rows(x2), B2, C2, D2))
    first = X.apply_i8(c, x), X.apply_i8(c2, x2)
    a, b = torch.ones(1 << 26, device="cuda"), torch.empty(1 << 26, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(40):
            b.copy_(a)
    again = [(X.apply_i8(c, x), X.apply_i8(c2, x2)) for _ in range(60)]
    torch.cuda.synchronize()
    for y, y2 in again:
        assert torch.equal(y, first[0]) and torch.equal(y2, first[1])


def test_many_rows_of_a_narrow_product():
    """More rows than one pass of the dense product quantises, and 64-bit
    offsets in the output."""
    t, n, m = 70001, 16, 8
    x, w = _x(t, n, torch.float16, 1), _held(m, n, 2)
    R.check(X.matmul_i8(x, w), *R.dense(*R.rows(x), w.q, w.scale))


def test_offsets_past_32_bits():
    """Outputs and inputs of more than 2^31 elements."""
    t, m, n = 65000, 40000, 32
    x, w = _held(t, n, 1), _held(m, n, 2)
    y = X.matmul_i8(x, w, out_dtype=torch.bfloat16)
    for i in (0, 1, 33000, 53690, 53688, t - 1):  # 53687 m is just below 2^31
        R.check(y[i:i + 1], *R.dense(x.q[i:i + 1], x.scale[i:i + 1], w.q, w.scale))
    r = X.quantize_rows(y)
    for i in (0, 53688, t - 1):
        q, s = R.rows(y[i:i + 1])
        assert torch.equal(r.q[i:i + 1].double(), q) and torch.equal(r.scale[i:i + 1].double(), s)


# --- together, streams, graphs -----------------------------------------------

@pytest.mark.parametrize("t", [1, 5, 80])
def test_decomposed_projection(t):
    """A decomposed matrix used as a user does: the 8-bit factored product
    against the fp32 one on the same dequantised rows, the quantised
    reconstruction against both."""
    m, n = 200, 168
    A = torch.from_numpy(W.llm_like(m, n, 111, n_outliers=3)).cuda()
    f = X.decompose(A, 2.0, 0.5, 3)
    x = _x(t, n, torch.float32, t)
    xq = X.quantize_rows(x)
    xh = xq.q.float() * xq.scale[:, None]
    B, C, D = R.codes(f.packed_B, m), R.codes(f.packed_C, n), f.D.double()
    y = X.apply_i8(X.pack_codes(f), xq)
    exact = (xh.double() @ C.T * D) @ B
    # each component sum is rounded to a step of z: half a step times the
    # nonzeros of B's row, and the fp32 roundings: of the sum by D (half a
    # step of |D T|), and three of the result
    q, s = xq.q.double(), xq.scale.double()
    h, z = R.components(q, C, f.D)
    terms = (q @ C.T * D).abs() @ B.abs() * s[:, None]
    bound = 0.5 * z[:, None] * s[:, None] * B.abs().sum(0) + U(terms) + 3.01 * R.U32 * y.double().abs()
    xerr = R.U32 * ((xh.double().abs() @ C.abs().T * D.abs()) @ B.abs())  # xh rounds once
    assert ((y.double() - exact).abs() <= bound + xerr).all()
    y32 = X.apply(f, xh)
    # the fp32 kernel's own bound: n + k + 1026 additions on any path
    own = 2 * (n + f.k + 1026) * R.U32 * ((xh.double().abs() @ C.abs().T * D.abs()) @ B.abs())
    assert ((y32.double() - exact).abs() <= own).all()
    w = X.quantize_rows(X.reconstruct(f))
    R.check(X.matmul_i8(xq, w), *R.dense(xq.q, xq.scale, w.q, w.scale))
    # a shorter prefix of the same factors
    c = X.pack_codes(X.truncate(f, 77))
    R.check(X.apply_i8(c, xq), *R.factors(q, s, B[:77], C[:77], f.D[:77]))


def U(v):
    return 1.01 * R.U32 * v


@pytest.mark.parametrize("t", [1, 24, 200])
def test_on_another_stream(t):
    f, B, C, D = _factors(150, 100, 200, 1)
    c = X.pack_codes(f)
    x, w = _x(t, 100, torch.float32, 2), _held(150, 100, 3)
    q, s = R.rows(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    outs = [(X.matmul_i8(x, w, stream=st), X.apply_i8(c, x, stream=st), X.quantize_rows(x, stream=st))
            for _ in range(3)]
    st.synchronize()
    for a, b, r in outs:
        R.check(a, *R.dense(q, s, w.q, w.scale))
        R.check(b, *R.factors(q, s, B, C, D))
        assert torch.equal(r.q.double(), q)


@pytest.mark.parametrize("t", [1, 24, 200])
def test_two_streams_at_once(t):
    """Calls of two streams in flight together keep their own scratch."""
    f, B, C, D = _factors(400, 300, 600, 1)
    c = X.pack_codes(f)
    xs = [_x(t, 300, torch.float32, 10 + i) for i in range(2)]
    want = [X.apply_i8(c, x) for x in xs]
    sts = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(X.apply_i8(c, xs[i], stream=sts[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])


@pytest.mark.parametrize("t", [1, 24, 200])
def test_captured_and_replayed(t):
    """Two graphs of the operators, replayed in turn with new contents."""
    f, B, C, D = _factors(150, 100, 200, 1)
    c = X.pack_codes(f)
    w = _held(150, 100, 3)
    xs = [_x(t, 100, torch.float32, 20 + i) for i in range(2)]
    for x in xs:  # (first calls set the kernels up)
        X.matmul_i8(x, w)
        X.apply_i8(c, x)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((X.matmul_i8(x, w), X.apply_i8(c, x)))
        graphs.append(g)
    for r in range(3):
        for i in (0, 1):
            xs[i].copy_(_x(t, 100, torch.float32, 30 + 2 * r + i))
        for g in graphs:
            g.replay()
        graphs[r % 2].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            q, s = R.rows(xs[i])
            R.check(outs[i][0], *R.dense(q, s, w.q, w.scale))
            R.check(outs[i][1], *R.factors(q, s, B, C, D))
    del graphs


@pytest.mark.parametrize("t", [1, 3, 24, 200, 3000])
def test_operands_written_just_before(t):
    """Weights, scales and activations written by the kernels right in front of
    a call, and results read right behind it, over and over: the kernels start
    early and have to wait for what they read."""
    m, n = 700, 1030
    g = _gen(t)
    src = [(torch.randint(-127, 128, (m, 1040), generator=g, device="cuda", dtype=torch.int8),
            torch.rand(m, generator=g, device="cuda"), _x(t, n, torch.float32, 50 + i))
           for i in range(3)]
    fs = [_factors(300, n, 900, 60 + i) for i in range(3)]
    packed = [X.pack_codes(f[0]) for f in fs]
    want = [(X.matmul_i8(x, X.Quantized(w[:, :n], s)), X.apply_i8(c, x))
            for (w, s, x), c in zip(src, packed)]
    w, s, x = (v.clone() for v in src[0])
    c = packed[0]
    live = X.FactorCodes(c.codes_B.clone(), c.codes_C.clone(), c.D.clone(), c.bound.clone(), c.m, c.n)
    torch.cuda.synchronize()
    for r in range(30):
        i = r % 3
        for to, at in zip((w, s, x), src[i]):
            to.copy_(at)
        y = X.matmul_i8(x, X.Quantized(w[:, :n], s))
        for name in ("codes_B", "codes_C", "D", "bound"):
            getattr(live, name).copy_(getattr(packed[i], name))
        z = X.apply_i8(live, x)
        xq = X.quantize_rows(x)
        y2, z2 = X.matmul_i8(xq, X.Quantized(w[:, :n], s)).clone(), X.apply_i8(live, xq).clone()
        x.zero_()
        w.zero_()
        assert torch.equal(y, want[i][0]) and torch.equal(z, want[i][1])
        assert torch.equal(y2, want[i][0]) and torch.equal(z2, want[i][1])


@pytest.mark.parametrize("t", [1, 24, 3000])
def test_captured_behind_a_join(t):
    """Captured right behind a copy, a memset and two joined streams."""
    w, x = _held(200, 100, 3), _x(t, 100, torch.float32, 1)
    f, B, C, D = _factors(150, 100, 200, 1)
    c = X.pack_codes(f)
    src = x.clone()
    X.matmul_i8(x, w)
    X.apply_i8(c, x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        x.zero_()
        with torch.cuda.stream(side):
            y0 = X.matmul_i8(src, w)
        main.wait_stream(side)
        y1 = X.matmul_i8(x, w)
        x.copy_(src)
        y2 = X.matmul_i8(x, w)
        z = X.apply_i8(c, x)
    q, s = R.rows(src)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        ref = R.dense(q, s, w.q, w.scale)
        R.check(y0, *ref)
        R.check(y2, *ref)
        assert (y1 == 0).all()
        R.check(z, *R.factors(q, s, B, C, D))


def test_first_call_captured(tmp_path):
    """A graph may hold the first calls that a process makes."""
    code = """
import torch
from expanded_rank_matrix_b200 import externd as X
from tests import int8_ref as R
x = torch.randn(%d, 256, device='cuda')
wq = torch.randint(-127, 128, (64, 256), device='cuda', dtype=torch.int8)
w = X.Quantized(wq, torch.rand(64, device='cuda'))
q, s = R.rows(x)
torch.cuda.synchronize()
f = X.Factors(torch.full((96, 2, 2), 5, dtype=torch.int32, device='cuda'),
              torch.full((96, 2, 8), 3, dtype=torch.int32, device='cuda'),
              torch.rand(96, device='cuda'), None, 64, 256)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c = X.pack_codes(f)
    y = X.matmul_i8(x, w)
    z = X.apply_i8(c, x)
g.replay()
torch.cuda.synchronize()
R.check(y, *R.dense(q, s, w.q, w.scale))
R.check(z, *R.factors(q, s, R.codes(f.packed_B, 64), R.codes(f.packed_C, 256), f.D))
print('captured')
"""
    for t in (1, 60, 3000):
        r = subprocess.run([sys.executable, "-c", code % t], cwd=ROOT, capture_output=True, text=True,
                           timeout=120)
        assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_threads_at_once():
    """Calls from two host threads, each on its own stream."""
    f, *_ = _factors(300, 200, 500, 1)
    c = X.pack_codes(f)
    xs = [_x(t, 200, torch.float32, t) for t in (1, 90)]
    want = [X.apply_i8(c, x) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(x, y):
        st = torch.cuda.Stream()
        for _ in range(50):
            got = X.apply_i8(c, x, stream=st)
            st.synchronize()
            if not torch.equal(got, y):
                bad.append(1)
    threads = [threading.Thread(target=work, args=a) for a in zip(xs, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad


def test_binding_refusals():
    w, x = _held(8, 32, 1), _x(3, 32, torch.float32, 1)
    f, *_ = _factors(8, 32, 5, 2)
    c = X.pack_codes(f)
    with pytest.raises(ValueError):
        X.quantize_rows(x.double())
    with pytest.raises(ValueError):
        X.quantize_rows(x.cpu())
    with pytest.raises(ValueError):
        X.matmul_i8(x[:, :31], w)
    with pytest.raises(ValueError):
        X.matmul_i8(x, w, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        X.matmul_i8(x, w, bias=torch.zeros(8))
    with pytest.raises(ValueError):
        X.matmul_i8(x, w, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        X.matmul_i8(x, X.Quantized(w.q, w.scale[:7]))
    with pytest.raises(ValueError):
        X.matmul_i8(x, X.Quantized(w.q.float(), w.scale))
    with pytest.raises(ValueError):
        X.apply_i8(c, x[:, :31])
    with pytest.raises(ValueError):
        X.pack_codes(X.Factors(f.packed_B, f.packed_C[:4], f.D, None, 8, 32))
    with pytest.raises(X.ExterndError):
        X.quantize_rows(torch.zeros(1, X.I8_MAX_INNER + 1, device="cuda"))
    assert X.sync_status() == X.OK
