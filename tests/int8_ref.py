"""Plain 64-bit forms of the 8-bit inference operators, from their formulas,
and the error bounds of the fp32 arithmetic around their exact sums."""
import torch

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half the spacing of the subnormals
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def rows(x):
    """(q, scale) as fp64, scale already rounded to fp32; rows that are not
    finite have q = 0 and scale NaN."""
    x = x.double()
    finite = torch.isfinite(x).all(1)
    a = torch.where(finite[:, None], x.abs(), 0.0).amax(1)
    s = (a / torch.full_like(a, 127.0)).float().double()
    safe = torch.where(s > 0, s, 1.0)
    q = torch.where((finite & (s > 0))[:, None], torch.round(x / safe[:, None]), 0.0)
    q = q.clamp(-127, 127)
    return q, torch.where(finite, s, float("nan"))


def codes(planes, length):
    w = planes.to(torch.int64) & 0xFFFFFFFF
    at = torch.arange(length, device=planes.device)
    mask, sign = ((w[:, p][:, at // 32] >> (at % 32)) & 1 for p in (0, 1))
    return (mask * (1 - 2 * sign)).double()


def planes(codes_):
    """int codes [k][length] -> packed planes [k][2][words] (int32)."""
    k, length = codes_.shape
    w = (length + 31) // 32
    full = torch.zeros(k, w * 32, dtype=torch.int64, device=codes_.device)
    full[:, :length] = codes_.to(torch.int64)
    place = torch.arange(32, device=codes_.device)
    out = [((b.view(k, w, 32).to(torch.int64)) << place).sum(2) for b in (full != 0, full < 0)]
    v = torch.stack(out, 1)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32).contiguous()


def dense(q, s, wq, ws, bias=None):
    """y and the bound of |y_kernel - y| before the output rounding: the whole
    sum rounds once to fp32, then twice more with the scales (3 half steps of
    the product; the second-order terms are far below one), and once more when
    the bias is added (half a step of the result)."""
    p = (q.double() @ wq.double().T) * s.double()[:, None] * ws.double()
    y = p if bias is None else p + bias.double()
    return y, 3.01 * U32 * p.abs() + (0.0 if bias is None else U32 * y.abs() * 1.01)


def components(q, C, D):
    """(h, z): 16-bit component sums and their scale, from the definition."""
    p = (D.double() * (q.double() @ C.T)).float().double()
    rho = (D.double().abs() * C.abs().sum(1).sqrt()).amax().float().double()
    z = (rho * q.double().square().sum(1).sqrt() / torch.full((), 32512.0, dtype=torch.float64,
                                                              device=q.device)).float().double()
    safe = torch.where(z > 0, z, 1.0)[:, None]
    return torch.where(z[:, None] > 0, torch.round(p / safe), 0.0), z


def factors(q, s, B, C, D):
    """y and the bound before the output rounding (three fp32 roundings)."""
    h, z = components(q, C, D)
    y = (h @ B) * z[:, None] * s.double()[:, None]
    return y, 3.01 * U32 * y.abs()


def check(y, ref, bound):
    """y within the bound and half a step of its type (and of its subnormals);
    not-a-numbers where the reference has them."""
    assert y.shape == ref.shape
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(y), nan)
    top = torch.finfo(y.dtype).max
    got = y.double()
    half, tiny = HALF_STEP[y.dtype], TINY[y.dtype]
    # fp32 intermediates may be subnormal too
    allowed = bound * (1 + half) + half * ref.abs() * 1.0001 + tiny + 2.0 ** -148
    over = ref.abs() > top  # rounds to infinity (or to the largest value)
    bad = ((got - ref).abs() > allowed) & ~nan & ~over
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() / allowed)[~nan & ~over].max()))
