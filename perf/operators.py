"""The 8-bit inference operators on real shapes: quantising rows, the 8-bit
matrix product and the 8-bit product with ternary factors.

Shapes are those of one transformer block (hidden 2560, intermediate 9728, 32
query heads and 8 key-value heads of dimension 128) and of the decompositions
of its matrices.  Definitions (all of them row by row of X, one row a token):

quantize  a_t = max_j |x_tj|, s_t = fl32(a_t / 127), q_tj = x_tj / s_t rounded
          to the nearest whole number (ties to even; 0 where s_t is 0).
matmul    y_ti = s_t v_i sum_j q_tj w_ij + b_i, w [m][n] in 8 bits with one
          scale v_i for each output channel; x comes in floating point
          (quantised within the call) or in 8 bits with its scales.
apply     y = x (B diag(D) C)^T with ternary B [m][k] and C [k][n]:
            T_tc = sum_j q_tj C_cj                (whole numbers)
            p_tc = fl32(D_c T_tc)
            rho  = fl32(max_c |D_c| sqrt(nnz C_c)),  r_t = sum_j q_tj^2
            z_t  = fl32(rho sqrt(r_t) / 32512)    (|p_tc| <= rho sqrt(r_t))
            h_tc = p_tc / z_t rounded to the nearest whole number (ties to
                   even; 0 where z_t is 0): 16 bits, which is two 8-bit planes
            y_ti = s_t z_t sum_c B_ic h_tc
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FULL = 32512  # 127 * 256: the largest 16-bit value both of whose planes are 8-bit


def listed():
    return [
        # one new token entering a projection: the smallest call
        {"name": "quantize_token", "op": "quantize", "t": 1, "n": 2560, "x": "bf16"},
        # a prompt in front of the down projection
        {"name": "quantize_prompt", "op": "quantize", "t": 8192, "n": 9728, "x": "bf16"},
        # an fp32 weight matrix, one scale for each output channel, odd sizes
        {"name": "quantize_weight", "op": "quantize", "t": 4099, "n": 2559, "x": "f32"},
        # one token through the up projection
        {"name": "matmul_token", "op": "matmul", "t": 1, "m": 9728, "n": 2560, "x": "bf16",
         "y": "bf16", "bias": False},
        # a batch of decoding sequences through the down projection, quantised before
        {"name": "matmul_batch", "op": "matmul", "t": 32, "m": 2560, "n": 9728, "x": "i8",
         "y": "bf16", "bias": False},
        # a ragged short prompt, odd sizes everywhere, with a bias, in fp32
        {"name": "matmul_ragged", "op": "matmul", "t": 333, "m": 1371, "n": 2001, "x": "f32",
         "y": "f32", "bias": True},
        # a prompt through the output projection
        {"name": "matmul_prompt", "op": "matmul", "t": 4096, "m": 2560, "n": 4096, "x": "i8",
         "y": "f16", "bias": False},
        # a long prompt through the up projection: the largest product
        {"name": "matmul_long", "op": "matmul", "t": 8192, "m": 9728, "n": 2560, "x": "bf16",
         "y": "bf16", "bias": False},
        # one token through the factors of a square projection (three times its rank)
        {"name": "apply_token", "op": "apply", "t": 1, "m": 2560, "n": 2560, "k": 7680,
         "x": "bf16", "y": "bf16"},
        # a decoding batch through the factors of the up projection (twice its rank)
        {"name": "apply_batch", "op": "apply", "t": 16, "m": 9728, "n": 2560, "k": 5120,
         "x": "f16", "y": "f16"},
        # a ragged short prompt, odd sizes, in fp32
        {"name": "apply_ragged", "op": "apply", "t": 201, "m": 1000, "n": 1533, "k": 2001,
         "x": "f32", "y": "f32"},
        # a prompt through the factors of a square projection
        {"name": "apply_prompt", "op": "apply", "t": 4096, "m": 2560, "n": 2560, "k": 7680,
         "x": "i8", "y": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantize", "matmul", "matmul", "apply", "apply"])
    top = max((work(c) for c in listed() if c["op"] == op), key=lambda w: (w["flops"], w["bytes"]))
    while True:
        c = {"op": op, "t": spread(1, 8192)}
        if op == "quantize":
            c |= {"n": spread(64, 9728), "x": rng.choice(["f32", "f16", "bf16"])}
        else:
            # half of the sizes are whole multiples of 32, the others as they come
            m, n = (spread(64, 9728) for _ in range(2))
            if rng.random() < 0.5:
                m, n = 32 * max(2, m // 32), 32 * max(2, n // 32)
            c |= {"m": m, "n": n, "x": rng.choice(["f32", "f16", "bf16", "i8"]),
                  "y": rng.choice(["f32", "f16", "bf16"])}
            if op == "matmul":
                c["bias"] = rng.random() < 0.5
            else:
                c["k"] = int(rng.uniform(1.0, 3.43) * min(m, n))
        w = work(c)
        if w["flops"] <= top["flops"] and w["bytes"] <= max(top["bytes"], 1 << 28):
            return c


def _activations(g, t, n, dtype):
    """Token rows of different loudness with a few loud channels."""
    x = torch.randn(t, n, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(t, 1, generator=g, device="cuda"))
    loud = torch.randint(0, n, (max(1, n // 400),), generator=g, device="cuda")
    x[:, loud] *= 8.0
    return x.to(dtype)


def _weights(g, m, n):
    w = 0.02 * torch.randn(m, n, generator=g, device="cuda")
    w[:, torch.randint(0, n, (max(1, n // 300),), generator=g, device="cuda")] *= 10.0
    return w


def _held(w):
    """Rows of 8-bit values as they are kept: row starts on 16-byte boundaries."""
    s = w.abs().amax(1) / 127
    q = torch.zeros(w.shape[0], (w.shape[1] + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    q[:, :w.shape[1]] = torch.round(w / s[:, None]).to(torch.int8)
    return q[:, :w.shape[1]], s


def _planes(g, k, length):
    """[k][2][ceil(length / 32)] words of ternary vectors: a mask and a sign plane;
    62 % of the entries are not 0, as at the threshold of half the rms."""
    w = (length + 31) // 32
    place = torch.arange(32, device="cuda", dtype=torch.int64)
    out = torch.empty(k, 2, w, dtype=torch.int32, device="cuda")
    mask = torch.rand(k, w * 32, generator=g, device="cuda") < 0.62
    mask[:, length:] = False
    sign = (torch.rand(k, w * 32, generator=g, device="cuda") < 0.5) & mask
    for p, bits in enumerate((mask, sign)):
        v = (bits.view(k, w, 32).to(torch.int64) << place).sum(2)
        out[:, p] = torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    x = _activations(g, c["t"], c["n"], TYPES.get(c["x"], torch.float32))
    if c["x"] == "i8":
        s["x"], s["sx"] = _held(x)
    else:
        s["x"] = x
    if c["op"] == "matmul":
        s["w"], s["sw"] = _held(_weights(g, c["m"], c["n"]))
        s["bias"] = torch.randn(c["m"], generator=g, device="cuda") if c["bias"] else None
    if c["op"] == "apply":
        k = c["k"]
        s["B"], s["C"] = _planes(g, k, c["m"]), _planes(g, k, c["n"])
        # greedy components come largest first, with a spread around the trend
        trend = 0.02 * torch.arange(1, k + 1, device="cuda").float() ** -0.5
        s["D"] = trend * torch.exp(0.2 * torch.randn(k, generator=g, device="cuda"))
    if own:
        from expanded_rank_matrix_b200 import externd as X
        s["X"] = X
        if c["x"] == "i8":
            s["x"] = X.Quantized(s["x"], s["sx"])
        if c["op"] == "matmul":
            s["w"] = X.Quantized(s["w"], s["sw"])
        if c["op"] == "apply":
            f = X.Factors(s["B"], s["C"], s["D"], None, c["m"], c["n"])
            s["codes"] = X.pack_codes(f)
    return s


def run(s):
    c = s["case"]
    if own:
        X = s["X"]
        if c["op"] == "quantize":
            r = X.quantize_rows(s["x"])
            return {"q": r.q, "scale": r.scale}
        if c["op"] == "matmul":
            return {"y": X.matmul_i8(s["x"], s["w"], bias=s["bias"], out_dtype=TYPES[c["y"]])}
        return {"y": X.apply_i8(s["codes"], s["x"], out_dtype=TYPES[c["y"]])}
    if c["op"] == "quantize":
        q, scale = _plain_rows(s["x"])
        return {"q": q.to(torch.int8), "scale": scale}
    q, scale = (s["x"].float(), s["sx"]) if c["x"] == "i8" else _plain_rows(s["x"])
    if c["op"] == "matmul":
        y = scale[:, None] * ((q @ s["w"].float().T) * s["sw"])
        if s["bias"] is not None:
            y = y + s["bias"]
    else:
        y = _plain_apply(q, scale, s["B"], s["C"], s["D"], c["m"], c["n"])
    return {"y": y.to(TYPES[c["y"]])}


def _plain_rows(x):
    """Whole numbers (as floats) and scales; 64 bits where a value may lie next to a border."""
    x = x.double()
    scale = (x.abs().amax(1) / 127).float()
    d = scale.double()[:, None]
    return torch.where(d > 0, torch.round(x / d), 0.0).float(), scale


def _codes(planes, length):
    """Bit planes -> entries -1, 0, +1 as floats [k][length]."""
    place = torch.arange(32, dtype=torch.int32, device=planes.device)
    bits = (planes[..., None] >> place) & 1
    v = bits[:, 0] * (1 - 2 * bits[:, 1])
    return v.reshape(planes.shape[0], -1)[:, :length].float()


def _plain_apply(q, scale, B, C, D, m, n):
    C, B = _codes(C, n), _codes(B, m)
    # whole numbers below 2^24 at every step, so 32 bits are exact in both products
    p = D * (q @ C.T)
    d = D.double()
    rho = (d.abs() * C.abs().sum(1).double().sqrt()).amax().float().double()
    full = torch.full((), float(FULL), dtype=torch.float64, device=q.device)
    z = (rho * q.double().square().sum(1).sqrt() / full).float()
    zd = z.double()[:, None]
    h = torch.where(zd > 0, torch.round(p.double() / zd), 0.0)
    hi = torch.floor((h + 128) / 256)
    total = 256.0 * (hi.float() @ B).double() + ((h - 256 * hi).float() @ B).double()
    return scale[:, None] * (z[:, None] * total.float())


def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}
    t, n = c["t"], c["n"]
    x = t * n * size[c["x"]] + (4 * t if c["x"] == "i8" else 0)
    if c["op"] == "quantize":
        return {"bytes": x + t * n + 4 * t, "flops": 3 * t * n}
    m = c["m"]
    y = t * m * size[c["y"]]
    if c["op"] == "matmul":
        return {"bytes": x + y + m * n + 4 * m * (2 if c["bias"] else 1), "flops": 2 * t * m * n}
    k = c["k"]
    # two bits an entry, and the scales
    return {"bytes": x + y + k * (m + n) // 4 + 4 * k, "flops": 2 * t * k * (m + n)}


def _exact_rows(x):
    peak = torch.linalg.vector_norm(x.double(), ord=float("inf"), dim=1)
    scale = torch.div(peak, torch.full_like(peak, 127.0)).to(torch.float32).to(torch.float64)
    safe = torch.where(scale == 0, torch.ones_like(scale), scale)
    return torch.div(x.double(), safe.unsqueeze(1)).round(), scale


def _exact_ternary(planes, length):
    words = planes.to(torch.int64) & 0xFFFFFFFF
    at = torch.arange(length, device=planes.device)
    mask, sign = ((words[:, p][:, at // 32] >> (at % 32)) & 1 for p in (0, 1))
    return (mask - 2 * (mask & sign)).double()


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["x"] == "i8":
        q, scale = s["x"].double(), s["sx"].double()
    else:
        q, scale = _exact_rows(s["x"])
    if c["op"] == "quantize":
        return {"q": q.to(torch.int8), "scale": scale}
    if c["op"] == "matmul":
        w = s["w"].double().mul_(s["sw"].double().unsqueeze(1))
        y = torch.einsum("tj,ij->ti", q.mul_(scale.unsqueeze(1)), w)
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    B, C = _exact_ternary(s["B"], c["m"]), _exact_ternary(s["C"], c["n"])
    D = s["D"].double()
    # the definition's one rounding of each component sum to 32 bits
    p = (torch.einsum("tj,cj->tc", q, C) * D).to(torch.float32).double()
    rho = torch.sqrt(C.pow(2).sum(1)).mul(D.abs()).max().to(torch.float32).double()
    z = torch.div(rho * torch.sqrt(q.pow(2).sum(1)), torch.tensor(float(FULL), device=q.device)
                  .double()).to(torch.float32).double()
    h = torch.div(p, torch.where(z == 0, torch.ones_like(z), z).unsqueeze(1)).round()
    h = h * (z != 0).unsqueeze(1)
    return {"y": torch.einsum("tc,ci->ti", h.mul_((scale * z).unsqueeze(1)), B)}
