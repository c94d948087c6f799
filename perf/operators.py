"""Cases, plain forms and 64-bit definitions of the normalisation and dropout operators.

Three operators over rows of C channels (the last axis of a channels-last tensor):

  layer norm      y = (x - mean) * rstd * gamma + beta, mean and rstd = 1/sqrt(var + eps) of the
                  row; backward: dx, dgamma, dbeta.
  dropout         y = keep ? x / (1 - q) : 0, keep from a counter-based generator; q is p
                  rounded to a multiple of 2^-16, so that the expected value is kept exactly.
  add layer norm  z = res + dropout(x), y = layer_norm(z): the end of one residual branch and
                  the norm in front of the next; backward: dx, dres, dgamma, dbeta.

The generator is Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
easy as 1, 2, 3", 2011): element i of the tensor in row-major order takes the 16-bit value
i % 8 (of each word the low half first) of the block with the 128-bit counter (i // 8, offset)
and the 64-bit key seed, and is kept where that value is at least q * 2^16.

`run` computes these with elementary torch operations in fp32 (`own` false) or through the
framework's entry points (`own` true).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
OPS = ("ln_fwd", "ln_bwd", "dropout_fwd", "dropout_bwd", "add_ln_fwd", "add_ln_bwd")

# The most a drawn case moves or draws: no more than the largest listed case of its operator.
MOST_BYTES = 1.0e9
MOST_RANDOM = 6.0e7


def _case(name, op, rows, C, dtype, wide, p=0.0, serve=False):
    """dtype: of x (add layer norm), dy and y.  wide: of the stream (layer norm's x and dx; the
    residual, its sum and their gradients).  serve: no backward pass follows, so no statistics."""
    return {"name": name, "op": op, "rows": rows, "C": C, "dtype": dtype, "wide": wide, "p": p,
            "serve": serve}


def listed():
    return [
        # one token of a model of width 4096 in decoding: latency alone
        _case("ln_fwd_1x4096_bf16", "ln_fwd", 1, 4096, "bf16", "bf16", serve=True),
        # the norm behind the fp32 output of the depthwise layer of a 64x56x56x128 stage
        _case("ln_fwd_200704x128_f32", "ln_fwd", 64 * 56 * 56, 128, "f32", "f32"),
        # the same behind a 64x28x28x256 stage, written as the 16-bit input of the next product
        _case("ln_fwd_50176x256_f32_bf16", "ln_fwd", 64 * 28 * 28, 256, "bf16", "f32"),
        # its gradient in a 16-bit training step of the 64x56x56x128 stage
        _case("ln_bwd_200704x128_bf16", "ln_bwd", 64 * 56 * 56, 128, "bf16", "bf16"),
        # a batch of tokens of a wide model in training
        _case("ln_bwd_8192x4096_bf16", "ln_bwd", 8192, 4096, "bf16", "bf16"),
        # a ragged batch with a channel count that no vector divides
        _case("ln_bwd_4099x1001_f16", "ln_bwd", 4099, 1001, "f16", "f16"),
        # dropout of a feed-forward layer's hidden activations (a batch of 8192 tokens)
        _case("dropout_fwd_8192x8192_bf16", "dropout_fwd", 8192, 8192, "bf16", "bf16", p=0.1),
        # a small ragged activation
        _case("dropout_bwd_1009x991_f32", "dropout_bwd", 1009, 991, "f32", "f32", p=0.5),
        # 32 sequences in decoding, 16-bit residual stream, no dropout
        _case("add_ln_fwd_32x8192_bf16", "add_ln_fwd", 32, 8192, "bf16", "bf16", serve=True),
        # a training step over 16384 tokens, fp32 residual stream, 16-bit branches
        _case("add_ln_fwd_16384x4096_bf16_f32", "add_ln_fwd", 16384, 4096, "bf16", "f32", p=0.1),
        _case("add_ln_bwd_16384x4096_bf16_f32", "add_ln_bwd", 16384, 4096, "bf16", "f32", p=0.1),
        # the last stage (64x7x7x1024) of a depthwise network trained with dropout on its branches
        _case("add_ln_bwd_3136x1024_f32", "add_ln_bwd", 64 * 7 * 7, 1024, "f32", "f32", p=0.2),
    ]


def draw(rng):
    """A case of the same ranges: 1 to 200704 rows, 32 to 16384 channels, every operator, type
    and residual type."""
    op = rng.choice(OPS)
    dtype = rng.choice(("f32", "bf16", "f16"))
    wide = dtype if op.startswith("dropout") else rng.choice((dtype, "f32"))
    dropout = op.startswith("dropout")
    p = 0.0
    if dropout or (op.startswith("add") and rng.random() < 0.7):
        p = rng.choice((0.1, 0.2, 0.5, round(rng.uniform(0.01, 0.9), 3)))
    while True:
        C = int(round(math.exp(rng.uniform(math.log(32), math.log(16384)))))
        if rng.random() < 0.7:
            C = max(32, C // 32 * 32)
        rows = int(round(math.exp(rng.uniform(0, math.log(200704)))))
        case = _case("", op, rows, C, dtype, wide, p, serve=op.endswith("fwd") and rows <= 256)
        del case["name"]
        if (C != 3072 and work(case)["bytes"] <= MOST_BYTES
                and (p == 0.0 or rows * C <= MOST_RANDOM)):
            return case


def work(case):
    """Every input read once, every output written once; operations a value cannot do without
    (sums, differences, products; a draw of the generator is 10 rounds of 2 products and 4
    exclusive-ors for 8 values)."""
    op, rows, C = case["op"], case["rows"], case["C"]
    n, e, w = rows * C, BYTES[case["dtype"]], BYTES[case["wide"]]
    rng = 7.5 * n if case["p"] else 0
    stats = 0 if case["serve"] else 8 * rows
    if op == "ln_fwd":
        return {"bytes": n * (w + e) + 8 * C + stats, "flops": 8 * n}
    if op == "ln_bwd":
        return {"bytes": n * (e + 2 * w) + 8 * rows + 12 * C, "flops": 14 * n}
    if op.startswith("dropout"):
        return {"bytes": 2 * n * e, "flops": n + rng}
    if op == "add_ln_fwd":
        return {"bytes": n * (2 * e + 2 * w) + 8 * C + stats, "flops": 10 * n + rng}
    return {"bytes": n * (2 * e + 3 * w) + 8 * rows + 12 * C, "flops": 16 * n + rng}


def prepare(case, seed):
    op, rows, C = case["op"], case["rows"], case["C"]
    dt, wide = TYPES[case["dtype"]], TYPES[case["wide"]]
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {"case": case, "seed": (int(seed) * 0x9E3779B97F4A7C15 + 12345) % 2 ** 63,
         "offset": int(seed) % 1000}
    if op.startswith("dropout"):
        s["x"] = rand(rows, C).to(dt)
        return s
    s["gamma"], s["beta"] = 1 + 0.2 * rand(C), 0.1 * rand(C)
    # channels with their own means and spreads, a few of them far larger than the rest
    centre, spread = 0.5 * rand(C) + 0.3, torch.exp(0.4 * rand(C))
    spread[rand(C) > 2.6] *= 12
    h = rand(rows, C).mul_(spread).add_(centre).to(wide)
    if op == "ln_fwd":
        s["x"] = h
    elif op == "add_ln_fwd":
        s["res"], s["x"] = h, (0.5 * rand(rows, C)).to(dt)
    else:
        # what the forward pass kept: the normalised tensor and its statistics
        f = h.float()
        s["mean"] = f.mean(-1)
        s["rstd"] = torch.rsqrt(f.var(-1, unbiased=False) + EPS)
        s["z"], s["dy"] = h, (0.05 * rand(rows, C)).to(dt)
        if op == "add_ln_bwd":
            s["dz"] = (0.05 * rand(rows, C)).to(wide)
    if case["serve"]:
        # a serving loop writes into buffers that it keeps
        s["y"] = torch.empty((rows, C), device="cuda", dtype=dt)
        s["sum"] = torch.empty((rows, C), device="cuda", dtype=wide)
    return s


# ------------------------------------------------------------------------- plain form

def _philox(groups, seed, offset):
    """The 16-bit values of the blocks with counters (0..groups-1, offset): groups x 8 of int64."""
    m32 = 0xFFFFFFFF
    i = torch.arange(groups, device="cuda", dtype=torch.int64)
    c0, c1 = i & m32, i >> 32
    c2, c3 = torch.full_like(i, offset & m32), torch.full_like(i, offset >> 32)
    k0, k1 = seed & m32, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57   # 64-bit products, their low bits wrap exactly
        c0, c1, c2, c3 = (((b >> 32) & m32) ^ c1 ^ k0, b & m32,
                          ((a >> 32) & m32) ^ c3 ^ k1, a & m32)
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    words = torch.stack((c0, c1, c2, c3), 1)
    return torch.stack((words & 0xFFFF, words >> 16), 2)


def _dropout(x, p, seed, offset):
    if p == 0.0:
        return x
    n = x.numel()
    values = _philox((n + 7) // 8, seed, offset).reshape(-1)[:n].reshape(x.shape)
    dropped = math.floor(p * 65536 + 0.5)
    return torch.where(values >= dropped, x * (65536 / (65536 - dropped)), torch.zeros_like(x))


def _norm(x, gamma, beta):
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    return d * rstd * gamma + beta, mean.squeeze(-1), rstd.squeeze(-1)


def _norm_grad(dy, x, mean, rstd, gamma):
    xhat = (x - mean.unsqueeze(-1)) * rstd.unsqueeze(-1)
    dg = dy * gamma
    dx = (dg - dg.mean(-1, keepdim=True)
          - xhat * (dg * xhat).mean(-1, keepdim=True)) * rstd.unsqueeze(-1)
    return dx, (dy * xhat).sum(0), dy.sum(0)


def _plain(s):
    case = s["case"]
    op, p, dt, wide = case["op"], case["p"], TYPES[case["dtype"]], TYPES[case["wide"]]
    if op.startswith("dropout"):
        return {"y": _dropout(s["x"].float(), p, s["seed"], s["offset"]).to(dt)}
    if op == "ln_fwd":
        y, mean, rstd = _norm(s["x"].float(), s["gamma"], s["beta"])
        return {"y": y.to(dt)} if case["serve"] else {"y": y.to(dt), "mean": mean, "rstd": rstd}
    if op == "add_ln_fwd":
        z = s["res"].float() + _dropout(s["x"].float(), p, s["seed"], s["offset"])
        y, mean, rstd = _norm(z, s["gamma"], s["beta"])
        out = {"y": y.to(dt), "z": z.to(wide)}
        return out if case["serve"] else {**out, "mean": mean, "rstd": rstd}
    dx, dgamma, dbeta = _norm_grad(s["dy"].float(), s["z"].float(), s["mean"], s["rstd"],
                                   s["gamma"])
    if op == "ln_bwd":
        return {"dx": dx.to(wide), "dgamma": dgamma, "dbeta": dbeta}
    dres = s["dz"].float() + dx
    return {"dx": _dropout(dres, p, s["seed"], s["offset"]).to(dt), "dres": dres.to(wide),
            "dgamma": dgamma, "dbeta": dbeta}


# --------------------------------------------------------------------- framework's form

def _framework(s):
    import depthwise_convolution_nhwc_gb300 as dwc
    case = s["case"]
    op, p = case["op"], case["p"]
    if op == "dropout_fwd":
        return {"y": dwc.dropout_fwd(s["x"], p, s["seed"], s["offset"])}
    if op == "dropout_bwd":
        return {"y": dwc.dropout_bwd(s["x"], p, s["seed"], s["offset"])}
    if op == "ln_fwd":
        if case["serve"]:
            return {"y": dwc.layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS, out=s["y"])}
        y, mean, rstd = dwc.layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS,
                                           out_dtype=TYPES[case["dtype"]], stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx, dgamma, dbeta = dwc.layer_norm_bwd(s["dy"], s["z"], s["mean"], s["rstd"], s["gamma"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "add_ln_fwd":
        if case["serve"]:
            y, z = dwc.add_layer_norm_fwd(s["x"], s["res"], s["gamma"], s["beta"], EPS, p,
                                          s["seed"], s["offset"], out=s["y"], z=s["sum"])
            return {"y": y, "z": z}
        y, z, mean, rstd = dwc.add_layer_norm_fwd(s["x"], s["res"], s["gamma"], s["beta"], EPS, p,
                                                  s["seed"], s["offset"], stats=True)
        return {"y": y, "z": z, "mean": mean, "rstd": rstd}
    dx, dres, dgamma, dbeta = dwc.add_layer_norm_bwd(s["dy"], s["z"], s["mean"], s["rstd"],
                                                     s["gamma"], s["dz"], p, s["seed"],
                                                     s["offset"])
    return {"dx": dx, "dres": dres, "dgamma": dgamma, "dbeta": dbeta}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ 64-bit definition

def _kept(first, count, p, seed, offset):
    """Which of the elements first .. first+count-1 are kept (numpy, 64-bit integers)."""
    g0, g1 = first // 8, (first + count + 7) // 8
    m, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    block = np.arange(g0, g1, dtype=np.uint64)
    x = [block & m, block >> sh, np.full_like(block, offset & 0xFFFFFFFF),
         np.full_like(block, offset >> 32)]
    for r in range(10):
        k0 = np.uint64((seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32)
        k1 = np.uint64((seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32)
        u, v = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(v >> sh) ^ x[1] ^ k0, v & m, (u >> sh) ^ x[3] ^ k1, u & m]
    halves = np.stack(x, -1).astype("<u4").view("<u2").reshape(-1)
    at = first - 8 * g0
    return halves[at:at + count] >= round(p * 2 ** 16)


def exact(case, seed):
    """The definition in 64 bits on the values that `prepare` drew, some rows at a time."""
    s = prepare(case, seed)
    op, rows, C, p = case["op"], case["rows"], case["C"], case["p"]
    host = {k: v.double().cpu().numpy() for k, v in s.items()
            if isinstance(v, torch.Tensor) and v.dim() == 1}
    step = max(1, (1 << 18) // C)
    parts, sums = {}, {}

    def put(name, value):
        parts.setdefault(name, []).append(value)

    def add(name, value):
        sums[name] = sums.get(name, 0.0) + value.sum(0)

    big = {k: v.cpu() for k, v in s.items() if k in ("x", "res", "z", "dy", "dz")}
    for r in range(0, rows, step):
        t = {k: v[r:r + step].double().numpy() for k, v in big.items()}
        n = min(step, rows - r)

        def drop(v):
            if p == 0.0:
                return v
            keep = _kept(r * C, n * C, p, s["seed"], s["offset"]).reshape(n, C)
            return np.where(keep, v / (1.0 - round(p * 2 ** 16) / 2 ** 16), 0.0)

        if op.startswith("dropout"):
            put("y", drop(t["x"]))
        elif op.endswith("ln_fwd"):
            v = t["x"] if op == "ln_fwd" else t["res"] + drop(t["x"])
            mu = np.mean(v, axis=1)
            sigma = np.sqrt(np.var(v, axis=1) + EPS)
            put("y", (v - mu[:, None]) / sigma[:, None] * host["gamma"] + host["beta"])
            if op == "add_ln_fwd":
                put("z", v)
            if not case["serve"]:
                put("mean", mu)
                put("rstd", 1.0 / sigma)
        else:
            rs = host["rstd"][r:r + n, None]
            unit = (t["z"] - host["mean"][r:r + n, None]) * rs
            add("dbeta", t["dy"])
            add("dgamma", t["dy"] * unit)
            a = t["dy"] * host["gamma"]
            along = np.einsum("ij,ij->i", a, unit)[:, None] / C
            grad = rs * (a - np.mean(a, axis=1, keepdims=True) - along * unit)
            if op == "ln_bwd":
                put("dx", grad)
            else:
                grad = grad + t["dz"]
                put("dres", grad)
                put("dx", drop(grad))
    return {**{k: np.concatenate(v) for k, v in parts.items()}, **sums}
