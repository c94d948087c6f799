"""Cases, plain forms and 64-bit definitions of the sequence operators and of the block norm.

Three families over channels-last rows (positions x C):

  causal conv     depthwise filter of K taps that looks back along the positions of a sequence:
                  y[t,c] = act(bias[c] + sum_k w[k,c] * x[t-K+1+k,c]), act the identity or SiLU; the
                  K - 1 inputs before a sequence's first position are its state (zero if not given).
  selective scan  per-channel recurrence with N states and a decay that depends on the input:
                  delta = softplus(dt + dt_bias), h_t = exp(delta A) h_{t-1} + delta u B_t,
                  y_t = (C_t . h_t + D u) * silu(z); B and C are shared by the channels of a group.
  block norm      the norms on either side of a residual connection, with a gate and residual scales:
                  z = alpha res + scale * act(gate) * rms_norm(x) * gamma_post,
                  y = rms_norm(z) * gamma_pre.

Each has its backward pass; the first two also a step for one token with the state updated in
place.  Sequences are a batch (B x T x C) or packed one behind the other (L x C with the offsets of
their first rows; some are empty).

`run` computes these with elementary torch operations in fp32 (`own` false) or through the
framework's entry points (`own` true).
"""
import math
import random

import torch

own = False

EPS = 1e-5
ALPHA = 0.9
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
OPS = ("conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_train", "scan_step", "norm_fwd", "norm_bwd")

# The most a drawn case takes: channels x positions, the same times the states (a scan's plain form
# holds several fp32 tensors of that size), and rows x channels of a norm.
MOST_CONV = 8 * 2048 * 4096
MOST_SCAN = 8 * 2048 * 4096 * 16
MOST_NORM = 16384 * 4096


def _conv(name, op, B, T, C, K, dtype, act="silu", packed=False, state=False):
    """B sequences of T positions; packed: B sequences that have B * T positions together."""
    return {"name": name, "op": op, "B": B, "T": T, "C": C, "K": K, "dtype": dtype, "act": act,
            "packed": packed, "state": state}


def _scan(name, op, B, T, C, N, G, dtype, packed=False, state=False, gate=True):
    return {"name": name, "op": op, "B": B, "T": T, "C": C, "N": N, "G": G, "dtype": dtype,
            "packed": packed, "state": state, "gate": gate}


def _norm(name, op, rows, C, dtype, wide, gate="silu", serve=False):
    """dtype: of x, the gate and y.  wide: of the residual stream.  serve: no backward pass follows."""
    return {"name": name, "op": op, "rows": rows, "C": C, "dtype": dtype, "wide": wide, "gate": gate,
            "serve": serve}


def listed():
    return [
        # a training batch: 8 sequences of 2048 tokens, inner width 4096
        _conv("conv_fwd_8x2048x4096_k4_bf16", "conv_fwd", 8, 2048, 4096, 4, "bf16"),
        _conv("conv_bwd_8x2048x4096_k4_bf16", "conv_bwd", 8, 2048, 4096, 4, "bf16"),
        # packed sequences of ragged lengths that go on from earlier parts, odd channel count
        _conv("conv_bwd_packed_7x715x1001_k3_f32", "conv_bwd", 7, 715, 1001, 3, "f32", packed=True, state=True),
        # one token for each of 64 sequences in decoding
        _conv("conv_step_64x4096_k4_bf16", "conv_step", 64, 1, 4096, 4, "bf16"),
        # one long prompt, its final state kept for decoding
        _scan("scan_fwd_1x16384x2048x16_bf16", "scan_fwd", 1, 16384, 2048, 16, 1, "bf16", state=True),
        # a training step of the batch above, forward and backward
        _scan("scan_train_8x2048x4096x16_bf16", "scan_train", 8, 2048, 4096, 16, 1, "bf16"),
        # packed ragged sequences in fp32, two groups, an odd number of states
        _scan("scan_train_packed_5x601x1002x11_f32", "scan_train", 5, 601, 1002, 11, 2, "f32", packed=True),
        # decoding: one token for each of 64 sequences
        _scan("scan_step_64x4096x16_bf16", "scan_step", 64, 1, 4096, 16, 1, "bf16"),
        # one token of a model of width 4096 in decoding: latency alone
        _norm("norm_fwd_1x4096_bf16", "norm_fwd", 1, 4096, "bf16", "bf16", "none", serve=True),
        # a training step over 16384 tokens, fp32 residual stream, 16-bit branches
        _norm("norm_fwd_16384x4096_bf16_f32", "norm_fwd", 16384, 4096, "bf16", "f32"),
        _norm("norm_bwd_16384x4096_bf16_f32", "norm_bwd", 16384, 4096, "bf16", "f32"),
        # a ragged batch with a channel count that no vector divides
        _norm("norm_bwd_4099x1001_f16", "norm_bwd", 4099, 1001, "f16", "f16", "sigmoid"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """A case of the same ranges: 1 to 64 sequences, 1 to 16384 positions, 32 to 8192 channels, 1 to
    64 states; 1 to 16384 rows and 32 to 16384 channels of a norm; every operator and type."""
    op = rng.choice(OPS)
    dtype = rng.choice(("f32", "bf16", "f16"))
    while True:
        C = _spread(rng, 32, 16384 if op.startswith("norm") else 8192)
        if rng.random() < 0.6:
            C = max(32, C // 32 * 32)
        if op.startswith("norm"):
            rows = _spread(rng, 1, 16384)
            case = _norm("", op, rows, C, dtype, rng.choice((dtype, "f32")), rng.choice(("none", "sigmoid", "silu")),
                         serve=op == "norm_fwd" and rows <= 256)
            fits = rows * C <= MOST_NORM
        else:
            step = op.endswith("step")
            B, T = _spread(rng, 1, 256 if step else 64), 1 if step else _spread(rng, 1, 16384)
            packed, state = not step and rng.random() < 0.4, not step and rng.random() < 0.4
            if op.startswith("conv"):
                case = _conv("", op, B, T, C, rng.choice((2, 3, 4, 4, 5, 8)), dtype, rng.choice(("silu", "none")),
                             packed, state)
                fits = B * T * C <= MOST_CONV
            else:
                G = rng.choice((1, 1, 2, 4))
                C = C // G * G
                N = rng.choice((16, 16, 8, 32, 64, rng.randint(1, 40)))
                case = _scan("", op, B, T, C, N, G, dtype, packed, state, gate=rng.random() < 0.7)
                fits = B * T * C * N <= MOST_SCAN and B * T <= 65536
        del case["name"]
        if fits:
            return case


def work(case):
    """Every input read once, every output written once; operations a value cannot do without (an
    exponential, a quotient or a root counts as one)."""
    op = case["op"]
    e = BYTES[case["dtype"]]
    if op.startswith("norm"):
        n, w, C = case["rows"] * case["C"], BYTES[case["wide"]], case["C"]
        gate, stats = case["gate"] != "none", 0 if case["serve"] else 8 * case["rows"]
        if op == "norm_fwd":
            return {"bytes": n * ((2 + gate) * e + 2 * w) + 12 * C + stats, "flops": (10 + 5 * gate) * n}
        return {"bytes": n * ((3 + 2 * gate) * e + 3 * w) + 24 * C + stats, "flops": (28 + 12 * gate) * n}
    B, T, C = case["B"], case["T"], case["C"]
    n = B * T * C
    if op.startswith("conv"):
        K, silu = case["K"], case["act"] == "silu"
        kept = B * (K - 1) * C * e
        par = (K + 1) * C * 4
        if op == "conv_step":
            return {"bytes": 2 * n * e + 2 * kept + par, "flops": (2 * K + 4 * silu) * n}
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + (2 * kept if case["state"] else 0) + par, "flops": (2 * K + 4 * silu) * n}
        return {"bytes": 3 * n * e + (2 * kept if case["state"] else 0) + 2 * par,
                "flops": (4 * K + 1 + silu * (2 * K + 8)) * n}
    N, G, gate = case["N"], case["G"], case["gate"]
    bc = 2 * B * T * G * N * e
    par = C * (N + 2) * 4
    held = B * C * N * 4
    if op == "scan_step":
        return {"bytes": (3 + gate) * n * e + bc + 2 * held + par, "flops": (7 * N + 6 + 5 * gate) * n}
    if op == "scan_fwd":
        return {"bytes": (3 + gate) * n * e + bc + (2 * held if case["state"] else held) + par,
                "flops": (7 * N + 6 + 5 * gate) * n}
    # forward and backward: u, dt, z, dy, B, C in, y and their gradients out
    return {"bytes": (6 + 2 * gate) * n * e + 2 * bc + (2 * held if case["state"] else 0) + 2 * par,
            "flops": (21 * N + 16 + 14 * gate) * n}


# ------------------------------------------------------------------------------ inputs

def _offsets(case, seed):
    """First rows of the packed sequences: random cuts, so lengths differ widely; the second of three
    or more is empty, the third has one position where that many are left."""
    B, total = case["B"], case["B"] * case["T"]
    r = random.Random(int(seed) * 7919 + 17)
    cuts = sorted(r.randint(0, total) for _ in range(B - 1))
    at = [0] + cuts + [total]
    if B >= 3:
        at[2] = at[1]
        at[3] = min(max(at[3], at[2] + 1), total) if B > 3 else total
        at = [max(at[:i + 1]) for i in range(B + 1)]
    return at


def prepare(case, seed):
    op, C = case["op"], case["C"]
    dt = TYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {"case": case}
    if op.startswith("norm"):
        rows, wide = case["rows"], TYPES[case["wide"]]
        s["gamma_post"], s["gamma_pre"] = 1 + 0.2 * rand(C), 1 + 0.2 * rand(C)
        s["scale"] = 0.3 + 0.1 * rand(C)
        s["x"] = (rand(rows, C) * torch.exp(0.4 * rand(C)) * 2).to(dt)
        s["gate"] = rand(rows, C).to(dt) if case["gate"] != "none" else None
        stream = rand(rows, C) * torch.exp(0.4 * rand(C)) + 0.3 * rand(C)
        if op == "norm_fwd":
            s["res"] = stream.to(wide)
        else:
            # what the forward pass kept: the sum and the two statistics
            s["z"] = stream.to(wide)
            s["rstd_post"] = torch.rsqrt(s["x"].float().square().mean(-1) + EPS)
            s["rstd_pre"] = torch.rsqrt(s["z"].float().square().mean(-1) + EPS)
            s["dy"], s["dz"] = (0.05 * rand(rows, C)).to(dt), (0.05 * rand(rows, C)).to(wide)
        if case["serve"]:
            # a serving loop writes into buffers that it keeps
            s["y"] = torch.empty((rows, C), device="cuda", dtype=dt)
            s["sum"] = torch.empty((rows, C), device="cuda", dtype=wide)
        return s
    B, T = case["B"], case["T"]
    step = op.endswith("step")
    lead = (B,) if step else (B * T,) if case["packed"] else (B, T)
    s["offsets"] = None
    if case["packed"]:
        s["bounds"] = _offsets(case, seed)
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda")
    if op.startswith("conv"):
        K = case["K"]
        s["w"], s["bias"] = rand(K, C) / math.sqrt(K), 0.2 * rand(C)
        s["x"] = rand(*lead, C).to(dt)
        s["state"] = rand(B, K - 1, C).to(dt) if case["state"] or step else None
        if op == "conv_bwd":
            s["dy"] = (0.1 * rand(*lead, C)).to(dt)
        if step:
            s["y"] = torch.empty((B, C), device="cuda", dtype=dt)
        return s
    N, G = case["N"], case["G"]
    # decays and steps as such layers are initialised: A near -1 .. -N, delta between 0.001 and 0.1
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * rand(C, N))
    start = torch.exp(torch.rand(C, generator=g, device="cuda") * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = start + torch.log(-torch.expm1(-start))
    s["D"] = 1 + 0.1 * rand(C)
    s["u"], s["dt"] = rand(*lead, C).to(dt), (0.5 * rand(*lead, C)).to(dt)
    s["B"], s["C"] = rand(*lead, G, N).to(dt), rand(*lead, G, N).to(dt)
    s["z"] = rand(*lead, C).to(dt) if case["gate"] else None
    s["state"] = 0.5 * rand(B, C, N) if case["state"] or step else None
    if op == "scan_train":
        s["dy"] = (0.1 * rand(*lead, C)).to(dt)
    if step:
        s["y"] = torch.empty((B, C), device="cuda", dtype=dt)
    return s


# -------------------------------------------------------------------------- plain form

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(x, kind):
    return x if kind == "none" else _sigmoid(x) if kind == "sigmoid" else x * _sigmoid(x)


def _act_slope(x, kind):
    if kind == "none":
        return torch.ones_like(x)
    p = _sigmoid(x)
    return p * (1 - p) if kind == "sigmoid" else p * (1 + x * (1 - p))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _sequence_of(s, total):
    """Of every packed row its sequence, and whether it is the sequence's first one."""
    at = s["offsets"].long()
    row = torch.arange(total, device="cuda")
    seq = torch.searchsorted(at[1:].contiguous(), row, right=True)
    return seq, row == at[seq]


def _with_state(s, x, K):
    """x with each sequence's K - 1 earlier rows in front of it, and the place of every row of x in it."""
    case, C = s["case"], x.shape[-1]
    B = case["B"]
    state = s["state"].float() if s["state"] is not None else x.new_zeros(B, K - 1, C)
    if not case["packed"]:
        return torch.cat((state, x), 1), None
    seq, _ = _sequence_of(s, x.shape[0])
    place = torch.arange(x.shape[0], device="cuda") + (seq + 1) * (K - 1)
    first = s["offsets"][:-1].long() + torch.arange(B, device="cuda") * (K - 1)
    ext = x.new_zeros(x.shape[0] + B * (K - 1), C)
    ext[(first[:, None] + torch.arange(K - 1, device="cuda")).reshape(-1)] = state.reshape(-1, C)
    ext[place] = x
    return ext, place


def _tap(ext, place, T, j):
    """The rows j positions back (dense: T rows of each sequence; packed: at `place`)."""
    if place is not None:
        return ext[place - j]
    return ext[:, ext.shape[1] - T - j:ext.shape[1] - j]


def _last_rows(s, ext, K):
    """The K - 1 last rows of each sequence with its state in front."""
    if not s["case"]["packed"]:
        return ext[:, ext.shape[1] - (K - 1):]
    end = s["offsets"][1:].long() + torch.arange(1, s["case"]["B"] + 1, device="cuda") * (K - 1)
    return ext[end[:, None] - (K - 1) + torch.arange(K - 1, device="cuda")]


def _plain_conv(s):
    case = s["case"]
    K, T, dt, kind = case["K"], case["T"], TYPES[case["dtype"]], case["act"]
    w, x = s["w"], s["x"].float()
    if case["op"] == "conv_step":
        rows = torch.cat((s["state"].float(), x[:, None]), 1)
        s["state"].copy_(rows[:, 1:])
        return {"y": _act((rows * w).sum(1) + s["bias"], kind).to(dt), "state": s["state"]}
    ext, place = _with_state(s, x, K)
    pre = s["bias"] + sum(w[k] * _tap(ext, place, T, K - 1 - k) for k in range(K))
    if case["op"] == "conv_fwd":
        y = _act(pre, kind).to(dt)
        return {"y": y, "final": _last_rows(s, ext, K).to(dt)} if case["state"] else {"y": y}
    dpre = s["dy"].float() * _act_slope(pre, kind)
    every = tuple(range(dpre.dim() - 1))
    dw = torch.stack([(dpre * _tap(ext, place, T, K - 1 - k)).sum(every) for k in range(K)])
    dext = torch.zeros_like(ext)
    for k in range(K):
        if place is not None:
            dext[place - (K - 1 - k)] += w[k] * dpre
        else:
            dext[:, k:k + T] += w[k] * dpre
    out = {"dx": (dext[place] if place is not None else dext[:, K - 1:]).to(dt), "dw": dw, "dbias": dpre.sum(every)}
    if case["state"]:
        first = s["offsets"][:-1].long() + torch.arange(case["B"], device="cuda") * (K - 1) if place is not None else None
        ahead = dext[first[:, None] + torch.arange(K - 1, device="cuda")] if place is not None else dext[:, :K - 1]
        out["dstate"] = ahead.to(dt)
    return out


def _prefix(a, b, reverse=False):
    """h_t = a_t h_{t-1} + b_t along axis 1 by doubling (the other way round: h_t = a_t h_{t+1} + b_t)."""
    T, step = a.shape[1], 1
    while step < T:
        here, there = (slice(0, T - step), slice(step, T)) if reverse else (slice(step, T), slice(0, T - step))
        rest = slice(T - step, T) if reverse else slice(0, step)
        h, p = b[:, here] + a[:, here] * b[:, there], a[:, here] * a[:, there]
        b, a = ((torch.cat((h, b[:, rest]), 1), torch.cat((p, a[:, rest]), 1)) if reverse else
                (torch.cat((b[:, rest], h), 1), torch.cat((a[:, rest], p), 1)))
        step *= 2
    return b


def _plain_scan(s):
    case = s["case"]
    op, C, N, G, dt, packed = case["op"], case["C"], case["N"], case["G"], TYPES[case["dtype"]], case["packed"]
    step = op == "scan_step"

    def rows(t):
        """sequences x positions x groups x channels of a group x 1, in fp32"""
        t = t.float()[:, None] if step else t.float()[None] if packed else t.float()
        return t.reshape(t.shape[0], t.shape[1], G, C // G, 1)

    def states(t):
        t = t.float()[:, None] if step else t.float()[None] if packed else t.float()
        return t.reshape(t.shape[0], t.shape[1], G, 1, N)

    def back(t, like):
        return t.reshape(like.shape).to(like.dtype)

    A, D = s["A"].reshape(G, C // G, N), s["D"].reshape(G, C // G, 1)
    u, raw = rows(s["u"]), rows(s["dt"]) + s["dt_bias"].reshape(G, C // G, 1)
    Bm, Cm = states(s["B"]), states(s["C"])
    delta = _softplus(raw)
    a = torch.exp(delta * A)
    b = delta * u * Bm
    h0 = s["state"].reshape(-1, G, C // G, N) if s["state"] is not None else None
    if packed:
        seq, first = _sequence_of(s, u.shape[1])
        if h0 is not None:
            b[0, first] += a[0, first] * h0[seq[first]]
        a[0, first] = 0
    elif h0 is not None:
        b[:, 0] += a[:, 0] * h0
    h = _prefix(a, b)
    y = (h * Cm).sum(-1, keepdim=True) + D * u
    z = rows(s["z"]) if case["gate"] else None
    out = {"y": back(y * _act(z, "silu") if case["gate"] else y, s["u"])}
    if step:
        s["state"].copy_(h[:, 0].reshape(s["state"].shape))
        return {**out, "state": s["state"]}
    if op == "scan_fwd":
        if packed:
            at = s["offsets"].long()
            last = h[0, (at[1:] - 1).clamp(min=0)]
            none = h0 if h0 is not None else torch.zeros_like(last)
            last = torch.where((at[1:] > at[:-1])[:, None, None, None], last, none)
        else:
            last = h[:, -1]
        return {**out, "final": last.reshape(-1, C, N)}
    g = rows(s["dy"])
    if case["gate"]:
        out["dz"] = back(g * y * _act_slope(z, "silu"), s["z"])
        g = g * _act(z, "silu")
    # h_t reaches h_{t+1} through a_{t+1}
    ahead = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)
    dh = _prefix(ahead, g * Cm, reverse=True)
    del ahead
    ph = h - delta * u * Bm          # a_t h_{t-1}, with a sequence's first state
    dh_ph = dh * ph
    dpre = (dh * Bm).sum(-1, keepdim=True)
    ddelta = (dh_ph * A).sum(-1, keepdim=True) + dpre * u
    draw_ = ddelta * _sigmoid(raw)
    out.update(du=back(dpre * delta + D * g, s["u"]), ddt=back(draw_, s["dt"]), dA=(dh_ph * delta).sum((0, 1)).reshape(C, N),
               dB=back((dh * (delta * u)).sum(3), s["B"]), dC=back((h * g).sum(3), s["C"]),
               dD=(g * u).sum((0, 1)).reshape(C), ddt_bias=draw_.sum((0, 1)).reshape(C))
    if h0 is not None:
        if packed:
            at = s["offsets"].long()
            lead = at[:-1].clamp(max=u.shape[1] - 1)
            decay = torch.exp(delta[0, lead] * A)
            dstate = torch.where((at[1:] > at[:-1])[:, None, None, None], dh[0, lead] * decay, torch.zeros_like(h0))
        else:
            dstate = dh[:, 0] * a[:, 0]
        out["dstate"] = dstate.reshape(-1, C, N)
    return out


def _plain_norm(s):
    case = s["case"]
    dt, wide, kind = TYPES[case["dtype"]], TYPES[case["wide"]], case["gate"]
    x = s["x"].float()
    if case["op"] == "norm_fwd":
        rstd_post = torch.rsqrt((x * x).mean(-1) + EPS)
        m = x * rstd_post[:, None] * s["gamma_post"]
        if s["gate"] is not None:
            m = m * _act(s["gate"].float(), kind)
        z = ALPHA * s["res"].float() + s["scale"] * m
        rstd_pre = torch.rsqrt((z * z).mean(-1) + EPS)
        out = {"y": (z * rstd_pre[:, None] * s["gamma_pre"]).to(dt), "z": z.to(wide)}
        return out if case["serve"] else {**out, "rstd_post": rstd_post, "rstd_pre": rstd_pre}
    dy, zhat = s["dy"].float(), s["z"].float() * s["rstd_pre"][:, None]
    a = dy * s["gamma_pre"]
    dz = s["dz"].float() + s["rstd_pre"][:, None] * (a - zhat * (a * zhat).mean(-1, keepdim=True))
    xhat = x * s["rstd_post"][:, None]
    n = xhat * s["gamma_post"]
    gate = _act(s["gate"].float(), kind) if s["gate"] is not None else 1.0
    dm = s["scale"] * dz
    dn = dm * gate
    b = dn * s["gamma_post"]
    dx = s["rstd_post"][:, None] * (b - xhat * (b * xhat).mean(-1, keepdim=True))
    out = {"dx": dx.to(dt), "dres": (ALPHA * dz).to(wide), "dgamma_post": (dn * xhat).sum(0),
           "dgamma_pre": (dy * zhat).sum(0), "dscale": (dz * n * gate).sum(0)}
    if s["gate"] is not None:
        out["dgate"] = (dm * n * _act_slope(s["gate"].float(), kind)).to(dt)
    return out


def _plain(s):
    op = s["case"]["op"]
    return _plain_conv(s) if op.startswith("conv") else _plain_scan(s) if op.startswith("scan") else _plain_norm(s)


# --------------------------------------------------------------------- framework's form

def _framework(s):
    import depthwise_convolution_nhwc_gb300 as dwc
    case = s["case"]
    op = case["op"]
    if op == "conv_fwd":
        r = dwc.causal_conv_fwd(s["x"], s["w"], s["bias"], case["act"], s["state"], s["offsets"], final=case["state"])
        return {"y": r[0], "final": r[1]} if case["state"] else {"y": r}
    if op == "conv_bwd":
        dx, dw, dbias, dstate = dwc.causal_conv_bwd(s["dy"], s["x"], s["w"], s["bias"], case["act"], s["state"], s["offsets"])
        out = {"dx": dx, "dw": dw, "dbias": dbias}
        return {**out, "dstate": dstate} if case["state"] else out
    if op == "conv_step":
        y = dwc.causal_conv_step(s["x"], s["state"], s["w"], s["bias"], case["act"], out=s["y"])
        return {"y": y, "state": s["state"]}
    if op == "scan_step":
        y = dwc.selective_scan_step(s["u"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["D"], s["z"], s["dt_bias"],
                                    out=s["y"])
        return {"y": y, "state": s["state"]}
    if op == "scan_fwd":
        y, last = dwc.selective_scan_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                                         state=s["state"], offsets=s["offsets"], final=True)
        return {"y": y, "final": last}
    if op == "scan_train":
        y, saved = dwc.selective_scan_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                                          state=s["state"], offsets=s["offsets"], save=True)
        du, ddt, dA, dB, dC, dD, dz, ddt_bias, dstate = dwc.selective_scan_bwd(
            s["dy"], s["u"], s["dt"], s["A"], s["B"], s["C"], saved, s["D"], s["z"], s["dt_bias"], offsets=s["offsets"],
            state_grad=case["state"])
        out = {"y": y, "du": du, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": dD, "ddt_bias": ddt_bias}
        if case["gate"]:
            out["dz"] = dz
        return {**out, "dstate": dstate} if case["state"] else out
    if op == "norm_fwd":
        if case["serve"]:
            y, z = dwc.block_norm_fwd(s["x"], s["res"], s["gamma_post"], s["gamma_pre"], s["gate"], s["scale"], ALPHA,
                                      case["gate"], EPS, out=s["y"], z=s["sum"])
            return {"y": y, "z": z}
        y, z, rstd_post, rstd_pre = dwc.block_norm_fwd(s["x"], s["res"], s["gamma_post"], s["gamma_pre"], s["gate"],
                                                       s["scale"], ALPHA, case["gate"], EPS, stats=True)
        return {"y": y, "z": z, "rstd_post": rstd_post, "rstd_pre": rstd_pre}
    dx, dres, dgate, dgamma_post, dgamma_pre, dscale = dwc.block_norm_bwd(
        s["dy"], s["x"], s["z"], s["rstd_post"], s["rstd_pre"], s["gamma_post"], s["gamma_pre"], s["gate"], s["scale"],
        ALPHA, case["gate"], s["dz"])
    out = {"dx": dx, "dres": dres, "dgamma_post": dgamma_post, "dgamma_pre": dgamma_pre, "dscale": dscale}
    return out if s["gate"] is None else {**out, "dgate": dgate}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ 64-bit definition

def _silu64(v, slope=False):
    q = torch.sigmoid(v)
    return q + v * q * (1 - q) if slope else v * q


def _pieces(s, case):
    """(rows of the flattened positions, sequence) of each sequence."""
    at = s["bounds"] if case["packed"] else [i * case["T"] for i in range(case["B"] + 1)]
    return [(slice(at[i], at[i + 1]), i) for i in range(case["B"])]


def _exact_conv(s, case):
    C, K, silu = case["C"], case["K"], case["act"] == "silu"
    w, bias = s["w"].double(), s["bias"].double()
    lead = s["x"].shape
    x = s["x"].double().reshape(-1, C)
    dy = s["dy"].double().reshape(-1, C) if "dy" in s else None
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, dbias = torch.zeros_like(w), torch.zeros_like(bias)
    kept = []
    for rows, i in _pieces(s, case):
        past = s["state"][i].double() if s["state"] is not None else x.new_zeros(K - 1, C)
        line = torch.cat((past, x[rows]))
        n = line.shape[0] - (K - 1)
        windows = line.unfold(0, K, 1) if n > 0 else line.new_zeros(0, C, K)
        pre = torch.einsum("tck,kc->tc", windows, w) + bias
        if dy is None:
            y[rows] = _silu64(pre) if silu else pre
            kept.append(line[n:])
            continue
        d = dy[rows] * _silu64(pre, True) if silu else dy[rows]
        dw += torch.einsum("tc,tck->kc", d, windows)
        dbias += d.sum(0)
        back = torch.zeros_like(line)
        for t in range(K):
            back[t:t + n] += d * w[t]
        dx[rows] = back[K - 1:]
        kept.append(back[:K - 1])
    if case["op"] == "conv_step":
        return {"y": y.reshape(lead), "state": torch.stack(kept)}
    if dy is None:
        return {"y": y.reshape(lead), "final": torch.stack(kept)} if case["state"] else {"y": y.reshape(lead)}
    out = {"dx": dx.reshape(lead), "dw": dw, "dbias": dbias}
    return {**out, "dstate": torch.stack(kept)} if case["state"] else out


def _exact_scan(s, case):
    """Position by position; a batch side by side, packed sequences one after another."""
    B, C, N, G, packed, step = case["B"], case["C"], case["N"], case["G"], case["packed"], case["op"] == "scan_step"
    per = C // G
    one = lambda v: v.double()[:, None] if step else v.double()[None] if packed else v.double()  # noqa: E731
    u, x = one(s["u"]), one(s["dt"]) + s["dt_bias"].double()
    delta = torch.where(x > 40, x, torch.log1p(torch.exp(x.clamp(max=40))))
    A, D = s["A"].double(), s["D"].double()
    wide = lambda v, t: v[:, t].double().repeat_interleave(per, dim=1)  # noqa: E731
    Bm, Cm = ((v[:, None] if step else v[None] if packed else v) for v in (s["B"], s["C"]))
    rows, length = u.shape[0], u.shape[1]
    at = s["bounds"] if packed else []
    begin = {at[i]: i for i in range(len(at) - 1) if at[i + 1] > at[i]}     # first position: sequence
    init = s["state"].double() if s["state"] is not None else torch.zeros(B, C, N, device="cuda", dtype=torch.float64)
    train = case["op"] == "scan_train"
    last = init.clone()
    h = None if packed else init
    y = torch.empty_like(u)
    past = torch.empty((length, rows, C, N), device="cuda", dtype=torch.float64) if train else None
    seq = None
    for t in range(length):
        if packed and t in begin:
            seq = begin[t]
            h = init[seq:seq + 1]
        if train:
            past[t] = h
        h = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * u[:, t])[..., None] * wide(Bm, t)
        y[:, t] = torch.einsum("bcn,bcn->bc", h, wide(Cm, t)) + D * u[:, t]
        if packed and not train and (t + 1 == length or t + 1 in begin):
            last[seq] = h[0]
    gate = one(s["z"]) if case["gate"] else None
    out = {"y": (y * _silu64(gate) if case["gate"] else y).reshape(s["u"].shape)}
    if step:
        return {**out, "state": h}
    if not train:
        return {**out, "final": last if packed else h}
    g = one(s["dy"])
    if case["gate"]:
        out["dz"] = (g * y * _silu64(gate, True)).reshape(s["z"].shape)
        g = g * _silu64(gate)
    du, dx, dA = torch.empty_like(u), torch.empty_like(u), torch.zeros_like(A)
    dB, dC = (torch.empty((rows, length, G, N), device="cuda", dtype=torch.float64) for _ in range(2))
    dstate = torch.zeros_like(init)
    carry = torch.zeros((rows, C, N), device="cuda", dtype=torch.float64)
    ends = {i - 1 for i in at}
    for t in range(length - 1, -1, -1):
        if packed and t in ends:
            carry = torch.zeros_like(carry)
        dt_, in_ = delta[:, t, :, None], (delta[:, t] * u[:, t])[..., None]
        decay = torch.exp(dt_ * A)
        held = decay * past[t]
        dh = carry + g[:, t, :, None] * wide(Cm, t)
        dC[:, t] = ((held + in_ * wide(Bm, t)) * g[:, t, :, None]).reshape(rows, G, per, N).sum(2)
        dB[:, t] = (dh * in_).reshape(rows, G, per, N).sum(2)
        into = torch.einsum("bcn,bcn->bc", dh, wide(Bm, t))
        du[:, t] = into * delta[:, t] + D * g[:, t]
        dx[:, t] = into * u[:, t] + (dh * held * A).sum(-1)
        dA += (dh * held * dt_).sum(0)
        carry = dh * decay
        if packed and t in begin:
            dstate[begin[t]] = carry[0]
    dx *= torch.sigmoid(x)
    out.update(du=du.reshape(s["u"].shape), ddt=dx.reshape(s["dt"].shape), dA=dA, dB=dB.reshape(s["B"].shape),
               dC=dC.reshape(s["C"].shape), dD=(g * u).sum((0, 1)), ddt_bias=dx.sum((0, 1)))
    return {**out, "dstate": dstate if packed else carry} if case["state"] else out


def _exact_norm(s, case):
    v = {k: t.double() for k, t in s.items() if isinstance(t, torch.Tensor)}
    C, kind = case["C"], case["gate"]
    q = torch.sigmoid(v["gate"]) if kind != "none" else None
    gate = 1.0 if kind == "none" else q if kind == "sigmoid" else q * v["gate"]
    if case["op"] == "norm_fwd":
        post = 1 / torch.sqrt(torch.linalg.vector_norm(v["x"], dim=1) ** 2 / C + EPS)
        z = ALPHA * v["res"] + v["scale"] * gate * v["gamma_post"] * post[:, None] * v["x"]
        pre = 1 / torch.sqrt(torch.linalg.vector_norm(z, dim=1) ** 2 / C + EPS)
        out = {"y": pre[:, None] * z * v["gamma_pre"], "z": z}
        return out if case["serve"] else {**out, "rstd_post": post, "rstd_pre": pre}
    pre, post = v["rstd_pre"][:, None], v["rstd_post"][:, None]

    def back(d, t, r):
        return r * d - t * r ** 3 * torch.einsum("rc,rc->r", d, t)[:, None] / C

    dz = v["dz"] + back(v["dy"] * v["gamma_pre"], v["z"], pre)
    unit = post * v["x"]
    out = {"dres": ALPHA * dz, "dgamma_pre": torch.einsum("rc,rc->c", v["dy"], pre * v["z"]),
           "dscale": (dz * gate * unit).sum(0) * v["gamma_post"],
           "dgamma_post": (dz * gate * unit).sum(0) * v["scale"],
           "dx": back(dz * v["scale"] * gate * v["gamma_post"], v["x"], post)}
    if kind != "none":
        slope = q * (1 - q) if kind == "sigmoid" else q + v["gate"] * q * (1 - q)
        out["dgate"] = dz * v["scale"] * unit * v["gamma_post"] * slope
    return out


def exact(case, seed):
    """The definition in 64 bits on the values that `prepare` drew."""
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_conv(s, case) if op.startswith("conv") else _exact_scan(s, case) if op.startswith("scan") else
            _exact_norm(s, case))
