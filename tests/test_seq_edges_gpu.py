"""Sequence operators where the ordinary inputs of the other tests do not lead: decay rates past fp32's range, states that
grow, views of one cache, calls whose sequences stay whole, many short sequences, long backward passes and ones of many states."""
import numpy as np
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from oracle import seq as ref
from test_seq_gpu import added, check_conv, check_scan, d, device, inside, joined, rand, scan_inputs, want_scan, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dwc.build()
    dwc.load_library()
    yield
    assert dwc.device_status() == 0, "a kernel reported a timed-out wait"


def parts(s):
    return [s[k] for k in ("u", "dt", "A", "B", "C")], [s[k] for k in ("D", "z", "dt_bias")]


@pytest.mark.parametrize("rate", [-float("inf"), -3e38])
@pytest.mark.parametrize("lead,C,N,offsets", [((2, 1), 8, 4, None), ((2, 17), 8, 4, None), ((3, 39), 24, 16, None), ((1, 333), 16, 8, None),
                                              ((2, 21), 16, 100, None), ((200,), 12, 5, [0, 3, 20, 36, 199])])
def test_scan_of_states_that_keep_nothing(lead, C, N, offsets, rate):
    """A of minus infinity, and a finite one that log2(e) takes past fp32: exp(delta A) is 0 at every position and its
    derivatives are, as they are of A = -1e6 (delta is 1e-3 and more, exp(-1000) is 0 in 64 bits too)."""
    rng = np.random.default_rng(N)
    count = lead[0] if offsets is None else len(offsets) - 1
    s = scan_inputs(rng, lead, C, N, 1, "f32")
    dy, h0, df = rand(rng, (*lead, C), "f32"), rand(rng, (count, C, N), "f32"), rand(rng, (count, C, N), "f32")
    plain = {**s, "A": s["A"].clone()}
    s["A"][::3, N // 2:], plain["A"][::3, N // 2:] = rate, -1e6
    off = device(offsets)
    args, rest = parts(s)
    y, last, saved = dwc.selective_scan_fwd(*args, *rest, state=h0, offsets=off, final=True, save=True)
    got = dwc.selective_scan_bwd(dy, *args, saved, *rest, offsets=off, dfinal=df, state_grad=True)
    fwd, bwd = want_scan(plain, dy, True, offsets, count, h0, df)
    within(inside(y, offsets), joined([f[0] for f in fwd], offsets), "y")
    within(last, ref.stack([f[1] for f in fwd]), "final")
    for k, t in zip(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"), got):
        rows = k in ("du", "ddt", "dB", "dC", "dz")
        within(inside(t, offsets) if rows else t, joined([f[k] for f in bwd], offsets) if rows else added([f[k] for f in bwd]), k)
    within(got[8], ref.stack([f["dstate"] for f in bwd]), "dstate")


def test_scan_step_of_states_that_keep_nothing():
    """A prompt of 16 positions and one token are a prompt of 17."""
    rng = np.random.default_rng(1)
    s = scan_inputs(rng, (3, 17), 24, 8, 1, "f32")
    s["A"][::3, 4:] = -float("inf")
    args, rest = parts(s)
    y, last = dwc.selective_scan_fwd(*args, *rest, final=True)
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    first, state = dwc.selective_scan_fwd(cut(args[0], 0, 16), cut(args[1], 0, 16), s["A"], cut(args[3], 0, 16), cut(args[4], 0, 16),
                                          rest[0], cut(rest[1], 0, 16), rest[2], final=True)
    one = dwc.selective_scan_step(s["u"][:, 16], s["dt"][:, 16], s["A"], s["B"][:, 16], s["C"][:, 16], state, s["D"], s["z"][:, 16],
                                  s["dt_bias"])
    s["A"][::3, 4:] = -1e6
    fwd, _ = want_scan(s, s["u"], True, None, 3, None, None)
    for got in (y, torch.cat((first, one[:, None]), 1)):
        within(got, ref.stack([f[0] for f in fwd]), "y")
    for got in (last, state):
        within(got, ref.stack([f[1] for f in fwd]), "final")


@pytest.mark.parametrize("T", [37, 300])
def test_scan_of_positions_that_are_left_out(T):
    """delta = 0 leaves the states alone, whatever the (finite) rate."""
    rng = np.random.default_rng(T)
    s = scan_inputs(rng, (2, T), 16, 8, 1, "f32", bias=False, plus=False)
    keep = torch.from_numpy(rng.random((2, T, 1)) < 0.5).cuda()
    s["dt"] = (s["dt"] + 0.01) * keep
    s["A"][:, 4:] = -3e38
    args, rest = parts(s)
    y, last = dwc.selective_scan_fwd(*args, *rest, False, final=True)
    s["A"][:, 4:] = -1e6
    fwd, _ = want_scan(s, s["u"], False, None, 2, None, None)
    within(y, ref.stack([f[0] for f in fwd]), "y")
    within(last, ref.stack([f[1] for f in fwd]), "final")


def test_scan_of_states_that_grow():
    """A > 0, chunks over which a state grows past fp32: one of zero stays zero, forward and backward.  (The definition runs over
    the positions behind the zeros alone, since its bounds of zero states grow as well.)"""
    rng = np.random.default_rng(2)
    T, C, N = 700, 16, 8
    s = scan_inputs(rng, (1, T), C, N, 1, "f32", plus=False, bias=False)
    s["dt"] = torch.ones_like(s["dt"])
    s["A"][:, 1:] = 3.0
    s["u"][:, :-20] = 0                # (exp(3 * 20) in the end)
    args, rest = parts(s)
    y, last = dwc.selective_scan_fwd(*args, *rest, False, final=True)
    part = lambda a, b: {k: t[:, a:b] if k in ("u", "dt", "z", "B", "C") else t for k, t in s.items()}  # noqa: E731
    fwd, _ = want_scan(part(-20, T), s["u"][:, -20:], False, None, 1, None, None)
    within(y[:, -20:], ref.stack([f[0] for f in fwd]), "y")
    within(last, ref.stack([f[1] for f in fwd]), "final")
    assert not y[:, :-20].any()
    s["u"] = torch.zeros_like(s["u"])
    args, rest = parts(s)
    dy = rand(rng, (1, T, C), "f32")
    dy[:, 20:] = 0
    _, saved = dwc.selective_scan_fwd(*args, *rest, False, save=True)
    got = dwc.selective_scan_bwd(dy, *args, saved, *rest, False)
    _, bwd = want_scan(part(0, 20), dy[:, :20], False, None, 1, None, None)
    for k, t in zip(("du", "ddt", "dB", "dC"), (got[0], got[1], got[3], got[4])):
        within(t[:, :20], ref.stack([f[k] for f in bwd]), k)
        assert not t[:, 20:].any()


def test_scan_of_large_states_that_shrink():
    """A chunk leaves less than fp32's smallest number of a state, but the state is large."""
    rng = np.random.default_rng(4)
    T, C, N = 80, 16, 8
    s = scan_inputs(rng, (1, T), C, N, 1, "f32", plus=False, bias=False)
    s["dt"], s["u"] = torch.ones_like(s["dt"]), torch.zeros_like(s["u"])
    s["A"][:, ::2] = -1.5              # exp(-1.5 * 64) = 2e-42
    h0 = rand(rng, (1, C, N), "f32") * 1e30
    args, rest = parts(s)
    y, last = dwc.selective_scan_fwd(*args, *rest, False, h0, final=True)
    # a decay's relative error in fp32 is 4 u of the exponential's and 2 u |delta A| of its argument's, a product u: 8 u a position;
    # the join's: 120 * 2 u of the sum's and the product's roundings, four times 4 u, four products: 300 u beside them
    want = h0.double() * torch.exp(s["A"].double() * T)
    assert ((last.double() - want).abs() <= (8 * T + 300) * 2 ** -24 * want.abs() + 1e-37).all()
    assert (want[:, :, ::2].abs() > 1e-24).any()


def test_scan_of_small_states_that_grow():
    """A chunk's growth is past fp32, the state that it grows is not."""
    rng = np.random.default_rng(4)
    T, C, N = 80, 16, 8
    s = scan_inputs(rng, (1, T), C, N, 1, "f32", plus=False, bias=False)
    s["dt"], s["u"] = torch.ones_like(s["dt"]), torch.zeros_like(s["u"])
    s["A"][:, ::2] = 1.6               # exp(1.6 * 64) = 3e44
    h0 = rand(rng, (1, C, N), "f32") * 1e-30
    args, rest = parts(s)
    y, last = dwc.selective_scan_fwd(*args, *rest, False, h0, final=True)
    fwd, _ = want_scan(s, s["u"], False, None, 1, h0, None)
    within(last, ref.stack([f[1] for f in fwd]), "final")
    within(y, ref.stack([f[0] for f in fwd]), "y")


# ------------------------------------------------------------------------ views of one cache

def test_steps_on_views_of_one_cache():
    """A sequence's state and its next input side by side in one row of a cache: nothing is shared, whatever the range of addresses."""
    rng = np.random.default_rng(6)
    B, K, C, N = 3, 4, 16, 8
    cache, w = rand(rng, (B, K, C), "f32"), rand(rng, (K, C), "f32")
    state, x = cache[:, :K - 1], cache[:, K - 1]
    kept, one = state.clone(), x.clone()
    want = dwc.causal_conv_step(one, kept, w, None, "silu")
    got = dwc.causal_conv_step(x, state, w, None, "silu")
    assert torch.equal(got, want) and torch.equal(state, kept) and torch.equal(x, one)
    s = scan_inputs(rng, (B, 1), C, N, 1, "f32")
    s = {k: t[:, 0] if k in ("u", "dt", "z", "B", "C") else t for k, t in s.items()}
    row = rand(rng, (B, C * N + 2 * C), "f32")
    h, u, dt = row[:, C:C + C * N].view(B, C, N), row[:, :C], row[:, C + C * N:]
    args = lambda u, dt, h: (u, dt, s["A"], s["B"], s["C"], h, s["D"], s["z"], s["dt_bias"])  # noqa: E731
    kept = h.clone()
    want = dwc.selective_scan_step(*args(u.clone(), dt.clone(), kept))
    got = dwc.selective_scan_step(*args(u, dt, h))
    assert torch.equal(got, want) and torch.equal(h, kept)
    for call in (lambda: dwc.causal_conv_step(cache[:, K - 2], state, w), lambda: dwc.causal_conv_step(cache[:, 0], state, w),
                 lambda: dwc.causal_conv_step(cache.view(B, -1)[:, 40:56], state, w),
                 lambda: dwc.selective_scan_step(*args(row[:, C - 1:2 * C - 1], dt, h)),
                 lambda: dwc.selective_scan_step(*args(u, row[:, C * N:C * N + C], h))):
        with pytest.raises(ValueError, match="overlap"):
            call()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", range(1, 17))
def test_causal_conv_step_of_every_number_of_taps(K, dtype):
    rng = np.random.default_rng(K)
    for B, C in ((3, 24), (2, 33)):
        x, w, b, state = rand(rng, (B, 3, C), dtype), rand(rng, (K, C), "f32", 0.7), rand(rng, C, "f32"), rand(rng, (B, K - 1, C), dtype)
        start = d(state)
        ys = torch.stack([dwc.causal_conv_step(x[:, t], state, w, b, "silu") for t in range(3)], 1)
        want = [ref.causal_conv(d(x[i]), d(w), d(b), "silu", start[i]) for i in range(B)]
        within(ys, ref.stack([f[0] for f in want]), "y")
        assert torch.equal(state, torch.from_numpy(np.stack([f[1] for f in want])).to(state.dtype).cuda())


# ------------------------------------------------------------------ which sequences are cut

def chunk_floats(count, length, C, N, offsets=None):
    """Floats of the forward pass's workspace: none where no sequence is cut."""
    v = dwc.Rows(1 << 16, length * C, C)
    scan = dwc.Scan(dwc.Seqs(count, length, offsets.data_ptr() if offsets is not None else None), C, N, 1, 1, 0, v, v, v, v, v, 1 << 16, None,
                    None)
    return dwc.load_library().dwc_selective_scan_fwd_workspace_size(scan) // 4


def enough(C):
    """Sequences of C channels and 16 states (blocks of 32 channels) that fill half the CTAs of the backward pass, seven to an
    SM, and so a third of the forward pass's ten."""
    return -(-7 * torch.cuda.get_device_properties(0).multi_processor_count // 2 // (C // 32)) + 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_of_sequences_that_stay_whole(dtype):
    """A batch that fills the GPU is not cut, although its sequences are longer than the shortest chunk."""
    C, N, T = 1024, 16, 70
    count = enough(C)
    assert chunk_floats(count, T, C, N) == 0 and chunk_floats(1, T, C, N) > 0
    check_scan(np.random.default_rng(1), (count, T), C, N, 1, dtype)


def test_scan_of_packed_sequences_whole_and_cut():
    """Packed sequences that fill the GPU: those past twice the mean length are cut, the others are not."""
    C, N = 1024, 16
    lengths = [40] * (enough(C) - 3) + [150, 300, 0]
    offsets = [0] + [int(o) for o in np.cumsum(lengths)]
    rows, count = offsets[-1], len(lengths)
    span = -(-2 * (rows // count) // 16) * 16
    assert 64 < span < 150
    assert chunk_floats(count, rows, C, N, device(offsets)) == (rows // span + count) * C * (N + 1)
    check_scan(np.random.default_rng(2), (rows,), C, N, 1, "f32", offsets=offsets)


@pytest.mark.parametrize("C,K,T", [(128, 4, 5), (128, 4, 32), (33, 3, 7), (64, 1, 1), (64, 12, 3)])
def test_causal_conv_of_many_short_sequences(C, K, T):
    check_conv(np.random.default_rng(C), (512, T), C, K, "bf16")


@pytest.mark.parametrize("C,N,T", [(64, 16, 3), (24, 8, 17)])
def test_scan_of_many_short_sequences(C, N, T):
    check_scan(np.random.default_rng(C), (300, T), C, N, 1, "bf16")


def test_many_short_packed_sequences():
    offsets = [int(o) for o in np.cumsum([0] + [i * i % 8 for i in range(400)])]
    check_conv(np.random.default_rng(3), (offsets[-1] + 3,), 64, 4, "bf16", offsets=offsets)
    check_scan(np.random.default_rng(3), (offsets[-1] + 3,), 32, 16, 1, "bf16", offsets=offsets)


def test_scan_backward_past_32_bits():
    """More than 2^31 elements: gradients at both ends of the sequence, the last ones from the state that was kept in front of them, the
    first ones from a part in whose rest a state is forgotten (delta A is -0.4 a position in the mean, 500 of them)."""
    C, T, N, tail, head = 4096, 530000, 2, 70, 600
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    assert x.numel() > 2 ** 31
    A = -torch.rand(C, N, device="cuda", generator=g) - 0.5
    B, Cm = (torch.randn(1, T, 1, N, device="cuda", generator=g).bfloat16() for _ in range(2))
    _, saved = dwc.selective_scan_fwd(x, x, A, B, Cm, save=True)
    at = (T - tail) // 16 * 16
    state = saved[at // 16:at // 16 + 1].clone()
    got = dwc.selective_scan_bwd(x, x, x, A, B, Cm, saved)
    names = ("du", "ddt", "dB", "dC")
    got = dict(zip(names, (got[0], got[1], got[3], got[4])))
    for a, b, keep, h in ((at, T, slice(0, T - at), state), (0, head, slice(0, 100), None)):
        s = {"u": x[:, a:b], "dt": x[:, a:b], "z": None, "A": A, "B": B[:, a:b], "C": Cm[:, a:b], "D": None, "dt_bias": None}
        _, bwd = want_scan(s, x[:, a:b], True, None, 1, h, None)
        for k in names:
            within(got[k][0, a:b][keep], bwd[0][k][keep], k)


# -------------------------------------------------- backward passes of more partial rows than fit

GRADS = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate")


def many_states(lead, G, dtype, seed):
    """4096 channels of 128 states, 512 KB of partial rows a position: 8 GB are 16384 positions.  Memories are short (delta |A| is
    0.5 and more in the mean)."""
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dtype)  # noqa: E731
    C, N = 4096, 128
    s = {"u": r(*lead, C), "dt": r(*lead, C), "z": r(*lead, C), "B": r(*lead, G, N), "C": r(*lead, G, N)}
    s["A"] = -0.5 - torch.rand(C, N, device="cuda", generator=g)
    s["D"], s["dt_bias"] = r(C).float(), torch.full((C,), 0.5, device="cuda")
    return s, r(*lead, C)


def bwd_bytes(s, offsets=None):
    """Bytes of the backward pass's workspace, and of its partial rows' bound with what the parameters take beside them."""
    u, N = s["u"], s["A"].shape[1]
    C = u.shape[-1]
    seqs = dwc.Seqs(*u.shape[:2], None) if offsets is None else dwc.Seqs(offsets.numel() - 1, u.shape[0], offsets.data_ptr())
    v = dwc.Rows(1 << 16, u.shape[-2] * C, C)
    scan = dwc.Scan(seqs, C, N, s["B"].shape[-2], 1, 1, v, v, v, v, v, 1 << 16, None, None)
    return dwc.load_library().dwc_selective_scan_bwd_workspace_size(scan), 2 ** 33


def test_scan_backward_of_a_batch_in_parts():
    """Nine sequences of which eight fit: the bits of each sequence's own call; parameters' gradients are the sums of theirs, in fp32 nine
    terms (8 roundings)."""
    s, dy = many_states((9, 2000), 1, torch.bfloat16, 1)
    need, most = bwd_bytes(s)
    assert 0.9 * most < need <= most + 9 * 4096 * 130 * 4
    args, rest = parts(s)
    _, saved = dwc.selective_scan_fwd(*args, *rest, save=True)
    got = dict(zip(GRADS, dwc.selective_scan_bwd(dy, *args, saved, *rest, state_grad=True)))
    n = saved.shape[0] // 9
    sums = {k: [] for k in ("dA", "dD", "ddt_bias")}
    for i in range(9):
        one = {k: t[i:i + 1] if k in ("u", "dt", "z", "B", "C") else t for k, t in s.items()}
        args, rest = parts(one)
        want = dict(zip(GRADS, dwc.selective_scan_bwd(dy[i:i + 1], *args, saved[i * n:(i + 1) * n], *rest, state_grad=True)))
        for k in GRADS:
            if k in sums:
                sums[k].append(want[k].double())
            else:
                assert torch.equal(got[k][i:i + 1], want[k]), (k, i)
    for k, list_ in sums.items():
        terms = torch.stack(list_)
        assert ((got[k].double() - terms.sum(0)).abs() <= 8 * 2 ** -24 * terms.abs().sum(0) + 1e-30).all(), k


def test_scan_backward_of_packed_sequences_in_parts():
    """Packed sequences of which one lies across the border, empty ones and rows beside them: the bits of each one's own call."""
    lengths = [700, 1500, 0, 1100, 900] * 4
    offsets = [5] + [5 + int(o) for o in np.cumsum(lengths)]
    s, dy = many_states((offsets[-1] + 3,), 1, torch.bfloat16, 2)
    off = device(offsets)
    need, most = bwd_bytes(s, off)
    # (and of every piece that there may be parameters' gradients, the state behind it and a sum: 2 N + 3 values a channel)
    assert 0.9 * most < need <= most + (len(lengths) + s["u"].shape[0] // 1500) * 4096 * 259 * 4
    args, rest = parts(s)
    _, saved = dwc.selective_scan_fwd(*args, *rest, offsets=off, save=True)
    got = dict(zip(GRADS, dwc.selective_scan_bwd(dy, *args, saved, *rest, offsets=off, state_grad=True)))
    sums = {k: 0 for k in ("dA", "dD", "ddt_bias")}
    size = dict(sums)
    for i, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
        if a == b:
            assert not got["dstate"][i].any()
            continue
        one = {k: t[a:b][None] if k in ("u", "dt", "z", "B", "C") else t for k, t in s.items()}
        args, rest = parts(one)
        slot = a // 16 + i
        want = dict(zip(GRADS, dwc.selective_scan_bwd(dy[a:b][None], *args, saved[slot:slot + -(-(b - a) // 16)].contiguous(), *rest,
                                                      state_grad=True)))
        for k in GRADS:
            if k in sums:
                sums[k], size[k] = sums[k] + want[k].double(), size[k] + want[k].double().abs()
            else:
                assert torch.equal(got[k][i] if k == "dstate" else got[k][a:b], want[k][0]), (k, i)
    for k in sums:
        assert ((got[k].double() - sums[k]).abs() <= len(lengths) * 2 ** -24 * size[k] + 1e-30).all(), k
    for k in ("du", "ddt", "dz", "dB", "dC"):
        assert not got[k][:5].any() and not got[k][-3:].any()


def test_scan_backward_of_one_long_sequence_in_parts():
    """A sequence that is cut for it, against a call of one group's channels, whose chunks are others: what crosses a border between
    chunks is off by at most 16 roundings for each of the some 100 positions that it is remembered for, 1e-4 of terms of which an
    output adds up 128 of either sign (their sum of magnitudes is a few times the largest output: 5e-4 of that).  The
    gradients of parameters add up 20000 such terms, which err apart."""
    s, dy = many_states((1, 20000), 64, torch.float32, 3)
    need, most = bwd_bytes(s)
    assert 0.9 * most < need <= most + 8 * 4096 * 259 * 4
    args, rest = parts(s)
    _, saved = dwc.selective_scan_fwd(*args, *rest, save=True)
    got = dict(zip(GRADS, dwc.selective_scan_bwd(dy, *args, saved, *rest, state_grad=True)))
    for group in (0, 37, 63):
        c = slice(group * 64, group * 64 + 64)
        one = {k: s[k][..., c] for k in ("u", "dt", "z", "D", "dt_bias")}
        one.update({k: s[k][:, :, group] for k in ("B", "C")}, A=s["A"][c])
        args, rest = parts(one)
        want = dict(zip(GRADS, dwc.selective_scan_bwd(dy[..., c], *args, saved[:, c].contiguous(), *rest, state_grad=True)))
        for k in GRADS:
            mine = got[k][:, :, group] if k in ("dB", "dC") else got[k][c] if k in ("dA", "dD", "ddt_bias") else \
                got[k][:, c] if k == "dstate" else got[k][..., c]
            assert (mine - want[k]).abs().max() <= 5e-4 * want[k].abs().max(), (k, group)
