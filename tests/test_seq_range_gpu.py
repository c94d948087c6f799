"""Sequence operators at the ends of their ranges: no positions or sequences, tensors past 2^31 elements, sequences of
chunks (few long ones, packed ones of very different length), states carried through them, updates in place."""
import numpy as np
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from oracle import seq as ref
from test_seq_gpu import check_norm, check_scan, d, rand, scan_inputs, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dwc.build()
    dwc.load_library()
    yield
    assert dwc.device_status() == 0, "a kernel reported a timed-out wait"


@pytest.mark.parametrize("B,T", [(0, 5), (3, 0), (0, 0)])
def test_nothing_to_do(B, T):
    """No positions: states pass through, gradients of parameters are zero."""
    rng = np.random.default_rng(0)
    C, N = 16, 8
    x, w, b = rand(rng, (B, T, C), "f32"), rand(rng, (4, C), "f32"), rand(rng, C, "f32")
    st, h = rand(rng, (B, 3, C), "f32"), rand(rng, (B, C, N), "f32")
    y, last = dwc.causal_conv_fwd(x, w, b, "silu", st, final=True)
    assert y.shape == x.shape and torch.equal(last, st)
    dx, dw, db, ds = dwc.causal_conv_bwd(x, x, w, b, "silu", st, dfinal=st)
    assert dx.shape == x.shape and not dw.any() and not db.any() and torch.equal(ds, st)
    s = scan_inputs(rng, (B, T), C, N, 1, "f32")
    args, rest = [s[k] for k in ("u", "dt", "A", "B", "C")], [s[k] for k in ("D", "z", "dt_bias")]
    y, last, saved = dwc.selective_scan_fwd(*args, *rest, state=h, final=True, save=True)
    assert y.shape == x.shape and torch.equal(last, h)
    g = dwc.selective_scan_bwd(x, *args, saved, *rest, dfinal=h, state_grad=True)
    assert torch.equal(g[8], h) and not g[2].any() and not g[5].any() and not g[7].any()
    if T == 0:
        none = x.reshape(0, C)
        off = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        y, last = dwc.causal_conv_fwd(none, w, b, "silu", st, off, final=True)
        assert torch.equal(last, st)
    one = rand(rng, (0, C), "f32")
    assert dwc.causal_conv_step(one, st[:0], w).shape == one.shape


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lead,C,N,offsets", [((1, 700), 32, 16, None), ((2, 1031), 24, 8, None), ((1, 400), 8, 100, None),
                                              ((900,), 20, 11, [0, 3, 700, 700, 899]), ((640,), 16, 16, [1, 640])])
def test_scan_in_chunks(lead, C, N, offsets, dtype):
    """Few sequences, which the passes cut into chunks of 64 positions and more."""
    check_scan(np.random.default_rng(C), lead, C, N, 1, dtype, offsets=offsets)


def test_scan_in_chunks_of_groups_and_without_options():
    check_scan(np.random.default_rng(5), (1, 333), 12, 5, 3, "f32", gate=False, skip=False, bias=False, plus=False, state=False,
               dfinal=False)


def test_many_sequences_stay_whole():
    """Enough CTAs without chunks, lengths that differ (batch and packed)."""
    check_scan(np.random.default_rng(1), (70, 40), 128, 4, 1, "f32")
    offsets = list(np.cumsum([0] + [7 * (i % 9) for i in range(80)]))
    check_scan(np.random.default_rng(2), (int(offsets[-1]),), 256, 4, 1, "f32", offsets=[int(o) for o in offsets])


def test_gradients_match_differences():
    """The kernels' gradients against central differences of the kernels' forward pass in one direction.  The loss is a sum of
    n = 2 * 40 * 8 products of fp32 values, each off by about e = 1e-6 (bounds of the forward tests): with a step of h = 1e-2
    along a unit direction the rounding is at most n^0.5 e |dy y| / h = 2.5e-3 |..| of the loss' scale 1, the truncation
    h^2 times a third derivative of order 10."""
    rng = np.random.default_rng(3)
    s = scan_inputs(rng, (2, 40), 8, 4, 1, "f32")
    dy = rand(rng, (2, 40, 8), "f32")
    names = ("u", "dt", "A", "B", "C", "D", "z", "dt_bias")
    out = lambda t: dwc.selective_scan_fwd(*(t[k] for k in names))  # noqa: E731
    _, saved = dwc.selective_scan_fwd(*(s[k] for k in names), save=True)
    got = dwc.selective_scan_bwd(dy, *(s[k] for k in names[:5]), saved, *(s[k] for k in names[5:]))
    grads = dict(zip(("u", "dt", "A", "B", "C", "D", "z", "dt_bias"), (got[0], got[1], got[2], got[3], got[4], got[5], got[6], got[7])))
    h = 1e-2
    for k in names:
        v = rand(rng, s[k].shape, "f32")
        v /= v.norm()
        side = [(out({**s, k: s[k] + sign * h * v}).double() * dy.double()).sum() for sign in (1, -1)]
        want, g = float(side[0] - side[1]) / (2 * h), float((grads[k].double() * v.double()).sum())
        assert abs(want - g) <= 1e-2 * max(1.0, abs(g)), (k, want, g)


def test_past_32_bits():
    """More than 2^31 elements: the last positions' values are those of a call of their own from the states before them."""
    C, T, tail = 4096, 530000, 70
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    assert x.numel() > 2 ** 31
    w = torch.randn(4, C, device="cuda", generator=g)
    y, last = dwc.causal_conv_fwd(x, w, None, "silu", final=True)
    part = dwc.causal_conv_fwd(x[:, -tail - 3:], w, None, "silu")
    assert torch.equal(y[:, -tail:], part[:, 3:]) and torch.equal(last, x[:, -3:])
    dx, dw, _, _ = dwc.causal_conv_bwd(x, x, w, None, "silu")
    part = dwc.causal_conv_bwd(x[:, -tail - 3:], x[:, -tail - 3:], w, None, "silu")[0]
    assert torch.equal(dx[:, -tail:], part[:, 3:]) and dw.isfinite().all()
    del dx, part, dw
    A = -torch.rand(C, 2, device="cuda", generator=g) - 0.5
    B, Cm = (torch.randn(1, T, 2, device="cuda", generator=g).bfloat16() for _ in range(2))
    y, last, saved = dwc.selective_scan_fwd(x, x, A, B, Cm, final=True, save=True, out=y)
    at = (T - tail) // 16 * 16
    state = saved[at // 16:at // 16 + 1].clone()
    y2, last2 = dwc.selective_scan_fwd(x[:, at:], x[:, at:], A, B[:, at:], Cm[:, at:], state=state, final=True)
    # (chunks of another length: the states in front of them are joined in another order, rounded to bf16 in the end)
    assert torch.allclose(y[:, at:].float(), y2.float(), rtol=2 ** -7, atol=1e-4)
    assert torch.allclose(last, last2, rtol=1e-5, atol=1e-6)
    del saved, last, y2
    rows = x[0]
    g1 = torch.ones(C, device="cuda")
    y, z, post, pre = dwc.block_norm_fwd(rows, rows, g1, g1, None, g1, out=y[0], stats=True)
    # (a call of fewer rows may add a row up in another order, so the last rows are held to the definition's bounds)
    last, one = d(rows[-tail:]), np.ones(C)
    for got, want in zip((y, z, post, pre), ref.block_norm(last, last, one, one, None, one, 1.0, "none", 1e-5)):
        within(got[-tail:], want, "block norm past 32 bits")
    dx, dres = dwc.block_norm_bwd(rows, rows, z, post, pre, g1, g1, None, g1)[:2]
    want = ref.block_norm_bwd(last, last, d(z[-tail:]), d(post[-tail:]), d(pre[-tail:]), one, one, None, one, 1.0, "none",
                              np.zeros_like(last))
    within(dx[-tail:], want["dx"], "dx")
    within(dres[-tail:], want["dres"], "dres")


@pytest.mark.parametrize("dtype,K,C", [("f32", 4, 2048), ("bf16", 4, 2048), ("f16", 8, 2048), ("bf16", 1, 2048), ("f32", 3, 1001),
                                       ("bf16", 2, 1001), ("bf16", 13, 2048)])
def test_causal_conv_of_long_runs(dtype, K, C):
    """So many positions that a thread walks its longest runs.  dx depends on a position's neighbours alone: the bits of each
    sequence's own call, whose runs are shorter.  Without an activation dw is a sum of products, in fp32 128 in a run, 4 runs
    to a row of partial sums, at most 160 such rows: off by 300 roundings of the sum of magnitudes at most."""
    rng = np.random.default_rng(K)
    T = 10001
    x, dy = (torch.from_numpy(rng.standard_normal((2, T, C), np.float32)).to("cuda", {"f32": torch.float32, "bf16": torch.bfloat16,
                                                                                    "f16": torch.float16}[dtype]) for _ in range(2))
    w, b = rand(rng, (K, C), "f32"), rand(rng, C, "f32")
    dx = dwc.causal_conv_bwd(dy, x, w, b, "silu")[0]
    for s in range(2):
        one = dwc.causal_conv_bwd(dy[s:s + 1], x[s:s + 1], w, b, "silu")[0]
        assert torch.equal(dx[s], one[0])
    _, dw, db, _ = dwc.causal_conv_bwd(dy, x, w, b)
    x, dy = x.double(), dy.double()
    for k in range(K):
        back = K - 1 - k
        terms = dy[:, back:] * x[:, :T - back]
        assert ((dw[k].double() - terms.sum((0, 1))).abs() <= 300 * 2 ** -24 * terms.abs().sum((0, 1))).all()
    assert ((db.double() - dy.sum((0, 1))).abs() <= 300 * 2 ** -24 * dy.abs().sum((0, 1))).all()


@pytest.mark.parametrize("pair", [("f32", "f32"), ("bf16", "bf16"), ("f32", "f16")], ids="-".join)
@pytest.mark.parametrize("rows,C", [(1000, 1536), (700, 2304), (700, 2501), (500, 2816), (340, 4104), (340, 5001), (340, 5120), (170, 6144),
                                    (170, 7001)])
def test_block_norm_widths_between(rows, C, pair):
    """Rows whose groups of warps do not fill a CTA of 512 threads, several to a CTA and several rounds of them."""
    check_norm(np.random.default_rng(C), (rows, C), *pair, dz=C % 2 == 0)


@pytest.mark.parametrize("pair", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("rows,C", [(64, 1000), (300, 129), (37, 1001), (257, 2048), (40, 8192), (9, 20001)])
def test_block_norm_in_place(rows, C, pair):
    """z over the stream, y over x or the gate: the bits of outputs of their own."""
    rng = np.random.default_rng(rows)
    x, gate, res = rand(rng, (rows, C), pair[1]), rand(rng, (rows, C), pair[1]), rand(rng, (rows, C), pair[0])
    g = rand(rng, C, "f32", 0.2, 1.0)
    y, z = dwc.block_norm_fwd(x, res, g, g, gate, g)
    for over in ("x", "gate", None):
        t = {"x": x.clone(), "gate": gate.clone(), "res": res.clone()}
        y2, z2 = dwc.block_norm_fwd(t["x"], t["res"], g, g, t["gate"], g, out=t[over] if over else None, z=t["res"])
        assert torch.equal(y, y2) and torch.equal(z, z2) and z2 is t["res"] and (over is None or y2 is t[over])
    with pytest.raises(ValueError):
        dwc.block_norm_fwd(x[:-1], res[:-1], out=x[1:])


@pytest.mark.parametrize("pair", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("rows,C", [(65, 1001), (130, 2048), (6, 20001)])
def test_block_norm_backward_in_place(rows, C, pair):
    """Through the C ABI: dx over dy, dres over dz, dgate over the gate."""
    rng = np.random.default_rng(rows)
    x, gate, dy = (rand(rng, (rows, C), pair[1]) for _ in range(3))
    res, dz = (rand(rng, (rows, C), pair[0]) for _ in range(2))
    g = rand(rng, C, "f32", 0.2, 1.0)
    _, z, post, pre = dwc.block_norm_fwd(x, res, g, g, gate, g, stats=True)
    want = dwc.block_norm_bwd(dy, x, z, post, pre, g, g, gate, g, dz=dz)
    lib = dwc.load_library()
    n = lib.dwc_block_norm_bwd_workspace_size(rows, C)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    grads = [torch.empty(C, device="cuda") for _ in range(3)]
    p = lambda t: t.data_ptr()  # noqa: E731
    code = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    st = lib.dwc_block_norm_bwd(p(dy), C, p(dz), C, p(x), C, p(z), C, p(gate), C, 2, p(post), p(pre), p(g), p(g), p(g), 0, 1.0, p(dy), p(dz),
                                p(gate), *(p(t) for t in grads), rows, C, code[x.dtype], code[res.dtype], p(ws), n,
                                torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for a, b in zip((dy, dz, gate, *grads), want):
        assert torch.equal(a, b)


def test_block_norm_over_several_rounds():
    """More rows than the groups of one round, aligned and shifted."""
    for rows, C in ((5000, 264), (3001, 1001), (1500, 4096), (40000, 33)):
        check_norm(np.random.default_rng(rows), (rows, C), "f32", "bf16")


@pytest.mark.parametrize("scale", [1e-12, 1e12])
def test_block_norm_scale_does_not_matter(scale):
    """Rows far from 1 in size (their squares still normal fp32 numbers)."""
    rng = np.random.default_rng(1)
    x, res, dy = rand(rng, (9, 512), "f32") * scale, rand(rng, (9, 512), "f32") * scale, rand(rng, (9, 512), "f32")
    y, z, post, pre = dwc.block_norm_fwd(x, res, eps=0.0, stats=True)
    one = np.ones(512)
    want = ref.block_norm(d(x), d(res), one, one, None, one, 1.0, "none", 0.0)
    within(y, want[0], "y")
    got = dwc.block_norm_bwd(dy, x, z, post, pre)
    want = ref.block_norm_bwd(d(dy), d(x), d(z), d(post), d(pre), one, one, None, one, 1.0, "none", np.zeros((9, 512)))
    within(got[0], want["dx"], "dx")
    within(got[1], want["dres"], "dres")


def test_overlaps_are_refused():
    x = torch.zeros(4, 6, 16, device="cuda")
    w = torch.zeros(4, 16, device="cuda")
    A, B = torch.zeros(16, 4, device="cuda"), torch.zeros(4, 6, 4, device="cuda")
    buf = torch.zeros(2, 4, 6, 16, device="cuda").view(-1)
    shifted = buf[8:8 + x.numel()].view_as(x)
    inside = buf[:x.numel()].view_as(x)
    for call in (lambda: dwc.causal_conv_fwd(inside, w, out=shifted), lambda: dwc.selective_scan_fwd(inside, x, A, B, B, out=shifted),
                 lambda: dwc.selective_scan_step(x[:, 0], x[:, 1], A, B[:, 0], B[:, 0], buf[:256].view(4, 16, 4), out=buf[:64].view(4, 16)),
                 lambda: dwc.causal_conv_step(x[:, 0], x[:, :3], w)):
        with pytest.raises(ValueError, match="overlap"):
            call()
