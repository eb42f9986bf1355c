"""GPU parity of the gated norm and the residual norm, forward and backward, against the fp64 definitions.

Tolerances.  Every output is one rounding (half a step: 2^-8 relative for bf16, 2^-24 for fp32) of an fp32
value.  That value is a product of a few factors, each with a relative error of a few 2^-24: the row sum of
squares adds at most N/32 + 5 roundings along its longest chain and enters under a square root, the
exponential of a gate in [-8, 8] carries at most 16 units (its argument's rounding times the argument), and
the remaining products and the quotient some ten more.  REL = 2^-18 (64 units) covers rows up to 2,048 wide
and ABS-terms below are REL times the magnitude of the terms that a difference is taken of.  Sums over rows:
at most 64 further roundings along a chain (rows / 592 blocks, then the fixed tree), so 2^-17 times the sum
of magnitudes."""
import numpy as np
import pytest

from oracle import operators as op
from tests.gpu_util import cuda_or_skip, f64

pytestmark = pytest.mark.gpu
REL = 2.0 ** -18
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 1e-6


def _dt(torch, dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _make(torch, seed, rows, d, dtype, names, weights):
    gen = torch.Generator().manual_seed(seed)
    out = {n: torch.randn(rows, d, generator=gen).clamp(-8, 8).to(_dt(torch, dtype)).cuda() for n in names}
    return out | {n: (1 + 0.3 * torch.randn(d, generator=gen)).cuda() for n in weights}


def close(got, ref, half, magnitude, rel=REL):
    err = np.abs(f64(got) - ref)
    bar = half * np.abs(ref) * (1 + rel) + rel * magnitude + 1e-37
    assert np.isfinite(f64(got)).all()
    assert (err <= bar).all(), f"worst {np.max(err / bar):.2f} of the bar"


def check_gated(g, torch, t, act, dtype, eps=EPS, y=None):
    half = HALF[dtype]
    x = {n: f64(a) for n, a in t.items()}
    if y is None:
        y = g.gated_norm_fwd(t["o"], t["gate"], t["weight"], act=act, eps=eps)
    ref = op.gated_norm(x["o"], x["gate"], x["weight"], act, eps)
    close(y, ref, half, np.abs(ref))
    do, dgate, dweight = g.gated_norm_bwd(t["o"], t["gate"], t["weight"], t["dy"], act=act, eps=eps)
    rdo, rdg, rdw = op.gated_norm_backward(x["o"], x["gate"], x["weight"], x["dy"], act, eps)
    a, slope = op._act(x["gate"], act)
    r = 1 / np.sqrt((x["o"] ** 2).mean(-1, keepdims=True) + eps)
    dxn = np.abs(x["dy"] * a * x["weight"])
    close(do, rdo, half, r * dxn + np.abs(x["o"]) * r ** 3 * (dxn * np.abs(x["o"])).mean(-1, keepdims=True))
    # silu's slope s (1 + g (1 - s)) is a sum of two terms
    terms = np.abs(x["dy"] * x["o"] * r * x["weight"]) * (1 + np.abs(x["gate"]))
    close(dgate, rdg, half, terms)
    close(dweight, rdw, HALF["f32"], np.abs(x["dy"] * a * x["o"] * r).sum(0), 2.0 ** -17)


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("bf16", 7), ("bf16", 1000), ("bf16", 9001), ("f32", 1),
                                        ("f32", 33), ("f32", 5003)])
def test_gated_norm(dtype, rows, d, act):
    torch, g = cuda_or_skip()
    t = _make(torch, rows + d, rows, d, dtype, ("o", "gate", "dy"), ("weight",))
    check_gated(g, torch, t, act, dtype)


@pytest.mark.parametrize("dtype,d,rows", [("bf16", 128, 18943), ("bf16", 128, 18944), ("bf16", 128, 18977),
                                          ("bf16", 64, 37887), ("bf16", 64, 37888), ("bf16", 64, 37901),
                                          ("f32", 128, 9471), ("f32", 128, 9472), ("f32", 128, 9475),
                                          ("f32", 64, 18943), ("f32", 64, 18944), ("f32", 64, 18951)])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gated_norm_of_many_rows(dtype, d, rows, act):
    """Both sides of the row counts from which a forward thread has four rows, with and without a remainder."""
    torch, g = cuda_or_skip()
    check_gated(g, torch, _make(torch, rows, rows, d, dtype, ("o", "gate", "dy"), ("weight",)), act, dtype)


def test_gated_norm_rows_of_zeros_and_wide_gates():
    torch, g = cuda_or_skip()
    t = _make(torch, 5, 6, 128, "f32", ("o", "gate", "dy"), ("weight",))
    t["o"][0] = 0                        # r = eps^-1/2: y = 0, do = dn weight / sqrt(eps)
    t["gate"][1, ::2], t["gate"][1, 1::2] = 200.0, -200.0    # the sigmoid's ends: exactly 1 and 0
    t["o"][2] = 1e15                     # squares near the top of fp32's range
    y = g.gated_norm_fwd(t["o"], t["gate"], t["weight"])
    check_gated(g, torch, {n: a[[0, 2, 3, 4, 5]] if a.dim() == 2 else a for n, a in t.items()}, "silu", "f32")
    x = {n: f64(a) for n, a in t.items()}
    with np.errstate(over="ignore"):
        ref = op.gated_norm(x["o"], x["gate"], x["weight"])
    close(y, ref, HALF["f32"], np.abs(ref))
    assert (f64(y)[1, 1::2] == 0).all()


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("bf16", 2), ("bf16", 3), ("bf16", 45), ("bf16", 9003), ("f32", 1),
                                        ("f32", 3), ("f32", 5001)])
def test_gated_norm_without_an_eps(dtype, rows, d, act):
    """eps = 0, the rows not filling the last warp: a place without a row takes no part in dweight."""
    torch, g = cuda_or_skip()
    t = _make(torch, rows + d, rows, d, dtype, ("o", "gate", "dy"), ("weight",))
    check_gated(g, torch, t, act, dtype, eps=0.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_norm_slope_of_wide_open_gates(dtype, d):
    """dgate of sigmoid gates is a product alone, so it is right to a few units of its own size however far the gate is
    open: s (1 - s) is 2e-9 at 20, where a difference of two fp32 has lost all digits.  The argument's rounding adds 20
    units of 2^-24 there to what REL counts otherwise."""
    torch, g = cuda_or_skip()
    t = _make(torch, d, 301, d, dtype, ("o", "gate", "dy"), ("weight",))
    t["gate"].copy_(torch.linspace(-20, 20, 301 * d).view(301, d))
    _, dgate, _ = g.gated_norm_bwd(t["o"], t["gate"], t["weight"], t["dy"], act="sigmoid")
    x = {n: f64(a) for n, a in t.items()}
    slope = 1 / (1 + np.exp(-x["gate"])) / (1 + np.exp(x["gate"]))
    r = 1 / np.sqrt((x["o"] ** 2).mean(-1, keepdims=True) + EPS)
    ref = x["dy"] * x["o"] * r * x["weight"] * slope
    close(dgate, ref, HALF[dtype], np.abs(ref))


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("d", [64, 128])
def test_gated_norm_in_fp32_is_fp32(d, act):
    """fp32 rows keep fp32's precision over all gates.  In units of 2^-24: expf 4 (2 ulp), its sum 1, the quotient 1, its
    product 1; the row's sum of squares at most 4 + 5 roundings and eps 1, halved by the root, rsqrtf 4 (2 ulp); four
    products, the last the output's rounding: 20.  dgate's product has five factors more for the sigmoid (24 in all); the
    bar for both is 32."""
    torch, g = cuda_or_skip()
    t = _make(torch, d, 603, d, "f32", ("o", "gate", "dy"), ("weight",))
    t["gate"].copy_(torch.linspace(-80, 80, 603 * d).view(603, d))
    y = g.gated_norm_fwd(t["o"], t["gate"], t["weight"], act=act)
    x = {n: f64(a) for n, a in t.items()}
    ref = op.gated_norm(x["o"], x["gate"], x["weight"], act)
    assert (np.abs(f64(y) - ref) <= 32 * 2.0 ** -24 * np.abs(ref)).all(), np.max(np.abs(f64(y) / ref - 1)) * 2 ** 24
    if act == "sigmoid":
        _, dgate, _ = g.gated_norm_bwd(t["o"], t["gate"], t["weight"], t["dy"], act=act)
        r = 1 / np.sqrt((x["o"] ** 2).mean(-1, keepdims=True) + EPS)
        ref = x["dy"] * x["o"] * r * x["weight"] / (1 + np.exp(-x["gate"])) / (1 + np.exp(x["gate"]))
        assert (np.abs(f64(dgate) - ref) <= 32 * 2.0 ** -24 * np.abs(ref)).all()


def test_gated_norm_in_place_shapes_and_empty():
    torch, g = cuda_or_skip()
    t = _make(torch, 6, 60, 128, "bf16", ("o", "gate", "dy"), ("weight",))
    want = g.gated_norm_fwd(t["o"], t["gate"], t["weight"])
    for into in ("o", "gate"):
        c = {n: t[n].clone() for n in ("o", "gate")}
        g.gdn2_gated_norm_fwd(c["o"], c["gate"], t["weight"], c[into])
        assert torch.equal(c[into], want)
    shaped = g.gated_norm_fwd(t["o"].view(3, 5, 4, 128), t["gate"].view(3, 5, 4, 128), t["weight"])
    assert torch.equal(shaped.view(60, 128), want)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert g.gated_norm_fwd(e, e, t["weight"]).shape == (0, 128)
    _, _, dw = g.gated_norm_bwd(e, e, t["weight"], e)
    assert (dw == 0).all()


def check_add(g, torch, t, dtype, scale=True, residual=True, dh=True, eps=EPS):
    half = HALF[dtype]
    x = {n: f64(a) for n, a in t.items()}
    sc, res = t["scale"] if scale else None, t["residual"] if residual else None
    y, h = g.add_norm_fwd(t["x"], res, sc, t["weight"], eps=eps)
    ry, rh = op.add_norm(x["x"], x["residual"] if residual else None, x["scale"] if scale else None, x["weight"], eps)
    terms = np.abs(x["x"]) * (np.abs(x["scale"]) if scale else 1) + (np.abs(x["residual"]) if residual else 0)
    close(h, rh, half, terms)
    r = 1 / np.sqrt((rh ** 2).mean(-1, keepdims=True) + eps)
    close(y, ry, half, terms * r * np.abs(x["weight"]))
    dres, dx, dscale, dweight = g.add_norm_bwd(h, t["x"], sc, t["weight"], t["dy"], t["dh"] if dh else None, eps=eps)
    xh = f64(h)                          # the gradients are those at the stored sum
    ref = op.add_norm_backward(xh, x["x"], x["scale"] if scale else None, x["weight"], x["dy"],
                               x["dh"] if dh else None, eps)
    r = 1 / np.sqrt((xh ** 2).mean(-1, keepdims=True) + eps)
    d = np.abs(x["dy"] * x["weight"])
    terms = (np.abs(x["dh"]) if dh else 0) + r * d + np.abs(xh) * r ** 3 * (d * np.abs(xh)).mean(-1, keepdims=True)
    close(dres, ref[0], half, terms)
    if scale:
        close(dx, ref[1], half, terms * np.abs(x["scale"]))
        close(dscale, ref[2], HALF["f32"], (terms * np.abs(x["x"])).sum(0), 2.0 ** -17)
    else:
        assert dscale is None and torch.equal(dx, dres)
    close(dweight, ref[3], HALF["f32"], np.abs(x["dy"] * xh * r).sum(0), 2.0 ** -17)


@pytest.mark.parametrize("dtype,rows,width", [("bf16", 1, 8), ("bf16", 5, 72), ("bf16", 700, 256), ("bf16", 64, 2048),
                                              ("bf16", 1300, 2048), ("bf16", 9, 4096), ("bf16", 3, 5000),
                                              ("bf16", 2, 8192), ("f32", 1, 8), ("f32", 30, 136), ("f32", 600, 2048),
                                              ("f32", 3, 3400), ("f32", 2, 4104), ("f32", 2, 8192)])
def test_add_norm(dtype, rows, width):
    torch, g = cuda_or_skip()
    t = _make(torch, rows + width, rows, width, dtype, ("x", "residual", "dy", "dh"), ("scale", "weight"))
    check_add(g, torch, t, dtype)


@pytest.mark.parametrize("scale,residual,dh", [(False, True, True), (True, False, True), (False, False, False),
                                               (True, True, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_add_norm_optional_inputs(dtype, scale, residual, dh):
    torch, g = cuda_or_skip()
    t = _make(torch, 11, 50, 264, dtype, ("x", "residual", "dy", "dh"), ("scale", "weight"))
    check_add(g, torch, t, dtype, scale, residual, dh)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", [(9, 8), (33, 32), (4001, 64), (5, 72), (3001, 128), (5001, 208), (13, 264), (1201, 392), (7, 520), (3, 776), (2001, 1032), (3, 1304)])
def test_add_norm_rows_that_share_a_block(dtype, rows, width):
    """Eight lanes to six warps a row, the last block partly empty; an empty place takes no part, whatever eps is."""
    torch, g = cuda_or_skip()
    t = _make(torch, 3, rows, width, dtype, ("x", "residual", "dy", "dh"), ("scale", "weight"))
    check_add(g, torch, t, dtype)
    y, h = g.add_norm_fwd(t["x"], t["residual"], t["scale"], t["weight"])
    small, none = (g.add_norm_bwd(h, t["x"], t["scale"], t["weight"], t["dy"], t["dh"], eps=eps) for eps in (1e-20, 0.0))
    assert all(torch.equal(a, b) and torch.isfinite(a.float()).all() for a, b in zip(small, none))


@pytest.mark.parametrize("dtype,rows,width", [("bf16", 40003, 64), ("bf16", 20011, 128), ("bf16", 30001, 72),
                                              ("bf16", 9999, 208), ("f32", 40003, 32), ("f32", 20011, 64), ("f32", 5003, 264)])
@pytest.mark.parametrize("scale", [True, False])
def test_add_norm_of_more_rows_than_the_blocks_take_at_once(dtype, rows, width, scale):
    """The backward's blocks (at most 592, of up to 32 rows) walk on to further rows and carry the columns' sums: along a
    sum's longest chain here 3 rows of a thread, 31 of the block's others, 18 blocks of a group and 5 steps of the last
    sum, 57 additions of the 64 that the tolerance for sums counts."""
    torch, g = cuda_or_skip()
    t = _make(torch, rows, rows, width, dtype, ("x", "residual", "dy", "dh"), ("scale", "weight"))
    check_add(g, torch, t, dtype, scale=scale)


def test_add_norm_in_place_and_empty():
    torch, g = cuda_or_skip()
    t = _make(torch, 12, 40, 512, "bf16", ("x", "residual"), ("scale", "weight"))
    y, h = g.add_norm_fwd(t["x"], t["residual"], t["scale"], t["weight"])
    r, x = t["residual"].clone(), t["x"].clone()
    g.gdn2_add_norm_fwd(x, r, t["scale"], t["weight"], r, x)      # the stream and the input both overwritten
    assert torch.equal(r, h) and torch.equal(x, y)
    y2 = torch.empty_like(y)
    g.gdn2_add_norm_fwd(t["x"], t["residual"], t["scale"], t["weight"], None, y2)
    assert torch.equal(y2, y)
    e = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    _, _, ds, dw = g.add_norm_bwd(e, e, t["scale"], t["weight"], e)
    assert (ds == 0).all() and (dw == 0).all()


def test_backward_is_deterministic_with_a_shared_workspace():
    torch, g = cuda_or_skip()
    t = _make(torch, 13, 30000, 128, "bf16", ("o", "gate", "dy"), ("weight",))
    ws = g.new_workspace(g.gdn2_gated_norm_bwd_workspace_bytes(30000, 128))
    ws[256:].fill_(0xFF)
    first = g.gated_norm_bwd(t["o"], t["gate"], t["weight"], t["dy"], workspace=ws)
    for _ in range(3):
        again = g.gated_norm_bwd(t["o"], t["gate"], t["weight"], t["dy"], workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_backward_without_a_workspace_zeroes_nothing(monkeypatch):
    """The gradients' workspace holds no status: nothing of it is read before it is written, and a call that makes its own
    launches no memset for it."""
    torch, g = cuda_or_skip()
    t = _make(torch, 17, 300, 128, "bf16", ("o", "gate", "dy", "h", "x"), ("weight", "scale"))
    calls = [lambda ws: g.gated_norm_bwd(t["o"], t["gate"], t["weight"], t["dy"], workspace=ws),
             lambda ws: g.add_norm_bwd(t["h"], t["x"], t["scale"], t["weight"], t["dy"], workspace=ws)]
    sizes = g.gdn2_gated_norm_bwd_workspace_bytes(300, 128), g.gdn2_add_norm_bwd_workspace_bytes(300, 128)
    wants = [call(torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")) for call, n in zip(calls, sizes)]
    monkeypatch.setattr(g, "new_workspace", None)            # it zeroes the status header
    for call, want in zip(calls, wants):
        assert all(torch.equal(a, b) for a, b in zip(call(None), want))


def test_autograd_of_both_norms():
    """One block's tail and the next one's head, gradients against fp64 autograd of the same formulas."""
    torch, g = cuda_or_skip()
    rows, d = 37, 128
    t = _make(torch, 14, rows, d, "f32", ("o", "gate", "residual", "c1", "c2"), ("w1", "w2", "scale"))
    leaves = {n: t[n].clone().requires_grad_() for n in ("o", "gate", "residual", "w1", "w2", "scale")}
    z = g.gdn2_gated_norm(leaves["o"], leaves["gate"], leaves["w1"])
    y, h = g.gdn2_add_norm(z, leaves["residual"], leaves["w2"], leaves["scale"])
    (y * t["c1"] + h * t["c2"]).sum().backward()
    ref = {n: t[n].double().cpu().requires_grad_() for n in leaves}
    norm = lambda x: x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)  # noqa: E731
    z = norm(ref["o"]) * ref["w1"] * torch.nn.functional.silu(ref["gate"])
    h = ref["residual"] + ref["scale"] * z
    y = norm(h) * ref["w2"]
    (y * t["c1"].double().cpu() + h * t["c2"].double().cpu()).sum().backward()
    for n in leaves:
        # a chain of two backward passes over 37 rows of 128: each within 2^-17 of its terms, whose largest
        # is at most some 16 times the largest gradient
        want = ref[n].grad.numpy()
        assert np.abs(f64(leaves[n].grad) - want).max() <= 2.0 ** -12 * np.abs(want).max(), n


def test_autograd_gradients_that_are_not_wanted_or_missing():
    torch, g = cuda_or_skip()
    t = _make(torch, 15, 20, 64, "f32", ("x", "residual", "c"), ("weight",))
    x, r, w = (t[n].clone().requires_grad_() for n in ("x", "residual", "weight"))
    y, h = g.gdn2_add_norm(x, r, w)
    gx, gr = torch.autograd.grad((h * t["c"]).sum(), (x, r))     # no gradient at y
    assert torch.equal(gx, t["c"]) and torch.equal(gr, t["c"]) and gx.data_ptr() != gr.data_ptr()
    y, h = g.gdn2_add_norm(x, None, t["weight"])                 # no residual, a fixed weight
    (gx,) = torch.autograd.grad((y * t["c"]).sum(), (x,))
    want = op.add_norm_backward(f64(h), None, None, f64(t["weight"]), f64(t["c"]))[0]
    assert np.abs(f64(gx) - want).max() <= 2.0 ** -15 * np.abs(want).max()
    with pytest.raises(RuntimeError):
        (gx,) = torch.autograd.grad(g.gdn2_gated_norm(x, r, w).sum(), (x,), create_graph=True)
        torch.autograd.grad(gx.sum(), (x,))


def test_captured_forward_and_backward_on_a_side_stream():
    torch, g = cuda_or_skip()
    t = _make(torch, 16, 500, 128, "bf16", ("o", "gate", "dy"), ("weight",))
    ws = g.new_workspace(g.gdn2_gated_norm_bwd_workspace_bytes(500, 128))
    out = [torch.empty_like(t["o"]) for _ in range(3)] + [torch.empty_like(t["weight"])]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            g.gdn2_gated_norm_fwd(t["o"], t["gate"], t["weight"], out[0])
            g.gdn2_gated_norm_bwd(t["o"], t["gate"], t["weight"], t["dy"], *out[1:], workspace=ws)
    for seed in (1, 2):
        new = _make(torch, seed, 500, 128, "bf16", ("o", "gate", "dy"), ("weight",))
        for n in new:
            t[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        want = [g.gated_norm_fwd(t["o"], t["gate"], t["weight"]), *g.gated_norm_bwd(t["o"], t["gate"], t["weight"], t["dy"])]
        assert all(torch.equal(a, b) for a, b in zip(out, want))
