"""Pins of oracle/operators.py (CPU): gradients against central differences and torch's fp64 autograd,
trees and runs against the sequential recurrence oracle, copies against their definition."""
import numpy as np
import pytest

import oracle
from oracle import operators as op


def _cases(rng, rows=5, d=7):
    return {n: rng.standard_normal((rows, d)) for n in ("o", "gate", "dy", "x", "residual", "dh")} | \
        {n: 1 + 0.3 * rng.standard_normal(d) for n in ("weight", "scale")}


def _differences(loss, at, h=1e-5):
    g = np.zeros_like(at)
    for i in np.ndindex(at.shape):
        keep = at[i]
        at[i] = keep + h
        up = loss()
        at[i] = keep - h
        g[i] = (up - loss()) / (2 * h)
        at[i] = keep
    return g


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gated_norm_gradients_against_differences(rng, act):
    c = _cases(rng)
    loss = lambda: float((c["dy"] * op.gated_norm(c["o"], c["gate"], c["weight"], act, 1e-3)).sum())  # noqa: E731
    got = op.gated_norm_backward(c["o"], c["gate"], c["weight"], c["dy"], act, 1e-3)
    for g, name in zip(got, ("o", "gate", "weight")):
        # central differences at h = 1e-5: truncation O(h^2) and rounding 1e-16/h, both below 1e-9
        np.testing.assert_allclose(g, _differences(loss, c[name]), rtol=0, atol=1e-8)


@pytest.mark.parametrize("with_scale,with_residual", [(True, True), (False, True), (True, False)])
def test_add_norm_gradients_against_differences(rng, with_scale, with_residual):
    c = _cases(rng)
    scale = c["scale"] if with_scale else None
    residual = c["residual"] if with_residual else None

    def loss():
        y, h = op.add_norm(c["x"], residual, scale, c["weight"], 1e-3)
        return float((c["dy"] * y).sum() + (c["dh"] * h).sum())

    _, h = op.add_norm(c["x"], residual, scale, c["weight"], 1e-3)
    dres, dx, dscale, dweight = op.add_norm_backward(h, c["x"], scale, c["weight"], c["dy"], c["dh"], 1e-3)
    for g, at in ((dx, c["x"]), (dweight, c["weight"])) + (((dscale, scale),) if with_scale else ()) + \
            (((dres, residual),) if with_residual else ()):
        np.testing.assert_allclose(g, _differences(loss, at), rtol=0, atol=1e-8)
    if not with_scale:
        assert dscale is None and np.array_equal(dx, dres)


def test_norms_against_torch_autograd(rng):
    torch = pytest.importorskip("torch")
    c = _cases(rng, 4, 16)
    t = {n: torch.tensor(a, dtype=torch.float64, requires_grad=True) for n, a in c.items()}
    norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    y = norm(t["o"]) * t["weight"] * torch.nn.functional.silu(t["gate"])
    ref = torch.autograd.grad(y, (t["o"], t["gate"], t["weight"]), t["dy"])
    np.testing.assert_allclose(op.gated_norm(c["o"], c["gate"], c["weight"]), y.detach().numpy(), atol=1e-13)
    for g, r in zip(op.gated_norm_backward(c["o"], c["gate"], c["weight"], c["dy"]), ref):
        np.testing.assert_allclose(g, r.numpy(), atol=1e-12)
    h = t["residual"] + t["scale"] * t["x"]
    y = norm(h) * t["weight"]
    ref = torch.autograd.grad((y * t["dy"] + h * t["dh"]).sum(), (t["residual"], t["x"], t["scale"], t["weight"]))
    for g, r in zip(op.add_norm_backward(h.detach().numpy(), c["x"], c["scale"], c["weight"], c["dy"], c["dh"]), ref):
        np.testing.assert_allclose(g, r.numpy(), atol=1e-12)


def tokens(rng, n, H=2, K=8, V=6):
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    gate = lambda *s: 1 / (1 + np.exp(-rng.standard_normal(s)))  # noqa: E731
    return [unit(rng.standard_normal((n, H, K))), unit(rng.standard_normal((n, H, K))), rng.standard_normal((n, H, V)),
            gate(n, H, K), gate(n, H, K), gate(n, H, V)]


def test_tree_is_the_recurrence_along_every_path(rng):
    x, pool = tokens(rng, 9), rng.standard_normal((3, 2, 8, 6))
    cu, parents, slots = [0, 6, 6, 9], [-1, 0, 0, 2, -1, 3, -1, 0, 1], [2, 0, -1]
    o = op.tree(*x, pool, slots, cu, parents)
    for i, lo in enumerate(cu[:-1]):
        for t in range(lo, cu[i + 1]):
            path = [t]
            while parents[path[0]] >= 0:
                path.insert(0, lo + parents[path[0]])
            S0 = pool[slots[i]][None] if slots[i] >= 0 else None
            ref, _ = oracle.recurrence(*(a[path][None] for a in x), S0)
            np.testing.assert_allclose(o[t], ref[0, -1], atol=1e-13)


def test_recurrent_is_the_recurrence_of_each_run(rng):
    x, pool = tokens(rng, 8), rng.standard_normal((5, 2, 8, 6))
    index, cu, src, dst = [7, 1, 2, 2, 0, 5], [0, 3, 3, 6], [4, 0, -1], [4, 1, 2]
    o, after = op.recurrent(*x, pool, src, dst, cu, index)
    for i in (0, 2):
        rows = index[cu[i]:cu[i + 1]]
        ref, S = oracle.recurrence(*(a[rows][None] for a in x), pool[src[i]][None] if src[i] >= 0 else None)
        np.testing.assert_allclose(o[cu[i]:cu[i + 1]], ref[0], atol=1e-13)
        np.testing.assert_allclose(after[dst[i]], S[0], atol=1e-13)
    assert np.array_equal(after[1], pool[0]) and np.array_equal(after[3], pool[3])   # an empty run; an untouched slot


def test_state_copy_definition(rng):
    pool = rng.standard_normal((5, 3))
    out = op.state_copy(pool, pool, [0, 1, 4, -1, 3, 3], [1, 0, -1, 2, 2, 4])
    for got, want in zip(out, (pool[1], pool[0], pool[2], pool[4], np.zeros(3))):
        assert np.array_equal(got, want)
