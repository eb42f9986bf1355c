"""Argument checks of the norms and of the operators over a state cache, on the CPU: the C entry points
refuse before they touch the device, and the binding marshals its tensors in the declared order."""
import ctypes

import pytest
import torch

import gated_delta_rule_96_b200 as g
from tests.test_binding_host import addr, rec  # noqa: F401  (the recorder fixture)

P = ctypes.c_void_p
F = P(0x10000)       # never dereferenced: every call below fails validation first or has nothing to do
ODD = P(0x10004)


@pytest.fixture(scope="module")
def lib():
    return g.load_library()


def gated(lib, o=F, gate=F, weight=F, y=F, rows=4, d=128, act=0, eps=1e-6, dtype=1):
    return lib.gdn2_gated_norm_fwd(o, gate, weight, y, rows, d, act, eps, dtype, None)


def gated_bwd(lib, p=F, weight=F, dweight=F, rows=4, d=128, act=0, eps=1e-6, dtype=1, ws=F, n=1 << 30):
    return lib.gdn2_gated_norm_bwd(p, p, weight, p, p, p, dweight, rows, d, act, eps, dtype, ws, n, None)


def add(lib, x=F, residual=F, scale=F, weight=F, h=F, y=F, rows=4, width=64, eps=1e-6, dtype=1):
    return lib.gdn2_add_norm_fwd(x, residual, scale, weight, h, y, rows, width, eps, dtype, None)


def add_bwd(lib, h=F, x=F, scale=F, weight=F, dh=F, dx=F, dscale=F, dweight=F, rows=4, width=64, eps=1e-6, dtype=1,
            ws=F, n=1 << 30):
    return lib.gdn2_add_norm_bwd(h, x, scale, weight, h, dh, h, dx, dscale, dweight, rows, width, eps, dtype, ws, n,
                                 None)


def tree(lib, p=F, S=F, stride=2 * 128 * 128, num=4, idx=F, o=F, batch=2, H=2, total=8, most=4, K=128, V=128, dtype=1,
         ws=F, n=256):
    return lib.gdn2_tree_fwd(p, p, p, p, p, p, S, stride, num, idx, idx, idx, o, batch, H, total, most, K, V, dtype, ws,
                             n, None)


def recurrent(lib, p=F, S=F, stride=2 * 128 * 128, num=4, idx=F, index=F, o=F, batch=2, H=2, total=8, rows=8, K=128,
              V=128, dtype=1, ws=F, n=256):
    return lib.gdn2_recurrent_fwd(p, p, p, p, p, p, S, stride, num, idx, idx, idx, index, o, batch, H, total, rows, K,
                                  V, dtype, ws, n, None)


def copy(lib, dst=F, dstride=64, dnum=4, src=F, sstride=64, snum=4, idx=F, pairs=3, floats=64, ws=F, n=256):
    return lib.gdn2_state_copy(dst, dstride, dnum, src, sstride, snum, idx, idx, pairs, floats, ws, n, None)


NAN = float("nan")


@pytest.mark.parametrize("call,want", [
    (lambda l: gated(l, rows=-1), -2), (lambda l: gated(l, dtype=2), -3), (lambda l: gated(l, d=96), -4),
    (lambda l: gated(l, o=None), -1), (lambda l: gated(l, weight=None), -1), (lambda l: gated(l, y=ODD), -7),
    (lambda l: gated(l, act=2), -10), (lambda l: gated(l, eps=-1.0), -10), (lambda l: gated(l, eps=NAN), -10),
    (lambda l: gated(l, rows=0, o=None, y=None), 0),
    (lambda l: gated_bwd(l, rows=-1), -2), (lambda l: gated_bwd(l, d=32), -4), (lambda l: gated_bwd(l, p=None), -1),
    (lambda l: gated_bwd(l, dweight=None), -1), (lambda l: gated_bwd(l, act=-1), -10),
    (lambda l: gated_bwd(l, ws=None), -5), (lambda l: gated_bwd(l, ws=P(0x10008)), -7), (lambda l: gated_bwd(l, n=300), -5),
    (lambda l: add(l, rows=-1), -2), (lambda l: add(l, width=60), -4), (lambda l: add(l, width=8200), -4),
    (lambda l: add(l, width=0), -4), (lambda l: add(l, dtype=5), -3), (lambda l: add(l, x=None), -1),
    (lambda l: add(l, residual=ODD), -7), (lambda l: add(l, scale=ODD), -7), (lambda l: add(l, h=ODD), -7),
    (lambda l: add(l, eps=2.0), -10), (lambda l: add(l, rows=0), 0),
    (lambda l: add_bwd(l, width=4), -4), (lambda l: add_bwd(l, x=None), -1), (lambda l: add_bwd(l, dx=None), -1),
    (lambda l: add_bwd(l, dscale=None), -1), (lambda l: add_bwd(l, dh=ODD), -7), (lambda l: add_bwd(l, n=256), -5),
    (lambda l: tree(l, batch=-1), -2), (lambda l: tree(l, total=-1), -2), (lambda l: tree(l, most=-1), -2),
    (lambda l: tree(l, most=65), -4), (lambda l: tree(l, K=96), -4), (lambda l: tree(l, dtype=9), -3),
    (lambda l: tree(l, p=None), -1), (lambda l: tree(l, p=ODD), -7), (lambda l: tree(l, S=None), -1),
    (lambda l: tree(l, stride=128 * 128), -2), (lambda l: tree(l, stride=2 * 128 * 128 + 2), -7),
    (lambda l: tree(l, idx=None), -1), (lambda l: tree(l, idx=P(0x10002)), -7), (lambda l: tree(l, ws=None), -5),
    (lambda l: tree(l, n=16), -5), (lambda l: tree(l, batch=65536), -4), (lambda l: tree(l, batch=0), 0),
    (lambda l: tree(l, total=0, p=None, o=None), 0), (lambda l: tree(l, most=0), 0),
    (lambda l: recurrent(l, rows=-1), -2), (lambda l: recurrent(l, index=None, rows=7), -2),
    (lambda l: recurrent(l, V=96), -4), (lambda l: recurrent(l, p=None), -1), (lambda l: recurrent(l, idx=None), -1),
    (lambda l: recurrent(l, index=P(0x10001)), -7), (lambda l: recurrent(l, ws=None), -5),
    (lambda l: recurrent(l, stride=64), -2), (lambda l: recurrent(l, batch=70000), -4),
    (lambda l: recurrent(l, H=0), 0), (lambda l: recurrent(l, batch=0), 0),
    (lambda l: copy(l, pairs=-1), -2), (lambda l: copy(l, pairs=1025), -4), (lambda l: copy(l, floats=62), -7),
    (lambda l: copy(l, dstride=32), -2), (lambda l: copy(l, dstride=66), -7), (lambda l: copy(l, dstride=128), -2),
    (lambda l: copy(l, dst=None), -1), (lambda l: copy(l, idx=None), -1), (lambda l: copy(l, src=P(0x20008)), -7),
    (lambda l: copy(l, ws=None), -5), (lambda l: copy(l, n=0), -5), (lambda l: copy(l, pairs=0, idx=None), 0),
])
def test_entry_points_refuse(lib, call, want):
    assert call(lib) == want
    assert g.gdn2_status_str(want) != "unknown status"


def test_workspace_sizes():
    assert g.gdn2_gated_norm_bwd_workspace_bytes(-1, 128) == 0 and g.gdn2_gated_norm_bwd_workspace_bytes(4, 96) == 0
    assert g.gdn2_gated_norm_bwd_workspace_bytes(0, 128) >= 256 + 4 * 128
    assert g.gdn2_add_norm_bwd_workspace_bytes(4, 12) == 0 and g.gdn2_add_norm_bwd_workspace_bytes(-1, 16) == 0
    # bounded: at most 592 blocks write partial sums, whatever the number of rows
    assert g.gdn2_gated_norm_bwd_workspace_bytes(1 << 40, 128) <= 256 + 592 * 128 * 4
    assert g.gdn2_add_norm_bwd_workspace_bytes(1 << 40, 8192) <= 256 + 592 * 2 * 8192 * 4


def test_norm_marshalling(rec):  # noqa: F811
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    o, gate, y, dy, do, dg = (bf(2, 3, 4, 64) for _ in range(6))
    w, dw = torch.ones(64), torch.zeros(64)
    g.gdn2_gated_norm_fwd(o, gate, w, y, act="sigmoid", eps=1e-5)
    name, a = rec.calls[-1]
    assert name == "gdn2_gated_norm_fwd" and [addr(p) for p in a[:4]] == [t.data_ptr() for t in (o, gate, w, y)]
    assert a[4:7] == (24, 64, 1) and a[7] == 1e-5 and a[8] == g.GDN2_BF16
    g.gdn2_gated_norm_bwd(o, gate, w, dy, do, dg, dw)
    name, a = rec.calls[-1]
    assert [addr(p) for p in a[:7]] == [t.data_ptr() for t in (o, gate, w, dy, do, dg, dw)]
    assert a[7:10] == (24, 64, 0) and a[13] >= g.gdn2_gated_norm_bwd_workspace_bytes(24, 64)
    with pytest.raises(ValueError):
        g.gdn2_gated_norm_fwd(o, gate, w, y, act="tanh")
    with pytest.raises(TypeError):
        g.gdn2_gated_norm_fwd(o, gate.float(), w, y)
    with pytest.raises(ValueError):
        g.gdn2_gated_norm_fwd(o, gate, torch.ones(128), y)

    x, r, h, y, dy, dh, dr, dx = (torch.zeros(5, 96) for _ in range(8))
    s, w, ds, dw = (torch.ones(96) for _ in range(4))
    g.gdn2_add_norm_fwd(x, None, s, w, None, y)
    _, a = rec.calls[-1]
    assert [addr(p) for p in a[:6]] == [x.data_ptr(), None, s.data_ptr(), w.data_ptr(), None, y.data_ptr()]
    assert a[6:8] == (5, 96) and a[9] == g.GDN2_F32
    g.gdn2_add_norm_bwd(h, x, s, w, dy, None, dr, dx, ds, dw)
    _, a = rec.calls[-1]
    assert [addr(p) for p in a[:10]] == [h.data_ptr(), x.data_ptr(), s.data_ptr(), w.data_ptr(), dy.data_ptr(), None,
                                         dr.data_ptr(), dx.data_ptr(), ds.data_ptr(), dw.data_ptr()]
    with pytest.raises(ValueError):
        g.gdn2_add_norm_fwd(x, r[:4], s, w, h, y)
    with pytest.raises(TypeError):
        g.gdn2_add_norm_bwd(h, x, s, w.bfloat16(), dy, None, dr, dx, ds, dw)


def test_slot_marshalling(rec, monkeypatch):  # noqa: F811
    monkeypatch.setattr(g, "_check_pool", lambda S, H, K, V, device: g._slot_stride(S))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    n, H, K, V = 6, 2, 128, 64
    q, k, b, v, w, o = bf(n, H, K), bf(n, H, K), bf(n, H, K), bf(n, H, V), bf(n, H, V), bf(n, H, V)
    alpha, pool = torch.zeros(n, H, K), torch.zeros(4, 3, H, K, V)
    layer = pool[:, 1]                       # one layer's part: slots a layer apart
    slots, cu, par = i32(3, 0), i32(0, 4, 6), i32(-1, 0, 0, 1, -1, -1)
    g.gdn2_tree_fwd(q, k, v, alpha, b, w, layer, slots, cu, par, o, 4)
    name, a = rec.calls[-1]
    assert name == "gdn2_tree_fwd"
    assert [addr(p) for p in a[:7]] == [t.data_ptr() for t in (q, k, v, alpha, b, w, layer)]
    assert a[7:9] == (3 * H * K * V, 4) and [addr(p) for p in a[9:13]] == [t.data_ptr() for t in (slots, cu, par, o)]
    assert a[13:20] == (2, H, n, 4, K, V, g.GDN2_BF16) and a[21] >= 256
    index = i32(5, 4, 0)
    cu = i32(0, 1, 3)
    o = bf(3, H, V)
    g.gdn2_recurrent_fwd(q, k, v, alpha, b, w, layer, slots, slots, cu, index, o)
    _, a = rec.calls[-1]
    assert [addr(p) for p in a[9:14]] == [t.data_ptr() for t in (slots, slots, cu, index, o)]
    assert a[14:21] == (2, H, 3, n, K, V, g.GDN2_BF16)
    with pytest.raises(ValueError):
        g.gdn2_recurrent_fwd(q, k, v, alpha, b, w, layer, slots, slots, cu, None, o)     # o is not one row an entry
    with pytest.raises(TypeError):
        g.gdn2_recurrent_fwd(q, k, v, alpha, b, w, layer, slots.long(), slots, cu, index, o)
    with pytest.raises(ValueError):
        g.gdn2_tree_fwd(q, k, v, alpha, b, w, layer, slots, cu[:2], par, bf(n, H, V), 4)


def test_slot_stride_refuses_overlap():
    pool = torch.zeros(4, 2, 64, 64)
    assert g._slot_stride(pool) == 2 * 64 * 64 and g._slot_stride(pool[::2]) == 4 * 64 * 64
    with pytest.raises(ValueError):
        g._slot_stride(pool[:1].expand(4, 2, 64, 64))
    with pytest.raises(ValueError):
        g._slot_stride(pool.transpose(2, 3))


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        g.gdn2_gated_norm(x, x, torch.ones(64))
    with pytest.raises(ValueError):
        g.gdn2_add_norm(x, x, torch.ones(64))
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.gdn2_state_copy(x, x, i, i)
