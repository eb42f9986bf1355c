"""Argument checks of the norms and of the operators over a state cache, on the CPU: the C entry points
refuse before they touch the device, and the binding names what is wrong with a tensor."""
import ctypes

import pytest
import torch

import gated_delta_rule_96_b200 as g

P = ctypes.c_void_p
F = P(0x10000)       # never dereferenced: every call below fails validation first or has nothing to do
ODD = P(0x10004)
at = lambda floats: P(0x10000 + 4 * floats)  # noqa: E731


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
    # two caches of 4 slots of 64 floats that share memory (a later part of one, from the end of one slot into the
    # next, the last slot alone, other strides), and ones that do not (behind, before, between one another)
    (lambda l: copy(l, src=at(64)), -2), (lambda l: copy(l, src=at(-64)), -2), (lambda l: copy(l, src=at(192), snum=1), -2),
    (lambda l: copy(l, dstride=128, sstride=128, src=at(60)), -2), (lambda l: copy(l, dstride=128, sstride=128, src=at(-60)), -2),
    (lambda l: copy(l, dstride=128, sstride=64, src=at(64), pairs=0), -2),
    (lambda l: copy(l, dnum=1, snum=1, src=at(60), pairs=0), -2), (lambda l: copy(l, src=at(256), pairs=0), 0),
    (lambda l: copy(l, src=at(-256), pairs=0), 0), (lambda l: copy(l, dstride=128, sstride=128, src=at(64), pairs=0), 0),
    (lambda l: copy(l, dstride=128, sstride=128, src=at(-64), pairs=0), 0),
    (lambda l: copy(l, dnum=1, sstride=128, src=at(-64), pairs=0), 0), (lambda l: copy(l, dnum=1, sstride=128, src=at(-128)), -2),
    (lambda l: copy(l, snum=0, src=at(64), pairs=0), 0),
])
def test_entry_points_refuse(lib, call, want):
    assert call(lib) == want
    assert g.gdn2_status_str(want) != "unknown status"


@pytest.mark.parametrize("change,want", [
    # one slot has no stride: the first slot of a cache, with the cache's own stride or any other, is part of that cache
    (dict(dnum=1, dstride=64, sstride=128), 0), (dict(snum=1, sstride=64, dstride=128), 0), (dict(dnum=1, snum=1, dstride=128), 0),
    (dict(dnum=1, dstride=4096, sstride=128), 0), (dict(dnum=0, sstride=128), 0),
    # two of one address with more slots each and other strides share memory without being one
    (dict(dnum=2, snum=2, dstride=128), -2), (dict(dnum=2, dstride=64, sstride=128), -2)])
def test_state_copy_of_a_one_slot_part(lib, change, want):
    assert copy(lib, pairs=0, **change) == want


def test_wait_limit(lib):
    assert [lib.gdn2_set_wait_limit(n) for n in (-2, 1 << 32, 0, (1 << 32) - 1, -1)] == [-10, -10, 0, 0, 0]
    with pytest.raises(g.GDN2Error):
        g.gdn2_set_wait_limit(-5)


def test_workspace_sizes():
    assert g.gdn2_gated_norm_bwd_workspace_bytes(-1, 128) == 0 and g.gdn2_gated_norm_bwd_workspace_bytes(4, 96) == 0
    assert g.gdn2_gated_norm_bwd_workspace_bytes(0, 128) >= 256 + 4 * 128
    assert g.gdn2_add_norm_bwd_workspace_bytes(4, 12) == 0 and g.gdn2_add_norm_bwd_workspace_bytes(-1, 16) == 0
    # bounded: at most 592 blocks write partial sums, whatever the number of rows
    assert g.gdn2_gated_norm_bwd_workspace_bytes(1 << 40, 128) <= 256 + 592 * 128 * 4
    assert g.gdn2_add_norm_bwd_workspace_bytes(1 << 40, 8192) <= 256 + 592 * 2 * 8192 * 4


# The binding: types and shapes are refused first, wherever the tensors are, then tensors that are not on the GPU.

BF = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
I32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
NO_CUDA = "must be CUDA tensors"


def norm_args(**change):
    a = dict(o=BF(2, 3, 64), gate=BF(2, 3, 64), weight=torch.ones(64), y=BF(2, 3, 64))
    return g.gdn2_gated_norm_fwd(**(a | change))


def norm_bwd_args(**change):
    a = dict(o=BF(6, 64), gate=BF(6, 64), weight=torch.ones(64), dy=BF(6, 64), do=BF(6, 64), dgate=BF(6, 64),
             dweight=torch.ones(64), workspace=torch.zeros(256, dtype=torch.uint8))
    return g.gdn2_gated_norm_bwd(**(a | change))


def add_args(**change):
    a = dict(x=torch.zeros(5, 96), residual=None, scale=None, weight=torch.ones(96), h=None, y=torch.zeros(5, 96))
    return g.gdn2_add_norm_fwd(**(a | change))


def add_bwd_args(**change):
    z, one = torch.zeros(5, 96), torch.ones(96)
    a = dict(h=z, x=z, scale=one, weight=one, dy=z, dh=None, dresidual=z, dx=z, dscale=one, dweight=one,
             workspace=torch.zeros(256, dtype=torch.uint8))
    return g.gdn2_add_norm_bwd(**(a | change))


def token_args(n=6, H=2, K=128, V=64):
    return dict(q=BF(n, H, K), k=BF(n, H, K), v=BF(n, H, V), alpha=torch.zeros(n, H, K), b=BF(n, H, K), w=BF(n, H, V),
                S=torch.zeros(4, 3, H, K, V)[:, 1], workspace=torch.zeros(256, dtype=torch.uint8))


def tree_args(**change):
    a = token_args() | dict(slots=I32(3, 0), cu_nodes=I32(0, 4, 6), parents=I32(-1, 0, 0, 1, -1, -1), o=BF(6, 2, 64),
                            max_nodes=4)
    return g.gdn2_tree_fwd(**(a | change))


def recurrent_args(**change):
    a = token_args() | dict(slots_in=I32(3, 0), slots_out=I32(1, 0), cu_tokens=I32(0, 1, 3), index=I32(5, 4, 0), o=BF(3, 2, 64))
    return g.gdn2_recurrent_fwd(**(a | change))


def copy_args(**change):
    a = dict(dst=torch.zeros(4, 2, 64), src=torch.zeros(9, 2, 64), dst_index=I32(0, 1), src_index=I32(5, -1),
             workspace=torch.zeros(256, dtype=torch.uint8))
    return g.gdn2_state_copy(**(a | change))


@pytest.mark.parametrize("call,change,error,text", [
    (norm_args, {}, ValueError, NO_CUDA), (norm_args, {"act": "tanh"}, ValueError, "act must be one of"),
    (norm_args, {"gate": torch.zeros(2, 3, 64)}, TypeError, "gate must be bfloat16"),
    (norm_args, {"weight": torch.ones(128)}, ValueError, "weight has shape"),
    (norm_args, {"weight": BF(64)}, TypeError, "weight must be float32"),
    (norm_args, {"o": torch.zeros(2, 3, 64, dtype=torch.float16)}, TypeError, "bfloat16 or float32"),
    (norm_args, {"y": None}, TypeError, "outputs"), (norm_args, {"y": BF(6, 64)}, ValueError, "y has shape"),
    (norm_args, {"o": 3}, TypeError, "o must be a tensor"), (norm_args, {"eps": "a"}, TypeError, "real number"),
    (norm_bwd_args, {}, ValueError, NO_CUDA), (norm_bwd_args, {"dweight": BF(64)}, TypeError, "dweight must be float32"),
    (norm_bwd_args, {"dgate": BF(6, 32)}, ValueError, "dgate has shape"),
    (norm_bwd_args, {"do": None}, TypeError, "outputs"),
    (add_args, {}, ValueError, NO_CUDA), (add_args, {"residual": torch.zeros(4, 96)}, ValueError, "residual has shape"),
    (add_args, {"h": BF(5, 96)}, TypeError, "h must be float32"), (add_args, {"y": None}, TypeError, "y must be a tensor"),
    (add_args, {"scale": torch.ones(95)}, ValueError, "scale has shape"),
    (add_bwd_args, {}, ValueError, NO_CUDA), (add_bwd_args, {"weight": BF(96)}, TypeError, "weight must be float32"),
    (add_bwd_args, {"dh": torch.zeros(5, 95)}, ValueError, "dh has shape"),
    (tree_args, {}, ValueError, NO_CUDA), (tree_args, {"cu_nodes": I32(0, 4)}, ValueError, "cu_nodes has shape"),
    (tree_args, {"parents": I32(-1)}, ValueError, "parents has shape"),
    (tree_args, {"slots": torch.zeros(2, dtype=torch.int64)}, TypeError, "slots must be a one-dimensional int32"),
    (tree_args, {"S": torch.zeros(4, 2, 64, 128)}, ValueError, "S has shape"),
    (tree_args, {"S": BF(4, 2, 128, 64)}, TypeError, "S must be float32"),
    (tree_args, {"S": torch.zeros(1, 2, 128, 64).expand(4, 2, 128, 64)}, ValueError, "must not overlap"),
    (tree_args, {"S": torch.zeros(4, 2, 64, 128).transpose(2, 3)}, ValueError, "must be contiguous"),
    (tree_args, {"k": BF(6, 2, 64)}, ValueError, "k has shape"), (tree_args, {"v": BF(6, 2)}, ValueError, "v has shape"),
    (tree_args, {"alpha": BF(6, 2, 128)}, TypeError, "alpha must be float32"), (tree_args, {"o": None}, TypeError, "outputs"),
    (tree_args, {"max_nodes": 1 << 40}, ValueError, "max_nodes"), (tree_args, {"max_nodes": 1.5}, TypeError, "integer"),
    (recurrent_args, {}, ValueError, NO_CUDA), (recurrent_args, {"index": None}, ValueError, "o has shape"),
    (recurrent_args, {"o": None}, ValueError, NO_CUDA),
    (recurrent_args, {"slots_out": I32(1)}, ValueError, "slots_out has shape"),
    (recurrent_args, {"cu_tokens": I32(0, 1)}, ValueError, "cu_tokens has shape"),
    (copy_args, {}, ValueError, NO_CUDA), (copy_args, {"src": torch.zeros(9, 2, 32)}, ValueError, "src has shape"),
    (copy_args, {"src_index": I32(0)}, ValueError, "src_index has shape"),
    (copy_args, {"dst": torch.zeros(4)}, ValueError, "dst has shape"), (copy_args, {"dst": BF(4, 2, 64)}, TypeError, "float32"),
])
def test_binding_refuses(call, change, error, text):
    with pytest.raises(error, match=text):
        call(**change)


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        g.gdn2_gated_norm(x, x, torch.ones(64))
    with pytest.raises(ValueError):
        g.gdn2_add_norm(x, x, torch.ones(64))
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.gdn2_state_copy(x, x, i, i)


def test_native_half_is_rebuilt_when_it_has_to_be(monkeypatch, tmp_path):
    """For a newer source, another torch or another Python; not otherwise."""
    import os
    import sys

    from gated_delta_rule_96_b200 import build
    source, made = tmp_path / "gdn2_torch.cpp", []
    source.write_text("")
    os.utime(source, (1, 1))
    monkeypatch.setattr(build, "TORCH_SOURCE", str(source))
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path))
    (tmp_path / "gdn2.h").write_text("")
    os.utime(tmp_path / "gdn2.h", (1, 1))
    monkeypatch.setattr(build, "TORCH_LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "TORCH_STAMP", str(tmp_path / "made" / "stamp"), raising=False)

    def compile_(cmd):
        made.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
    monkeypatch.setattr(build.subprocess, "check_call", compile_)

    def built():
        made.clear()
        assert build.build_torch() == build.TORCH_LIB and os.path.exists(build.TORCH_LIB)
        return len(made)
    assert built() == 1 and built() == 0
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert built() == 1 and built() == 0
    monkeypatch.setattr(sys, "version", "another one")
    assert built() == 1 and built() == 0
    os.utime(source)
    os.utime(build.TORCH_LIB, (2, 2))
    assert built() == 1 and built() == 0
