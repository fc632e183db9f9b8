"""Host checks of the draft-tree calls: a refused call launches nothing (no
GPU needed), and the binding's own checks."""
from __future__ import annotations

import ctypes

import pytest
import torch

import paged_kv_cache_14_gb300 as pa


@pytest.fixture(scope="module")
def lib():
    return pa.load()


def _tree(lib, name="pa_decode_tree", **over):
    a = dict(q=0x1000, tq=12, cu=0x1100, par=0x1200, k=0x2000, v=0x3000, sc=0x3100, bt=0x4000, mb=8, ctx=0x5000, n=3,
             mq=8, mkv=100, hq=8, hkv=2, d=128, bs=16, nb=10, scale=0.1, out=0x6000, ws=None, wsb=0, dt=pa.PA_BF16,
             stream=None)
    a.update(over)
    if name == "pa_decode_tree":
        a.pop("sc")
    return getattr(lib, name)(*a.values())


NO_WORKSPACE = -5  # what a call that passes every other check answers here


def test_tree_host_checks(lib):
    for name in ("pa_decode_tree", "pa_decode_tree_fp8", "pa_decode_tree_e5m2"):
        go = lambda **o: _tree(lib, name, **o)  # noqa: E731
        assert go() == NO_WORKSPACE
        assert go(ws=0x7000, wsb=10) == NO_WORKSPACE
        assert go(hq=9) == -3
        assert go(bs=8) == -4
        assert go(dt=5) == -2
        assert go(d=96) == -10
        assert go(hq=258, hkv=2) == -10                   # group 129
        assert go(hq=256, hkv=2) == NO_WORKSPACE
        assert go(n=65536) == -10 and go(n=65535) == NO_WORKSPACE
        assert go(mq=1025) == -10 and go(mq=1024) == NO_WORKSPACE
        assert go(nb=2 ** 27) == -10
        for name2 in ("q", "cu", "par", "k", "v", "bt", "ctx", "out"):
            assert go(**{name2: None}) == -1
        for name2 in ("q", "k", "v", "out"):
            assert go(**{name2: 0x9004}) == -12
        for over in (dict(n=-1), dict(tq=-1), dict(mb=0), dict(nb=0), dict(mq=0), dict(mkv=0), dict(hkv=0),
                     dict(scale=float("inf")), dict(scale=0.0), dict(scale=-1.0)):
            assert go(**over) == -1, over
        assert go(n=0) == 0 and go(tq=0) == 0
        assert go(ws=0x7008, wsb=1 << 40) == -12
    assert _tree(lib, "pa_decode_tree_fp8", sc=None) == -1
    assert _tree(lib, "pa_decode_tree_fp8", sc=0x3104) == -12
    assert _tree(lib, "pa_decode_tree_fp8", d=64) == -10
    assert _tree(lib, "pa_decode_tree_fp8", dt=pa.PA_F32) == -2
    assert _tree(lib, dt=pa.PA_F32, d=96, scale=-1.0) == NO_WORKSPACE
    assert _tree(lib, dt=pa.PA_F32, d=288) == -10


def test_tree_workspace(lib):
    size = pa.pa_decode_tree_workspace_size
    assert size(0, 8, 2, 128, 16, 0, 8, 100) == 0
    small = size(1, 8, 8, 128, 16, 1, 1, 10)
    large = size(64, 64, 8, 128, 16, 4096, 64, 100000)
    assert 0 < small < large < 1 << 28
    # It does not grow with the context once the machine is full.
    assert large == size(64, 64, 8, 128, 16, 4096, 64, 10 ** 6)
    assert size(1, 9, 8, 128, 16, 1, 1, 10) == 0  # refused


def _verify(lib, **over):
    a = dict(t=0x1000, ts=100, d=0x2000, ds=100, tok=0x3000, cu=0x3100, par=0x3200, ua=0x3300, us=0x3400, n=2, tq=9,
             mq=8, v=100, mp=8, path=0x4000, lens=0x4100, nxt=0x4200, dt=pa.PA_F32, stream=None)
    a.update(over)
    return lib.pa_verify_tree(*a.values())


def test_verify_host_checks(lib):
    for over in (dict(n=-1), dict(tq=-1), dict(v=0), dict(mp=0), dict(mq=-1), dict(ts=99), dict(ds=99), dict(t=None),
                 dict(tok=None), dict(cu=None), dict(par=None), dict(ua=None), dict(us=None), dict(path=None),
                 dict(lens=None), dict(nxt=None)):
        assert _verify(lib, **over) == -1, over
    assert _verify(lib, dt=3) == -2
    assert _verify(lib, v=262145, ts=262145, ds=262145) == -10
    assert _verify(lib, mq=1025) == -10
    for over in (dict(t=0x1002), dict(d=0x2001), dict(t=0x1001, dt=pa.PA_F16)):
        assert _verify(lib, **over) == -12, over
    assert _verify(lib, n=0) == 0


def _compact(lib, name="pa_compact_tree", **over):
    two = (ctypes.c_void_p * 2)
    a = dict(k=two(0x1000, 0x2000), v=two(0x3000, 0x4000), sc=two(0x5000, 0x5100), layers=2, bt=0x6000, mb=8,
             ctx=0x6100, path=0x6200, lens=0x6300, n=3, mp=8, nb=10, bs=16, hkv=2, d=64, dt=pa.PA_BF16, stream=None)
    a.update(over)
    a.pop("sc" if name == "pa_compact_tree" else "dt")
    return getattr(lib, name)(*a.values())


def test_compact_host_checks(lib):
    two = (ctypes.c_void_p * 2)
    for name in ("pa_compact_tree", "pa_compact_tree_fp8", "pa_compact_tree_e5m2"):
        go = lambda **o: _compact(lib, name, **o)  # noqa: E731
        for over in (dict(n=-1), dict(layers=-1), dict(mb=0), dict(nb=0), dict(hkv=0), dict(d=0), dict(mp=0),
                     dict(k=None), dict(v=None), dict(bt=None), dict(ctx=None), dict(path=None), dict(lens=None),
                     dict(k=two(0x1000, None))):
            assert go(**over) == -1, over
        assert go(bs=4) == -4
        assert go(mp=1025) == -10
        assert go(v=two(0x1000, 0x1008)) == -12
        assert go(n=0) == 0 and go(layers=0) == 0
    assert _compact(lib, d=4) == -10 and _compact(lib, dt=9) == -2
    assert _compact(lib, "pa_compact_tree_fp8", d=32) == -10
    assert _compact(lib, "pa_compact_tree_fp8", sc=two(0x5000, None)) == -1
    assert _compact(lib, "pa_compact_tree_fp8", sc=two(0x5000, 0x5002)) == -12


def test_binding_refuses_host_tensors():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i32 = torch.int32
    with pytest.raises(TypeError, match="CUDA"):
        pa.pa_decode_tree(z(4, 8, 128), z(2, dt=i32), z(4, dt=i32), z(3, 2, 16, 128), z(3, 2, 16, 128), z(1, 3, dt=i32),
                          z(1, dt=i32), 4, 20, 0.1, out=z(4, 8, 128), workspace=z(16, dt=torch.uint8))
    with pytest.raises(TypeError, match="CUDA"):
        pa.pa_verify_tree(z(4, 10), None, z(4, dt=i32), z(2, dt=i32), z(4, dt=i32), z(4), z(1), 4, 4)
    with pytest.raises(TypeError, match="CUDA"):
        pa.pa_compact_tree([z(3, 2, 16, 64)], [z(3, 2, 16, 64)], z(1, 3, dt=i32), z(1, dt=i32), z(1, 4, dt=i32),
                           z(1, dt=i32))


def test_binding_refuses_layer_lists():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i32 = torch.int32
    with pytest.raises(ValueError, match="same layers"):
        pa.pa_compact_tree([z(3, 2, 16, 64)], [], z(1, 3, dt=i32), z(1, dt=i32), z(1, 4, dt=i32), z(1, dt=i32))


def test_tree_workspace_at_the_largest_bounds():
    """Bounds up to 2^31 - 1 do not wrap: the workspace is that of a full machine."""
    size = pa.pa_decode_tree_workspace_size
    for dtype in (torch.bfloat16, torch.float32):
        full = size(64, 64, 8, 128, 16, 4096, 64, 10 ** 6, dtype)
        for bound in (2 ** 31 - 64, 2 ** 31 - 63, 2 ** 31 - 32, 2 ** 31 - 1):
            assert size(64, 64, 8, 128, 16, 4096, 64, bound, dtype) == full


def test_tree_pool_sizes(lib):
    """Pools of 2^31 rows: refused where tensor maps address them, taken by
    the fp32 call, whose offsets are 64-bit."""
    for nb, hkv in ((2 ** 27, 2), (2 ** 26, 2), (2 ** 27, 1)):
        assert _tree(lib, nb=nb, hkv=hkv) == -10
        assert _tree(lib, "pa_decode_tree_fp8", nb=nb, hkv=hkv) == -10
        assert _tree(lib, nb=nb, hkv=hkv, dt=pa.PA_F32) == NO_WORKSPACE
    assert _tree(lib, nb=2 ** 26 - 1, hkv=2) == NO_WORKSPACE


def test_compact_refuses_pools_listed_twice(lib):
    """Two layers that share a pool, or a layer's K and V, would be moved twice."""
    two, many = ctypes.c_void_p * 2, ctypes.c_void_p * 200
    for name in ("pa_compact_tree", "pa_compact_tree_fp8", "pa_compact_tree_e5m2"):
        go = lambda **o: _compact(lib, name, **o)  # noqa: E731
        assert go(k=two(0x1000, 0x1000)) == -1
        assert go(v=two(0x3000, 0x3000)) == -1
        assert go(v=two(0x3000, 0x1000)) == -1
        far = [0x100000 + 0x100 * i for i in range(400)]
        far[399] = far[0]  # a V pool of another launch's layer
        assert go(layers=200, k=many(*far[:200]), v=many(*far[200:]),
                  sc=many(*[0x900000 + 0x10 * i for i in range(200)])) == -1
    assert _compact(lib, "pa_compact_tree_fp8", sc=two(0x5000, 0x5000)) == -1
