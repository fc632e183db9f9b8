"""Host checks of the long-context calls: a refused call launches nothing (no
GPU needed), and the binding's own checks."""
from __future__ import annotations

import pytest
import torch

import paged_kv_cache_14_gb300 as pa
from paged_kv_cache_14_gb300.step import SparseStep


@pytest.fixture(scope="module")
def lib():
    return pa.load()


# Calls with an argument that the last check refuses: what passes every other
# check answers that check's code, and none gets as far as a launch.
def _table(lib, **over):
    a = dict(out=0x1000, first=0, n=0, rot=128, base=1e4, kind=0, factor=1.0, orig=0, low=1.0, high=4.0, amp=1.0,
             stream=None)
    a.update(over)
    return lib.pa_rope_table(*a.values())


def test_table_checks(lib):
    assert _table(lib) == 0  # no positions
    for over in (dict(n=-1), dict(first=-1), dict(n=1, first=2 ** 31), dict(n=2 ** 31 - 1, first=2), dict(base=1.0),
                 dict(base=float("nan")), dict(base=float("inf")), dict(kind=5), dict(kind=-1),
                 dict(kind=1, factor=0.0), dict(kind=2, factor=-1.0), dict(kind=1, factor=float("inf")),
                 dict(kind=3, orig=0), dict(kind=3, orig=10, low=4.0), dict(kind=4, orig=10, low=0.0),
                 dict(kind=4, orig=10, high=float("inf")), dict(amp=float("nan")), dict(n=1, out=None)):
        assert _table(lib, **over) == -1, over
    for rot in (0, 1, 3, 258, -2):
        assert _table(lib, rot=rot) == -10
    assert _table(lib, n=1, out=0x1004) == -12
    assert _table(lib, kind=3, orig=8192, factor=8.0) == 0 and _table(lib, kind=4, orig=1, factor=0.5, high=32.0) == 0


def _rope(lib, name="pa_rope_and_cache", **over):
    a = dict(q=0x1000, qs=1024, k=0x2000, ks=256, v=0x3000, vs=256, pos=0x3100, slots=0x3200, cs=0x3300, np=50, rot=128,
             inter=0, t=0, out=0x4000, kc=0x5000, vc=0x6000, sc=0x6100, nb=10, bs=16, hq=8, hkv=2, d=128,
             dt=pa.PA_BF16, stream=None)
    a.update(over)
    if name == "pa_rope_and_cache":
        a.pop("sc")
    return getattr(lib, name)(*a.values())


def test_rope_checks(lib):
    for name in ("pa_rope_and_cache", "pa_rope_and_cache_fp8", "pa_rope_and_cache_e5m2"):
        go = lambda **o: _rope(lib, name, **o)  # noqa: E731
        assert go() == 0
        for over in (dict(t=-1), dict(nb=0), dict(hq=-1), dict(hkv=0), dict(np=0)):
            assert go(**over) == -1, over
        assert go(bs=8) == -4 and go(dt=7) == -2
        for over in (dict(rot=0), dict(rot=3), dict(rot=130), dict(rot=-2)):
            assert go(**over) == -10, over
        for key in ("q", "k", "v", "pos", "slots", "cs", "out", "kc", "vc"):
            assert go(t=1, **{key: None}) == -1, key
        for key in ("q", "k", "v", "cs", "out", "kc", "vc"):
            assert go(t=1, **{key: 0x9004}) == -12, key
        assert go(t=1, ks=255) == -1 and go(t=1, vs=128) == -1 and go(t=1, qs=1023) == -1
        assert go(t=1, ks=257) == -12 and go(t=1, qs=1028) == -12
        assert go(t=1, out=0x1000, qs=1280) == -1   # in place, but rows apart
        assert go(t=2 ** 40) == -10
    assert _rope(lib, d=100, rot=64) == -10 and _rope(lib, d=1032, rot=64) == -10
    assert _rope(lib, d=1024, rot=256) == 0 and _rope(lib, d=1024, rot=258) == -10
    assert _rope(lib, "pa_rope_and_cache_fp8", d=96, rot=64) == -10
    assert _rope(lib, "pa_rope_and_cache_fp8", t=1, sc=None) == -1
    assert _rope(lib, "pa_rope_and_cache_e5m2", t=1, sc=0x6104) == -12


def _summary(lib, name="pa_block_summaries", **over):
    a = dict(k=0x1000, sc=0x1100, bt=0x2000, mb=8, first=0x2100, lens=0x2200, n=0, mn=100, nb=10, bs=16, hkv=2, d=128,
             out=0x3000, os=0x3100, dt=pa.PA_BF16, stream=None)
    a.update(over)
    a.pop("sc" if name == "pa_block_summaries" else "dt")
    return getattr(lib, name)(*a.values())


def test_summary_checks(lib):
    for name in ("pa_block_summaries", "pa_block_summaries_fp8", "pa_block_summaries_e5m2"):
        go = lambda **o: _summary(lib, name, **o)  # noqa: E731
        assert go() == 0 and go(n=3, mn=0) == 0
        for over in (dict(n=-1), dict(mn=-1), dict(mb=0), dict(nb=0), dict(hkv=0)):
            assert go(**over) == -1, over
        assert go(bs=64) == -4
        assert go(d=96) == -10 and go(d=256) == -10
        for key in ("k", "bt", "first", "lens", "out", "os"):
            assert go(n=1, **{key: None}) == -1, key
        for key in ("k", "out", "os"):
            assert go(n=1, **{key: 0x9004}) == -12, key
        assert go(n=2 ** 31 - 1, mn=2 ** 31 - 1, mb=2 ** 31 - 1, hkv=2 ** 20) == -10
    assert _summary(lib, dt=9) == -2
    assert _summary(lib, dt=pa.PA_F32, d=96) == 0 and _summary(lib, dt=pa.PA_F32, d=288) == -10
    assert _summary(lib, "pa_block_summaries_fp8", n=1, sc=None) == -1
    assert _summary(lib, "pa_block_summaries_e5m2", n=1, sc=0x1104) == -12


def _select(lib, **over):
    a = dict(q=0x1000, s=0x2000, ss=0x2100, bt=0x2200, mb=8, lens=0x2300, n=0, maxlen=100, hq=8, hkv=2, d=128, bs=16,
             nb=10, keep=4, sink=1, recent=1, lists=0x3000, ll=0x3100, dt=pa.PA_BF16, stream=None)
    a.update(over)
    return lib.pa_select_blocks(*a.values())


def test_select_checks(lib):
    go = lambda **o: _select(lib, **o)  # noqa: E731
    assert go() == 0 and go(keep=2) == 0
    for over in (dict(n=-1), dict(mb=0), dict(maxlen=0), dict(nb=0), dict(hq=0), dict(hkv=0), dict(keep=0),
                 dict(sink=-1), dict(recent=-1), dict(keep=1), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert go(**over) == -1, over
    assert go(dt=3) == -2 and go(hq=9) == -3 and go(bs=24) == -4
    for over in (dict(d=48), dict(d=288), dict(d=16), dict(hq=258), dict(n=65536)):
        assert go(**over) == -10, over
    assert go(hq=256) == 0 and go(d=256) == 0 and go(d=32) == 0
    for key in ("q", "s", "ss", "bt", "lens", "lists", "ll"):
        assert go(n=1, **{key: None}) == -1, key
    for key in ("q", "s", "ss", "lists", "ll"):
        assert go(n=1, **{key: 0x9004}) == -12, key


def _sparse(lib, name="pa_decode_sparse", **over):
    a = dict(q=0x1000, k=0x2000, v=0x3000, sc=0x3100, bt=0x4000, mb=8, lens=0x4100, lists=0x4200, ll=0x4300, keep=4,
             n=0, hq=8, hkv=2, d=128, bs=16, nb=10, scale=0.1, out=0x5000, dt=pa.PA_BF16, stream=None)
    a.update(over)
    if name == "pa_decode_sparse":
        a.pop("sc")
    return getattr(lib, name)(*a.values())


def test_sparse_checks(lib):
    for name in ("pa_decode_sparse", "pa_decode_sparse_fp8", "pa_decode_sparse_e5m2"):
        go = lambda **o: _sparse(lib, name, **o)  # noqa: E731
        assert go() == 0
        for over in (dict(n=-1), dict(mb=0), dict(keep=0), dict(hq=0), dict(hkv=0), dict(nb=0),
                     dict(scale=float("nan")), dict(scale=float("inf"))):
            assert go(**over) == -1, over
        assert go(dt=4) == -2 and go(hq=9) == -3 and go(bs=17) == -4
        for over in (dict(d=96), dict(hq=258), dict(n=65536), dict(keep=2 ** 26 + 1)):
            assert go(**over) == -10, over
        assert go(hq=256) == 0 and go(scale=-1.0) == 0 and go(scale=0.0) == 0
        for key in ("q", "k", "v", "bt", "lens", "lists", "ll", "out"):
            assert go(n=1, **{key: None}) == -1, key
        for key in ("q", "k", "v", "out"):
            assert go(n=1, **{key: 0x9004}) == -12, key
    assert _sparse(lib, d=64) == 0 and _sparse(lib, "pa_decode_sparse_fp8", d=64) == -10
    assert _sparse(lib, dt=pa.PA_F32, d=96) == 0 and _sparse(lib, dt=pa.PA_F32, d=288) == -10
    assert _sparse(lib, "pa_decode_sparse_e5m2", dt=pa.PA_F32) == -2
    assert _sparse(lib, "pa_decode_sparse_fp8", n=1, sc=None) == -1
    assert _sparse(lib, "pa_decode_sparse_fp8", n=1, sc=0x3104) == -12


def test_binding_refuses_cpu_tensors():
    t = torch.zeros(2, 4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(3, 2, 16, 64)
    with pytest.raises(TypeError):
        pa.pa_rope_and_cache(t, t, t, i, i.long(), t[0], cache, cache)
    with pytest.raises(TypeError):
        pa.pa_block_summaries(cache, i[None], i, i, 4, cache, cache)
    with pytest.raises(TypeError):
        pa.pa_select_blocks(t, cache, cache, i[None], i, 4, 16, 4)
    with pytest.raises(TypeError):
        pa.pa_decode_sparse(t, cache, cache, i[None], i, i[None, None], i[None], 1.0)
    with pytest.raises(ValueError):
        pa.pa_rope_table(4, 64, scaling="stretched")


def test_table_refuses_infinite_frequencies(lib):
    """A factor may take base or a frequency out of the doubles' range: base 0
    makes all but the first frequency infinite, an infinite one makes them 0."""
    assert _table(lib, kind=2, rot=4, factor=1e-200) == -1
    for kind in (1, 3, 4):  # (over one original position no pair makes a turn: all frequencies are scaled)
        assert _table(lib, kind=kind, factor=1e-310, orig=1) == -1, kind
    assert _table(lib, kind=2, rot=4, factor=1e200) == 0
    for kind in (1, 2, 3, 4):
        assert _table(lib, kind=kind, factor=0.25, orig=4096) == 0, kind


@pytest.mark.parametrize("scale", [-0.1, float("nan"), float("inf")])
def test_step_refuses_scales(scale):
    """A negative scale would choose the blocks that weigh least."""
    i32, f32 = (lambda *s: torch.zeros(s, dtype=torch.int32)), (lambda *s: torch.zeros(s))
    step = lambda scale: SparseStep(  # noqa: E731
        k_caches=[f32(4, 1, 16, 32)], v_caches=[f32(4, 1, 16, 32)], block_tables=i32(1, 4), ctx_lens=i32(1),
        seq_lens=i32(1), new_seq_ids=i32(1), new_positions=i32(1), cos_sin=f32(64, 32), num_q_heads=1,
        dtype=torch.float32, max_seq_len=64, max_new_tokens=1, max_list_len=2, scale=scale)
    assert step(0.25).scale == 0.25
    with pytest.raises(ValueError, match="scale"):
        step(scale)
