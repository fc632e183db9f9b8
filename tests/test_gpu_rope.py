"""Rotary positions: the table against float64, the rotation with the cache
write bit for bit against the oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import oracle.sparse as osp
from sparse_helpers import SUFFIX, dev, normal
from tree_helpers import CODEC, DT

pytestmark = pytest.mark.gpu

SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
            dict(scaling="bands", factor=16.0, original_len=8192), dict(scaling="ramp", factor=4.0, original_len=4096),
            dict(scaling="bands", factor=2.0, original_len=100, low=0.5, high=3.0, base=500000.0)]

# The header's bound: x is off by its rounding, the polynomials' by theirs (a
# few half steps of 1) and the series' next term, 2^-28.
TABLE_ERROR = 2.0 ** -22


@pytest.mark.parametrize("how", range(len(SCALINGS)))
@pytest.mark.parametrize("first,positions,rot", [(0, 1, 2), (0, 300, 128), (1, 77, 34), (131000, 200, 64),
                                                 (2 ** 20 - 5, 9, 256), (2 ** 31 - 3, 3, 96)])
def test_table(lib, how, first, positions, rot):
    kw = SCALINGS[how]
    got = lib.pa_rope_table(positions, rot, first_position=first, **kw).cpu().double().numpy()
    freqs = osp.rope_frequencies(rot, **kw)
    ref = osp.rope_table(first, positions, freqs)
    # float64's own angle is off by half a step of it, and so is a frequency.
    own = (first + positions) * freqs.max() * 2.0 ** -51
    assert np.abs(got - ref).max() <= TABLE_ERROR + own


def test_table_amplitude_and_whole_turns(lib):
    out = lib.pa_rope_table(5, 8, amplitude=1.25)
    ref = osp.rope_table(0, 5, osp.rope_frequencies(8), 1.25)
    assert np.abs(out.cpu().double().numpy() - ref).max() <= 1.25 * TABLE_ERROR + 2.0 ** -24
    assert torch.equal(out[0], torch.tensor([1.25] * 4 + [0.0] * 4).cuda())
    assert lib.pa_rope_table(0, 8).shape == (0, 8)
    # Parts of a table are the whole's rows.
    whole = lib.pa_rope_table(1000, 128)
    assert torch.equal(whole[700:], lib.pa_rope_table(300, 128, first_position=700))


def tokens(seed, seqs, hq, hkv, d, block, dtype, pad=True, fused=True, most=3):
    """New tokens of ragged sequences: (q, k, v), positions, slots, pool size."""
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, 100, seqs)
    new = rng.integers(1, most, seqs)
    blocks = [-(-int(a + b) // block) for a, b in zip(ctx, new)]
    P = sum(blocks) + 2
    perm = rng.permutation(P)
    pos, slots, at = [], [], 0
    for a, b, nb in zip(ctx, new, blocks):
        for x in range(a, a + b):
            pos.append(x)
            slots.append(int(perm[at + x // block]) * block + x % block)
        at += nb
    T = len(pos)
    if fused:
        qkv = normal(rng, T, hq + 2 * hkv, d).to(DT[dtype])
        q, k, v = qkv.split([hq, hkv, hkv], 1)
    else:
        q, k, v = (normal(rng, T, h, d).to(DT[dtype]) for h in (hq, hkv, hkv))
    slots = np.array(slots, np.int64)
    if pad and T > 2:
        slots[T // 2] = -1
    return rng, (q, k, v), np.array(pos, np.int32), slots, P


def on_device(qkv):
    """The same parts of one tensor on the device."""
    q, k, v = qkv
    if q.data_ptr() + q.shape[1] * q.shape[2] * q.element_size() == k.data_ptr():
        whole = torch.cat([q, k, v], 1).cuda()
        return whole.split([q.shape[1], k.shape[1], v.shape[1]], 1)
    return tuple(x.cuda() for x in qkv)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,rot", [(8, 2, 64, 64), (32, 8, 128, 128), (4, 4, 128, 64), (6, 2, 96, 24),
                                          (3, 1, 80, 20), (5, 5, 128, 2), (2, 1, 256, 256), (7, 1, 64, 46)])
def test_rotation_and_cache(lib, interleaved, dtype, hq, hkv, d, rot):
    rng, qkv, pos, slots, P = tokens(1, 9, hq, hkv, d, 16, dtype)
    cs = osp.rope_table(0, 128, osp.rope_frequencies(rot)).astype(np.float32)
    k0, v0 = normal(rng, P, hkv, 16, d).to(DT[dtype]), normal(rng, P, hkv, 16, d).to(DT[dtype])
    kd, vd = dev(k0, v0)
    q, k, v = on_device(qkv)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    got = lib.pa_rope_and_cache(q, k, v, *dev(pos, slots, cs), kd, vd, interleaved=interleaved, q_out=out)
    assert lib.pa_get_status() == 0 and got is out
    ref = torch.from_numpy(osp.rotate(qkv[0], cs, pos, interleaved)).to(DT[dtype])
    ref[slots < 0] = 7.0  # a padded token's row stays
    assert torch.equal(got.cpu(), ref)
    oracle.reshape_and_cache(torch.from_numpy(osp.rotate(qkv[1], cs, pos, interleaved)).to(DT[dtype]), qkv[2], slots,
                             k0, v0, 16)
    assert torch.equal(kd.cpu(), k0) and torch.equal(vd.cpu(), v0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,fmt", [("bf16", "e4m3"), ("f16", "e5m2"), ("f32", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("hq,hkv,d,rot", [(8, 2, 64, 64), (32, 8, 128, 128), (4, 4, 128, 64), (6, 1, 128, 46),
                                          (0, 2, 64, 20)])
@pytest.mark.parametrize("most,block", [(2, 16), (40, 16), (90, 32)])
def test_rotation_and_8bit_cache(lib, interleaved, dtype, fmt, hq, hkv, d, rot, most, block):
    rng, qkv, pos, slots, P = tokens(2, 7, hq, hkv, d, block, dtype, most=most)
    cs = osp.rope_table(0, 256, osp.rope_frequencies(rot)).astype(np.float32)
    fine = np.arange(256, dtype=np.uint8)
    fine = fine[np.isfinite(CODEC[fmt][0](fine))]
    k0, v0 = (rng.choice(fine, size=(P, hkv, block, d)) for _ in range(2))
    sc = np.exp2(rng.uniform(-12, -4, (P, hkv, 2))).astype(np.float32)
    kd, vd, sd = dev(k0.copy(), v0.copy(), sc.copy())
    q, k, v = on_device(qkv)
    call = getattr(lib, "pa_rope_and_cache" + SUFFIX[fmt])
    got = call(q if hq else None, k, v, *dev(pos, slots, cs), kd, vd, sd, interleaved=interleaved)
    assert lib.pa_get_status() == 0
    live = slots >= 0
    if hq:
        ref = torch.from_numpy(osp.rotate(qkv[0], cs, pos, interleaved)).to(DT[dtype])
        assert torch.equal(got.cpu()[live], ref[live])
    else:
        assert got is None
    osp.cache_write_8bit(fmt, osp.rotate(qkv[1], cs, pos, interleaved), qkv[2].float().numpy(), slots, k0, v0, sc, block)
    assert np.array_equal(sd.cpu().numpy(), sc)
    assert np.array_equal(kd.cpu().numpy(), k0) and np.array_equal(vd.cpu().numpy(), v0)


def test_rotation_in_place_and_far_positions(lib):
    rng, qkv, pos, slots, P = tokens(3, 12, 16, 4, 128, 16, "bf16", pad=False, fused=False)
    far = (pos.astype(np.int64) + 130900).astype(np.int32)
    cs = lib.pa_rope_table(131072, 128, base=500000.0)
    kd, vd = (torch.zeros(P, 4, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (x.cuda() for x in qkv)
    lib.pa_rope_and_cache(q, k, v, *dev(far, slots), cs, kd, vd, q_out=q)
    assert lib.pa_get_status() == 0
    assert torch.equal(q.cpu(), torch.from_numpy(osp.rotate(qkv[0], cs.cpu().numpy(), far, False)).bfloat16())


def test_many_tokens(lib):
    """A prompt's worth, each token in its place."""
    T, hq, hkv, d = 5000, 8, 2, 64
    rng = np.random.default_rng(4)
    q, k, v = (normal(rng, T, h, d).half() for h in (hq, hkv, hkv))
    slots = rng.permutation(T + 64)[:T].astype(np.int64)
    P = (T + 64 + 15) // 16
    pos = np.arange(T, dtype=np.int32)
    cs = osp.rope_table(0, T, osp.rope_frequencies(d)).astype(np.float32)
    kd, vd = (torch.zeros(P, hkv, 16, d, dtype=torch.float16, device="cuda") for _ in range(2))
    got = lib.pa_rope_and_cache(*dev(q, k, v, pos, slots, cs), kd, vd)
    assert lib.pa_get_status() == 0
    assert torch.equal(got.cpu(), torch.from_numpy(osp.rotate(q, cs, pos, False)).half())
    kr = torch.from_numpy(osp.rotate(k, cs, pos, False)).half()
    flat = lambda x: x.cpu().transpose(1, 2).reshape(-1, hkv, d)[slots]  # noqa: E731
    assert torch.equal(flat(kd), kr) and torch.equal(flat(vd), v)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_bad_slots_and_positions(lib, fmt):
    """A token without a place or a position is reported and skipped; the others are written."""
    T, hq, hkv, d, P = 6, 4, 2, 64, 6
    rng = np.random.default_rng(5)
    q, k, v = (normal(rng, T, h, d).bfloat16() for h in (hq, hkv, hkv))
    cs = osp.rope_table(0, 50, osp.rope_frequencies(d)).astype(np.float32)
    ok_slots, ok_pos = np.arange(T, dtype=np.int64) * 16, np.arange(T, dtype=np.int32)
    dt = torch.bfloat16 if fmt is None else torch.uint8
    for slot, pos, code in ((P * 16, 2, -7), (2 ** 40, 2, -7), (32, 50, -8), (32, -1, -8)):
        slots, posn = ok_slots.copy(), ok_pos.copy()
        slots[2], posn[2] = slot, pos
        kd, vd = (torch.zeros(P, hkv, 16, d, dtype=dt, device="cuda") for _ in range(2))
        out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        sc = () if fmt is None else (torch.ones(P, hkv, 2, device="cuda"),)
        getattr(lib, "pa_rope_and_cache" + SUFFIX[fmt])(*dev(q, k, v, posn, slots, cs), kd, vd, *sc, q_out=out)
        assert lib.pa_get_status() == code and lib.pa_get_status() == 0
        ref = torch.from_numpy(osp.rotate(q, cs, np.clip(posn, 0, 49), False)).bfloat16()
        ref[2] = 7.0
        assert torch.equal(out.cpu(), ref)
        written = (kd != 0).flatten(1).any(1).cpu().tolist()
        assert written == [True, True, False, True, True, True]


def test_other_stream_and_graph(lib):
    rng, qkv, pos, slots, P = tokens(6, 20, 8, 2, 128, 16, "bf16", pad=False, fused=False)
    cs = lib.pa_rope_table(128, 128)
    q, k, v = (x.cuda() for x in qkv)
    pools = [torch.zeros(P, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    pd, sd = dev(pos, slots)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = lib.pa_rope_and_cache(q, k, v, pd, sd, cs, pools[0], pools[1], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    held = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.pa_rope_and_cache(q, k, v, pd, sd, cs, pools[2], pools[3], q_out=held)
    q.copy_(q.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert lib.pa_get_status() == 0
    ref = torch.from_numpy(osp.rotate(qkv[0], cs.cpu().numpy(), pos, False)).bfloat16()
    assert torch.equal(out.cpu(), ref)
    assert torch.equal(held.cpu(), torch.from_numpy(osp.rotate(qkv[0].flip(0), cs.cpu().numpy(), pos, False)).bfloat16())
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    t = lib.pa_rope_table(64, 128, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(t, cs[:64])
