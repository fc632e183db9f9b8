"""Measured cases of the operators of a long-context decode step over the paged
cache: the table of rotary positions, rotation of queries and keys with the
cache write on the way, summaries of the cached blocks' keys, the choice of
blocks by a cheap score, and attention over the chosen blocks.

Each case names its operator in "op":
  table      cosines and sines of every position, frequencies scaled for long contexts
  rope       new tokens' q rotated, their k rotated and cached, their v cached
  summary    the largest and smallest value of every key dimension of a block, in 8 bits
  select     the blocks of each sequence and KV head that a decode query attends to
  sparse     decode attention over listed blocks
"""
import math

import torch

own = False  # True: run() calls this repository's kernels

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


def listed():
    return [
        # A model's table at start-up, plain frequencies.
        {"name": "table_short", "op": "table", "positions": 8192, "rot": 128, "base": 10000.0, "scaling": "none",
         "factor": 1.0, "original": 8192},
        # The table of a model stretched from 8192 to 131072 positions, band by band.
        {"name": "table_long_bands", "op": "table", "positions": 131072, "rot": 128, "base": 500000.0,
         "scaling": "bands", "factor": 16.0, "original": 8192},
        # One user's decode step: nothing but latency counts.
        {"name": "rope_one_user", "op": "rope", "seqs": 1, "new": 1, "ctx": 5000, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "block": 16, "dtype": "bf16"},
        # Prefill chunks of a mixed batch: pairs side by side, half of each head rotated.
        {"name": "rope_chunks", "op": "rope", "seqs": 16, "new": 1024, "ctx": 16384, "hq": 64, "hkv": 8, "d": 128,
         "rot": 64, "interleaved": True, "block": 32, "dtype": "f16"},
        # A serving batch of a 70B-shaped layer over the 8-bit cache.
        {"name": "rope_batch_e4m3", "op": "rope", "seqs": 256, "new": 1, "ctx": 8192, "hq": 64, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "block": 16, "dtype": "e4m3"},
        # Each decode step: the newest block of every sequence.
        {"name": "summary_step", "op": "summary", "seqs": 64, "new": 1, "ctx": 4096, "hkv": 8, "d": 128, "block": 16,
         "dtype": "bf16"},
        # After a long prompt: all of its blocks.
        {"name": "summary_prompt", "op": "summary", "seqs": 4, "new": 65536, "ctx": 65536, "hkv": 8, "d": 128,
         "block": 16, "dtype": "bf16"},
        # A serving batch of an 8B-shaped layer.
        {"name": "select_batch", "op": "select", "seqs": 64, "ctx": 8192, "keep": 64, "sink": 1, "recent": 2,
         "hq": 32, "hkv": 8, "d": 128, "block": 16, "dtype": "bf16"},
        # Few sequences of a very long context.
        {"name": "select_long", "op": "select", "seqs": 8, "ctx": 131072, "keep": 256, "sink": 1, "recent": 4,
         "hq": 64, "hkv": 8, "d": 128, "block": 16, "dtype": "bf16"},
        # One user of a long document: 64 blocks of it.
        {"name": "sparse_one_user", "op": "sparse", "seqs": 1, "ctx": 32768, "keep": 64, "hq": 32, "hkv": 8, "d": 128,
         "block": 16, "dtype": "bf16"},
        # A serving batch of a 70B-shaped layer, 2048 tokens of each context.
        {"name": "sparse_batch", "op": "sparse", "seqs": 64, "ctx": 16384, "keep": 128, "hq": 64, "hkv": 8, "d": 128,
         "block": 16, "dtype": "bf16"},
        # Very long contexts in the 8-bit cache.
        {"name": "sparse_long_e4m3", "op": "sparse", "seqs": 8, "ctx": 131072, "keep": 256, "hq": 64, "hkv": 8,
         "d": 128, "block": 16, "dtype": "e4m3"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "rope", "summary", "select", "select", "sparse", "sparse"])
    if op == "table":
        rot = 2 * rng.randint(8, 64)
        return {"op": op, "positions": _log(rng, 1, 131072), "rot": rot, "base": rng.choice([10000.0, 500000.0]),
                "scaling": rng.choice(["none", "linear", "base", "bands", "ramp"]),
                "factor": rng.choice([2.0, 4.0, 7.5, 16.0]), "original": rng.choice([2048, 4096, 8192])}
    hq, hkv = rng.choice([(32, 8), (64, 8), (8, 8), (16, 2), (12, 4), (28, 4)])
    d = rng.choice([128, 128, 64])
    block = rng.choice([16, 32])
    seqs = _log(rng, 1, 64)
    if op == "rope":
        return {"op": op, "seqs": seqs, "new": 1 if rng.random() < 0.5 else _log(rng, 2, 8192 // seqs),
                "ctx": _log(rng, 1, 65536), "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]), "interleaved": rng.random() < 0.5,
                "block": block, "dtype": rng.choice(["bf16", "bf16", "f16", "f32", "e4m3", "e5m2"])}
    if op == "summary":
        ctx = _log(rng, 1, 262144 // seqs)
        return {"op": op, "seqs": seqs, "new": 1 if rng.random() < 0.3 else _log(rng, 1, ctx), "ctx": ctx,
                "hkv": hkv, "d": d, "block": block,
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32", "e4m3", "e5m2"])}
    ctx = _log(rng, 16, min(131072, 1048576 // seqs))
    if op == "select":
        return {"op": op, "seqs": seqs, "ctx": ctx, "keep": _log(rng, 4, 512), "sink": rng.randint(0, 2),
                "recent": rng.randint(1, 2), "hq": hq, "hkv": hkv, "d": d, "block": block,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32", "e4m3", "e5m2"])
    if dtype == "f32":
        return {"op": op, "seqs": _log(rng, 1, 8), "ctx": _log(rng, 16, 8192), "keep": _log(rng, 1, 64), "hq": hq,
                "hkv": hkv, "d": rng.choice([32, 64, 96, 128]), "block": block, "dtype": dtype}
    ctx = min(ctx, 262144 // seqs)
    return {"op": op, "seqs": seqs, "ctx": ctx, "keep": _log(rng, 1, 256), "hq": hq, "hkv": hkv,
            "d": d if dtype in DTYPES else 128, "block": block, "dtype": dtype}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _lengths(case, lo, hi):
    """Ragged lengths from lo to hi, the same for every seed; the first
    sequence has the longest."""
    g = torch.Generator().manual_seed(case["seqs"] * 1009 + hi)
    out = torch.randint(lo, hi + 1, (case["seqs"],), generator=g).tolist()
    out[0] = hi
    return out


def _paged(case, g, dev, lens):
    """Block tables (every sequence's blocks scattered over the pool) and the pool's size."""
    b = case["block"]
    nb = [-(-x // b) for x in lens]
    perm = torch.randperm(sum(nb) + 3, generator=g).to(torch.int32)
    table = torch.zeros(len(lens), max(nb) + 1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(nb):
        table[i, :k] = perm[at:at + k]
        at += k
    return table.to(dev), sum(nb) + 3


def _pool(case, gg, dev, blocks, pools):
    """`pools` pools in the cache's type, and the scales of an 8-bit one."""
    out, scales = [], []
    for _ in range(pools):
        x = torch.randn(blocks, case["hkv"], case["block"], case["d"], generator=gg, device=dev,
                        dtype=torch.float32 if case["dtype"] == "f32" else torch.float16)
        if case["dtype"] in DTYPES:
            out.append(x.to(DTYPES[case["dtype"]]))
            continue
        t, top = FP8[case["dtype"]]
        # Blocks of different magnitude, as layers and tokens have.
        x = x * (0.5 + torch.rand(blocks, case["hkv"], 1, 1, generator=gg, device=dev)).half()
        s = x.abs().amax((2, 3), keepdim=True).float() / torch.tensor(top, device=dev)
        out.append((x.float() / s).to(t).view(torch.uint8))
        scales.append(s[..., 0, 0])
    return out, torch.stack(scales, -1).contiguous() if scales else None


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": dict(case)}
    if case["op"] == "table":
        # A part of a sequence's positions is asked for: where it starts is the input.
        s["first"] = int(torch.randint(0, 4096, (1,), generator=g))
        return s
    n, b, hkv, d = case["seqs"], case["block"], case["hkv"], case["d"]
    io = DTYPES.get(case["dtype"], torch.bfloat16)
    if case["op"] == "rope":
        counts = _lengths(case, case["new"] - case["new"] // 2, case["new"])
        ctx = _lengths(case, case["ctx"] // 4, case["ctx"])
        # The pool holds the blocks that the new tokens touch; those before them play no part.
        lead = [x % b for x in ctx]
        table, blocks = _paged(case, g, dev, [a + c for a, c in zip(lead, counts)])
        pos = torch.cat([torch.arange(x, x + c) for x, c in zip(ctx, counts)])
        at = torch.cat([torch.arange(x, x + c) for x, c in zip(lead, counts)]).to(dev)
        seq = torch.repeat_interleave(torch.arange(n), torch.tensor(counts)).to(dev)
        s["positions"] = pos.to(torch.int32).to(dev)
        s["slots"] = table[seq, at // b].long() * b + at % b
        # q, k and v are parts of one product's rows.
        total = pos.numel()
        qkv = torch.randn(total, case["hq"] + 2 * hkv, d, generator=gg, device=dev).to(io)
        s["q"], s["k"], s["v"] = qkv.split([case["hq"], hkv, hkv], 1)
        angle = torch.arange(max(ctx) + case["new"], device=dev).double()[:, None] * 10000.0 ** (
            -torch.arange(0, case["rot"], 2, device=dev).double() / case["rot"])
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        (s["k_cache"], s["v_cache"]), s["scales"] = _pool(case, gg, dev, blocks, 2)
        s["blocks"] = blocks
        return s
    lens = _lengths(case, max(1, case["ctx"] // 2), case["ctx"])
    s["table"], blocks = _paged(case, g, dev, lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["max_len"] = max(lens)
    if case["op"] == "summary":
        new = [min(x, y) for x, y in zip(lens, _lengths(case, case["new"] - case["new"] // 2, case["new"]))]
        s["first"] = torch.tensor([x - y for x, y in zip(lens, new)], dtype=torch.int32, device=dev)
        s["max_new"] = max(new)
        (s["k_cache"],), sc = _pool(case, gg, dev, blocks, 1)
        s["scales"] = None if sc is None else sc.expand(blocks, hkv, 2).contiguous()
        s["summaries"] = torch.zeros(blocks, hkv, 2, d, dtype=torch.int8, device=dev)
        s["summary_scales"] = torch.zeros(blocks, hkv, device=dev)
        return s
    s["q"] = torch.randn(n, case["hq"], d, generator=gg, device=dev).to(io)
    if case["op"] == "select":
        # Blocks' ranges as rotated keys have them: channels of different size, blocks of different place and width.
        channel = (0.7 * torch.randn(hkv, d, generator=gg, device=dev)).exp()
        mid = channel * torch.randn(blocks, hkv, d, generator=gg, device=dev)
        wide = channel * (0.5 + torch.rand(blocks, hkv, d, generator=gg, device=dev))
        s["summaries"] = torch.empty(blocks, hkv, 2, d, dtype=torch.int8, device=dev)
        s["summary_scales"] = torch.empty(blocks, hkv, device=dev)
        codes, scales = _codes(mid + wide, mid - wide)
        s["summaries"].copy_(codes)
        s["summary_scales"].copy_(scales)
        return s
    (s["k"], s["v"]), s["scales"] = _pool(case, gg, dev, blocks, 2)
    s["scale"] = d ** -0.5
    # The first and the last block of a sequence and others between them; some lists are shorter.
    lists = torch.full((n, hkv, case["keep"]), -1, dtype=torch.int32)
    some = torch.zeros(n, hkv, dtype=torch.int32)
    for i, x in enumerate(lens):
        nb = -(-x // b)
        for h in range(hkv):
            k = min(nb, case["keep"] - (i + h) % 3 if case["keep"] > 3 else case["keep"])
            pick = torch.randperm(nb, generator=g)[:k]
            pick[0] = nb - 1 if nb - 1 not in pick else pick[0]
            lists[i, h, :k] = pick.sort()[0]
            some[i, h] = k
    s["lists"], s["list_lens"] = lists.to(dev), some.to(dev)
    return s


def _codes(hi, lo):
    """Largest and smallest values [..., d] in 8 bits: codes [..., 2, d] and scales [...]."""
    top = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    scale = top / torch.full_like(top, 127.0)
    div = scale[..., None]
    up = torch.where(div > 0, hi / div, torch.zeros_like(hi)).ceil().clamp(max=127.0)
    dn = torch.where(div > 0, lo / div, torch.zeros_like(lo)).floor().clamp(min=-127.0)
    return torch.stack([up, dn], -2).to(torch.int8), scale


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"table": _own_table, "rope": _own_rope, "summary": _own_summary, "select": _own_select,
                "sparse": _own_sparse}[op](s)
    return {"table": _plain_table, "rope": _plain_rope, "summary": _plain_summary, "select": _plain_select,
            "sparse": _plain_sparse}[op](s)


def _own_table(s):
    import paged_kv_cache_14_gb300 as pa
    c = s["case"]
    return pa.pa_rope_table(c["positions"], c["rot"], base=c["base"], scaling=c["scaling"], factor=c["factor"],
                            original_len=c["original"], first_position=s["first"])


def _own_rope(s):
    import paged_kv_cache_14_gb300 as pa
    c = s["case"]
    args = (s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], s["k_cache"], s["v_cache"])
    if s["scales"] is None:
        q = pa.pa_rope_and_cache(*args, interleaved=c["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    call = pa.pa_rope_and_cache_fp8 if c["dtype"] == "e4m3" else pa.pa_rope_and_cache_e5m2
    q = call(*args, s["scales"], interleaved=c["interleaved"])
    t = FP8[c["dtype"]][0]
    return q, s["k_cache"].view(t), s["v_cache"].view(t), s["scales"]


def _own_summary(s):
    import paged_kv_cache_14_gb300 as pa
    c = s["case"]
    rest = (s["table"], s["first"], s["lens"], s["max_new"], s["summaries"], s["summary_scales"])
    if s["scales"] is None:
        pa.pa_block_summaries(s["k_cache"], *rest)
    else:
        call = pa.pa_block_summaries_fp8 if c["dtype"] == "e4m3" else pa.pa_block_summaries_e5m2
        call(s["k_cache"], s["scales"], *rest)
    return s["summaries"], s["summary_scales"]


def _own_select(s):
    import paged_kv_cache_14_gb300 as pa
    c = s["case"]
    return pa.pa_select_blocks(s["q"], s["summaries"], s["summary_scales"], s["table"], s["lens"], s["max_len"],
                               c["block"], c["keep"], num_sink=c["sink"], num_recent=c["recent"])


def _own_sparse(s):
    import paged_kv_cache_14_gb300 as pa
    c = s["case"]
    rest = (s["table"], s["lens"], s["lists"], s["list_lens"], s["scale"])
    if s["scales"] is None:
        return pa.pa_decode_sparse(s["q"], s["k"], s["v"], *rest)
    call = pa.pa_decode_sparse_fp8 if c["dtype"] == "e4m3" else pa.pa_decode_sparse_e5m2
    return call(s["q"], s["k"], s["v"], s["scales"], *rest)


# ----- the plain forms -----

def _plain_table(s):
    c = s["case"]
    rot = c["rot"]
    i = torch.arange(0, rot, 2, device="cuda").double()
    base = c["base"] * c["factor"] ** (rot / (rot - 2)) if c["scaling"] == "base" else c["base"]
    f = base ** (-i / rot)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "bands":  # short waves stay, long ones stretch, those between are mixed
        turns = c["original"] * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = keep * f + (1 - keep) * f / c["factor"]
    elif c["scaling"] == "ramp":  # the same by the pair's number, from 32 turns to one
        lo, hi = (rot * math.log(c["original"] / (2 * math.pi * x)) / (2 * math.log(c["base"])) for x in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        stretch = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f = (1 - stretch) * f + stretch * f / c["factor"]
    pos = torch.arange(s["first"], s["first"] + c["positions"], device="cuda").double()
    angle = pos[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _rotated(x, cos, sin, rot, interleaved):
    x = x.float()
    y, rest = x[..., :rot], x[..., rot:]
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, rest], -1)


def _plain_rope(s):
    c = s["case"]
    b, rot = c["block"], c["rot"]
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    q = _rotated(s["q"], cos, sin, rot, c["interleaved"]).to(s["q"].dtype)
    k = _rotated(s["k"], cos, sin, rot, c["interleaved"])
    blk, off = s["slots"] // b, s["slots"] % b
    if s["scales"] is None:
        s["k_cache"][blk, :, off] = k.to(s["k_cache"].dtype)
        s["v_cache"][blk, :, off] = s["v"]
        return q, s["k_cache"], s["v_cache"]
    t, top = FP8[c["dtype"]]
    # Rows below the first written offset stay, under the block's new scale.
    first = torch.full((s["blocks"],), b, device=blk.device).scatter_reduce(0, blk, off, "amin")
    for which, (x, pool) in enumerate(((k, s["k_cache"]), (s["v"].float(), s["v_cache"]))):
        most = torch.zeros(s["blocks"], c["hkv"], device=x.device)
        most = most.scatter_reduce(0, blk[:, None].expand(-1, c["hkv"]), x.abs().amax(-1), "amax")
        old = torch.where((first > 0)[:, None], s["scales"][..., which], 0.0)
        new = torch.maximum(old, most / torch.full_like(most, top))
        ratio = torch.where((new > old) & (old > 0), old / new, torch.ones_like(new))
        again = (pool.view(t).float() * ratio[:, :, None, None]).to(t).view(torch.uint8)
        under = (torch.arange(b, device=x.device) < first[:, None]) & (first < b)[:, None]
        pool.copy_(torch.where(under[:, None, :, None], again, pool))
        row = new[blk][..., None]
        pool[blk, :, off] = torch.where(row > 0, x / row, torch.zeros_like(x)).to(t).view(torch.uint8)
        s["scales"][..., which] = torch.where((first < b)[:, None], new, s["scales"][..., which])
    return q, s["k_cache"].view(t), s["v_cache"].view(t), s["scales"]


def _plain_summary(s):
    c = s["case"]
    b = c["block"]
    lens, first = s["lens"].long()[:, None], s["first"].long()[:, None]
    lb = first // b + torch.arange((s["max_new"] + b - 2) // b + 1, device=lens.device)
    lb = torch.where(lb * b < lens, lb, first // b)  # past the end: the first block once more
    blk = s["table"].long().gather(1, lb)
    x = s["k_cache"][blk]
    if s["scales"] is not None:
        x = x.view(FP8[c["dtype"]][0]).float() * s["scales"][blk][..., 0, None, None]
    x = x.float()
    held = (lb[..., None] * b + torch.arange(b, device=lens.device) < lens[..., None])[:, :, None, :, None]
    codes, scales = _codes(torch.where(held, x, -math.inf).amax(3), torch.where(held, x, math.inf).amin(3))
    s["summaries"][blk] = codes
    s["summary_scales"][blk] = scales
    return s["summaries"], s["summary_scales"]


def _plain_select(s):
    c = s["case"]
    n, b, hkv, d = c["seqs"], c["block"], c["hkv"], c["d"]
    q = s["q"].float()
    sq = q.abs().amax(-1, keepdim=True)
    sq = sq / torch.full_like(sq, 127.0)
    q = torch.where(sq > 0, q / sq, torch.zeros_like(q)).round()
    parts = torch.stack([q.clamp(min=0.0), q.clamp(max=0.0)], -2).reshape(n, hkv, -1, 2 * d)
    width = -(-s["max_len"] // b)
    table = s["table"][:, :width].long()
    codes = s["summaries"][table].float().reshape(n, width, hkv, 2 * d).transpose(1, 2)
    whole = parts @ codes.transpose(2, 3)  # [n, hkv, g, blocks], whole numbers
    score = (whole * sq.reshape(n, hkv, -1, 1)).amax(2) * s["summary_scales"][table].transpose(1, 2)
    at = torch.arange(width, device=q.device)
    some = ((s["lens"] + b - 1) // b).long()[:, None]
    forced = (at < c["sink"]) | (at >= some - c["recent"])
    score = torch.where(forced[:, None], math.inf, score)
    score = torch.where((at < some)[:, None], score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :c["keep"]]
    best = torch.nn.functional.pad(best, (0, c["keep"] - best.shape[-1]), value=width)
    best = torch.where(best < some[..., None], best, width).sort(-1)[0]
    lens = some.clamp(max=c["keep"]).expand(n, hkv)
    return torch.where(best < width, best, -1).to(torch.int32), lens.to(torch.int32).contiguous()


def _plain_sparse(s):
    c = s["case"]
    n, hq, hkv, d, b = c["seqs"], c["hq"], c["hkv"], c["d"], c["block"]
    lists = s["lists"].long()
    live = torch.arange(lists.shape[2], device=lists.device) < s["list_lens"][..., None]
    lists = torch.where(live, lists, 0)
    blk = s["table"].long()[:, None].expand(n, hkv, -1).gather(2, lists)
    head = torch.arange(hkv, device=lists.device)[None, :, None]

    def values(pool, which):  # [n, hkv, tokens, d] in 32 bits
        x = pool[blk, head]
        if s["scales"] is not None:
            x = x.view(FP8[c["dtype"]][0]).float() * s["scales"][blk, head, which][..., None, None]
        return x.float().reshape(n, hkv, -1, d)

    pos = lists[..., None] * b + torch.arange(b, device=lists.device)
    seen = (live[..., None] & (pos < s["lens"].long()[:, None, None, None])).reshape(n, hkv, 1, -1)
    q = s["q"].float().reshape(n, hkv, hq // hkv, d)
    score = (q @ values(s["k"], 0).transpose(2, 3) * s["scale"]).masked_fill(~seen, -math.inf)
    w = (score - score.amax(-1, keepdim=True)).exp()
    return ((w @ values(s["v"], 1)) / w.sum(-1, keepdim=True)).reshape(n, hq, d).to(s["q"].dtype)


# ---------------------------------------------------------------------------
# What a pass costs at least
# ---------------------------------------------------------------------------

def work(case):
    op, b = case["op"], case.get("block")
    if op == "table":
        # Each pair's angle, its reduction, and a sine and a cosine of some ten operations each.
        return {"bytes": 4 * case["positions"] * case["rot"], "flops": 12 * case["positions"] * case["rot"]}
    d, hkv = case["d"], case["hkv"]
    size = {"f32": 4, "f16": 2, "bf16": 2}.get(case["dtype"], 1)
    io = max(size, 2)
    if op == "rope":
        counts = _lengths(case, case["new"] - case["new"] // 2, case["new"])
        t = sum(counts)
        old = 0
        if size == 1:  # rows of a block under way, which a larger scale encodes again
            old = 4 * hkv * d * sum(x % b for x in _lengths(case, case["ctx"] // 4, case["ctx"])) / 2
        return {"bytes": t * (d * (2 * case["hq"] * io + 2 * hkv * (io + size)) + 4 * case["rot"]) + old,
                "flops": 3 * t * (case["hq"] + hkv) * case["rot"]}
    lens = _lengths(case, max(1, case["ctx"] // 2), case["ctx"])
    if op == "summary":
        new = [min(x, y) for x, y in zip(lens, _lengths(case, case["new"] - case["new"] // 2, case["new"]))]
        blocks = sum((x - 1) // b - (x - y) // b + 1 for x, y in zip(lens, new))
        rows = sum(x - (x - y) // b * b for x, y in zip(lens, new))
        return {"bytes": hkv * (rows * d * size + blocks * (2 * d + 4)), "flops": 2 * hkv * d * rows}
    if op == "select":
        blocks = sum(-(-x // b) for x in lens)
        return {"bytes": hkv * blocks * (2 * d + 4) + case["seqs"] * (case["hq"] * d * io + 4 * hkv * case["keep"]),
                "flops": 4 * blocks * case["hq"] * d}
    rows = sum(min(x, (case["keep"] - (case["keep"] > 3)) * b) for x in lens)  # some lists are one or two shorter
    return {"bytes": 2 * rows * hkv * d * size + 2 * case["seqs"] * case["hq"] * d * io,
            "flops": 4 * rows * case["hq"] * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sparse" and case["seqs"] * case["hkv"] > 4096:
        return None
    return {"table": _exact_table, "rope": _exact_rope, "summary": _exact_summary, "select": _exact_select,
            "sparse": _exact_sparse}[case["op"]](s)


def _exact_table(s):
    c = s["case"]
    rot, stretch, old = c["rot"], c["factor"], c["original"]
    freqs = []
    for i in range(rot // 2):
        f = c["base"] ** (-2.0 * i / rot)
        if c["scaling"] == "linear":
            f /= stretch
        elif c["scaling"] == "base":
            f = (c["base"] * stretch ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif c["scaling"] == "bands":
            wave = 2 * math.pi / f
            if wave > old:
                f /= stretch
            elif wave > old / 4.0:
                part = (old / wave - 1.0) / 3.0
                f = (1 - part) * f / stretch + part * f
        elif c["scaling"] == "ramp":
            ends = [rot * math.log(old / (x * 2 * math.pi)) / (2 * math.log(c["base"])) for x in (32, 1)]
            a, z = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rot - 1)
            part = min(1.0, max(0.0, (i - a) / max(z - a, 0.001)))
            f = f / stretch * part + f * (1 - part)
        freqs.append(f)
    pos = torch.arange(c["positions"], dtype=torch.float64) + s["first"]
    angle = torch.outer(pos, torch.tensor(freqs, dtype=torch.float64))
    return torch.hstack([torch.cos(angle), torch.sin(angle)])


def _exact_turn(x, cs, rot, interleaved):
    """Rows x [t, h, d] in 64 bits, turned pair by pair."""
    out = x.double().clone()
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        co, si = cs[:, i, None].double(), cs[:, half + i, None].double()
        out[:, :, a] = x[:, :, a].double() * co - x[:, :, b].double() * si
        out[:, :, b] = x[:, :, a].double() * si + x[:, :, b].double() * co
    return out


def _nearest(x, name):
    """The 8-bit value nearest to each x, ties to the even code."""
    t = FP8[name][0]
    codes = torch.arange(128, dtype=torch.uint8)
    val = codes.view(t).double()
    val = val[torch.isfinite(val)].to(x.device)
    a = x.abs()
    up = torch.searchsorted(val, a.contiguous()).clamp(max=val.numel() - 1)
    dn = (up - 1).clamp(min=0)
    du, dd = val[up] - a, a - val[dn]
    pick = torch.where((dd < du) | ((dd == du) & (dn % 2 == 0)), dn, up)
    return torch.copysign(val[pick], x)


def _exact_rope(s):
    c, b = s["case"], s["case"]["block"]
    cs = s["cos_sin"][s["positions"].long()]
    q = _exact_turn(s["q"], cs, c["rot"], c["interleaved"])
    rows = [_exact_turn(s["k"], cs, c["rot"], c["interleaved"]), s["v"].double()]
    slots = s["slots"].tolist()
    if s["scales"] is None:
        pools = []
        for x, pool in zip(rows, (s["k_cache"], s["v_cache"])):
            flat = pool.double().transpose(1, 2).reshape(-1, c["hkv"], c["d"]).clone()
            flat[s["slots"]] = x
            pools.append(flat.reshape(-1, b, c["hkv"], c["d"]).transpose(1, 2).contiguous())
        return q, pools[0], pools[1]
    t, top = FP8[c["dtype"]]
    by_block = {}
    for j, x in enumerate(slots):
        by_block.setdefault(x // b, []).append(j)
    if len(by_block) > 2000:
        return None
    scales, pools = s["scales"].double(), []
    for which, (x, pool) in enumerate(zip(rows, (s["k_cache"], s["v_cache"]))):
        val = pool.view(t).double()
        for blk, js in by_block.items():
            offs = [slots[j] % b for j in js]
            new = x[js].abs().amax((0, 2)) / top
            if min(offs) > 0:
                old = scales[blk, :, which].clone()
                new = torch.maximum(new, old)
                again = _nearest(val[blk, :, :min(offs)] * (old / new)[:, None, None], c["dtype"])
                val[blk, :, :min(offs)] = torch.where((new > old)[:, None, None], again, val[blk, :, :min(offs)])
            val[blk][:, offs] = _nearest(x[js].transpose(0, 1) / new[:, None, None], c["dtype"])
            scales[blk, :, which] = new
        pools.append(val)
    return q, pools[0], pools[1], scales


def _exact_summary(s):
    c, b = s["case"], s["case"]["block"]
    lens, first, table = s["lens"].tolist(), s["first"].tolist(), s["table"].long()
    codes, scales = s["summaries"].clone(), s["summary_scales"].double()
    if sum((x - y) // b + 1 for x, y in zip(lens, first)) > 20000:
        return None
    for i, x in enumerate(lens):
        for lb in range(first[i] // b, -(-x // b)):
            blk = table[i, lb]
            v = s["k_cache"][blk, :, :min(b, x - lb * b)]
            if s["scales"] is not None:
                v = v.view(FP8[c["dtype"]][0]).float() * s["scales"][blk, :, 0, None, None]
            v = v.double()
            hi, lo = v.amax(1), v.amin(1)
            # The scale and the quotients are 32-bit numbers by definition; 64 bits round to the same.
            sc = (v.abs().amax((1, 2)) / 127.0).float().double()
            codes[blk, :, 0] = (hi / sc[:, None]).float().ceil().clamp(max=127).to(torch.int8)
            codes[blk, :, 1] = (lo / sc[:, None]).float().floor().clamp(min=-127).to(torch.int8)
            scales[blk] = sc
    return codes, scales


def _exact_select(s):
    c, b = s["case"], s["case"]["block"]
    n, hkv, d, keep = c["seqs"], c["hkv"], c["d"], c["keep"]
    g = c["hq"] // hkv
    lists, some = torch.full((n, hkv, keep), -1, dtype=torch.int32), torch.zeros(n, hkv, dtype=torch.int32)
    if n * hkv > 4096:
        return None
    for i, x in enumerate(s["lens"].tolist()):
        nb = -(-x // b)
        blk = s["table"][i, :nb].long()
        for h in range(hkv):
            q = s["q"][i, h * g:(h + 1) * g].double()
            sq = (q.abs().amax(1) / 127.0).float().double()
            q = (q / sq[:, None]).float().round().double()
            hi, lo = s["summaries"][blk, h, 0].double(), s["summaries"][blk, h, 1].double()
            whole = q.clamp(min=0) @ hi.T + q.clamp(max=0) @ lo.T
            score = ((sq[:, None] * whole).float().amax(0).double() * s["summary_scales"][blk, h].double()).float()
            must = [j for j in range(nb) if j < c["sink"] or j >= nb - c["recent"]]
            rest = [j for j in torch.sort(-score, stable=True)[1].tolist() if c["sink"] <= j < nb - c["recent"]]
            mine = sorted((must + rest)[:keep])
            lists[i, h, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            some[i, h] = len(mine)
    return lists, some


def _exact_sparse(s):
    c, b = s["case"], s["case"]["block"]
    g = c["hq"] // c["hkv"]
    lens, table = s["lens"].tolist(), s["table"].long()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    counts, lists = s["list_lens"].tolist(), s["lists"].long()
    for i in range(c["seqs"]):
        for h in range(c["hkv"]):
            lb = lists[i, h, :counts[i][h]]
            blk = table[i, lb]
            kv = []
            for which, pool in enumerate((s["k"], s["v"])):
                x = pool[blk, h]
                if s["scales"] is None:
                    x = x.double()
                else:
                    x = x.view(FP8[c["dtype"]][0]).double() * s["scales"][blk, h, which].double()[:, None, None]
                kv.append(x.reshape(-1, c["d"])[:(lb.numel() - 1) * b + min(b, lens[i] - int(lb[-1]) * b)])
            score = s["q"][i, h * g:(h + 1) * g].double() @ kv[0].T * s["scale"]
            out[i, h * g:(h + 1) * g] = torch.softmax(score, 1) @ kv[1]
    return out
