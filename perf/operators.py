"""Measured cases of the draft-tree operators: attention of a tree of drafted
tokens over a paged cache, verification of the drafted tokens against the
target's probabilities, and compaction of the accepted path in the cache.

Each case names its operator in "op":
  tree    q rows of every sequence's tree nodes against its paged context
  verify  which drafted tokens are kept, and the next token
  compact K/V rows of the kept nodes moved to the end of the context
A tree is a list of parents: node j of a sequence (node 0 is the newest
committed token) has parents[j] < j, and parents[0] = -1.
"""
import math

import torch

own = False  # True: run() calls this repository's kernels

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


def listed():
    return [
        # One user, a short answer so far: nothing but latency counts.
        {"name": "tree_one_user", "op": "tree", "seqs": 1, "ctx": 700, "nodes": 8, "hq": 32, "hkv": 8, "d": 128,
         "block": 16, "dtype": "bf16"},
        # A serving batch of an 8B-shaped layer, trees of up to 16 nodes.
        {"name": "tree_batch_8b", "op": "tree", "seqs": 64, "ctx": 4096, "nodes": 16, "hq": 32, "hkv": 8, "d": 128,
         "block": 16, "dtype": "bf16"},
        # A serving batch of a 70B-shaped layer with wide trees.
        {"name": "tree_batch_70b_wide", "op": "tree", "seqs": 48, "ctx": 8192, "nodes": 40, "hq": 64, "hkv": 8,
         "d": 128, "block": 32, "dtype": "f16"},
        # Few sequences of a very long context: one sequence has to fill the machine.
        {"name": "tree_long", "op": "tree", "seqs": 4, "ctx": 131072, "nodes": 12, "hq": 64, "hkv": 8, "d": 128,
         "block": 16, "dtype": "bf16"},
        # The 70B-shaped batch over the 8-bit cache.
        {"name": "tree_batch_e4m3", "op": "tree", "seqs": 64, "ctx": 4096, "nodes": 16, "hq": 64, "hkv": 8, "d": 128,
         "block": 16, "dtype": "e4m3"},
        # fp32 I/O, as the fp32 decode is used: for checking, on small models.
        {"name": "tree_f32", "op": "tree", "seqs": 3, "ctx": 1500, "nodes": 11, "hq": 12, "hkv": 4, "d": 96,
         "block": 16, "dtype": "f32"},
        # A chain of drafts of a few users against the draft's own probabilities.
        {"name": "verify_chain", "op": "verify", "seqs": 4, "nodes": 5, "branch": 1, "vocab": 32000, "dtype": "f32",
         "draft": True},
        # A serving batch, trees whose children were drawn from the draft's probabilities.
        {"name": "verify_tree", "op": "verify", "seqs": 96, "nodes": 16, "branch": 3, "vocab": 131072,
         "dtype": "f32", "draft": True},
        # Drafts without probabilities (a lookup or the likeliest few), an odd vocabulary, 16 bits.
        {"name": "verify_lookup", "op": "verify", "seqs": 64, "nodes": 24, "branch": 4, "vocab": 100003,
         "dtype": "bf16", "draft": False},
        # One layer of a few sequences.
        {"name": "compact_few", "op": "compact", "seqs": 4, "ctx": 900, "nodes": 8, "layers": 1, "hkv": 8, "d": 128,
         "block": 16, "dtype": "bf16"},
        # Every layer of a serving batch.
        {"name": "compact_batch", "op": "compact", "seqs": 128, "ctx": 256, "nodes": 24, "layers": 32, "hkv": 8,
         "d": 128, "block": 16, "dtype": "bf16"},
        # The same over an 8-bit cache: rows that change their block are encoded with its scale.
        {"name": "compact_e4m3", "op": "compact", "seqs": 64, "ctx": 300, "nodes": 40, "layers": 16, "hkv": 8,
         "d": 128, "block": 16, "dtype": "e4m3"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "compact"])
    if op == "verify":
        seqs = _log(rng, 1, 96)
        return {"op": op, "seqs": seqs, "nodes": _log(rng, 1, 24), "branch": rng.randint(1, 4),
                "vocab": _log(rng, 1000, 131072), "dtype": rng.choice(["f32", "f32", "bf16", "f16"]),
                "draft": rng.random() < 0.6}
    dtype = rng.choice(["bf16", "bf16", "f16", "e4m3", "e5m2", "f32"])
    block = rng.choice([16, 32])
    if op == "compact":
        return {"op": op, "seqs": _log(rng, 1, 96), "ctx": _log(rng, 1, 300), "nodes": _log(rng, 1, 64),
                "layers": _log(rng, 1, 24), "hkv": rng.choice([1, 2, 4, 8]), "d": rng.choice([64, 128]),
                "block": block, "dtype": dtype}
    hq, hkv = rng.choice([(32, 8), (64, 8), (8, 8), (16, 2), (12, 4), (28, 4)])
    if dtype == "f32":
        return {"op": op, "seqs": _log(rng, 1, 4), "ctx": _log(rng, 1, 1500), "nodes": _log(rng, 1, 24), "hq": hq,
                "hkv": hkv, "d": rng.choice([32, 64, 96, 128]), "block": block, "dtype": dtype}
    seqs = _log(rng, 1, 96)
    d = rng.choice([128, 128, 64]) if dtype in DTYPES else 128
    ctx = _log(rng, 16, min(65536, 262144 // seqs))
    return {"op": op, "seqs": seqs, "ctx": ctx, "nodes": _log(rng, 1, min(96, 12000000 // (seqs * ctx))), "hq": hq,
            "hkv": hkv, "d": d, "block": block, "dtype": dtype}


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


def _trees(case, g):
    """Ragged trees: (node counts, parents, child counts) as host lists."""
    n, t = case["seqs"], case["nodes"]
    branch = case.get("branch", 4)
    draws = torch.rand(n, t, generator=g).tolist()
    counts = _lengths(case, t - t // 2, t)
    parents, children = [], []
    for i in range(n):
        kids = [0] * counts[i]
        mine = [-1]
        for j in range(1, counts[i]):
            # Nodes early in the list get children first; a full node passes its turn on.
            p = int(draws[i][j] * draws[i][j] * j)
            while kids[p] >= branch:
                p += 1
            kids[p] += 1
            mine.append(p)
        parents += mine
        children += kids
    return counts, parents, children


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


def _pool(case, gg, dev, layers, blocks):
    """K and V of `layers` pools in the cache's type, and the scales of an 8-bit one."""
    out = []
    for _ in range(2):
        x = torch.randn(layers, blocks, case["hkv"], case["block"], case["d"], generator=gg, device=dev,
                        dtype=torch.float32 if case["dtype"] == "f32" else torch.float16)
        if case["dtype"] in DTYPES:
            out.append((x.to(DTYPES[case["dtype"]]), None))
            continue
        t, top = FP8[case["dtype"]]
        # Blocks of different magnitude, as layers and tokens have.
        x = x * (0.5 + torch.rand(layers, blocks, case["hkv"], 1, 1, generator=gg, device=dev)).half()
        s = x.abs().amax((3, 4), keepdim=True).float() / top
        out.append(((x.float() / s).to(t).view(torch.uint8), s[..., 0, 0]))
    (k, ks), (v, vs) = out
    return k, v, None if ks is None else torch.stack([ks, vs], -1).contiguous()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device=dev).manual_seed(seed)
    counts, parents, children = _trees(case, g)
    n, t = case["seqs"], case["nodes"]
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    total = cu[-1]
    s = {"case": dict(case), "cu": torch.tensor(cu, dtype=torch.int32, device=dev),
         "parents": torch.tensor(parents, dtype=torch.int32, device=dev), "max_nodes": t, "total": total}
    if case["op"] == "verify":
        v, dt = case["vocab"], DTYPES[case["dtype"]]
        logits = 3.0 * torch.randn(total, v, generator=gg, device=dev)
        draft = torch.softmax(logits + torch.randn(total, v, generator=gg, device=dev), -1).to(dt)
        s["target"] = torch.softmax(logits, -1).to(dt)
        # A child's token is drawn from the draft's distribution after its parent.
        rows = torch.tensor([cu[i] + max(parents[cu[i] + j], 0) for i in range(n) for j in range(counts[i])],
                            device=dev)
        cum = draft.float().cumsum(-1)
        pick = torch.rand(total, generator=gg, device=dev) * cum[rows, -1]
        tok = [torch.searchsorted(cum[rows[i:i + 256]], pick[i:i + 256, None])[:, 0] for i in range(0, total, 256)]
        s["tokens"] = torch.cat(tok).clamp(max=v - 1).to(torch.int32)
        s["draft"] = draft if case["draft"] else None
        s["u_accept"] = torch.rand(total, generator=gg, device=dev)
        s["u_sample"] = torch.rand(n, generator=gg, device=dev)
        s["max_path"] = t
        # The trees' shape, which the program that drew the drafts knows: rows with more than k children.
        s["with_more"] = [torch.tensor(r, device=dev) for k in range(1, max(children))
                          if (r := [i for i, c in enumerate(children) if c > k])]
        return s
    if case["op"] == "tree":
        ctx = _lengths(case, max(1, case["ctx"] // 4), case["ctx"])
        lens = [a + b for a, b in zip(ctx, counts)]
        s["table"], blocks = _paged(case, g, dev, lens)
        k, v, sc = _pool(case, gg, dev, 1, blocks)
        s["k"], s["v"], s["scales"] = k[0], v[0], None if sc is None else sc[0].contiguous()
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s["max_kv"] = max(lens)
        s["q"] = torch.randn(total, case["hq"], case["d"], generator=gg, device=dev).to(
            DTYPES.get(case["dtype"], torch.bfloat16))
        s["scale"] = case["d"] ** -0.5
        return s
    ctx = _lengths(case, max(1, case["ctx"] // 2), case["ctx"])
    s["table"], blocks = _paged(case, g, dev, [a + b for a, b in zip(ctx, counts)])
    s["k"], s["v"], s["scales"] = _pool(case, gg, dev, case["layers"], blocks)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    # The kept path of a tree: the root and some of the later nodes, in order.
    paths = []
    for i in range(n):
        keep = 1 + int(torch.randint(0, min(8, counts[i]), (1,), generator=g))
        rest = (1 + torch.randperm(max(counts[i] - 1, 1), generator=g)[:keep - 1]).tolist() if keep > 1 else []
        paths.append([0] + sorted(rest))
    width = min(8, t)
    s["path"] = torch.tensor([p + [-1] * (width - len(p)) for p in paths], dtype=torch.int32, device=dev)
    s["path_lens"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"tree": _own_tree, "verify": _own_verify, "compact": _own_compact}[op](s)
    return {"tree": _plain_tree, "verify": _plain_verify, "compact": _plain_compact}[op](s)


def _own_tree(s):
    import paged_kv_cache_14_gb300 as pa
    c, q, k = s["case"], s["q"], s["k"]
    if "workspace" not in s:  # kept by a serving program from step to step, like the output
        s["workspace"] = torch.empty(pa.pa_decode_tree_workspace_size(
            c["seqs"], c["hq"], c["hkv"], c["d"], c["block"], s["total"], s["max_nodes"], s["max_kv"],
            q.dtype), dtype=torch.uint8, device=q.device)
        s["out"] = torch.empty_like(q)
    if s["scales"] is None:
        return pa.pa_decode_tree(q, s["cu"], s["parents"], k, s["v"], s["table"], s["ctx"], s["max_nodes"],
                                 s["max_kv"], s["scale"], out=s["out"], workspace=s["workspace"])
    call = pa.pa_decode_tree_fp8 if c["dtype"] == "e4m3" else pa.pa_decode_tree_e5m2
    return call(q, s["cu"], s["parents"], k, s["v"], s["scales"], s["table"], s["ctx"], s["max_nodes"], s["max_kv"],
                s["scale"], out=s["out"], workspace=s["workspace"])


def _own_verify(s):
    import paged_kv_cache_14_gb300 as pa
    return pa.pa_verify_tree(s["target"], s["draft"], s["tokens"], s["cu"], s["parents"], s["u_accept"],
                             s["u_sample"], s["max_nodes"], s["max_path"])


def _own_compact(s):
    import paged_kv_cache_14_gb300 as pa
    if "layers" not in s:  # a program holds its layers' pools as separate tensors
        s["layers"] = [list(x.unbind(0)) if x is not None else None for x in (s["k"], s["v"], s["scales"])]
    k, v, sc = s["layers"]
    if sc is None:
        pa.pa_compact_tree(k, v, s["table"], s["ctx"], s["path"], s["path_lens"])
        return s["k"], s["v"]
    call = pa.pa_compact_tree_fp8 if s["case"]["dtype"] == "e4m3" else pa.pa_compact_tree_e5m2
    call(k, v, sc, s["table"], s["ctx"], s["path"], s["path_lens"])
    return _cache_values(s)


def _cache_values(s):
    t = FP8[s["case"]["dtype"]][0]
    return s["k"].view(t), s["v"].view(t), s["scales"]


# ----- the plain forms -----

def _square(m):
    return (m @ m).clamp(max=1.0)


def _layout(s):
    """Padded trees: row of node j of sequence i, which nodes exist, parents,
    and ancestors-or-self as a 0/1 matrix."""
    cu, t = s["cu"].long(), s["max_nodes"]
    node = torch.arange(t, device=cu.device)
    rows = cu[:-1, None] + node
    there = rows < cu[1:, None]
    rows = torch.where(there, rows, torch.zeros_like(rows))
    par = torch.where(there, s["parents"].long()[rows], torch.full_like(rows, -1))
    link = (par[:, :, None] == node).float() + (node[:, None] == node).float()
    reach = _square(_square(_square(_square(_square(_square(_square(link)))))))  # paths of up to 128 steps
    return rows, there, par, reach > 0


def _plain_tree(s):
    c = s["case"]
    n, t, hq, hkv, d, b = c["seqs"], s["max_nodes"], c["hq"], c["hkv"], c["d"], c["block"]
    rows, there, par, reach = _layout(s)
    length = -(-s["max_kv"] // b) * b
    table = s["table"][:, :length // b].long()

    def values(pool, which):  # [n, hkv, length, d] in 32 bits
        x = pool[table]
        if s["scales"] is not None:
            x = x.view(FP8[c["dtype"]][0]).float() * s["scales"][table][..., which, None, None]
        return x.float().transpose(1, 2).reshape(n, hkv, length, d)

    ctx = s["ctx"].long()[:, None, None]
    pos = torch.arange(length, device=ctx.device)
    at = (pos - ctx).clamp(0, t - 1).expand(n, t, length)
    seen = (pos < ctx) | (reach.gather(2, at) & (pos >= ctx) & (pos < ctx + there.sum(1)[:, None, None]))
    q = s["q"][rows].float().reshape(n, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)  # [n, hkv, g, t, d]
    score = (q.reshape(n, hkv, -1, d) @ values(s["k"], 0).transpose(2, 3)).reshape(n, hkv, hq // hkv, t, length)
    score = (score * s["scale"]).masked_fill(~seen[:, None, None], -math.inf)
    score = score - score.amax(-1, keepdim=True)
    w = score.exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.reshape(n, hkv, -1, length) @ values(s["v"], 1)).reshape(n, hkv, hq // hkv, t, d) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(n * t, hq, d)
    r = torch.arange(s["total"], device=o.device)
    seq = torch.searchsorted(s["cu"].long()[1:], r, right=True)
    return o[seq * t + r - s["cu"].long()[seq]].to(s["q"].dtype)


def _plain_verify(s):
    rows, there, par, reach = _layout(s)
    n, t = rows.shape
    node = torch.arange(t, device=rows.device)
    target, draft = s["target"], s["draft"]
    tok = s["tokens"].long()[rows]
    prow = rows.gather(1, par.clamp(min=0))  # the row whose distribution a node's token is judged by
    child = there & (par >= 0)
    sib = (par[:, :, None] == par[:, None, :]) & child[:, :, None] & child[:, None, :]  # [n, node, other]
    before = sib & (node[None, None, :] < node[None, :, None])
    rank = before.sum(2)
    kids = torch.zeros_like(rows).scatter_add(1, par.clamp(min=0), child.long())
    u = s["u_accept"].double()[rows]
    px = target[prow, tok].double()
    if draft is None:
        again = (before & (tok[:, :, None] == tok[:, None, :])).any(2)  # the same token was refused already
        w = px.masked_fill(again, 0.0)
        mass = 1.0 - (before.double() @ w[:, :, None])[..., 0]
        accept = u * mass < w
    else:
        qx = draft[prow, tok].double()
        # After k refusals at a row the weights are max(0, p - C q), C the sum of the masses so far.
        mult = torch.zeros(8, s["total"], dtype=torch.float64, device=rows.device)
        mass = torch.ones_like(mult)
        mult[1:] = 1.0
        for k, r in enumerate(s["with_more"], 1):
            mass[k, r] = (target[r].double() - mult[k, r, None] * draft[r].double()).clamp(min=0.0).sum(-1)
            mult[k + 1:, r] = mult[k, r] + mass[k, r]
        w = (px - mult[rank.clamp(max=7), prow] * qx).clamp(min=0.0)
        accept = u * qx * mass[rank.clamp(max=7), prow] < w
    accept = accept & child
    taken = accept & ~(before & accept[:, None, :]).any(2)
    broken = (~taken & (par >= 0)).float()
    kept = there & ((reach.float() @ broken[:, :, None])[..., 0] == 0)
    last = torch.where(kept, node, torch.zeros_like(rows)).amax(1)
    lens = kept.sum(1)
    path = torch.full((n, s["max_path"] + 1), -1, dtype=torch.int32, device=rows.device)
    place = torch.where(kept, kept.cumsum(1) - 1, torch.full_like(rows, s["max_path"]))
    path = path.scatter(1, place, node.to(torch.int32).expand(n, t))[:, :s["max_path"]]
    row = rows.gather(1, last[:, None])[:, 0]
    p = target[row].double()
    if draft is None:
        tried = child & (par == last[:, None])
        wide = torch.cat([p, p[:, :1]], 1)
        w = wide.scatter(1, torch.where(tried, tok, torch.full_like(tok, p.shape[1])), 0.0)[:, :-1]
    else:
        m = kids.gather(1, last[:, None])[:, 0]
        w = (p - mult[m, row][:, None] * draft[row].double()).clamp(min=0.0)
    cum = w.cumsum(1)
    # Nothing left after the refusals: drawn from the target itself.
    cum = torch.where(cum[:, -1:] > 0, cum, p.cumsum(1))
    tau = s["u_sample"].double()[:, None] * cum[:, -1:]
    return path.contiguous(), lens.to(torch.int32), (cum <= tau).sum(1).to(torch.int32)


def _plain_compact(s):
    b = s["case"]["block"]
    k = torch.arange(s["path"].shape[1], device=s["path"].device)
    ctx = s["ctx"].long()[:, None]
    # Past the path's end: the first row once more.
    live = k < s["path_lens"][:, None]
    src = ctx + torch.where(live, s["path"].long(), s["path"].long()[:, :1])
    dst = ctx + torch.where(live, k, torch.zeros_like(k))
    table = s["table"].long()
    sb, so = table.gather(1, src // b), src % b
    db, do = table.gather(1, dst // b), dst % b
    if s["scales"] is None:
        s["k"][:, db, :, do] = s["k"][:, sb, :, so]
        s["v"][:, db, :, do] = s["v"][:, sb, :, so]
        return s["k"], s["v"]
    first = ctx // b
    keep = ctx % b  # offsets below it hold committed tokens, in the first block alone
    b0 = table.gather(1, first)[:, 0]
    same = (dst // b)[:, :, None] == (dst // b)[:, None, :]  # rows that land in one block
    scales = s["scales"].clone()
    _move_8bit(s, s["k"], scales, 0, sb, so, db, do, b0, keep, same, dst // b == first)
    _move_8bit(s, s["v"], scales, 1, sb, so, db, do, b0, keep, same, dst // b == first)
    return _cache_values(s)


def _move_8bit(s, pool, old, which, sb, so, db, do, b0, keep, same, in_first):
    """Rows of one 8-bit pool into their new places, each block under the
    largest scale of the rows that stay in it."""
    t = FP8[s["case"]["dtype"]][0]
    one = torch.ones((), device=pool.device)
    sc = old[..., which]  # [layers, blocks, heads]
    s_src = sc[:, sb]  # [layers, n, k, heads]
    s_new = torch.where(same[None, :, :, :, None], s_src[:, :, None], 0.0).amax(3)
    s_kept = torch.where(keep > 0, sc[:, b0].permute(0, 2, 1).unsqueeze(-1), 0.0).permute(0, 2, 3, 1)
    s_new = torch.maximum(s_new, torch.where(in_first[None, :, :, None], s_kept, 0.0))
    codes = pool[:, sb, :, so]  # [n, k, layers, heads, d]
    ratio = torch.where(s_new > 0, s_src / s_new, one).permute(1, 2, 0, 3).unsqueeze(-1)
    moved = (codes.view(t).float() * ratio).to(t).view(torch.uint8)
    block = pool[:, b0]  # [layers, n, heads, block, d]
    n0 = s_new[:, :, 0]  # the first row always lands in the first block
    o0 = sc[:, b0]
    r0 = torch.where((n0 > o0) & (o0 > 0), o0 / n0, one)[..., None, None]
    again = (block.view(t).float() * r0).to(t).view(torch.uint8)
    under = torch.arange(block.shape[3], device=pool.device) < keep
    pool[:, b0] = torch.where(under[None, :, None, :, None], again, block)
    pool[:, db, :, do] = moved
    s["scales"][:, db, :, which] = s_new


# ---------------------------------------------------------------------------
# What a pass costs at least
# ---------------------------------------------------------------------------

def work(case):
    t = case["nodes"]
    counts = _lengths(case, t - t // 2, t)
    nodes = sum(counts)
    size = {"f32": 4, "f16": 2, "bf16": 2}.get(case["dtype"], 1)
    if case["op"] == "tree":
        io = 4 if case["dtype"] == "f32" else 2
        lens = [a + b for a, b in zip(_lengths(case, max(1, case["ctx"] // 4), case["ctx"]), counts)]
        kv = sum(lens) * 2 * case["hkv"] * case["d"] * size
        pairs = sum(a * b for a, b in zip(counts, lens))
        return {"bytes": kv + 2 * nodes * case["hq"] * case["d"] * io, "flops": 4 * pairs * case["hq"] * case["d"]}
    if case["op"] == "verify":
        # The row that the next token is drawn from, and two values a node.
        wide = 2 if case["draft"] else 1
        return {"bytes": case["seqs"] * case["vocab"] * size * wide + nodes * (8 + 2 * size * wide),
                "flops": 3 * case["seqs"] * case["vocab"]}
    # About (1 + min(8, nodes)) / 2 rows a sequence, read and written, K and V.
    rows = case["seqs"] * (1 + min(8, case["nodes"])) / 2
    return {"bytes": rows * 4 * case["layers"] * case["hkv"] * case["d"] * size, "flops": 0}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "compact": _exact_compact}[case["op"]](s)


def _ancestors(parents, j):
    up = []
    while j >= 0:
        up.append(j)
        j = parents[j]
    return up


def _exact_tree(s):
    c, b = s["case"], s["case"]["block"]
    cu, ctx, parents = s["cu"].tolist(), s["ctx"].tolist(), s["parents"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    g = c["hq"] // c["hkv"]
    for i in range(c["seqs"]):
        lo, hi = cu[i], cu[i + 1]
        n, length = hi - lo, ctx[i] + hi - lo
        blocks = s["table"][i, :-(-length // b)].long()
        keep = torch.zeros(n, n, dtype=torch.bool)
        for j in range(n):
            keep[j, _ancestors(parents[lo:hi], j)] = True
        keep = keep.to(out.device).repeat_interleave(g, 0)
        for h in range(c["hkv"]):
            kv = []
            for which, pool in enumerate((s["k"], s["v"])):
                x = pool[blocks, h]
                if s["scales"] is None:
                    x = x.double()
                else:
                    x = x.view(FP8[c["dtype"]][0]).double() * s["scales"][blocks, h, which].double()[:, None, None]
                kv.append(x.reshape(-1, c["d"])[:length])
            q = s["q"][lo:hi, h * g:(h + 1) * g].double().reshape(n * g, c["d"])
            score = (q @ kv[0].T) * s["scale"]
            score[:, ctx[i]:].masked_fill_(~keep, -math.inf)
            out[lo:hi, h * g:(h + 1) * g] = (torch.softmax(score, 1) @ kv[1]).reshape(n, g, c["d"])
    return out


def _exact_verify(s):
    cu, parents, tokens = s["cu"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    ua, us = s["u_accept"].double().tolist(), s["u_sample"].double().tolist()
    n = len(us)
    path = torch.full((n, s["max_path"]), -1, dtype=torch.int32)
    lens, nexts = [], []
    for i in range(n):
        lo, hi = cu[i], cu[i + 1]
        at, kept = 0, [0]
        while True:
            p = s["target"][lo + at].double().cpu()
            q = None if s["draft"] is None else s["draft"][lo + at].double().cpu()
            w, mass, step = p.clone(), 1.0, None
            for j in range(at + 1, hi - lo):
                if parents[lo + j] != at:
                    continue
                x = tokens[lo + j]
                if ua[lo + j] * (1.0 if q is None else float(q[x])) * mass < float(w[x]):
                    step = j
                    break
                if q is None:
                    mass -= float(w[x])
                    w[x] = 0.0
                else:
                    w = (w - mass * q).clamp(min=0.0)
                    mass = float(w.sum())
            if step is None:
                break
            at = step
            kept.append(at)
        cum = w.cumsum(0)
        if float(cum[-1]) <= 0:
            cum = p.cumsum(0)
        nexts.append(int((cum <= us[i] * cum[-1]).sum()))
        path[i, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
        lens.append(len(kept))
    return path, torch.tensor(lens, dtype=torch.int32), torch.tensor(nexts, dtype=torch.int32)


def _nearest(x, name):
    """The 8-bit value nearest to each x, ties to the even code."""
    t = FP8[name][0]
    codes = torch.arange(128, dtype=torch.uint8)
    val = codes.view(t).double()
    val = val[torch.isfinite(val)].to(x.device)
    a = x.abs()
    up = torch.searchsorted(val, a).clamp(max=val.numel() - 1)
    dn = (up - 1).clamp(min=0)
    du, dd = val[up] - a, a - val[dn]
    pick = torch.where((dd < du) | ((dd == du) & (dn % 2 == 0)), dn, up)
    return torch.copysign(val[pick], x)


def _exact_compact(s):
    c, b = s["case"], s["case"]["block"]
    ctx, lens, path, table = (s[x].tolist() for x in ("ctx", "path_lens", "path", "table"))
    if s["scales"] is None:
        pools = [s["k"].clone(), s["v"].clone()]
        for i in range(c["seqs"]):
            for new, old in zip(pools, (s["k"], s["v"])):
                for j in range(lens[i]):
                    x, y = ctx[i] + path[i][j], ctx[i] + j
                    new[:, table[i][y // b], :, y % b] = old[:, table[i][x // b], :, x % b]
        return tuple(pools)
    t = FP8[c["dtype"]][0]
    scales = s["scales"].clone()
    pools = []
    for which, pool in enumerate((s["k"], s["v"])):
        val = pool.view(t).float()
        old = s["scales"][..., which]
        new = val.clone()
        for i in range(c["seqs"]):
            moves = [(ctx[i] + path[i][j], ctx[i] + j) for j in range(lens[i])]
            for lb in sorted({y // b for _, y in moves}):
                here = [(x, y) for x, y in moves if y // b == lb]
                blk, kept = table[i][lb], here[0][1] % b
                sc = [old[:, table[i][x // b]] for x, _ in here] + ([old[:, blk]] if kept else [])
                top = torch.stack(sc).amax(0)
                safe = torch.where(top > 0, top, torch.ones_like(top))
                if kept:
                    r = torch.where(top > 0, old[:, blk] / safe, 1.0)[..., None, None]
                    r = torch.where(old[:, blk][..., None, None] > 0, r, torch.ones_like(r))
                    new[:, blk, :, :kept] = _nearest((val[:, blk, :, :kept] * r).double(), c["dtype"]).float()
                for x, y in here:
                    r = torch.where(top > 0, old[:, table[i][x // b]] / safe, 1.0)[..., None]
                    new[:, blk, :, y % b] = _nearest((val[:, table[i][x // b], :, x % b] * r).double(),
                                                     c["dtype"]).float()
                scales[:, blk, :, which] = top
        pools.append(new)
    return pools[0], pools[1], scales
