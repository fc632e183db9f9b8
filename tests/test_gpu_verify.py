"""Verification of drafted tokens against the fp64 oracle: whole numbers, so
equal. A drawn token could differ only where the sample lies within the
sums' rounding (2^-43 a weight) of a border, about one sample in 10^6."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.draft_tree as ot
from tree_helpers import DT, random_parents

pytestmark = pytest.mark.gpu


def case(seed, dtype, nodes, vocab, draft=True, kind="random", temp=3.0, near=1.0):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    T = int(cu[-1])
    parents = np.array(sum((random_parents(rng, n, kind) for n in nodes), []), np.int32)
    lg = torch.from_numpy(rng.standard_normal((T, vocab)).astype(np.float32)) * temp
    lq = lg + near * torch.from_numpy(rng.standard_normal((T, vocab)).astype(np.float32))
    p, q = torch.softmax(lg, -1).to(DT[dtype]), torch.softmax(lq, -1).to(DT[dtype])
    tok = np.zeros(T, np.int32)
    for i in range(len(nodes)):
        for j in range(nodes[i]):
            row = q[cu[i] + max(parents[cu[i] + j], 0)].double().numpy()
            tok[cu[i] + j] = rng.choice(vocab, p=row / row.sum())
    return dict(target=p, draft=q if draft else None, tokens=tok, cu=cu, parents=parents,
                ua=rng.random(T, dtype=np.float32), us=rng.random(len(nodes), dtype=np.float32),
                max_path=max(1, max(nodes)))


def call(lib, c, pad=0, **over):
    t = lambda x: torch.as_tensor(x).cuda()  # noqa: E731

    def rows(x):
        if x is None:
            return None
        wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, :x.shape[1]] = x.cuda()
        return wide[:, :x.shape[1]]

    a = dict(target_probs=rows(c["target"]), draft_probs=rows(c["draft"]), draft_tokens=t(c["tokens"]),
             cu_q_lens=t(c["cu"]), parents=t(c["parents"]), uniform_accept=t(c["ua"]), uniform_sample=t(c["us"]),
             max_q_len=max(1, int(np.diff(c["cu"]).max())), max_path_len=c["max_path"])
    a.update(over)
    return lib.pa_verify_tree(**a)


def check(lib, c, pad=0, status=0):
    got = call(lib, c, pad)
    assert lib.pa_get_status() == status
    ref = ot.verify_tree(c["target"], c["draft"], c["tokens"], c["cu"], c["parents"], c["ua"], c["us"], c["max_path"])
    for name, g, r in zip(("path", "path_lens", "next_tokens"), got, ref):
        assert g.dtype == torch.int32
        assert np.array_equal(g.cpu().numpy(), r), (name, g.cpu().numpy(), r)
    return ref


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 32, 33, 127, 1000, 4099, 32000])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_trees(lib, dtype, vocab, draft, pad):
    nodes = [1, 2, 5, 16, 40, 3, 8, 8]
    check(lib, case(vocab + 10 * len(dtype), dtype, nodes, vocab, draft, near=0.7), pad)


@pytest.mark.parametrize("kind", ["chain", "star", "forest"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("near", [0.0, 0.3, 3.0])
def test_kinds(lib, kind, draft, near):
    check(lib, case(5, "f32", [30, 9, 64, 1], 500, draft, kind, near=near))


@pytest.mark.parametrize("seqs", [1, 3, 9, 20, 40, 80, 160, 400])
@pytest.mark.parametrize("draft", [True, False])
def test_batches(lib, seqs, draft):
    """Every split of a row over the machine."""
    check(lib, case(seqs, "f32", [1 + i % 5 for i in range(seqs)], 3001, draft))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_vocabulary(lib, dtype):
    check(lib, case(6, dtype, [4, 3], 262144))


def test_largest_tree(lib):
    for kind in ("chain", "star"):
        for draft in (True, False):
            c = case(7, "f32", [1024], 50, draft, kind, near=0.05)
            if kind == "star":
                c["ua"][:] = 0.999999  # many refusals
            check(lib, c)


def test_the_same_token_twice(lib):
    for draft in (True, False):
        c = case(8, "f32", [9, 9], 40, draft, "star")
        c["tokens"][:] = 5
        c["tokens"][3] = 6
        c["ua"][:] = 0.9999
        check(lib, c)


def test_short_paths(lib):
    for longest in (1, 2, 3):
        c = case(9, "f32", [20, 7, 1], 300, kind="chain", near=0.0)
        c["max_path"] = longest
        ref = check(lib, c)
        assert ref[1].max() == longest


def test_padding_tokens_and_no_nodes(lib):
    c = case(10, "f32", [6, 0, 9, 0], 300, near=0.1)
    c["tokens"][[1, 8]] = -1
    c["tokens"][[3, 9]] = 300
    ref = check(lib, c)
    assert list(ref[1][[1, 3]]) == [0, 0] and list(ref[2][[1, 3]]) == [-1, -1]


@pytest.mark.parametrize("us", [0.0, 2.0 ** -30, 0.5, 1.0 - 2.0 ** -24])
def test_ends_of_the_distribution(lib, us):
    """Rows with zeros at both ends: a token without weight is never drawn."""
    for dtype in ("f32", "bf16"):
        c = case(11, dtype, [3] * 6, 1003)
        for x in (c["target"], c["draft"]):
            x[:, :17] = 0
            x[:, -29:] = 0
        c["us"][:] = us
        ref = check(lib, c)
        assert ref[2].min() >= 17 and ref[2].max() < 1003 - 29


def test_one_sure_token(lib):
    c = case(12, "f32", [4, 4], 777)
    c["target"].zero_()
    c["target"][:, 776] = 1.0
    ref = check(lib, c)
    assert (ref[2] == 776).all()


def test_equal_rows_leave_nothing(lib):
    """p = q and a refusal (u q < p fails for u = 1 - 2^-24 only by rounding,
    so the token is given no probability): the residual is empty."""
    c = case(13, "f32", [2, 2, 2], 64, near=0.0)
    c["draft"] = c["target"].clone()
    for i in range(3):
        c["target"][2 * i, c["tokens"][2 * i + 1]] = 0
        c["draft"][2 * i, c["tokens"][2 * i + 1]] = 0
    ref = check(lib, c)
    assert (ref[1] == 1).all()


def test_not_probabilities(lib):
    c = case(14, "f32", [4, 4, 4], 100)
    c["target"][0, 3], c["target"][4, 50], c["target"][8, 99] = float("nan"), -1.0, 2.0
    c["draft"][0, 5], c["draft"][4, 51], c["draft"][8, 0] = float("nan"), -3.0, float("inf")
    check(lib, c)
    c["target"][4:8] = float("nan")
    ref = check(lib, c, status=-1)
    assert ref[2][1] == -1


def test_the_tokens_follow_the_target(lib):
    """One drafted token, many sequences: kept or not, the first token is
    distributed as the target says (5 standard deviations)."""
    rng = np.random.default_rng(15)
    n, vocab = 60000, 12
    p = rng.dirichlet(np.ones(vocab)).astype(np.float32)
    q = rng.dirichlet(np.ones(vocab)).astype(np.float32)
    for draft, children in ((True, 1), (True, 3), (False, 3)):
        T = n * (1 + children)
        cu = np.arange(0, T + 1, 1 + children).astype(np.int32)
        tok = rng.choice(vocab, size=(n, 1 + children), p=q.astype(np.float64) / q.astype(np.float64).sum())
        if not draft:
            tok[:, 1:] = [3, 1, 7]
        c = dict(target=torch.from_numpy(np.tile(p, (T, 1))), draft=torch.from_numpy(np.tile(q, (T, 1))) if draft else None,
                 tokens=tok.reshape(-1).astype(np.int32), cu=cu,
                 parents=np.tile([-1] + [0] * children, n).astype(np.int32), ua=rng.random(T, dtype=np.float32),
                 us=rng.random(n, dtype=np.float32), max_path=2)
        path, lens, nxt = (x.cpu().numpy() for x in call(lib, c))
        assert lib.pa_get_status() == 0
        first = np.where(lens == 2, tok[np.arange(n), np.maximum(path[:, 1], 0)], nxt)
        got = np.bincount(first, minlength=vocab) / n
        dev = 5 * np.sqrt(p * (1 - p) / n)
        assert (np.abs(got - p) <= dev).all()


def test_bad_trees(lib):
    c = case(16, "f32", [5, 5, 5], 100)
    ref = [x.cpu() for x in call(lib, c)]
    for node, up in ((5, 0), (7, 2), (7, 4), (7, -2), (9, 2 ** 30)):
        b = dict(c, parents=c["parents"].copy())
        b["parents"][node] = up
        got = [x.cpu() for x in call(lib, b)]
        assert lib.pa_get_status() == -1
        assert got[1][1] == 0 and got[2][1] == -1 and (got[0][1] == -1).all()
        for g, r in zip(got, ref):
            assert torch.equal(g[[0, 2]], r[[0, 2]])
    for cu in ([0, 5, 3, 15], [0, 5, 10, 99], [-1, 5, 10, 15]):
        got = call(lib, dict(c, cu=np.array(cu, np.int32)), max_q_len=20)
        assert lib.pa_get_status() == -8
    got = call(lib, c, max_q_len=4)
    assert lib.pa_get_status() == -8 and (got[1] == 0).all()


def test_captured_and_replayed(lib):
    c = case(17, "f32", [9, 4, 1], 5000)
    t = lambda x: torch.as_tensor(x).cuda()  # noqa: E731
    a = dict(target_probs=t(c["target"]), draft_probs=t(c["draft"]), draft_tokens=t(c["tokens"]), cu_q_lens=t(c["cu"]),
             parents=t(c["parents"]), uniform_accept=t(c["ua"]), uniform_sample=t(c["us"]), max_q_len=16,
             max_path_len=c["max_path"], path=torch.empty(3, c["max_path"], dtype=torch.int32, device="cuda"),
             path_lens=torch.empty(3, dtype=torch.int32, device="cuda"),
             next_tokens=torch.empty(3, dtype=torch.int32, device="cuda"))
    lib.pa_verify_tree(**a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.pa_verify_tree(**a)
    for seed in (18, 19):
        d = case(seed, "f32", [9, 4, 1], 5000)
        for name, key in (("target_probs", "target"), ("draft_probs", "draft"), ("draft_tokens", "tokens"),
                          ("parents", "parents"), ("uniform_accept", "ua"), ("uniform_sample", "us")):
            a[name].copy_(t(d[key]))
        g.replay()
        torch.cuda.synchronize()
        ref = ot.verify_tree(d["target"], d["draft"], d["tokens"], d["cu"], d["parents"], d["ua"], d["us"],
                             d["max_path"])
        for x, r in zip((a["path"], a["path_lens"], a["next_tokens"]), ref):
            assert np.array_equal(x.cpu().numpy(), r)


def test_weights_between_neighbouring_floats(lib):
    """Two refusals leave C = 1 + S with S just above 2^-24: token 3 weighs
    p - C q > 0 although p < fl(fl(C) q), which lies across a multiple of
    2^-22 from p. It weighs little, token 599 a thousand times as much."""
    c = case(15, "f32", [3], 600, kind="star")
    ulp = 2.0 ** -33
    p3 = 7782.5 * 2.0 ** -22
    for name, at3, at599 in (("target", p3, 0.75), ("draft", p3 - ulp, 0.75 - 2.0 ** -24)):
        c[name].zero_()
        c[name][0, 3], c[name][0, 599] = at3, at599
    c["tokens"][:] = [0, 5, 6]  # no probability: refused
    c["us"][:] = 0.5
    ref = check(lib, c)
    assert ref[2][0] == 599


def test_rows_in_different_lines(lib):
    """Target and draft rows that start at different places of their 16-byte lines."""
    for seed, dtype in ((16, "f32"), (17, "bf16")):
        c = case(seed, dtype, [5, 1, 7], 5000)
        t, d = (torch.zeros(13, 5000 + 16, dtype=DT[dtype], device="cuda") for _ in range(2))
        t[:, 3:5003], d[:, 1:5001] = c["target"].cuda(), c["draft"].cuda()
        got = call(lib, c, target_probs=t[:, 3:5003], draft_probs=d[:, 1:5001])
        ref = ot.verify_tree(c["target"], c["draft"], c["tokens"], c["cu"], c["parents"], c["ua"], c["us"],
                             c["max_path"])
        for g, r in zip(got, ref):
            assert np.array_equal(g.cpu().numpy(), r)


def test_on_another_stream(lib):
    """Outputs made for another stream do not take memory that the current
    stream still has to read."""
    c = case(18, "f32", [6] * 500, 200)
    a = dict(target_probs=c["target"].cuda(), draft_probs=c["draft"].cuda(), draft_tokens=torch.as_tensor(c["tokens"]).cuda(),
             cu_q_lens=torch.as_tensor(c["cu"]).cuda(), parents=torch.as_tensor(c["parents"]).cuda(),
             uniform_accept=torch.as_tensor(c["ua"]).cuda(), uniform_sample=torch.as_tensor(c["us"]).cuda(),
             max_q_len=6, max_path_len=6)
    ref = [x.clone() for x in lib.pa_verify_tree(**a)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.full(sh, 7, dtype=torch.int32, device="cuda") for sh in ((500, 6), (500,), (500,))]
    torch.cuda._sleep(50_000_000)
    kept = [x.clone() for x in old]
    del old
    got = lib.pa_verify_tree(**a, stream=s)
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in kept)
    for g, r in zip(got, ref):
        assert torch.equal(g, r)


def test_subnormal_probabilities(lib):
    """u q < p for equal subnormal p and q and the largest u below 1: kept."""
    c = case(19, "f32", [2, 2, 2], 40)
    for i, tiny in enumerate((2.0 ** -149, 2.0 ** -140, 3.0 * 2.0 ** -130)):
        token = c["tokens"][2 * i + 1]
        for name in ("target", "draft"):
            c[name][2 * i, token] = tiny
    c["ua"][:] = 1 - 2.0 ** -24
    ref = check(lib, c)
    assert (ref[1] == 2).all()


def test_masses_above_one(lib):
    """p sums to 1.8, so the first refusal leaves S = 1.3: 0.7 * 0.5 is below
    the second child's weight 0.4, 0.7 * 0.5 * S is not."""
    c = case(20, "f32", [3], 4, kind="star")
    c["target"][0] = torch.tensor([0.0, 0.0, 0.9, 0.9])
    c["draft"][0] = torch.tensor([0.5, 0.0, 0.5, 0.0])
    c["tokens"][:] = [0, 0, 2]
    c["ua"][:] = [0.0, 0.5, 0.7]
    ref = check(lib, c)
    assert ref[1][0] == 1


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rounded_rows_with_masses_above_one(lib, dtype):
    """16-bit rows that sum to a little more than 1 and drafts of other tokens:
    S after the first refusal passes 1, with the second child's random number
    between w / (q S) and w / q."""
    rng = np.random.default_rng(21)
    n, vocab = 64, 2000
    c = case(21, dtype, [3] * n, vocab, kind="star")
    p = torch.softmax(3.0 * torch.from_numpy(rng.standard_normal((3 * n, vocab)).astype(np.float32)), -1).to(DT[dtype])
    q = torch.zeros_like(p)
    between = 0
    for r in range(0, 3 * n, 3):
        order = p[r].argsort()
        low, x = int(order[0]), int((p[r].double() - 1e-6).abs().argmin())
        q[r, x], q[r, low] = 0.75 * p[r, x], 1.0 - 2.0 ** -8
        pr, qr = p[r].double(), q[r].double()
        S, w = float((pr - qr).clamp(min=0).sum()), float(pr[x] - qr[x])
        u = np.float32(w / float(qr[x]) * (1 - 2.0 ** -22))
        c["tokens"][r + 1], c["tokens"][r + 2], c["ua"][r + 1], c["ua"][r + 2] = low, x, 0.999, u
        between += float(u) * float(qr[x]) < w <= float(u) * float(qr[x]) * S
    c["target"], c["draft"] = p, q
    assert between > n // 8
    check(lib, c)


def test_empty_sequences_outside_the_rows(lib):
    """A cu_q_lens that leaves [0, total_q] is reported for a sequence without
    nodes too."""
    c = case(22, "f32", [5, 0, 5], 100)
    check(lib, c)
    for first in (-1, 11, 2 ** 31 - 1):
        got = call(lib, dict(c, cu=np.full(4, first, np.int32)), max_q_len=5)
        assert lib.pa_get_status() == -8
        assert (got[1] == 0).all() and (got[2] == -1).all()
