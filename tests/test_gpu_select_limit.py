"""Choice among as many blocks as a call takes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group,blocks", [(256, 128, 169984), (128, 8, 378752), (128, 1, 378751)])
def test_longest_rows(lib, d, group, blocks):
    g = torch.Generator(device="cuda").manual_seed(d + group)
    P, block, keep = blocks + 3, 16, 700
    hi = torch.randint(-100, 128, (P, 1, d), generator=g, device="cuda")
    lo = hi - torch.randint(0, 28, hi.shape, generator=g, device="cuda")
    codes = torch.stack([hi, lo], 2).to(torch.int8)
    scales = torch.rand(P, 1, generator=g, device="cuda") + 0.5
    q = torch.randn(1, group, d, generator=g, device="cuda")
    table = torch.randperm(P, generator=g, device="cuda")[:blocks].to(torch.int32)[None]
    lens = torch.tensor([blocks * block - 5], dtype=torch.int32, device="cuda")
    lists, counts = lib.pa_select_blocks(q, codes, scales, table, lens, blocks * block, block, keep, 2, 3)
    assert lib.pa_get_status() == 0 and counts.tolist() == [[keep]]
    # The scores, in the header's steps: whole numbers below 2^53, then fp32.
    row = q[0].cpu().numpy()
    sq = np.abs(row).max(1) / np.float32(127)
    qc = torch.from_numpy(np.clip(np.rint(row / sq[:, None]), -127, 127)).cuda().double()
    t = table[0].long()
    whole = qc.clamp(min=0) @ hi[t, 0].double().T + qc.clamp(max=0) @ lo[t, 0].double().T
    best = (torch.from_numpy(sq).cuda()[:, None] * whole.float()).amax(0)
    score = best * scales[t, 0]
    some = score[2:blocks - 3]
    order = torch.sort(some, descending=True, stable=True).indices[:keep - 5] + 2
    mine = torch.cat([torch.arange(2, device="cuda"), order.sort().values, torch.arange(blocks - 3, blocks, device="cuda")])
    assert torch.equal(lists[0, 0].long(), mine)
