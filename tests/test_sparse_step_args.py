"""What SparseStep takes and refuses when it is made (no GPU needed)."""
from __future__ import annotations

import pytest
import torch

from paged_kv_cache_14_gb300.step import SparseStep


def make(d=128, dtype=torch.bfloat16, kv=None, layers=2, **over):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool = lambda: torch.zeros(4, 2, 16, d, dtype=torch.uint8 if kv else dtype)  # noqa: E731
    a = dict(k_caches=[pool() for _ in range(layers)], v_caches=[pool() for _ in range(layers)], block_tables=i32(1, 4),
             ctx_lens=i32(1), seq_lens=i32(1), new_seq_ids=i32(1), new_positions=i32(1), cos_sin=torch.zeros(64, d),
             num_q_heads=4, dtype=dtype, max_seq_len=64, max_new_tokens=1, max_list_len=2, scale=0.1)
    if kv:
        a.update(kv_scales=[torch.zeros(4, 2, 2) for _ in range(layers)], kv_format=kv)
    a.update(over)
    return SparseStep(**a)


@pytest.mark.parametrize("dtype,kv,d", [
    (torch.bfloat16, "e4m3", 64), (torch.float16, "e5m2", 64), (torch.float32, "e4m3", 128), (torch.bfloat16, None, 96),
    (torch.float16, None, 256), (torch.float32, None, 48), (torch.float32, None, 288)])
def test_shapes_that_attend_would_refuse(dtype, kv, d):
    """Such a step could write its cache but never attend to it."""
    with pytest.raises(ValueError, match="head_dim"):
        make(d, dtype, kv)


@pytest.mark.parametrize("dtype,kv,d", [
    (torch.bfloat16, "e4m3", 128), (torch.float16, "e5m2", 128), (torch.bfloat16, None, 64), (torch.float16, None, 128),
    (torch.float32, None, 32), (torch.float32, None, 256)])
def test_shapes(dtype, kv, d):
    step = make(d, dtype, kv)
    assert len(step.summaries) == 2 and step.summaries[0].shape == (4, 2, 2, d)


def test_summaries_are_shared():
    """Steps over the same caches (a prompt's chunks, then decode) use one set."""
    prompt = make()
    decode = make(summaries=prompt.summaries, summary_scales=prompt.summary_scales)
    for layer in range(2):
        assert decode.summaries[layer] is prompt.summaries[layer]
        assert decode.summary_scales[layer] is prompt.summary_scales[layer]


def test_summaries_that_do_not_fit():
    step = make()
    for over in (dict(summaries=step.summaries), dict(summary_scales=step.summary_scales),
                 dict(summaries=step.summaries[:1], summary_scales=step.summary_scales[:1]),
                 dict(summaries=[x[:3] for x in step.summaries], summary_scales=step.summary_scales),
                 dict(summaries=step.summaries, summary_scales=[x[:, :1] for x in step.summary_scales]),
                 dict(summaries=[x.float() for x in step.summaries], summary_scales=step.summary_scales)):
        with pytest.raises(ValueError, match="summar"):
            make(**over)
