"""The training calls at the edges of what they allow: shared memory and
workspaces that earlier work left full, limits of sizes, scales and logits that
are not finite, waits that give up."""
import math

import pytest
import torch

from speculative_decoding_verify_ssd_b200 import binding as ssd

from train_testlib import logits_like, top_ref

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
def test_top_blocks_on_used_shared_memory():
    """Thousands of blocks one after the other on shared memory (their barriers'
    places too) that the blocks before them left full."""
    z = logits_like((3000,), 1500, BF16, 71)
    tokens, values, _, _ = top_ref(z, 8, 1.0)
    first = None
    for _ in range(20):
        ssd.ssd_distill(z, tokens, values.float())
        r = ssd.ssd_teacher_top(z, 8)
        assert (r.status == 0).all() and torch.equal(r.tokens, tokens) and torch.equal(r.values.double(), values)
        first = r if first is None else first
        assert torch.equal(r.lse, first.lse) and torch.equal(r.tail, first.tail)
