"""Attention with modified scores where calls, workspaces and roundings meet: runs of calls without
a wait between them, ragged tiles under a cap, weights and slopes of the smallest sizes, what padded
rows may hold in every form, scratch under memory pressure and capture, overlaps, and tensors that a
caller lets go of.
"""
import numpy as np
import pytest
import torch

import encoder_inputs as EI
from oracle import scored_oracle as SO
from parity_utils import encoder_from_inputs, to_dev
from test_gpu_scored import Case, encoder

pytestmark = pytest.mark.gpu


def fresh_encoder(nh, d, mode):
    """A handle that holds no scratch yet."""
    enc = encoder_from_inputs(EI.make_inputs(EI.Workload("scored", EI.EncoderShape(nh, d, 64, 1), 1, 1, mode[:4], 1, 1, seed=0)))
    enc.set_option("tc_attention", mode != "fp16-simt")
    return enc


# ---------------------------------------------------------------- calls one after the other
@pytest.mark.parametrize("mode", ["fp16", "fp16-simt", "fp32"])
@pytest.mark.parametrize("nh,d,s", [(3, 64, 300), (2, 128, 700), (4, 32, 131)], ids=str)
@pytest.mark.parametrize("pdl", [True, False], ids=["pdl", "no-pdl"])
def test_inputs_that_alternate_through_one_handle(pdl, nh, d, s, mode):
    """Backward calls of different data one behind the other share the scratch: each gets its own statistics."""
    cases = [Case("table-docs", mode, 2, nh, s, d, seed=20 + i, std=(1.0, 0.3, 2.0)[i]) for i in range(3)]
    enc = encoder(nh, d, mode)
    enc.set_option("pdl", pdl)
    try:
        args, want = [], []
        for c in cases:
            ctx, lse = c.forward()
            want.append(c.backward(ctx, lse))
            args.append((c.scores(), to_dev(c.qkv), to_dev(c.valid), ctx, lse, to_dev(c.dctx).view(2 * s, -1)))
        order = [0, 1, 2, 1, 0, 2, 2, 0, 1] * 3
        got = [(torch.empty_like(want[i][0]), torch.empty_like(want[i][1])) for i in order]
        torch.cuda.synchronize()
        for i, (dqkv, dtable) in zip(order, got):
            enc.op_scored_attention_backward(*args[i], dqkv, 2, s, dtable=dtable)
        torch.cuda.synchronize()
    finally:
        enc.set_option("pdl", True)
    assert enc.device_status() == 0
    for i, x in zip(order, got):
        assert torch.equal(want[i][0], x[0]) and torch.equal(want[i][1], x[1])
