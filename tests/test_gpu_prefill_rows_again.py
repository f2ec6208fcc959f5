"""m3_prefill_rows again after m3_kv_alloc: what a context holds for packed prompts fits any cache of it."""
import dataclasses

import pytest
import torch

import synth
from gpu_util import Model, bits, f32, rel_err

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first,then", [(1, 4), (2, 3), (4, 2)])
def test_a_cache_of_other_rows(ora, first, then):
    from autoregressive_audio_token_b200 import m3
    s = dataclasses.replace(synth.TINY, n_layers=2)
    m = Model(s, seed=5, max_rows=4, oracle=False)
    try:
        lens = [9, 4, 17, 6]
        x = synth.normal((sum(lens), s.hidden), 5, "p", std=0.02).cuda()
        h = torch.zeros((4, s.hidden), dtype=torch.bfloat16, device="cuda")
        m3.m3_kv_alloc(m.ctx, first, 32, 0, 32)
        m3.m3_prefill_rows(m.ctx, list(range(first)), lens[:first], x[:sum(lens[:first])].contiguous(), h[:first])
        m3.m3_kv_alloc(m.ctx, then, 32, 0, 32)
        # the new cache's pages are the one allocation that the second call makes
        m3.m3_inject_fault(m.ctx, m3.M3_FAULT_ALLOC, 2)
        h.zero_()
        rows = list(range(then))[::-1]
        m3.m3_prefill_rows(m.ctx, rows, lens[:then], x[:sum(lens[:then])].contiguous(), h[:then])
        m3.m3_inject_fault(m.ctx, m3.M3_FAULT_NONE, 1)
        one, at = torch.zeros_like(h), 0
        m3.m3_kv_alloc(m.ctx, then, 32, 0, 32)
        for i, (r, n) in enumerate(zip(rows, lens)):
            m3.m3_prefill(m.ctx, r, 0, x[at:at + n].contiguous(), one[i])
            at += n
        torch.cuda.synchronize()
        m3.m3_sync_status(m.ctx)
        assert rel_err(f32(bits(h[:then])), f32(bits(one[:then]))) <= 2e-2
    finally:
        m.close()
