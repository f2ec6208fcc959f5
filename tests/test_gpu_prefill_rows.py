"""GPU parity of the packed prompt prefill (m3_prefill_rows) against the CPU oracle.

Prefilling several cache rows at once is defined as m3_prefill row by row, that is as decoding each
prompt's tokens one by one; the oracle runs exactly that.  Compared: every row's K/V of every layer,
each prompt's last hidden state, the rows that were not named, and a decode frame on the result.
Tolerance: the bf16 logit bar, 2e-2 of the largest magnitude (int8: 5e-2), as for m3_prefill.
"""
import dataclasses

import numpy as np
import pytest
import torch

import synth
from gpu_util import Model, bits, check_codes_teacher_forced, f32, rel_err

pytestmark = pytest.mark.gpu

TWO_LAYERS = dataclasses.replace(synth.TINY, n_layers=2)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def f16(a):
    return a.view(np.float16).astype(np.float32)


@pytest.mark.parametrize("rows,lens,chunk,wdtype,kv_f16", [
    ([0, 1], [37, 150], 256, 0, False),
    ([3, 0, 2], [1, 70, 129], 2048, 0, False),
    ([2, 1], [64, 33], 256, 0, True),         # f16 cache
    ([1, 0, 3, 2], [30, 33, 70, 20], 64, 0, False),  # two packed passes around a prompt past the chunk
    ([1, 0], [20, 9], 64, 1, False),          # int8: one by one
])
def test_prefill_rows_matches_sequential_decode(ora, rows, lens, chunk, wdtype, kv_f16, monkeypatch):
    monkeypatch.setenv("M3_PREFILL_CHUNK", str(chunk))
    s = TWO_LAYERS
    m = Model(s, seed=41, max_rows=4, wdtype=wdtype, kv_f16=kv_f16)
    try:
        top = max(lens) + 8
        kc, vc = m.kv_setup(rows=4, n_prefill=0, max_pos=top, bucket=32)
        xs = [synth.normal((n, s.hidden), 41, f"prompt{i}", std=0.02) for i, n in enumerate(lens)]
        h_last = torch.empty((len(rows), s.hidden), dtype=torch.bfloat16, device="cuda")
        m.m3.m3_prefill_rows(m.ctx, rows, lens, torch.cat(xs).cuda(), h_last)
        torch.cuda.synchronize()
        m.m3.m3_sync_status(m.ctx)
        tol = 2e-2 if wdtype == 0 else 5e-2
        val = f16 if kv_f16 else f32
        for i, (r, n) in enumerate(zip(rows, lens)):
            xb = bits(xs[i])
            for t in range(n):
                x_out = m.ora.body(kc[r:r + 1], vc[r:r + 1], [t], xb[t:t + 1].copy())
            gk, gv = m.m3.m3_kv_get(m.ctx, r, s.n_layers, n, s.n_kv_heads, s.head_dim)
            gk, gv = gk.numpy().view(np.uint16), gv.numpy().view(np.uint16)
            for l in range(s.n_layers):
                assert rel_err(val(gk[l]), val(kc[r, l, :n])) <= tol, ("K", r, l)
                assert rel_err(val(gv[l]), val(vc[r, l, :n])) <= tol, ("V", r, l)
            href = ora.rmsnorm(f32(x_out[0]), bits(m.final_norm), s.rms_eps)
            assert rel_err(f32(bits(h_last[i])), href) <= tol, r
        for r in set(range(4)) - set(rows):
            gk, _ = m.m3.m3_kv_get(m.ctx, r, s.n_layers, max(lens), s.n_kv_heads,
                                   s.head_dim)
            assert not gk.numpy().any()
        # a frame decoded on the prefilled rows
        pos = [0] * 4
        for r, n in zip(rows, lens):
            pos[r] = n
        x = synth.frame_input(s, 4, 42, 0)
        codes, h, lg = m.decode(pos, seed=4, frame=7, x_in=x)
        oc, oh, olg = m.ora.decode_frame(kc, vc, pos, 4, 7, bits(x))
        assert rel_err(lg, olg) <= tol
        check_codes_teacher_forced(m, h, codes, 4, 7)
    finally:
        m.close()


def test_prefill_rows_8b_layer(ora):
    # one Qwen3-8B layer, a pair of prompts: four query heads a KV head, 128 dims
    s = synth.LAYER8B
    m = Model(s, seed=43, device="cuda", max_rows=2)
    try:
        lens = [70, 41]
        kc, vc = m.kv_setup(rows=2, n_prefill=0, max_pos=80, bucket=64)
        xs = synth.normal((sum(lens), s.hidden), 43, "prompts8b", std=0.02)
        h_last = torch.empty((2, s.hidden), dtype=torch.bfloat16, device="cuda")
        m.m3.m3_prefill_rows(m.ctx, [1, 0], lens, xs.cuda(), h_last)
        torch.cuda.synchronize()
        m.m3.m3_sync_status(m.ctx)
        xb, at = bits(xs), 0
        for i, (r, n) in enumerate(zip([1, 0], lens)):
            for t in range(n):
                x_out = m.ora.body(kc[r:r + 1], vc[r:r + 1], [t], xb[at + t:at + t + 1].copy())
            at += n
            gk, gv = m.m3.m3_kv_get(m.ctx, r, s.n_layers, n, s.n_kv_heads, s.head_dim)
            assert rel_err(f32(gk.numpy().view(np.uint16)[0]), f32(kc[r, 0, :n])) <= 2e-2
            assert rel_err(f32(gv.numpy().view(np.uint16)[0]), f32(vc[r, 0, :n])) <= 2e-2
            href = ora.rmsnorm(f32(x_out[0]), bits(m.final_norm), s.rms_eps)
            assert rel_err(f32(bits(h_last[i])), href) <= 2e-2
    finally:
        m.close()


def test_prefill_rows_argument_errors(ora):
    from autoregressive_audio_token_b200 import m3
    s = TWO_LAYERS
    m = Model(s, seed=2, max_rows=4, oracle=False)
    try:
        x = synth.normal((10, s.hidden), 2, "p", std=0.02).cuda()

        def code(rows, lens, xx=x):
            with pytest.raises(m3.M3Error) as e:
                m3.m3_prefill_rows(m.ctx, rows, lens, xx)
            return e.value.code

        assert code([0], [10]) == m3.M3_ESTATE  # no KV cache yet
        m3.m3_kv_alloc(m.ctx, 2, 16, 0, 32)
        assert code([0, 0], [5, 5]) == m3.M3_EINVAL
        assert code([0, 2], [5, 5]) == m3.M3_EINVAL
        assert code([-1], [10]) == m3.M3_EINVAL
        assert code([0, 1], [10, 0]) == m3.M3_EINVAL
        assert code([0, 1, 1], [4, 4, 2]) == m3.M3_EINVAL
        assert code([], [], x[:0]) == m3.M3_EINVAL
        big = synth.normal((17, s.hidden), 2, "p", std=0.02).cuda()
        assert code([1], [17], big) == m3.M3_ECAPACITY
        m3.m3_prefill_rows(m.ctx, [1, 0], [4, 6], x)
        # a failed allocation leaves the context usable
        m3.m3_sync_status(m.ctx)
    finally:
        m.close()


def test_prefill_rows_after_a_failed_allocation(ora):
    from autoregressive_audio_token_b200 import m3
    s = TWO_LAYERS
    m = Model(s, seed=3, max_rows=2, oracle=False)
    try:
        x = synth.normal((12, s.hidden), 3, "p", std=0.02).cuda()
        m3.m3_kv_alloc(m.ctx, 2, 32, 0, 32)
        h = torch.zeros((2, s.hidden), dtype=torch.bfloat16, device="cuda")
        failed = 0
        while failed < 30:  # each time one allocation further: the cache, the pass's buffers, copies, maps
            m3.m3_inject_fault(m.ctx, m3.M3_FAULT_ALLOC, 2)
            try:
                m3.m3_prefill_rows(m.ctx, [0, 1], [5, 7], x, h)
                break
            except m3.M3Error as e:
                assert e.code == m3.M3_ENOMEM
                failed += 1
        assert 8 <= failed < 30
        m3.m3_inject_fault(m.ctx, m3.M3_FAULT_NONE, 1)
        m3.m3_prefill_rows(m.ctx, [0, 1], [5, 7], x, h)
        one = torch.zeros_like(h)
        m3.m3_prefill(m.ctx, 0, 0, x[:5].contiguous(), one[0])
        m3.m3_prefill(m.ctx, 1, 0, x[5:].contiguous(), one[1])
        torch.cuda.synchronize()
        m3.m3_sync_status(m.ctx)
        assert rel_err(f32(bits(h)), f32(bits(one))) <= 2e-2
    finally:
        m.close()
