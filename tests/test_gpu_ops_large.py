"""The serving operators (include/m3_ops.h) where offsets pass 32 bits: pools, prompts and logits of more than 2^31
elements, checked at their far ends."""
import pytest
import torch

import test_gpu_ops as T
from test_gpu_ops import BF16, F16, F32, _status, gen, i32, ops  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("24 GB of device memory wanted")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_store_and_attend_far_into_a_pool(ops, dtype):
    hq, hk, d, page, n_pages = 16, 8, 128, 256, 4500  # 2.36e9 elements
    pool = torch.zeros(n_pages, 2, hk, page, d, dtype=dtype, device="cuda")
    assert pool.numel() > 2**31
    g = gen(1)
    for n, prefix, lens in ((20, 1500, [13 * i % 400 for i in range(20)]), (2, 300, [40, 256]), (1, 2600, [700])):
        new = lambda k: torch.randn(2, k, hk, d, generator=g, device="cuda").to(dtype)  # noqa: E731
        numbers = iter(range(n_pages - 1, 0, -1))  # from the far end; a near page now and then
        shared, own, pages, table, used = new(prefix), [new(x) for x in lens], [], [], []
        most = max(-(-x // page) for x in lens)
        for i, kv in enumerate([shared] + own):
            mine = [next(numbers) if (i + j) % 3 else 1 + 20 * i + j for j in range(-(-kv.shape[1] // page))]
            used += mine
            slots = torch.tensor([mine[t // page] * page + t % page for t in range(kv.shape[1])], dtype=torch.int64, device="cuda")
            ops.m3_kv_store(kv[0], kv[1], slots, pool)
            if i:
                table.append(mine + [-1] * (most - len(mine)))
            else:
                pages = mine
        assert len(used) == len(set(used))
        q = torch.randn(n, hq, d, generator=g, device="cuda").to(dtype)
        out, lse = torch.empty_like(q), torch.empty(n, hq, device="cuda")
        ops.m3_attn_prefix(q, pool, i32(pages), prefix, i32(table), i32(lens), out, lse)
        T.check_prefix(out, lse, q, shared, own, lens, d ** -0.5, dtype)
        for kv, row, x in zip(own, table, lens):
            if x:
                assert torch.equal(pool[row[0], 0, :, 0], kv[0, 0]) and torch.equal(pool[row[0], 1, :, 0], kv[1, 0])


def test_prompts_of_many_tokens(ops):
    # 8192 sequences, 2.2e9 elements of q and of out; the first, some in between and the last against plain attention
    hq, hk, d = 32, 8, 128
    lens = [65 if i % 4 else 64 for i in range(8191)] + [300]
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    n, g = cu[-1], gen(2)
    q = torch.empty(n, hq, d, dtype=BF16, device="cuda").normal_(generator=g)
    k, v = (torch.empty(n, hk, d, dtype=BF16, device="cuda").normal_(generator=g) for _ in range(2))
    assert q.numel() > 2**31
    out, lse = torch.empty_like(q), torch.empty(n, hq, device="cuda")
    ops.m3_attn_prompt(q, k, v, i32(cu), out, lse)
    for s in (0, 1, 4095, 8063, 8190, 8191):
        a, b = cu[s], cu[s + 1]
        T.check_prompt(out[a:b], lse[a:b], q[a:b], k[a:b], v[a:b], [0, b - a], [0, b - a], d ** -0.5, BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rules_far_into_the_logits(ops, dtype):
    r, n = 11000, 200001  # 2.2e9 logits
    x = torch.empty(r, n, dtype=dtype, device="cuda").normal_(generator=gen(3))
    rows = [0, 1, 5461, 10737, r - 1]  # 10737: the row that holds logit 2^31
    want = x[rows].clone()
    history, hist_len, rep, freq, pres, ids, bias, mask, row = T.rule_inputs(r, n, 40, 5, 2, 3)
    use = (history, hist_len, rep, freq, pres, ids, bias, mask, row)
    pick = [None if t is None else t[rows] if t.shape[0] == r else t for t in use]
    ops.m3_logit_rules(x, x, *use)
    T.check_rules(x[rows], want, *pick)
