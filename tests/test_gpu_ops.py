"""The serving operators (include/m3_ops.h) on the GPU against plain 64-bit forms (ops_ref.py)."""
import math
import random

import pytest
import torch

import ops_ref as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from autoregressive_audio_token_b200 import ops
    return ops


@pytest.fixture(autouse=True)
def _status(request):
    yield
    if torch.cuda.is_available():
        from autoregressive_audio_token_b200 import ops
        ops.m3_ops_sync_status()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------- map ---

def run_map(ops, fresh, cached, free, table, page, n_pages, start, n_tokens, free_at=None):
    n = len(fresh)
    t = i32(table) if len(table[0]) else torch.empty(n, 0, dtype=torch.int32, device="cuda")
    cu, lens, taken = i32([-7] * (n + 1)), i32([-7] * n), i32([-7])
    pos, seqs = i32([-7] * n_tokens), i32([-7] * n_tokens)
    slots = torch.full((n_tokens,), -7, dtype=torch.int64, device="cuda")
    ops.m3_kv_map(i32(fresh), i32(cached) if cached else None, i32(free), t, page, n_pages, cu, pos, slots, seqs,
                  lens, taken, start=start, free_at=None if free_at is None else i32([free_at]))
    return [x.tolist() for x in (t, cu, pos, slots, seqs, lens)] + [int(taken)]


def check_map(ops, fresh, cached, free, table, page, n_pages, start=0, pad=0, free_at=None):
    n_tokens = sum(max(f, 0) for f in fresh) + pad
    got = run_map(ops, fresh, cached, free, table, page, n_pages, start, max(n_tokens, 0), free_at)
    want = R.kv_map(fresh, cached or [0] * len(fresh), free, table, page, n_pages, start, n_tokens, free_at or 0)
    for name, g, w in zip(("table", "cu", "positions", "slots", "seqs", "lens", "taken"), got, want):
        assert g == w, name


@pytest.mark.parametrize("n,most_fresh,most_cached,page", [
    (1, 1, 0, 16), (1, 0, 0, 16), (3, 40, 100, 16), (16, 1, 9000, 256), (33, 300, 70, 32), (257, 90, 600, 64),
    (1000, 5, 0, 1024), (5119, 2, 3, 16), (6143, 2, 3, 16), (8192, 3, 50, 128)])
@pytest.mark.parametrize("pad", [0, 5])
def test_map(ops, n, most_fresh, most_cached, page, pad):
    rnd = random.Random(n * 7 + page)
    fresh = [rnd.randint(0, most_fresh) if i % 5 else most_fresh for i in range(n)]
    cached = [rnd.randint(0, most_cached) for _ in range(n)]
    cols = max(-(-(f + c) // page) for f, c in zip(fresh, cached)) + 2
    need = sum(-(-(f + c) // page) for f, c in zip(fresh, cached)) + 9
    numbers = list(range(need))
    rnd.shuffle(numbers)
    table = [[-1] * cols for _ in range(n)]
    for r, c in enumerate(cached):
        for i in range(-(-c // page)):
            table[r][i] = numbers.pop()
    check_map(ops, fresh, cached, numbers, table, page, need, start=11, pad=pad)


def test_map_page_edges(ops):
    # lengths that end on, before and behind a page's last place
    fresh, cached = [1, 1, 1, 16, 17, 15, 0, 0], [15, 16, 17, 16, 15, 1, 0, 16]
    table = [[20 + 3 * r + i for i in range(3)] for r in range(8)]
    check_map(ops, fresh, cached, list(range(20)), table, 16, 60)


def test_map_runs_out_of_pages_columns_and_bounds(ops):
    table = [[-1] * 3 for _ in range(4)]
    check_map(ops, [40, 40, 40, 2], None, [5, 3, 9, 1], table, 16, 10, pad=3)              # the list ends
    check_map(ops, [100, 20, 49, 2], None, list(range(12)), table, 16, 12, pad=3)          # max_pages
    check_map(ops, [40, 40, 40, 2], None, [5, -3, 77, 1] * 3, table, 16, 10)               # bad numbers in the list
    check_map(ops, [3, 4], [10, 20], [1, 2], [[-1, 5, 5], [99, 6, 6]], 16, 10)             # bad cached pages
    check_map(ops, [3, 4], [10, 200], [1, 2], [[0, 5, 5], [3, 6, 6]], 16, 10)              # cached past the table
    check_map(ops, [-3, 4], [10, -20], [1, 2], [[0, 5, 5], [3, 6, 6]], 16, 10)             # negative lengths
    check_map(ops, [30, 4], None, [1, 2, 8, 7, 4], [[-1] * 3] * 2, 16, 10, free_at=2)      # further down the list
    check_map(ops, [30, 4], None, [1, 2], [[-1] * 3] * 2, 16, 10, free_at=50)
    check_map(ops, [30, 4], None, [], [[-1] * 3] * 2, 16, 10)
    check_map(ops, [30, 4], None, [1, 2], [[]] * 2, 16, 10)                                # a table without columns


def test_map_drops_tokens_past_the_arrays_and_saturates(ops):
    got = run_map(ops, [7, 9], None, [0, 1, 2], [[-1] * 2] * 2, 16, 3, 0, 10)
    want = R.kv_map([7, 9], [0, 0], [0, 1, 2], [[-1] * 2] * 2, 16, 3, 0, 10)
    assert got == list(want)
    big = 2**31 - 1
    t, cu, _, _, _, lens, taken = run_map(ops, [big, big, 1], [0, big, 0], [4], [[-1] * 2] * 3, 16, 5, 0, 4)
    assert cu == [0, big, big, big] and lens == [big, big, 1] and taken == 3 and t[0] == [4, -1]


def test_map_slots_past_32_bits(ops):
    t, _, _, slots, _, _, _ = run_map(ops, [2], [1023], [2**31 - 2], [[2**31 - 3, -1]], 1024, 2**31 - 1, 0, 2)
    assert slots == [(2**31 - 3) * 1024 + 1023, (2**31 - 2) * 1024]


def test_map_strided_table(ops):
    t = i32([[-1] * 8 for _ in range(3)])
    ops_args = (i32([5, 20, 1]), None, i32([4, 3, 2, 1]), t[:, 2:5], 16, 9)
    out = [i32([0] * 4), i32([0] * 26), torch.zeros(26, dtype=torch.int64, device="cuda"), i32([0] * 26), i32([0] * 3),
           i32([0])]
    ops.m3_kv_map(*ops_args, *out)
    assert t.tolist() == [[-1, -1, 4] + [-1] * 5, [-1, -1, 3, 2] + [-1] * 4, [-1, -1, 1] + [-1] * 5]


# ----------------------------------------------------------------- store ---

@pytest.mark.parametrize("n,hk,d,page,dtype", [(1, 1, 64, 16, BF16), (16, 8, 128, 256, BF16), (37, 3, 64, 32, F16),
                                               (1000, 16, 128, 64, F16), (5, 2, 8, 16, BF16), (70, 40, 256, 16, BF16),
                                               (2500, 2, 1024, 1024, F16)])
@pytest.mark.parametrize("layout", ["plain", "fused", "unaligned"])
def test_store(ops, n, hk, d, page, dtype, layout):
    g = gen(n)
    n_pages = -(-n // page) + 2
    pool = torch.randn(n_pages, 2, hk, page, d, generator=g, device="cuda").to(dtype)
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:n]
    slots[n // 2::7] = -1
    if n > 3:
        slots[1], slots[3] = n_pages * page, -2**40
    if layout == "fused":
        kv = torch.randn(n, 2 * hk + 3, d, generator=g, device="cuda").to(dtype)
        k, v = kv[:, 1:1 + hk], kv[:, 2 + hk:2 + 2 * hk]
    elif layout == "unaligned":
        k = torch.randn(n * hk * (d + 1) + 1, generator=g, device="cuda").to(dtype)[1:].view(n, hk, d + 1)[..., :d]
        v = torch.randn(hk, n, d, generator=g, device="cuda").to(dtype).transpose(0, 1)
    else:
        k, v = (torch.randn(n, hk, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    want = pool.clone()
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < n_pages * page:
            want[s // page, 0, :, s % page] = k[i]
            want[s // page, 1, :, s % page] = v[i]
    ops.m3_kv_store(k, v, slots, pool)
    assert torch.equal(pool, want)


# ---------------------------------------------------------------- prompt ---

def prompt_case(fresh, cached, hq, hk, d, dtype, seed, extra=3, scale=None):
    """Inputs with `extra` rows behind the last sequence; K and V behind the last key are NaN."""
    g = gen(seed)
    keys = [f + c for f, c in zip(fresh, cached)]
    cu_q, cu_k = [0], [0]
    for f, k in zip(fresh, keys):
        cu_q.append(cu_q[-1] + f)
        cu_k.append(cu_k[-1] + max(k, 0))
    q = torch.randn(cu_q[-1] + extra, hq, d, generator=g, device="cuda").to(dtype)
    k = torch.randn(cu_k[-1] + extra, hk, d, generator=g, device="cuda").to(dtype)
    v = torch.randn(cu_k[-1] + extra, hk, d, generator=g, device="cuda").to(dtype)
    k[cu_k[-1]:] = math.nan
    v[cu_k[-1]:] = math.nan
    return q, k, v, cu_q, cu_k


def check_prompt(out, lse, q, k, v, cu_q, cu_k, scale, dtype):
    d = q.shape[2]
    for a, b, ka, kb in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        if a == b:
            continue
        seen = torch.arange(kb - ka, device="cuda") <= (torch.arange(b - a, device="cuda") + (kb - ka) - (b - a))[:, None]
        ref = R.attend(q[a:b], k[ka:kb], v[ka:kb], seen, scale)
        bound, lbound = R.attention_bounds(ref, kb - ka, d, scale, dtype)
        err = (out[a:b].double() - ref[0]).abs()
        assert bool((err <= bound).all()), (a, b, float((err - bound).max()), float(err.max()))
        empty = ref[1] == -math.inf
        assert torch.equal(lse[a:b] == -math.inf, empty)
        lerr = (lse[a:b].double() - ref[1]).nan_to_num(0, 0, 0).abs()
        assert bool((lerr <= lbound).all()), (a, b, float(lerr.max()))


PROMPTS = [
    ([1], [0]), ([2], [0]), ([127], [0]), ([128], [0]), ([129], [0]), ([300, 237], [0, 0]), ([0, 5, 0, 0, 64, 1], [0] * 6),
    ([1, 1, 1], [0, 127, 128]), ([3, 40, 65], [500, 0, 63]), ([700], [0]), ([513, 31, 1500], [0, 600, 1]),
    ([5, 9], [-3, 4]),  # fewer keys than queries: the first rows attend to nothing
    ([6, 2], [-6, 0]),  # no key at all
]


@pytest.mark.parametrize("hq,hk,d,dtype", [(4, 1, 128, BF16), (8, 8, 64, F16), (6, 2, 128, F16), (4, 2, 64, BF16)])
@pytest.mark.parametrize("lengths", PROMPTS, ids=lambda p: "x".join(map(str, p[0][:3])))
def test_prompt(ops, lengths, hq, hk, d, dtype):
    fresh, cached = lengths
    q, k, v, cu_q, cu_k = prompt_case(fresh, cached, hq, hk, d, dtype, sum(fresh) + hq)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ops.m3_attn_prompt(q, k, v, i32(cu_q), out, lse, cu_k=i32(cu_k))
    check_prompt(out, lse, q, k, v, cu_q, cu_k, d ** -0.5, dtype)
    assert bool((out[cu_q[-1]:] == 7).all()) and bool((lse[cu_q[-1]:] == 7).all())


@pytest.mark.parametrize("hq,hk", [(1, 1), (16, 1), (24, 4), (5, 1), (64, 1), (7, 7), (32, 8), (33, 3)])
def test_prompt_head_groups(ops, hq, hk):
    q, k, v, cu_q, cu_k = prompt_case([90, 200], [30, 0], hq, hk, 128, BF16, hq)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ops.m3_attn_prompt(q, k, v, i32(cu_q), out, lse, cu_k=i32(cu_k), scale=0.2)
    check_prompt(out, lse, q, k, v, cu_q, cu_k, 0.2, BF16)


def test_prompt_strided_without_lse_and_cu_k(ops):
    hq, hk, d = 8, 2, 128
    g = gen(5)
    qkv = torch.randn(333, hq + 2 * hk, d, generator=g, device="cuda").to(BF16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    out = torch.empty(hq, 333, d, dtype=BF16, device="cuda").transpose(0, 1)
    cu = [0, 100, 101, 333]
    ops.m3_attn_prompt(q, k, v, i32(cu), out)
    lse = torch.empty(333, hq, device="cuda")
    plain = torch.empty(333, hq, d, dtype=BF16, device="cuda")
    ops.m3_attn_prompt(q.contiguous(), k.contiguous(), v.contiguous(), i32(cu), plain, lse)
    assert torch.equal(out, plain)
    check_prompt(out, lse, q, k, v, cu, cu, d ** -0.5, BF16)


@pytest.mark.parametrize("big", [30.0, 300.0])
def test_prompt_wide_scores(ops, big):
    # maxima that grow along the keys, so that the running maximum is raised again and again
    q, k, v, cu_q, cu_k = prompt_case([400], [0], 4, 2, 64, F16, 9)
    k *= torch.linspace(0.1, big / 10, k.shape[0], device="cuda")[:, None, None].to(F16)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ops.m3_attn_prompt(q, k, v, i32(cu_q), out, lse, cu_k=i32(cu_k))
    check_prompt(out, lse, q, k, v, cu_q, cu_k, 64 ** -0.5, F16)


def test_prompt_other_sequences_and_bad_lengths(ops):
    # infinities and NaN of a neighbour stay there
    q, k, v, cu_q, cu_k = prompt_case([70, 60, 90], [0, 0, 0], 4, 2, 128, BF16, 3, extra=0)
    k[70:130] = math.nan
    v[70:130] = math.inf
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ops.m3_attn_prompt(q, k, v, i32(cu_q), out, lse)
    keep = lambda x: torch.cat([x[:70], x[130:]])  # noqa: E731
    check_prompt(keep(out), keep(lse), keep(q), keep(k), keep(v), [0, 70, 160], [0, 70, 160], 128 ** -0.5, BF16)
    assert bool(out[70:130].isnan().all())
    # sums past the arrays are cut
    out2, lse2 = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ops.m3_attn_prompt(q, k, v, i32([0, 70, 130, 5000]), out2, lse2)
    assert torch.equal(out2[:70], out[:70]) and torch.equal(out2[130:], out[130:])


@pytest.mark.parametrize("hq,hk,d,dtype", [(4, 1, 128, BF16), (2, 2, 64, F16)])
def test_prompt_values_ahead_of_a_query_stay_there(ops, hq, hk, d, dtype):
    # infinities and NaN in keys and values that later queries alone attend to
    q, k, v, cu_q, cu_k = prompt_case([300, 150], [40, 0], hq, hk, d, dtype, 21, extra=0)
    ends = [(0, 340), (340, 490)]
    places = [(200, "v", math.nan), (205, "v", math.inf), (206, "v", -math.inf), (339, "v", math.nan), (339, "k", math.inf),
              (350, "v", math.inf), (480, "v", math.nan), (485, "k", math.nan)]
    for at, which, x in places:
        (k if which == "k" else v)[at, 0, ::3 if at % 2 else 5] = x
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ops.m3_attn_prompt(q, k, v, i32(cu_q), out, lse, cu_k=i32(cu_k))
    g = hq // hk
    for (ka, kb), a, b in zip(ends, cu_q, cu_q[1:]):
        n = kb - ka
        for i in range(b - a):
            seen = i + n - (b - a) + 1  # keys this query attends to
            for h in range(hq):
                z = (k[ka:ka + seen, h // g].double() @ q[a + i, h].double()) * d ** -0.5
                p = torch.softmax(z, 0)[:, None] * v[ka:ka + seen, h // g].double()
                want, got = p.sum(0), out[a + i, h].double()
                if not bool(z.isfinite().all()):
                    continue  # a score of its own is none
                fin = want.isfinite()
                assert torch.equal(got.isnan(), want.isnan()), (a + i, h)
                assert torch.equal(got[want.isinf()], want[want.isinf()]), (a + i, h)
                # as attention_bounds, with the mean of |v| and of the scores' terms bounded by their largest
                tol = (3 * R.HALF[dtype] + 2.0 ** -10) * float(v[ka:ka + seen][v[ka:ka + seen].isfinite()].abs().max())
                assert float((got - want)[fin].abs().max()) <= tol, (a + i, h)


def test_prompt_many_sequences(ops):
    rnd = random.Random(4)
    fresh = [rnd.choice([0, 1, 2, 3, 17, 40]) for _ in range(300)]
    q, k, v, cu_q, cu_k = prompt_case(fresh, [rnd.choice([0, 5]) for _ in fresh], 2, 1, 64, BF16, 12)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ops.m3_attn_prompt(q, k, v, i32(cu_q), out, lse, cu_k=i32(cu_k))
    check_prompt(out, lse, q, k, v, cu_q, cu_k, 64 ** -0.5, BF16)


# ---------------------------------------------------------------- prefix ---

def prefix_case(n, prefix, lens, hq, hk, d, page, dtype, seed, spare=2):
    """A pool whose places past the lengths, and whose unused pages, are NaN."""
    g = gen(seed)
    np_, most = -(-prefix // page), max([-(-max(x, 0) // page) for x in lens] + [1])
    n_pages = np_ + sum(-(-max(x, 0) // page) for x in lens) + spare
    numbers = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    pool = torch.full((n_pages, 2, hk, page, d), math.nan, dtype=dtype, device="cuda")
    q = torch.randn(n, hq, d, generator=g, device="cuda").to(dtype)

    def fill(count):
        mine, kv = [], torch.randn(2, count, hk, d, generator=g, device="cuda").to(dtype)
        for i in range(-(-count // page)):
            p = numbers.pop()
            part = kv[:, i * page:(i + 1) * page]
            pool[p, :, :, :part.shape[1]] = part.transpose(1, 2)
            mine.append(p)
        return mine, kv

    pages, shared = fill(prefix)
    table, own = [], []
    for x in lens:
        mine, kv = fill(max(x, 0))
        table.append(mine + [-1] * (most - len(mine)))
        own.append(kv)
    return q, pool, pages, shared, table, own


def check_prefix(out, lse, q, shared, own, lens, scale, dtype):
    n, d = q.shape[0], q.shape[2]
    for b in range(n):
        if lens[b] < 0:
            assert bool((out[b] == 7).all()) and bool((lse[b] == 7).all())
            continue
        kv = torch.cat([shared, own[b]], 1)
        seen = torch.ones(1, kv.shape[1], dtype=torch.bool, device="cuda")
        ref = R.attend(q[b:b + 1], kv[0], kv[1], seen, scale)
        bound, lbound = R.attention_bounds(ref, kv.shape[1], d, scale, dtype)
        err = (out[b:b + 1].double() - ref[0]).abs()
        assert bool((err <= bound).all()), (b, float((err - bound).max()), float(err.max()))
        assert torch.equal(lse[b:b + 1] == -math.inf, ref[1] == -math.inf)
        assert bool(((lse[b:b + 1].double() - ref[1]).nan_to_num(0, 0, 0).abs() <= lbound).all()), b


PREFIXES = [(1, 0, [0]), (1, 1, [0]), (1, 0, [1]), (2, 300, [5, 40]), (3, 128, [0, 128, 17]), (4, 129, [-1, 3, 0, 250]),
            (5, 1000, [16, 15, 17, 700, 1]), (40, 2000, [7 * i % 300 for i in range(40)]), (3, 0, [0, 33, -1]),
            (1, 2500, [70]), (2, 1100, [0, 9]), (140, 1100, [i % 37 - 1 for i in range(140)])]


@pytest.mark.parametrize("hq,hk,d,page,dtype", [(8, 2, 128, 16, BF16), (4, 4, 64, 256, F16), (6, 1, 64, 32, BF16),
                                                (32, 8, 128, 64, F16), (8, 2, 64, 1024, BF16)])
@pytest.mark.parametrize("n,prefix,lens", PREFIXES)
def test_prefix(ops, n, prefix, lens, hq, hk, d, page, dtype):
    q, pool, pages, shared, table, own = prefix_case(n, prefix, lens, hq, hk, d, page, dtype, n + prefix)
    out, lse = torch.full_like(q, 7.0), torch.full((n, hq), 7.0, device="cuda")
    ops.m3_attn_prefix(q, pool, i32(pages), prefix, i32(table), i32(lens), out, lse)
    check_prefix(out, lse, q, shared, own, lens, d ** -0.5, dtype)


@pytest.mark.parametrize("hq,hk", [(1, 1), (17, 1), (24, 4), (5, 1), (64, 1), (7, 7), (66, 2)])
def test_prefix_head_groups(ops, hq, hk):
    lens = [3, 0, 190]
    q, pool, pages, shared, table, own = prefix_case(3, 333, lens, hq, hk, 128, 32, BF16, hq)
    out, lse = torch.empty_like(q), torch.empty(3, hq, device="cuda")
    ops.m3_attn_prefix(q, pool, i32(pages), 333, i32(table), i32(lens), out, lse, scale=0.11)
    check_prefix(out, lse, q, shared, own, lens, 0.11, BF16)


def test_prefix_bad_pages_are_left_out(ops):
    page, hk = 16, 2
    q, pool, pages, shared, table, own = prefix_case(3, 400, [40, 70, 16], 8, hk, 128, page, BF16, 2)
    pages[3], pages[24], pages[10] = -1, pool.shape[0], 2**31 - 1
    table[0][1], table[1][0], table[2][0] = -5, pool.shape[0] + 3, -1
    keep = torch.ones(400, dtype=torch.bool, device="cuda")
    for p in (3, 24, 10):
        keep[p * page:(p + 1) * page] = False
    shared = shared[:, keep]
    own[0] = torch.cat([own[0][:, :16], own[0][:, 32:]], 1)
    own[1], own[2] = own[1][:, 16:], own[2][:, :0]
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    ops.m3_attn_prefix(q, pool, i32(pages), 400, i32(table), i32([40, 70, 16]), out, lse)
    check_prefix(out, lse, q, shared, own, [40, 70, 16], 128 ** -0.5, BF16)


def test_prefix_without_own_pages(ops):
    # a table without columns: the prefix alone, and with none of it nothing
    for prefix in (400, 0):
        q, pool, pages, shared, table, own = prefix_case(2, prefix, [0, 0], 8, 2, 64, 16, BF16, 4)
        none = torch.empty(2, 0, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(q, 7.0), torch.full((2, 8), 7.0, device="cuda")
        ops.m3_attn_prefix(q, pool, i32(pages), prefix, none, i32([0, -1]), out, lse)
        check_prefix(out, lse, q, shared, own, [0, -1], 64 ** -0.5, BF16)


def test_prefix_strides_and_lengths_past_the_table(ops):
    lens = [20, 32]
    q, pool, pages, shared, table, own = prefix_case(2, 50, lens, 8, 2, 64, 16, F16, 8)
    wide = torch.zeros(2, 3 * 8 * 64, dtype=F16, device="cuda")
    wide[:, 512:1024] = q.flatten(1)
    big_table = i32([row + [9, 9] for row in table])
    out = torch.empty(8, 2, 64, dtype=F16, device="cuda").transpose(0, 1)
    lse = torch.empty(2, 8, device="cuda")
    ops.m3_attn_prefix(wide[:, 512:1024].unflatten(1, (8, 64)), pool, i32(pages), 50, big_table[:, :2], i32([20, 10**9]),
                       out, lse)
    check_prefix(out, lse, q, shared, own, lens, 64 ** -0.5, F16)


# ----------------------------------------------------------------- rules ---

def check_rules(got, x, *rules):
    want, mag = R.logit_rules(x, *rules)
    half = R.HALF[x.dtype]
    # fp32 steps: the quotient or product, count times frequency, the two differences and the biases' sums
    n_bias = 0 if rules[6] is None else rules[6].shape[1]
    bound = half * want.abs().nan_to_num(0, 0, 0) * (1 + 2.0 ** -7) + (6 + n_bias) * 2.0 ** -24 * mag.nan_to_num(0, 0, 0)
    if x.dtype is F16:
        bound = bound + 2.0 ** -25
    fin = want.isfinite()
    assert torch.equal(got.double()[~fin], want[~fin])
    err = (got.double() - want).abs()
    assert bool((err[fin] <= bound[fin]).all()), float((err - bound)[fin].max())


def rule_inputs(r, n, nh, nb, nm, seed):
    g = gen(seed)
    u = lambda a, b: a + (b - a) * torch.rand(r, generator=g, device="cuda")  # noqa: E731
    history = torch.randint(-2, n + 2, (r, nh), generator=g, device="cuda").to(torch.int32) if nh else None
    if nh > 4:
        history[:, ::3] = history[:, :1].clamp(0, n - 1)  # a token that comes often
    hist_len = torch.randint(0, nh + 1, (r,), generator=g, device="cuda").to(torch.int32) if nh else None
    ids = bias = mask = row = None
    if nb:
        ids = torch.randint(-1, n + 1, (r, nb), generator=g, device="cuda").to(torch.int32)
        bias = 3 * torch.randn(r, nb, generator=g, device="cuda")
    if nm:
        mask = torch.randint(-2**31, 2**31, (nm, -(-n // 32)), generator=g, device="cuda").to(torch.int32)
        row = torch.randint(-1, nm + 1, (r,), generator=g, device="cuda").to(torch.int32)
    return history, hist_len, u(1, 1.6), u(-0.2, 0.4), u(-0.3, 0.7), ids, bias, mask, row


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("r,n,nh,nb,nm", [(1, 1, 1, 1, 1), (2, 16385, 1500, 16, 1), (3, 31, 9, 40, 2), (5, 1000, 0, 7, 0),
                                          (4, 4097, 70, 0, 3), (700, 8191, 33, 5, 4), (300, 20000, 50, 0, 0),
                                          (300, 20000, 0, 9, 0), (300, 20001, 0, 0, 2),
                                          (120, 130001, 600, 40, 3), (110, 140000, 9000, 300, 1),  # two launches
                                          (2, 50001, 4096, 300, 2)])
def test_rules(ops, r, n, nh, nb, nm, dtype):
    x = (4 * torch.randn(r, n, generator=gen(n), device="cuda")).to(dtype)
    history, hist_len, rep, freq, pres, ids, bias, mask, row = rule_inputs(r, n, nh, nb, nm, n + r)
    out = torch.empty_like(x)
    ops.m3_logit_rules(x, out, history, hist_len, rep, freq, pres, ids, bias, mask, row)
    check_rules(out, x, history, hist_len, rep, freq, pres, ids, bias, mask, row)
    y = x.clone()
    ops.m3_logit_rules(y, y, history, hist_len, rep, freq, pres, ids, bias, mask, row)
    assert torch.equal(y, out)
    y = x.clone()  # in place without a mask: only the named tokens are touched
    ops.m3_logit_rules(y, y, history, hist_len, rep, freq, pres, ids, bias)
    check_rules(y, x, history, hist_len, rep, freq, pres, ids, bias, None, None)


@pytest.mark.parametrize("dtype", [F32, F16])
def test_rules_strides_and_single_rules(ops, dtype):
    big = (4 * torch.randn(3, 2100, generator=gen(1), device="cuda")).to(dtype)
    to = torch.zeros(3, 2300, dtype=dtype, device="cuda")
    history, hist_len, rep, freq, pres, ids, bias, mask, row = rule_inputs(3, 2003, 21, 9, 3, 4)
    wide = torch.full((3, 40), 1, dtype=torch.int32, device="cuda")
    wide[:, 3:24] = history
    for a, b in ((5, 5), (3, 8), (0, 1), (17, 290)):
        x, out = big[:, a:a + 2003], to[:, b:b + 2003]
        for use in ((wide[:, 3:24], hist_len, rep, freq, pres, ids, bias, mask, row),
                    (history, None, None, None, None, None, None, None, None),
                    (history, None, rep, None, None, None, None, mask, None),
                    (None, None, rep, freq, pres, None, None, mask[:1], None),
                    (None,) * 5 + (ids, bias, None, None)):
            ops.m3_logit_rules(x, out, *use)
            check_rules(out, x, *use)
        assert bool((to[:, :b] == 0).all()) and bool((to[:, b + 2003:] == 0).all())
        to.zero_()


def test_rules_infinities_masks_and_repeated_biases(ops):
    x = torch.zeros(2, 70, device="cuda")
    x[0, 3], x[0, 4], x[0, 5], x[0, 6] = math.nan, math.inf, -math.inf, torch.finfo(F32).min
    mask = torch.zeros(2, 3, dtype=torch.int32, device="cuda")  # row 0: nothing but 5 and 6, row 1: nothing
    mask[0, 0] = (1 << 5) | (1 << 6)
    out = torch.empty_like(x)
    ops.m3_logit_rules(x, out, mask=mask)
    want = torch.full_like(x, -math.inf)
    want[0, 6] = torch.finfo(F32).min
    assert torch.equal(out, want)
    # one token named several times: its biases add up in their order
    ids = i32([[7, 9, 7, 7, 9, -1, 70]])
    bias = torch.tensor([[1e8, 1.0, 1.0, -1e8, 2.0, 5.0, 5.0]], device="cuda")
    ops.m3_logit_rules(x[1:], out[1:], bias_ids=ids, bias=bias)
    want = torch.zeros(70, device="cuda")
    want[7], want[9] = (torch.tensor(1e8) + 1.0) - 1e8, 3.0
    assert torch.equal(out[1], want)


# -------------------------------------------- streams, graphs, one after another --

def serve_inputs(ops, seed=0):
    """Requests that share a prompt: everything two steps of a server need."""
    g = gen(seed)
    page, hq, hk, d, n = 32, 8, 2, 64, 3
    n_pages = 64
    pool = torch.full((n_pages, 2, hk, page, d), math.nan, dtype=BF16, device="cuda")
    free = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    return g, page, hq, hk, d, n, n_pages, pool, free


def maps(ops, fresh, cached, free, table, page, n_pages, n_tokens, start, free_at):
    n = fresh.numel()
    e = lambda k, t=torch.int32: torch.empty(k, dtype=t, device="cuda")  # noqa: E731
    cu, pos, slots, seqs, lens, taken = e(n + 1), e(n_tokens), e(n_tokens, torch.int64), e(n_tokens), e(n), e(1)
    ops.m3_kv_map(fresh, cached, free, table, page, n_pages, cu, pos, slots, seqs, lens, taken, start=start,
                  free_at=free_at)
    return cu, pos, slots, seqs, lens, taken


def test_operators_together(ops):
    """A shared prompt, each request's own prompt, then single tokens, through the five operators; the attention of
    every step against plain attention over the tokens so far."""
    g, page, hq, hk, d, n, n_pages, pool, free = serve_inputs(ops)
    scale = d ** -0.5
    new = lambda t: tuple(torch.randn(t, h, d, generator=g, device="cuda").to(BF16) for h in (hq, hk, hk))  # noqa: E731
    # the shared prompt of 75 tokens: a table of one request
    shared_len = 75
    ptable = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    cu, _, slots, _, _, taken = maps(ops, i32([shared_len]), None, free, ptable, page, n_pages, shared_len, 0, None)
    qs, ks, vs = new(shared_len)
    ops.m3_kv_store(ks, vs, slots, pool)
    out = torch.empty_like(qs)
    lse = torch.empty(shared_len, hq, device="cuda")
    ops.m3_attn_prompt(qs, ks, vs, cu, out, lse)
    check_prompt(out, lse, qs, ks, vs, [0, shared_len], [0, shared_len], scale, BF16)
    at = taken.clone()
    # single tokens of three requests, each ending pages at its own time
    table = torch.full((n, 4), -1, dtype=torch.int32, device="cuda")
    cached, own = i32([0] * n), [torch.empty(2, 0, hk, d, dtype=BF16, device="cuda") for _ in range(n)]
    for step in range(70):
        fresh = i32([1, int(step % 2 == 0), int(step < 40)])
        cu, pos, slots, seqs, lens, taken = maps(ops, fresh, cached, free, table, page, n_pages, 4, shared_len, at)
        at = at + taken
        q, k, v = new(4)
        ops.m3_kv_store(k, v, slots, pool)
        who = seqs.tolist()
        for i, r in enumerate(who):
            if r >= 0:
                assert int(pos[i]) == shared_len + own[r].shape[1]
                own[r] = torch.cat([own[r], torch.stack([k[i], v[i]])[:, None]], 1)
        cached = lens
        # rows of requests without a token this step are padding
        rows = torch.randn(n, hq, d, generator=g, device="cuda").to(BF16)
        row_lens = torch.where(fresh > 0, lens, -1).to(torch.int32)
        o, l2 = torch.full_like(rows, 7.0), torch.full((n, hq), 7.0, device="cuda")
        ops.m3_attn_prefix(rows, pool, ptable[0, :3].contiguous(), shared_len, table, row_lens, o, l2)
        if step % 13 == 0 or step > 66:
            check_prefix(o, l2, rows, torch.stack([ks, vs]), own, row_lens.tolist(), scale, BF16)
    # a draw among what a grammar allows
    logits = torch.randn(n, 500, generator=g, device="cuda")
    mask = torch.zeros(1, 16, dtype=torch.int32, device="cuda")
    mask[0, 3] = 1 << 4
    ops.m3_logit_rules(logits, logits, history=i32([[1, 2, 3]] * n), frequency=torch.ones(n, device="cuda"), mask=mask)
    assert logits.argmax(1).tolist() == [100] * n


def all_calls(ops, seed):
    """(run, outputs) over inputs of one seed: every operator once, one after another."""
    g, page, hq, hk, d, n, n_pages, pool, free = serve_inputs(ops, seed)
    pool.zero_()
    lens0 = [40, 90, 7]
    table = torch.full((n, 4), -1, dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(sum(lens0), h, d, generator=g, device="cuda").to(BF16) for h in (hq, hk, hk))
    fresh = i32(lens0)
    e = lambda m, t=torch.int32: torch.zeros(m, dtype=t, device="cuda")  # noqa: E731
    t = sum(lens0)
    outs = [e(n + 1), e(t), e(t, torch.int64), e(t), e(n), e(1)]
    o1, l1 = torch.zeros_like(q), torch.zeros(t, hq, device="cuda")
    q2 = torch.randn(n, hq, d, generator=g, device="cuda").to(BF16)
    o2, l2 = torch.zeros_like(q2), torch.zeros(n, hq, device="cuda")
    ws = torch.empty(ops.m3_attn_prefix_workspace(n, hq, hk, d, 3, page, 4), dtype=torch.uint8, device="cuda")
    x = torch.randn(n, 3001, generator=g, device="cuda")
    y = torch.zeros_like(x)
    history = torch.randint(0, 3001, (n, 50), generator=g, device="cuda").to(torch.int32)
    pen = torch.full((n,), 1.3, device="cuda")

    def run(stream=None):
        ops.m3_kv_map(fresh, None, free, table, page, n_pages, *outs, stream=stream)
        ops.m3_kv_store(k, v, outs[2], pool, stream=stream)
        ops.m3_attn_prompt(q, k, v, outs[0], o1, l1, stream=stream)
        ops.m3_attn_prefix(q2, pool, table[1, :3].contiguous(), 90, table, outs[4], o2, l2, workspace=ws, stream=stream)
        ops.m3_logit_rules(x, y, history=history, repetition=pen, stream=stream)

    return run, [table, pool, o1, l1, o2, l2, y] + outs


def test_captured_replayed_and_side_by_side(ops):
    """Two captured graphs of all operators, replayed at once on two streams, and eager calls on a third: the same
    bits every time."""
    torch.cuda.synchronize()
    sets = [all_calls(ops, s) for s in range(3)]
    torch.cuda.synchronize()
    want = []
    for run, outs in sets:
        run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    graphs, streams = [], [torch.cuda.Stream() for _ in range(3)]
    for (run, outs), st in zip(sets[:2], streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            run()
        graphs.append(gr)
    torch.cuda.synchronize()
    for _, outs in sets:
        for o in outs[2:]:
            o.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        with torch.cuda.stream(streams[2]):
            sets[2][0]()
    torch.cuda.synchronize()
    for (_, outs), w in zip(sets, want):
        for i, (o, x) in enumerate(zip(outs, w)):
            assert torch.equal(o.nan_to_num(), x.nan_to_num()) if o.is_floating_point() else torch.equal(o, x), i


def test_a_stream_passed_by_hand(ops):
    run, outs = all_calls(ops, 5)
    run()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs[2:]:
        o.zero_()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(stream=st)
    st.synchronize()
    for o, x in zip(outs, want):
        assert torch.equal(o, x)


def test_refusals_leave_no_error_behind(ops):
    from autoregressive_audio_token_b200.m3 import M3Error
    q = torch.zeros(4, 4, 64, dtype=BF16, device="cuda")
    for call in (lambda: ops.m3_attn_prompt(q, q[:, :3], q[:, :3], i32([0, 4]), torch.empty_like(q)),
                 lambda: ops.m3_attn_prompt(q, q, q, i32([0, 4]), torch.empty_like(q), scale=-1.0),
                 lambda: ops.m3_attn_prompt(q, q, q, torch.tensor([0, 4], dtype=torch.int32), torch.empty_like(q)),
                 lambda: ops.m3_kv_store(q, q, torch.zeros(4, dtype=torch.int64, device="cuda"),
                                         torch.zeros(2, 2, 4, 24, 64, dtype=BF16, device="cuda"))):
        with pytest.raises(M3Error):
            call()
    ops.m3_ops_sync_status()


def large_calls(ops, seed):
    """The forms of many CTAs: a shared prefix beside the rows' own pages, logits in two launches, long prompts."""
    lens = [(7 * i + seed) % 300 for i in range(40)]
    q, pool, pages, shared, table, own = prefix_case(40, 2000, lens, 8, 2, 64, 32, BF16, seed)
    o1, l1 = torch.zeros_like(q), torch.zeros(40, 8, device="cuda")
    ws = torch.empty(ops.m3_attn_prefix_workspace(40, 8, 2, 64, len(pages), 32, len(table[0])), dtype=torch.uint8,
                     device="cuda")
    pages, table, lens_t = i32(pages), i32(table), i32(lens)
    x = torch.randn(120, 130001, generator=gen(seed), device="cuda")
    y = torch.zeros_like(x)
    history, hist_len, rep, freq, pres, ids, bias, mask, row = rule_inputs(120, 130001, 600, 40, 3, seed)
    p, k, v, cu_q, _ = prompt_case([2000, 700, 1500], [0, 0, 0], 8, 2, 128, F16, seed, extra=0)
    o2, l2, cu = torch.zeros_like(p), torch.zeros(p.shape[:2], device="cuda"), i32(cu_q)

    def run():
        ops.m3_attn_prefix(q, pool, pages, 2000, table, lens_t, o1, l1, workspace=ws)
        ops.m3_logit_rules(x, y, history, hist_len, rep, freq, pres, ids, bias, mask, row)
        ops.m3_attn_prompt(p, k, v, cu, o2, l2)

    return run, [o1, l1, y, o2, l2]


def test_large_calls_captured_and_side_by_side(ops):
    sets = [large_calls(ops, s) for s in (1, 2)]
    torch.cuda.synchronize()
    want, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for run, outs in sets:
        run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    for (run, outs), st in zip(sets, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            run()
            run()
        graphs.append(g)
    torch.cuda.synchronize()
    for _, outs in sets:
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    for _ in range(6):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_, outs), w in zip(sets, want):
        for i, (o, x) in enumerate(zip(outs, w)):
            assert torch.equal(o, x), i
