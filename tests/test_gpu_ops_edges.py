"""The serving operators (include/m3_ops.h) on the GPU where their forms differ: values that are no numbers, scores far
apart, and the shapes at which m3_attn_prefix and m3_logit_rules change how they split their work."""
import math

import pytest
import torch

import test_gpu_ops as T
from test_gpu_ops import BF16, F16, F32, _status, gen, i32, ops  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- prefix ---
# The forms of m3_attn_prefix by rows and positions: splits of few positions joined by a cluster, one row whose
# splits a second launch joins, a shared prefix beside the rows' own pages, and the same with a warp per join.

CLUSTER = dict(n=2, prefix=300, lens=[40, 100], hq=8, hk=2, d=64, page=64, dtype=BF16)
ONE_ROW = dict(n=1, prefix=2500, lens=[700], hq=8, hk=2, d=128, page=16, dtype=F16)
SHARED = dict(n=16, prefix=2000, lens=[60 * i for i in range(16)], hq=8, hk=2, d=128, page=16, dtype=BF16)
MANY = dict(n=150, prefix=1000, lens=[3 * i % 290 for i in range(150)], hq=32, hk=8, d=64, page=32, dtype=F16)
FORMS = {"cluster": CLUSTER, "one_row": ONE_ROW, "shared": SHARED, "many": MANY}


def case_of(form, seed=3):
    f = FORMS[form]
    return f, T.prefix_case(f["n"], f["prefix"], f["lens"], f["hq"], f["hk"], f["d"], f["page"], f["dtype"], seed)


def run_prefix(ops, f, q, pool, pages, table, scale=None):
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    ops.m3_attn_prefix(q, pool, i32(pages), f["prefix"], i32(table), i32(f["lens"]), out, lse, scale=scale)
    return out, lse


def put(pool, pages, page, first, last, side, head, value):
    """Positions first..last - 1 of these pages: K (side 0) or V (1) of a head."""
    for p in range(first, last):
        pool[pages[p // page], side, head, p % page] = value


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("first,last", [(128, 256), (0, 128), (200, 201)])
def test_prefix_scores_that_are_no_numbers(ops, form, first, last):
    # keys of NaN that a row attends to, a whole run of positions among them, make its result NaN
    f, (q, pool, pages, shared, table, own) = case_of(form)
    g = f["hq"] // f["hk"]
    plain, plain_lse = run_prefix(ops, f, q, pool, pages, table)
    put(pool, pages, f["page"], first, last, 0, 1, math.nan)
    out, lse = run_prefix(ops, f, q, pool, pages, table)
    hit = torch.zeros(f["hq"], dtype=torch.bool, device="cuda")
    hit[g:2 * g] = True
    assert bool(out[:, hit].isnan().all()) and bool(lse[:, hit].isnan().all())
    assert torch.equal(out[:, ~hit], plain[:, ~hit]) and torch.equal(lse[:, ~hit], plain_lse[:, ~hit])


@pytest.mark.parametrize("form", FORMS)
def test_prefix_own_scores_that_are_no_numbers(ops, form):
    # among one row's own positions: that row alone
    f, (q, pool, pages, shared, table, own) = case_of(form)
    row = max(range(f["n"]), key=lambda b: f["lens"][b])
    g, plain = f["hq"] // f["hk"], run_prefix(ops, f, q, pool, pages, table)
    for first, last in ((0, 64), (f["lens"][row] - 1, f["lens"][row])):
        put(pool, table[row], f["page"], first, last, 0, 0, math.nan)
        out, lse = run_prefix(ops, f, q, pool, pages, table)
        assert bool(out[row, :g].isnan().all()) and bool(lse[row, :g].isnan().all())
        keep = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
        keep[row, :g] = False
        assert torch.equal(out[keep], plain[0][keep]) and torch.equal(lse[keep], plain[1][keep])
        put(pool, table[row], f["page"], first, last, 0, 0, 0.0)
        plain = run_prefix(ops, f, q, pool, pages, table)


@pytest.mark.parametrize("form", FORMS)
def test_prefix_infinite_values(ops, form):
    # every weight is above 0: an infinite value comes out, and opposite ones make NaN; lse does not see them
    f, (q, pool, pages, shared, table, own) = case_of(form)
    g, (plain, plain_lse) = f["hq"] // f["hk"], run_prefix(ops, f, q, pool, pages, table)
    for p, d, x in ((130, 3, math.inf), (140, 5, -math.inf), (10, 7, math.inf), (290, 7, -math.inf), (150, 9, math.nan)):
        pool[pages[p // f["page"]], 1, 0, p % f["page"], d] = x
    out, lse = run_prefix(ops, f, q, pool, pages, table)
    assert torch.equal(lse, plain_lse)
    assert bool((out[:, :g, 3] == math.inf).all()) and bool((out[:, :g, 5] == -math.inf).all())
    assert bool(out[:, :g, 7].isnan().all()) and bool(out[:, :g, 9].isnan().all())
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[:, :g, [3, 5, 7, 9]] = False
    assert torch.equal(out[keep], plain[keep])


@pytest.mark.parametrize("form", FORMS)
def test_prefix_infinite_values_of_weights_too_small(ops, form):
    # weights under the smallest number beside a far larger one: 0 times an infinity is no number, in every form
    f, (q, pool, pages, shared, table, own) = case_of(form)
    g, d = f["hq"] // f["hk"], f["d"]
    for p in (10, 200):
        for at, x in ((p, 12.0), (p ^ 128, -12.0)):
            put(pool, pages, f["page"], at, at + 1, 0, 0, (x * torch.sign(q[0, 0].float())).to(f["dtype"]))
        pool[pages[(p ^ 128) // f["page"]], 1, 0, (p ^ 128) % f["page"], 2] = math.inf
        out, lse = run_prefix(ops, f, q, pool, pages, table, scale=0.25)
        assert bool(out[0, 0, 2].isnan()) and bool(out[0, 0, 3:].isfinite().all()) and bool(lse.isfinite().all())
        pool[pages[(p ^ 128) // f["page"]], 1, 0, (p ^ 128) % f["page"], 2] = 0.0


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("at", [0, 130, 299])
def test_prefix_scores_far_apart(ops, form, at):
    # one run of keys so far above the rest that what the other splits hold is less than the smallest number beside it
    f, (q, pool, pages, shared, table, own) = case_of(form)
    g, d = f["hq"] // f["hk"], f["d"]
    for p in range(at, min(at + 3, f["prefix"])):
        for h in range(f["hk"]):
            k = (12 * torch.sign(q[0, h * g].float())).to(f["dtype"])  # |score| = 12 sum |q| scale: 77 at D 64
            pool[pages[p // f["page"]], 0, h, p % f["page"]] = k
            shared[0, p, h] = k
    out, lse = run_prefix(ops, f, q, pool, pages, table, scale=0.25)
    T.check_prefix(out, lse, q, shared, own, f["lens"], 0.25, f["dtype"])


@pytest.mark.parametrize("n,prefix,page,d,dtype", [(3, 2500, 16, 128, BF16), (40, 2000, 64, 64, F16),
                                                   (10, 3000, 256, 128, F16), (33, 2999, 16, 64, BF16),
                                                   (5, 4600, 1024, 64, BF16), (2, 2100, 128, 128, BF16),
                                                   (1, 2500, 16, 128, BF16)])  # the last: one row, no shared form
def test_prefix_bad_pages_of_a_long_prefix(ops, n, prefix, page, d, dtype):
    # missing pages in the first, a middle and the last key tile, a run of tiles without any page, and in rows' own
    lens = [(97 * i + 700) % 900 for i in range(n)]
    q, pool, pages, shared, table, own = T.prefix_case(n, prefix, lens, 8, 2, d, page, dtype, n)
    last, bad = len(pages) - 1, [-1, pool.shape[0], 2**31 - 1, -2**31]
    middle = list(range(len(pages) // 2, len(pages) // 2 + max(1, 256 // page)))  # two tiles or more
    gone = sorted({0, *middle, last})
    keep = torch.ones(prefix, dtype=torch.bool, device="cuda")
    for i, p in enumerate(gone):
        pages[p] = bad[i % 4]
        keep[p * page:(p + 1) * page] = False
    shared = shared[:, keep]
    for b in range(0, n, 2):
        if lens[b] > 0:
            p = (lens[b] - 1) // page // 2
            table[b][p] = bad[b % 4]
            own[b] = torch.cat([own[b][:, :p * page], own[b][:, (p + 1) * page:]], 1)
    out, lse = torch.full_like(q, 7.0), torch.full((n, 8), 7.0, device="cuda")
    ops.m3_attn_prefix(q, pool, i32(pages), prefix, i32(table), i32(lens), out, lse)
    T.check_prefix(out, lse, q, shared, own, lens, d ** -0.5, dtype)


@pytest.mark.parametrize("hq,hk,n", [(16, 1, 64), (16, 1, 65), (16, 1, 71), (64, 1, 16), (64, 1, 17), (5, 1, 200),
                                     (33, 1, 24), (32, 8, 256)])
@pytest.mark.parametrize("d,dtype,page,prefix", [(128, BF16, 64, 1000), (64, F16, 16, 1153)])
def test_prefix_rows_of_two_tiles(ops, hq, hk, n, d, dtype, page, prefix):
    # rows enough for CTAs of two row tiles, the second one short or empty
    lens = [(11 * i) % 45 - 1 for i in range(n)]
    q, pool, pages, shared, table, own = T.prefix_case(n, prefix, lens, hq, hk, d, page, dtype, n + hq)
    out, lse = torch.full_like(q, 7.0), torch.full((n, hq), 7.0, device="cuda")
    ops.m3_attn_prefix(q, pool, i32(pages), prefix, i32(table), i32(lens), out, lse)
    T.check_prefix(out, lse, q, shared, own, lens, d ** -0.5, dtype)


@pytest.mark.parametrize("hq,hk", [(1, 1), (17, 1), (24, 4), (5, 1), (64, 1), (7, 7), (66, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix_head_groups_of_a_long_prefix(ops, hq, hk, d):
    lens = [3, 0, 190]
    q, pool, pages, shared, table, own = T.prefix_case(3, 2133, lens, hq, hk, d, 32, BF16, hq)
    out, lse = torch.empty_like(q), torch.empty(3, hq, device="cuda")
    ops.m3_attn_prefix(q, pool, i32(pages), 2133, i32(table), i32(lens), out, lse, scale=0.11)
    T.check_prefix(out, lse, q, shared, own, lens, 0.11, BF16)


@pytest.mark.parametrize("form", FORMS)
def test_prefix_forms(ops, form):
    f, (q, pool, pages, shared, table, own) = case_of(form, 5)
    out, lse = run_prefix(ops, f, q, pool, pages, table)
    T.check_prefix(out, lse, q, shared, own, f["lens"], f["d"] ** -0.5, f["dtype"])


def test_prefix_shorter_than_its_pages(ops):
    # the plan goes by the pages given: splits behind prefix_len have nothing
    for form in FORMS:
        f, (q, pool, pages, shared, table, own) = case_of(form, 6)
        for short in (1, 127, 130):
            out, lse = run_prefix(ops, {**f, "prefix": short}, q, pool, pages, table)
            T.check_prefix(out, lse, q, shared[:, :short], own, f["lens"], f["d"] ** -0.5, f["dtype"])


def test_prefix_workspace_of_a_given_stream(ops):
    # without a workspace the call takes one of the stream it runs on, not memory that the current stream has freed
    # and may still be using
    f, (q, pool, pages, shared, table, own) = case_of("shared", 8)
    want = run_prefix(ops, f, q, pool, pages, table)
    size = ops.m3_attn_prefix_workspace(f["n"], f["hq"], f["hk"], f["d"], len(pages), f["page"], len(table[0]))
    pages_t, table_t, lens_t = i32(pages), i32(table), i32(f["lens"])
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    held = lambda s: [x for x in torch.cuda.memory_snapshot() if x["stream"] == s.cuda_stream]  # noqa: E731
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    st = next(s for s in (torch.cuda.Stream() for _ in range(64)) if not held(s))
    marks = torch.full((size,), 5, dtype=torch.uint8, device="cuda")
    copy = torch.empty_like(marks)
    torch.cuda.synchronize()
    torch.cuda._sleep(2_000_000)  # the current stream is busy, its copy from `marks` yet to come
    copy.copy_(marks)
    del marks
    ops.m3_attn_prefix(q, pool, pages_t, f["prefix"], table_t, lens_t, out, lse, stream=st)
    assert held(st)  # the stream's own memory
    torch.cuda.synchronize()
    assert bool((copy == 5).all())
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("current", ["captured", "other"])
def test_prefix_workspace_of_a_captured_stream(ops, current):
    # a captured call keeps its workspace for its replays, also when another stream is the current one
    f, (q, pool, pages, shared, table, own) = case_of("shared", 8)
    want = run_prefix(ops, f, q, pool, pages, table)
    pages_t, table_t, lens_t = i32(pages), i32(table), i32(f["lens"])
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    st, other, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        with torch.cuda.stream(other if current == "other" else st):
            ops.m3_attn_prefix(q, pool, pages_t, f["prefix"], table_t, lens_t, out, lse, stream=st)
    size = ops.m3_attn_prefix_workspace(f["n"], f["hq"], f["hk"], f["d"], len(pages), f["page"], len(table[0]))
    taken = []
    for s in (torch.cuda.current_stream(), st, other):  # whoever asks now gets other memory
        with torch.cuda.stream(s):
            taken += [torch.full((size,), 5, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(2):
        out.zero_()
        lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert all(bool((x == 5).all()) for x in taken)


def test_prefix_on_the_default_stream_by_hand(ops):
    f, (q, pool, pages, shared, table, own) = case_of("shared", 9)
    want = run_prefix(ops, f, q, pool, pages, table)
    pages_t, table_t, lens_t = i32(pages), i32(table), i32(f["lens"])
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        ops.m3_attn_prefix(q, pool, pages_t, f["prefix"], table_t, lens_t, out, lse, stream=torch.cuda.default_stream())
        assert torch.cuda.current_stream() == other
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ----------------------------------------------------------------- rules ---
# One launch, and the two that many runs (or penalties and biases alone, in place) take.

def rules_both_ways(ops, x, **rules):
    """The same rules out of place, in place (without a mask: two launches), and as many rows (two launches)."""
    out = torch.empty_like(x)
    ops.m3_logit_rules(x, out, **rules)
    if rules.get("mask") is None:
        y = x.clone()
        ops.m3_logit_rules(y, y, **rules)
        assert torch.equal(y.nan_to_num(), out.nan_to_num()) and torch.equal(y.isnan(), out.isnan())
    return out


def test_rules_add_biases_to_the_logit_in_their_order(ops):
    x = torch.tensor([[1.0, 1.0, -3.0, 0.5, 1e8]], device="cuda")
    ids = i32([[0, 1, 0, 1, 3, 4, 4, 4]])
    bias = torch.tensor([[1e8, -1e8, -1e8, 1e8, 2.0, 1.0, 1.0, -1e8]], device="cuda")
    want = x[0].clone()
    for i, b in zip(ids[0].tolist(), bias[0]):
        want[i] += b
    assert want.tolist() == [0.0, 0.0, -3.0, 2.5, 0.0]  # 1 is lost beside 1e8
    assert torch.equal(rules_both_ways(ops, x, bias_ids=ids, bias=bias)[0], want)


def test_rules_divide_by_any_repetition(ops):
    # quotients where 1 / repetition is no normal number, or rounds
    rep = [1e-39, 1e-45, 3e38, 3.4e38, 3.0, 1.1]
    x = torch.tensor([[2.5e-5, -1.0, 0.0, 1e-30, 7.3]] * len(rep), device="cuda")
    r = torch.tensor(rep, device="cuda")
    want = torch.where(x > 0, x / r[:, None], x * r[:, None])
    got = rules_both_ways(ops, x, history=i32([[0, 1, 2, 3, 4]] * len(rep)), repetition=r)
    assert torch.equal(got, want)


@pytest.mark.parametrize("n,r", [(8192, 80), (8192, 2), (60000, 3)])
@pytest.mark.parametrize("ids", ["distinct", "one", "pairs"])
def test_rules_with_the_most_biases(ops, n, r, ids):
    g = gen(n + r)
    x = torch.randn(r, n, generator=g, device="cuda")
    which = torch.rand(r, n, generator=g, device="cuda").topk(4096).indices.to(torch.int32)
    if ids == "one":
        which[:] = 77
    elif ids == "pairs":
        which[:, 2048:] = which[:, :2048].flip(1)
    bias = torch.randn(r, 4096, generator=g, device="cuda")
    history = torch.randint(0, n, (r, 100), generator=g, device="cuda").to(torch.int32)
    pen = torch.full((r,), 0.3, device="cuda")
    want = x.clone()
    for i in range(r):
        seen, c = history[i].long().unique(return_counts=True)
        want[i, seen] -= pen[i] * c
    if ids == "one":
        for e in range(4096):
            want[:, 77] += bias[:, e]
    else:
        half = 2048 if ids == "pairs" else 4096
        for part in range(0, 4096, half):  # the earlier entry of a token first
            want.scatter_add_(1, which[:, part:part + half].long(), bias[:, part:part + half])
    got = rules_both_ways(ops, x, history=history, frequency=pen, bias_ids=which, bias=bias)
    # the penalty's product and difference may be one rounding or two: 2^-24 of their magnitudes each, and then the
    # biases' additions round differently from there, each by as much
    steps = 4 + (4096 if ids == "one" else 2)
    mag = (x.abs() + 0.3 * 100 + (bias.abs().sum(1, keepdim=True) if ids == "one" else 2 * bias.abs().amax()))
    assert bool(((got - want).abs() <= steps * 2.0 ** -23 * mag).all())


def test_rules_time_of_the_most_biases(ops):
    # far from the square of their number (a quarter of a second here): one token's are added one after another
    x, out = torch.zeros(2, 16385, device="cuda"), torch.empty(2, 16385, device="cuda")
    ids, bias = torch.full((2, 4096), 9, dtype=torch.int32, device="cuda"), torch.ones(2, 4096, device="cuda")
    for to in (out, x):  # one launch; in place, the other form
        ops.m3_logit_rules(x, to, bias_ids=ids, bias=bias)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        ops.m3_logit_rules(x, to, bias_ids=ids, bias=bias)
        end.record()
        end.synchronize()
        assert start.elapsed_time(end) < 20.0
    assert out[0, 9] == 4096 and x[0, 9] == 2 * 4096


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rules_between_columns_of_one_buffer(ops, dtype):
    # logits and out side by side in the same rows do not overlap
    for n, gap in ((1000, 0), (1000, 13), (37, 3)):
        buf = torch.zeros(3, 2 * n + gap, dtype=dtype, device="cuda")
        for a, b in ((0, n + gap), (n + gap, 0)):
            x, out = buf[:, a:a + n], buf[:, b:b + n]
            x.copy_(torch.randn(3, n, generator=gen(n), device="cuda"))
            want = x.clone()
            ops.m3_logit_rules(x, out, bias_ids=i32([[5]] * 3), bias=torch.ones(3, 1, device="cuda"))
            assert torch.equal(x, want)
            want[:, 5] = (want[:, 5].float() + 1).to(dtype)
            assert torch.equal(out, want)
