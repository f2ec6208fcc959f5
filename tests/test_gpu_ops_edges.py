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
