"""Overlapping and misshapen arguments of the serving operators, refused before anything is launched (no GPU needed)."""
import pytest
import torch

from test_ops_checks import RULES, _lib

# disjoint, aligned addresses that are never followed
MAP = dict(n_req=4, fresh=0x10000, cached=0x20000, free=0x30000, n_free=4, free_at=0x40000, table=0x50000, max_pages=3,
           ld=3, page=16, n_pages=8, start=0, n_tokens=8, cu=0x60000, positions=0x70000, slots=0x80000, seqs=0x90000,
           lens=0xA0000, taken=0xB0000, stream=None)
INPUTS = dict(fresh=16, cached=16, free=16, free_at=4)
OUTPUTS = dict(cu=20, lens=16, taken=4, positions=32, seqs=32, slots=64)


def refusal(**changed):
    m3, _, lib = _lib()
    assert lib.m3_kv_map(*{**MAP, **changed}.values()) == m3.M3_EINVAL
    return m3.m3_last_error()


@pytest.mark.parametrize("i", INPUTS)
@pytest.mark.parametrize("o", OUTPUTS)
def test_map_outputs_are_no_inputs(i, o):
    at = MAP[i]
    wide = o in ("positions", "seqs", "slots")  # aligned to 16 bytes: the input is moved instead
    for where in {0, INPUTS[i] - 4}:  # the output starts on the input's first word, on its last
        moved = {i: MAP[o] - where} if wide else {o: at + where}
        assert "an output overlaps" in refusal(**moved), where
    last = OUTPUTS[o] - 4  # the input starts on the output's last word
    assert "an output overlaps" in refusal(**{i: MAP[o] + last})


@pytest.mark.parametrize("i", INPUTS)
@pytest.mark.parametrize("o", OUTPUTS)
def test_map_neighbours_are_no_overlap(i, o):
    # what touches without overlapping gets as far as the next check, here an unaligned map
    bad = "positions" if o == "seqs" else "seqs"
    for at in (MAP[o] - INPUTS[i], MAP[o] + OUTPUTS[o]):
        assert "16-byte aligned" in refusal(**{i: at, bad: MAP[bad] + 4})


@pytest.mark.parametrize("o", OUTPUTS)
def test_map_a_list_without_pages_overlaps_nothing(o):
    bad = "positions" if o == "seqs" else "seqs"
    assert "16-byte aligned" in refusal(free=MAP[o] + 4 * (OUTPUTS[o] > 4), n_free=0, **{bad: MAP[bad] + 4})


@pytest.mark.parametrize("x,out,ld", [(0, 1, 200), (0, 99, 200), (0, 101, 200), (99, 0, 200), (101, 0, 200), (0, 100, 199),
                                      (100, 0, 199), (0, 199, 200), (0, 201, 200), (301, 0, 200), (0, 50, 100)])
def test_rules_columns_that_overlap(x, out, ld):
    # rows of 100 in one buffer of fp32 whose columns share places, in the same rows or the next
    m3, _, lib = _lib()
    base = RULES["x"]
    call = {**RULES, "n": 3, "x": base + 4 * x, "out": base + 4 * out, "ldx": ld, "ldo": ld, "nm": 3}
    assert lib.m3_logit_rules(*call.values()) == m3.M3_EINVAL
    assert "out overlaps" in m3.m3_last_error()


@pytest.mark.parametrize("bad", [dict(bias_ids=torch.zeros(2, 1, dtype=torch.int32), bias=torch.tensor(1.0)),
                                 dict(bias_ids=torch.tensor(3, dtype=torch.int32), bias=torch.tensor(1.0)),
                                 dict(bias_ids=torch.zeros(2, dtype=torch.int32), bias=torch.zeros(2)),
                                 dict(mask=torch.tensor(0, dtype=torch.int32)), dict(mask=torch.zeros(1, dtype=torch.int32)),
                                 dict(history=torch.tensor(1, dtype=torch.int32))])
def test_rules_of_too_few_dimensions(bad):
    m3, ops, _ = _lib()
    x = torch.zeros(2, 8)
    with pytest.raises(m3.M3Error) as e:
        ops.m3_logit_rules(x, x, **bad)
    assert e.value.code == m3.M3_EINVAL
