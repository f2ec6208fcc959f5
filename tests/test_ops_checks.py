"""Host-side checks of the serving operators (no GPU needed): the binding covers the header, and what
a call refuses is refused before anything is launched."""
import ctypes as C

import pytest
import torch

from test_abi import _declared


VP, I32, I64, F32 = C.c_void_p, C.c_int, C.c_int64, C.c_float
ARGS = {
    "m3_kv_map": [I32, VP, VP, VP, I32, VP, VP, I32, I64, I32, I32, I32, I32, VP, VP, VP, VP, VP, VP, VP],
    "m3_kv_store": [I32, I32, I32, I32, VP, I64, I64, VP, I64, I64, VP, VP, I32, I32, VP],
    "m3_attn_prompt": [I32, I32, I32, I32, I32, I32, I32, VP, I64, I64, VP, I64, I64, VP, I64, I64, VP, VP, F32, VP,
                       I64, I64, VP, VP],
    "m3_attn_prefix": [I32, I32, I32, I32, I32, VP, I64, I64, VP, I32, I32, VP, I32, I32, VP, I32, I64, VP, F32, VP,
                       I64, I64, VP, VP, I64, VP],
    "m3_logit_rules": [I32, I32, I32, VP, I64, VP, I64, VP, I32, I64, VP, VP, VP, VP, VP, VP, I32, VP, I32, VP, VP],
}


def _lib():
    from autoregressive_audio_token_b200 import m3, ops
    for name, args in ARGS.items():
        getattr(m3.lib, name).argtypes = args
    return m3, ops, m3.lib


P = 1 << 20  # a non-null, aligned address that is never followed


def test_binding_covers_the_operators():
    _, ops, lib = _lib()
    assert sorted(ops.EXPORTED) == _declared("m3_ops.h")
    for n in ops.EXPORTED:
        assert hasattr(ops, n) and hasattr(lib, n), n


MAP = dict(n_req=2, fresh=P, cached=None, free=P, n_free=4, free_at=None, table=P, max_pages=3, ld=3,
           page=16, n_pages=8, start=0, n_tokens=4, cu=P + 64, positions=P, slots=P, seqs=P, lens=P + 128,
           taken=P, stream=None)


@pytest.mark.parametrize("bad", [dict(n_req=0), dict(n_req=8193), dict(page=24), dict(page=8), dict(page=2048),
                                 dict(n_free=-1), dict(max_pages=-1), dict(n_pages=-1), dict(start=-1),
                                 dict(n_tokens=-1), dict(ld=2), dict(fresh=None), dict(table=None), dict(cu=None),
                                 dict(slots=None), dict(taken=None), dict(free=None), dict(lens=None),
                                 dict(free_at=P), dict(lens=P + 4), dict(cu=P), dict(cached=P + 128), dict(cached=P + 72), dict(positions=P + 4), dict(slots=P + 8), dict(seqs=P + 4)])
def test_map_refuses(bad):
    m3, _, lib = _lib()
    assert lib.m3_kv_map(*{**MAP, **bad}.values()) == m3.M3_EINVAL
    assert m3.m3_last_error()


STORE = dict(dtype=0, n=4, hk=2, d=64, k=P, kt=128, kh=64, v=P, vt=128, vh=64, slots=P, pool=P, n_pages=2,
             page=16, stream=None)


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(n=-1), dict(hk=0), dict(d=4), dict(d=12), dict(d=1032),
                                 dict(page=15), dict(k=None), dict(v=None), dict(slots=None), dict(pool=None),
                                 dict(pool=P + 2), dict(n_pages=-1)])
def test_store_refuses(bad):
    m3, _, lib = _lib()
    assert lib.m3_kv_store(*{**STORE, **bad}.values()) == m3.M3_EINVAL


PROMPT = dict(dtype=0, n_seq=1, n_q=4, n_k=4, hq=4, hk=2, d=64, q=P, qt=256, qh=64, k=P, kt=128, kh=64, v=P,
              vt=128, vh=64, cu_q=P, cu_k=None, scale=0.125, out=P, ot=256, oh=64, lse=None, stream=None)


@pytest.mark.parametrize("bad", [dict(dtype=-1), dict(n_seq=-1), dict(n_seq=8193), dict(n_q=-1), dict(n_k=3), dict(hq=3), dict(hk=0),
                                 dict(hq=130, hk=2), dict(d=96), dict(q=None), dict(k=None), dict(v=None), dict(out=None),
                                 dict(cu_q=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                 dict(scale=float("inf")), dict(q=P + 8), dict(k=P + 2), dict(v=P + 8), dict(out=P + 8),
                                 dict(qt=250), dict(kh=60), dict(vt=0), dict(ot=252), dict(kt=-128)])
def test_prompt_refuses(bad):
    m3, _, lib = _lib()
    assert lib.m3_attn_prompt(*{**PROMPT, **bad}.values()) == m3.M3_EINVAL


PREFIX = dict(dtype=0, n=2, hq=4, hk=2, d=64, q=P, qr=256, qh=64, pool=P, n_pages=4, page=16, pages=P, n_prefix=2,
              prefix_len=20, table=P, max_pages=2, ld=2, lens=P, scale=0.125, out=P, orow=256, oh=64, lse=None, ws=P,
              ws_bytes=1 << 24, stream=None)


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(n=-1), dict(hq=5), dict(d=32), dict(page=17), dict(prefix_len=33),
                                 dict(prefix_len=-1), dict(n_prefix=-1), dict(max_pages=-1), dict(ld=1), dict(q=None),
                                 dict(pool=None), dict(pages=None), dict(table=None), dict(lens=None), dict(out=None),
                                 dict(scale=0.0), dict(q=P + 2), dict(pool=P + 8), dict(out=P + 4), dict(qr=252),
                                 dict(oh=0), dict(ws=None), dict(ws=P + 4), dict(ws_bytes=16),
                                 dict(n_prefix=1 << 27, prefix_len=5, page=1024)])
def test_prefix_refuses(bad):
    m3, _, lib = _lib()
    assert lib.m3_attn_prefix(*{**PREFIX, **bad}.values()) == m3.M3_EINVAL


def test_prefix_workspace_is_zero_for_what_is_refused():
    _, ops, _ = _lib()
    assert ops.m3_attn_prefix_workspace(2, 4, 2, 64, 2, 16, 2) > 0
    for bad in ((0, 4, 2, 64, 2, 16, 2), (2, 5, 2, 64, 2, 16, 2), (2, 4, 2, 80, 2, 16, 2), (2, 4, 2, 64, 2, 20, 2),
                (2, 4, 2, 64, -1, 16, 2)):
        assert ops.m3_attn_prefix_workspace(*bad) == 0


RULES = dict(dtype=0, n=2, vocab=100, x=P, ldx=100, out=P, ldo=100, hist=P, nh=5, ldh=5, hl=None, rep=None, freq=None,
             pres=None, ids=P, bias=P, nb=3, mask=P, nm=2, mr=None, stream=None)


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(n=-1), dict(vocab=0), dict(x=None), dict(out=None), dict(nb=4097), dict(nh=(1 << 24) + 1, ldh=1 << 25),
                                 dict(nb=-1), dict(ids=None), dict(bias=None), dict(hist=None), dict(nh=-1), dict(ldx=99),
                                 dict(ldo=99), dict(ldh=4), dict(nm=0), dict(nm=3), dict(out=P + 400), dict(x=P + 2),
                                 dict(out=P, ldo=104)])
def test_rules_refuse(bad):
    m3, _, lib = _lib()
    assert lib.m3_logit_rules(*{**RULES, **bad}.values()) == m3.M3_EINVAL


def test_calls_without_work_are_fine():
    m3, _, lib = _lib()
    assert lib.m3_kv_store(*{**STORE, "n": 0}.values()) == m3.M3_OK
    assert lib.m3_attn_prompt(*{**PROMPT, "n_seq": 0}.values()) == m3.M3_OK
    assert lib.m3_attn_prefix(*{**PREFIX, "n": 0}.values()) == m3.M3_OK
    assert lib.m3_logit_rules(*{**RULES, "n": 0}.values()) == m3.M3_OK


def test_binding_refuses_shapes_types_and_host_tensors():
    m3, ops, _ = _lib()
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    calls = [
        lambda: ops.m3_attn_prompt(q, kv, kv, cu, torch.empty_like(q)),                      # on the host
        lambda: ops.m3_attn_prompt(q.float(), kv, kv, cu, q),                                # type
        lambda: ops.m3_attn_prompt(q, kv.half(), kv, cu, torch.empty_like(q)),               # mixed types
        lambda: ops.m3_attn_prompt(q, kv, kv[:3], cu, torch.empty_like(q)),                  # rows
        lambda: ops.m3_attn_prompt(q, kv, kv, cu.long(), torch.empty_like(q)),               # cu type
        lambda: ops.m3_attn_prompt(q.transpose(1, 2), kv, kv, cu, torch.empty_like(q)),      # D strided
        lambda: ops.m3_kv_store(kv, kv, torch.zeros(3, dtype=torch.int64), torch.zeros(2, 2, 2, 16, 64)),
        lambda: ops.m3_logit_rules(torch.zeros(2, 8, dtype=torch.float64), torch.zeros(2, 8)),
        lambda: ops.m3_logit_rules(torch.zeros(2, 8), torch.zeros(2, 9)),
        lambda: ops.m3_logit_rules(torch.zeros(2, 8), torch.zeros(2, 8), bias=torch.zeros(2, 1)),
    ]
    for call in calls:
        with pytest.raises(m3.M3Error) as e:
            call()
        assert e.value.code == m3.M3_EINVAL
