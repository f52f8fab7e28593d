"""Refusals of the attention entry points, on the host: nothing is enqueued, no device is needed."""
import ctypes

import pytest
import torch

from linear_attention_token_gdn_b200 import build as gbuild
from linear_attention_token_gdn_b200 import gdn

BAD, NOT_BUILT = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


def at(i):
    """A made-up aligned address, far from the others: checks never dereference it."""
    return ctypes.c_void_p((i + 1) << 40)


MIS = ctypes.c_void_p((99 << 40) + 4)


def prep(L, **over):
    a = dict(q=at(0), k=at(1), qs=16 * 128, ks=2 * 128, wq=at(2), wk=at(3), eps=1e-6, pos=at(4), f=at(5), rot=128, N=8, Hq=16,
             Hkv=2, d=128, i=gdn.BF16, o=gdn.BF16, qo=at(6), ko=at(7))
    a.update(over)
    return L.gdn_attn_prep(a["q"], a["k"], a["qs"], a["ks"], a["wq"], a["wk"], a["eps"], a["pos"], a["f"], a["rot"], a["N"],
                           a["Hq"], a["Hkv"], a["d"], a["i"], a["o"], a["qo"], a["ko"], None)


@pytest.mark.parametrize("over", [
    dict(q=None), dict(k=MIS), dict(qs=16 * 128 - 8), dict(qs=16 * 128 + 4), dict(ks=0), dict(wq=None), dict(eps=-1.0),
    dict(pos=None), dict(f=None), dict(rot=24), dict(rot=144), dict(rot=-16), dict(N=-1), dict(Hq=15), dict(Hkv=0), dict(d=48),
    dict(d=512), dict(i=3), dict(o=-1), dict(qo=None), dict(ko=MIS), dict(eps=float("nan")),
    dict(qo=at(7)),                                            # q_out over k_out
    dict(qo=ctypes.c_void_p((1 << 40) + 4096)),                # q_out inside q
    dict(qo=at(0), qs=16 * 128 + 8),                           # in place, but strided
    dict(qo=at(0), o=gdn.F32),                                 # in place, but of another type
    dict(ko=at(0)),                                            # k_out over q
    dict(N=1 << 30, Hq=64, Hkv=64, qs=64 * 128, ks=64 * 128),  # too many rows for the grid
])
def test_prep_refuses(L, over):
    assert prep(L, **over) == BAD
    assert gdn.last_error_message() != ""


def test_prep_of_no_tokens_is_a_no_op(L):
    assert prep(L, N=0, q=None, k=None, qo=None, ko=None, pos=None) == gdn.GDN_OK


def prep_cache(L, **over):
    a = dict(q=at(0), k=at(1), v=at(2), qs=16 * 128, ks=256, vs=256, wq=at(3), wk=at(4), eps=1e-6, pos=at(5), f=at(6), rot=64,
             cu=None, ns=4, N=8, Hq=16, Hkv=2, d=128, table=at(7), mp=10, np=100, ps=64, i=gdn.BF16, o=gdn.BF16, qo=at(8),
             kc=at(9), vc=at(10))
    a.update(over)
    return L.gdn_attn_prep_cache(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["wq"], a["wk"], a["eps"], a["pos"],
                                 a["f"], a["rot"], a["cu"], a["ns"], a["N"], a["Hq"], a["Hkv"], a["d"], a["table"], a["mp"],
                                 a["np"], a["ps"], a["i"], a["o"], a["qo"], a["kc"], a["vc"], None)


@pytest.mark.parametrize("over,status", [
    (dict(v=None), BAD), (dict(vs=248), BAD), (dict(vs=260), BAD), (dict(ns=0), BAD), (dict(ns=3), BAD), (dict(N=-1), BAD),
    (dict(table=None), BAD), (dict(mp=0), BAD), (dict(np=0), BAD), (dict(ps=0), BAD), (dict(ps=24), NOT_BUILT),
    (dict(ps=2048), NOT_BUILT), (dict(o=gdn.F32), NOT_BUILT), (dict(mp=1 << 25), BAD), (dict(kc=None), BAD), (dict(vc=MIS), BAD),
    (dict(vc=at(9)), BAD), (dict(kc=at(0)), BAD), (dict(qo=at(9)), BAD), (dict(qo=at(2)), BAD), (dict(cu=MIS), BAD),
    (dict(f=None), BAD), (dict(rot=8), BAD), (dict(d=96), BAD), (dict(Hq=3), BAD),
])
def test_prep_cache_refuses(L, over, status):
    assert prep_cache(L, **over) == status
    assert gdn.last_error_message() != ""


def test_prep_cache_of_no_tokens_is_a_no_op(L):
    assert prep_cache(L, N=0, q=None, k=None, v=None, kc=None, vc=None) == gdn.GDN_OK


def prep_bwd(L, **over):
    a = dict(gq=at(0), gk=at(1), q=at(2), k=at(3), qs=16 * 128, ks=256, wq=at(4), wk=at(5), eps=1e-6, pos=at(6), f=at(7), rot=128,
             N=8, Hq=16, Hkv=2, d=128, i=gdn.BF16, g=gdn.BF16, dq=at(8), dk=at(9), dwq=at(10), dwk=at(11), ws=at(12), n=1 << 30)
    a.update(over)
    return L.gdn_attn_prep_bwd(a["gq"], a["gk"], a["q"], a["k"], a["qs"], a["ks"], a["wq"], a["wk"], a["eps"], a["pos"], a["f"],
                               a["rot"], a["N"], a["Hq"], a["Hkv"], a["d"], a["i"], a["g"], a["dq"], a["dk"], a["dwq"],
                               a["dwk"], a["ws"], a["n"], None)


@pytest.mark.parametrize("over", [
    dict(gq=None), dict(gk=MIS), dict(q=None), dict(qs=8), dict(eps=-1.0), dict(rot=20), dict(N=-1), dict(Hq=5), dict(d=100),
    dict(i=4), dict(g=4), dict(dq=None), dict(dwq=None), dict(dwk=MIS), dict(ws=None), dict(n=100), dict(dq=at(0)), dict(dk=at(2)),
    dict(dq=at(9)), dict(f=None),
])
def test_prep_bwd_refuses(L, over):
    assert prep_bwd(L, **over) == BAD
    assert gdn.last_error_message() != ""


def decode(L, **over):
    a = dict(q=at(0), kc=at(1), vc=at(2), table=at(3), lens=at(4), pages=None, ns=0, B=4, Hq=16, Hkv=2, d=128, mp=10, np=100, ps=64,
             scale=0.1, i=gdn.BF16, y_dt=gdn.BF16, y=at(5), ws=at(6), n=1 << 30)
    a.update(over)
    return L.gdn_attn_decode(a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["pages"], a["ns"], a["B"], a["Hq"], a["Hkv"],
                             a["d"], a["mp"], a["np"], a["ps"], a["scale"], a["i"], a["y_dt"], a["y"], a["ws"], a["n"], None)


@pytest.mark.parametrize("over,status", [
    (dict(q=None), BAD), (dict(kc=MIS), BAD), (dict(table=None), BAD), (dict(lens=None), BAD), (dict(pages=MIS, ns=4), BAD),
    (dict(pages=at(7), ns=0), BAD), (dict(pages=at(7), ns=1 << 25), BAD), (dict(B=-1), BAD), (dict(Hq=15), BAD), (dict(Hkv=0), BAD),
    (dict(d=0), BAD), (dict(d=16), NOT_BUILT), (dict(d=96), NOT_BUILT), (dict(i=gdn.F32), NOT_BUILT), (dict(i=5), BAD),
    (dict(y_dt=5), BAD), (dict(ps=40), NOT_BUILT), (dict(ps=0), BAD), (dict(mp=0), BAD), (dict(mp=1 << 26), BAD),
    (dict(scale=float("nan")), BAD), (dict(y=at(0)), BAD), (dict(y=None), BAD), (dict(ws=None), BAD), (dict(n=4096), BAD),
    (dict(y=at(1)), BAD), (dict(y=at(2)), BAD),
])
def test_decode_refuses(L, over, status):
    assert decode(L, **over) == status
    assert gdn.last_error_message() != ""


def test_decode_workspace_does_not_depend_on_the_batch(L):
    size = L.gdn_attn_decode_workspace_size
    assert size(16, 2, 128) == 640 * 2 * 4 + 640 * 2 * 8 * 130 * 4
    assert size(32, 2, 128) == 640 * 2 * 4 + 640 * 2 * 16 * 130 * 4
    assert size(32, 2, 256) == 640 * 2 * 4 + 640 * 2 * 8 * 258 * 4
    assert size(16, 3, 128) == 0 and size(16, 2, 100) == 0


def test_no_rows_is_a_no_op(L):
    assert decode(L, B=0, q=None, y=None, ws=None) == gdn.GDN_OK
    assert page_mean(L, B=0, kc=None) == gdn.GDN_OK
    assert select(L, B=0, q=None, ws=None) == gdn.GDN_OK


def page_mean(L, **over):
    a = dict(kc=at(0), table=at(1), lens=at(2), starts=None, B=4, Hkv=2, d=128, mp=10, np=100, ps=64, i=gdn.BF16, mean=at(3))
    a.update(over)
    return L.gdn_attn_page_mean(a["kc"], a["table"], a["lens"], a["starts"], a["B"], a["Hkv"], a["d"], a["mp"], a["np"],
                                a["ps"], a["i"], a["mean"], None)


@pytest.mark.parametrize("over,status", [
    (dict(kc=None), BAD), (dict(starts=MIS), BAD), (dict(B=-1), BAD), (dict(Hkv=0), BAD), (dict(d=0), BAD), (dict(d=16), NOT_BUILT),
    (dict(i=gdn.F32), NOT_BUILT), (dict(mean=MIS), BAD), (dict(ps=17), NOT_BUILT), (dict(np=0), BAD), (dict(mean=at(0)), BAD),
])
def test_page_mean_refuses(L, over, status):
    assert page_mean(L, **over) == status
    assert gdn.last_error_message() != ""


def select(L, **over):
    a = dict(q=at(0), mean=at(1), table=at(2), lens=at(3), B=4, Hq=16, Hkv=2, d=128, mp=10, np=100, ps=64, ns=4, first=1, last=1,
             i=gdn.BF16, pages=at(4), ws=at(5), n=1 << 30)
    a.update(over)
    return L.gdn_attn_select(a["q"], a["mean"], a["table"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["d"], a["mp"], a["np"],
                             a["ps"], a["ns"], a["first"], a["last"], a["i"], a["pages"], a["ws"], a["n"], None)


@pytest.mark.parametrize("over,status", [
    (dict(q=None), BAD), (dict(mean=MIS), BAD), (dict(ns=0), BAD), (dict(first=-1), BAD), (dict(last=-1), BAD),
    (dict(first=3, last=2), BAD), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), BAD), (dict(d=16), NOT_BUILT),
    (dict(i=gdn.F32), NOT_BUILT), (dict(Hq=3), BAD), (dict(pages=None), BAD), (dict(ws=None), BAD),
    (dict(n=4 * 2 * 10 * 8 - 1), BAD), (dict(ps=8), NOT_BUILT), (dict(mp=-1), BAD),
])
def test_select_refuses(L, over, status):
    assert select(L, **over) == status
    assert gdn.last_error_message() != ""


def test_the_binding_refuses_host_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    w, pos = torch.zeros(64), torch.zeros(2, dtype=torch.int32)
    cache, table = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: gdn.attn_prep(x, x, w, w, pos, None),
                 lambda: gdn.attn_prep_cache(x, x, x, w, w, pos, None, cache, cache, table),
                 lambda: gdn.attn_prep_bwd(x, x, x, x, w, w, pos, None),
                 lambda: gdn.attn_decode(x, cache, cache, table, pos),
                 lambda: gdn.attn_page_mean(cache, table, pos),
                 lambda: gdn.attn_select(x, torch.zeros(4, 2, 64), table, pos, 16, 2)):
        with pytest.raises(ValueError):
            call()
