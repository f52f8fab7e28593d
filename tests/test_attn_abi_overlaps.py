"""Outputs and workspaces of the attention entry points that lie on another tensor are refused, on the host: nothing is
enqueued, no device is needed."""
import ctypes

import pytest

from linear_attention_token_gdn_b200 import build as gbuild
from linear_attention_token_gdn_b200 import gdn
from test_attn_abi import at, decode, page_mean, prep, prep_bwd, prep_cache, select


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


def inside(i, offset):
    """`offset` bytes behind at(i)."""
    return ctypes.c_void_p(at(i).value + offset)


def refused(status):
    assert status == gdn.GDN_ERR_INVALID_ARG and "overlaps" in gdn.last_error_message()


# Of 8 tokens, 16 heads over 2 of 128 channels: w, dw and inv_freq (half of it in the cache form, whose table has 160) of 512
# bytes, positions of 32.
@pytest.mark.parametrize("over", [dict(qo=at(2)), dict(qo=at(4)), dict(qo=inside(5, 496)), dict(ko=inside(3, 496)),
                                  dict(ko=inside(4, 16)), dict(ko=at(5)), dict(wq=inside(6, 16 * 128 * 2 * 8 - 16))])
def test_prep_refuses_outputs_on_its_small_inputs(L, over):
    refused(prep(L, **over))


@pytest.mark.parametrize("over", [dict(qo=at(3)), dict(qo=at(5)), dict(kc=inside(6, 240)), dict(vc=at(7)), dict(vc=inside(7, 144)),
                                  dict(cu=inside(9, 64)), dict(cu=at(8)), dict(wk=inside(10, 1 << 20)), dict(table=inside(8, 16))])
def test_prep_cache_refuses_outputs_on_its_small_inputs(L, over):
    refused(prep_cache(L, **over))


OUTPUTS = dict(dq=16 * 128 * 2 * 8, dk=2 * 128 * 2 * 8, dwq=512, dwk=512, ws=2048 * 128 * 4)  # bytes
INPUTS = dict(gq=16 * 128 * 2 * 8, gk=2 * 128 * 2 * 8, q=16 * 128 * 2 * 8, k=2 * 128 * 2 * 8, wq=512, wk=512, pos=32, f=512)


@pytest.mark.parametrize("of", INPUTS)
@pytest.mark.parametrize("out", OUTPUTS)
def test_prep_bwd_refuses_outputs_on_inputs(L, out, of):
    where = at(20)
    refused(prep_bwd(L, **{out: where, of: where}))
    refused(prep_bwd(L, **{out: where, of: inside(20, OUTPUTS[out] - 16)}))
    refused(prep_bwd(L, **{out: inside(20, INPUTS[of] - 16), of: where}))


@pytest.mark.parametrize("a,b", [(a, b) for i, a in enumerate(OUTPUTS) for b in list(OUTPUTS)[i + 1:]])
def test_prep_bwd_refuses_outputs_on_outputs(L, a, b):
    where = at(20)
    refused(prep_bwd(L, **{a: where, b: where}))
    refused(prep_bwd(L, **{a: where, b: inside(20, OUTPUTS[a] - 16)}))
    refused(prep_bwd(L, **{a: inside(20, OUTPUTS[b] - 16), b: where}))


def on_one_another(call, a, na, b, nb):
    """The call with tensor `b` on `a`, and each on the other's last 16 bytes."""
    for where in ({a: at(20), b: at(20)}, {a: at(20), b: inside(20, na - 16)}, {a: inside(20, nb - 16), b: at(20)}):
        refused(call(**where))


# 4 rows, 16 heads over 2 of 128 channels, 10 pages a row of 100 of 64 places
ROWS = dict(q=4 * 16 * 128 * 2, table=4 * 10 * 4, lens=16)
CACHES = dict(kc=100 * 2 * 64 * 128 * 2, vc=100 * 2 * 64 * 128 * 2)


@pytest.mark.parametrize("out,n", [("y", 4 * 16 * 128 * 2), ("ws", 640 * 2 * 4 + 640 * 2 * 8 * 130 * 4)])
@pytest.mark.parametrize("of", [*ROWS, *CACHES, "pages"])
def test_decode_refuses_outputs_on_inputs(L, out, n, of):
    sizes = dict(ROWS, **CACHES, pages=4 * 2 * 6 * 4)
    lists = dict(pages=at(7), ns=6)
    on_one_another(lambda **over: decode(L, **dict(lists, **over)), out, n, of, sizes[of])


def test_decode_refuses_its_output_in_its_workspace(L):
    on_one_another(lambda **over: decode(L, **over), "y", 4 * 16 * 128 * 2, "ws", 640 * 2 * 4 + 640 * 2 * 8 * 130 * 4)


@pytest.mark.parametrize("of,n", [("kc", CACHES["kc"]), ("table", 160), ("lens", 16), ("starts", 16)])
def test_page_mean_refuses_means_on_inputs(L, of, n):
    on_one_another(lambda **over: page_mean(L, **over), "mean", 100 * 2 * 128 * 4, of, n)


@pytest.mark.parametrize("out,n", [("pages", 4 * 2 * 4 * 4), ("ws", 4 * 2 * 10 * 8)])
@pytest.mark.parametrize("of", [*ROWS, "mean"])
def test_select_refuses_outputs_on_inputs(L, out, n, of):
    on_one_another(lambda **over: select(L, **over), out, n, of, dict(ROWS, mean=100 * 2 * 128 * 4)[of])


def test_select_refuses_its_list_in_its_workspace(L):
    on_one_another(lambda **over: select(L, **over), "pages", 4 * 2 * 4 * 4, "ws", 4 * 2 * 10 * 8)
