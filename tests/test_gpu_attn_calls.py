"""The attention operators called in ways that the documentation allows or names an error: lists and offsets that
do not fit, arguments by name, new memory as torch's settings want it."""
import pytest
import torch

from attn_cases import cache, frequencies, gen, normal
from linear_attention_token_gdn_b200 import build as gbuild
from linear_attention_token_gdn_b200 import gdn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    gbuild.build()
    gdn.lib()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def test_an_empty_list_of_pages_is_refused():
    """[B, Hkv, 0] is a list without a place, not the absence of a list."""
    kc, vc, table, lens = cache(1, [40, 17], 2, 64, 16, BF16)
    q = normal(gen(1), 2, 4, 64, dtype=BF16)
    with pytest.raises(ValueError):
        gdn.attn_decode(q, kc, vc, table, lens, pages=torch.empty(2, 2, 0, dtype=torch.int32, device="cuda"))
    none = torch.full((2, 2, 1), -1, dtype=torch.int32, device="cuda")  # a list without a page: zeros
    assert not gdn.attn_decode(q, kc, vc, table, lens, pages=none).any()
    gdn.check_device_error()


def fill_cache(cu, N, Hq=2, Hkv=2, d=64):
    """Tokens 0 .. N - 1 at positions 0 .. N - 1 of sequences with a page of 16 places each."""
    g, num_seqs = gen(2), len(cu) - 1
    q, k, v = (normal(g, N, h, d, dtype=BF16) for h in (Hq, Hkv, Hkv))
    w = torch.zeros(d, device="cuda")
    kc, vc = (torch.zeros(num_seqs, Hkv, 16, d, device="cuda", dtype=BF16) for _ in range(2))
    table = torch.arange(num_seqs, dtype=torch.int32, device="cuda")[:, None].contiguous()
    gdn.attn_prep_cache(q, k, v, w, w, torch.arange(N, dtype=torch.int32, device="cuda"), None, kc, vc, table, cu_seqlens=ints(cu))
    return v, vc


MALFORMED = [[0, 6, 2, 8], [0, 5, 3], [-4, 3, 8], [0, 4, 12], [3, 5, 8], [2, 8], [0, -1, 8], [0, 8, 7], [0, 9, 8]]


@pytest.mark.parametrize("cu", MALFORMED, ids=str)
def test_the_cache_form_flags_malformed_offsets(cu):
    fill_cache(cu, 8)
    with pytest.raises(gdn.GDNError) as e:
        gdn.check_device_error()
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG and "cu_seqlens" in str(e.value)
    gdn.check_device_error()  # cleared


@pytest.mark.parametrize("at,value", [(0, 1), (1, -1), (650, 2), (699, -3), (700, 2)])
def test_the_cache_form_checks_every_offset_of_many_sequences(at, value):
    """One token with one query and one key head of 16 channels: two threads look at 700 sequences."""
    cu = [0] * 300 + [1] * 401
    fill_cache(cu, 1, 1, 1, 16)
    gdn.check_device_error()
    cu[at] = value
    fill_cache(cu, 1, 1, 1, 16)
    with pytest.raises(gdn.GDNError):
        gdn.check_device_error()


@pytest.mark.parametrize("cu", [[0, 8], [0, 0, 8], [0, 8, 8, 8], [0, 3, 3, 5], [0, 0], [0, 0, 0, 1, 1, 7]], ids=str)
def test_the_cache_form_takes_empty_sequences_and_tokens_behind_the_last(cu):
    v, vc = fill_cache(cu, 8)
    gdn.check_device_error()
    for b in range(len(cu) - 1):
        places = set(range(cu[b], cu[b + 1]))
        for p in range(16):
            assert torch.equal(vc[b, :, p], v[p]) if p in places else not vc[b, :, p].any()


def test_every_argument_by_name():
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 16
    kc, vc, table, lens = cache(4, [40, 7, 100], Hkv, d, page, BF16)
    g, f, pos = gen(4), frequencies(64), ints([39, 6, 99])
    q, k, v = (normal(g, B, h, d, dtype=BF16) for h in (Hq, Hkv, Hkv))
    wq, wk = normal(g, d), normal(g, d)
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    assert same(gdn.attn_prep(q=q, k=k, w_q=wq, w_k=wk, positions=pos, inv_freq=f), gdn.attn_prep(q, k, wq, wk, pos, f))
    a = gdn.attn_prep_bwd(dq_out=q, dk_out=k, q=q, k=k, w_q=wq, w_k=wk, positions=pos, inv_freq=f)
    assert same(a.values(), gdn.attn_prep_bwd(q, k, q, k, wq, wk, pos, f).values())
    kc2, vc2 = kc.clone(), vc.clone()
    a = gdn.attn_prep_cache(q=q, k=k, v=v, w_q=wq, w_k=wk, positions=pos, inv_freq=f, k_cache=kc2, v_cache=vc2, page_table=table)
    assert torch.equal(a, gdn.attn_prep_cache(q, k, v, wq, wk, pos, f, kc, vc, table))
    mean = gdn.attn_page_mean(k_cache=kc, page_table=table, lens=lens)
    assert torch.equal(mean, gdn.attn_page_mean(kc, table, lens))
    pages = gdn.attn_select(q=q, page_mean=mean, page_table=table, lens=lens, page_size=page, n_sel=3)
    assert torch.equal(pages, gdn.attn_select(q, mean, table, lens, page, 3))
    y = gdn.attn_decode(q=q, k_cache=kc, v_cache=vc, page_table=table, lens=lens, pages=pages)
    assert torch.equal(y, gdn.attn_decode(q, kc, vc, table, lens, pages=pages))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = gdn.attn_decode(q=q, k_cache=kc, v_cache=vc, page_table=table, lens=lens, pages=pages, stream=side)
    side.synchronize()
    assert torch.equal(y, z)
    gdn.check_device_error()


def test_new_outputs_are_filled_as_the_deterministic_setting_wants():
    """torch fills new memory with NaN under deterministic algorithms; a padding token's row of q_out is such memory."""
    g = gen(5)
    q, k, v = (normal(g, 2, h, 64, dtype=BF16) for h in (4, 2, 2))
    w, pos = torch.zeros(64, device="cuda"), ints([3, -1])
    kc, vc = (torch.zeros(2, 2, 16, 64, device="cuda", dtype=BF16) for _ in range(2))
    table = ints([[0], [1]])
    call = lambda: gdn.attn_prep_cache(q, k, v, w, w, pos, None, kc, vc, table)  # noqa: E731
    want = call()[0].clone()
    torch.cuda.synchronize()
    before = torch.are_deterministic_algorithms_enabled(), torch.is_deterministic_algorithms_warn_only_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        old = torch.full((2, 4, 64), 3.0, device="cuda", dtype=BF16)  # what the new output's memory may hold
        del old
        got = call()
    finally:
        torch.use_deterministic_algorithms(before[0], warn_only=before[1])
    gdn.check_device_error()
    assert torch.equal(got[0], want) and got[1].isnan().all()
