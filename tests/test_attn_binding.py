"""The attention functions of the binding on the host: how they take their arguments; no device is needed."""
import pytest
import torch

from linear_attention_token_gdn_b200 import gdn


def test_the_binding_takes_its_first_argument_by_name():
    """Host tensors are refused for being host tensors, however they are passed; without a first argument the call
    names the parameter that is missing."""
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    w, pos = torch.zeros(64), torch.zeros(2, dtype=torch.int32)
    cache, table = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    rows = dict(k=x, w_q=w, w_k=w, positions=pos, inv_freq=None)
    pages = dict(page_table=table, lens=pos)
    calls = [(gdn.attn_prep, "q", rows), (gdn.attn_prep_bwd, "dq_out", dict(rows, dk_out=x, q=x)),
             (gdn.attn_prep_cache, "q", dict(rows, v=x, k_cache=cache, v_cache=cache, page_table=table)),
             (gdn.attn_decode, "q", dict(pages, k_cache=cache, v_cache=cache)), (gdn.attn_page_mean, "k_cache", pages),
             (gdn.attn_select, "q", dict(pages, page_mean=torch.zeros(4, 2, 64), page_size=16, n_sel=2))]
    for call, first, others in calls:
        with pytest.raises(ValueError, match="device tensors"):
            call(**{first: cache if first == "k_cache" else x}, **others)
        with pytest.raises(TypeError, match=f"'{first}'"):
            call(**others)
