"""The attention operators called in ways that the documentation allows or names an error: lists that do not
fit."""
import pytest
import torch

from attn_cases import cache, gen, normal
from linear_attention_token_gdn_b200 import build as gbuild
from linear_attention_token_gdn_b200 import gdn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    gbuild.build()
    gdn.lib()


def test_an_empty_list_of_pages_is_refused():
    """[B, Hkv, 0] is a list without a place, not the absence of a list."""
    kc, vc, table, lens = cache(1, [40, 17], 2, 64, 16, BF16)
    q = normal(gen(1), 2, 4, 64, dtype=BF16)
    with pytest.raises(ValueError):
        gdn.attn_decode(q, kc, vc, table, lens, pages=torch.empty(2, 2, 0, dtype=torch.int32, device="cuda"))
    none = torch.full((2, 2, 1), -1, dtype=torch.int32, device="cuda")  # a list without a page: zeros
    assert not gdn.attn_decode(q, kc, vc, table, lens, pages=none).any()
    gdn.check_device_error()
