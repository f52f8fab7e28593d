"""Gradients of keys and their norm weights against differences of attn_prep itself."""
import pytest
import torch

from attn_cases import frequencies, gen, normal
from linear_attention_token_gdn_b200 import build as gbuild
from linear_attention_token_gdn_b200 import gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    gbuild.build()
    gdn.lib()


def test_key_gradients_against_differences_of_the_forward():
    """L = sum dk . k_out of attn_prep along a direction of k and one of w_k, by central differences of the kernel's own fp32
    forward.  With step h = 2^-6 they miss by h^2 / 6 times a third derivative (a few units here) and by 2^-20 / h of fp32
    noise in outputs of size 1 to 4, over sqrt(384) random terms: 1e-2 covers both against |dL| of about 20."""
    g = gen(6)
    q, k, dq, dk, along = (normal(g, 6, 2, 32) for _ in range(5))
    wq, wk, dw = normal(g, 32, std=0.2), normal(g, 32, std=0.2), normal(g, 32)
    pos, f = torch.arange(6, device="cuda", dtype=torch.int32), frequencies(32)
    out = gdn.attn_prep_bwd(dq, dk, q, k, wq, wk, pos, f)
    h = 2.0 ** -6
    loss = lambda x, w: (dk.double() * gdn.attn_prep(q, x, wq, w, pos, f)[1].double()).sum().item()  # noqa: E731
    slope = (loss(k + h * along, wk) - loss(k - h * along, wk)) / (2 * h)
    assert abs(slope - (out["dk"].double() * along.double()).sum().item()) < 1e-2
    slope = (loss(k, wk + h * dw) - loss(k, wk - h * dw)) / (2 * h)
    assert abs(slope - (out["dw_k"].double() * dw.double()).sum().item()) < 1e-2
