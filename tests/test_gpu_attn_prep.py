"""attn_prep, attn_prep_bwd and attn_prep_cache against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from attn_cases import assert_within, f64, frequencies, gen, normal, prep_slack
from linear_attention_token_gdn_b200 import build as gbuild
from linear_attention_token_gdn_b200 import gdn

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    gbuild.build()
    gdn.lib()


def make(seed, N, Hq, Hkv, d, dtype, fused=False):
    g = gen(seed)
    if fused:  # slices of one projection's output, with eight more channels behind
        rows = normal(g, N, (Hq + 2 * Hkv) * d + 8, dtype=dtype)
        q, k, v = (rows[:, a * d:(a + n) * d].view(N, n, d) for a, n in ((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv)))
    else:
        q, k, v = (normal(g, N, n, d, dtype=dtype) for n in (Hq, Hkv, Hkv))
    return q, k, v, normal(g, d, std=0.2), normal(g, d, std=0.2)


SHAPES = [  # N, Hq, Hkv, d, rot
    (1, 1, 1, 16, 16), (3, 4, 4, 16, 0), (33, 5, 1, 32, 16), (7, 3, 3, 64, 48), (65, 16, 2, 128, 128), (130, 12, 3, 128, 64),
    (5, 8, 8, 256, 64), (257, 2, 1, 256, 256), (2000, 20, 4, 64, 64),
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,Hq,Hkv,d,rot", SHAPES)
def test_forward(N, Hq, Hkv, d, rot, dtype):
    q, k, _, wq, wk = make(N + d, N, Hq, Hkv, d, dtype, fused=N % 2 == 1)
    pos = torch.randint(0, 1 << 20, (N,), generator=gen(1), device="cuda", dtype=torch.int32)
    f = frequencies(rot)
    got = gdn.attn_prep(q, k, wq, wk, pos, f if rot else None)
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        want = oracle.attn_prep(x, w, pos, f)
        assert y.dtype == dtype
        assert_within(y, want, prep_slack(want))


@pytest.mark.parametrize("in_dtype,out_dtype", [(F32, BF16), (BF16, F32), (F16, BF16)])
def test_forward_to_another_type(in_dtype, out_dtype):
    q, k, _, wq, wk = make(5, 19, 6, 2, 64, in_dtype)
    pos, f = torch.arange(19, device="cuda", dtype=torch.int32), frequencies(32)
    for x, w, y in zip((q, k), (wq, wk), gdn.attn_prep(q, k, wq, wk, pos, f, out_dtype=out_dtype)):
        want = oracle.attn_prep(x, w, pos, f)
        assert y.dtype == out_dtype
        assert_within(y, want, prep_slack(want))


def test_far_and_negative_positions():
    q, k, _, wq, wk = make(6, 4, 2, 2, 32, F32)
    pos = torch.tensor([2 ** 31 - 1, -(2 ** 31), -5, 12345678], dtype=torch.int32, device="cuda")
    f = torch.tensor([1.0, 0.37, 1e-3, 0.0, 3.5, 1e-9, 2.0, 0.11], dtype=torch.float64, device="cuda")
    want = oracle.attn_prep(q, wq, pos, f)
    # angles reach 7.5e9 radians: the oracle's one fp64 rounding of them and the kernel's three are 2^-53 of that each
    assert_within(gdn.attn_prep(q, k, wq, wk, pos, f)[0], want, prep_slack(want) + 4e-6 * np.abs(want).max())


def test_in_place_and_a_zero_row():
    q, k, _, wq, wk = make(7, 40, 8, 2, 128, BF16)
    q[3, 2] = 0
    pos, f = torch.arange(40, device="cuda", dtype=torch.int32), frequencies(128)
    want = gdn.attn_prep(q, k, wq, wk, pos, f)
    q2, k2 = q.clone(), k.clone()
    gdn.attn_prep(q2, k2, wq, wk, pos, f, out=(q2, k2))
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    assert not want[0][3, 2].any()


def test_no_tokens():
    q, k, _, wq, wk = make(8, 0, 4, 2, 64, BF16)
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    a, b = gdn.attn_prep(q, k, wq, wk, pos, frequencies(64))
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)
    g = gdn.attn_prep_bwd(a, b, q, k, wq, wk, pos, frequencies(64))
    assert not g["dw_q"].any() and not g["dw_k"].any()


# ---------------------------------------------------------------- gradients

def bwd_slack(dy, x, w, pos, f, dw):
    """fp32 as in prep_slack: dx is r (gn - u mean(gn u)), so its error is below 2^-18 of r (max |gn| + max |u| mean |gn u|);
    a channel of dw adds at most 64 terms in a row in fp32 (then in pairs, then in fp64), each with an error of
    2^-19 from r and the angle: below 2^-17 of the sum of their magnitudes."""
    x, w, dy = f64(x), f64(w), f64(dy)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    size = np.abs(dy).max(-1, keepdims=True) * np.sqrt(2)
    gn, u = size * (1 + np.abs(w).max()), np.abs(x * r)
    dx = 2.0 ** -18 * r * (gn + u.max(-1, keepdims=True) * gn * u.mean(-1, keepdims=True))
    return dx, 2.0 ** -17 * (size * u).sum((0, 1))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N,Hq,Hkv,d,rot", SHAPES)
def test_gradients(N, Hq, Hkv, d, rot, dtype):
    q, k, _, wq, wk = make(N + d + 1, N, Hq, Hkv, d, dtype, fused=N % 2 == 0)
    g = gen(2)
    pos = torch.randint(0, 1 << 20, (N,), generator=g, device="cuda", dtype=torch.int32)
    f = frequencies(rot)
    dq, dk = normal(g, N, Hq, d, dtype=dtype), normal(g, N, Hkv, d, dtype=dtype)
    out = gdn.attn_prep_bwd(dq, dk, q, k, wq, wk, pos, f if rot else None)
    for dy, x, w, dx, dw in ((dq, q, wq, out["dq"], out["dw_q"]), (dk, k, wk, out["dk"], out["dw_k"])):
        want_x, want_w = oracle.attn_prep_backward(dy, x, w, pos, f)
        slack_x, slack_w = bwd_slack(dy, x, w, pos, f, dw)
        assert dx.dtype == dtype and dw.dtype == F32
        assert_within(dx, want_x, slack_x, "dx")
        assert_within(dw, want_w, slack_w, "dw")


def test_gradients_from_fp32_ones_and_repeat_bits():
    q, k, _, wq, wk = make(9, 300, 16, 4, 128, BF16)
    g = gen(3)
    pos, f = torch.arange(300, device="cuda", dtype=torch.int32), frequencies(64)
    dq, dk = normal(g, 300, 16, 128), normal(g, 300, 4, 128)
    a = gdn.attn_prep_bwd(dq, dk, q, k, wq, wk, pos, f)
    want_x, want_w = oracle.attn_prep_backward(dq, q, wq, pos, f)
    slack_x, slack_w = bwd_slack(dq, q, wq, pos, f, None)
    assert_within(a["dq"], want_x, slack_x)
    assert_within(a["dw_q"], want_w, slack_w)
    b = gdn.attn_prep_bwd(dq, dk, q, k, wq, wk, pos, f)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_gradients_against_differences_of_the_forward():
    """L = sum dy * attn_prep(x): the change of L along a direction, from the kernel's own fp32 forward.  Central
    differences with step h = 2^-6 miss by h^2 / 6 times a third derivative (a few units here) and by 2^-20 / h of
    fp32 noise in outputs of size 1 to 4, over sqrt(384) random terms: 1e-2 covers both against |dL| of about 20."""
    q, k, _, wq, wk = make(10, 6, 2, 2, 32, F32)
    g = gen(4)
    pos, f = torch.arange(6, device="cuda", dtype=torch.int32), frequencies(32)
    dq, dk, along, zero = normal(g, 6, 2, 32), normal(g, 6, 2, 32), normal(g, 6, 2, 32), torch.zeros(6, 2, 32, device="cuda")
    out = gdn.attn_prep_bwd(dq, dk, q, k, wq, wk, pos, f)
    h = 2.0 ** -6
    loss = lambda a, w: (dq.double() * gdn.attn_prep(a, k, w, wk, pos, f)[0].double()).sum().item()  # noqa: E731
    slope = (loss(q + h * along, wq) - loss(q - h * along, wq)) / (2 * h)
    assert abs(slope - (out["dq"].double() * along.double()).sum().item()) < 1e-2
    dw = normal(g, 32)
    slope = (loss(q, wq + h * dw) - loss(q, wq - h * dw)) / (2 * h)
    assert abs(slope - (out["dw_q"].double() * dw.double()).sum().item()) < 1e-2
    assert not zero.any()


# ---------------------------------------------------------------- the cache

def pages_for(seed, counts, num, width):
    order = torch.randperm(num, generator=gen(seed), device="cuda").to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda")
    i = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[i:i + n]
        i += n
    return table


@pytest.mark.parametrize("d,rot,page,Hq,Hkv", [(128, 128, 16, 16, 2), (64, 32, 48, 5, 5), (256, 64, 64, 4, 1), (16, 16, 32, 3, 3)])
@pytest.mark.parametrize("in_dtype,dtype", [(BF16, BF16), (F16, F16), (F32, BF16)])
def test_cache_of_ragged_sequences(d, rot, page, Hq, Hkv, in_dtype, dtype):
    new, past = [5, 0, 1, 70], [0, 9, page - 1, 30]
    N = sum(new) + 3  # three tokens behind the last sequence
    q, k, v, wq, wk = make(d + page, N, Hq, Hkv, d, in_dtype, fused=True)
    counts = [-(-(a + n) // page) for a, n in zip(past, new)]
    num, width = sum(counts) + 2, max(counts)
    table = pages_for(3, counts, num, width)
    cu = torch.tensor([0, *np.cumsum(new)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([p for a, n in zip(past, new) for p in range(a, a + n)] + [0, 1, 2], dtype=torch.int32, device="cuda")
    f = frequencies(rot)
    kc, vc = (torch.full((num, Hkv, page, d), 7.0, device="cuda", dtype=dtype) for _ in range(2))
    q_out = torch.full((N, Hq, d), 7.0, device="cuda", dtype=dtype)
    gdn.attn_prep_cache(q, k, v, wq, wk, pos, f, kc, vc, table, cu_seqlens=cu, q_out=q_out)
    gdn.check_device_error()
    want_q, want_k = oracle.attn_prep(q, wq, pos, f), oracle.attn_prep(k, wk, pos, f)
    n = sum(new)
    assert_within(q_out[:n], want_q[:n], prep_slack(want_q[:n]))
    assert (q_out[n:] == 7).all()
    seen = torch.zeros(num, page, dtype=torch.bool, device="cuda")
    rows = [b for b, m in enumerate(new) for _ in range(m)]
    pg = torch.tensor([int(table[b, p // page]) for b, p in zip(rows, pos.tolist())], device="cuda")
    off = pos[:n].long() % page
    seen[pg, off] = True
    assert_within(kc[pg, :, off], want_k[:n], prep_slack(want_k[:n]))
    assert torch.equal(vc[pg, :, off], v[:n].to(dtype))
    for c in (kc, vc):
        assert (c.transpose(1, 2)[~seen] == 7).all()


def test_cache_decode_step_with_padding_rows():
    B, Hq, Hkv, d, page = 6, 8, 2, 128, 16
    q, k, v, wq, wk = make(11, B, Hq, Hkv, d, BF16)
    table = pages_for(4, [3] * B, 3 * B, 3)
    pos = torch.tensor([0, -1, 47, 16, -7, 15], dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((3 * B, Hkv, page, d), 7.0, device="cuda", dtype=BF16) for _ in range(2))
    q_out = torch.full((B, Hq, d), 7.0, device="cuda", dtype=BF16)
    f = frequencies(128)
    gdn.attn_prep_cache(q, k, v, wq, wk, pos, f, kc, vc, table, q_out=q_out)
    gdn.check_device_error()
    for b, p in enumerate(pos.tolist()):
        if p < 0:
            assert (q_out[b] == 7).all()
            continue
        want = oracle.attn_prep(q[b:b + 1], wq, pos[b:b + 1], f)
        assert_within(q_out[b:b + 1], want, prep_slack(want))
        assert torch.equal(vc[int(table[b, p // page]), :, p % page], v[b])
    assert int((vc != 7).any(-1).any(1).sum()) == 4  # four places written


@pytest.mark.parametrize("what", ["position", "entry", "negative entry"])
def test_cache_flags_a_place_outside(what):
    B, Hkv, d, page = 2, 2, 64, 16
    q, k, v, wq, wk = make(12, B, 4, Hkv, d, BF16)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([5, 20], dtype=torch.int32, device="cuda")
    if what == "position":
        pos[1] = 32
    else:
        table[1, 1] = 4 if what == "entry" else -1
    kc, vc = (torch.zeros(4, Hkv, page, d, device="cuda", dtype=BF16) for _ in range(2))
    gdn.attn_prep_cache(q, k, v, wq, wk, pos, frequencies(64), kc, vc, table)
    with pytest.raises(gdn.GDNError) as e:
        gdn.check_device_error()
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    assert torch.equal(vc[0, :, 5], v[0]) and not vc[1:].any() and not kc[1:].any()
    gdn.check_device_error()  # cleared


def test_cache_flags_malformed_cu_seqlens():
    q, k, v, wq, wk = make(13, 8, 2, 2, 64, BF16)
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(1, 2, 16, 64, device="cuda", dtype=BF16) for _ in range(2))
    cu = torch.tensor([3, 5, 8], dtype=torch.int32, device="cuda")  # tokens 0 to 2 are in no sequence
    gdn.attn_prep_cache(q, k, v, wq, wk, torch.arange(8, device="cuda", dtype=torch.int32), None, kc, vc, table, cu_seqlens=cu)
    with pytest.raises(gdn.GDNError):
        gdn.check_device_error()


# ---------------------------------------------------------------- streams and graphs

def test_on_another_stream_and_in_a_graph():
    q, k, _, wq, wk = make(14, 64, 16, 4, 128, BF16)
    pos, f = torch.arange(64, device="cuda", dtype=torch.int32), frequencies(128)
    want = gdn.attn_prep(q, k, wq, wk, pos, f)
    grads = gdn.attn_prep_bwd(q, k, q, k, wq, wk, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdn.attn_prep(q, k, wq, wk, pos, f, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q2 = q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = gdn.attn_prep(q2, k, wq, wk, pos, f)
        b = gdn.attn_prep_bwd(q, k, q2, k, wq, wk, pos, f)
    q2.zero_()
    q2.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    assert all(torch.equal(b[n], grads[n]) for n in grads)
