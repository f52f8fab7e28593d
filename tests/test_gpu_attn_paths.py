"""Where the attention operators change their way of working: few keys or many, few pairs or many, long lists of pages,
far positions, launches that overlap, and the bounds-checking build."""
import types

import numpy as np
import pytest
import torch

import oracle
from attn_cases import assert_within, cache, decode_slack, f64, frequencies, gen, normal, prep_slack
from linear_attention_token_gdn_b200 import build as gbuild
from linear_attention_token_gdn_b200 import gdn

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    gbuild.build()
    gdn.lib()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# Up to 256 keys (512 from 64 pairs on) a pair is one CTA's; above, pairs are cut up, and when they are fewer than a quarter
# of the resident CTAs (592 at d = 128, 296 at d = 256) the pieces are found by pair instead of by CTA.
@pytest.mark.parametrize("B,tiles", [(1, 16), (1, 17), (31, 32), (32, 32), (33, 33), (55, 33), (56, 40), (200, 33)])
@pytest.mark.parametrize("d,Hq,dtype", [(128, 4, BF16), (256, 20, F16)])
def test_one_cta_a_pair_or_pieces(B, tiles, d, Hq, dtype):
    lengths = [0 if b % 7 == 3 else 1 + (211 * b) % (16 * tiles) for b in range(B)]
    lengths[-1] = 16 * tiles
    kc, vc, table, lens = cache(B + tiles, lengths, 2, d, 16, dtype)
    assert table.shape[1] == tiles
    q = normal(gen(B), B, Hq, d, dtype=dtype)
    y = gdn.attn_decode(q, kc, vc, table, lens)
    gdn.check_device_error()
    slack = decode_slack(q, kc, vc, lens, d ** -0.5)
    want = oracle.attn_decode(q, kc, vc, table, lens)
    assert_within(y, want, slack)
    wide = torch.cat([table, torch.full((B, 700), -1, dtype=torch.int32, device="cuda")], 1)  # room for far more keys
    split = gdn.attn_decode(q, kc, vc, wide, lens)
    gdn.check_device_error()
    assert_within(split, want, slack)


@pytest.mark.parametrize("n_sel", [3, 16, 17, 40])
def test_listed_pages_alone_or_in_pieces(n_sel):
    kc, vc, table, lens = cache(n_sel, [0, 5, 16 * n_sel, 2000], 2, 64, 16, BF16)
    pages = torch.full((4, 2, n_sel), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate((0, 5, 16 * n_sel, 2000)):
        have = min(-(-n // 16), n_sel)
        pages[b, 0, :have] = torch.arange(have, device="cuda")
        pages[b, 1, n_sel - have:] = torch.arange(have, device="cuda").flip(0)
    q = normal(gen(1), 4, 12, 64, dtype=BF16)
    y = gdn.attn_decode(q, kc, vc, table, lens, pages=pages)
    gdn.check_device_error()
    assert not y[0].any()
    assert_within(y, oracle.attn_decode(q, kc, vc, table, lens, pages=pages), decode_slack(q, kc, vc, lens, 0.125))


def test_few_keys_in_a_graph_with_other_lengths():
    kc, vc, table, lens = cache(2, [64, 33, 1], 2, 128, 16, BF16)
    q = normal(gen(2), 3, 8, 128, dtype=BF16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gdn.attn_decode(q, kc, vc, table, lens)
    for other in ([64, 33, 1], [0, 0, 0], [1, 16, 0], [17, 2, 1]):
        lens.copy_(torch.tensor(other, dtype=torch.int32))
        graph.replay()
        gdn.check_device_error()
        assert_within(y, oracle.attn_decode(q, kc, vc, table, lens), decode_slack(q, kc, vc, lens, 128 ** -0.5))


@pytest.mark.parametrize("n_sel,n_first", [(3000, 0), (2049, 5), (1, 0), (4999, 10)])
def test_choice_among_thousands_of_equal_pages(n_sel, n_first):
    """Only the last pages of the first 2048 and two behind them stand out; of the rest the first are taken."""
    n = 5000
    q = torch.ones(1, 2, 32, device="cuda", dtype=BF16)
    mean = torch.zeros(n, 1, 32, device="cuda")
    table = torch.randperm(n, generator=gen(3), device="cuda").to(torch.int32)[None]
    for p in (2047, 2048, 4500):
        mean[int(table[0, p])] = 1.0
    got = gdn.attn_select(q, mean, table, ints([16 * n - 3]), 16, n_sel, n_first=n_first, n_last=1)
    gdn.check_device_error()
    want = oracle.attn_select(q, mean, table, ints([16 * n - 3]), 16, n_sel, n_first, 1)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("Hq,Hkv", [(16, 1), (7, 7), (33, 3)])
def test_choice_keeps_no_page_back(Hq, Hkv):
    """n_first + n_last = n_sel: nothing is chosen by score, and groups of 1, 11 and 16 heads."""
    g = gen(4)
    q, mean = normal(g, 3, Hq, 64, dtype=F16), normal(g, 900, Hkv, 64)
    table = torch.randperm(900, generator=g, device="cuda").to(torch.int32).view(3, 300)
    lens = ints([16 * 300, 16 * 20, 100])
    for n_first, n_last, n_sel in ((3, 4, 7), (0, 2, 9), (5, 0, 250)):
        got = gdn.attn_select(q, mean, table, lens, 16, n_sel, n_first=n_first, n_last=n_last)
        gdn.check_device_error()
        assert np.array_equal(got.cpu().numpy(), oracle.attn_select(q, mean, table, lens, 16, n_sel, n_first, n_last))


def test_far_and_negative_positions():
    """Angles up to 2^31 radians.  Both sides round position * frequency in 64 bits, to 2^-53 of it: 2^-21 radians each, which
    moves an output by 2^-20 of its pair, within a second prep_slack."""
    pos = [0, 1, -1, 2 ** 31 - 1, 2 ** 30 + 12345, -2 ** 31, -2 ** 30 - 7, 2 ** 24 + 1, 10 ** 9]
    g, f = gen(5), frequencies(128)
    q, k = normal(g, len(pos), 6, 128), normal(g, len(pos), 2, 128)
    wq, wk = normal(g, 128, std=0.1), normal(g, 128, std=0.1)
    qo, ko = gdn.attn_prep(q, k, wq, wk, ints(pos), f)
    grads = gdn.attn_prep_bwd(q, k, q, k, wq, wk, ints(pos), f)
    gdn.check_device_error()
    for x, w, out, dx in ((q, wq, qo, grads["dq"]), (k, wk, ko, grads["dk"])):
        want = oracle.attn_prep(x, w, np.array(pos), f)
        assert_within(out, want, 2 * prep_slack(want))
        dwant, _ = oracle.attn_prep_backward(x, x, w, np.array(pos), f)
        assert_within(dx, dwant, 2.0 ** -15 * np.abs(f64(x)).max())  # 8 times the forward's bound: products of three such terms


def test_calls_that_follow_one_another_without_waiting():
    """Later kernels may start while earlier ones end: 60 steps of changing inputs in one queue give the bits that the
    same steps give one at a time."""
    B, Hq, Hkv, d, page, n_sel = 3, 8, 2, 64, 16, 20
    kc, vc, table, lens = cache(6, [3000, 900, 40], Hkv, d, page, BF16)
    mean = gdn.attn_page_mean(kc, table, lens)
    qs = [normal(gen(100 + i), B, Hq, d, dtype=BF16) for i in range(60)]
    room = torch.empty(gdn.lib().gdn_attn_decode_workspace_size(Hq, Hkv, d), dtype=torch.uint8, device="cuda")

    def step(q):
        pages = gdn.attn_select(q, mean, table, lens, page, n_sel)
        y = gdn.attn_decode(q, kc, vc, table, lens, pages=pages, workspace=room)
        return pages, y, gdn.attn_decode(q, kc, vc, table, lens, workspace=room)

    want = []
    for q in qs:
        want.append(step(q))
        torch.cuda.synchronize()
    got = [step(q) for q in qs]
    torch.cuda.synchronize()
    gdn.check_device_error()
    assert all(torch.equal(x, y) for w, g in zip(want, got) for x, y in zip(w, g))


def test_a_stream_of_another_device_is_refused():
    kc, vc, table, lens = cache(7, [5], 1, 64, 16, BF16)
    with pytest.raises(ValueError):
        gdn.attn_decode(normal(gen(7), 1, 1, 64, dtype=BF16), kc, vc, table, lens,
                        stream=types.SimpleNamespace(device=torch.device("cuda", 7)))


def test_bounds_checking_build():
    """Every operator in the build whose kernels check their indexes: no check trips, the results are the release build's."""
    gbuild.build(debug=True)
    debug = gdn.load(gdn.DEBUG_LIB_PATH)
    g, f = gen(8), frequencies(64)
    wq, wk = normal(g, 128, std=0.1), normal(g, 128, std=0.1)
    prompt = [37, 0, 700, 5]
    N = sum(prompt)
    q, k, v = (normal(g, N, h, 128, dtype=BF16) for h in (10, 2, 2))
    pos = ints([p for n in prompt for p in range(n)])
    counts = [-(-n // 16) for n in prompt]
    table = torch.zeros(4, max(counts), dtype=torch.int32, device="cuda")
    for b in range(4):
        table[b, :counts[b]] = torch.arange(sum(counts[:b]), sum(counts[:b + 1]), device="cuda")
    lens = ints(prompt)

    def run():
        kc, vc = (torch.zeros(sum(counts), 2, 16, 128, device="cuda", dtype=BF16) for _ in range(2))
        out = [*gdn.attn_prep(q, k, wq, wk, pos, f), *gdn.attn_prep_bwd(q, k, q, k, wq, wk, pos, f).values()]
        out += [gdn.attn_prep_cache(q, k, v, wq, wk, pos, f, kc, vc, table, cu_seqlens=ints([0, *np.cumsum(prompt)])), kc, vc]
        mean = gdn.attn_page_mean(kc, table, lens)
        new = q[:4].contiguous()
        pages = gdn.attn_select(new, mean, table, lens, 16, 9, n_first=1, n_last=2)
        out += [mean, pages, gdn.attn_decode(new, kc, vc, table, lens, pages=pages), gdn.attn_decode(new, kc, vc, table, lens),
                gdn.attn_decode(new, kc, vc, table[:, :3].contiguous(), lens.clamp(max=48))]
        gdn.check_device_error()
        return out

    release = run()
    with gdn.using(debug):
        checked = run()
    for a, b in zip(release, checked):
        torch.testing.assert_close(b, a, rtol=1e-6, atol=1e-6)
