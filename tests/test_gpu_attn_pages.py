"""attn_page_mean and attn_select against the fp64 oracle, and a serving run of the attention operators together."""
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


# ---------------------------------------------------------------- mean keys

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,Hkv,page", [(128, 2, 64), (64, 3, 16), (32, 1, 48), (256, 2, 1024), (128, 1, 80)])
def test_means(d, Hkv, page, dtype):
    lengths = [0, 1, page - 1, page, page + 1, 5 * page + 7]
    kc, _, table, lens = cache(d + page, lengths, Hkv, d, page, dtype)
    for starts in (None, [0, 0, page - 2, page - 1, page, 3 * page + 5], [0, 1, 0, page, 0, 5 * page + 6]):
        mean = torch.full((kc.shape[0], Hkv, d), 7.0, device="cuda")
        out = gdn.attn_page_mean(kc, table, lens, mean, starts=None if starts is None else ints(starts))
        gdn.check_device_error()
        assert out is mean
        want = oracle.page_mean(torch.nan_to_num(kc), table, lens, np.full(mean.shape, 7.0), starts)
        # at most page roundings of a running sum, relative to the sum of |k|: the mean of |k| is below 1 at 64 keys and
        # more, and below the largest |k| < 6 always
        assert_within(mean, want, 2.0 ** -24 * (page + 8) * np.where(want == 7.0, 0.0, 6.0))


def test_means_of_many_rows_and_a_new_tensor():
    B = 333
    kc, _, table, lens = cache(5, [(29 * b) % 70 for b in range(B)], 2, 64, 16, BF16)
    mean = gdn.attn_page_mean(kc, table, lens)
    gdn.check_device_error()
    want = oracle.page_mean(torch.nan_to_num(kc), table, lens, np.zeros(mean.shape))
    assert_within(mean, want, 2.0 ** -24 * 24 * 6)


def test_means_flag_what_lies_outside():
    kc, _, table, lens = cache(6, [40, 40], 1, 64, 16, BF16, spare=0)
    table[0, 1] = kc.shape[0]
    mean = torch.zeros(kc.shape[0], 1, 64, device="cuda")
    gdn.attn_page_mean(kc, table, lens, mean)
    with pytest.raises(gdn.GDNError):
        gdn.check_device_error()
    assert mean[int(table[0, 0])].any() and mean[int(table[1, 1])].any()
    gdn.attn_page_mean(kc, table, ints([40, 49]), mean)
    with pytest.raises(gdn.GDNError):
        gdn.check_device_error()


# ---------------------------------------------------------------- choice

def select_case(seed, lengths, Hq, Hkv, d, page, dtype, width=None):
    g = gen(seed)
    counts = [-(-n // page) for n in lengths]
    num = max(1, sum(counts))
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max([1, *counts]) if width is None else width), -1, dtype=torch.int32, device="cuda")
    i = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[i:i + n]
        i += n
    return normal(g, len(lengths), Hq, d, dtype=dtype), normal(g, num, Hkv, d), table, ints(lengths)


def same_choice(q, mean, table, lens, page, n_sel, **kw):
    got = gdn.attn_select(q, mean, table, lens, page, n_sel, **kw)
    gdn.check_device_error()
    want = oracle.attn_select(q, mean, table, lens, page, n_sel, **kw)
    assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want)
    return got


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,d,page", [(16, 2, 128, 64), (4, 4, 64, 16), (40, 2, 32, 32), (9, 1, 256, 128)])
@pytest.mark.parametrize("n_sel,n_first,n_last", [(1, 0, 0), (1, 0, 1), (6, 1, 2), (64, 0, 1), (20, 20, 0)])
def test_choice(Hq, Hkv, d, page, n_sel, n_first, n_last, dtype):
    lengths = [0, 1, page * n_sel, page * n_sel + 1, 150 * page - 5, 7, 600 * page, 128 * page, 129 * page]
    case = select_case(d + n_sel, lengths, Hq, Hkv, d, page, dtype)
    same_choice(*case, page, n_sel, n_first=n_first, n_last=n_last)


def test_choice_of_many_rows_and_long_ones():
    same_choice(*select_case(1, [16 * (b % 40) for b in range(300)], 4, 2, 64, 16, BF16), 16, 5)
    same_choice(*select_case(2, [16 * 9000 - 3, 16 * 513], 2, 1, 32, 16, BF16), 16, 700, n_first=3, n_last=2)


def test_choice_among_ties():
    """Integer means and queries: scores are exact and mostly equal."""
    q, mean, table, lens = select_case(3, [16 * 400, 16 * 1100], 4, 2, 32, 16, BF16)
    q = torch.zeros_like(q)
    q[..., 0] = 1
    mean = torch.zeros_like(mean)
    mean[..., 0] = torch.randint(-1, 2, mean.shape[:2], generator=gen(4), device="cuda").float()
    mean[..., 0] = torch.where(mean[..., 0] == 0, torch.where(torch.rand(mean.shape[:2], device="cuda", generator=gen(5)) < 0.5, -0.0, 0.0),
                               mean[..., 0])  # zeros of both signs are one score
    for n_sel in (1, 64, 200, 399):
        same_choice(q, mean, table, lens, 16, n_sel)
    same_choice(q, torch.zeros_like(mean), table, lens, 16, 50, n_last=0)


def test_choice_with_scores_a_last_bit_apart():
    """Means that differ in one fp32 last place, under queries of the same sign: fp32 sums would not tell them apart."""
    q, mean, table, lens = select_case(6, [16 * 300], 2, 1, 128, 16, BF16)
    mean = torch.ones_like(mean)
    for p in range(300):
        mean[int(table[0, p]), 0, p % 128] = 1 + 2.0 ** -23 * (1 + p % 7)
    same_choice(q.abs() + 0.5, mean, table, lens, 16, 40)


def test_choice_with_infinities_and_nan():
    q, mean, table, lens = select_case(7, [16 * 40], 2, 1, 64, 16, BF16)
    q = q.abs() + 0.1
    mean[int(table[0, 3])] = float("inf")
    mean[int(table[0, 9])] = float("-inf")
    mean[int(table[0, 12])] = float("nan")
    got = gdn.attn_select(q, mean, table, lens, 16, 37, n_last=1)[0, 0].tolist()
    assert 3 in got and 9 not in got and 12 not in got
    got = gdn.attn_select(q, mean, table, lens, 16, 39, n_last=1)[0, 0].tolist()
    assert 9 in got and 12 not in got


def test_choice_flags_what_lies_outside():
    q, mean, table, lens = select_case(8, [16 * 30, 16 * 30], 2, 1, 64, 16, BF16)
    table[0, 4] = mean.shape[0]
    got = gdn.attn_select(q, mean, table, lens, 16, 29)
    with pytest.raises(gdn.GDNError):
        gdn.check_device_error()
    assert 4 not in got[0, 0].tolist()  # the page that is not there comes last
    gdn.attn_select(q, mean, table.clamp(max=mean.shape[0] - 1), ints([16 * 31, 3]), 16, 4)
    with pytest.raises(gdn.GDNError):
        gdn.check_device_error()


# ---------------------------------------------------------------- together

def test_prefill_and_decode_steps_of_a_layer():
    """A ragged prefill fills the cache; then each step takes one token per row through norm and rotation into the
    cache, keeps up the mean keys, chooses pages and attends to them.  Every stage is checked on what it got."""
    B, Hq, Hkv, d, page, n_sel = 3, 8, 2, 128, 16, 4
    prompt, steps = [37, 0, 130], 20
    counts = [-(-(n + steps) // page) for n in prompt]
    num = sum(counts) + 1
    order = torch.randperm(num, generator=gen(1), device="cuda").to(torch.int32)
    table = torch.zeros(B, max(counts), dtype=torch.int32, device="cuda")
    for b in range(B):
        table[b, :counts[b]] = order[sum(counts[:b]):sum(counts[:b + 1])]
    kc, vc = (torch.full((num, Hkv, page, d), float("nan"), device="cuda", dtype=BF16) for _ in range(2))
    mean = torch.full((num, Hkv, d), float("nan"), device="cuda")
    g, f = gen(2), frequencies(64)
    wq, wk = normal(g, d, std=0.1), normal(g, d, std=0.1)
    N = sum(prompt)
    q, k, v = (normal(g, N, h, d, dtype=BF16) for h in (Hq, Hkv, Hkv))
    pos = ints([p for n in prompt for p in range(n)])
    gdn.attn_prep_cache(q, k, v, wq, wk, pos, f, kc, vc, table, cu_seqlens=ints([0, *np.cumsum(prompt)]))
    lens = ints(prompt)
    gdn.attn_page_mean(kc, table, lens, mean)
    keys = [[oracle.attn_prep(k[sum(prompt[:b]):sum(prompt[:b + 1])], wk, pos[sum(prompt[:b]):sum(prompt[:b + 1])], f)]
            for b in range(B)]
    values = [[f64(v[sum(prompt[:b]):sum(prompt[:b + 1])])] for b in range(B)]
    seen_sparse = False
    for step in range(steps):
        q, k, v = (normal(g, B, h, d, dtype=BF16) for h in (Hq, Hkv, Hkv))
        before = lens.clone()
        lens = lens + 1
        qr = gdn.attn_prep_cache(q, k, v, wq, wk, before, f, kc, vc, table)
        gdn.attn_page_mean(kc, table, lens, mean, starts=before)
        pages = gdn.attn_select(qr, mean, table, lens, page, n_sel, n_first=1, n_last=1)
        y = gdn.attn_decode(qr, kc, vc, table, lens, pages=pages)
        dense = gdn.attn_decode(qr, kc, vc, table, lens)
        gdn.check_device_error()
        want_q, want_k = oracle.attn_prep(q, wq, before, f), oracle.attn_prep(k, wk, before, f)
        assert_within(qr, want_q, prep_slack(want_q))
        for b in range(B):
            keys[b].append(want_k[b:b + 1])
            values[b].append(f64(v[b:b + 1]))
            kb, vb = np.concatenate(keys[b]), np.concatenate(values[b])
            at = np.arange(int(lens[b]))
            held = kc[table[b, at // page].long(), :, torch.from_numpy(at % page).cuda()]
            assert_within(held, kb, prep_slack(kb))
            assert np.array_equal(f64(vc[table[b, at // page].long(), :, torch.from_numpy(at % page).cuda()]), vb)
        counts_now = [-(-int(n) // page) for n in lens]
        for b in range(B):
            for p in range(counts_now[b]):
                i, n = int(table[b, p]), min(page, int(lens[b]) - p * page)
                assert_within(mean[i], f64(kc[i, :, :n]).mean(1), 2.0 ** -24 * 24 * 6)
        clean = torch.nan_to_num(mean)
        assert np.array_equal(pages.cpu().numpy(), oracle.attn_select(qr, clean, table, lens, page, n_sel, 1, 1))
        slack = decode_slack(qr, kc, vc, lens, d ** -0.5)
        assert_within(y, oracle.attn_decode(qr, kc, vc, table, lens, pages=pages), slack)
        assert_within(dense, oracle.attn_decode(qr, kc, vc, table, lens), slack)
        seen_sparse |= any(n > n_sel for n in counts_now)
    assert seen_sparse


def test_a_whole_step_in_a_graph():
    """The step of the test above captured once, lengths advanced on the device, replayed; against eager calls."""
    B, Hq, Hkv, d, page, n_sel, steps = 2, 4, 1, 64, 16, 3, 40
    table = torch.arange(2 * 8, dtype=torch.int32, device="cuda").view(2, 8)
    g, f = gen(3), frequencies(64)
    wq, wk = normal(g, d, std=0.1), normal(g, d, std=0.1)
    tokens = [tuple(normal(g, B, h, d, dtype=F16) for h in (Hq, Hkv, Hkv)) for _ in range(steps)]

    def fresh():
        return [torch.zeros(16, Hkv, page, d, device="cuda", dtype=F16) for _ in range(2)] + [torch.zeros(16, Hkv, d, device="cuda"),
                                                                                           ints([0, 5])]

    def step(q, k, v, kc, vc, mean, lens):
        before = lens.clone()
        lens.add_(1)
        qr = gdn.attn_prep_cache(q, k, v, wq, wk, before, f, kc, vc, table)
        gdn.attn_page_mean(kc, table, lens, mean, starts=before)
        pages = gdn.attn_select(qr, mean, table, lens, page, n_sel)
        return pages, gdn.attn_decode(qr, kc, vc, table, lens, pages=pages)

    eager = fresh()
    want = [tuple(x.clone() for x in step(*t, *eager)) for t in tokens]
    held, slot = fresh(), [x.clone() for x in tokens[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*slot, *held)
    for x, y in zip(held, fresh()):
        x.copy_(y)
    for t, w in zip(tokens, want):
        for s, x in zip(slot, t):
            s.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])
    gdn.check_device_error()
