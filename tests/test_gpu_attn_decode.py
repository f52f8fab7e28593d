"""attn_decode against the fp64 oracle.  Every place of the cache that no row owns holds NaN."""
import numpy as np
import pytest
import torch

import oracle
from attn_cases import assert_within, cache, decode_slack, gen, normal
from linear_attention_token_gdn_b200 import build as gbuild
from linear_attention_token_gdn_b200 import gdn

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    gbuild.build()
    gdn.lib()


def check(q, kc, vc, table, lens, pages=None, scale=None, y_dtype=None, **kw):
    y = gdn.attn_decode(q, kc, vc, table, lens, pages=pages, scale=scale, y_dtype=y_dtype, **kw)
    gdn.check_device_error()
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    want = oracle.attn_decode(q, kc, vc, table, lens, pages=pages, scale=scale)
    assert_within(y, want, decode_slack(q, kc, vc, lens, scale))
    return y


LENS = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 200, 0, 1000]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,Hq,Hkv,page", [
    (128, 8, 1, 64), (128, 16, 2, 16), (128, 3, 3, 48), (128, 32, 2, 64), (128, 20, 1, 128), (128, 12, 1, 1024),
    (64, 4, 2, 16), (64, 18, 2, 80), (32, 5, 1, 32), (32, 16, 1, 16), (256, 8, 4, 64), (256, 16, 1, 32), (256, 1, 1, 16),
])
def test_ragged_rows(d, Hq, Hkv, page, dtype):
    kc, vc, table, lens = cache(d + Hq, LENS, Hkv, d, page, dtype)
    q = normal(gen(1), len(LENS), Hq, d, dtype=dtype)
    y = check(q, kc, vc, table, lens)
    assert not y[0].any() and not y[11].any()


@pytest.mark.parametrize("y_dtype", [F32, F16, BF16])
def test_output_types_and_scales(y_dtype):
    kc, vc, table, lens = cache(2, [40, 300], 2, 128, 16, BF16)
    q = normal(gen(2), 2, 8, 128, dtype=BF16)
    for scale in (1e-3, 0.3, -0.2, 0.0):
        assert check(q, kc, vc, table, lens, scale=scale, y_dtype=y_dtype).dtype == y_dtype


def test_one_row_split_over_all_of_the_gpu():
    kc, vc, table, lens = cache(3, [70001], 1, 128, 64, BF16)
    check(normal(gen(3), 1, 8, 128, dtype=BF16), kc, vc, table, lens)


def test_one_long_row_among_short_ones():
    lens = [1] * 40 + [30000] + [17] * 9
    kc, vc, table, lens = cache(4, lens, 2, 64, 32, F16)
    check(normal(gen(4), 50, 6, 64, dtype=F16), kc, vc, table, lens)


@pytest.mark.parametrize("B", [128, 129, 300, 700])
def test_many_rows(B):
    lens = [(37 * b) % 41 for b in range(B)]
    kc, vc, table, lens = cache(B, lens, 2, 64, 16, BF16)
    check(normal(gen(5), B, 4, 64, dtype=BF16), kc, vc, table, lens)


def test_no_row_has_a_key():
    kc, vc, table, lens = cache(6, [0] * 200, 2, 128, 16, BF16, width=4)
    y = torch.full((200, 8, 128), 3.0, device="cuda", dtype=BF16)
    gdn.attn_decode(normal(gen(6), 200, 8, 128, dtype=BF16), kc, vc, table, lens, y=y)
    gdn.check_device_error()
    assert not y.any()


def test_scores_that_rise_along_the_row_and_one_far_above():
    """The running maximum moves in every tile, and once by far more than fp32's exponent range."""
    kc, vc, table, lens = cache(7, [640, 640], 1, 64, 64, BF16)
    q = torch.ones(2, 4, 64, device="cuda", dtype=BF16)
    for b in range(2):
        for p in range(640):
            kc[int(table[b, p // 64]), 0, p % 64] = p * 0.0625
    kc[int(table[1, 5]), 0, 3] = 300.0
    y = gdn.attn_decode(q, kc, vc, table, lens, scale=1.0, y_dtype=F32)
    want = oracle.attn_decode(q, kc, vc, table, lens, scale=1.0)
    # scores up to 2560 are exact in fp32, times log2 e they are off by 2^-23 of 3700 each: weights by 2^-11, |v| < 5
    assert_within(y, want, 2 * 2.0 ** -11 * 5.0)
    assert torch.equal(y[1], vc[int(table[1, 5]), 0, 3].float().expand(4, 64))


def test_equal_keys_give_the_mean_value():
    kc, vc, table, lens = cache(8, [4097], 1, 32, 16, F16)
    q = torch.zeros(1, 2, 32, device="cuda", dtype=F16)
    check(q, kc, vc, table, lens, y_dtype=F32)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_infinities_and_nan_behind_the_length_stay_out(bad):
    kc, vc, table, lens = cache(9, [5, 33], 1, 128, 16, BF16)
    q = normal(gen(9), 2, 8, 128, dtype=BF16)
    want = gdn.attn_decode(q, kc, vc, table, lens)
    kc2, vc2 = (torch.where(c.isnan(), torch.full_like(c, bad), c) for c in (kc, vc))
    assert torch.equal(gdn.attn_decode(q, kc2, vc2, table, lens), want)


def test_minus_infinite_scores():
    kc, vc, table, lens = cache(10, [20, 20], 1, 64, 16, F16)
    q = torch.ones(2, 2, 64, device="cuda", dtype=F16)
    kc[int(table[0, 0]), 0, 4] = float("-inf")       # one key out
    for p in range(20):                                # all keys out
        kc[int(table[1, p // 16]), 0, p % 16] = float("-inf")
    y = gdn.attn_decode(q, kc, vc, table, lens)
    keep = torch.tensor([p for p in range(20) if p != 4], device="cuda")
    rows = lambda c: torch.stack([c[int(table[0, p // 16]), 0, p % 16] for p in keep.tolist()]).double()  # noqa: E731
    s = torch.softmax(q[0].double() @ rows(kc).T / 8, -1) @ rows(vc)
    assert_within(y[0], s.cpu().numpy(), 5e-4)  # decode_slack for |v| < 4 and |q| |k| < 80
    assert not y[1].any()


@pytest.mark.parametrize("what", ["entry", "negative entry", "length", "negative length"])
def test_what_lies_outside_is_skipped_and_flagged(what):
    kc, vc, table, lens = cache(11, [40, 40, 40], 2, 128, 16, BF16, spare=0)
    q = normal(gen(11), 3, 8, 128, dtype=BF16)
    want = oracle.attn_decode(q, kc, vc, table, lens)
    slack = decode_slack(q, kc, vc, lens, 128 ** -0.5)
    if what == "entry":
        table[1, 1] = kc.shape[0]
    elif what == "negative entry":
        table[1, 1] = -1
    elif what == "length":
        lens[1] = 49  # the table holds 48; the last 8 places hold NaN, so only the other rows are looked at
    else:
        lens[1] = -3
    y = gdn.attn_decode(q, kc, vc, table, lens)
    with pytest.raises(gdn.GDNError) as e:
        gdn.check_device_error()
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    assert_within(y[[0, 2]], want[[0, 2]], slack)
    if "entry" in what:  # the row without its second page
        one = oracle.attn_decode(q[1:2], kc, vc, torch.where((table[1:2] < 0) | (table[1:2] >= kc.shape[0]), 0, table[1:2]),
                                 lens[1:2], pages=np.broadcast_to([0, 2], (1, 2, 2)))
        assert_within(y[1:2], one, slack)
    if what == "negative length":
        assert not y[1].any()


# ---------------------------------------------------------------- listed pages

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(128, 16, 2, 64), (64, 24, 2, 16), (256, 8, 2, 48), (32, 3, 3, 32)])
def test_listed_pages(d, Hq, Hkv, page, dtype):
    lengths = [0, 1, page, page + 1, 7 * page - 3, 20 * page]
    kc, vc, table, lens = cache(d, lengths, Hkv, d, page, dtype)
    g = np.random.default_rng(d)
    pages = np.full((len(lengths), Hkv, 6), -1)
    for b, n in enumerate(lengths):
        for h in range(Hkv):
            have = g.permutation(-(-n // page))[:6]
            pages[b, h, g.permutation(6)[:len(have)]] = have  # in no order, -1 in between
    pages[4, 0] = -1  # a row with a length, and no page for one head
    pages = torch.tensor(pages, dtype=torch.int32, device="cuda")
    y = check(normal(gen(d), len(lengths), Hq, d, dtype=dtype), kc, vc, table, lens, pages=pages)
    assert not y[4, :Hq // Hkv].any() and y[4, Hq // Hkv:].any()


def test_all_pages_listed_is_all_of_the_row():
    kc, vc, table, lens = cache(12, [100, 1000, 333], 2, 128, 16, BF16)
    pages = torch.full((3, 2, 63), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate((100, 1000, 333)):
        m = -(-n // 16)
        pages[b, :, :m] = torch.arange(m, device="cuda")
    q = normal(gen(12), 3, 8, 128, dtype=BF16)
    dense = oracle.attn_decode(q, kc, vc, table, lens)
    assert_within(gdn.attn_decode(q, kc, vc, table, lens, pages=pages), dense, decode_slack(q, kc, vc, lens, 128 ** -0.5))
    doubled = torch.cat([pages, pages], -1)  # each twice: the weights double, the result stays
    assert_within(gdn.attn_decode(q, kc, vc, table, lens, pages=doubled), dense, decode_slack(q, kc, vc, lens, 128 ** -0.5))


def test_a_listed_page_beyond_the_row_is_flagged():
    kc, vc, table, lens = cache(13, [40], 1, 64, 16, BF16, width=5)
    pages = torch.tensor([[[0, 3, 1]]], dtype=torch.int32, device="cuda")
    q = normal(gen(13), 1, 4, 64, dtype=BF16)
    y = gdn.attn_decode(q, kc, vc, table, lens, pages=pages)
    with pytest.raises(gdn.GDNError):
        gdn.check_device_error()
    want = oracle.attn_decode(q, kc, vc, table, lens, pages=np.array([[[0, 1]]]))
    assert_within(y, want, decode_slack(q, kc, vc, lens, 0.125))


# ---------------------------------------------------------------- calls in company

def test_the_same_bits_again_whatever_the_workspace_held():
    kc, vc, table, lens = cache(14, [3000, 0, 17, 5000, 64], 4, 128, 64, BF16)
    q = normal(gen(14), 5, 16, 128, dtype=BF16)
    n = gdn.lib().gdn_attn_decode_workspace_size(16, 4, 128)
    a = gdn.attn_decode(q, kc, vc, table, lens, workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda"))
    b = gdn.attn_decode(q, kc, vc, table, lens, workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a, b)


def test_rows_that_share_pages():
    kc, vc, table, lens = cache(15, [500, 300], 2, 64, 16, F16)
    both = table[[0, 0, 1, 0]].contiguous()
    lens = torch.tensor([500, 123, 300, 500], dtype=torch.int32, device="cuda")
    q = normal(gen(15), 4, 4, 64, dtype=F16)
    check(q, kc, vc, both, lens)


def test_two_streams_at_once():
    args = [cache(16 + i, [2000 + 100 * i, 7], 2, 128, 16, BF16) for i in range(2)]
    qs = [normal(gen(30 + i), 2, 16, 128, dtype=BF16) for i in range(2)]
    want = [gdn.attn_decode(q, *a) for q, a in zip(qs, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [gdn.attn_decode(q, *a, stream=s) for q, a, s in zip(qs, args, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip(got, want))


def test_graph_replays_with_other_lengths():
    kc, vc, table, lens = cache(18, [1200, 900, 64], 2, 128, 64, BF16)
    q = normal(gen(18), 3, 8, 128, dtype=BF16)
    graph = torch.cuda.CUDAGraph()
    gdn.attn_decode(q, kc, vc, table, lens)
    with torch.cuda.graph(graph):
        y = gdn.attn_decode(q, kc, vc, table, lens)
    for other in ([1200, 900, 64], [0, 1, 63], [1, 0, 0], [700, 900, 0]):
        lens.copy_(torch.tensor(other, dtype=torch.int32))
        graph.replay()
        gdn.check_device_error()
        assert_within(y, oracle.attn_decode(q, kc, vc, table, lens), decode_slack(q, kc, vc, lens, 128 ** -0.5))


def test_a_cache_of_more_than_32_bits_of_elements():
    """2^32 + elements (9 GB) in each cache: the row's pages are the last ones and one in the middle."""
    d, page, Hkv = 128, 64, 8
    num = (1 << 32) // (d * page * Hkv) + 3
    kc, vc = (torch.empty(num, Hkv, page, d, device="cuda", dtype=BF16) for _ in range(2))
    ids = [num - 1, num // 2, num - 2]
    g = gen(19)
    for i in ids:
        kc[i], vc[i] = normal(g, Hkv, page, d, dtype=BF16), normal(g, Hkv, page, d, dtype=BF16)
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    q = normal(g, 1, 16, d, dtype=BF16)
    small = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    ks, vs = kc[ids].cpu(), vc[ids].cpu()
    y = gdn.attn_decode(q, kc, vc, table, lens)
    mean = torch.zeros(num, Hkv, d, device="cuda")
    gdn.attn_page_mean(kc, table, lens, mean)
    gdn.check_device_error()
    assert_within(y, oracle.attn_decode(q.cpu(), ks, vs, small, lens.cpu()), decode_slack(q, ks, vs, lens, d ** -0.5))
    want = oracle.page_mean(ks, small, lens.cpu(), np.zeros((3, Hkv, d)))
    assert_within(mean[ids], want, 2.0 ** -24 * 72 * 4)  # 64 + 8 roundings of sums of |k| < 4, over the count
    pages = gdn.attn_select(q, mean, table, lens, page, 2)
    assert torch.equal(pages.cpu().long(), torch.from_numpy(oracle.attn_select(q.cpu(), mean[ids].cpu(), small, lens.cpu(), page, 2)))
    # and written there: position 149 of the row
    x = normal(g, 1, 16, d, dtype=BF16)
    k, v = normal(g, 1, Hkv, d, dtype=BF16), normal(g, 1, Hkv, d, dtype=BF16)
    w = torch.zeros(d, device="cuda")
    gdn.attn_prep_cache(x, k, v, w, w, torch.tensor([149], dtype=torch.int32, device="cuda"), None, kc, vc, table)
    gdn.check_device_error()
    assert torch.equal(vc[num - 2, :, 149 - 128], v[0])
