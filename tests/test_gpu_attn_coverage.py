"""Every tile of every row counts once in attn_decode, whatever the row's length and however it is cut up.

The values of tile t (16 keys) are 1 in one channel and 0 in the others, so that channel c of the output is the weight of
the tiles t = c - 5 hk mod d alone: a tile that is lost, read twice or taken with another tile's keys moves it by
a percent, where the mean of random values would hide it.  No term has the other sign, so the bound is relative to
each output."""
import math

import numpy as np
import pytest
import torch

from attn_cases import gen
from linear_attention_token_gdn_b200 import build as gbuild
from linear_attention_token_gdn_b200 import gdn

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    gbuild.build()
    gdn.lib()


def steps(t, b):
    """Score of tile t of row b under a query of 1: eighths, exact in 16 bits."""
    return ((7 * t + 3 * b) % 16) / 8


def build_case(seed, lens, Hkv, d, page, dtype, width):
    counts = [-(-n // page) for n in lens]
    num = sum(counts) + 2
    order = torch.randperm(num, generator=gen(seed), device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(counts), width)), -1, dtype=torch.int32, device="cuda")
    kc = torch.full((num, Hkv, page, d), float("nan"), device="cuda", dtype=dtype)
    vc = kc.clone()
    i = 0
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = order[i:i + counts[b]].long()
        table[b, :counts[b]] = ids.to(torch.int32)
        i += counts[b]
        at = torch.arange(counts[b] * page, device="cuda")
        t = at // 16
        k = torch.zeros(len(at), d, device="cuda")
        k[:, 0] = steps(t, b)
        k[n:] = float("nan")
        for hk in range(Hkv):
            v = torch.zeros(len(at), d, device="cuda")
            v[at, (t + 5 * hk) % d] = 1.0
            v[n:] = float("nan")
            kc[ids, hk], vc[ids, hk] = k.view(-1, page, d).to(dtype), v.view(-1, page, d).to(dtype)
    return kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def query(b, h):
    return ((3 * h + b) % 9) / 8  # 0: equal weights


def expected(lens, Hq, Hkv, d, page, lists):
    """[B, Hq, d] in 64 bits, and the least relative change that one tile's absence makes anywhere."""
    want, least = np.zeros((len(lens), Hq, d)), math.inf
    for b, n in enumerate(lens):
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            t = np.arange(-(-n // 16))
            if lists is not None:
                listed = [p for p in lists[b][hk] if p >= 0]
                t = np.concatenate([np.arange(p * page // 16, min((p + 1) * page // 16, len(t))) for p in listed]
                                   + [np.zeros(0, int)]).astype(int)
            if len(t) == 0:
                continue
            weight = np.minimum(16, n - 16 * t) * np.exp(query(b, h) * steps(t, b))
            c = (t + 5 * hk) % d
            of_channel = np.bincount(c, weights=weight, minlength=d)
            want[b, h] = of_channel / weight.sum()
            least = min(least, float((weight / of_channel[c]).min()))
    return want, least


CASES = [  # lens, Hq, Hkv, d, page, dtype, width of the table, pages listed of each row
    ([70001], 8, 1, 128, 64, BF16, 0, 0),                       # one row over the whole GPU, joined by slices of channels
    ([131001], 16, 2, 256, 64, F16, 0, 0),
    ([50007], 40, 2, 64, 16, BF16, 0, 0),                       # groups of 20: two blocks of heads, two tiles of heads each
    ([33000], 12, 1, 32, 48, F16, 0, 0),
    ([20000, 1, 17003, 0, 9999], 64, 8, 128, 64, BF16, 0, 0),   # pieces found by pair, all channels joined together
    ([1] * 40 + [30000] + [17] * 9, 6, 2, 64, 32, F16, 0, 0),   # one long row among short ones
    ([1000 + 37 * b for b in range(20)], 16, 8, 128, 16, BF16, 0, 0),  # pieces found by CTA
    ([2000 - 61 * b for b in range(30)], 48, 3, 256, 64, F16, 0, 0),
    ([700 + 13 * b for b in range(45)], 10, 5, 32, 16, BF16, 0, 0),
    ([8 * b for b in range(64)], 16, 8, 128, 16, BF16, 0, 0),   # one CTA a pair
    ([8 * b for b in range(64)], 16, 8, 128, 16, BF16, 4000, 0),  # the same rows under a wide table: pieces
    ([256, 255, 1, 0, 129], 4, 2, 64, 64, F16, 0, 0),
    ([256, 255, 1, 0, 129], 4, 2, 64, 64, F16, 4000, 0),
    ([20000, 6401, 130000, 0], 32, 4, 128, 64, BF16, 0, 100),   # listed pages, pieces found by pair
    ([900, 5000, 17, 3000] * 12, 24, 6, 64, 16, F16, 0, 40),    # listed pages, pieces found by CTA
    ([900, 5000, 17, 3000], 8, 2, 256, 48, BF16, 0, 5),         # listed pages, one CTA a pair
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,dtype,width,n_sel", CASES)
def test_every_tile_counts_once(lens, Hq, Hkv, d, page, dtype, width, n_sel):
    """The bound, relative to each output: a weight is off by 2^-18 (the remainder's rounding in bf16) and a few 2^-22 (the
    exponent, exp2f); a warp adds T tiles by two products each, of at most four roundings of 2^-23 a product; the warps',
    pieces' and lanes' sums are below 64 roundings more, twice (numerator and denominator)."""
    kc, vc, table, ln = build_case(len(lens) + d, lens, Hkv, d, page, dtype, width)
    lists = pages = None
    if n_sel:
        g = np.random.default_rng(d)
        lists = np.full((len(lens), Hkv, n_sel), -1)
        for b, n in enumerate(lens):
            for hk in range(Hkv):
                have = g.permutation(-(-n // page))[:n_sel]
                lists[b, hk, g.permutation(n_sel)[:len(have)]] = have
        pages = torch.tensor(lists, dtype=torch.int32, device="cuda")
    q = torch.zeros(len(lens), Hq, d, device="cuda", dtype=dtype)
    for b in range(len(lens)):
        for h in range(Hq):
            q[b, h, 0] = query(b, h)
    y = gdn.attn_decode(q, kc, vc, table, ln, pages=pages, scale=1.0, y_dtype=torch.float32)
    gdn.check_device_error()
    want, least = expected(lens, Hq, Hkv, d, page, lists)
    tiles = (n_sel * page // 16 * len(lens) if n_sel else sum(-(-n // 16) for n in lens)) * Hkv * (1 + (Hq // Hkv - 1) // 16)
    of_warp = max(8, tiles // (4 * 148) + 2)                    # at least a CTA an SM; alone, a CTA has up to 32 tiles
    bound = 2.0 ** -17 + (8 * of_warp + 2 * 64) * 2.0 ** -23
    assert least > 20 * bound                                   # a tile that is lost shows in every one of its channels
    off = np.abs(y.double().cpu().numpy() - want) - bound * want
    assert (off <= 0).all(), (float(off.max()), np.unravel_index(off.argmax(), off.shape))
