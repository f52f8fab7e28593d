"""Inputs and error bounds of the attention tests.

A paged cache is drawn with every place that no row owns set to NaN, so that a read of one shows.
The bounds count roundings: u is half a step of the output's type relative to the value, and fp32 work is
bounded by its number of sequential roundings (2^-24 each; tensor-core sums 2^-23)."""
import numpy as np
import torch

HALF_STEP = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # half of fp16's smallest step


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=g.device) * std).to(dtype)


def frequencies(rot, device="cuda", base=10000.0):
    return torch.tensor([base ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=device)


def assert_within(got, want, slack, what=""):
    """|got - want| <= u |want| + slack, elementwise (want, slack in float64)."""
    g, u = f64(got), HALF_STEP[got.dtype]
    assert g.shape == want.shape, (g.shape, want.shape)
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    over = np.abs(g - want) - (u * np.abs(want) + TINY[got.dtype] + slack)
    worst = float(over.max()) if over.size else 0.0
    assert worst <= 0.0, f"{what}: {worst:.3g} above the bound at {np.unravel_index(over.argmax(), over.shape)}"


def prep_slack(want):
    """attn_prep in fp32: the sum of squares has at most 16 + 4 sequential roundings (half of them count in r), rsqrt, the
    three products and the rotation's four operations about 12 more, cos and sin 2^-22 absolute: below 2^-18 of
    the larger of a pair, which is at most sqrt(2) times the row's largest output."""
    return 2.0 ** -18 * np.abs(want).max(axis=-1, keepdims=True)


def cache(seed, lens, Hkv, d, page, dtype, spare=3, width=None):
    """(k_cache, v_cache, page_table, lens): rows of the given lengths on shuffled pages, NaN everywhere else."""
    g = gen(seed)
    counts = [-(-n // page) for n in lens]
    num = sum(counts) + spare
    width = max(1, max(counts)) if width is None else width
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
    caches = [torch.full((num, Hkv, page, d), float("nan"), device="cuda", dtype=dtype) for _ in range(2)]
    at = 0
    for b, n in enumerate(lens):
        ids = order[at:at + counts[b]]
        at += counts[b]
        table[b, :counts[b]] = ids
        for c in caches:
            full = normal(g, counts[b], Hkv, page, d, dtype=dtype)
            if counts[b]:
                full[-1, :, n - (counts[b] - 1) * page:] = float("nan")
            c[ids.long()] = full
    return caches[0], caches[1], table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def decode_slack(q, k_cache, v_cache, lens, scale):
    """attn_decode: a score's error is at most 2^-23 (d / 16 + 16) of scale times its sum of |q k|, a weight's relative
    error twice that with m's; the weights' split leaves 2^-17 (bf16), the sums 2^-23 for each of a warp's tiles, the
    exponentials and joins a few 2^-22; all relative to the largest |v|."""
    d, n = q.shape[-1], int(lens.max()) if len(lens) else 0
    qs, ks = np.abs(f64(q)).max(), np.nanmax(np.abs(f64(k_cache)), initial=0.0)
    v = np.nanmax(np.abs(f64(v_cache)), initial=0.0)
    rows = np.sqrt((f64(q) ** 2).sum(-1).max() * np.nanmax(np.nan_to_num(f64(k_cache) ** 2).sum(-1), initial=0.0))
    reach = min(rows, qs * ks * d)  # of sum |q k|, by Cauchy-Schwarz
    return v * (4 * 2.0 ** -23 * (d / 16 + 16) * abs(scale) * reach + 2.0 ** -16 + 2.0 ** -23 * (n / 32 + 64))
