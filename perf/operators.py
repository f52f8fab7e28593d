"""What the attention-side operators are timed and compared on: their cases, inputs, plain forms and 64-bit values.

A stack of gated-delta mixers keeps an attention layer between them.  The operators are that layer's parts:

* ``train``:  zero-centred RMSNorm of each query and key head with the position rotation in the same pass, and its
  gradients (inputs and norm weights);
* ``append``: the same pass for serving: queries come back, rotated keys and the values go to a paged cache;
* ``mean``:   the mean key of the cache pages that new tokens touched;
* ``decode``: attention of one new token per row over the paged cache;
* ``sparse``: pages chosen for each row and key head by the score of their mean key, then attention over these alone.

A cache is [num_pages, kv_heads, page_size, d]; a row's pages stand in its row of the page table.
``own`` selects the framework's operators; otherwise the plain torch forms run.
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 1e6  # of the rotation's frequencies: BASE ** (-2 i / rot)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # a numerics-sized training step of a small fp32 model, odd token count, every head its own keys
        {"name": "train small f32", "kind": "train", "dtype": "f32", "seqs": 1, "T": 77, "Hq": 4, "Hkv": 4, "d": 16, "rot": 16, "start": 0},
        # an ordinary training step: two sequences of 4096 tokens
        {"name": "train 2x4096", "kind": "train", "dtype": "bf16", "seqs": 2, "T": 4096, "Hq": 16, "Hkv": 4, "d": 128, "rot": 128, "start": 0},
        # a long-context training step, part of each head rotated, positions that continue far into a document
        {"name": "train 1x32768", "kind": "train", "dtype": "bf16", "seqs": 1, "T": 32768, "Hq": 32, "Hkv": 8, "d": 128, "rot": 64, "start": 950000},
        # one token for each of a few requests: launch latency
        {"name": "append 4 tokens", "kind": "append", "dtype": "bf16", "B": 4, "new_lo": 1, "new_hi": 1, "past_lo": 7, "past_hi": 999, "Hq": 16, "Hkv": 2, "d": 128, "rot": 128, "page": 16},
        # a ragged prefill of four requests, one of them in its second piece, wide heads
        {"name": "append ragged prefill", "kind": "append", "dtype": "f16", "B": 4, "new_lo": 1024, "new_hi": 8192, "past_lo": 0, "past_hi": 5000, "Hq": 16, "Hkv": 2, "d": 256, "rot": 64, "page": 64},
        # the pages touched by one new token of each request
        {"name": "mean step", "kind": "mean", "dtype": "bf16", "B": 64, "new_lo": 1, "new_hi": 1, "past_lo": 3, "past_hi": 8191, "Hkv": 8, "d": 128, "page": 64},
        # all pages of a few requests after their prefill
        {"name": "mean after prefill", "kind": "mean", "dtype": "bf16", "B": 4, "new_lo": 1024, "new_hi": 32768, "past_lo": 0, "past_hi": 0, "Hkv": 8, "d": 128, "page": 64},
        # one short request alone: latency; its length ends one key into a page
        {"name": "decode short", "kind": "decode", "dtype": "bf16", "B": 1, "len_lo": 129, "len_hi": 129, "Hq": 16, "Hkv": 2, "d": 128, "page": 16},
        # a serving batch of uneven requests, one of them without a key yet
        {"name": "decode batch", "kind": "decode", "dtype": "bf16", "B": 64, "len_lo": 0, "len_hi": 8192, "Hq": 32, "Hkv": 8, "d": 128, "page": 64},
        # one request far into a long document, wide heads
        {"name": "decode long", "kind": "decode", "dtype": "f16", "B": 1, "len_lo": 131001, "len_hi": 131001, "Hq": 16, "Hkv": 2, "d": 256, "page": 64},
        # a few long requests, 32 of about 2000 pages each
        {"name": "sparse 4 long", "kind": "sparse", "dtype": "bf16", "B": 4, "len_lo": 120000, "len_hi": 131072, "Hq": 32, "Hkv": 4, "d": 128, "page": 64, "n_sel": 32, "n_first": 1, "n_last": 2},
        # a serving batch whose shorter requests have fewer pages than are chosen
        {"name": "sparse batch", "kind": "sparse", "dtype": "f16", "B": 64, "len_lo": 1, "len_hi": 32768, "Hq": 32, "Hkv": 8, "d": 128, "page": 64, "n_sel": 64, "n_first": 1, "n_last": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["train", "append", "mean", "decode", "decode", "sparse"])
    if kind == "train":
        dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
        d = rng.choice([16, 32, 64, 128, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        most = 32768 * 40 * 128 * 2 // (SIZES[dtype] * d * (Hq + Hkv))
        T = _log(rng, 1, max(2, min(32768, most)))
        seqs = rng.randint(1, max(1, min(8, most // T)))
        return {"kind": kind, "dtype": dtype, "seqs": seqs, "T": T, "Hq": Hq, "Hkv": Hkv, "d": d,
                "rot": 16 * rng.randint(0, d // 16), "start": rng.choice([0, 0, _log(rng, 1, 1 << 20)])}
    dtype = rng.choice(["bf16", "f16"])
    d = rng.choice([32, 64, 128, 128, 256])
    page = rng.choice([16, 32, 48, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 12, 16])
    if kind in ("append", "mean"):
        B = _log(rng, 1, 256)
        hi = _log(rng, 1, max(2, min(16384, 33_000_000 // (B * Hkv * d))))
        c = {"kind": kind, "dtype": dtype, "B": B, "new_lo": rng.randint(0, hi), "new_hi": hi, "past_lo": 0, "past_hi": rng.choice([0, _log(rng, 1, 4096)]), "Hkv": Hkv, "d": d, "page": page}
        return dict(c, Hq=Hq, rot=16 * rng.randint(0, d // 16)) if kind == "append" else c
    B = _log(rng, 1, 256)
    hi = _log(rng, 1, max(2, min(131072, 250_000_000 // (B * Hkv * d))))
    c = {"kind": kind, "dtype": dtype, "B": B, "len_lo": rng.randint(0, hi), "len_hi": hi, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page}
    if kind == "sparse":
        n_first, n_last = rng.randint(0, 2), rng.randint(1, 3)
        c |= {"n_sel": n_first + n_last + _log(rng, 1, 100), "n_first": n_first, "n_last": n_last}
    return c


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, uneven and in no order, the first lo and the last hi."""
    if n == 1:
        return [hi]
    mid = [lo + int((hi - lo + 1) * (0.6180339887498949 * (b + 1) % 1.0)) for b in range(n - 2)]
    return [lo, *mid, hi]


def _lengths(c):
    """(keys before the call, new tokens) of each row."""
    if c["kind"] in ("append", "mean"):
        return _spread(c["B"], c["past_lo"], c["past_hi"])[::-1], _spread(c["B"], c["new_lo"], c["new_hi"])
    return _spread(c["B"], c["len_lo"], c["len_hi"]), [0] * c["B"]


def work(c):
    e = SIZES[c["dtype"]]
    d, Hkv = c["d"], c["Hkv"]
    if c["kind"] == "train":  # forward: x in, y out; backward: dy and x in, dx out
        n = c["seqs"] * c["T"] * (c["Hq"] + Hkv) * d
        return {"bytes": 5 * n * e, "flops": 30 * n}
    past, new = _lengths(c)
    if c["kind"] == "append":  # q, k, v in; q, k, v out
        n = sum(new) * (c["Hq"] + 2 * Hkv) * d
        return {"bytes": 2 * n * e + 4 * sum(new), "flops": 10 * n}
    p = c["page"]
    if c["kind"] == "mean":  # the keys of the touched pages in, one fp32 mean each out
        keys = sum(a + n - a // p * p for a, n in zip(past, new) if n)
        pages = sum(-(-(a + n) // p) - a // p for a, n in zip(past, new) if n)
        return {"bytes": Hkv * d * (keys * e + 4 * pages), "flops": keys * Hkv * d}
    Hq = c["Hq"]
    if c["kind"] == "decode":  # keys and values in
        return {"bytes": sum(past) * Hkv * d * 2 * e + 2 * c["B"] * Hq * d * e, "flops": 4 * sum(past) * Hq * d}
    pages = [-(-a // p) for a in past]  # the mean keys in, then the chosen pages' keys and values
    keys = sum(a if n <= c["n_sel"] else (c["n_sel"] - 1) * p + (a - (n - 1) * p) for a, n in zip(past, pages))
    return {"bytes": sum(pages) * Hkv * d * 4 + keys * Hkv * d * 2 * e + 3 * c["B"] * Hq * d * e + 4 * c["B"] * Hkv * c["n_sel"],
            "flops": 2 * sum(pages) * Hq * d + 4 * keys * Hq * d}


def _frequencies(rot, device):
    i = torch.arange(rot // 2, device=device, dtype=torch.float64)
    return BASE ** (-2 * i / rot) if rot else i


def prepare(case, seed):
    c = case
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, d, Hkv = DTYPES[c["dtype"]], c["d"], c["Hkv"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * std).to(dtype)

    s = {"case": c}
    if c["kind"] == "train":
        N = c["seqs"] * c["T"]
        s |= {"q": normal(N, c["Hq"], d), "k": normal(N, Hkv, d), "dq": normal(N, c["Hq"], d), "dk": normal(N, Hkv, d),
              "positions": (torch.arange(c["T"], device=dev, dtype=torch.int32) + c["start"]).repeat(c["seqs"])}
    if c["kind"] in ("train", "append"):
        s |= {"w_q": normal(d, std=0.1, dtype=torch.float32), "w_k": normal(d, std=0.1, dtype=torch.float32), "inv_freq": _frequencies(c["rot"], dev)}
    if c["kind"] == "train":
        return s
    past, new = _lengths(c)
    total = [a + n for a, n in zip(past, new)]
    page, counts = c["page"], [-(-t // c["page"]) for t in total]
    width = max(1, max(counts))
    num_pages = sum(counts) + 3
    order = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(c["B"], width, dtype=torch.int32, device=dev)
    used = torch.arange(width, device=dev)[None] < torch.tensor(counts, device=dev)[:, None]
    table[used] = order[:sum(counts)]
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s |= {"page_table": table, "lens": whole(total), "past": whole(past), "k_cache": normal(num_pages, Hkv, page, d)}
    if c["kind"] == "mean":
        return s | {"page_mean": torch.zeros(num_pages, Hkv, d, device=dev)}
    s["v_cache"] = normal(num_pages, Hkv, page, d)
    if c["kind"] == "append":
        N = sum(new)
        rows = torch.repeat_interleave(torch.arange(c["B"], device=dev), torch.tensor(new, device=dev))
        cu = torch.zeros(c["B"] + 1, dtype=torch.int32, device=dev)
        cu[1:] = torch.cumsum(whole(new), 0)
        positions = torch.arange(N, device=dev) - cu[rows] + s["past"][rows]
        # queries, keys and values as the three parts of one projection's output
        qkv = normal(N, c["Hq"] + 2 * Hkv, d)
        return s | {"q": qkv[:, :c["Hq"]], "k": qkv[:, c["Hq"]:c["Hq"] + Hkv], "v": qkv[:, c["Hq"] + Hkv:], "cu_seqlens": cu, "rows": rows, "positions": positions.to(torch.int32)}
    s["q"] = normal(c["B"], c["Hq"], d)
    if c["kind"] == "sparse":
        s["page_mean"] = normal(num_pages, Hkv, d, std=page ** -0.5, dtype=torch.float32)
    return s


def run(state):
    s, c = state, state["case"]
    if own:
        return _framework(s, c)
    return {"train": _train, "append": _append, "mean": _mean, "decode": _decode, "sparse": _sparse}[c["kind"]](s, c)


def _framework(s, c):
    from linear_attention_token_gdn_b200 import gdn

    if c["kind"] == "train":
        q, k = gdn.attn_prep(s["q"], s["k"], s["w_q"], s["w_k"], s["positions"], s["inv_freq"], eps=EPS)
        g = gdn.attn_prep_bwd(s["dq"], s["dk"], s["q"], s["k"], s["w_q"], s["w_k"], s["positions"], s["inv_freq"], eps=EPS)
        return q, k, g["dq"], g["dk"], g["dw_q"], g["dw_k"]
    if c["kind"] == "append":
        q = gdn.attn_prep_cache(s["q"], s["k"], s["v"], s["w_q"], s["w_k"], s["positions"], s["inv_freq"], s["k_cache"], s["v_cache"], s["page_table"],
                                cu_seqlens=s["cu_seqlens"], eps=EPS)
        return q, s["k_cache"], s["v_cache"]
    if c["kind"] == "mean":
        return gdn.attn_page_mean(s["k_cache"], s["page_table"], s["lens"], s["page_mean"], starts=s["past"])
    if c["kind"] == "decode":
        return gdn.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"])
    pages = gdn.attn_select(s["q"], s["page_mean"], s["page_table"], s["lens"], c["page"], c["n_sel"], n_first=c["n_first"], n_last=c["n_last"])
    return pages, gdn.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"], pages=pages)


# ------------------------------------------------------------------ plain forms

def _turn(positions, inv_freq):
    angle = positions.double()[:, None] * inv_freq  # in 64 bits: 2^20 radians leave few bits of a float32's angle
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _rotate(x, cos, sin):
    r = cos.shape[-1]
    a, b = x[..., :r], x[..., r:2 * r]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * r:]], -1)


def _norm_rotate(x, w, cos, sin):
    x = x.float()
    return _rotate(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (1 + w), cos, sin)


def _norm_rotate_grad(dy, x, w, cos, sin):
    dn, x = _rotate(dy.float(), cos, -sin), x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    g, unit = dn * (1 + w), x * r
    return r * (g - unit * (g * unit).mean(-1, keepdim=True)), (dn * unit).sum((0, 1))


def _train(s, c):
    dt = DTYPES[c["dtype"]]
    cos, sin = _turn(s["positions"], s["inv_freq"])
    dq, dw_q = _norm_rotate_grad(s["dq"], s["q"], s["w_q"], cos, sin)
    dk, dw_k = _norm_rotate_grad(s["dk"], s["k"], s["w_k"], cos, sin)
    return _norm_rotate(s["q"], s["w_q"], cos, sin).to(dt), _norm_rotate(s["k"], s["w_k"], cos, sin).to(dt), dq.to(dt), dk.to(dt), dw_q, dw_k


def _append(s, c):
    dt = DTYPES[c["dtype"]]
    cos, sin = _turn(s["positions"], s["inv_freq"])
    at = s["positions"].long()
    pages, places = s["page_table"][s["rows"], at // c["page"]].long(), at % c["page"]
    s["k_cache"][pages, :, places] = _norm_rotate(s["k"], s["w_k"], cos, sin).to(dt)
    s["v_cache"][pages, :, places] = s["v"]
    return _norm_rotate(s["q"], s["w_q"], cos, sin).to(dt), s["k_cache"], s["v_cache"]


def _mean(s, c):
    p = c["page"]
    at = torch.arange(s["page_table"].shape[1], device=s["lens"].device)[None] * p
    lens, past = s["lens"][:, None], s["past"][:, None]
    touched = (at < lens) & (at + p > past) & (lens > past)
    pages = s["page_table"][touched].long()
    count = (lens - at).clamp(0, p)[touched]
    inside = torch.arange(p, device=at.device)[None] < count[:, None]
    keys = torch.where(inside[:, None, :, None], s["k_cache"][pages].float(), torch.zeros((), device=at.device))
    s["page_mean"][pages] = keys.sum(2) / count[:, None, None]
    return s["page_mean"]


def _attend(q, k, v, valid):
    """q [B, Hkv, G, d]; k, v [B, Hkv, L, d] fp32; valid [B, 1 or Hkv, L].  Rows without a key give zeros."""
    score = torch.matmul(q, k.transpose(-1, -2)) * q.shape[-1] ** -0.5
    score = score.masked_fill(~valid[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    y = torch.matmul(e, v)
    return torch.where(total > 0, y / total, torch.zeros_like(y))


def _decode(s, c):
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    table = s["page_table"].long()
    k, v = (s[n][table].float().transpose(1, 2).reshape(B, Hkv, -1, d) for n in ("k_cache", "v_cache"))
    valid = torch.arange(k.shape[2], device=table.device)[None, None] < s["lens"][:, None, None]
    return _attend(s["q"].float().view(B, Hkv, -1, d), k, v, valid).view(B, c["Hq"], d).to(DTYPES[c["dtype"]])


def _choose(s, c):
    B, Hkv, d, p = c["B"], c["Hkv"], c["d"], c["page"]
    counts = (s["lens"] + p - 1) // p
    # in 64 bits: which page is the last to be chosen may hang on the last bits of two scores
    means = s["page_mean"][s["page_table"].long()].double().transpose(1, 2)
    score = torch.matmul(s["q"].double().view(B, Hkv, -1, d), means.transpose(-1, -2)).amax(2)
    at = torch.arange(score.shape[-1], device=score.device)[None]
    n = counts[:, None]
    score = score.masked_fill(((at < c["n_first"]) | (at >= n - c["n_last"]))[:, None], math.inf).masked_fill((at >= n)[:, None], -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :c["n_sel"]]
    best = torch.nn.functional.pad(best, (0, c["n_sel"] - best.shape[-1]), value=1 << 30)
    best = best.masked_fill(best >= n[:, None], 1 << 30).sort(-1).values
    return best.masked_fill(best == 1 << 30, -1).to(torch.int32)


def _sparse(s, c):
    B, Hkv, d, p = c["B"], c["Hkv"], c["d"], c["page"]
    chosen = _choose(s, c)
    logical = chosen.clamp(min=0).long()
    pages = torch.gather(s["page_table"].long()[:, None].expand(B, Hkv, -1), 2, logical)
    heads = torch.arange(Hkv, device=pages.device)[None, :, None]
    k, v = (s[n][pages, heads].float().reshape(B, Hkv, -1, d) for n in ("k_cache", "v_cache"))
    at = logical[..., None] * p + torch.arange(p, device=pages.device)
    valid = ((chosen >= 0)[..., None] & (at < s["lens"][:, None, None, None])).reshape(B, Hkv, -1)
    return chosen, _attend(s["q"].float().view(B, Hkv, -1, d), k, v, valid).view(B, c["Hq"], d).to(DTYPES[c["dtype"]])


# ------------------------------------------------------------------ the definitions in 64 bits, row by row

def exact(case, seed):
    c = case
    if c["kind"] == "append" and c["Hkv"] * c["d"] * sum(map(sum, _lengths(c))) > 80_000_000:
        return None  # whole caches in 64 bits
    s = prepare(case, seed)
    return {"train": _exact_train, "append": _exact_append, "mean": _exact_mean, "decode": _exact_attention, "sparse": _exact_attention}[c["kind"]](s, c)


def _exact_rows(x, w, turns):
    """One head at a time; each pair of channels is a complex number that the rotation multiplies."""
    out, r = torch.empty(x.shape, dtype=torch.float64, device=x.device), turns.shape[1]
    for h in range(x.shape[1]):
        row = x[:, h].double()
        row = (1 + w.double()) * row / (row.pow(2).sum(1, keepdim=True) / x.shape[2] + EPS).sqrt()
        z = torch.complex(row[:, :r].contiguous(), row[:, r:2 * r].contiguous()) * turns
        out[:, h] = torch.cat([z.real, z.imag, row[:, 2 * r:]], 1)
    return out


def _exact_grads(dy, x, w, turns):
    """The gradients as directional derivatives of the normalised row: d(x / |x|_rms) has no part along x but that of eps."""
    dx, dw, r, d = torch.empty(x.shape, dtype=torch.float64, device=x.device), torch.zeros(x.shape[2], dtype=torch.float64, device=x.device), turns.shape[1], x.shape[2]
    for h in range(x.shape[1]):
        row, top = x[:, h].double(), dy[:, h].double()
        z = torch.complex(top[:, :r].contiguous(), top[:, r:2 * r].contiguous()) * turns.conj()
        back = torch.cat([z.real, z.imag, top[:, 2 * r:]], 1)
        size = (row.pow(2).sum(1, keepdim=True) / d + EPS).sqrt()
        dw += (back * row / size).sum(0)
        back = back * (1 + w.double())
        dx[:, h] = back / size - row * (back * row).sum(1, keepdim=True) / (d * size.pow(3))
    return dx, dw


def _turns(s):
    angle = s["positions"].double().outer(s["inv_freq"])
    return torch.polar(torch.ones_like(angle), angle)


def _exact_train(s, c):
    t = _turns(s)
    dq, dw_q = _exact_grads(s["dq"], s["q"], s["w_q"], t)
    dk, dw_k = _exact_grads(s["dk"], s["k"], s["w_k"], t)
    return _exact_rows(s["q"], s["w_q"], t), _exact_rows(s["k"], s["w_k"], t), dq, dk, dw_q, dw_k


def _exact_append(s, c):
    t = _turns(s)
    q, k, v = _exact_rows(s["q"], s["w_q"], t), _exact_rows(s["k"], s["w_k"], t), s["v"].double()
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    past, new = _lengths(c)
    table, n = s["page_table"].tolist(), 0
    for b in range(c["B"]):
        at = past[b]
        while at < past[b] + new[b]:
            page, place = table[b][at // c["page"]], at % c["page"]
            m = min(c["page"] - place, past[b] + new[b] - at)
            k_cache[page, :, place:place + m] = k[n:n + m].transpose(0, 1)
            v_cache[page, :, place:place + m] = v[n:n + m].transpose(0, 1)
            at, n = at + m, n + m
    return q, k_cache, v_cache


def _exact_mean(s, c):
    out = s["page_mean"].double()
    past, new = _lengths(c)
    table = s["page_table"].tolist()
    for b in range(c["B"]):
        total = past[b] + new[b]
        for j in range(past[b] // c["page"], -(-total // c["page"])) if new[b] else ():
            out[table[b][j]] = s["k_cache"][table[b][j], :, :min(c["page"], total - j * c["page"])].double().mean(1)
    return out


def _exact_attention(s, c):
    B, Hkv, Hq, d, p = c["B"], c["Hkv"], c["Hq"], c["d"], c["page"]
    G = Hq // Hkv
    y = torch.zeros(B, Hq, d, dtype=torch.float64, device=s["q"].device)
    lens = _lengths(c)[0]
    chosen = torch.full((B, Hkv, c["n_sel"]), -1, dtype=torch.int32) if c["kind"] == "sparse" else None
    for b in range(B):
        if not lens[b]:
            continue
        n = -(-lens[b] // p)
        pages = s["page_table"][b, :n].long()
        for h in range(Hkv):
            q = s["q"][b, h * G:(h + 1) * G].double()
            if chosen is None:
                keep = list(range(n))
            else:
                score = (s["page_mean"][pages, h].double() @ q.T).max(1).values.tolist()
                rank = sorted(range(n), key=lambda j: (not (j < c["n_first"] or j >= n - c["n_last"]), 0.0 if j < c["n_first"] or j >= n - c["n_last"] else -score[j], j))
                keep = sorted(rank[:c["n_sel"]])
                chosen[b, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
            held = torch.tensor(keep, device=q.device)
            inside = (held[:, None] * p + torch.arange(p, device=q.device)).reshape(-1) < lens[b]
            k, v = (s[name][pages[held], h].reshape(-1, d)[inside].double() for name in ("k_cache", "v_cache"))
            y[b, h * G:(h + 1) * G] = torch.softmax(q @ k.T / math.sqrt(d), 1) @ v
    return y if chosen is None else (chosen.to(y.device), y)
