"""Cases and plain forms of the 8-bit integer operators: rows quantized to int8 with one scale
each (quantize_i8_rows), their matrix product (gemm_i8), and a paged key/value cache held in
int8 with one scale per page and head: writing it (kv8_append), reading it back (kv8_gather)
and attention over it (kv8_attention).

A case is timed through run(): with `own` false in elementary torch operations, with `own`
true through the library.

Definitions (d is held in binary32):
  rows       d = fl32(amax/127), 0 where amax < 2^-119; q = rint(x/d), ties to even, 0 where d = 0
  product    y[t,n] = a_d[t] * w_d[n] * sum_k a[t,k] w[n,k] (+ bias[n])
  append     a page's d grows to max(d_old, fl32(amax_new/127)); the codes it already holds
             become rint(q * d_old/d); a page whose first token is among the new ones starts at 0
  attention  softmax over the tokens j <= len - new + i of q_i . (d_k k_j) * scale, times d_v v_j
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = 2.0 ** -119  # amax below this: the row's (or page's) values are taken as zero


def listed():
    return [
        # one token through a 4096x4096 projection: decoding, where the launches' latency counts
        {"name": "linear_1x4096x4096", "op": "linear", "tokens": 1, "k": 4096, "n": 4096, "x": "bf16", "y": "bf16",
         "bias": False},
        # a decoding batch through the wide projection of the benchmark's layer set
        {"name": "linear_16x4096x11008", "op": "linear", "tokens": 16, "k": 4096, "n": 11008, "x": "bf16",
         "y": "bf16", "bias": False},
        # an odd batch of short prompts, rows that fill no whole 16-byte unit, binary32 and a bias
        {"name": "linear_777x11000x4099_f32", "op": "linear", "tokens": 777, "k": 11000, "n": 4099, "x": "f32",
         "y": "f32", "bias": True},
        # a long prompt through the wide projection: the tensor cores' case
        {"name": "linear_4096x4096x11008", "op": "linear", "tokens": 4096, "k": 4096, "n": 11008, "x": "bf16",
         "y": "bf16", "bias": False},
        # the product alone on rows that are quantized already, a batch of 192 decoded together
        {"name": "product_192x14336x4096", "op": "product", "tokens": 192, "k": 14336, "n": 4096, "x": "f16",
         "y": "f16", "bias": True},
        # a prompt batch written to the cache, several sequences continuing inside a page
        {"name": "append_prompts", "op": "append", "batch": 12, "new_lo": 100, "new_hi": 1500, "len_lo": 0,
         "len_hi": 300, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # one token of each of 96 sequences written to the cache: a decoding step
        {"name": "append_decode", "op": "append", "batch": 96, "new_lo": 1, "new_hi": 1, "len_lo": 1,
         "len_hi": 4000, "kv_heads": 8, "dim": 128, "page": 32, "dtype": "bf16"},
        # one short sequence, as many key heads as query heads: the smallest decoding call
        {"name": "attention_1x600_mha", "op": "attention", "batch": 1, "new_lo": 1, "new_hi": 1, "len_lo": 600,
         "len_hi": 600, "heads": 32, "kv_heads": 32, "dim": 128, "page": 64, "dtype": "bf16"},
        # a decoding batch of unequal lengths with grouped heads
        {"name": "attention_64x8000_gqa", "op": "attention", "batch": 64, "new_lo": 1, "new_hi": 1, "len_lo": 50,
         "len_hi": 8000, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # one very long sequence: few rows, the length split over the machine
        {"name": "attention_1x131000_gqa", "op": "attention", "batch": 1, "new_lo": 1, "new_hi": 1,
         "len_lo": 131000, "len_hi": 131000, "heads": 32, "kv_heads": 4, "dim": 128, "page": 32, "dtype": "f16"},
        # a few drafted tokens of each sequence checked at once, narrow heads
        {"name": "attention_24x5_drafts", "op": "attention", "batch": 24, "new_lo": 2, "new_hi": 7, "len_lo": 300,
         "len_hi": 5000, "heads": 16, "kv_heads": 8, "dim": 64, "page": 16, "dtype": "f16"},
        # two prompt chunks against what the cache already holds
        {"name": "attention_2x2000_prompts", "op": "attention", "batch": 2, "new_lo": 1600, "new_hi": 2100,
         "len_lo": 3000, "len_hi": 6500, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "product", "append", "attention", "attention", "attention"))
    if op in ("linear", "product"):
        t, n = _log(rng, 1, 4096), _log(rng, 64, 11008)
        k = _log(rng, 128, 14336)
        if rng.random() < 0.5:
            n, k = max(64, n // 64 * 64), k // 128 * 128
        t = max(1, min(t, 4096 * 4096 * 11008 // (k * n)))
        return {"op": op, "tokens": t, "k": k, "n": n, "x": rng.choice(("f32", "bf16", "bf16", "f16")),
                "y": rng.choice(("f32", "bf16", "bf16", "f16")), "bias": rng.random() < 0.4}
    kv = rng.choice((1, 2, 4, 8, 16))
    shape = {"kv_heads": kv, "dim": rng.choice((64, 128, 128)), "page": rng.choice((16, 32, 64, 128)),
             "dtype": rng.choice(("bf16", "bf16", "f16"))}
    if op == "append":
        new_hi = _log(rng, 1, 2000)
        batch = max(1, min(_log(rng, 1, 128), 12000 // new_hi))
        return {"op": op, "batch": batch, "new_lo": rng.randint(1, new_hi), "new_hi": new_hi,
                "len_lo": 0, "len_hi": _log(rng, 16, 3000), **shape}
    heads = kv * rng.choice((1, 2, 4, 5, 8))
    new_hi = rng.choice((1, 1, 1, _log(rng, 2, 16), _log(rng, 16, 2000)))
    hi = _log(rng, 64, 131000)
    most = 4.0e5 if new_hi == 1 else 6.0e4          # tokens that the batch holds in the cache
    batch = max(1, min(_log(rng, 1, 64), int(most / hi), int(2.4e8 / (hi * new_hi * heads))))
    hi = max(16, min(hi, int(6.0e8 / (batch * new_hi * heads))))
    return {"op": op, "batch": batch, "new_lo": rng.randint(1, new_hi), "new_hi": new_hi,
            "len_lo": rng.randint(1, hi), "len_hi": hi, "heads": heads, **shape}


def _lengths(case):
    """New tokens and cached tokens (before them) of each sequence; part of the case, whatever the seed."""
    r = random.Random(case["batch"] * 7919 + case["len_hi"] * 31 + case["new_hi"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    old = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    if case["op"] == "attention" and case["batch"] > 1:
        old[-1] = case["len_hi"]
    return new, old


def _quantize(x):
    """The rows' codes (in binary64: a quotient next to a half decides a code) and scales (one rounding
    of amax/127: in binary32 a device tensor over a number is a product with fl32(1/127), often an ulp off)."""
    amax = x.abs().amax(-1).float()
    d = torch.where(amax < TINY, torch.zeros_like(amax), (amax.double() / 127.0).float())
    q = torch.round(x.double() / torch.where(d > 0, d, torch.ones_like(d)).double()[..., None])
    return torch.where((d > 0)[..., None], q, torch.zeros_like(q)), d


def _pitched(codes):
    """int8 codes [rows, n] as a view of rows of a multiple of 16 bytes, zeros behind the row."""
    rows, n = codes.shape
    buf = torch.zeros(rows, -(-n // 16) * 16, dtype=torch.int8, device=codes.device)
    buf[:, :n] = codes.to(torch.int8)
    return buf[:, :n]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] in ("linear", "product"):
        t, k, n = case["tokens"], case["k"], case["n"]
        # activations with a few channels much larger than the others; weights of a trained matrix's size
        x = randn(t, k) * (1.0 + 15.0 * (torch.rand(k, generator=g, device="cuda") < 0.01))
        s["x_data"] = x.to(DTYPES[case["x"]])
        w, s["w_scales"] = _quantize(randn(n, k) * 0.02)
        s["w_codes"] = _pitched(w)
        s["bias_data"] = randn(n) * 0.1 if case["bias"] else None
        if case["op"] == "product":
            a, s["a_scales"] = _quantize(s.pop("x_data").float())
            s["a_codes"] = _pitched(a)
        return s
    new, old = _lengths(case)
    page, kv, dim = case["page"], case["kv_heads"], case["dim"]
    lens = [a + b for a, b in zip(new, old)]
    width = max(-(-m // page) for m in lens)
    pages = [-(-m // page) for m in lens]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    tables = torch.zeros(len(new), width, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(pages):
        tables[b, :m] = order[at:at + m]
        at += m
    s["tables"], s["width"] = tables, width
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    s["most_new"], s["total"] = max(new), sum(new)
    for name in ("k", "v"):
        codes = torch.empty(n_pages, kv, page, dim, dtype=torch.int8, device="cuda")
        for part in codes.split(max(1, (1 << 26) // (kv * page * dim))):
            part.copy_((randn(*part.shape) * 38.0).round().clamp(-127, 127))
        s[name + "_codes"] = codes
        s[name + "_scales"] = torch.exp(randn(n_pages, kv) * 0.15) * 0.026
    if case["op"] == "append":
        s["k_new"] = (randn(s["total"], kv, dim) * 1.05).to(DTYPES[case["dtype"]])
        s["v_new"] = (randn(s["total"], kv, dim) * 1.05).to(DTYPES[case["dtype"]])
        # what is read back: from the start of each sequence's first page that the new tokens reach
        back = [m - o // page * page for m, o in zip(lens, old)]
        s["back"] = torch.tensor([sum(back[:b]) for b in range(len(back) + 1)], dtype=torch.int32, device="cuda")
        s["total_back"] = sum(back)
    else:
        s["q_data"] = (randn(s["total"], case["heads"], dim) * 1.3).to(DTYPES[case["dtype"]])
    return s


def _own(s):
    import post_weight_quantization_rowwise_b200 as iqq
    if s["op"] == "linear":
        a, d = iqq.quantize_i8_rows(s["x_data"])
        return iqq.gemm_i8(a, d, s["w_codes"], s["w_scales"], bias=s["bias_data"], dtype=DTYPES[s["y"]])
    if s["op"] == "product":
        return iqq.gemm_i8(s["a_codes"], s["a_scales"], s["w_codes"], s["w_scales"], bias=s["bias_data"],
                           dtype=DTYPES[s["y"]])
    if "cache" not in s:  # the handle that a program keeps for its cache's tensors
        s["cache"] = iqq.Kv8Cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
    cache = s["cache"]
    if s["op"] == "append":
        iqq.iqq_kv8_append(cache, s["k_new"], s["v_new"], s["tables"], s["lens"], s["cu"])
        k, v = iqq.kv8_gather(cache, s["tables"], s["lens"], s["back"], s["total_back"], dtype=DTYPES[s["dtype"]])
        return {"k": k, "v": v, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    return iqq.kv8_attention(cache, s["q_data"], s["tables"], s["lens"], s["cu"])


def _spans(cu, lens, total):
    """Sequence and position of each row of a packed span: the last cu[b+1]-cu[b] tokens of sequence b."""
    row = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu.long(), row, right=True) - 1
    return seq, lens.long()[seq] - cu.long()[seq + 1] + row


def _plain_append(s, name):
    codes, scales, page = s[name + "_codes"], s[name + "_scales"], s["page"]
    x = s[name + "_new"].float()
    seq, pos = _spans(s["cu"], s["lens"], s["total"])
    where = s["tables"].long()[seq, pos // page]
    amax = x.abs().amax(-1)
    need = torch.where(amax < TINY, torch.zeros_like(amax), (amax.double() / 127.0).float())
    # only the first page that a sequence's new tokens reach can hold older ones
    start = s["lens"].long() - (s["cu"][1:] - s["cu"][:-1]).long()
    first = s["tables"].long().gather(1, (start // page).clamp(max=s["width"] - 1)[:, None])[:, 0]
    held = scales[first]
    grown = scales.clone()
    grown[where] = 0.0
    grown[first] = torch.where((start % page > 0)[:, None], held, grown[first])
    grown.scatter_reduce_(0, where[:, None].expand_as(need), need, "amax")
    d = grown[first]
    old = codes[first].double()
    again = torch.round(old * held.double()[..., None, None] / torch.where(d > 0, d, 1.0).double()[..., None, None])
    keep = (torch.arange(page, device=x.device)[None, :] < (start % page)[:, None])[:, None, :, None]
    codes[first] = torch.where(keep, again, old).to(torch.int8)
    dt = grown[where][..., None].double()
    codes[where, :, pos % page] = torch.where(dt > 0, torch.round(x.double() / torch.where(dt > 0, dt, 1.0)),
                                              0.0).to(torch.int8)
    scales.copy_(grown)
    seq, pos = _spans(s["back"], s["lens"], s["total_back"])
    where = s["tables"].long()[seq, pos // page]
    return (codes[where, :, pos % page].float() * scales[where][..., None]).to(s[name + "_new"].dtype)


def _plain_attention(s):
    q, page, kv, dim, most = s["q_data"].float(), s["page"], s["kv_heads"], s["dim"], s["most_new"]
    batch, heads, length = s["batch"], s["heads"], s["width"] * s["page"]
    group = heads // kv
    pages = s["tables"].long()
    lay = lambda c, d: ((c[pages].float() * d[pages][..., None, None]).permute(0, 2, 1, 3, 4)  # noqa: E731
                        .reshape(batch, kv, length, dim))
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(most, device=q.device)
    row = (s["cu"][:-1].long()[:, None] + i[None, :]).clamp(max=s["total"] - 1)
    qs = q[row].reshape(batch, most, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv, group * most, dim)
    score = torch.matmul(qs, lay(s["k_codes"], s["k_scales"]).transpose(-1, -2)) * dim ** -0.5
    score = score.reshape(batch, kv, group, most, length)
    last = (s["lens"].long() - new)[:, None] + i[None, :]
    hidden = torch.arange(length, device=q.device)[None, None, :] > last[:, :, None]
    score = score.masked_fill_(hidden[:, None, None], -math.inf)
    score = torch.exp(score.sub_(score.amax(-1, keepdim=True)))
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.reshape(batch, kv, group * most, length), lay(s["v_codes"], s["v_scales"]))
    out = out.reshape(batch, kv, group, most, dim) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(batch * most, heads, dim)
    seq, pos = _spans(s["cu"], s["lens"], s["total"])
    return out[seq * most + pos - (s["lens"].long() - new)[seq]].to(s["q_data"].dtype)


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] in ("linear", "product"):
        a, d = _quantize(s["x_data"]) if s["op"] == "linear" else (s["a_codes"], s["a_scales"])
        y = torch.matmul(a.float(), s["w_codes"].float().t()) * d[:, None] * s["w_scales"][None, :]
        if s["bias_data"] is not None:
            y = y + s["bias_data"]
        return y.to(DTYPES[s["y"]])
    if s["op"] == "append":
        k, v = _plain_append(s, "k"), _plain_append(s, "v")
        return {"k": k, "v": v, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    return _plain_attention(s)


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] in ("linear", "product"):
        t, k, n = case["tokens"], case["k"], case["n"]
        x = t * k * size[case["x"]] if case["op"] == "linear" else t * (k + 4)
        return {"bytes": x + n * (k + 4) + t * n * size[case["y"]] + (4 * n if case["bias"] else 0),
                "flops": 2.0 * t * k * n}
    new, old = _lengths(case)
    page, kv, dim = case["page"], case["kv_heads"], case["dim"]
    lens = [a + b for a, b in zip(new, old)]
    if case["op"] == "append":
        # new values in, codes out; the codes already in a reached page in (and out, when its scale
        # grows); the reached pages read back
        held = sum(o % page for o in old)
        back = sum(m - o // page * page for m, o in zip(lens, old))
        each = sum(new) * (size[case["dtype"]] + 1) + 2 * held + back * (1 + size[case["dtype"]])
        return {"bytes": 2 * each * kv * dim, "flops": 0}
    pairs = sum(n * o + n * (n + 1) // 2 for n, o in zip(new, old))
    cells = sum(-(-m // page) for m in lens)
    return {"bytes": 2 * sum(lens) * kv * dim + 8 * cells * kv + 2 * sum(new) * case["heads"] * dim
            * size[case["dtype"]], "flops": 4.0 * pairs * case["heads"] * dim}


def _rows64(x):
    """The definition's codes and scales in 64 bits (the scale is a binary32 number by definition)."""
    top = x.double().abs().max(dim=-1, keepdim=True).values
    d = (top / 127.0).to(torch.float32).double() * (top >= TINY)
    return (x.double() / d).round().nan_to_num(0.0), d


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("linear", "product"):
        a, d = _rows64(s["x_data"]) if case["op"] == "linear" else (s["a_codes"].double(),
                                                                   s["a_scales"].double()[:, None])
        y = (a @ s["w_codes"].double().mT) * (d * s["w_scales"].double())
        return y if s["bias_data"] is None else y + s["bias_data"].double()
    page, lens, cu = case["page"], s["lens"].tolist(), s["cu"].tolist()
    if case["op"] == "append":
        out = {}
        for name in ("k", "v"):
            scales, parts = s[name + "_scales"].double(), []
            for b, m in enumerate(lens):
                start, rows = m - (cu[b + 1] - cu[b]), s[name + "_new"][cu[b]:cu[b + 1]].double()
                for p in range(start // page, -(-m // page)):
                    lo, hi = max(start, p * page), min(m, (p + 1) * page)
                    cell = int(s["tables"][b, p])
                    x, was = rows[lo - start:hi - start], scales[cell] * (lo > p * page)
                    top = x.abs().amax(dim=(0, 2))
                    d = torch.maximum(was, (top / 127.0).float().double() * (top >= TINY))
                    inv = torch.where(d > 0, d, math.inf)[:, None, None]
                    held = s[name + "_codes"][cell, :, :lo - p * page].double() * was[:, None, None]
                    every = torch.cat([held, x.transpose(0, 1)], 1)
                    parts.append(((every / inv).round() * d[:, None, None]).transpose(0, 1))
                    scales[cell] = d
            out[name], out[name + "_scales"] = torch.cat(parts), scales
        return out
    if 8.0 * sum(lens) * case["kv_heads"] * case["dim"] > 2e10:
        return None
    group, outs = case["heads"] // case["kv_heads"], []
    for b, m in enumerate(lens):
        n = cu[b + 1] - cu[b]
        cells = s["tables"][b, :-(-m // page)].long()
        seen = torch.arange(m, device="cuda")[None, :] <= (m - n + torch.arange(n, device="cuda"))[:, None]
        q = s["q_data"][cu[b]:cu[b + 1]].double()
        o = torch.empty_like(q)
        for h in range(case["kv_heads"]):
            k, v = ((s[c + "_codes"][cells, h].double() * s[c + "_scales"][cells, h].double()[:, None, None])
                    .flatten(0, 1)[:m] for c in ("k", "v"))
            for e in range(h * group, (h + 1) * group):
                p = torch.softmax((q[:, e] @ k.mT / math.sqrt(case["dim"])).masked_fill(~seen, -math.inf), -1)
                o[:, e] = p @ v
        outs.append(o)
    return torch.cat(outs)
