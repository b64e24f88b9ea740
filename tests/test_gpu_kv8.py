"""The paged int8 key/value cache against plain forms in 64 bits.

Append: scales and codes are exact by definition (correctly rounded quotients), so they are
compared for equality, page after page.  Gather: fl(scale * code), rounded to the type once.

Attention, with u = eps/2 of the output's type: the scores' dot products round in binary32
(about head_dim + 4 roundings of terms that sum to S = sum |q k| scale, so a weight is off by
the factor exp(+-2 (D+8) 2^-24 S)), the weights are rounded to the output's type or finer
before they meet the values (a factor 1 +- u each), sums are binary32 and the result is rounded
once (u).  Hence with V = sum_j p_j |v_j|
    |out - o| <= V (u + 2 (D + 8) 2^-24 max S + (n_keys + 64) 2^-24) + u |o| (1 + u) + step.
"""
import math
import random

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
STEP = {BF16: 2.0 ** -133, F16: 2.0 ** -24}


@pytest.fixture(scope="module")
def iqq():
    import post_weight_quantization_rowwise_b200 as m
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(new):
    return _i32([sum(new[:b]) for b in range(len(new) + 1)])


class Case:
    """A cache of random codes and scales whose sequences hold lens tokens, pages in random order."""

    def __init__(self, iqq, lens, kv, dim, page, seed, spare=3):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        counts = [-(-m // page) for m in lens]
        order = list(range(sum(counts) + spare))
        random.Random(seed).shuffle(order)
        width = max(counts + [1]) + 1
        rows, at = [], 0
        for c in counts:
            rows.append(order[at:at + c] + [0] * (width - c))
            at += c
        self.spare = order[at:]
        self.tables = _i32(rows).reshape(len(lens), width)
        self.lens, self.kv, self.dim, self.page = lens, kv, dim, page
        shape = (len(order), kv, page, dim)
        k, v = (torch.randint(-127, 128, shape, generator=self.g, device="cuda").to(torch.int8) for _ in range(2))
        ks, vs = (torch.rand(shape[:2], generator=self.g, device="cuda") * 0.02 + 0.002 for _ in range(2))
        self.cache = iqq.Kv8Cache(k, v, ks, vs)

    def randn(self, *shape, dtype=F32):
        return torch.randn(*shape, generator=self.g, device="cuda").to(dtype)

    def values(self, b, which, head):
        codes, scales = ((self.cache.k_codes, self.cache.k_scales), (self.cache.v_codes, self.cache.v_scales))[which]
        cells = self.tables[b, :-(-self.lens[b] // self.page)].long()
        return (codes[cells, head].double() * scales[cells, head].double()[:, None, None]).flatten(0, 1)[:self.lens[b]]


def _append64(codes, scales, x, table, start, n, page):
    """The definition for one sequence, in place, on the CPU, in 64 bits."""
    if n == 0:
        return
    for p in range(start // page, -(-(start + n) // page)):
        lo, hi = max(start, p * page), min(start + n, (p + 1) * page)
        cell = table[p]
        new = x[lo - start:hi - start].double()
        amax = new.abs().amax((0, 2))
        held = scales[cell].double() * (lo > p * page)
        need = torch.where(amax < 2.0 ** -119, 0.0, (amax / 127).float().double())
        d = torch.maximum(held, need)
        safe = torch.where(d > 0, d, 1.0)[:, None, None]
        old = codes[cell, :, :lo - p * page].double()
        again = torch.round(old * held[:, None, None] / safe)
        codes[cell, :, :lo - p * page] = torch.where((d > held)[:, None, None], again, old).to(torch.int8)
        fresh = torch.where(d[:, None, None] > 0, torch.round(new.transpose(0, 1) / safe), 0.0)
        codes[cell, :, lo - p * page:hi - p * page] = fresh.to(torch.int8)
        scales[cell] = d.float()


def _append_and_check(iqq, c, old, new, dtype, k=None, v=None, flags=None):
    total = sum(new)
    k = c.randn(total, c.kv, c.dim, dtype=dtype) if k is None else k
    v = c.randn(total, c.kv, c.dim, dtype=dtype) * 3 if v is None else v
    want = [t.cpu().clone() for t in (c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales)]
    at, tables = 0, c.tables.tolist()
    for b, n in enumerate(new):
        for x, codes, scales in ((k, want[0], want[1]), (v, want[2], want[3])):
            _append64(codes, scales, x[at:at + n].cpu(), tables[b], old[b], n, c.page)
        at += n
    iqq.iqq_kv8_append(c.cache, k, v, c.tables, _i32([a + b for a, b in zip(old, new)]), _cu(new), flags=flags)
    for got, ref in zip((c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales), want):
        assert torch.equal(got.cpu(), ref)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("page,dim,kv", [(16, 64, 1), (32, 128, 3), (64, 128, 2), (128, 64, 2), (128, 128, 1)])
def test_append_exact(iqq, dtype, page, dim, kv):
    """Sequences that begin, continue inside a page, end on and off page borders, take nothing,
    and cross many pages; pages no new token reaches, and codes behind the last token, stay."""
    old = [0, 0, 5, page - 1, page, page + 3, 7, 2 * page + 1]
    new = [1, page, 1, 1, page, 3 * page + 5, 0, 40]
    c = Case(iqq, [a + b for a, b in zip(old, new)], kv, dim, page, page + dim)
    _append_and_check(iqq, c, old, new, dtype)


def test_append_token_after_token(iqq):
    """A page filled one token a call, its scale growing now and then."""
    c = Case(iqq, [40, 33], 2, 64, 32, 5)
    for i in range(33):
        k = c.randn(2, 2, 64) * (1.0 + (i % 5))
        _append_and_check(iqq, c, [i, i], [1, 1], F32, k=k, v=k * 2.0 ** -130 if i % 7 == 0 else k)


def test_append_strided_and_ties(iqq):
    """k and v as parts of one fused projection; values on and next to halves of the scale."""
    c = Case(iqq, [70], 2, 64, 64, 6)
    fused = c.randn(70, 8, 64, dtype=BF16)
    _append_and_check(iqq, c, [0], [70], BF16, k=fused[:, 4:6], v=fused[:, 6:8])
    half = (torch.arange(64, device="cuda") + 0.5) * 0.037
    k = half.expand(70, 2, 64).clone()
    k[:, :, 1::3] = torch.nextafter(k[:, :, 1::3], torch.zeros_like(k[:, :, 1::3]))
    k[:, :, 63] = 127 * 0.037
    _append_and_check(iqq, c, [0], [70], F32, k=k, v=-k)


def test_append_nonfinite_and_bad_indices(iqq):
    c = Case(iqq, [20, 20, 20], 2, 64, 16, 7)
    k = c.randn(6, 2, 64)
    k[0, 1, 3], k[3, 0, 0] = float("nan"), float("inf")
    before = c.cache.k_scales.clone()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    iqq.iqq_kv8_append(c.cache, k, k, c.tables, _i32([20, 20, 20]), _i32([0, 2, 4, 6]), flags=flags)
    assert int(flags.item()) == iqq.FLAG_NONFINITE_INPUT
    for b, h in ((0, 1), (1, 0)):
        assert torch.isnan(c.cache.k_scales[c.tables[b, 1], h])
    assert torch.isfinite(c.cache.k_scales[c.tables[0, 1], 0])
    # every index that is refused on the device: nothing of the cache changes
    good = (c.tables, _i32([20, 20, 20]), _i32([0, 2, 4, 6]))
    for tables, lens, cu in ((torch.full_like(c.tables, -1), *good[1:]),
                             (torch.full_like(c.tables, c.cache.n_pages), *good[1:]),
                             (good[0], _i32([1, -5, 1]), good[2]),
                             (good[0], good[1], _i32([9, 9, 12, 13])),
                             (good[0], good[1], _i32([6, 4, 2, 0])),
                             (good[0], _i32([10 ** 9] * 3), good[2])):
        state = [t.clone() for t in (c.cache.k_codes, c.cache.v_codes, c.cache.k_scales, c.cache.v_scales)]
        flags.zero_()
        x = c.randn(6, 2, 64) * 50
        iqq.iqq_kv8_append(c.cache, x, x, tables, lens, cu, flags=flags)
        assert int(flags.item()) == iqq.FLAG_BAD_INDEX, (tables, lens, cu)
        for t, was in zip((c.cache.k_codes, c.cache.v_codes, c.cache.k_scales, c.cache.v_scales), state):
            assert torch.equal(t.nan_to_num(9.0), was.nan_to_num(9.0))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("page,dim,kv", [(16, 64, 1), (64, 128, 3)])
def test_gather(iqq, dtype, page, dim, kv):
    lens = [1, 100, page, 0, 3 * page + 1]
    c = Case(iqq, lens, kv, dim, page, 8)
    for new in (lens, [1, 7, 0, 0, page + 2]):
        k = torch.full((sum(new) + 2, kv, dim), 7.0, dtype=dtype, device="cuda")
        v = k.clone()
        iqq.iqq_kv8_gather(c.cache, c.tables, _i32(lens), _cu(new), k, v)
        assert (k[-2:] == 7.0).all() and (v[-2:] == 7.0).all()  # rows behind the last sequence
        at = 0
        for b, n in enumerate(new):
            for h in range(kv):
                for which, got in ((0, k), (1, v)):
                    ref = c.values(b, which, h)[lens[b] - n:].float().to(dtype) if n else got[:0, 0]
                    assert torch.equal(got[at:at + n, h], ref)
            at += n


def _attention64(c, b, h, group, q, n, scale):
    """Outputs, lse and the error bound's parts (sum p |v|, largest sum |q k| scale) of n rows."""
    k, v = c.values(b, 0, h // group), c.values(b, 1, h // group)
    m = c.lens[b]
    last = m - n + torch.arange(n, device="cuda")
    seen = torch.arange(m, device="cuda")[None] <= last[:, None]
    s = (q.double() @ k.t()) * scale
    big = (q.double().abs() @ k.abs().t() * abs(scale)).amax(1) if m else torch.zeros(n, device="cuda").double()
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, 1) if m else torch.full((n,), -math.inf, device="cuda").double()
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p @ v, lse, p @ v.abs(), big


def _check_attention(iqq, c, new, heads, dtype, q=None, scale=None, pad=0):
    total = sum(new)
    q = c.randn(total + pad, heads, c.dim, dtype=dtype) if q is None else q
    out = torch.full((total + pad, heads, c.dim), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((total + pad, heads), 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = iqq.kv8_attention_workspace_bytes(c.cache, len(new), c.tables.shape[1], heads, total + pad)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
    iqq.iqq_kv8_attention(c.cache, q, c.tables, _i32(c.lens), _cu(new), out, lse=lse, scale=scale, workspace=ws,
                          flags=flags)
    assert int(flags.item()) == 0
    if pad:
        assert (out[total:] == 7.0).all() and (lse[total:] == 7.0).all()
    u, at = torch.finfo(dtype).eps / 2, 0
    sc = c.dim ** -0.5 if scale is None else scale
    for b, n in enumerate(new):
        for h in range(heads):
            o, l, mass, big = _attention64(c, b, h, heads // c.kv, q[at:at + n, h], n, sc)
            keys = c.lens[b]
            bound = mass * (u + 2 * (c.dim + 8) * 2.0 ** -24 * big[:, None] + (keys + 64) * 2.0 ** -24)
            # binary16 weights below 2^-14 round by an absolute 2^-25, where a row's largest is at least
            # 2^7 and a code's unit at most twice the largest value scale: 2^-25 127 2 vs / 2^7 a key
            bound = bound + keys * 127 * 2.0 ** -31 * float(c.cache.v_scales.max())
            bound = bound + u * o.abs() * (1 + u) + STEP[dtype]
            got, gl = out[at:at + n, h].double(), lse[at:at + n, h].double()
            real = torch.isfinite(q[at:at + n, h]).all(1)  # a row of q that holds an infinity or NaN gives NaN
            assert got[~real].isnan().all() and not torch.isfinite(gl[~real]).any()
            got, gl, o, l, big, bound = (t[real] for t in (got, gl, o, l, big, bound))
            assert ((got - o).abs() <= bound).all(), (b, h, float(((got - o).abs() - bound).max()))
            fine = torch.isfinite(l)
            assert torch.equal(fine, torch.isfinite(gl)) and (gl[~fine] == -math.inf).all()
            off = (gl - l).abs()[fine] - (2 * (c.dim + 8) * 2.0 ** -24 * big[fine] + (keys + 64) * 2.0 ** -24
                                          + 2.0 ** -22 * l[fine].abs())
            assert off.numel() == 0 or off.max() <= 0, float(off.max())
        at += n
    return out


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page,dim,kv,group", [(16, 64, 2, 1), (32, 128, 1, 4), (64, 128, 2, 8), (128, 64, 1, 5),
                                               (64, 64, 1, 16), (128, 128, 1, 3), (16, 128, 1, 24)])
def test_attention_one_token(iqq, dtype, page, dim, kv, group):
    """Lengths from one token, on and next to page and tile borders."""
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000, 1025]
    c = Case(iqq, lens, kv, dim, page, 11 + page)
    _check_attention(iqq, c, [1] * len(lens), kv * group, dtype, pad=1)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page,dim,kv,group", [(16, 64, 2, 1), (32, 128, 1, 4), (64, 128, 2, 2), (128, 64, 1, 5)])
def test_attention_ragged_chunks(iqq, dtype, page, dim, kv, group):
    """Chunks that are the whole sequence, its end, a few tokens, none, and longer than the
    sequence (rows that see nothing)."""
    lens = [1, 70, 300, 129, 64, 500, 257, 3, 0]
    new = [1, 70, 5, 128, 0, 33, 200, 7, 2]
    c = Case(iqq, lens, kv, dim, page, 13 + page)
    out = _check_attention(iqq, c, new, kv * group, dtype, pad=3)
    at = sum(new[:7])
    assert (out[at:at + 4] == 0).all() and (out[at + 7:at + 9] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,new,kv,group", [([9000], [1], 1, 4), ([40000], [1], 2, 8), ([5000, 3, 8111], [1, 1, 1], 1, 2),
                                               ([3000], [1500], 1, 2), ([6100], [17], 2, 4),
                                               ([30000], [60], 1, 8), ([20000, 700, 70], [100, 64, 70], 1, 1),
                                               ([9000, 0, 5], [200, 3, 9], 2, 4)])
def test_attention_long(iqq, dtype, lens, new, kv, group):
    c = Case(iqq, lens, kv, 128, 64, 17)
    _check_attention(iqq, c, new, kv * group, dtype)


def test_attention_steep_scores_and_scale(iqq):
    """Weights that one key takes almost whole, late and early, negative scale, scale 0."""
    c = Case(iqq, [400, 90], 1, 64, 32, 19)
    q = c.randn(2, 2, 64, dtype=BF16) * 8
    for scale in (1.0, -0.5, 0.0, 2.0 ** -20):
        _check_attention(iqq, c, [1, 1], 2, BF16, q=q, scale=scale)


def test_attention_scales_of_pages(iqq):
    """Pages of zeros (scale 0) and of scales many binades apart."""
    for dtype in (BF16, F16):
        c = Case(iqq, [300, 40], 2, 64, 16, 23)
        c.cache.v_scales.mul_(torch.exp2(torch.randint(-12, 1, c.cache.v_scales.shape, generator=c.g, device="cuda").float()))
        c.cache.k_scales.mul_(torch.exp2(torch.randint(-6, 2, c.cache.k_scales.shape, generator=c.g, device="cuda").float()))
        for t in (c.cache.k_scales, c.cache.v_scales):
            t[c.tables[0, 2]] = 0.0
            t[c.tables[0, 18]] = 0.0
        c.cache.v_scales[c.tables[1].long()] = 0.0
        _check_attention(iqq, c, [9, 40], 4, dtype)


def test_attention_nan_page_is_contained(iqq):
    """A page whose scale is NaN makes NaN of the rows that see it, and of no others: rows that
    end before the page, other heads, other sequences; pages behind the end are not looked at."""
    c = Case(iqq, [100, 100], 2, 64, 16, 29)
    c.cache.k_scales[c.tables[0, 4], 1] = float("nan")
    c.cache.v_scales[c.tables[0, 5], 0] = float("nan")
    c.cache.k_scales[c.spare] = float("nan")
    q = c.randn(200, 4, 64, dtype=BF16)
    out = iqq.kv8_attention(c.cache, q, c.tables, _i32([100, 100]), _i32([0, 100, 200]))
    bad = torch.isnan(out).any(2)
    want = torch.zeros_like(bad)
    want[64:100, 2:] = True
    want[80:100, :2] = True
    assert torch.equal(bad, want)


def test_attention_bad_indices_are_left_out(iqq):
    c = Case(iqq, [100, 50], 1, 64, 16, 31)
    q = c.randn(2, 2, 64, dtype=BF16)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (_i32([100, 50]), _i32([0, 1, 2]))
    good = iqq.kv8_attention(c.cache, q, c.tables, *args, flags=flags)
    assert int(flags.item()) == 0
    bad = c.tables.clone()
    bad[0, 3], bad[0, 6] = -7, 10 ** 6
    out = iqq.kv8_attention(c.cache, q, bad, *args, flags=flags)
    assert int(flags.item()) == iqq.FLAG_BAD_INDEX and torch.equal(out[1], good[1]) and torch.isfinite(out).all()
    # the pages left out are hidden: the same as the 80 other tokens alone
    flags.zero_()
    keep = torch.cat([c.tables[:1, [0, 1, 2, 4, 5]], c.tables[1:, :5]])
    short = iqq.kv8_attention(c.cache, q, keep, _i32([80, 50]), args[1])
    torch.testing.assert_close(out.float(), short.float(), rtol=2.0 ** -7, atol=1e-3)
    # a table too narrow for the length: its tokens only
    out = iqq.kv8_attention(c.cache, q, c.tables[:, :4], *args, flags=flags)
    assert int(flags.item()) == iqq.FLAG_BAD_INDEX
    short = iqq.kv8_attention(c.cache, q, c.tables, _i32([64, 50]), args[1])
    torch.testing.assert_close(out.float(), short.float(), rtol=2.0 ** -7, atol=1e-3)
    # spans out of range: their rows stay as they were
    for cu in ([0, 3, 2], [-4, 1, 2], [2, 1, 0]):
        flags.zero_()
        out = torch.full_like(q, 7.0)
        ws = torch.empty(iqq.kv8_attention_workspace_bytes(c.cache, 2, c.tables.shape[1], 2, 2), dtype=torch.uint8, device="cuda")
        iqq.iqq_kv8_attention(c.cache, q, c.tables, args[0], _i32(cu), out, workspace=ws, flags=flags)
        assert int(flags.item()) == iqq.FLAG_BAD_INDEX
        assert torch.isfinite(out).all()


def test_rows_before_the_first_sequence(iqq):
    """cu_tokens that begins above 0: the rows before belong to nobody, in append, gather and both
    forms of attention."""
    for new, lens in (([1, 1, 1], [40, 7, 130]), ([90, 60, 100], [90, 200, 140])):
        c = Case(iqq, lens, 2, 64, 16, 51)
        skip, total = 40, 40 + sum(new)
        cu = _cu(new) + skip
        k = c.randn(total, 2, 64)
        want = [t.cpu().clone() for t in (c.cache.k_codes, c.cache.k_scales)]
        at = skip
        for b, n in enumerate(new):
            _append64(want[0], want[1], k[at:at + n].cpu(), c.tables[b].tolist(), lens[b] - n, n, 16)
            at += n
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        iqq.iqq_kv8_append(c.cache, k, k, c.tables, _i32(lens), cu, flags=flags)
        assert torch.equal(c.cache.k_codes.cpu(), want[0]) and torch.equal(c.cache.k_scales.cpu(), want[1])
        ko = torch.full((total, 2, 64), 7.0, device="cuda")
        iqq.iqq_kv8_gather(c.cache, c.tables, _i32(lens), cu, ko, ko.clone(), flags=flags)
        assert (ko[:skip] == 7.0).all() and torch.equal(ko[skip], c.values(0, 0, 0).float()[lens[0] - new[0]].new_tensor(
            torch.stack([c.values(0, 0, h).float()[lens[0] - new[0]] for h in range(2)]).tolist()))
        q = c.randn(total, 4, 64, dtype=BF16)
        out = torch.full_like(q, 7.0)
        need = iqq.kv8_attention_workspace_bytes(c.cache, 3, c.tables.shape[1], 4, total)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        iqq.iqq_kv8_attention(c.cache, q, c.tables, _i32(lens), cu, out, workspace=ws, flags=flags)
        ref = iqq.kv8_attention(c.cache, q[skip:].contiguous(), c.tables, _i32(lens), _cu(new))
        assert (out[:skip] == 7.0).all() and int(flags.item()) == 0
        torch.testing.assert_close(out[skip:].float(), ref.float(), rtol=2.0 ** -7, atol=2e-3)


def test_attention_rows_without_a_maximum_beside_rising_scores(iqq):
    """A prompt whose first pages are left out: some rows never see a key, beside rows whose scores
    rise steeply from tile to tile."""
    c = Case(iqq, [900], 1, 128, 64, 53)
    c.cache.k_scales.fill_(0.02)
    c.cache.k_codes[c.tables[0, :15].long()] = (torch.arange(15, device="cuda") * 8)[:, None, None, None].to(torch.int8)
    q = torch.full((880, 1, 128), 4.0, device="cuda").to(BF16)
    bad = c.tables.clone()
    bad[0, :4] = -1
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = iqq.kv8_attention(c.cache, q, bad, _i32([900]), _i32([0, 880]), flags=flags)
    assert int(flags.item()) == iqq.FLAG_BAD_INDEX
    k, v = c.values(0, 0, 0), c.values(0, 1, 0)
    s = (q[:, 0].double() @ k.t()) * 128 ** -0.5
    seen = torch.arange(900, device="cuda")[None] <= 20 + torch.arange(880, device="cuda")[:, None]
    seen[:, :256] = False
    p = torch.softmax(s.masked_fill(~seen, -math.inf), 1).nan_to_num(0.0)
    ref, mass = p @ v, p @ v.abs()
    # scores of one page are equal, so weights are equal up to binary32 and binary16 roundings
    bound = mass * (2.0 ** -8 + 2.0 ** -10) + 2.0 ** -8 * ref.abs() + 2.0 ** -133
    assert (out[:236] == 0).all()
    assert ((out[:, 0].double() - ref).abs() <= bound).all()


def test_attention_largest_and_smallest_q(iqq):
    """Rows of q at the ends of bfloat16's range: the scores, brought back by the scale, are ordinary.
    A drawn 4 times 2^126 is an infinity, whose row alone is NaN."""
    c = Case(iqq, [200, 90], 1, 64, 16, 57)
    for size in (2.0 ** 126, 2.0 ** -126):
        base = c.randn(91, 2, 64, dtype=BF16)
        q = (base.double() * size).to(BF16)
        scale = 0.125 / size
        if not 2.0 ** -126 <= scale <= 2.0 ** 127:
            scale = 2.0 ** -126
        _check_attention(iqq, c, [1, 90], 2, BF16, q=q, scale=scale)


def test_attention_strided_q_and_offsets_past_32_bits(iqq):
    """q as part of a fused projection; a cache larger than 4 GiB, its last pages in use."""
    kv, dim, page = 8, 128, 128
    n_pages = (1 << 32) // (kv * dim * page) + 40
    codes = torch.zeros(2, n_pages, kv, page, dim, dtype=torch.int8, device="cuda")
    tail = torch.randint(-127, 128, (2, 40, kv, page, dim), dtype=torch.int8, device="cuda")
    codes[:, -40:] = tail
    scales = torch.full((n_pages, kv), 0.01, device="cuda")
    big = iqq.Kv8Cache(codes[0], codes[1], scales, scales.clone())
    small = iqq.Kv8Cache(tail[0].contiguous(), tail[1].contiguous(), scales[-40:].clone(), scales[-40:].clone())
    fused = torch.randn(3, 24, dim, device="cuda").to(BF16)
    q, tables = fused[:, 8:24], torch.randperm(40, device="cuda")[:36].reshape(3, 12).to(torch.int32)
    lens, cu = _i32([1500, 1, 700]), _i32([0, 1, 2, 3])
    a = iqq.kv8_attention(big, q, tables + (n_pages - 40), lens, cu)
    b = iqq.kv8_attention(small, q.contiguous(), tables, lens, cu)
    assert torch.equal(a, b)
    k, v = torch.randn(3, kv, dim, device="cuda"), torch.randn(3, kv, dim, device="cuda")
    iqq.iqq_kv8_append(big, k, v, tables + (n_pages - 40), lens, cu)
    iqq.iqq_kv8_append(small, k, v, tables, lens, cu)
    assert torch.equal(big.k_codes[-40:], small.k_codes) and torch.equal(big.v_codes[-40:], small.v_codes)
    ka, va = iqq.kv8_gather(big, tables + (n_pages - 40), lens, _cu([1500, 1, 700]), 2201)
    kb, vb = iqq.kv8_gather(small, tables, lens, _cu([1500, 1, 700]), 2201)
    assert torch.equal(ka, kb) and torch.equal(va, vb)


def test_append_then_attend_as_a_model_does(iqq):
    """A prompt and decoding steps through append and attention, captured as a graph with its
    lengths on the device: each step's output against the values the cache then holds."""
    kv, heads, dim, page = 2, 8, 128, 32
    c = Case(iqq, [0, 0], kv, dim, page, 37, spare=20)
    c.tables = _i32([c.spare[:8], c.spare[8:16]])
    prompt = [45, 70]
    k, v = c.randn(115, kv, dim, dtype=BF16), c.randn(115, kv, dim, dtype=BF16)
    iqq.iqq_kv8_append(c.cache, k, v, c.tables, _i32(prompt), _cu(prompt))
    c.lens = prompt
    _check_attention(iqq, c, prompt, heads, BF16)
    lens, cu = _i32(prompt), _i32([0, 1, 2])
    k1, v1, q1 = (torch.zeros(2, n, dim, dtype=BF16, device="cuda") for n in (kv, kv, heads))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens += 1
        iqq.iqq_kv8_append(c.cache, k1, v1, c.tables, lens, cu)
        out = iqq.kv8_attention(c.cache, q1, c.tables, lens, cu)
    for step in range(40):
        for t in (k1, v1, q1):
            t.copy_(c.randn(*t.shape))
        graph.replay()
        c.lens = [m + step + 1 for m in prompt]
        assert lens.tolist() == c.lens
        eager = _check_attention(iqq, c, [1, 1], heads, BF16, q=q1)
        assert torch.equal(out, eager)


def test_attention_on_two_streams_at_once(iqq):
    """Two calls on two streams, each with its own workspace, give what each gives alone."""
    a, b = Case(iqq, [30000], 2, 128, 64, 41), Case(iqq, [20000, 9000], 2, 128, 64, 43)
    qa, qb = a.randn(1, 8, 128, dtype=F16), b.randn(2, 8, 128, dtype=F16)
    args_a, args_b = (a.tables, _i32(a.lens), _i32([0, 1])), (b.tables, _i32(b.lens), _i32([0, 1, 2]))
    alone = iqq.kv8_attention(a.cache, qa, *args_a), iqq.kv8_attention(b.cache, qb, *args_b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        x = iqq.kv8_attention(a.cache, qa, *args_a, stream=s1)
        y = iqq.kv8_attention(b.cache, qb, *args_b, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(x, alone[0]) and torch.equal(y, alone[1])


def test_attention_prompts_beside_single_tokens(iqq):
    """One call that holds whole prompts, chunks, drafts, single tokens and idle sequences."""
    lens = [700, 33, 2000, 1, 260, 0, 90, 5000]
    for new in ([700, 1, 1, 1, 4, 0, 0, 130], [1, 1, 1, 1, 3, 0, 2, 1], [40, 1, 300, 1, 1, 0, 90, 1]):
        c = Case(iqq, lens, 2, 128, 32, 61)
        _check_attention(iqq, c, new, 8, BF16, pad=2)


@pytest.mark.parametrize("count", [33, 200, 1100])
def test_many_sequences(iqq, count):
    """More sequences than a warp's lanes, its square and a launch's CTAs; append, gather, attention."""
    rng = random.Random(count)
    lens = [rng.choice([0, 1, 5, 16, 17, 40]) for _ in range(count)]
    new = [min(m, rng.choice([0, 1, 1, 2])) for m in lens]
    c = Case(iqq, lens, 1, 64, 16, 63)
    k = c.randn(sum(new), 1, 64)
    want = [t.cpu().clone() for t in (c.cache.k_codes, c.cache.k_scales)]
    at = 0
    for b, n in enumerate(new):
        _append64(want[0], want[1], k[at:at + n].cpu(), c.tables[b].tolist(), lens[b] - n, n, 16)
        at += n
    iqq.iqq_kv8_append(c.cache, k, k, c.tables, _i32(lens), _cu(new))
    assert torch.equal(c.cache.k_codes.cpu(), want[0]) and torch.equal(c.cache.k_scales.cpu(), want[1])
    ko, vo = iqq.kv8_gather(c.cache, c.tables, _i32(lens), _cu(new), sum(new), dtype=F32)
    at = 0
    for b, n in enumerate(new):
        assert torch.equal(ko[at:at + n, 0], c.values(b, 0, 0)[lens[b] - n:].float())
        assert torch.equal(vo[at:at + n, 0], c.values(b, 1, 0)[lens[b] - n:].float())
        at += n
    _check_attention(iqq, c, new, 2, F16)


@pytest.mark.parametrize("kv,group,new", [(1, 64, [1, 2]), (1, 71, [1, 1]), (2, 33, [9, 1]), (1, 300, [2, 3])])
def test_attention_large_groups(iqq, kv, group, new):
    c = Case(iqq, [150, 77], kv, 64, 16, 67)
    _check_attention(iqq, c, new, kv * group, BF16)


def test_attention_shared_pages_and_lowest_codes(iqq):
    """Two sequences whose first pages are the same, and codes of -128."""
    c = Case(iqq, [300, 290], 1, 128, 16, 71)
    c.tables[1, :12] = c.tables[0, :12]
    c.cache.k_codes[c.tables[0, 3].long(), :, 5] = -128
    c.cache.v_codes[c.tables[0, 7].long(), :, :, ::3] = -128
    for new in ([1, 1], [200, 280]):
        _check_attention(iqq, c, new, 4, BF16)


def test_captured_prompts_with_split_keys(iqq):
    """A long chunk whose keys are split, captured and replayed on new q, lengths and pages."""
    c = Case(iqq, [9000], 1, 128, 64, 73)
    q, lens, cu = torch.zeros(100, 8, 128, dtype=BF16, device="cuda"), _i32([9000]), _i32([0, 100])
    assert iqq.kv8_attention_workspace_bytes(c.cache, 1, c.tables.shape[1], 8, 100) > 0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = iqq.kv8_attention(c.cache, q, c.tables, lens, cu)
    for m in (9000, 100, 4321):
        q.copy_(c.randn(100, 8, 128))
        lens.fill_(m)
        c.tables[0, :140] = c.tables[0, torch.randperm(140, device="cuda")]
        c.lens = [m]
        graph.replay()
        assert torch.equal(out, _check_attention(iqq, c, [100], 8, BF16, q=q))


def test_attention_smallest_and_largest_value_scales(iqq):
    """Pages whose value scales are all near 2^-87, or near 2^93: denominators and outputs stay finite."""
    for size in (2.0 ** -80, 2.0 ** 100):
        for new in ([1, 3], [300, 64]):
            c = Case(iqq, [3000, 500], 1, 64, 64, 79)
            c.cache.v_scales.mul_(size)
            _check_attention(iqq, c, new, 4, BF16, scale=1.0)


def test_captured_tokens_over_long_and_short_tables(iqq):
    """Single tokens, captured over tables wider than the lengths (shares of stages) and as narrow as
    they (a tile a CTA), replayed on new q and lengths: the same values as uncaptured, within the
    bounds both ways."""
    c = Case(iqq, [4000, 900, 1000], 2, 128, 64, 83)
    q, lens, cu = torch.zeros(3, 8, 128, dtype=F16, device="cuda"), _i32(c.lens), _cu([1, 1, 1])
    short = c.tables[:, :16]
    assert iqq.kv8_attention_workspace_bytes(c.cache, 3, c.tables.shape[1], 8, 3) > 0
    assert iqq.kv8_attention_workspace_bytes(c.cache, 3, 16, 8, 3) == 0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wide = iqq.kv8_attention(c.cache, q, c.tables, lens, cu)
        narrow = iqq.kv8_attention(c.cache, q, short, lens, cu)
    full = c.tables
    for m in ([1000, 900, 1000], [1, 0, 130], [1024, 63, 64]):
        q.copy_(c.randn(3, 8, 128))
        lens.copy_(_i32(m))
        graph.replay()
        c.lens = m
        for tables, out in ((full, wide), (short, narrow)):
            c.tables = tables
            assert torch.equal(out, _check_attention(iqq, c, [1, 1, 1], 8, F16, q=q))


@pytest.mark.parametrize("lens,new", [([1], [1]), ([200, 90, 1], [1, 1, 1]), ([5000], [1]), ([300, 4], [3, 2]),
                                      ([260, 1], [260, 1]), ([9000], [100])])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_rows_whose_scores_are_all_minus_infinity(iqq, lens, new, dim):
    """Keys of one sign, so that an infinity in q, or products beyond binary32, give every visible score
    the value -Inf: the softmax of such a row is NaN, and so is its log-sum; zeros and -Inf belong to
    rows that see nothing.  Every form of the launch: whole tiles, shares, prompts, split keys."""
    c = Case(iqq, lens, 1, dim, 64, 91)
    c.cache.k_codes.clamp_(min=1)
    q = c.randn(sum(new), 4, dim, dtype=BF16)
    q[:, 1, 5] = -math.inf
    q[:, 2] = -3.0e38
    c.cache.k_scales.mul_(64.0)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    need = iqq.kv8_attention_workspace_bytes(c.cache, len(new), c.tables.shape[1], 4, sum(new))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    iqq.iqq_kv8_attention(c.cache, q, c.tables, _i32(lens), _cu(new), out, lse=lse, workspace=ws, scale=4.0)
    assert out[:, 1:3].isnan().all() and lse[:, 1:3].isnan().all()
    assert torch.isfinite(out[:, ::3]).all() and torch.isfinite(lse[:, ::3]).all()


def test_attention_rows_that_see_nothing_with_infinities(iqq):
    """More rows than tokens, q infinite: the rows that see no token give zeros and -Inf all the same,
    and so do rows whose only pages have no place."""
    for lens, new in (([2, 70], [4, 3]), ([30, 40], [90, 200])):
        c = Case(iqq, lens, 1, 64, 16, 93)
        c.cache.k_codes.clamp_(min=1)
        q = torch.full((sum(new), 2, 64), -math.inf, device="cuda").to(BF16)
        lse = torch.zeros(sum(new), 2, device="cuda")
        out = iqq.kv8_attention(c.cache, q, c.tables, _i32(lens), _cu(new), lse=lse)
        pos = torch.cat([torch.arange(n, device="cuda") + m - n for m, n in zip(lens, new)])
        assert (out[pos < 0] == 0).all() and (lse[pos < 0] == -math.inf).all()
        assert out[pos >= 0].isnan().all() and lse[pos >= 0].isnan().all()
        out = iqq.kv8_attention(c.cache, q, torch.full_like(c.tables, -1), _i32(lens), _cu(new), lse=lse)
        assert (out == 0).all() and (lse == -math.inf).all()


def _check_scales(iqq, c, new, heads, dtype, q):
    """Attention where value scales lie far apart.  The weights p_j times their page's value scale are
    rounded to binary16, 2^-11 of each or 2^-31 of the row's largest such product (a page of zeros counts
    as the scale 2^-40 there, or 2^-100 of the largest): a code of 127 in each of the keys."""
    out = iqq.kv8_attention(c.cache, q, c.tables, _i32(c.lens), _cu(new))
    u, at = torch.finfo(dtype).eps / 2, 0
    for b, n in enumerate(new):
        for h in range(heads):
            k, v = c.values(b, 0, h // (heads // c.kv)), c.values(b, 1, h // (heads // c.kv))
            cells = c.tables[b, :-(-c.lens[b] // c.page)].long()
            vs = c.cache.v_scales[cells, h // (heads // c.kv)].double().repeat_interleave(c.page)[:c.lens[b]]
            seen = torch.arange(c.lens[b], device="cuda")[None] <= c.lens[b] - n + torch.arange(n, device="cuda")[:, None]
            qh = q[at:at + n, h].double()
            s = (qh @ k.t() * c.dim ** -0.5).masked_fill(~seen, -math.inf)
            big = (qh.abs() @ k.abs().t() * c.dim ** -0.5).amax(1)
            p = torch.softmax(s, 1)
            ref, mass = p @ v, p @ v.abs()
            as_if = torch.where(vs > 0, vs, max(2.0 ** -40, 2.0 ** -100 * float(vs.max())))
            bound = mass * (u + 2 * (c.dim + 8) * 2.0 ** -24 * big[:, None] + (c.lens[b] + 64) * 2.0 ** -24)
            bound = bound + c.lens[b] * 127 * 2.0 ** -31 * (p * as_if).amax(1)[:, None] + u * ref.abs() * (1 + u) + STEP[dtype]
            off = (out[at:at + n, h].double() - ref).abs()
            assert (off <= bound).all(), (b, h, float((off / bound).max()))
        at += n


def _zero_pages_before_small_values(iqq, new, small):
    """Pages of zeros (scale 0), then values whose scales are near 2^small, which bfloat16 holds; one of
    the sequences begins with such zeros, the other has them behind a page of the scale 1 that gets
    next to no weight."""
    c = Case(iqq, [640, 500], 1, 64, 64, 97)
    c.cache.v_scales.mul_(100.0 * 2.0 ** small)
    c.cache.v_scales[c.tables[0, :5].long()] = 0.0
    c.cache.v_scales[c.tables[1, 1:3].long()] = 0.0
    c.cache.v_scales[c.tables[1, 0].long()] = 1.0
    c.cache.k_codes[c.tables[1, 0].long()] = -127
    q = c.randn(sum(new), 2, 64, dtype=BF16)
    at = sum(new[:1])
    q[at:] = q[at:].abs() + 6.0
    c.cache.k_codes[c.tables[1, 1:].long()] = c.cache.k_codes[c.tables[1, 1:].long()] // 16
    c.cache.k_scales.fill_(0.02)
    _check_scales(iqq, c, new, 2, BF16, q)


def _zero_pages_beside_the_largest_values(iqq, new):
    """Pages of zeros before, between and behind pages of scales near 2^93: they keep their share of the
    weights."""
    c = Case(iqq, [900], 1, 64, 64, 103)
    c.cache.v_scales.mul_(2.0 ** 100)
    c.cache.v_scales[c.tables[0, [0, 1, 6, 14]].long()] = 0.0
    q = c.randn(new[0], 2, 64, dtype=BF16)
    _check_scales(iqq, c, new, 2, BF16, q)


@pytest.mark.parametrize("small", [-21, -32, -45, -70])
def test_prompts_with_zero_pages_before_small_values(iqq, small):
    _zero_pages_before_small_values(iqq, [300, 200], small)


def test_prompts_with_zero_pages_beside_the_largest_values(iqq):
    _zero_pages_beside_the_largest_values(iqq, [150])


@pytest.mark.parametrize("new", [[1, 1], [3, 4]])
@pytest.mark.parametrize("small", [-21, -32, -45, -70])
def test_tokens_with_zero_pages_before_small_values(iqq, new, small):
    _zero_pages_before_small_values(iqq, new, small)


def test_tokens_with_zero_pages_beside_the_largest_values(iqq):
    _zero_pages_beside_the_largest_values(iqq, [1])


@pytest.mark.parametrize("new", [[1], [4], [200]])
@pytest.mark.parametrize("lens", [[700], [5000]])
@pytest.mark.parametrize("apart", [20, 26, 34, 60])
def test_attention_negligible_page_of_large_values(iqq, new, lens, apart):
    """A page whose value scale is 2^apart times the others' and whose keys get next to no weight: the
    others' weights keep their bits, wherever the page lies."""
    for where in (0, 1, 9):
        c = Case(iqq, lens, 1, 128, 64, 101)
        c.cache.k_scales.fill_(0.02)
        c.cache.k_codes[:] = c.cache.k_codes // 16
        c.cache.k_codes[c.tables[0, where].long()] = -127
        c.cache.v_scales[c.tables[0, where].long()] *= 2.0 ** apart
        q = c.randn(new[0], 2, 128, dtype=BF16).abs() + 5.0
        _check_scales(iqq, c, new, 2, BF16, q)


def test_calls_in_turn_on_the_same_buffers(iqq):
    """Append and gather, and append and attention, over and over on the same pages with other data, and
    nothing that waits for the device between the calls: every call sees what the one before wrote."""
    lens = [130, 64, 1, 40]
    c = Case(iqq, lens, 4, 128, 64, 109)
    args, total = (c.tables, _i32(lens), _cu(lens)), sum(lens)
    data = [c.randn(total, 4, 128, dtype=BF16) * 2.0 ** (i % 5 - 2) for i in range(24)]
    q, last = c.randn(4, 8, 128, dtype=BF16), _i32([0, 1, 2, 3, 4])
    alone = []
    for x in data:
        iqq.iqq_kv8_append(c.cache, x, -x, *args)
        torch.cuda.synchronize()
        k, v = iqq.kv8_gather(c.cache, *args, total, dtype=BF16)
        torch.cuda.synchronize()
        alone.append((k, v, iqq.kv8_attention(c.cache, q, c.tables, args[1], last)))
        torch.cuda.synchronize()
    got = []
    for x in data:
        iqq.iqq_kv8_append(c.cache, x, -x, *args)
        k, v = iqq.kv8_gather(c.cache, *args, total, dtype=BF16)
        got.append((k, v, iqq.kv8_attention(c.cache, q, c.tables, args[1], last)))
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("lens,new,heads", [([100, 80, 50], [2, 1, 2], 2), ([9000, 700, 300], [1, 2, 1], 4),
                                            ([700, 650, 900], [300, 200, 400], 4), ([20000, 9000, 900], [40, 60, 50], 8)])
def test_attention_bad_spans_leave_their_rows(iqq, lens, new, heads):
    """A span below 0, beyond the rows, of negative length, and a negative length of the sequence: its
    rows and their log-sums stay as they were, and the other sequences' rows are what a good call
    gives.  Whole tiles, shares joined, the prompt kernel, and its keys split."""
    c = Case(iqq, lens, 1, 64, 16, 107)
    total, n = sum(new), len(lens)
    q = c.randn(total, heads, 64, dtype=BF16)
    need = iqq.kv8_attention_workspace_bytes(c.cache, n, c.tables.shape[1], heads, total)
    assert (need > 0) == (max(lens) > 5000)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(m, cu):
        out, lse = torch.full_like(q, 7.0), torch.full((total, heads), 7.0, device="cuda")
        flags.zero_()
        iqq.iqq_kv8_attention(c.cache, q, c.tables, _i32(m), _i32(cu), out, lse=lse, workspace=ws, flags=flags)
        return out, lse, int(flags.item())

    cu = _cu(new).tolist()
    good, good_lse, f = call(lens, cu)
    assert f == 0
    for m, at, bad in ((lens, [-4] + cu[1:], [0]), (lens, cu[:-1] + [total + 9], [2]),
                       ([lens[0], -3, lens[2]], cu, [1]), ([-1, lens[1], lens[2]], cu, [0]),
                       (lens, [cu[0], cu[2], cu[1], cu[1]], [1]), (lens, [-2, -1, total + 1, 2 ** 31 - 1], [0, 1, 2])):
        out, lse, f = call(m, at)
        assert f == iqq.FLAG_BAD_INDEX, (m, at)
        written = torch.zeros(total, dtype=torch.bool, device="cuda")
        for b in range(n):
            if b not in bad:
                written[at[b]:at[b + 1]] = True
        assert (out[~written] == 7.0).all() and (lse[~written] == 7.0).all(), (m, at)
        for b in range(n):
            if b not in bad and (at[b], at[b + 1]) == (cu[b], cu[b + 1]):
                torch.testing.assert_close(out[cu[b]:cu[b + 1]].float(), good[cu[b]:cu[b + 1]].float(),
                                           rtol=2.0 ** -7, atol=2e-3)
                torch.testing.assert_close(lse[cu[b]:cu[b + 1]], good_lse[cu[b]:cu[b + 1]], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("keys", [1, 63, 500, 640, 704, 705, 960, 1024, 1100])
@pytest.mark.parametrize("kv,group,dim", [(1, 8, 128), (8, 4, 64), (40, 1, 128)])
def test_attention_one_short_sequence(iqq, keys, kv, group, dim):
    """One token over tables on both sides of the lengths up to which a CTA takes a whole tile."""
    c = Case(iqq, [keys], kv, dim, 64, 113)
    c.tables = c.tables[:, :-(-keys // 64)].contiguous()
    _check_attention(iqq, c, [1], kv * group, F16)
