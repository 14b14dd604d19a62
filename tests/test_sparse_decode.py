"""Block-sparse decoding: norm + rotation + append, page bounds, page selection and the attention over
selected pages, each against its formula in 64 bits; refusals on the host.

Tolerances, derived from the arithmetic: a 16-bit or E4M3 result is one rounding (at most half a step,
finfo.eps / 2 of the value) of an fp32 value, and that value carries at most 32 fp32 roundings of the magnitudes
it is made of (a chain of at most 32 products and 5 additions halved by the root, the root, three products and the
rotation's two).  Bounds and selected pages are equal.  The attention keeps the library's own tolerance (2e-3 of a
row's largest element, 1e-4 on lse) plus the output's rounding."""
import math

import numpy as np
import pytest
import torch

import paged_split_kv_gather_gb300 as fd
from tests.helpers import LSE_TOL, OUT_TOL

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
gpu = pytest.mark.gpu


def half_step(t):
    return torch.finfo(t).eps / 2


def make_pool(pages, hk, page, d, dtype, layout, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    t = torch.float8_e4m3fn if dtype == "fp8" else DT[dtype]

    def rand(*shape):
        return (torch.randn(shape, generator=g) * (8.0 if dtype == "fp8" else 1.0)).to(t).to(device)

    if layout == "interleaved":
        kv = rand(pages, 2, hk, page, d)
        return kv[:, 0], kv[:, 1]
    if layout == "nhd":
        return rand(pages, page, hk, d).permute(0, 2, 1, 3), rand(pages, page, hk, d).permute(0, 2, 1, 3)
    return rand(pages, hk, page, d), rand(pages, hk, page, d)


def bits(t):
    return t.contiguous().view(torch.uint8)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


# ------------------------------------------------------------------------------------------- norm, rotation, append

def norm_rope_reference(x, w, cos_sin, positions, interleaved, eps):
    """(64-bit result, magnitudes its fp32 error is relative to) of rows [n, H, D]."""
    x = x.double().cpu()
    n, _, d = x.shape
    rs = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = x * rs * (1.0 if w is None else w.double().cpu())
    mag = y.abs()
    if cos_sin is None:
        return y, mag
    rot = cos_sin.shape[1]
    cs = cos_sin.double().cpu()[torch.as_tensor(positions).long()]
    out, m = y.clone(), mag.clone()
    for e in range(rot // 2):
        ia, ib = (2 * e, 2 * e + 1) if interleaved else (e, e + rot // 2)
        c, s = cs[:, e, None], cs[:, rot // 2 + e, None]
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        m[..., ia], m[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out, m


def assert_rounded(got, ref, mag, scale=1.0):
    """got is ref / scale rounded to its own type, the fp32 value behind it off by 32 roundings of mag."""
    t = got.dtype
    got = got.double().cpu()
    slack = 32 * 2.0 ** -24 * mag / scale
    ref = ref / scale
    if t == torch.float8_e4m3fn:
        ref = ref.clamp(-448, 448)
        smallest = 2.0 ** -10  # half a step below the smallest normal value
    else:
        smallest = 2.0 ** -25 if t == torch.float16 else 0.0
    tol = half_step(t) * (ref.abs() + slack) + slack + smallest
    bad = (got - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}: worst {((got - ref).abs() - tol).max():.3g}"


ROWS = [
    # dtype, kv, D, hq, hk, rot, interleaved, page, layout, seqs, tokens
    ("bf16", "", 64, 4, 1, 64, False, 16, "hnd", 1, 1),
    ("bf16", "", 128, 32, 4, 128, False, 64, "hnd", 1, 1),
    ("f16", "", 128, 12, 3, 64, False, 1, "nhd", 3, 5),
    ("bf16", "", 192, 6, 2, 192, False, 8, "interleaved", 2, 33),
    ("f16", "", 192, 5, 5, 96, True, 32, "hnd", 7, 1),
    ("f16", "", 256, 16, 8, 128, False, 16, "interleaved", 64, 1),
    ("bf16", "", 512, 3, 1, 512, False, 256, "nhd", 2, 19),
    ("f16", "", 512, 8, 8, 32, True, 128, "hnd", 1, 40),
    ("bf16", "fp8", 128, 8, 2, 128, True, 16, "nhd", 3, 21),
    ("f16", "fp8", 256, 8, 4, 16, False, 32, "interleaved", 5, 1),
    ("bf16", "", 128, 32, 8, 0, False, 16, "hnd", 2, 700),
]


@gpu
@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c)))
def test_norm_rope_append(case):
    dtype, kv, d, hq, hk, rot, inter, page, layout, seqs, tokens = case
    t = DT[dtype]
    rng = np.random.default_rng(d + tokens)
    starts = rng.integers(0, 3 * page + 2, seqs)
    width = int(max(starts) + tokens) // page + 1
    pages = seqs * width + 3
    table = rng.permutation(pages)[: seqs * width].reshape(seqs, width)
    k, v = make_pool(pages, hk, page, d, kv or dtype, layout, seed=d)
    n = seqs * tokens
    g = torch.Generator().manual_seed(n)
    qkv = (torch.randn(n, hq + 2 * hk, d, generator=g) * 3).to(t)
    qkv[0, 0] = 0  # a row of zeros: eps keeps it finite
    qkv = qkv.cuda()
    q, k_new, v_new = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    qw = (1 + 0.3 * torch.randn(d, generator=g)).to(t).cuda()
    kw = None if hq == 12 else (1 + 0.3 * torch.randn(d, generator=g)).to(t).cuda()
    cos_sin = None
    if rot:
        ang = np.arange(4096)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
        cos_sin = torch.as_tensor(np.concatenate([np.cos(ang), np.sin(ang)], 1), dtype=torch.float32).cuda()
    bi = np.repeat(np.arange(seqs), tokens)
    pos = np.concatenate([np.arange(s, s + tokens) for s in starts])
    rope = pos + 1000 if dtype == "f16" else pos
    perm = rng.permutation(n)
    bi, pos, rope = bi[perm], pos[perm], rope[perm]
    ks, vs = (0.0625, 0.02) if kv else (1.0, 1.0)
    before = [bits(k).clone(), bits(v).clone(), bits(qkv).clone()]
    k0, v0 = k.clone(), v.clone()
    q_out = torch.full((n, hq, d), float("nan"), dtype=t, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fd.fdec_norm_rope_append(q, k_new, v_new, qw, kw, cos_sin, i32(bi), i32(pos), q_out, k, v, i32(table), page,
                             eps=1e-5, interleaved=inter, rope_positions=i32(rope) if dtype == "f16" else None,
                             k_scale=ks, v_scale=vs, device_errors=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(bits(qkv), before[2])
    assert_rounded(q_out, *norm_rope_reference(q, qw, cos_sin, rope, inter, 1e-5))
    at = (torch.as_tensor(table[bi, pos // page]).long().cuda(), slice(None), torch.as_tensor(pos % page).long().cuda())
    view = (lambda x: x.view(torch.uint8)) if kv else (lambda x: x)
    got_k, got_v = view(k)[at], view(v)[at]
    if kv:
        got_k, got_v = got_k.view(torch.float8_e4m3fn), got_v.view(torch.float8_e4m3fn)
    assert_rounded(got_k, *norm_rope_reference(k_new, kw, cos_sin, rope, inter, 1e-5), scale=ks)
    if kv:
        assert_rounded(got_v, v_new.double().cpu(), v_new.double().cpu().abs(), scale=vs)
    else:
        assert torch.equal(got_v, v_new)
    # every other row of the cache is as it was
    for pool, old in ((k, k0), (v, v0)):
        view(pool)[at] = view(old)[at]
        assert torch.equal(bits(pool), bits(old))
    # in place
    fd.fdec_norm_rope_append(q, k_new, v_new, qw, kw, cos_sin, i32(bi), i32(pos), q, k, v, i32(table), page,
                             eps=1e-5, interleaved=inter, rope_positions=i32(rope) if dtype == "f16" else None,
                             k_scale=ks, v_scale=vs)
    assert torch.equal(q, q_out)


@gpu
def test_norm_rope_append_skips_and_flags_bad_tokens():
    k, v = make_pool(6, 2, 16, 128, "bf16", "hnd", 1)
    before = (k.clone(), v.clone())
    qkv = torch.randn(4, 8, 128, device="cuda").bfloat16()
    cos_sin = torch.ones(40, 128, device="cuda")
    q_out = torch.zeros(4, 4, 128, dtype=torch.bfloat16, device="cuda")
    table = i32([[0, 1, 2], [3, 99, 5]])

    def call(bi, pos, rope=None):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        fd.fdec_norm_rope_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], None, None, cos_sin, i32(bi), i32(pos), q_out, k, v,
                                 table, 16, rope_positions=None if rope is None else i32(rope), device_errors=err)
        return int(err.item())

    assert call([2, -1, 0, 0], [0, 0, -1, 48]) == fd.DEVERR_SEQ_LEN  # bad sequences, bad positions
    assert call([0, 0, 1, 1], [47, 46, 47, 46], [40, -1, 40, 41]) == fd.DEVERR_SEQ_LEN  # rows outside cos_sin
    assert call([1, 1, 1, 1], [16, 17, 18, 19]) == fd.DEVERR_PAGE_ID
    assert torch.equal(k, before[0]) and torch.equal(v, before[1]) and not q_out.any()


# ----------------------------------------------------------------------------------------------------- page bounds

@gpu
@pytest.mark.parametrize("expected", [0, 1, 77])
@pytest.mark.parametrize("dtype,kv,d,hk,page,layout", [
    ("bf16", "", 64, 3, 16, "hnd"), ("f16", "", 128, 4, 64, "nhd"), ("bf16", "", 192, 2, 8, "interleaved"),
    ("f16", "", 256, 8, 16, "interleaved"), ("bf16", "", 512, 1, 128, "hnd"), ("bf16", "fp8", 128, 2, 256, "nhd"),
    ("f16", "fp8", 256, 2, 1, "hnd"), ("bf16", "", 128, 4, 2, "hnd")])
def test_page_bounds(dtype, kv, d, hk, page, layout, expected):
    lens = [0, 1, page, page + 1, 5 * page - 1, 300]
    begins = [0, 0, page - 1, 0, 2 * page + page // 2, 300 - min(300, 77)]
    width = max(-(-n // page) for n in lens) + 1
    rng = np.random.default_rng(page)
    pages = len(lens) * width + 2
    table = rng.permutation(pages)[: len(lens) * width].reshape(len(lens), width)
    k, _ = make_pool(pages, hk, page, d, kv or dtype, layout, seed=page)
    t = DT[dtype]
    # what lies past a length is never read: NaN there changes nothing; a NaN key shows
    for b, n in enumerate(lens):
        if n % page:
            k.view(torch.uint8)[table[b, n // page], :, n % page:] = 0x7F if kv else 0xFF
    nan_at = (int(table[5, (300 - 1) // page]), hk - 1, (300 - 1) % page, d - 1)
    k.view(torch.uint8)[nan_at[0], nan_at[1], nan_at[2], -1] = 0x7F if kv else 0xFF
    if not kv:
        k.view(torch.uint8)[nan_at[0], nan_at[1], nan_at[2], -2] = 0xFF
    bounds = torch.full((pages, hk, 2, d), 7.0, dtype=t, device="cuda")
    want = bounds.clone().double().cpu()
    kd = k.float().double().cpu()
    for b, (n, begin) in enumerate(zip(lens, begins)):
        for j in range(begin // page, -(-n // page)):
            rows = kd[table[b, j], :, : min(page, n - j * page)]
            want[table[b, j], :, 0], want[table[b, j], :, 1] = rows.amin(1), rows.amax(1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fd.fdec_page_bounds(k, bounds, i32(table), i32(begins), i32(lens), page, expected_tokens=expected,
                        device_errors=err)
    got = bounds.double().cpu()
    assert int(err.item()) == 0 and bool(want.isnan().any())
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0), want.nan_to_num(0))


@gpu
def test_page_bounds_without_begins_and_bad_pages():
    k, _ = make_pool(8, 2, 16, 128, "f16", "hnd", 3)
    bounds = torch.zeros(8, 2, 2, 128, dtype=torch.float16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fd.fdec_page_bounds(k, bounds, i32([[0, 8, 2], [-1, 4, 5]]), None, i32([48, 20]), 16, device_errors=err)
    assert int(err.item()) == fd.DEVERR_PAGE_ID
    touched = [0, 2, 4]
    for page in range(8):
        rows = k[page, :, :4] if page == 4 else k[page]
        want = torch.stack([rows.amin(1), rows.amax(1)], 1) if page in touched else torch.zeros_like(bounds[page])
        assert torch.equal(bounds[page], want), page
    err.zero_()
    fd.fdec_page_bounds(k, bounds, i32([[0, 1], [2, 3]]), i32([-5, 0]), i32([40, -3]), 16, device_errors=err)
    assert int(err.item()) == fd.DEVERR_SEQ_LEN  # 40 > 2 pages: clamped; negative: nothing
    assert torch.equal(bounds[1, :, 1], k[1].amax(1))


# --------------------------------------------------------------------------------------------------- page selection

def select_reference(q, bounds, table, lens, page, budget, first, last, causal):
    q, bounds = q.double().cpu().numpy(), bounds.double().cpu().numpy()
    b_, q_len, hq, d = q.shape
    hk = bounds.shape[1]
    g = hq // hk
    ids = np.full((b_ * q_len, hk, budget), -1, dtype=np.int32)
    index, counts = ids.copy(), np.zeros((b_ * q_len, hk), dtype=np.int32)
    for b in range(b_):
        for i in range(q_len):
            seen = max(0, lens[b] - q_len + i + 1 if causal else lens[b])
            m = -(-seen // page)
            for h in range(hk):
                if m <= budget:
                    take = list(range(m))
                else:
                    qq = q[b, i, h * g:(h + 1) * g]
                    with np.errstate(invalid="ignore", over="ignore"):
                        rows = bounds[table[b, :m], h]  # [m, 2, D]
                        neg, pos = np.where(qq > 0, 0, qq).sum(0), np.where(qq < 0, 0, qq).sum(0)
                        s = (rows[:, 0] * neg + rows[:, 1] * pos).sum(-1)
                    s = np.where(np.isnan(s), np.inf, s)
                    cand = list(range(first, m - last))
                    cand.sort(key=lambda j: (-s[j], j))
                    take = sorted(list(range(first)) + cand[: budget - first - last] + list(range(m - last, m)))
                row = b * q_len + i
                ids[row, h, : len(take)] = table[b, take]
                index[row, h, : len(take)] = take
                if m:
                    counts[row, h] = (len(take) - 1) * page + seen - (m - 1) * page
    return ids, counts, index


def run_select(q, bounds, table, lens, page, budget, first, last, causal=True, max_pages=None, twice=True):
    b, q_len, hq, d = q.shape
    sel = fd.PageSelect(b, q_len, page, hq, bounds.shape[1], d, max_pages or table.shape[1], budget,
                        "bf16" if q.dtype == torch.bfloat16 else "f16", first, last, causal)
    tb, ln = i32(table), i32(lens)
    got = [x.cpu().numpy().copy() for x in sel.run(q, bounds, tb, ln)]
    if twice:  # the workspace is as a next call expects it
        for a, c in zip(got, sel.run(q, bounds, tb, ln)):
            assert np.array_equal(a, c.cpu().numpy())
    assert sel.device_errors() == 0
    return got


def check_select(q, bounds, table, lens, page, budget, first=1, last=1, causal=True, max_pages=None):
    got = run_select(q, bounds, table, lens, page, budget, first, last, causal, max_pages)
    want = select_reference(q, bounds, table, lens, page, budget, first, last, causal)
    for name, a, c in zip(("page_ids", "counts", "page_indices"), got, want):
        assert np.array_equal(a, c), name


def bounds_like(pages, hk, d, t, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    mean = torch.randn(pages, hk, 1, d, generator=g) * 0.5
    half = torch.rand(pages, hk, 2, d, generator=g) * spread + 0.5
    half[:, :, 0].neg_()
    return (mean + half).to(t).cuda()


@gpu
@pytest.mark.parametrize("dtype,d,hq,hk,q_len,page,budget,first,last", [
    ("bf16", 64, 4, 1, 1, 16, 9, 1, 1), ("f16", 128, 32, 4, 1, 64, 16, 0, 1), ("bf16", 128, 32, 8, 4, 16, 33, 2, 3),
    ("f16", 192, 16, 8, 1, 16, 20, 1, 2), ("bf16", 256, 6, 6, 3, 1, 50, 0, 4), ("f16", 512, 8, 1, 1, 8, 13, 3, 1),
    ("bf16", 64, 33, 3, 2, 32, 5, 1, 4), ("f16", 128, 5, 5, 1, 256, 1, 0, 1), ("bf16", 192, 40, 2, 1, 128, 7, 1, 1)])
def test_select_pages(dtype, d, hq, hk, q_len, page, budget, first, last):
    rng = np.random.default_rng(d + budget)
    n = [0, q_len - 1, 1, page, budget * page, budget * page + 1, (budget + 1) * page, 300 * page - 1, 177 * page + page // 2]
    width = 300
    pages = len(n) * width
    table = rng.permutation(pages).reshape(len(n), width)
    t = DT[dtype]
    q = torch.randn(len(n), q_len, hq, d, generator=torch.Generator().manual_seed(d)).to(t).cuda()
    bounds = bounds_like(pages, hk, d, t, seed=budget)
    check_select(q, bounds, table, n, page, budget, first, last)
    if q_len > 1:
        check_select(q, bounds, table, n, page, budget, first, last, causal=False)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_select_pages_ties_go_to_the_lower_index(dtype):
    t = DT[dtype]
    table = np.random.default_rng(1).permutation(900).reshape(1, 900)
    q = torch.randn(1, 1, 8, 128, generator=torch.Generator().manual_seed(2)).to(t).cuda()
    lens = [900 * 16 - 5]
    same = bounds_like(1, 2, 128, t, 3).expand(900, -1, -1, -1).contiguous()
    check_select(q, same, table, lens, 16, 40, 1, 1)                      # every page alike
    check_select(torch.zeros_like(q), bounds_like(900, 2, 128, t, 4), table, lens, 16, 40, 2, 3)  # every score 0
    few = bounds_like(7, 2, 128, t, 5)[torch.arange(900) % 7].contiguous()  # long runs of equal scores
    check_select(q, few, table, lens, 16, 200, 0, 1)
    pairs = bounds_like(450, 2, 128, t, 6)[torch.arange(900) // 2].contiguous()
    for budget in (17, 18, 19, 20):
        check_select(q, pairs, table, lens, 16, budget, 1, 1)


@gpu
def test_select_pages_orders_by_the_64_bit_score():
    """Scores whose differences are far below an fp32 rounding of their terms."""
    d, pages = 128, 600
    rng = np.random.default_rng(7)
    bounds = torch.zeros(pages, 1, 2, d)
    bounds[:, :, :, 0], bounds[:, :, :, 1] = 4096.0, -4096.0  # cancels, at a size that drowns the rest in 32 bits
    small = torch.as_tensor(rng.permutation(pages).astype(np.float64) + 1) * 2.0 ** -20
    bounds[:, 0, :, 2] = small[:, None].bfloat16().float()
    q = torch.ones(1, 1, 1, d)
    q[..., 2:] = 2.0 ** -3
    perm = rng.permutation(pages).reshape(1, pages)
    check_select(q.bfloat16().cuda(), bounds.bfloat16().cuda(), perm, [pages * 16], 16, 100, 1, 1)


@gpu
def test_select_pages_with_infinities_and_nans():
    table = np.random.default_rng(8).permutation(500).reshape(1, 500)
    q = torch.randn(1, 1, 4, 64, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    lens = [500 * 16]
    base = bounds_like(500, 2, 64, torch.bfloat16, 10)
    one = base.clone()
    one[table[0, 321], :, 1, 5] = float("nan")
    one[table[0, 123], 0, 0, 7] = float("nan")
    check_select(q, one, table, lens, 16, 12)
    inf = base.clone()
    inf[table[0, 77], :, 1] = float("inf")
    inf[table[0, 78], :, 0] = float("-inf")
    inf[table[0, 200:220], 1, 1, 3] = float("inf")
    check_select(q, inf, table, lens, 16, 12)
    huge = base * 1e38  # products past fp32's range, sums within 64 bits
    check_select(q * 64, huge, table, lens, 16, 12)
    tiny = base * 1e-30
    check_select(q * 1e-20, tiny, table, lens, 16, 12)
    qn = q.clone()
    qn[0, 0, 1, 3] = float("nan")  # every score of the first KV head is NaN: lowest indices
    check_select(qn, base, table, lens, 16, 12)
    qi = q.clone()
    qi[0, 0, 3, 3] = float("inf")
    check_select(qi, base, table, lens, 16, 12)


@gpu
def test_select_pages_of_a_very_long_sequence():
    pages = 70001
    table = np.random.default_rng(11).permutation(pages).reshape(1, pages)
    q = torch.randn(1, 1, 16, 128, generator=torch.Generator().manual_seed(12)).half().cuda()
    bounds = bounds_like(pages, 2, 128, torch.float16, 13)
    check_select(q, bounds, table, [pages * 16 - 3], 16, 500, 4, 8)
    check_select(q, bounds, table, [pages * 16 - 3], 16, 60000, 4, 8)


@gpu
@pytest.mark.parametrize("b", [2, 20])
def test_select_pages_of_rows_around_a_tile(b):
    """Rows of about 4096, 8192 and 16384 pages, few (16) and more than one an SM (160)."""
    pages, lens = 16500, [4096, 16384, 4097, 16385, 8193, 8192, 4098, 16500] + [7, 0, 5000, 12289, 1, 16386, 8194, 300, 4000, 2, 9999, 40]
    lens = lens[:b] if b > 2 else [16386, 16384]
    table = np.tile(np.random.default_rng(14).permutation(pages), (b, 1))
    q = torch.randn(b, 1, 16, 64, generator=torch.Generator().manual_seed(15)).bfloat16().cuda()
    check_select(q, bounds_like(pages, 8, 64, torch.bfloat16, 16), table, lens, 1, 128, 1, 1)


@gpu
def test_select_pages_flags_lengths_and_page_ids():
    table = np.arange(100).reshape(1, 100)
    q = torch.randn(1, 1, 4, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    bounds = bounds_like(100, 1, 64, torch.float16, 2)
    sel = fd.PageSelect(1, 1, 16, 4, 1, 64, 100, 10, "f16")
    want = select_reference(q, bounds, table, [1600], 16, 10, 1, 1, True)
    got = sel.run(q, bounds, i32(table), i32([1700]))  # clamped to the 100 pages
    assert sel.device_errors() == fd.DEVERR_SEQ_LEN
    for a, c in zip(got, want):
        assert np.array_equal(a.cpu().numpy(), c)
    sel.run(q, bounds, i32(table), i32([-4]))
    assert sel.device_errors() == fd.DEVERR_SEQ_LEN and int(sel.counts.sum()) == 0
    bad = table.copy()
    bad[0, 50], bad[0, 60] = 100, -7
    ids, counts, index = sel.run(q, bounds, i32(bad), i32([1600]))
    assert sel.device_errors() == fd.DEVERR_PAGE_ID
    assert not np.isin(index.cpu().numpy(), [50, 60]).any() and int(counts[0, 0]) == 160


# ------------------------------------------------------------------------------- attention over selected pages

def attend_reference(q, k, v, ids, counts, scale):
    q, k, v = q.double().cpu().numpy(), k.float().double().cpu().numpy(), v.float().double().cpu().numpy()
    n, _, hq, d = q.shape
    hk, page = k.shape[1], k.shape[2]
    g = hq // hk
    out, lse = np.zeros((n, 1, hq, d)), np.full((n, 1, hq), -np.inf)
    for r in range(n):
        for h in range(hk):
            c = counts[r, h]
            if c == 0:
                continue
            pages = ids[r, h, : -(-c // page)]
            kk, vv = k[pages, h].reshape(-1, d)[:c], v[pages, h].reshape(-1, d)[:c]
            for x in range(h * g, (h + 1) * g):
                z = kk @ q[r, 0, x] * scale
                top = z.max()
                e = np.exp(z - top)
                out[r, 0, x] = e @ vv / e.sum()
                lse[r, 0, x] = top + np.log(e.sum())
    return out, lse


def assert_attention(out, lse, ref_out, ref_lse):
    half = 0.0 if out.dtype == torch.float32 else half_step(out.dtype)
    o = out.double().cpu().numpy()
    peak = np.abs(ref_out).max(-1, keepdims=True)
    assert np.isfinite(o).all()
    # + the smallest binary16 step for rows of tiny values
    assert (np.abs(o - ref_out) <= (OUT_TOL + half) * peak + 2.0 ** -25).all()
    got = lse.double().cpu().numpy()
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got), empty) and not o[empty].any()
    assert (np.abs(got[~empty] - ref_lse[~empty]) <= LSE_TOL).all()


ATTEND = [
    # dtype, kv, D, hq, hk, page, budget, rows, layout
    ("bf16", "", 64, 4, 1, 16, 3, 2, "hnd"), ("bf16", "", 128, 32, 4, 64, 64, 1, "hnd"),
    ("f16", "", 128, 32, 8, 16, 40, 9, "interleaved"), ("bf16", "", 192, 16, 8, 8, 30, 5, "nhd"),
    ("f16", "", 256, 16, 8, 32, 17, 6, "interleaved"), ("bf16", "", 512, 4, 2, 16, 9, 7, "hnd"),
    ("bf16", "", 128, 8, 2, 1, 130, 4, "nhd"), ("f16", "", 64, 6, 3, 4, 33, 4, "hnd"),
    ("bf16", "", 128, 64, 2, 16, 21, 3, "hnd"), ("f16", "", 256, 70, 2, 64, 6, 3, "nhd"),
    ("bf16", "fp8", 128, 32, 8, 16, 40, 5, "nhd"), ("f16", "fp8", 256, 8, 2, 64, 11, 5, "hnd"),
    ("bf16", "fp8", 128, 40, 2, 128, 3, 3, "interleaved"), ("f16", "", 128, 2, 2, 256, 20, 40, "hnd"),
    ("f16", "", 64, 4, 4, 64, 10, 1000, "hnd"), ("bf16", "", 64, 5, 1, 8, 65, 33, "nhd"),
]


def selected_lists(rows, hk, page, budget, pool_pages, seed):
    """Page lists of differing lengths for every row and head, -1 past them, and token counts, one list empty, one
    of a single token, one full."""
    rng = np.random.default_rng(seed)
    ids = np.full((rows, hk, budget), -1, dtype=np.int32)
    counts = np.zeros((rows, hk), dtype=np.int32)
    for r in range(rows):
        for h in range(hk):
            c = int(rng.integers(1, budget * page + 1))
            c = [budget * page, 0, 1][(r * hk + h) % 3] if r * hk + h < 3 else c
            counts[r, h] = c
            ids[r, h, : -(-c // page)] = rng.choice(pool_pages, -(-c // page), replace=False)
    return ids, counts


@gpu
@pytest.mark.parametrize("out_type", ["f32", "same"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(map(str, c)))
def test_run_selected(case, out_type):
    dtype, kv, d, hq, hk, page, budget, rows, layout = case
    t = DT[dtype]
    pool_pages = 2 * budget + 5
    k, v = make_pool(pool_pages, hk, page, d, kv or dtype, layout, seed=budget)
    ids, counts = selected_lists(rows, hk, page, budget, pool_pages, seed=rows)
    q = torch.randn(rows, 1, hq, d, generator=torch.Generator().manual_seed(d)).to(t).cuda()
    ks, vs = (0.125, 0.25) if kv else (1.0, 1.0)
    pd = fd.PagedDecode([budget * page] * rows, 1, page, hq, hk, d, dtype, kv_dtype=kv)
    out = torch.full((rows, 1, hq, d), float("nan"), dtype=torch.float32 if out_type == "f32" else t, device="cuda")
    lse = torch.full((rows, 1, hq), float("nan"), device="cuda")
    pd.run_selected(q, k, v, i32(ids), i32(counts), out, lse, k_scale=ks, v_scale=vs)
    assert pd.device_errors() == 0
    ref = attend_reference(q, k.float() * ks, v.float() * vs, ids, counts, 1 / math.sqrt(d))
    assert_attention(out, lse, *ref)
    if not kv and hq * d >= 64:  # q rows off 16 bytes: another split kernel
        odd = torch.zeros(rows * hq * d + 1, dtype=t, device="cuda")[1:].view(rows, 1, hq, d)
        odd.copy_(q)
        pd.run_selected(odd, k, v, i32(ids), i32(counts), out, lse)
        assert_attention(out, lse, *ref)


@gpu
@pytest.mark.parametrize("kv,d,hk,group,rows,page,budget", [
    ("", 512, 3, 4, 12, 32, 10), ("", 512, 1, 8, 5, 64, 5), ("", 256, 4, 4, 12, 16, 30), ("", 192, 4, 2, 9, 64, 10),
    ("", 128, 8, 20, 12, 8, 90), ("", 64, 8, 4, 40, 64, 12), ("", 64, 1, 33, 70, 16, 41), ("fp8", 256, 4, 8, 27, 16, 16),
    ("fp8", 128, 8, 4, 27, 64, 4)])
def test_run_selected_over_lists_of_a_few_blocks(kv, d, hk, group, rows, page, budget):
    """Lists around the sizes at which the work is cut at run time instead of as planned."""
    pool_pages, hq = 3 * budget, hk * group
    k, v = make_pool(pool_pages, hk, page, d, kv or "bf16", "nhd", seed=d)
    q = torch.randn(rows, 1, hq, d, generator=torch.Generator().manual_seed(rows)).bfloat16().cuda()
    pd = fd.PagedDecode([budget * page] * rows, 1, page, hq, hk, d, "bf16", kv_dtype=kv)
    out, lse = torch.empty(rows, 1, hq, d, device="cuda"), torch.empty(rows, 1, hq, device="cuda")
    for full in (False, True):
        ids, counts = selected_lists(rows, hk, page, budget, pool_pages, seed=budget)
        if full:
            counts[:] = budget * page
            ids[:] = np.random.default_rng(d).integers(0, pool_pages, ids.shape)
        out.fill_(float("nan")), lse.fill_(float("nan"))
        pd.run_selected(q, k, v, i32(ids), i32(counts), out, lse)
        assert pd.device_errors() == 0
        assert_attention(out, lse, *attend_reference(q, k.float(), v.float(), ids, counts, 1 / math.sqrt(d)))


@gpu
@pytest.mark.parametrize("path", [fd.FDEC_PATH_SIMT, fd.FDEC_PATH_MMA, fd.FDEC_PATH_TC])
@pytest.mark.parametrize("blocks_per_split", [0, 1])
def test_run_selected_on_every_path_equals_run_of_the_same_pages(path, blocks_per_split):
    """With every head given the sequence's own pages, the result is fdec_run's (bit for bit where the work is cut
    alike), and the same in every run."""
    rows, hq, hk, d, page, budget = 3, 32, 2, 128, 16, 20
    k, v = make_pool(80, hk, page, d, "bf16", "hnd", 4)
    ids, counts = selected_lists(rows, 1, page, budget, 80, seed=4)
    q = torch.randn(rows, 1, hq, d, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    pd = fd.PagedDecode([budget * page] * rows, 1, page, hq, hk, d, "bf16", path=path, blocks_per_split=blocks_per_split)
    a, b = (torch.full((rows, 1, hq, d), float("nan"), device="cuda") for _ in range(2))
    la, lb = (torch.full((rows, 1, hq), float("nan"), device="cuda") for _ in range(2))
    pd.run(q, k, v, i32(ids[:, 0]), i32(counts[:, 0]), a, la)
    pd.run_selected(q, k, v, i32(ids.repeat(hk, 1)), i32(counts.repeat(hk, 1)), b, lb)
    assert pd.device_errors() == 0
    if path != fd.FDEC_PATH_MMA:  # which cuts the lists into shares by their run-time lengths
        assert torch.equal(a, b) and torch.equal(la, lb)
    else:
        again, lagain = torch.empty_like(b), torch.empty_like(lb)
        pd.run_selected(q, k, v, i32(ids.repeat(hk, 1)), i32(counts.repeat(hk, 1)), again, lagain)
        assert torch.equal(again, b) and torch.equal(lagain, lb)
    ref = attend_reference(q, k, v, ids.repeat(hk, 1), counts.repeat(hk, 1), 1 / math.sqrt(d))
    assert_attention(b, lb, *ref)
    short = torch.empty((rows, 1, hq, d), dtype=torch.bfloat16, device="cuda")
    pd.run_selected(q, k, v, i32(ids.repeat(hk, 1)), i32(counts.repeat(hk, 1)), short, lb)
    assert torch.equal(short, b.bfloat16())  # the one rounding


@gpu
def test_run_selected_flags_bad_pages_and_counts():
    k, v = make_pool(8, 2, 16, 64, "f16", "hnd", 1)
    q = torch.randn(1, 1, 4, 64, device="cuda").half()
    out, lse = torch.empty(1, 1, 4, 64, device="cuda"), torch.empty(1, 1, 4, device="cuda")
    pd = fd.PagedDecode([64], 1, 16, 4, 2, 64, "f16", path=fd.FDEC_PATH_MMA)
    pd.run_selected(q, k, v, i32([[[0, 1, 2, 3], [0, 9, 2, 3]]]), i32([[64, 64]]), out, lse)
    assert pd.device_errors() == fd.DEVERR_PAGE_ID
    pd.run_selected(q, k, v, i32([[[0, 1, 2, 3], [0, 1, 2, 3]]]), i32([[65, -1]]), out, lse)
    assert pd.device_errors() == fd.DEVERR_SEQ_LEN
    assert bool(torch.isneginf(lse[0, 0, 2:]).all()) and bool(torch.isfinite(lse[0, 0, :2]).all())


# ------------------------------------------------------------------------------------------------- the whole step

def step_state(seed, q_len, page=16, dtype="bf16", kv=""):
    torch.manual_seed(seed)
    hq, hk, d, budget = 16, 4, 128, 12
    lens = [q_len, 333, 700, 129]
    width = 50
    k, v = make_pool(len(lens) * width, hk, page, d, kv or dtype, "interleaved", seed)
    table = np.random.default_rng(seed).permutation(len(lens) * width).reshape(len(lens), width)
    bounds = torch.zeros(len(lens) * width, hk, 2, d, dtype=DT[dtype], device="cuda")
    fd.fdec_page_bounds(k, bounds, i32(table), None, i32(lens) - q_len, page)
    n = len(lens) * q_len
    ang = torch.arange(800)[:, None] * 10000.0 ** (-torch.arange(d // 2) / (d // 2))
    return dict(hq=hq, hk=hk, d=d, budget=budget, lens=lens, k=k, v=v, table=table, bounds=bounds, n=n, page=page,
                qkv=(torch.randn(n, hq + 2 * hk, d) * 2).to(DT[dtype]).cuda(),
                qw=(1 + 0.2 * torch.randn(d)).to(DT[dtype]).cuda(), kw=(1 + 0.2 * torch.randn(d)).to(DT[dtype]).cuda(),
                cos_sin=torch.cat([ang.cos(), ang.sin()], 1).cuda())


@gpu
@pytest.mark.parametrize("q_len,kv", [(1, ""), (3, ""), (1, "fp8")])
def test_a_step_of_sparse_decoding(q_len, kv):
    s = step_state(3 + q_len, q_len, kv=kv)
    sd = fd.SparseDecode([800] * 4, q_len, s["page"], s["hq"], s["hk"], s["d"], s["budget"], kv_dtype=kv)
    ks, vs = (0.0625, 0.0625) if kv else (1.0, 1.0)
    hq, hk, n = s["hq"], s["hk"], s["n"]
    qkv = s["qkv"].clone()
    out = torch.empty(n, 1, hq, s["d"], dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, 1, hq, device="cuda")
    lens = i32(s["lens"])
    sd.step(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], s["qw"], s["kw"], s["cos_sin"], s["k"], s["v"],
            s["bounds"], i32(s["table"]), lens, out, lse, k_scale=ks, v_scale=vs)
    assert sd.device_errors() == 0
    pos = np.concatenate([np.arange(L - q_len, L) for L in s["lens"]])
    assert_rounded(qkv[:, :hq].clone(), *norm_rope_reference(s["qkv"][:, :hq], s["qw"], s["cos_sin"], pos, False, 1e-6))
    fresh = torch.zeros_like(s["bounds"])
    fd.fdec_page_bounds(s["k"], fresh, i32(s["table"]), None, lens, s["page"])
    assert torch.equal(fresh, s["bounds"])
    q = qkv[:, :hq]
    ids, counts, _ = select_reference(q.reshape(4, q_len, hq, s["d"]), s["bounds"], s["table"], s["lens"], s["page"],
                                      s["budget"], 1, 2, True)
    ref = attend_reference(q.reshape(n, 1, hq, s["d"]), s["k"].float() * ks, s["v"].float() * vs, ids, counts,
                           1 / math.sqrt(s["d"]))
    assert_attention(out, lse, *ref)


@gpu
def test_a_step_in_a_graph_and_on_another_stream():
    s = step_state(9, 1)
    hq, hk = s["hq"], s["hk"]
    table, lens = i32(s["table"]), i32(s["lens"])
    results = []
    for mode in ("eager", "stream", "graph"):
        sd = fd.SparseDecode([800] * 4, 1, s["page"], hq, hk, s["d"], s["budget"])
        qkv, k, v, bounds = (s[x].clone() for x in ("qkv", "k", "v", "bounds"))
        out = torch.zeros(s["n"], 1, hq, s["d"], dtype=torch.bfloat16, device="cuda")

        def step():
            sd.step(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], s["qw"], s["kw"], s["cos_sin"], k, v, bounds,
                    table, lens, out)

        torch.cuda.synchronize()
        if mode == "eager":
            step()
        elif mode == "stream":
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                step()
            side.synchronize()
        else:
            keep = [x.clone() for x in (qkv, k, v, bounds)]
            step()  # warm-up outside the capture
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for _ in range(3):
                for x, y in zip((qkv, k, v, bounds), keep):
                    x.copy_(y)
                out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        assert sd.device_errors() == 0
        results.append([x.clone() for x in (qkv, k, v, bounds, out)])
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------------------------- refusals (no device)

def cpu_rows(n=2, hq=4, hk=2, d=128, t=torch.bfloat16, page=16):
    qkv = torch.zeros(n, hq + 2 * hk, d, dtype=t)
    return dict(q=qkv[:, :hq], k_new=qkv[:, hq:hq + hk], v_new=qkv[:, hq + hk:], q_weight=None, k_weight=None,
                cos_sin=torch.zeros(64, d), batch_indices=torch.zeros(n, dtype=torch.int32),
                positions=torch.zeros(n, dtype=torch.int32), q_out=torch.zeros(n, hq, d, dtype=t),
                k=torch.zeros(4, hk, page, d, dtype=t), v=torch.zeros(4, hk, page, d, dtype=t),
                page_table=torch.zeros(1, 4, dtype=torch.int32), page_size=page)


def refused(status, fn, **kw):
    with pytest.raises(fd.FdecError) as e:
        fn(stream=0, **kw)
    assert e.value.status_name == status and str(e.value), e.value


def test_norm_rope_append_refusals():
    fn = fd.fdec_norm_rope_append
    ok = cpu_rows()
    empty = cpu_rows(n=0)
    fn(stream=0, **empty)  # nothing to do: no launch
    for bad in (cpu_rows(d=80), cpu_rows(page=48), cpu_rows(page=512)):
        bad["cos_sin"] = None
        refused("FDEC_ERR_UNSUPPORTED", fn, **bad)
    for rot in (24, 144):
        refused("FDEC_ERR_INVALID_ARG", fn, **{**ok, "cos_sin": torch.zeros(64, rot)})
    for eps in (-1.0, float("nan"), float("inf")):
        refused("FDEC_ERR_INVALID_ARG", fn, eps=eps, **ok)
    refused("FDEC_ERR_INVALID_ARG", fn, k_scale=2.0, **ok)  # a 16-bit cache has no scales
    codes = {**ok, "k": ok["k"].to(torch.float8_e4m3fn), "v": ok["v"].to(torch.float8_e4m3fn)}
    for scale in (0.0, -1.0, float("nan")):
        refused("FDEC_ERR_INVALID_ARG", fn, v_scale=scale, **codes)
    wide = cpu_rows(d=192)
    refused("FDEC_ERR_UNSUPPORTED", fn, **{**wide, "k": wide["k"].to(torch.float8_e4m3fn), "v": wide["v"].to(torch.float8_e4m3fn)})
    # rows, pools and weights off a 16-byte boundary
    odd = torch.zeros(2 * 8 * 128 + 1, dtype=torch.bfloat16)[1:].view(2, 8, 128)
    refused("FDEC_ERR_LAYOUT", fn, **{**ok, "q": odd[:, :4]})
    refused("FDEC_ERR_LAYOUT", fn, **{**ok, "q_out": odd[:, :4]})
    refused("FDEC_ERR_LAYOUT", fn, **{**ok, "q_weight": torch.zeros(129, dtype=torch.bfloat16)[1:]})
    refused("FDEC_ERR_LAYOUT", fn, **{**ok, "k": torch.zeros(4, 2, 16, 132, dtype=torch.bfloat16)[..., :128]})
    for key, value in {
            "positions": torch.zeros(2, dtype=torch.int64), "batch_indices": torch.zeros(3, dtype=torch.int32),
            "q_weight": torch.zeros(64, dtype=torch.bfloat16), "k_weight": torch.zeros(128), "q_out": ok["q_out"][:, :2],
            "k_new": ok["k_new"].half(), "v_new": ok["v_new"][:, :1], "cos_sin": torch.zeros(64, 128).half(),
            "page_size": 32, "v": ok["v"].half(), "q": ok["q"].transpose(0, 2), "page_table": torch.zeros(4, dtype=torch.int32),
    }.items():
        with pytest.raises(ValueError):
            fn(stream=0, **{**ok, key: value})


def test_page_bounds_refusals():
    fn = fd.fdec_page_bounds
    k = torch.zeros(4, 2, 16, 128, dtype=torch.float16)
    ok = dict(k=k, bounds=torch.zeros(4, 2, 2, 128, dtype=torch.float16), page_table=torch.zeros(1, 4, dtype=torch.int32),
              begins=None, seq_lens=torch.zeros(1, dtype=torch.int32), page_size=16)
    refused("FDEC_ERR_UNSUPPORTED", fn, **{**ok, "k": torch.zeros(4, 2, 48, 128, dtype=torch.float16), "page_size": 48})
    refused("FDEC_ERR_UNSUPPORTED", fn, **{**ok, "k": torch.zeros(4, 2, 16, 64, dtype=torch.uint8),
                                           "bounds": torch.zeros(4, 2, 2, 64, dtype=torch.float16)})
    refused("FDEC_ERR_LAYOUT", fn, **{**ok, "bounds": torch.zeros(4, 2, 2, 132, dtype=torch.float16)[..., :128]})
    refused("FDEC_ERR_INVALID_ARG", fn, **{**ok, "k": torch.zeros(0, 2, 16, 128, dtype=torch.float16)})
    for key, value in {"bounds": torch.zeros(4, 2, 1, 128, dtype=torch.float16), "k": k.bfloat16(), "page_size": 32,
                       "seq_lens": torch.zeros(2, dtype=torch.int32), "begins": torch.zeros(1, dtype=torch.int64)}.items():
        with pytest.raises(ValueError):
            fn(stream=0, **{**ok, key: value})


def test_select_pages_refusals():
    fn = fd.fdec_select_pages
    total = fd.fdec_select_pages_workspace(1, 1, 2, 8)
    buf = torch.zeros(total + 256, dtype=torch.uint8)
    ws = buf[(-buf.data_ptr()) % 256:][:total]
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok = dict(q=torch.zeros(1, 1, 4, 64, dtype=torch.float16), bounds=torch.zeros(4, 2, 2, 64, dtype=torch.float16),
              page_table=i(1, 8), seq_lens=i(1), page_size=16, max_pages=8, budget=4, page_ids=i(1, 2, 4), counts=i(1, 2),
              page_indices=None, workspace=ws)
    for first, last in ((-1, 1), (0, 0), (3, 2), (4, 1)):
        refused("FDEC_ERR_INVALID_ARG", fn, first_pages=first, last_pages=last, **ok)
    refused("FDEC_ERR_WORKSPACE", fn, **{**ok, "workspace": ws[:-1]})
    refused("FDEC_ERR_WORKSPACE", fn, **{**ok, "workspace": buf[(-buf.data_ptr()) % 256 + 16:]})
    refused("FDEC_ERR_CAPACITY", fn, **{**ok, "max_pages": 0})
    refused("FDEC_ERR_UNSUPPORTED", fn, **{**ok, "page_size": 24})
    refused("FDEC_ERR_INVALID_ARG", fn, **{**ok, "q": torch.zeros(1, 1, 3, 64, dtype=torch.float16)})
    refused("FDEC_ERR_LAYOUT", fn, **{**ok, "bounds": torch.zeros(4, 2, 2, 68, dtype=torch.float16)[..., :64]})
    for key, value in {"bounds": ok["bounds"].bfloat16(), "page_ids": i(1, 2, 5), "counts": i(2, 2), "max_pages": 9,
                       "seq_lens": i(2), "page_indices": torch.zeros(1, 2, 4)}.items():
        with pytest.raises(ValueError):
            fn(stream=0, **{**ok, key: value})
    for args in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (2**20, 2**12, 1, 1)):
        with pytest.raises(fd.FdecError):
            fd.fdec_select_pages_workspace(*args)


def test_run_selected_refusals():
    lib = fd._load()
    plan = fd.fdec_plan([64, 64], 1, 16, 4, 2, 64, "f16", num_sms=152)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.float16)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(4096, dtype=torch.uint8)
    ok = dict(plan=plan, q=q, k=k, v=k, page_ids=i(2, 2, 4), counts=i(2, 2), out=torch.zeros(2, 1, 4, 64), lse=None, workspace=ws)
    fn = fd.fdec_run_selected
    refused("FDEC_ERR_WORKSPACE", fn, **ok)  # never uploaded
    refused("FDEC_ERR_CAPACITY", fn, **{**ok, "page_ids": i(2, 2, 3)})
    refused("FDEC_ERR_INVALID_ARG", fn, **{**ok, "plan": fd.fdec_plan([64], 2, 16, 4, 2, 64, "f16", num_sms=152),
                                           "q": q[:1], "page_ids": i(1, 2, 4), "counts": i(1, 2), "out": ok["out"][:1]})
    refused("FDEC_ERR_LAYOUT", fn, **{**ok, "out": torch.zeros(2 * 4 * 64 + 1)[1:].view(2, 1, 4, 64)})
    q8 = fd.fdec_plan([64, 64], 1, 16, 4, 2, 128, "f16", num_sms=152, kv_dtype="q8_0")
    k8 = torch.zeros(4, 2, 16, 128, dtype=torch.int8)
    refused("FDEC_ERR_UNSUPPORTED", fn, **{**ok, "plan": q8, "q": torch.zeros(2, 1, 4, 128, dtype=torch.float16), "k": k8,
                                           "v": k8, "out": torch.zeros(2, 1, 4, 128)})
    for key, value in {"q": q.bfloat16(), "out": torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), "page_ids": i(2, 4),
                       "counts": i(2, 1), "k": k.to(torch.float8_e4m3fn)}.items():
        with pytest.raises(ValueError):
            fn(stream=0, **{**ok, key: value})
    assert lib.fdec_run_selected(None, None, 0, 0, fd.KVDesc(), fd.KVDesc(), None, 0, None, 1.0, 1.0, 1.0, None, 0, None,
                                 None, None) == 1  # a null plan


# ------------------------------------------------------------------------------- layouts, offsets, random shapes

@gpu
def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: the last pages are written, bounded, scored and attended to."""
    hk, d, page, pages = 8, 512, 16, 70000
    k = torch.empty(pages, hk, page, d, dtype=torch.bfloat16, device="cuda")  # 4.6e9 elements
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 32
    own = np.concatenate([np.arange(pages - 150, pages), [3]])
    k[torch.as_tensor(own).cuda()] = torch.randn(151, hk, page, d, device="cuda").bfloat16()
    v[torch.as_tensor(own).cuda()] = torch.randn(151, hk, page, d, device="cuda").bfloat16()
    table = np.random.default_rng(1).permutation(own)[None]
    L = 151 * page - 3
    qkv = torch.randn(1, 8 + 2 * hk, d, device="cuda").bfloat16()
    q_out = torch.empty(1, 8, d, dtype=torch.bfloat16, device="cuda")
    fd.fdec_norm_rope_append(qkv[:, :8], qkv[:, 8:16], qkv[:, 16:], None, None, None, i32([0]), i32([L - 1]), q_out, k, v,
                             i32(table), page)
    where = int(table[0, (L - 1) // page])
    assert torch.equal(v[where, :, (L - 1) % page], qkv[0, 16:])
    bounds = torch.zeros(pages, hk, 2, d, dtype=torch.bfloat16, device="cuda")
    fd.fdec_page_bounds(k, bounds, i32(table), None, i32([L]), page)
    for j in (0, 77, 150):
        rows = k[int(table[0, j]), :, : min(page, L - j * page)]
        assert torch.equal(bounds[int(table[0, j])], torch.stack([rows.amin(1), rows.amax(1)], 1))
    q = q_out.view(1, 1, 8, d)
    sel = fd.PageSelect(1, 1, page, 8, hk, d, 151, 30, "bf16")
    ids, counts, index = sel.run(q, bounds, i32(table), i32([L]))
    rows_of = torch.as_tensor(table[0]).cuda()
    want = select_reference(q, bounds[rows_of].contiguous(), np.arange(151)[None], [L], page, 30, 1, 1, True)
    assert np.array_equal(index.cpu().numpy(), want[2]) and np.array_equal(counts.cpu().numpy(), want[1])
    pd = fd.PagedDecode([30 * page], 1, page, 8, hk, d, "bf16")
    out, lse = torch.empty(1, 1, 8, d, device="cuda"), torch.empty(1, 1, 8, device="cuda")
    pd.run_selected(q, k, v, ids, counts, out, lse)
    assert pd.device_errors() == 0
    local = index.cpu().numpy()
    ref = attend_reference(q, k[rows_of].contiguous(), v[rows_of].contiguous(), local, counts.cpu().numpy(), 1 / math.sqrt(d))
    assert_attention(out, lse, *ref)


@gpu
def test_select_pages_of_other_layouts():
    """q off 16 bytes and head-major, bounds with the two sides apart, a page table wider than max_pages."""
    t, d, hk, hq, width = torch.float16, 128, 2, 8, 60
    table = np.random.default_rng(3).permutation(120).reshape(2, 60)
    wide = np.concatenate([table, np.full((2, 9), -1)], 1)
    lens = [60 * 16, 41 * 16 + 3]
    plain = bounds_like(120, hk, d, t, 4)
    sides = plain.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)      # [2, pages, Hk, D]
    heads = plain.transpose(0, 1).contiguous().transpose(0, 1)              # [Hk, pages, 2, D]
    q = torch.randn(2, 1, hq, d, generator=torch.Generator().manual_seed(5)).to(t).cuda()
    odd = torch.zeros(q.numel() + 1, dtype=t, device="cuda")[1:].view(q.shape)
    odd.copy_(q)
    major = q.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)          # [Hq, B, Q, D]
    want = select_reference(q, plain, table, lens, 16, 12, 1, 2, True)
    for qq in (q, odd, major):
        for bb in (plain, sides, heads):
            got = run_select(qq, bb, wide, lens, 16, 12, 1, 2, max_pages=width)
            for a, c in zip(got, want):
                assert np.array_equal(a, c)


@gpu
@pytest.mark.parametrize("seed", range(24))
def test_random_steps(seed):
    """Random shapes through the four operators in turn, each against its formula on what the last one wrote."""
    rng = np.random.default_rng(1000 + seed)
    d = int(rng.choice([64, 128, 128, 192, 256, 512]))
    kv = "fp8" if d in (128, 256) and rng.random() < 0.4 else ""
    dtype = str(rng.choice(["bf16", "f16"]))
    hk = int(rng.integers(1, 5))
    hq = hk * int(rng.choice([1, 2, 3, 4, 8, 17]))
    page = int(rng.choice([1, 2, 4, 8, 16, 32, 64, 128, 256]))
    seqs, q_len = int(rng.integers(1, 6)), int(rng.choice([1, 1, 2, 5]))
    width = int(rng.integers(3, 40))
    lens = [int(x) for x in rng.integers(q_len, width * page + 1, seqs)] if width * page > q_len else [q_len] * seqs
    width = max(width, -(-q_len // page))
    first, last = int(rng.integers(0, 3)), int(rng.integers(1, 4))
    budget = first + last + int(rng.integers(0, 12))
    rot = int(rng.choice([0, 16, d // 2, d]))
    layout = str(rng.choice(["hnd", "nhd", "interleaved"]))
    t = DT[dtype]
    pages = seqs * width + 1
    k, v = make_pool(pages, hk, page, d, kv or dtype, layout, seed)
    table = rng.permutation(pages)[: seqs * width].reshape(seqs, width)
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(seqs * q_len, hq + 2 * hk, d, generator=g).to(t).cuda()
    raw = qkv.clone()
    qw = (1 + 0.2 * torch.randn(d, generator=g)).to(t).cuda() if rng.random() < 0.7 else None
    cos_sin = None
    if rot:
        ang = np.arange(width * page)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
        cos_sin = torch.as_tensor(np.concatenate([np.cos(ang), np.sin(ang)], 1), dtype=torch.float32).cuda()
    bounds = torch.zeros(pages, hk, 2, d, dtype=t, device="cuda")
    fd.fdec_page_bounds(k, bounds, i32(table), None, i32(lens) - q_len, page)
    ks, vs = (0.125, 0.0625) if kv else (1.0, 1.0)
    inter = bool(rng.random() < 0.5)
    sd = fd.SparseDecode([width * page] * seqs, q_len, page, hq, hk, d, budget, dtype, first, last, kv_dtype=kv)
    out = torch.empty(seqs * q_len, 1, hq, d, dtype=t, device="cuda")
    lse = torch.empty(seqs * q_len, 1, hq, device="cuda")
    sd.step(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], qw, qw, cos_sin, k, v, bounds, i32(table), i32(lens), out,
            lse, interleaved=inter, k_scale=ks, v_scale=vs)
    assert sd.device_errors() == 0
    pos = np.concatenate([np.arange(L - q_len, L) for L in lens])
    assert_rounded(qkv[:, :hq].clone(), *norm_rope_reference(raw[:, :hq], qw, cos_sin, pos, inter, 1e-6))
    fresh = torch.zeros_like(bounds)
    fd.fdec_page_bounds(k, fresh, i32(table), None, i32(lens), page)
    assert torch.equal(fresh, bounds)
    q = qkv[:, :hq]
    ids, counts, _ = select_reference(q.reshape(seqs, q_len, hq, d), bounds, table, lens, page, budget, first, last, True)
    assert np.array_equal(sd.select.page_ids.cpu().numpy(), ids) and np.array_equal(sd.select.counts.cpu().numpy(), counts)
    ref = attend_reference(q.reshape(-1, 1, hq, d), k.float() * ks, v.float() * vs, ids, counts, 1 / math.sqrt(d))
    assert_attention(out, lse, *ref)


@gpu
def test_run_selected_over_e4m3_lists_in_splits_of_their_own():
    """128 lists of 2048 tokens: the planner's splits (of fdec_run_scaled) and those of the lists differ; both run from
    one plan and workspace, and the device errors of either are read."""
    rows, hq, hk, d, page, budget = 16, 16, 8, 128, 16, 128
    k, v = make_pool(400, hk, page, d, "fp8", "nhd", 6)
    ids, counts = selected_lists(rows, hk, page, budget, 400, seed=6)
    q = torch.randn(rows, 1, hq, d, generator=torch.Generator().manual_seed(7)).half().cuda()
    pd = fd.PagedDecode([budget * page] * rows, 1, page, hq, hk, d, "f16", kv_dtype="fp8")
    out, lse = torch.empty(rows, 1, hq, d, device="cuda"), torch.empty(rows, 1, hq, device="cuda")
    pd.run_selected(q, k, v, i32(ids), i32(counts), out, lse, k_scale=0.125, v_scale=0.25)
    assert pd.device_errors() == 0
    ref = attend_reference(q, k.float() * 0.125, v.float() * 0.25, ids, counts, 1 / math.sqrt(d))
    assert_attention(out, lse, *ref)
    pd.run(q, k, v, i32(ids[:, 0]), i32(counts[:, 0]), out, lse, k_scale=0.125, v_scale=0.25)
    assert pd.device_errors() == 0
    ref = attend_reference(q, k.float() * 0.125, v.float() * 0.25, ids[:, :1].repeat(hk, 1), counts[:, :1].repeat(hk, 1),
                           1 / math.sqrt(d))
    assert_attention(out, lse, *ref)
    bad = ids.copy()
    bad[0, 0, 3] = 400
    pd.run_selected(q, k, v, i32(bad), i32(counts), out, lse)
    assert pd.device_errors() == fd.DEVERR_PAGE_ID and pd.device_errors() == 0
    pd.run(q, k, v, i32(bad[:, 0]), i32(counts[:, 0]), out, lse, k_scale=0.125, v_scale=0.25)
    assert pd.device_errors() == fd.DEVERR_PAGE_ID
