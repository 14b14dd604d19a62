"""Block-sparse decoding where it can go wrong: the precision of attention over code caches, error flags, codes at
ties, stream order, refusals of tensors that are not on the GPU, plans with and without page lists.

Tolerances are derived beside each test."""
import math
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_split_kv_gather_gb300 as fd
from tests.test_sparse_decode import (DT, assert_attention, attend_reference, bounds_like, check_select, cpu_rows, gpu, i32,
                                       make_pool, select_reference, selected_lists)


# ------------------------------------------------------------------------------------------- attention over codes

@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,hq,hk,page,budget,rows", [(128, 8, 2, 16, 3, 40), (256, 8, 2, 16, 3, 40),
                                                      (128, 16, 8, 16, 128, 16), (256, 8, 4, 64, 40, 5),
                                                      (128, 24, 2, 16, 5, 30), (256, 64, 2, 32, 20, 3), (128, 70, 2, 64, 30, 4)])
def test_run_selected_over_codes_keeps_the_probabilities(d, hq, hk, page, budget, rows, dtype):
    """fp32 outputs over E4M3 lists, as near as those over 16-bit lists.

    Relative to sum p |v| / sum p: the logits are sums of D products in 16 fp32 accumulations of the tensor cores
    (2^-23 each, of sum |q k| scale log2(e) < 3 for the queries here: 2^-18 at most), the exponential 2^-22, a
    probability as two f16 values 2^-23, the sum over a list's tokens two of 16 accumulations and the merges 2^-18: in
    all below 2^-16.  (One f16 value alone is off by up to 2^-12.)"""
    t = DT[dtype]
    pool = 2 * budget + 5
    k, v = make_pool(pool, hk, page, d, "fp8", "nhd", seed=d)
    ids, counts = selected_lists(rows, hk, page, budget, pool, seed=rows)
    q = (torch.randn(rows, 1, hq, d, generator=torch.Generator().manual_seed(d)) / 8).to(t).cuda()
    ks, vs = 0.125, 0.25
    pd = fd.PagedDecode([budget * page] * rows, 1, page, hq, hk, d, dtype, kv_dtype="fp8")
    out = torch.full((rows, 1, hq, d), float("nan"), device="cuda")
    pd.run_selected(q, k, v, i32(ids), i32(counts), out, None, k_scale=ks, v_scale=vs)
    assert pd.device_errors() == 0
    kk, vv = k.float() * ks, v.float() * vs
    ref, _ = attend_reference(q, kk, vv, ids, counts, 1 / math.sqrt(d))
    mag, _ = attend_reference(q, kk, vv.abs(), ids, counts, 1 / math.sqrt(d))
    off = np.abs(out.double().cpu().numpy() - ref)
    assert (off <= 2.0 ** -16 * mag).all(), (off / np.maximum(mag, 1e-30)).max()


# ----------------------------------------------------------------------------------------------------- page bounds

@gpu
@pytest.mark.parametrize("hk,d,page", [(1, 128, 16), (2, 64, 8), (3, 128, 16), (1, 512, 256)])
@pytest.mark.parametrize("bad", range(6))
def test_page_bounds_flags_any_one_sequence(hk, d, page, bad):
    """A bad length or begin of one sequence alone, whichever it is: four of them share a CTA of one-warp units."""
    k, _ = make_pool(12, hk, page, d, "bf16", "hnd", 1)
    bounds = torch.zeros(12, hk, 2, d, dtype=torch.bfloat16, device="cuda")
    table = i32(np.arange(12).reshape(6, 2))
    for lens, begins in (({bad: 2 * page + 1}, {}), ({bad: -1}, {}), ({}, {bad: -1})):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        fd.fdec_page_bounds(k, bounds, table, i32([begins.get(b, page) for b in range(6)]),
                            i32([lens.get(b, 2 * page) for b in range(6)]), page, expected_tokens=1, device_errors=err)
        assert int(err.item()) == fd.DEVERR_SEQ_LEN
    err.zero_()
    fd.fdec_page_bounds(k, bounds, table, i32([page] * 6), i32([2 * page] * 6), page, expected_tokens=1, device_errors=err)
    assert int(err.item()) == 0


# ------------------------------------------------------------------------------------------- norm, rotation, append

def codes_of(x, scale):
    """E4M3 codes of x / scale, an fp32 division, to nearest even, saturating."""
    return (x.float() / torch.tensor(scale, dtype=torch.float32)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


@gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("scale", [7 / 256, 15 / 256, 0.03, 0.0234375, 3e-6, 1.7, 2 - 2.0 ** -23, 1 - 2.0 ** -24, 5e7])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_codes_are_those_of_the_quotient(dtype, scale, d):
    """Every 16-bit value as a value row, bit for bit; as a key those whose quotient's code a product with the
    reciprocal would miss (ties among them): rows of +-1 with eps 0 have norm 1, so the key is the weight itself."""
    t = DT[dtype]
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(t)
    x = torch.cat([x[torch.isfinite(x.float())], torch.tensor([math.inf, -math.inf, math.nan], dtype=t)])
    s = torch.tensor(scale, dtype=torch.float32)
    product = (x.float() * (1 / s)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    keys = torch.cat([x[codes_of(x, scale) != product], x[:-3:61]])[:d]
    weight = torch.ones(d, dtype=t)
    weight[:len(keys)] = keys
    n = -(-len(x) // d)
    v_new = torch.zeros(n * d, dtype=t)
    v_new[:len(x)] = x
    v_new = v_new.view(n, 1, d)
    sign = torch.where(torch.rand(n, 1, d, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0).to(t)
    page = 16
    pages = -(-n // page)
    k, v = (torch.zeros(pages, 1, page, d, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    q = torch.zeros(n, 1, d, dtype=t, device="cuda")
    fd.fdec_norm_rope_append(q, sign.cuda(), v_new.cuda(), None, weight.cuda(), None, i32(np.zeros(n)), i32(np.arange(n)), q,
                             k, v, i32(np.arange(pages)[None]), page, eps=0.0, k_scale=scale, v_scale=scale)
    got_k, got_v = (c.view(torch.uint8).reshape(-1, 1, d)[:n].cpu() for c in (k, v))
    magnitude = lambda c: torch.where((c & 0x7F) == 0, 0, c)  # noqa: E731  (the sign of a zero is not compared)
    assert torch.equal(magnitude(got_v), magnitude(codes_of(v_new, scale)))
    assert torch.equal(magnitude(got_k), magnitude(codes_of(sign * weight, scale)))


# ---------------------------------------------------------------------------------------------------- stream order

def kernel_bodies():
    """(file, name, body) of every __global__ function of the library's sources, comments taken out."""
    root = os.path.join(os.path.dirname(fd.__file__), "csrc")
    for name in sorted(os.listdir(root)):
        text = open(os.path.join(root, name)).read()
        text = re.sub(r"//[^\n]*", "", text)
        for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\((?=[^;{]*\{)", text):
            at = text.index("{", m.end())
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                if depth == 0:
                    break
                end += 1
            yield name, re.search(r"(\w+)\s*\((?:const\s|AppendParams)", text[m.start():at]).group(1), text[at:end]


def test_dependent_kernels_wait_on_every_way_out():
    """A kernel that is launched as a programmatic dependent completes only after the kernel before it: no return comes
    before a wait.  (The kernel after it waits for this one alone.)"""
    seen = {}
    for file, name, body in kernel_bodies():
        if "griddepcontrol.wait" not in body:
            continue
        first = body.index("griddepcontrol.wait")
        for m in re.finditer(r"\breturn;", body):
            assert m.start() > first, f"{file}: {name} returns before its wait"
        seen[name] = file
    assert {"norm_rope_kernel", "page_bounds_kernel", "score_pages_kernel", "choose_pages_kernel", "share_merge_kernel",
            "reduce_kernel", "split_mma_kernel", "split_mma_persist_kernel"} <= set(seen), seen


def test_dependent_kernels_read_fresh_data_with_ordinary_loads():
    """Read-only loads are for data that nobody writes while the kernel is resident; a dependent kernel is resident
    beside the one that writes its inputs."""
    root = os.path.join(os.path.dirname(fd.__file__), "csrc")
    for name in ("norm_rope.cu", "page_bounds.cu", "select_pages.cu"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(root, name)).read())
        assert "__ldg" not in text and ".nc." not in text, name
    text = re.sub(r"//[^\n]*", "", open(os.path.join(root, "split_persist_kernel.cuh")).read())
    assert not re.search(r"__ldg\([^;]*(seq_lens|pt \+|page_table)", text)


@gpu
def test_select_pages_of_short_rows_keeps_stream_order():
    """Inputs overwritten right after a selection in which every row is short (the scoring has nothing to do), and
    again after one in which every row is long."""
    t, d, hk, hq, page, width, budget, b = torch.bfloat16, 128, 2, 8, 16, 64, 12, 40
    table = np.random.default_rng(3).permutation(b * width).reshape(b, width)
    bounds = bounds_like(b * width, hk, d, t, 4)
    q = torch.randn(b, 1, hq, d, generator=torch.Generator().manual_seed(5)).to(t).cuda()
    short, full = [x % (budget * page + 1) for x in range(0, 5 * b, 5)], [width * page - x for x in range(b)]
    want = [select_reference(q, bounds, table, n, page, budget, 1, 1, True) for n in (short, full)]
    tb, lens = i32(table), i32(short)
    both = [i32(short), i32(full)]
    sel = fd.PageSelect(b, 1, page, hq, hk, d, width, budget, "bf16")
    got = []
    for i in range(60):
        lens.copy_(both[i % 2])
        got.append([x.clone() for x in sel.run(q, bounds, tb, lens)])
    lens.zero_()
    assert sel.device_errors() == 0
    for i, out in enumerate(got):
        for a, w in zip(out, want[i % 2]):
            assert np.array_equal(a.cpu().numpy(), w), i


# ---------------------------------------------------------------------------------------------- refusals (no device)

def test_tensors_that_are_not_on_a_gpu_are_refused():
    """Well-formed calls on host tensors: past every check of the library's own, and refused before a launch."""
    def refused(fn, *args, **kw):
        for stream in (0, None):
            with pytest.raises(ValueError, match="CUDA device"):
                fn(*args, stream=stream, **kw)

    rows = cpu_rows()
    refused(fd.fdec_norm_rope_append, **rows)
    k, bounds = torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(4, 2, 2, 64, dtype=torch.float16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    refused(fd.fdec_page_bounds, k, bounds, i(1, 4), None, i(1), 16)
    total = fd.fdec_select_pages_workspace(1, 1, 2, 8)
    buf = torch.zeros(total + 256, dtype=torch.uint8)
    ws = buf[(-buf.data_ptr()) % 256:][:total]
    refused(fd.fdec_select_pages, torch.zeros(1, 1, 4, 64, dtype=torch.float16), bounds, i(1, 8), i(1), 16, 8, 4, i(1, 2, 4),
            i(1, 2), None, ws)
    # the library's own refusals come first, and later calls of the thread are not held back
    with pytest.raises(fd.FdecError):
        fd.fdec_page_bounds(k[..., :60], bounds[..., :60], i(1, 4), None, i(1), 16, stream=0)
    with pytest.raises(ValueError):
        fd.fdec_page_bounds(k, bounds, i(1, 4), None, i(1), 16, device_errors=torch.zeros(1).double(), stream=0)
    fd.fdec_norm_rope_append(stream=0, **cpu_rows(n=0))  # no token: nothing to refuse


@gpu
def test_calls_use_the_current_stream_of_the_tensors_device():
    """After refusals on host tensors, a call on the GPU still launches, on the stream that is current."""
    test_tensors_that_are_not_on_a_gpu_are_refused()
    k, _ = make_pool(4, 2, 16, 64, "f16", "hnd", 3)
    bounds = torch.zeros(4, 2, 2, 64, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    table, lens = i32(np.arange(4)[None]), i32([64])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fd.fdec_page_bounds(k, bounds, table, None, lens, 16)
        copy = bounds.clone()
    side.synchronize()
    assert torch.equal(copy, torch.stack([k.amin(2), k.amax(2)], 2))


def test_a_workspace_of_repeated_bytes_is_refused():
    """numel bytes that are not all there: a tensor expanded from one byte."""
    total = fd.fdec_select_pages_workspace(1, 1, 2, 8)
    buf = torch.zeros(512, dtype=torch.uint8)
    at = (-buf.data_ptr()) % 256
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="contiguous"):
        fd.fdec_select_pages(torch.zeros(1, 1, 4, 64, dtype=torch.float16), torch.zeros(4, 2, 2, 64, dtype=torch.float16),
                             i(1, 8), i(1), 16, 8, 4, i(1, 2, 4), i(1, 2), None, buf[at:at + 1].expand(total), stream=0)


# ------------------------------------------------------------------------------------ plans with and without page lists

def test_plans_without_page_lists_have_no_workspace_for_them():
    """The workspace of fdec_plan is that of its splits: (capacities, page, Hq, Hk, D, cache) and bytes at 152 SMs."""
    for caps, page, hq, hk, d, kv, want in (
            ([2048] * 64, 64, 32, 8, 512, "", 8424960), ([32768] * 64, 64, 32, 8, 128, "", 5331456),
            ([262144], 64, 32, 4, 128, "", 1266688), ([700] * 5, 16, 4, 1, 64, "", 59904),
            ([2048] * 16, 16, 32, 8, 128, "fp8", 1066752), ([4096] * 16, 64, 16, 4, 256, "fp8", 1323008)):
        plan = fd.fdec_plan(caps, 1, page, hq, hk, d, num_sms=152, kv_dtype=kv)
        info = fd.fdec_plan_get_selected_info(plan)
        assert plan.workspace_bytes == want and not info["page_lists"] and not info["share_ctas"]
        # all that the other entry points see of a plan for page lists is the same
        lists = fd.fdec_plan(caps, 1, page, hq, hk, d, num_sms=152, kv_dtype=kv, page_lists=True)
        a, b = fd.fdec_plan_get_info(plan), fd.fdec_plan_get_info(lists)
        more = b.pop("workspace_bytes") - a.pop("workspace_bytes")
        assert a == b and np.array_equal(fd.fdec_plan_get_splits(plan), fd.fdec_plan_get_splits(lists))
        assert fd.fdec_plan_get_selected_info(lists)["page_lists"] == 1 and 0 <= more < 11 << 20
    info = fd.fdec_plan_get_selected_info(fd.fdec_plan([2048] * 64, 1, 16, 32, 8, 128, num_sms=152, page_lists=True))
    assert info["page_lists"] == 1 and info["share_ctas"] == 304 and info["launches"] == 2
    with pytest.raises(ValueError):
        fd.fdec_plan([64], 2, 16, 4, 2, 64, num_sms=152, page_lists=True)
    with pytest.raises(fd.FdecError) as e:
        fd.fdec_plan([64], 1, 16, 4, 2, 128, num_sms=152, page_lists=True, kv_dtype="q8_0")
    assert e.value.status_name == "FDEC_ERR_UNSUPPORTED"


@gpu
@pytest.mark.parametrize("kv", ["", "fp8"])
def test_run_selected_with_either_kind_of_plan(kv):
    rows, hq, hk, d, page, budget = 24, 16, 4, 128, 16, 60
    k, v = make_pool(2 * budget, hk, page, d, kv or "bf16", "hnd", 3)
    ids, counts = selected_lists(rows, hk, page, budget, 2 * budget, seed=2)
    q = torch.randn(rows, 1, hq, d, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    ref = attend_reference(q, k.float() * 0.125, v.float() * 0.25, ids, counts, 1 / math.sqrt(d))
    for page_lists in (True, False, None):
        pd = fd.PagedDecode([budget * page] * rows, 1, page, hq, hk, d, "bf16", kv_dtype=kv, page_lists=page_lists)
        assert fd.fdec_plan_get_selected_info(pd.plan)["page_lists"] == (page_lists is not False)
        out, lse = torch.empty(rows, 1, hq, d, device="cuda"), torch.empty(rows, 1, hq, device="cuda")
        pd.run_selected(q, k, v, i32(ids), i32(counts), out, lse, k_scale=0.125, v_scale=0.25)
        assert pd.device_errors() == 0
        assert_attention(out, lse, *ref)


# ------------------------------------------------------------------------------------------------- shares of lists

@gpu
@pytest.mark.parametrize("d,hq,hk,page,rows,caps", [
    (128, 32, 8, 16, 40, (2048, 64, 640, 1)), (64, 4, 4, 64, 64, (640, 1280)), (192, 8, 4, 8, 33, (1280, 320, 0)),
    (256, 16, 4, 32, 12, (960, 128)), (512, 8, 4, 32, 12, (640, 128)), (128, 40, 2, 16, 30, (2048, 100, 300))])
def test_run_selected_over_lists_of_unequal_capacities(d, hq, hk, page, rows, caps):
    """Shares of lists whose capacities differ (each is read on the device), ragged, full and empty, the same in every
    run whatever ran before."""
    cap = [caps[r % len(caps)] for r in range(rows)]
    width = max(1, -(-max(cap) // page))
    pool = 2 * width + 3
    k, v = make_pool(pool, hk, page, d, "bf16", "nhd", seed=d)
    q = torch.randn(rows, 1, hq, d, generator=torch.Generator().manual_seed(rows)).bfloat16().cuda()
    pd = fd.PagedDecode(cap, 1, page, hq, hk, d, "bf16", path=fd.FDEC_PATH_MMA)
    assert fd.fdec_plan_get_selected_info(pd.plan)["share_ctas"] > 0
    results = []
    for kind in ("ragged", "full", "empty", "ragged"):
        rng = np.random.default_rng(d)
        ids = rng.integers(0, pool, (rows, hk, width)).astype(np.int32)
        full = np.repeat(np.asarray(cap)[:, None], hk, 1)
        counts = {"full": full, "empty": 0 * full}.get(kind, rng.integers(0, full + 1)).astype(np.int32)
        out, lse = torch.full((rows, 1, hq, d), math.nan, device="cuda"), torch.full((rows, 1, hq), math.nan, device="cuda")
        pd.run_selected(q, k, v, i32(ids), i32(counts), out, lse)
        assert pd.device_errors() == 0
        assert_attention(out, lse, *attend_reference(q, k, v, ids, counts, 1 / math.sqrt(d)))
        results.append((out, lse))
    assert torch.equal(results[0][0], results[3][0]) and torch.equal(results[0][1], results[3][1])
    # counts above one list's capacity are clamped to it, and flagged
    over = np.asarray(counts)
    over[0] = cap[0] + 1
    pd.run_selected(q, k, v, i32(ids), i32(over), out, lse)
    assert pd.device_errors() == fd.DEVERR_SEQ_LEN
    over[0] = cap[0]
    assert_attention(out, lse, *attend_reference(q, k, v, ids, over, 1 / math.sqrt(d)))


@gpu
def test_run_selected_of_more_lists_than_shares_count():
    """4096 lists run in shares, 4100 as planned (every fourth token's lists longer than the others')."""
    d, page, width = 64, 64, 10
    k, v = make_pool(40, 4, page, d, "f16", "hnd", seed=1)
    for rows in (1024, 1025):
        ids, counts = selected_lists(rows, 4, page, width, 40, seed=rows)
        cap = np.asarray([page if r % 4 else width * page for r in range(rows)], dtype=np.int32)
        counts = np.minimum(counts, cap[:, None])
        q = torch.randn(rows, 1, 4, d, generator=torch.Generator().manual_seed(rows)).half().cuda()
        pd = fd.PagedDecode(cap, 1, page, 4, 4, d, "f16")
        assert (fd.fdec_plan_get_selected_info(pd.plan)["share_ctas"] > 0) == (rows == 1024)
        out, lse = torch.full((rows, 1, 4, d), math.nan, device="cuda"), torch.full((rows, 1, 4), math.nan, device="cuda")
        pd.run_selected(q, k, v, i32(ids), i32(counts), out, lse)
        assert pd.device_errors() == 0
        assert_attention(out, lse, *attend_reference(q, k, v, ids, counts, 1 / math.sqrt(d)))


@gpu
def test_run_selected_as_planned_equals_run_bit_for_bit():
    """Planned splits of one block: the partials and the reduction are fdec_run's."""
    rows, hq, hk, d, page, budget = 3, 32, 2, 128, 16, 20
    k, v = make_pool(80, hk, page, d, "bf16", "hnd", 4)
    ids, counts = selected_lists(rows, 1, page, budget, 80, seed=4)
    q = torch.randn(rows, 1, hq, d, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    pd = fd.PagedDecode([budget * page] * rows, 1, page, hq, hk, d, "bf16", path=fd.FDEC_PATH_MMA, blocks_per_split=1)
    assert fd.fdec_plan_get_selected_info(pd.plan)["share_ctas"] == 0
    a, b = (torch.full((rows, 1, hq, d), math.nan, device="cuda") for _ in range(2))
    la, lb = (torch.full((rows, 1, hq), math.nan, device="cuda") for _ in range(2))
    pd.run(q, k, v, i32(ids[:, 0]), i32(counts[:, 0]), a, la)
    pd.run_selected(q, k, v, i32(ids.repeat(hk, 1)), i32(counts.repeat(hk, 1)), b, lb)
    assert pd.device_errors() == 0 and torch.equal(a, b) and torch.equal(la, lb)


# --------------------------------------------------------------------------------------------------- page selection

def special_bounds(kind, pages, hk, d, t, seed):
    """Bounds of `pages` pages of which some hold what `kind` says; the pages that do."""
    b = bounds_like(pages, hk, d, t, seed)
    rng = np.random.default_rng(seed)
    some = torch.as_tensor(np.sort(rng.choice(pages, max(1, pages // 2), replace=False))).cuda()
    one = some[len(some) // 2:len(some) // 2 + 1]
    if kind == "one nan":
        b[one, :, 0, 3] = math.nan
    elif kind == "one infinity":
        b[one, :, 1, 3] = math.inf
    elif kind == "many nan":
        b[some, :, :, d - 1] = math.nan
    elif kind == "many infinities":
        b[some, :, 1] = math.inf
        b[some, :, 0] = -math.inf
    elif kind == "many minus infinities":  # both rows, so that every query is led to -inf or NaN
        b[some] = -math.inf
    elif kind == "all of them":
        third = len(some) // 3
        b[some[:third], :, 1, 0] = math.inf
        b[some[third:2 * third], :, :, 1] = -math.inf
        b[some[2 * third:], 0, 0, 2] = math.nan
    elif kind == "zeros":
        b[:] = 0
    elif kind == "many zeros":
        b[some] = 0
    elif kind == "largest":
        b[some, :, 1, :2] = torch.finfo(t).max
    return b


@gpu
@pytest.mark.parametrize("kind", ["one nan", "one infinity", "many nan", "many infinities", "many minus infinities",
                                  "all of them", "zeros", "many zeros", "largest"])
@pytest.mark.parametrize("dtype,d,hq,hk,q_len,pages", [("bf16", 128, 8, 2, 1, 1500), ("f16", 64, 4, 4, 2, 700),
                                                       ("bf16", 192, 4, 2, 4, 900), ("f16", 512, 6, 2, 1, 640),
                                                       ("bf16", 256, 8, 1, 3, 5000)])
def test_select_pages_of_special_bounds(dtype, d, hq, hk, q_len, pages, kind):
    t = DT[dtype]
    table = np.random.default_rng(pages).permutation(2 * pages).reshape(2, pages)
    bounds = special_bounds(kind, 2 * pages, hk, d, t, seed=pages)
    g = torch.Generator().manual_seed(d)
    q = torch.randn(2, q_len, hq, d, generator=g)
    lens = [pages * 16, pages * 16 - 70]
    for budget in (12, pages // 2 - 20, pages - 30):
        check_select(q.to(t).cuda(), bounds, table, lens, 16, budget, 1, 2)
    check_select(q.abs().to(t).cuda(), bounds, table, lens, 16, 40, 0, 1)  # weights of one sign: 0 x infinity is NaN


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["zero", "nan", "infinity", "minus infinity", "largest", "smallest"])
def test_select_pages_of_special_queries(dtype, kind):
    """One head (its group's scores are all NaN or infinite), one element, or every element; weights that are finite
    in 64 bits alone."""
    t = DT[dtype]
    value = {"zero": 0.0, "nan": math.nan, "infinity": math.inf, "minus infinity": -math.inf,
             "largest": torch.finfo(t).max, "smallest": torch.finfo(t).smallest_normal}[kind]
    pages, hq, hk, d = 900, 8, 2, 128
    table = np.random.default_rng(1).permutation(pages).reshape(1, pages)
    q = torch.randn(1, 1, hq, d, generator=torch.Generator().manual_seed(2)).to(t)
    element, head, every = q.clone(), q.clone(), torch.full_like(q, value)
    element[0, 0, 1, 5] = value
    head[0, 0, 6] = value
    for bounds in (bounds_like(pages, hk, d, t, 3), special_bounds("all of them", pages, hk, d, t, 4),
                   special_bounds("many zeros", pages, hk, d, t, 5)):
        for x in (element, head, every):
            for budget in (20, 500):
                check_select(x.cuda(), bounds, table, [pages * 16 - 1], 16, budget, 1, 1)


@gpu
def test_select_pages_leaves_bad_page_ids_behind_many_nan_pages():
    """Infinite scores of more pages than are compared each with each, and pages outside the pool, in one row."""
    pages, budget = 2000, 700
    bounds = bounds_like(pages, 1, 64, torch.float16, 2)
    bounds[400:1000, :, 1, 7] = math.nan
    q = torch.randn(1, 1, 4, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    table = np.arange(pages)[None]
    bad = table.copy()
    bad[0, [3, 555, 1500]] = [pages, -9, 1 << 30]
    want = select_reference(q, bounds, table, [pages * 16], 16, budget + 3, 1, 1, True)[2][0, 0]
    want = [j for j in want if j not in (3, 555, 1500)]
    sel = fd.PageSelect(1, 1, 16, 4, 1, 64, pages, budget, "f16")
    index = sel.run(q, bounds, i32(bad), i32([pages * 16]))[2].cpu().numpy()[0, 0]
    assert sel.device_errors() == fd.DEVERR_PAGE_ID
    assert not np.isin([3, 555, 1500], index).any()
    # (of the reference's budget + 3 pages, those that are not the bad ones, without its last free ones)
    scores = lambda j: math.inf if 400 <= j < 1000 else 0  # noqa: E731
    assert [j for j in want if scores(j)] == [j for j in index if scores(j)] and set(index) <= set(want)


@gpu
def test_special_values_do_not_make_a_row_slow():
    """One bad key in a long cache, an unwritten cache, a padded query: the call stays within a few times the ordinary
    one (it was a hundred times).  4096 pages, four rows; the best of several replays."""
    pages, hq, hk, d = 4096, 32, 4, 128
    table, lens = i32(np.random.default_rng(1).permutation(pages)[None]), i32([pages * 64])
    sel = fd.PageSelect(1, 1, 64, hq, hk, d, pages, 64, "bf16", 1, 2)
    ordinary = torch.randn(1, 1, hq, d, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()

    def best(q, bounds):
        sel.run(q, bounds, table, lens)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(10):
                sel.run(q, bounds, table, lens)
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    usual = best(ordinary, bounds_like(pages, hk, d, torch.bfloat16, 3))
    for kind in ("one nan", "one infinity", "zeros"):
        assert best(ordinary, special_bounds(kind, pages, hk, d, torch.bfloat16, 3)) < 10 * usual, kind
    for value in (0.0, math.nan):
        assert best(torch.full_like(ordinary, value), bounds_like(pages, hk, d, torch.bfloat16, 3)) < 10 * usual, value


_LITTLE_MEMORY = r'''
import resource, sys
sys.path.insert(0, sys.argv[1])
import paged_split_kv_gather_gb300 as fd
fd.fdec_plan([64], 1, 64, 4, 1, 128, num_sms=152)  # everything is loaded
now = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (now + (48 << 20), resource.RLIM_INFINITY))
for page_lists in (False, True):
    try:
        fd.fdec_plan([262144] * 4000, 1, 64, 32, 4, 128, blocks_per_split=1, num_sms=152, page_lists=page_lists)
    except fd.FdecError as e:
        assert "memory" in str(e), e
    else:
        raise AssertionError("planned")
fd.fdec_plan([64], 1, 64, 4, 1, 128, num_sms=152)
print("refused")
'''


def test_plans_without_host_memory_are_refused():
    """The plan's lists do not fit the process: a status, and the process goes on."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _LITTLE_MEMORY, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused" in r.stdout, (r.returncode, r.stdout, r.stderr[-2000:])
