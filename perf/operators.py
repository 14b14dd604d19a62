"""Block-sparse decoding over the paged KV cache: the four operators of a step, their plain forms and their cases.

A decoding step over a long context takes the fused projection's rows of the new tokens and

  norm_rope_append  norms every query and key head (RMS), rotates it by its position, and writes the keys and values
                    into the pages of the cache (16-bit, or E4M3 codes with a scale);
  page_bounds       writes the elementwise minimum and maximum of the keys of every page that changed;
  select_pages      bounds every page's logits for each query token and KV head from those two rows, and takes the
                    pages with the largest bounds (with the first and the newest ones always);
  run_selected      attends to the tokens of the taken pages.

``own`` False computes each with elementary torch operations, True through the library's entry points.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}
_DEV = "cuda"
_EPS = 1e-6
_K_SCALE, _V_SCALE = 0.03125, 0.0234375  # scales of the E4M3 caches: unit-variance rows use most of the range


# ---------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence decodes one token of a 32/4-head layer into a cache of 64-token pages: latency
        _rows("rows_decode_1", seqs=1, tokens=1, start=131071, hq=32, hk=4, d=128, page=64, dtype="bf16"),
        # a serving batch of 64, wide heads with half of each rotated, one tensor for K and V, small pages
        _rows("rows_decode_64", seqs=64, tokens=1, start=32767, hq=16, hk=8, d=256, page=16, dtype="f16", rot=128,
              layout="interleaved"),
        # ragged chunks of prompts into an 8-bit cache, adjacent pairs rotated
        _rows("rows_chunks_fp8", seqs=4, tokens=509, start=7683, hq=32, hk=8, d=128, page=16, dtype="bf16", kv="fp8",
              interleaved=True, layout="nhd"),
        # a whole prompt
        _rows("rows_prompt", seqs=1, tokens=32768, start=0, hq=32, hk=8, d=128, page=64, dtype="bf16"),
        # after a decoding step of a batch of 64: the newest page of each sequence
        _bounds("bounds_decode_64", seqs=64, new=1, length=32768, hk=8, d=256, page=16, dtype="f16",
                layout="interleaved"),
        # after a prompt of 131072 tokens
        _bounds("bounds_prompt", seqs=1, new=131072, length=131072, hk=4, d=128, page=64, dtype="bf16"),
        # one sequence of 262144 tokens, 64 pages of 64 tokens for every KV head
        _select("select_long", seqs=1, q_len=1, length=262144, hq=32, hk=4, d=128, page=64, budget=64, dtype="bf16"),
        # a batch of 64 of ragged lengths, pages of 16
        _select("select_batch", seqs=64, q_len=1, length=32768, hq=16, hk=8, d=192, page=16, budget=128, dtype="f16"),
        # speculative decoding: four query tokens, each with its own pages
        _select("select_spec", seqs=4, q_len=4, length=8196, hq=32, hk=8, d=128, page=16, budget=64, dtype="bf16"),
        # the attention of one long sequence: 4096 of its tokens for each KV head
        _attend("attend_long", rows=1, hq=32, hk=4, d=128, page=64, budget=64, dtype="bf16"),
        # the attention of a batch of 64: 2048 tokens for each KV head, some of them with less or none
        _attend("attend_batch", rows=64, hq=32, hk=8, d=128, page=16, budget=128, dtype="bf16", ragged=True),
        # four sequences with four query tokens each over an 8-bit cache
        _attend("attend_spec_fp8", rows=16, hq=32, hk=8, d=128, page=16, budget=128, dtype="bf16", kv="fp8"),
    ]


def _rows(name, *, seqs, tokens, start, hq, hk, d, page, dtype, kv="", rot=0, interleaved=False, layout="hnd"):
    return {"name": name, "op": "norm_rope_append", "seqs": seqs, "tokens": tokens, "start": start, "hq": hq, "hk": hk,
            "d": d, "page": page, "dtype": dtype, "kv": kv, "rot": rot or d, "interleaved": interleaved,
            "layout": layout}


def _bounds(name, *, seqs, new, length, hk, d, page, dtype, kv="", layout="hnd"):
    return {"name": name, "op": "page_bounds", "seqs": seqs, "new": new, "length": length, "hk": hk, "d": d,
            "page": page, "dtype": dtype, "kv": kv, "layout": layout}


def _select(name, *, seqs, q_len, length, hq, hk, d, page, budget, dtype, first=1, last=2):
    return {"name": name, "op": "select_pages", "seqs": seqs, "q_len": q_len, "length": length, "hq": hq, "hk": hk,
            "d": d, "page": page, "budget": budget, "dtype": dtype, "first": first, "last": last}


def _attend(name, *, rows, hq, hk, d, page, budget, dtype, kv="", ragged=False, layout="hnd"):
    return {"name": name, "op": "run_selected", "rows": rows, "hq": hq, "hk": hk, "d": d, "page": page,
            "budget": budget, "dtype": dtype, "kv": kv, "ragged": ragged, "layout": layout}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rows", "rows", "bounds", "select", "select", "attend", "attend"])
    hq, hk = rng.choice([(32, 4), (32, 8), (16, 8), (4, 1), (12, 3), (8, 8)])
    dtype = rng.choice(["bf16", "f16"])
    d = rng.choice([64, 128, 128, 192, 256, 512])
    page = rng.choice([8, 16, 16, 32, 64, 64, 128])
    layout = rng.choice(["hnd", "nhd", "interleaved"])
    kv = rng.choice(["", "", "fp8"]) if d in (128, 256) else ""
    if op == "rows":
        seqs = _log(rng, 1, 64)
        tokens = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 32768 * 48 * 128 // ((hq + 2 * hk) * d * seqs)))
        case = _rows("", seqs=seqs, tokens=min(tokens, 32768), start=rng.randrange(65536), hq=hq, hk=hk, d=d,
                     page=page, dtype=dtype, kv=kv, rot=rng.choice([d, d, d // 2, 32]),
                     interleaved=rng.random() < 0.4, layout=layout)
    elif op == "bounds":
        seqs = _log(rng, 1, 64)
        length = _log(rng, 64, max(64, 131072 * 4 * 128 // (hk * d * seqs)))
        new = rng.choice([1, length, _log(rng, 1, length)])
        case = _bounds("", seqs=seqs, new=new, length=length, hk=hk, d=d, page=page, dtype=dtype, kv=kv, layout=layout)
    elif op == "select":
        seqs, q_len = rng.choice([(1, 1), (_log(rng, 1, 64), 1), (_log(rng, 1, 8), rng.randrange(2, 9))])
        page = max(page, 16)
        pages = _log(rng, 8, max(16, 64 * 2048 * 8 * 192 // (seqs * q_len * hk * d)))
        case = _select("", seqs=seqs, q_len=q_len, length=min(pages, 8192) * page - rng.randrange(page), hq=hq, hk=hk,
                       d=d, page=page, budget=_log(rng, 8, 256), dtype=dtype, first=rng.randrange(3),
                       last=rng.randrange(1, 4))
    else:
        rows = _log(rng, 1, 64)
        budget = _log(rng, 1, max(2, min(512, 64 * 8 * 2048 * 128 // (rows * hk * d * page))))
        case = _attend("", rows=rows, hq=hq, hk=hk, d=d, page=page, budget=budget, dtype=dtype, kv=kv,
                       ragged=rng.random() < 0.5, layout=layout)
    del case["name"]
    return case


# --------------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(seed), random.Random(seed)


def _pools(g, pages, hk, page, d, dtype, kv, layout):
    """K and V as views [page, kv_head, slot, dim] of one or two tensors."""
    def values(shape):
        if kv:  # codes of unit-variance rows
            return (torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32) / _K_SCALE).clamp_(-448, 448).to(_TYPES[kv])
        return torch.randn(shape, generator=g, device=_DEV, dtype=_TYPES[dtype])

    if layout == "interleaved":
        both = values((pages, 2, hk, page, d))
        return both[:, 0], both[:, 1]
    if layout == "nhd":
        return values((pages, page, hk, d)).permute(0, 2, 1, 3), values((pages, page, hk, d)).permute(0, 2, 1, 3)
    return values((pages, hk, page, d)), values((pages, hk, page, d))


def _tables(g, seqs, width, pages):
    """Page tables of sequences that own disjoint runs of one shuffled pool."""
    order = torch.randperm(pages, generator=g, device=_DEV, dtype=torch.int64)
    return order[: seqs * width].view(seqs, width).to(torch.int32).contiguous()


def prepare(case, seed):
    g, rng = _gen(seed)
    return {"norm_rope_append": _prepare_rows, "page_bounds": _prepare_bounds, "select_pages": _prepare_select,
            "run_selected": _prepare_attend}[case["op"]](case, g, rng)


def _prepare_rows(case, g, rng):
    t = _TYPES[case["dtype"]]
    seqs, tokens, page, hq, hk, d = (case[k] for k in ("seqs", "tokens", "page", "hq", "hk", "d"))
    n = seqs * tokens
    starts = [case["start"] if seqs == 1 else rng.randrange(case["start"] + 1) for _ in range(seqs)]
    own_pages = -(-tokens // page) + 1  # those that the new tokens lie in
    pages = seqs * own_pages
    width = (case["start"] + tokens) // page + 2
    table = torch.full((seqs, width), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(rng.randrange(1 << 30))).to(torch.int32)
    for b, s in enumerate(starts):
        first = s // page
        table[b, first:first + own_pages] = order[b * own_pages:(b + 1) * own_pages][: width - first]
    k, v = _pools(g, pages, hk, page, d, case["dtype"], case["kv"], case["layout"])
    rows = torch.randn((n, hq + 2 * hk, d), generator=g, device=_DEV, dtype=torch.float32) * 3.0
    rows = rows.to(t)  # the fused projection's output
    half = case["rot"] // 2
    angle = torch.arange(case["start"] + tokens, dtype=torch.float64, device=_DEV)[:, None] * 10000.0 ** (
        -torch.arange(half, dtype=torch.float64, device=_DEV) / half)
    return {
        "case": case, "page": page, "k": k, "v": v, "table": table.to(_DEV),
        "q": rows[:, :hq], "k_new": rows[:, hq:hq + hk], "v_new": rows[:, hq + hk:],
        "q_weight": (1 + 0.2 * torch.randn(d, generator=g, device=_DEV)).to(t),
        "k_weight": (1 + 0.2 * torch.randn(d, generator=g, device=_DEV)).to(t),
        "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
        "batch_indices": torch.arange(seqs, dtype=torch.int32, device=_DEV).repeat_interleave(tokens),
        "positions": torch.cat([torch.arange(s, s + tokens, dtype=torch.int32) for s in starts]).to(_DEV),
        "q_out": torch.empty((n, hq, d), dtype=t, device=_DEV),
    }


def _prepare_bounds(case, g, rng):
    seqs, page, hk, d, length, new = (case[k] for k in ("seqs", "page", "hk", "d", "length", "new"))
    lens = [length if seqs == 1 else max(1, length - rng.randrange(length // 8 + 1)) for _ in range(seqs)]
    begins = [max(0, n - new) for n in lens]
    touched = max(-(-n // page) - b // page for n, b in zip(lens, begins))
    width = -(-length // page)
    pages = seqs * touched
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(rng.randrange(1 << 30))).to(torch.int32)
    table = torch.full((seqs, width), -1, dtype=torch.int32)
    for b, (n, s) in enumerate(zip(lens, begins)):
        count = -(-n // page) - s // page
        table[b, s // page:s // page + count] = order[b * touched:b * touched + count]
    k, _ = _pools(g, pages, hk, page, d, case["dtype"], case["kv"], case["layout"])
    return {
        "case": case, "page": page, "new": new, "touched": touched, "k": k, "table": table.to(_DEV),
        "bounds": torch.zeros((pages, hk, 2, d), dtype=_TYPES[case["dtype"]], device=_DEV),
        "begins": torch.tensor(begins, dtype=torch.int32, device=_DEV),
        "lens": torch.tensor(lens, dtype=torch.int32, device=_DEV),
    }


def _prepare_select(case, g, rng):
    t = _TYPES[case["dtype"]]
    seqs, q_len, page, hq, hk, d, length = (case[k] for k in ("seqs", "q_len", "page", "hq", "hk", "d", "length"))
    low = max(q_len, length // 16)
    lens = [length if b == 0 else int(round(math.exp(rng.uniform(math.log(low), math.log(length))))) for b in range(seqs)]
    width = -(-length // page)
    pages = seqs * width
    # the bounds of a page of unit-variance keys around a mean of its own
    mean = torch.randn((pages, hk, 1, d), generator=g, device=_DEV) * 0.5
    spread = torch.rand((pages, hk, 2, d), generator=g, device=_DEV) + 1.5
    spread[:, :, 0].neg_()
    state = {
        "case": case, "q": torch.randn((seqs, q_len, hq, d), generator=g, device=_DEV).to(t),
        "bounds": (mean + spread).to(t),
        "table": _tables(g, seqs, width, pages), "lens": torch.tensor(lens, dtype=torch.int32, device=_DEV),
    }
    if own:
        import paged_split_kv_gather_gb300 as fd

        state["select"] = fd.PageSelect(seqs, q_len, page, hq, hk, d, width, case["budget"], case["dtype"],
                                        first_pages=case["first"], last_pages=case["last"], device=_DEV)
    return state


def _prepare_attend(case, g, rng):
    t = _TYPES[case["dtype"]]
    rows, page, hq, hk, d, budget = (case[k] for k in ("rows", "page", "hq", "hk", "d", "budget"))
    context = min(4 * budget, max(budget, (1 << 30) // (rows * hk * page * d)))  # pages of each sequence
    pages = rows * context
    k, v = _pools(g, pages, hk, page, d, case["dtype"], case["kv"], case["layout"])
    table = _tables(g, rows, context, pages)
    # each row and KV head has taken `budget` of its sequence's pages, in order of their place in it
    taken = torch.rand((rows, hk, context), generator=g, device=_DEV).argsort(-1)[..., :budget].sort(-1)[0]
    ids = table[:, None, :].expand(rows, hk, context).gather(2, taken).contiguous()
    counts = [budget * page - rng.randrange(page) for _ in range(rows)]
    if case["ragged"]:  # sequences shorter than the budget, one in eight of them not begun
        counts = [c if rng.random() < 0.5 else 0 if rng.random() < 0.25 else rng.randrange(1, c + 1) for c in counts]
    counts = torch.tensor(counts, dtype=torch.int32, device=_DEV)[:, None].expand(rows, hk).contiguous()
    used = torch.arange(budget, device=_DEV) * page < counts[..., None]
    state = {
        "case": case, "page": page, "k": k, "v": v, "ids": torch.where(used, ids, -1), "counts": counts,
        "q": torch.randn((rows, 1, hq, d), generator=g, device=_DEV).to(t) * 2,
        "out": torch.empty((rows, 1, hq, d), dtype=t, device=_DEV), "lse": torch.empty((rows, 1, hq), device=_DEV),
        "k_scale": _K_SCALE if case["kv"] else 1.0, "v_scale": _V_SCALE if case["kv"] else 1.0,
    }
    if own:
        import paged_split_kv_gather_gb300 as fd

        state["plan"] = fd.PagedDecode([budget * page] * rows, 1, page, hq, hk, d, case["dtype"], device=_DEV,
                                       kv_dtype=case["kv"])
    return state


# ------------------------------------------------------------------------------------------------------ one pass

def run(state):
    return {"norm_rope_append": _run_rows, "page_bounds": _run_bounds, "select_pages": _run_select,
            "run_selected": _run_attend}[state["case"]["op"]](state)


def _bytes_view(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x


def _run_rows(s):
    c = s["case"]
    k_scale, v_scale = (_K_SCALE, _V_SCALE) if c["kv"] else (1.0, 1.0)
    if own:
        import paged_split_kv_gather_gb300 as fd

        fd.fdec_norm_rope_append(s["q"], s["k_new"], s["v_new"], s["q_weight"], s["k_weight"], s["cos_sin"],
                                 s["batch_indices"], s["positions"], s["q_out"], s["k"], s["v"], s["table"], s["page"],
                                 eps=_EPS, interleaved=c["interleaved"], k_scale=k_scale, v_scale=v_scale)
        return s["q_out"], s["k"], s["v"]
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    rot = c["rot"]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]

    def norm_rope(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w.float()
        r = x[..., :rot]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :rot // 2], r[..., rot // 2:])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        r = torch.stack([ra, rb], -1).flatten(-2) if c["interleaved"] else torch.cat([ra, rb], -1)
        return torch.cat([r, x[..., rot:]], -1)

    def stored(x, scale):
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn) if c["kv"] else x.to(s["q"].dtype)

    s["q_out"].copy_(norm_rope(s["q"], s["q_weight"]))
    position = s["positions"].long()
    page = s["table"][s["batch_indices"].long(), position // s["page"]].long()
    slot = position % s["page"]
    _bytes_view(s["k"])[page, :, slot] = _bytes_view(stored(norm_rope(s["k_new"], s["k_weight"]), k_scale))
    _bytes_view(s["v"])[page, :, slot] = _bytes_view(stored(s["v_new"].float(), v_scale))
    return s["q_out"], s["k"], s["v"]


def _run_bounds(s):
    c = s["case"]
    if own:
        import paged_split_kv_gather_gb300 as fd

        fd.fdec_page_bounds(s["k"], s["bounds"], s["table"], s["begins"], s["lens"], s["page"],
                            expected_tokens=s["new"])
        return s["bounds"]
    page = s["page"]
    at = s["begins"].long()[:, None] // page + torch.arange(s["touched"], device=_DEV)  # [B, T] pages in order
    live = at * page < s["lens"][:, None]
    ids = torch.where(live, s["table"].gather(1, at.clamp(max=s["table"].shape[1] - 1)).long(), 0)
    keys = _bytes_view(s["k"])[ids]  # [B, T, Hk, P, D]
    keys = (keys.view(torch.float8_e4m3fn) if c["kv"] else keys).float()
    there = (at[..., None] * page + torch.arange(page, device=_DEV) < s["lens"][:, None, None])[:, :, None, :, None]
    low = torch.where(there, keys, math.inf).amin(3)
    high = torch.where(there, keys, -math.inf).amax(3)
    # a page that is not there keeps its rows: it writes them to a page past the end
    wide = torch.cat([s["bounds"], s["bounds"][:1]])
    wide[torch.where(live, ids, len(s["bounds"]))] = torch.stack([low, high], 3).to(s["bounds"].dtype)
    s["bounds"].copy_(wide[:-1])
    return s["bounds"]


def _run_select(s):
    c = s["case"]
    if own:
        return s["select"].run(s["q"], s["bounds"], s["table"], s["lens"])
    seqs, q_len, hq, d = s["q"].shape
    hk, page, budget = c["hk"], c["page"], c["budget"]
    q = s["q"].double().view(seqs, q_len, hk, hq // hk, d)
    # the sum over the group's heads of the largest logit that a key within the bounds can have: a positive q takes
    # the maximum and a negative one the minimum (64 bits: near a border the order of two pages must not depend on
    # how the sums are rounded)
    weight = torch.stack([q.clamp(max=0).sum(3), q.clamp(min=0).sum(3)], 3)  # [B, Q, Hk, 2, D]
    rows = s["bounds"][s["table"].long()].double()  # [B, W, Hk, 2, D]
    score = torch.einsum("bqhtd,bwhtd->bqhw", weight, rows)
    seen = s["lens"].long()[:, None] - q_len + 1 + torch.arange(q_len, device=_DEV)  # tokens that a query sees
    there = (seen.clamp(min=0) + page - 1) // page
    w = torch.arange(score.shape[-1], device=_DEV)
    score = torch.where(score.isnan(), math.inf, score)
    always = (w < c["first"]) | (w >= there[..., None] - c["last"])
    score = torch.where(always[:, :, None], math.inf, score)
    score = torch.where((w < there[..., None])[:, :, None], score, -math.inf)
    # always-taken pages come before any other, then larger scores, then lower indices
    order = torch.argsort(score, dim=-1, descending=True, stable=True)
    rank = torch.arange(order.shape[-1], device=_DEV)
    order = torch.where(rank < there[..., None, None].clamp(max=budget), order, order.shape[-1])
    index = torch.nn.functional.pad(order, (0, max(0, budget - order.shape[-1])), value=order.shape[-1])
    index = index[..., :budget].sort(-1)[0].reshape(seqs * q_len, hk, budget)
    taken = (index < order.shape[-1]).sum(-1)
    none = index == order.shape[-1]
    ids = s["table"].repeat_interleave(q_len, 0)[:, None].expand(-1, hk, -1).gather(2, torch.where(none, 0, index))
    tail = (seen - (there - 1) * page).reshape(-1, 1)
    counts = torch.where(taken > 0, (taken - 1) * page + tail, 0)
    return torch.where(none, -1, ids).int(), counts.int(), torch.where(none, -1, index).int()


def _run_attend(s):
    c = s["case"]
    if own:
        s["plan"].run_selected(s["q"], s["k"], s["v"], s["ids"], s["counts"], s["out"], s["lse"],
                               k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"], s["lse"]
    rows, _, hq, d = s["q"].shape
    hk, page, budget = c["hk"], s["page"], c["budget"]
    ids = s["ids"].clamp(min=0).long()
    head = torch.arange(hk, device=_DEV)[None, :, None]

    def tokens(pool):  # [rows, Hk, budget * page, D]
        x = _bytes_view(pool)[ids, head]
        return (x.view(torch.float8_e4m3fn) if c["kv"] else x).float().view(rows, hk, budget * page, d)

    q = s["q"].float().view(rows, hk, hq // hk, d)
    z = torch.matmul(q, tokens(s["k"]).transpose(2, 3)) * (s["k_scale"] / math.sqrt(d))
    there = (torch.arange(budget * page, device=_DEV) < s["counts"][..., None])[:, :, None]
    z = torch.where(there, z, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, tokens(s["v"])) * s["v_scale"] / torch.where(total > 0, total, 1)
    return o.view(rows, 1, hq, d).to(s["q"].dtype), (total.log() + top).view(rows, 1, hq)


# ------------------------------------------------------------------------------------------------------- the work

def _seen_pages(case):
    """Pages that the queries of a select case score: the same draw of lengths costs differently, so its middle."""
    low = max(case["q_len"], case["length"] // 16)
    middle = case["length"] if low >= case["length"] else (case["length"] - low) / math.log(case["length"] / low)
    total = case["length"] + (case["seqs"] - 1) * middle
    return total / case["page"]


def work(case):
    d, hk = case["d"], case["hk"]
    eb = 1 if case.get("kv") else 2
    if case["op"] == "norm_rope_append":
        n, hq = case["seqs"] * case["tokens"], case["hq"]
        per = (hq + 2 * hk) * d * 2 + hq * d * 2 + 2 * hk * d * eb + case["rot"] * 4 + 12
        return {"bytes": n * per, "flops": n * ((hq + hk) * (4 * d + 3 * case["rot"]))}
    if case["op"] == "page_bounds":
        # whole pages are summed up again, the newest one half full
        pages = case["seqs"] * (-(-case["new"] // case["page"]))
        keys = case["seqs"] * max(case["new"], (case["page"] + 1) / 2)
        return {"bytes": hk * d * (keys * eb + pages * 4), "flops": 2 * hk * d * keys}
    if case["op"] == "select_pages":
        pages, n = _seen_pages(case), case["seqs"] * case["q_len"]
        out = n * hk * (2 * case["budget"] + 1) * 4
        flops = 4 * d * hk * pages * case["q_len"]
        return {"bytes": pages * hk * d * 4 + pages * 4 + n * case["hq"] * d * 2 + out, "flops": flops}
    share = 0.66 if case["ragged"] else 1.0
    tokens = case["rows"] * hk * case["budget"] * case["page"] * share
    group = case["hq"] // hk
    return {"bytes": tokens * 2 * d * eb + 2 * case["rows"] * case["hq"] * d * 2 + case["rows"] * hk * case["budget"] * 4,
            "flops": tokens * 4 * d * group}


# ------------------------------------------------------------------------------------------- the formulas in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope_append": _exact_rows, "page_bounds": _exact_bounds, "select_pages": lambda s: None,
            "run_selected": _exact_attend}[case["op"]](s)


def _exact_rows(s):
    c = s["case"]
    half = c["rot"] // 2
    turn = torch.complex(s["cos_sin"].double()[:, :half], s["cos_sin"].double()[:, half:])[s["positions"].long()]

    def rotated(x, w):
        x = x.double()
        x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + _EPS).sqrt() * w.double()
        pairs = x[..., :c["rot"]].unflatten(-1, (half, 2) if c["interleaved"] else (2, half))
        pairs = pairs if c["interleaved"] else pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
        z = z if c["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., c["rot"]:]], -1)

    k, v = s["k"].double(), s["v"].double()
    k_new, v_new = rotated(s["k_new"], s["k_weight"]), s["v_new"].double()
    if c["kv"]:
        k_new, v_new = (k_new / _K_SCALE).clamp(-448, 448), (v_new / _V_SCALE).clamp(-448, 448)
    ids = s["table"].long()[s["batch_indices"].long(), torch.div(s["positions"].long(), s["page"], rounding_mode="floor")]
    at = (ids[:, None], torch.arange(c["hk"], device=_DEV)[None], (s["positions"].long() % s["page"])[:, None])
    k.index_put_(at, k_new)
    v.index_put_(at, v_new)
    return rotated(s["q"], s["q_weight"]), k, v


def _exact_bounds(s):
    table, lens, begins = s["table"].tolist(), s["lens"].tolist(), s["begins"].tolist()
    if sum(-(-n // s["page"]) - b // s["page"] for n, b in zip(lens, begins)) > 20000:
        return None
    out = s["bounds"].double()
    for b, (n, begin) in enumerate(zip(lens, begins)):
        for j in range(begin // s["page"], -(-n // s["page"])):
            keys = s["k"][table[b][j], :, : min(s["page"], n - j * s["page"])].double()
            keys = keys.sort(1)[0]
            out[table[b][j]] = torch.stack([keys[:, 0], keys[:, -1]], 1)
    return out


def _exact_attend(s):
    rows, _, hq, d = s["q"].shape
    hk = s["case"]["hk"]
    group = hq // hk
    out = torch.zeros((rows, 1, hq, d), dtype=torch.float64, device=_DEV)
    lse = torch.full((rows, 1, hq), -math.inf, dtype=torch.float64, device=_DEV)
    counts = s["counts"].tolist()
    for n in range(rows):
        for h in range(hk):
            count = counts[n][h]
            if count == 0:
                continue
            ids = s["ids"][n, h, : -(-count // s["page"])].long()
            k = s["k"][:, h][ids].reshape(-1, d)[:count].double() * s["k_scale"]
            v = s["v"][:, h][ids].reshape(-1, d)[:count].double() * s["v_scale"]
            z = s["q"][n, 0, h * group:(h + 1) * group].double() @ k.T / math.sqrt(d)
            lse[n, 0, h * group:(h + 1) * group] = torch.logsumexp(z, -1)
            out[n, 0, h * group:(h + 1) * group] = torch.softmax(z, -1) @ v
    return out, lse
