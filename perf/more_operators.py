"""A round of speculative decoding over the paged KV cache: its four operators, their plain forms and their cases.

A sequence of the batch has a prefix in the cache and a tree of drafted tokens: node 0 is the newest token that stands,
every other node has a parent of a lower number, and node i's key and value lie behind the prefix at position
prefix + i.  One round

  reserve_pages   finds pages for the new positions among those that no sequence names (and makes sequences forks of
                  others: full pages shared, the last one copied);
  tree_attention  attends from every node to itself and its ancestors, and joins that with the state (output and
                  log-sum-exp) of its attention to the prefix;
  verify_drafts   walks the tree with the target's probabilities, those that the drafts were drawn with and given
                  random numbers: the path that stands, and the token after it;
  keep_path       moves the keys and values of that path behind the prefix, in every layer, and sets the lengths.

``own`` False computes each with elementary torch operations, True through the library's entry points.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
_DEV = "cuda"
_K_SCALE, _V_SCALE = 0.03125, 0.0234375  # scales of the E4M3 caches: unit-variance rows use most of the range


# ---------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence, a small tree, 32/4 heads over 64-token pages: latency
        _attend("attend_1", seqs=1, nodes=8, prefix=131072, hq=32, hk=4, d=128, page=64, dtype="bf16"),
        # a batch of 16 with trees of up to 13 nodes, wide heads, one tensor for K and V, 16-bit output
        _attend("attend_16", seqs=16, nodes=13, prefix=32768, hq=16, hk=8, d=256, page=16, dtype="f16", ragged=True,
                layout="interleaved", out="same"),
        # a batch of 32 over an 8-bit cache
        _attend("attend_32_fp8", seqs=32, nodes=24, prefix=8192, hq=32, hk=8, d=128, page=16, dtype="bf16", kv="fp8",
                ragged=True, layout="nhd"),
        # wide trees of a batch of 64
        _attend("attend_64", seqs=64, nodes=64, prefix=8192, hq=32, hk=8, d=128, page=16, dtype="bf16"),
        # one sequence, four drafted tokens in a row
        _verify("verify_1", seqs=1, nodes=5, vocab=32768, dtype="f32", drafts=True),
        # trees of a draft's most likely tokens (no probabilities of theirs), a vocabulary of odd size
        _verify("verify_16_tree", seqs=16, nodes=26, vocab=50021, dtype="f32", drafts=False, ragged=True),
        # a batch of 64, seven drafted tokens in a row, a large vocabulary
        _verify("verify_64", seqs=64, nodes=8, vocab=131072, dtype="f32", drafts=True),
        # the accepted path of one sequence, 32 layers
        _keep("keep_1", seqs=1, nodes=16, layers=32, hk=4, d=128, page=64, dtype="bf16"),
        # the accepted paths of a batch of 64, 32 layers, pages that a path crosses
        _keep("keep_64", seqs=64, nodes=24, layers=32, hk=8, d=128, page=16, dtype="bf16"),
        # room for 8 more tokens for a batch of 64 in a pool of 65536 pages
        _reserve("reserve_64", seqs=64, forks=0, length=8192, new=8, pages=65536, page=16),
        # the same for 256 long sequences in a pool of a million pages
        _reserve("reserve_256", seqs=256, forks=0, length=32768, new=8, pages=1 << 20, page=16),
        # four prompts answered 16 times each: 64 forks, their last pages copied in 16 layers
        _reserve("fork_64", seqs=4, forks=64, length=2048, new=16, pages=1024, page=16, layers=16, hk=8, d=128,
                 dtype="bf16"),
    ]


def _attend(name, *, seqs, nodes, prefix, hq, hk, d, page, dtype, kv="", ragged=False, layout="hnd", out="f32"):
    return {"name": name, "op": "tree_attention", "seqs": seqs, "nodes": nodes, "prefix": prefix, "hq": hq, "hk": hk,
            "d": d, "page": page, "dtype": dtype, "kv": kv, "ragged": ragged, "layout": layout, "out": out}


def _verify(name, *, seqs, nodes, vocab, dtype, drafts, ragged=False):
    return {"name": name, "op": "verify_drafts", "seqs": seqs, "nodes": nodes, "vocab": vocab, "dtype": dtype,
            "drafts": drafts, "ragged": ragged}


def _keep(name, *, seqs, nodes, layers, hk, d, page, dtype, kv="", layout="hnd"):
    return {"name": name, "op": "keep_path", "seqs": seqs, "nodes": nodes, "layers": layers, "hk": hk, "d": d,
            "page": page, "dtype": dtype, "kv": kv, "layout": layout}


def _reserve(name, *, seqs, forks, length, new, pages, page, layers=0, hk=1, d=64, dtype="bf16", layout="hnd"):
    return {"name": name, "op": "reserve_pages", "seqs": seqs, "forks": forks, "length": length, "new": new,
            "pages": pages, "page": page, "layers": layers, "hk": hk, "d": d, "dtype": dtype, "layout": layout}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "verify", "verify", "keep", "reserve"])
    hq, hk = rng.choice([(32, 4), (32, 8), (16, 8), (4, 1), (12, 3), (8, 8)])
    dtype = rng.choice(["bf16", "f16"])
    d = rng.choice([64, 128, 128, 192, 256, 512])
    page = rng.choice([8, 16, 16, 32, 64, 64, 128])
    layout = rng.choice(["hnd", "nhd", "interleaved"])
    kv = rng.choice(["", "", "fp8"]) if d in (128, 256) else ""
    if op == "attend":
        nodes = _log(rng, 1, 64)
        seqs = _log(rng, 1, max(1, min(256, 64 * 64 * 32 * 128 // (nodes * hq * d))))
        case = _attend("", seqs=seqs, nodes=nodes, prefix=_log(rng, 64, 131072), hq=hq, hk=hk, d=d, page=page,
                       dtype=dtype, kv=kv, ragged=rng.random() < 0.5, layout=layout, out=rng.choice(["f32", "same"]))
    elif op == "verify":
        vocab = _log(rng, 1000, 200000)
        vocab -= rng.choice([0, vocab % 64])
        nodes = _log(rng, 1, 64)
        seqs = _log(rng, 1, max(1, min(64, 64 * 8 * 131072 // (nodes * vocab))))
        case = _verify("", seqs=seqs, nodes=nodes, vocab=vocab, dtype=rng.choice(["f32", "f32", dtype]),
                       drafts=nodes > 1 and rng.random() < 0.6, ragged=rng.random() < 0.5)
    elif op == "keep":
        nodes, layers = _log(rng, 2, 64), rng.randrange(1, 33)
        seqs = _log(rng, 1, max(1, min(64, 64 * 8 * 32 * 8 * 128 // (min(8, nodes) * layers * hk * d),
                                       (1 << 30) // ((nodes + 2 * page) * layers * hk * d))))
        case = _keep("", seqs=seqs, nodes=nodes, layers=layers, hk=hk, d=d, page=page, dtype=dtype, kv=kv, layout=layout)
    elif rng.random() < 0.5:
        length, new = _log(rng, 64, 32768), _log(rng, 1, 128)
        per = (length + new) // page + 2
        seqs = _log(rng, 1, min(256, (1 << 20) // per))
        case = _reserve("", seqs=seqs, forks=0, length=length, new=new, page=page,
                        pages=min(1 << 20, seqs * per + rng.randrange(1 + seqs * per)))
    else:
        length, new, layers = _log(rng, 64, 2048), _log(rng, 1, 64), rng.randrange(1, 17)
        per = layers * hk * page * d  # elements of a page of keys in all layers
        seqs = _log(rng, 1, max(1, min(8, (1 << 29) // (per * (length // page + 1)))))
        forks = _log(rng, 1, max(1, min(128, 64 * 16 * 8 * 16 * 128 // per, (1 << 29) // (per * (new // page + 2)))))
        pages = seqs * (length // page + 1) + (seqs + forks) * (new // page + 2) + rng.randrange(50)
        case = _reserve("", seqs=seqs, forks=forks, length=length, new=new, pages=pages, page=page, layers=layers, hk=hk,
                        d=d, dtype=dtype, layout=layout)
    del case["name"]
    return case


# --------------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(seed), random.Random(seed)


def _caches(g, layers, pages, hk, page, d, dtype, kv, layout):
    """Keys and values of all layers, as views [layer, page, kv_head, slot, dim] of one or two tensors."""
    def values(shape):
        if kv:  # codes of unit-variance rows
            return (torch.randn(shape, generator=g, device=_DEV) / _K_SCALE).clamp_(-448, 448).to(_TYPES[kv])
        return torch.randn(shape, generator=g, device=_DEV, dtype=_TYPES[dtype])

    if layout == "interleaved":
        both = values((layers, pages, 2, hk, page, d))
        return both[:, :, 0], both[:, :, 1]
    if layout == "nhd":
        return tuple(values((layers, pages, page, hk, d)).transpose(2, 3) for _ in range(2))
    return tuple(values((layers, pages, hk, page, d)) for _ in range(2))


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=_DEV)


def _trees(rng, seqs, nodes, most, chain=False):
    """Parents of trees with at most `most` children a node, the levels one after another."""
    rows = []
    for _ in range(seqs):
        row, left = [-1], {0: most}
        for i in range(1, nodes):
            # rather the older of the nodes that have room
            p = i - 1 if chain else sorted(left)[min(len(left) - 1, int(rng.expovariate(0.7)))]
            if not chain:
                left[p] -= 1
                if not left[p]:
                    del left[p]
                left[i] = most
            row.append(p)
        rows.append(row)
    return _int(rows).view(seqs, nodes)


def _tail_table(rng, starts, nodes, page, width):
    """Page tables with pages for the positions of the nodes behind each prefix only, and the pages of their pool."""
    spans = [(s // page, -(-(s + nodes) // page)) for s in starts]
    pages = len(starts) * ((nodes - 1) // page + 2)
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.full((len(starts), width), -1, dtype=torch.int32)
    for b, (first, last) in enumerate(spans):
        table[b, first:last] = torch.tensor([order.pop() for _ in range(last - first)], dtype=torch.int32)
    return table.to(_DEV), pages


def prepare(case, seed):
    g, rng = _gen(seed)
    return {"tree_attention": _prepare_attend, "verify_drafts": _prepare_verify, "keep_path": _prepare_keep,
            "reserve_pages": _prepare_reserve}[case["op"]](case, g, rng)


def _prefixes(case, rng):
    most = case["prefix"]
    return [most if b == 0 else rng.randrange(most // 2, most + 1) for b in range(case["seqs"])]


def _prepare_attend(case, g, rng):
    t = _TYPES[case["dtype"]]
    seqs, nodes, page, hq, hk, d = (case[k] for k in ("seqs", "nodes", "page", "hq", "hk", "d"))
    prefix = _prefixes(case, rng)
    counts = [nodes] * seqs
    if case["ragged"]:  # trees of other sizes, one sequence in eight just begun, another without drafts
        prefix = [0 if rng.random() < 0.125 else n for n in prefix]
        counts = [nodes if b == 0 else 0 if rng.random() < 0.125 else rng.randrange(1, nodes + 1) for b in range(seqs)]
    table, pages = _tail_table(rng, prefix, nodes, page, (case["prefix"] + nodes) // page + 1)
    k, v = _caches(g, 1, pages, hk, page, d, case["dtype"], case["kv"], case["layout"])
    # the state of the prefix: an average of many values, and the log of the sum of as many exponentials
    there = torch.tensor(prefix, device=_DEV)
    empty = (there == 0)[:, None, None].expand(seqs, nodes, hq)
    lse = there.clamp(min=1).log()[:, None, None] + 1 + torch.randn((seqs, nodes, hq), generator=g, device=_DEV)
    o = 0.2 * torch.randn((seqs, nodes, hq, d), generator=g, device=_DEV)
    return {
        "case": case, "page": page, "k": k[0], "v": v[0], "table": table, "prefix": _int(prefix),
        "counts": _int(counts), "parents": _trees(rng, seqs, nodes, 4),
        "q": (torch.randn((seqs, nodes, hq, d), generator=g, device=_DEV) * 2).to(t),
        "o_prefix": torch.where(empty[..., None], 0.0, o), "lse_prefix": torch.where(empty, -math.inf, lse),
        "out": torch.zeros((seqs, nodes, hq, d), dtype=t if case["out"] == "same" else torch.float32, device=_DEV),
        "lse": torch.zeros((seqs, nodes, hq), device=_DEV),
        "k_scale": _K_SCALE if case["kv"] else 1.0, "v_scale": _V_SCALE if case["kv"] else 1.0,
    }


def _prepare_verify(case, g, rng):
    t = _TYPES[case["dtype"]]
    seqs, nodes, vocab = case["seqs"], case["nodes"], case["vocab"]
    counts = [nodes if b == 0 or not case["ragged"] else rng.randrange(1, nodes + 1) for b in range(seqs)]
    parents = _trees(rng, seqs, nodes, 4, chain=case["drafts"])
    logits = torch.randn((seqs, nodes, vocab), generator=g, device=_DEV) * 3
    target = torch.softmax(logits, -1).to(t)
    # the draft model is a noisy target
    logits += torch.randn((seqs, nodes, vocab), generator=g, device=_DEV) * 0.7
    draft = torch.softmax(logits, -1)
    del logits
    tokens = torch.randint(vocab, (seqs, nodes), generator=g, device=_DEV, dtype=torch.int32)
    if case["drafts"]:
        draft = draft[:, :-1].to(t)
        race = torch.empty(draft.shape, device=_DEV).exponential_(generator=g)
        tokens[:, 1:] = (draft.float() / race).argmax(-1).int()  # token i + 1 is drawn from row i
    else:
        best = draft.topk(4, -1)[1]  # a node's children are the draft's most likely tokens
        i = torch.arange(nodes, device=_DEV)
        rank = ((parents[:, :, None] == parents[:, None]) & (i < i[:, None])).sum(-1)
        at = parents.long().clamp(min=0)
        picked = best.gather(1, at[..., None].expand(-1, -1, 4)).gather(2, rank.clamp(max=3)[..., None])[..., 0]
        tokens = torch.where(i == 0, tokens, picked.int()).contiguous()
        draft = None
    return {
        "case": case, "target": target, "draft": draft, "tokens": tokens, "parents": parents, "counts": _int(counts),
        "uniforms": torch.rand((seqs, nodes), generator=g, device=_DEV),
        "path": torch.empty((seqs, nodes), dtype=torch.int32, device=_DEV),
        "lens": torch.empty(seqs, dtype=torch.int32, device=_DEV),
        "next": torch.empty((seqs, nodes), dtype=torch.int32, device=_DEV),
    }


def _prepare_keep(case, g, rng):
    seqs, nodes, page, hk, d = (case[k] for k in ("seqs", "nodes", "page", "hk", "d"))
    prefix = [rng.randrange(8192) for _ in range(seqs)]
    table, pages = _tail_table(rng, prefix, nodes, page, (8192 + nodes) // page + 1)
    k, v = _caches(g, case["layers"], pages, hk, page, d, case["dtype"], case["kv"], case["layout"])
    # The tree's levels follow one another, so the nodes of a path that is not simply the front of the tree lie
    # behind the path's own length; one sequence in four keeps nodes in a row, which move nothing.
    path, lens = torch.full((seqs, nodes), -1, dtype=torch.int32), []
    for b in range(seqs):
        n = rng.randrange(1, min(8, nodes) + 1)
        far = nodes >= 2 * n - 1 and (b == 0 or rng.random() < 0.75)
        kept = [0] + sorted(rng.sample(range(n, nodes), n - 1)) if far else list(range(n))
        path[b, :n] = torch.tensor(kept, dtype=torch.int32)
        lens.append(n)
    return {"case": case, "page": page, "k": k, "v": v, "table": table, "prefix": _int(prefix), "path": path.to(_DEV),
            "path_lens": _int(lens), "lens": torch.empty(seqs, dtype=torch.int32, device=_DEV)}


def _prepare_reserve(case, g, rng):
    seqs, forks, page, pages, length = (case[k] for k in ("seqs", "forks", "page", "pages", "length"))
    lens = [rng.randrange(length // 2, length + 1) for _ in range(seqs)]
    lens[0] = length
    used = [-(-n // page) for n in lens]
    order = torch.randperm(min(pages, sum(used) + pages // 16), generator=g, device=_DEV)[:sum(used)].int()
    width = (length + case["new"]) // page + 2
    table = torch.full((seqs + forks, width), -1, dtype=torch.int32, device=_DEV)
    table[:seqs][torch.arange(width, device=_DEV) < _int(used)[:, None]] = order
    sources = [-1] * seqs + [rng.randrange(seqs) for _ in range(forks)]
    now = lens + [lens[a] for a in sources[seqs:]]
    new = [n + (case["new"] if b < seqs else rng.randrange(case["new"] + 1)) for b, n in enumerate(now)]
    # the workspace's bytes are at most these for any sizes: see fdec_reserve_pages_workspace
    state = {
        "case": case, "page": page, "pages": pages, "table": table, "lens": _int(lens + [0] * forks), "new": _int(new),
        "sources": _int(sources) if forks else None, "granted": torch.empty(seqs + forks, dtype=torch.int32, device=_DEV),
        "workspace": torch.empty(64 + pages + 64 * (seqs + forks), dtype=torch.int32, device=_DEV), "k": None, "v": None,
    }
    if case["layers"]:
        state["k"], state["v"] = _caches(g, case["layers"], pages, case["hk"], page, case["d"], case["dtype"], "",
                                         case["layout"])
    return state


# ------------------------------------------------------------------------------------------------------ one pass

def run(state):
    return {"tree_attention": _run_attend, "verify_drafts": _run_verify, "keep_path": _run_keep,
            "reserve_pages": _run_reserve}[state["case"]["op"]](state)


def _bytes_view(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x


def _seen(parents):
    """[B, N, N] whether node j is node i or one of its ancestors: products of the step matrix with itself, since a
    path in a tree of up to 64 nodes has at most 63 steps."""
    n = parents.shape[1]
    j = torch.arange(n, device=parents.device)
    step = ((parents[..., None] == j) | (j[:, None] == j)).float()

    def twice(m):
        return torch.matmul(m, m).clamp(max=1)

    return twice(twice(twice(twice(twice(twice(step)))))) > 0


def _run_attend(s):
    c = s["case"]
    if own:
        import paged_split_kv_gather_gb300 as fd

        fd.fdec_tree_attention(s["q"], s["k"], s["v"], s["table"], s["prefix"], s["parents"], s["o_prefix"],
                               s["lse_prefix"], s["out"], s["lse"], s["page"], node_counts=s["counts"],
                               k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"], s["lse"]
    seqs, nodes, hq, d = s["q"].shape
    hk, page = c["hk"], s["page"]
    at = s["prefix"].long()[:, None] + torch.arange(nodes, device=_DEV)
    ids, slot = s["table"].long().gather(1, at // page), at % page

    def rows(pool):  # [B, Hk, N, D]
        x = _bytes_view(pool)[ids, :, slot]
        return (x.view(torch.float8_e4m3fn) if c["kv"] else x).float().transpose(1, 2)

    there = torch.arange(nodes, device=_DEV) < s["counts"][:, None]
    seen = (_seen(s["parents"]) & there[:, None])[:, None, None]  # [B, 1, 1, N, N]
    q = s["q"].float().view(seqs, nodes, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    z = torch.matmul(q, rows(s["k"]).transpose(2, 3)[:, :, None]) * (s["k_scale"] / math.sqrt(d))
    z = torch.where(seen, z, -math.inf)
    before = s["lse_prefix"].view(seqs, nodes, hk, hq // hk).permute(0, 2, 3, 1)
    top = torch.maximum(z.amax(-1), before)
    top = torch.where(top == -math.inf, 0, top)
    e = torch.exp(z - top[..., None])
    w = torch.exp(before - top)
    total = e.sum(-1) + w
    o = torch.matmul(e, rows(s["v"])[:, :, None]) * s["v_scale"]
    o = o + w[..., None] * s["o_prefix"].view(seqs, nodes, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    o = (o / torch.where(total > 0, total, 1)[..., None]).permute(0, 3, 1, 2, 4).reshape(seqs, nodes, hq, d)
    lse = (total.log() + top).permute(0, 3, 1, 2).reshape(seqs, nodes, hq)
    s["out"].copy_(torch.where(there[..., None, None], o, s["out"].float()))
    s["lse"].copy_(torch.where(there[..., None], lse, s["lse"]))
    return s["out"], s["lse"]


def _run_verify(s):
    c = s["case"]
    if own:
        import paged_split_kv_gather_gb300 as fd

        fd.fdec_verify_drafts(s["target"], s["draft"], s["tokens"], s["parents"], s["uniforms"], s["path"], s["lens"],
                              s["next"], node_counts=s["counts"])
        return s["path"], s["lens"], s["next"]
    seqs, nodes, vocab = s["target"].shape
    b, i = torch.arange(seqs, device=_DEV), torch.arange(nodes, device=_DEV)
    parents = s["parents"].long()
    up, tokens = parents.clamp(min=0), s["tokens"].long()
    drafted = (i > 0) & (i < s["counts"][:, None])
    u = s["uniforms"].double()
    # 64 bits: a number next to a border decides between two tokens
    p = s["target"][b[:, None], up, tokens].double()
    sibling = (parents[:, :, None] == parents[:, None]) & drafted[:, None] & drafted[..., None]
    older = sibling & (i < i[:, None])
    if c["drafts"]:  # a chain: one child a node
        stands = u * s["draft"][b[:, None], up, tokens].double() < p
    else:  # each token that falls takes its weight along
        left = torch.matmul(older.double(), p[..., None])[..., 0]
        weight = torch.where(older.any(-1), s["target"].double().sum(-1).gather(1, up) - left, 1)
        stands = u * weight < p
    stands = stands & drafted
    stands = stands & ~(older & stands[:, None]).any(-1)  # the first child that stands
    reached = (_seen(s["parents"]) & ~(stands | (i == 0))[:, None]).sum(-1) == 0
    reached = reached & (i < s["counts"][:, None])
    lens = reached.sum(-1)
    order = torch.where(reached, i, nodes).sort(-1)[0]
    path = torch.where(order < nodes, order, -1)
    last = order.gather(1, (lens - 1)[:, None])[:, 0]
    row = s["target"][b, last].double()
    child = (parents == last[:, None]) & drafted
    if c["drafts"]:
        fallen = child.any(-1)[:, None]
        rest = (row - s["draft"][b, last.clamp(max=nodes - 2)].double()).clamp(min=0)
        rest = torch.where(fallen, rest, row)
    else:
        gone = torch.zeros((seqs, vocab + 1), device=_DEV, dtype=torch.bool)
        gone = gone.scatter(1, torch.where(child, tokens, vocab), True)[:, :vocab]
        rest = torch.where(gone, 0, row)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, row)
    upto = rest.cumsum(-1)
    drawn = (upto <= u[:, :1] * upto[:, -1:]).sum(-1)
    after = torch.cat([path[:, 1:], torch.full_like(path[:, :1], -1)], 1)
    words = torch.where(after >= 0, tokens.gather(1, after.clamp(min=0)), -1)
    words = torch.where(i == (lens - 1)[:, None], drawn[:, None], words)
    return path.int(), lens.int(), words.int()


def _run_keep(s):
    if own:
        import paged_split_kv_gather_gb300 as fd

        fd.fdec_keep_path((s["k"], s["v"]), s["table"], s["prefix"], s["path"], s["path_lens"], s["lens"], s["page"])
        return s["k"], s["v"], s["lens"]
    page, table = s["page"], s["table"].long()
    nodes = s["path"].shape[1]
    i = torch.arange(nodes, device=_DEV)
    to = s["prefix"].long()[:, None] + i
    taken = torch.where(i < s["path_lens"][:, None], s["path"].long(), i)  # what is not kept stays where it is
    at = s["prefix"].long()[:, None] + taken
    for_page, from_page = table.gather(1, to // page), table.gather(1, at // page)
    k, v = _bytes_view(s["k"]), _bytes_view(s["v"])
    k[:, for_page, :, to % page] = k[:, from_page, :, at % page]
    v[:, for_page, :, to % page] = v[:, from_page, :, at % page]
    s["lens"].copy_(s["prefix"] + s["path_lens"])
    return s["k"], s["v"], s["lens"]


def _run_reserve(s):
    c, page, pages, table = s["case"], s["page"], s["pages"], s["table"]
    if own:
        import paged_split_kv_gather_gb300 as fd

        fd.fdec_reserve_pages(table, s["lens"], s["new"], s["granted"], pages, page, s["workspace"],
                              sources=s["sources"], caches=(s["k"], s["v"]) if c["layers"] else ())
        return tuple(x for x in (table, s["granted"], s["k"], s["v"]) if x is not None)
    col = torch.arange(table.shape[1], device=_DEV)
    me = torch.arange(table.shape[0], device=_DEV)
    lens, new = s["lens"].long(), s["new"].long()
    source = me if s["sources"] is None else torch.where(s["sources"] < 0, me, s["sources"].long())
    fork = source != me
    old = lens[source]
    # an entry that a sequence's length covers names a page in use
    live = col < ((lens + page - 1) // page)[:, None]
    used = torch.zeros(pages + 1, dtype=torch.bool, device=_DEV)
    used[torch.where(live, table.long(), pages)] = True
    free = torch.argsort(used[:pages].int(), stable=True)  # the free pages, the lowest first
    first = torch.where(fork, torch.minimum(old, new) // page, (old + page - 1) // page)
    want = (new + page - 1) // page
    need = (want - first).clamp(min=0)
    end = need.cumsum(0)
    granted = (end <= pages - used[:pages].sum()) | (need == 0)
    index = (end - need)[:, None] + col - first[:, None]
    take = (col >= first[:, None]) & (col < want[:, None]) & granted[:, None]
    shared = (fork & granted)[:, None] & (col < first[:, None])
    filled = torch.where(take, free[index.clamp(0, pages - 1)].int(), torch.where(shared, table[source], table))
    if c["layers"]:  # the filled part of a fork's last page
        n = c["seqs"]
        at = (torch.minimum(old, new) // page)[n:, None]
        kept = (torch.minimum(old, new) % page)[n:]
        moved = (torch.arange(page, device=_DEV) < kept[:, None]) & granted[n:, None]
        moved = moved[None, :, None, :, None]
        of, to = table[source[n:]].gather(1, at)[:, 0].long(), filled[n:].gather(1, at)[:, 0].long()
        # a fork without such a part writes a page of its source over itself
        none = (kept == 0) | ~granted[n:]
        of, to = torch.where(none, table[source[n:], 0].long(), of), torch.where(none, table[source[n:], 0].long(), to)
        s["k"][:, to] = torch.where(moved, s["k"][:, of], s["k"][:, to])
        s["v"][:, to] = torch.where(moved, s["v"][:, of], s["v"][:, to])
    table.copy_(filled)
    s["granted"].copy_(torch.where(granted, new, lens))
    return tuple(x for x in (table, s["granted"], s["k"], s["v"]) if x is not None)


# ------------------------------------------------------------------------------------------------------- the work

def work(case):
    d = case.get("d", 0)
    eb = 1 if case.get("kv") else 2
    if case["op"] == "tree_attention":
        rows = case["seqs"] * case["nodes"] * case["hq"] * (0.47 if case["ragged"] else 1.0)
        keys = case["seqs"] * case["nodes"] * case["hk"] * (0.47 if case["ragged"] else 1.0)
        out = 2 if case["out"] == "same" else 4
        depth = 1 + math.log(case["nodes"], 2)  # about the nodes of a path
        return {"bytes": rows * (d * (2 + 4 + out) + 8) + keys * 2 * d * eb, "flops": rows * 4 * d * depth}
    if case["op"] == "verify_drafts":
        # the last accepted node's row, and the draft's row where a draft has fallen (four in five)
        size = 4 if case["dtype"] == "f32" else 2
        rows = case["seqs"] * (1.8 if case["drafts"] else 1.0)
        return {"bytes": rows * case["vocab"] * size + case["seqs"] * case["nodes"] * 24,
                "flops": 3 * rows * case["vocab"]}
    if case["op"] == "keep_path":
        moved = case["seqs"] * 0.75 * max(0, min(8, case["nodes"]) - 1) / 2  # rows that are not in place already
        if case["seqs"] == 1:
            moved = max(0, min(8, case["nodes"]) - 1) / 2
        return {"bytes": moved * 2 * case["layers"] * case["hk"] * d * eb * 2 + case["seqs"] * 64, "flops": 0}
    entries = case["seqs"] * 0.75 * case["length"] / case["page"]
    new = (case["seqs"] + case["forks"]) * (case["new"] / case["page"] + 1)
    shared = case["forks"] * 0.75 * case["length"] / case["page"]
    copied = case["forks"] * (case["page"] - 1) / 2 * 2 * case["layers"] * case["hk"] * d * 2 * 2
    return {"bytes": 4 * entries + 4 * new + 4 * shared + copied + 12 * (case["seqs"] + case["forks"]), "flops": 0}


# ------------------------------------------------------------------------------------------- the formulas in 64 bits

def exact(case, seed):
    return {"tree_attention": _exact_attend, "verify_drafts": _exact_verify, "keep_path": _exact_keep,
            "reserve_pages": _exact_reserve}[case["op"]](prepare(case, seed))


def _exact_attend(s):
    seqs, nodes, hq, d = s["q"].shape
    group = hq // s["case"]["hk"]
    out, lse = s["out"].double(), s["lse"].double()
    prefix, counts, parents, table = (s[k].tolist() for k in ("prefix", "counts", "parents", "table"))
    for b in range(seqs):
        n = counts[b]
        if n == 0:
            continue
        line = torch.full((n, n), -math.inf, dtype=torch.float64)
        for i in range(n):
            j = i
            while j >= 0:
                line[i, j] = 0.0
                j = parents[b][j]
        where = [(table[b][t // s["page"]], t % s["page"]) for t in range(prefix[b], prefix[b] + n)]
        page = torch.tensor([w[0] for w in where], device=_DEV)
        slot = torch.tensor([w[1] for w in where], device=_DEV)
        k = s["k"].view(s["k"].dtype)[page, :, slot] if not s["case"]["kv"] else \
            _bytes_view(s["k"])[page, :, slot].view(torch.float8_e4m3fn)
        v = s["v"][page, :, slot] if not s["case"]["kv"] else _bytes_view(s["v"])[page, :, slot].view(torch.float8_e4m3fn)
        k = k.double().repeat_interleave(group, 1) * s["k_scale"]
        v = v.double().repeat_interleave(group, 1) * s["v_scale"]
        z = torch.einsum("ihd,jhd->hij", s["q"][b, :n].double(), k) / math.sqrt(d) + line.to(_DEV)
        inner = torch.logsumexp(z, -1)  # [H, n]
        before = s["lse_prefix"][b, :n].double().T
        both = torch.logaddexp(inner, before)
        o = torch.einsum("hij,jhd->ihd", torch.exp(z - both[..., None]), v)
        out[b, :n] = o + torch.exp(before - both).T[..., None] * s["o_prefix"][b, :n].double()
        lse[b, :n] = both.T
    return out, lse


def _exact_verify(s):
    seqs, nodes, vocab = s["target"].shape
    counts, parents, tokens, u = (s[k].tolist() for k in ("counts", "parents", "tokens", "uniforms"))
    path, words, lens = torch.full((seqs, nodes), -1), torch.full((seqs, nodes), -1), []
    for b in range(seqs):
        node, steps = 0, [0]
        while True:
            p = s["target"][b, node].double()
            rest, weight, next_node = p, 1.0, None
            for c in range(1, counts[b]):
                if parents[b][c] != node:
                    continue
                t = tokens[b][c]
                q = None if s["draft"] is None else s["draft"][b, node].double()
                chance = rest[t].item() / weight / (1.0 if q is None else q[t].item())
                if u[b][c] < chance:
                    next_node = c
                    break
                if q is None:
                    rest = rest.clone()
                    rest[t] = 0.0
                else:
                    rest = (rest / weight - q).clamp(min=0)
                weight = rest.sum().item()
            if next_node is None:
                break
            words[b, len(steps) - 1] = tokens[b][next_node]
            steps.append(next_node)
            node = next_node
        rest = rest if weight > 0 else p
        upto = rest.cumsum(0)
        words[b, len(steps) - 1] = int(torch.searchsorted(upto, upto[-1] * u[b][0], right=True))
        path[b, :len(steps)] = torch.tensor(steps)
        lens.append(len(steps))
    return path.int(), torch.tensor(lens, dtype=torch.int32), words.int()


def _exact_keep(s):
    page, table, prefix, path, lens = s["page"], *(s[k].tolist() for k in ("table", "prefix", "path", "path_lens"))
    both = []
    for pool in (s["k"], s["v"]):
        moved = pool.double()
        for b, n in enumerate(lens):
            for i in range(n):
                of, to = prefix[b] + path[b][i], prefix[b] + i
                row = pool[:, table[b][of // page], :, of % page]
                moved[:, table[b][to // page], :, to % page] = row.double()
        both.append(moved)
    return both[0], both[1], torch.tensor([p + n for p, n in zip(prefix, lens)], dtype=torch.int32)


def _exact_reserve(s):
    page, table, lens, new = s["page"], *(s[k].tolist() for k in ("table", "lens", "new"))
    sources = [-1] * len(lens) if s["sources"] is None else s["sources"].tolist()
    used = {p for row, n in zip(table, lens) for p in row[:-(-n // page)]}
    free = [p for p in range(s["pages"]) if p not in used]
    pools = [x.double() for x in (s["k"], s["v"]) if x is not None]
    filled, granted, wanted = [list(row) for row in table], list(lens), 0
    for b, a in enumerate(sources):
        a = b if a < 0 else a
        kept = min(lens[a], new[b])
        first = kept // page if a != b else -(-lens[b] // page)
        need = max(0, -(-new[b] // page) - first)
        taken = free[wanted:wanted + need]
        wanted += need
        if len(taken) < need:
            continue
        granted[b] = new[b]
        if a != b:
            filled[b][:first] = table[a][:first]
        filled[b][first:first + need] = taken
        if a != b and kept % page:
            for x, pool in zip(pools, (s["k"], s["v"])):
                x[:, taken[0], :, :kept % page] = pool[:, table[a][first], :, :kept % page].double()
    return (torch.tensor(filled, dtype=torch.int32), torch.tensor(granted, dtype=torch.int32), *pools)
