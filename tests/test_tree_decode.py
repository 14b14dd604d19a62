"""Speculative decoding: attention of drafted trees, verification of the drafts, the accepted path's rows, pages for
new lengths; each against its definition in 64 bits, or row by row; refusals on the host.

Tolerances of the attention, derived from the arithmetic (u = 2^-24, half a step of fp32).  A logit is a sum of D exact
products in fp32 (the tensor cores may cut instead of rounding: two half steps an addition), scaled once: off by at most
e = scale (2 D + 4) u sum_d |q_d k_d|, and rounded against the maximum, at most 3 u |z| more.  A probability is then off
by a factor exp(2 e) (its own logit and the maximum's or the sum's), the exponential's two units (4 u) and those of the
sums of 64 terms (128 u); the split into 16-bit terms leaves 2^-22.  So a row of out is off by at most
(2 e + 8 u zmax + 200 u) times the largest value it averages, and lse by e + 3 u zmax + 140 u + u |lse|.  A 16-bit result
is rounded once more: half a step of the value, or of the smallest normal number.  Tokens, paths, lengths and pages are
equal; moved rows are equal bit for bit."""
import inspect
import math
import os
import random
import re

import numpy as np
import pytest
import torch

import paged_split_kv_gather_gb300 as fd

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
PROB = {"f32": torch.float32, **DT}
U = 2.0 ** -24
gpu = pytest.mark.gpu


def i32(x, device="cuda"):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(device)


def bits(t):
    return t.contiguous().view(torch.uint8)


def make_pool(pages, hk, page, d, dtype, layout, seed, layers=0):
    """K and V views [page, kv_head, slot, dim], or [layer, ...]."""
    g = torch.Generator().manual_seed(seed)
    t = torch.float8_e4m3fn if dtype == "fp8" else DT[dtype]
    n = layers or 1

    def rand(*shape):
        return (torch.randn(shape, generator=g) * (8.0 if dtype == "fp8" else 1.0)).to(t).cuda()

    if layout == "interleaved":
        kv = rand(n, pages, 2, hk, page, d)
        out = kv[:, :, 0], kv[:, :, 1]
    elif layout == "nhd":
        out = tuple(rand(n, pages, page, hk, d).transpose(2, 3) for _ in range(2))
    else:
        out = tuple(rand(n, pages, hk, page, d) for _ in range(2))
    return out if layers else tuple(x[0] for x in out)


def random_parents(rng, nodes, kind):
    if kind == "chain":
        return [i - 1 for i in range(nodes)]
    if kind == "star":
        return [-1] + [0] * (nodes - 1)
    if kind == "forest":  # several nodes without a parent
        return [-1] + [rng.randrange(-1, i) for i in range(1, nodes)]
    return [-1] + [rng.randrange(max(0, i - 6), i) for i in range(1, nodes)]


def path_of(parents, i):
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out[::-1]


# ---------------------------------------------------------------------------------------------------- tree attention

class Tree:
    """Inputs of one call, and its definition in 64 bits."""

    def __init__(self, d, hq, hk, nodes, page, batch, dtype="bf16", kv="", layout="hnd", kind="tree", seed=0, counts=None,
                 prefix=None, state=True, k_scale=1.0, v_scale=1.0):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.d, self.hq, self.hk, self.nodes, self.page, self.batch = d, hq, hk, nodes, page, batch
        self.t = DT[dtype]
        self.prefix = prefix or [rng.randrange(0, 5 * page) if b else 0 for b in range(batch)]
        self.counts = counts or [nodes if b == 0 else rng.randrange(0, nodes + 1) for b in range(batch)]
        self.parents = [random_parents(rng, nodes, kind) for _ in range(batch)]
        width = (max(self.prefix) + nodes) // page + 2
        spans = [(p // page, -(-(p + nodes) // page)) for p in self.prefix]
        pages = sum(b - a for a, b in spans) + 2
        order = list(range(pages))
        rng.shuffle(order)
        self.table = np.full((batch, width), -7, dtype=np.int32)  # entries that no node needs are not looked at
        for b, (x, y) in enumerate(spans):
            self.table[b, x:y] = [order.pop() for _ in range(y - x)]
        self.k, self.v = make_pool(pages, hk, page, d, kv or dtype, layout, seed)
        self.k_scale, self.v_scale = (k_scale, v_scale)
        self.q = torch.randn((batch, nodes, hq, d), generator=g).to(self.t).cuda()
        self.o_prefix = self.lse_prefix = None
        if state:
            self.o_prefix = torch.randn((batch, nodes, hq, d), generator=g).cuda()
            self.lse_prefix = (torch.randn((batch, nodes, hq), generator=g) * 2 + 1).cuda()
            empty = torch.tensor(self.prefix)[:, None, None].expand(batch, nodes, hq) == 0
            self.lse_prefix[empty.cuda()] = -math.inf
            self.o_prefix[empty.cuda()] = math.nan  # an empty state counts for nothing, whatever its o
        self.scale = 1.0 / math.sqrt(d)

    def run(self, out=None, lse=None, err=None, **kw):
        out = torch.full_like(self.q, 3.0, dtype=torch.float32) if out is None else out
        lse = torch.full(self.q.shape[:3], 5.0, device="cuda") if lse is None else lse
        args = dict(node_counts=i32(self.counts), k_scale=self.k_scale, v_scale=self.v_scale, device_errors=err)
        args.update(kw)
        fd.fdec_tree_attention(self.q, self.k, self.v, i32(self.table), i32(self.prefix), i32(self.parents),
                               self.o_prefix, self.lse_prefix, out, lse, self.page, **args)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, parents=None, counts=None, unseen=()):
        """unseen: (sequence, node) whose rows nobody sees."""
        group = self.hq // self.hk
        half = 0.0 if out.dtype == torch.float32 else torch.finfo(out.dtype).eps / 2
        tiny = 0.0 if out.dtype == torch.float32 else torch.finfo(out.dtype).tiny
        for b in range(self.batch):
            for i in range((counts or self.counts)[b]):
                at = [(j, self.prefix[b] + j) for j in path_of((parents or self.parents)[b], i) if (b, j) not in unseen]
                where = [(int(self.table[b, p // self.page]), p % self.page) for _, p in at]
                for kvh in range(self.hk):
                    k, v = (torch.stack([x[pg, kvh, sl].double() for pg, sl in where]).cpu() if where
                            else torch.zeros(0, self.d, dtype=torch.float64) for x in (self.k, self.v))
                    k, v = k * self.k_scale, v * self.v_scale
                    q = self.q[b, i, kvh * group:(kvh + 1) * group].double().cpu()
                    z = q @ k.T * self.scale
                    mag = (q.abs() @ k.abs().T * abs(self.scale)).amax(-1) if where else torch.zeros(group).double()
                    rows = slice(kvh * group, (kvh + 1) * group)
                    if self.lse_prefix is not None:
                        before = self.lse_prefix[b, i, rows].double().cpu()
                        o = self.o_prefix[b, i, rows].double().cpu()
                        o = torch.where(before[:, None] == -math.inf, 0.0, o)
                    else:
                        before, o = torch.full((group,), -math.inf).double(), torch.zeros(group, self.d).double()
                    total = torch.logaddexp(torch.logsumexp(z, -1), before)
                    safe = torch.where(total == -math.inf, 0.0, total)
                    want = torch.exp(z - safe[:, None]) @ v + torch.exp(before - safe)[:, None] * o
                    want = torch.where(total[:, None] == -math.inf, 0.0, want)
                    e = (2 * self.d + 4) * U * mag
                    zmax = torch.maximum(z.abs().amax(-1) if where else torch.zeros(group).double(),
                                         torch.where(before == -math.inf, 0.0, before).abs())
                    largest = torch.maximum(v.abs().amax() if where else torch.zeros(()).double(), o.abs().amax(-1))
                    tol = (2 * e + 8 * U * zmax + 200 * U) * largest
                    got = out[b, i, rows].double().cpu()
                    off = (got - want).abs()
                    limit = tol[:, None] + half * torch.maximum(want.abs() + tol[:, None], torch.tensor(tiny).double())
                    assert (off <= limit).all(), (b, i, kvh, (off - limit).max().item(), off.max().item())
                    if lse is not None:
                        got = lse[b, i, rows].double().cpu()
                        assert torch.equal(got == -math.inf, total == -math.inf)
                        fine = total != -math.inf
                        off = (got - total).abs()[fine]
                        assert (off <= (e + 3 * U * zmax + 140 * U + U * total.abs())[fine]).all(), (b, i, kvh, off)


@gpu
@pytest.mark.parametrize("d,hq,hk,nodes,page,batch,dtype,kv,layout,kind", [
    (128, 8, 2, 8, 16, 3, "bf16", "", "hnd", "tree"),
    (128, 32, 4, 1, 64, 2, "bf16", "", "hnd", "chain"),        # one node: itself and the prefix
    (128, 4, 4, 64, 16, 2, "f16", "", "nhd", "tree"),          # every bit of the ancestors' word
    (64, 6, 2, 33, 8, 3, "bf16", "", "interleaved", "tree"),   # a group that does not divide a tile
    (64, 4, 1, 17, 1, 2, "f16", "", "hnd", "star"),            # pages of one token
    (192, 8, 8, 13, 32, 2, "f16", "", "nhd", "forest"),        # one query head a KV head
    (256, 16, 8, 24, 16, 2, "bf16", "", "hnd", "chain"),
    (512, 4, 2, 64, 256, 2, "bf16", "", "hnd", "tree"),        # the largest rows staged
    (512, 2, 1, 5, 4, 2, "f16", "", "interleaved", "tree"),
    (128, 8, 2, 26, 16, 3, "bf16", "fp8", "hnd", "tree"),
    (256, 4, 2, 9, 32, 2, "f16", "fp8", "nhd", "tree"),
    (128, 40, 2, 7, 16, 2, "bf16", "", "hnd", "tree"),         # more heads in a group than rows in a tile
    (128, 8, 2, 16, 16, 40, "bf16", "", "hnd", "tree"),
])
def test_tree_attention(d, hq, hk, nodes, page, batch, dtype, kv, layout, kind):
    scales = dict(k_scale=0.037, v_scale=0.21) if kv else {}
    c = Tree(d, hq, hk, nodes, page, batch, dtype, kv, layout, kind, seed=d + nodes, **scales)
    for out_type in (torch.float32, DT[dtype]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full(c.q.shape, 3.0, dtype=out_type, device="cuda")
        out, lse = c.run(out=out, err=err)
        assert int(err.item()) == 0
        c.check(out, lse)
        for b, n in enumerate(c.counts):  # rows past a sequence's nodes are left alone
            assert (out[b, n:] == 3.0).all() and (lse[b, n:] == 5.0).all()


@gpu
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (192, "f16")])
def test_tree_attention_in_place_of_the_state_and_without_one(d, dtype):
    c = Tree(d, 8, 2, 19, 16, 4, dtype, seed=5)
    out, lse = c.run()
    o, l2 = c.o_prefix.clone(), c.lse_prefix.clone()
    keep = c.o_prefix, c.lse_prefix
    c.o_prefix, c.lse_prefix = o, l2
    c.run(out=o, lse=l2)
    for b, n in enumerate(c.counts):
        assert torch.equal(bits(o[b, :n]), bits(out[b, :n])) and torch.equal(l2[b, :n], lse[b, :n])
        assert torch.equal(bits(o[b, n:]), bits(keep[0][b, n:])) and torch.equal(l2[b, n:], keep[1][b, n:])
    c = Tree(d, 8, 2, 19, 16, 4, dtype, seed=6, state=False)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.equal(c.run(lse=lse)[0], out)
    out2 = torch.empty_like(out)
    fd.fdec_tree_attention(c.q, c.k, c.v, i32(c.table), i32(c.prefix), i32(c.parents), None, None, out2, None, c.page)
    c.check(out2, None, counts=[c.nodes] * c.batch)  # without lse, and every sequence with all nodes


@gpu
def test_tree_attention_of_a_chain_without_parents():
    c = Tree(128, 8, 2, 12, 16, 3, seed=7, kind="chain", counts=[12, 12, 12])
    out, lse = c.run()
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    fd.fdec_tree_attention(c.q, c.k, c.v, i32(c.table), i32(c.prefix), None, c.o_prefix, c.lse_prefix, again, lse2, c.page)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@gpu
def test_tree_attention_takes_strided_queries_and_head_major_ones():
    c = Tree(128, 8, 2, 10, 16, 3, seed=8)
    want, _ = c.run()
    wide = torch.randn(3 * 10, 8 + 4, 128).to(c.t).cuda()
    wide[:, :8] = c.q.view(30, 8, 128)
    q = c.q
    c.q = wide[:, :8].view(3, 10, 8, 128)
    got, _ = c.run(out=torch.full(want.shape, 3.0, device="cuda"))
    assert torch.equal(want, got)
    c.q = q.view(30, 8, 128).transpose(0, 1).contiguous().transpose(0, 1).view(3, 10, 8, 128)
    assert c.q.stride(2) == 30 * 128
    got, _ = c.run(out=torch.full(want.shape, 3.0, device="cuda"))
    assert torch.equal(want, got)


@gpu
@pytest.mark.parametrize("d,dtype,kv", [(64, "bf16", ""), (128, "f16", ""), (256, "bf16", ""), (128, "bf16", "fp8"),
                                        (512, "f16", "")])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_rows_that_a_node_does_not_see_never_reach_it(d, dtype, kv, value):
    c = Tree(d, 6, 2, 22, 16, 2, dtype, kv, seed=9, counts=[22, 22])
    clean, lse = c.run()
    c.check(clean, lse)
    node = 3
    p = c.prefix[1] + node
    page, slot = int(c.table[1, p // 16]), p % 16
    for pool in (c.k, c.v):
        pool[page, 0, slot] = torch.tensor(value).to(pool.dtype)
        pool[page, 0, slot, 1::2] = torch.tensor(math.nan if value != value else -value).to(pool.dtype)
    # a slot behind the last node: in the page, of no node
    got, got_lse = c.run()
    for i in range(22):
        sees = node in path_of(c.parents[1], i)
        if not sees:
            c_rows, g_rows = clean[1, i], got[1, i]
            assert torch.isfinite(g_rows).all() and torch.isfinite(got_lse[1, i]).all()
            assert torch.equal(got_lse[1, i], lse[1, i])
            # (a tile with such a row is summed in another order: both are within the tolerance)
            assert (c_rows - g_rows).abs().max() <= 1e-4
        else:
            assert not torch.isfinite(got[1, i, :3]).all()  # the group of KV head 0
            assert torch.isfinite(got[1, i, 3:]).all()
    assert torch.equal(got[0], clean[0])
    for pool in (c.k, c.v):  # restored: a slot that no node holds may hold anything
        pool[page, 0, slot] = torch.zeros(d).to(pool.dtype)
    c.check(*c.run())


@gpu
def test_tree_attention_of_extreme_logits_and_states():
    c = Tree(128, 4, 2, 9, 16, 2, "bf16", seed=10, counts=[9, 9], prefix=[33, 70])
    c.q = c.q * 200
    c.check(*c.run())
    c.q = c.q / 200
    c.lse_prefix[0] = 120.0   # the prefix is everything
    c.lse_prefix[1] = -120.0  # and nothing
    out, lse = c.run()
    c.check(out, lse)
    assert torch.allclose(out[0], c.o_prefix[0]) and not torch.allclose(out[1], c.o_prefix[1])


@gpu
@pytest.mark.parametrize("dtype,power", [("bf16", 119), ("bf16", 60), ("bf16", -30), ("bf16", -90), ("bf16", -110),
                                         ("f16", 13), ("f16", -10)])
def test_tree_attention_of_values_of_any_size(dtype, power):
    """A bf16 cache's values are multiplied as f16 values: by a power of two that the largest sets."""
    for spread in (False, True):  # one row much smaller than the others: no worse than the tolerance of the largest
        c = Tree(128, 8, 2, 21, 16, 2, dtype, seed=13, counts=[21, 21])
        c.v = (c.v.double() * 2.0 ** power).to(c.t)
        if spread:
            c.v[:, :, ::3] = (c.v[:, :, ::3].double() * 2.0 ** -20).to(c.t)
        c.o_prefix = c.o_prefix * 2.0 ** power
        out, lse = c.run()
        c.check(out, lse)


@gpu
@pytest.mark.parametrize("d,dtype,kv", [(128, "bf16", ""), (256, "f16", ""), (128, "bf16", "fp8")])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-30])
def test_tree_attention_of_any_scale(d, dtype, kv, scale):
    c = Tree(d, 8, 2, 37, 16, 2, dtype, kv, seed=14, counts=[37, 20])
    c.scale = scale
    out, lse = c.run(scale=scale)
    c.check(out, lse)


@gpu
@pytest.mark.parametrize("hq,hk,nodes,batch", [(16, 8, 16, 70), (8, 8, 3, 90), (24, 3, 64, 160), (32, 4, 33, 115)])
def test_tree_attention_in_equal_shares(hq, hk, nodes, batch):
    """More sequences' heads than CTAs are resident: shares that begin inside a head, and span several."""
    c = Tree(64, hq, hk, nodes, 16, batch, "f16", seed=15)
    out, lse = c.run()
    few = random.Random(1).sample(range(batch), 6) + [0, batch - 1]
    counts = [n if b in few else 0 for b, n in enumerate(c.counts)]
    c.check(out, lse, counts=counts)
    # the others against calls of few sequences, which are not shared out
    for b in range(0, batch, 16):
        part = slice(b, min(batch, b + 16))
        o, l2 = torch.full_like(out[part], 3.0), torch.full_like(lse[part], 5.0)
        fd.fdec_tree_attention(c.q[part], c.k, c.v, i32(c.table[part]), i32(c.prefix[part]), i32(c.parents[part]),
                               c.o_prefix[part], c.lse_prefix[part], o, l2, 16, node_counts=i32(c.counts[part]))
        assert torch.equal(o, out[part]) and torch.equal(l2, lse[part])


@gpu
def test_tree_attention_flags_bad_trees_pages_and_lengths():
    def flags(c, parents=None, counts=None, prefix=None, table=None):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = torch.zeros(c.q.shape, device="cuda"), torch.zeros(c.q.shape[:3], device="cuda")
        fd.fdec_tree_attention(c.q, c.k, c.v, i32(c.table if table is None else table), i32(prefix or c.prefix),
                               i32(parents or c.parents), c.o_prefix, c.lse_prefix, out, lse, c.page,
                               node_counts=i32(counts or c.counts), device_errors=err)
        return int(err.item()), out, lse

    c = Tree(128, 8, 2, 11, 16, 3, seed=11, counts=[11, 11, 11], prefix=[0, 20, 45])
    bad = [list(p) for p in c.parents]
    bad[1][5], bad[2][7] = 5, -2
    got, out, lse = flags(c, parents=bad)
    bad[1][5] = bad[2][7] = -1
    assert got == fd.DEVERR_TREE
    c.check(out, lse, parents=bad)
    got, out, lse = flags(c, counts=[11, -1, 12])
    assert got == fd.DEVERR_SEQ_LEN
    c.check(out, lse, counts=[11, 0, 11])
    assert (out[1] == 0).all()
    for page in (-1, c.k.shape[0]):
        table = c.table.copy()
        table[2, 45 // 16] = page  # nodes 0 .. 2 of sequence 2
        got, out, lse = flags(c, table=table)
        assert got == fd.DEVERR_PAGE_ID
        c.check(out, lse, unseen={(2, 0), (2, 1), (2, 2)})
    width = c.table.shape[1]
    got, out, lse = flags(c, table=c.table[:, :3].copy())  # nodes from position 48 on
    assert width > 3 and got == fd.DEVERR_SEQ_LEN
    c.check(out, lse, unseen={(2, j) for j in range(3, 11)})
    # taken as 0, where this sequence's row has no page
    assert flags(c, prefix=[0, 20, -5])[0] == fd.DEVERR_SEQ_LEN | fd.DEVERR_PAGE_ID


# ------------------------------------------------------------------------------------------------------ verification

def verify_reference(target, draft, tokens, parents, u, count):
    """One sequence, in fp64 numpy: (path, out tokens, the smallest margin of any decision)."""
    if count == 0:
        return [], [], 1.0
    clamp = lambda x: np.clip(np.nan_to_num(x, nan=0.0, posinf=2.0, neginf=0.0), 0, 2)  # noqa: E731
    uniform = lambda x: 0.0 if not x >= 0 else min(float(x), 1 - 2.0 ** -24)  # noqa: E731
    target = clamp(target.astype(np.float64))
    vocab = target.shape[1]
    path, words, margin = [0], [], 1.0
    while True:
        x = path[-1]
        p = target[x]
        q = clamp(draft[x].astype(np.float64)) if draft is not None and x < len(draft) else None
        rest, weight, s, chosen = p, 1.0, 0.0, None
        for c in range(x + 1, count):
            if parents[c] != x or not 0 <= tokens[c] < vocab:
                continue
            t = tokens[c]
            left, right = uniform(u[c]) * weight * (1.0 if q is None else q[t]), rest[t]
            if left != right:
                margin = min(margin, abs(left - right) / max(left, right))
            if left < right:
                chosen = c
                break
            if q is None:
                rest = rest.copy()
                rest[t] = 0.0
            else:
                s += weight
                rest = np.maximum(p - s * q, 0)
            weight = rest.sum()
            if not weight > 0:
                break
        if chosen is None:
            break
        path.append(chosen)
        words.append(int(tokens[chosen]))
    rest = rest if rest.sum() > 0 else p
    if not rest.sum() > 0:
        return path, words + [-1], margin
    upto = np.cumsum(rest)
    goal = uniform(u[0]) * upto[-1]
    token = int(np.argmax(upto > goal))
    margin = min(margin, float(np.abs(upto - goal)[rest > 0].min() / upto[-1]) if goal > 0 else 1.0)
    return path, words + [token], margin


def run_verify(target, draft, tokens, parents, u, counts=None):
    b, n, _ = target.shape
    path, words = (torch.full((b, n), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    lens = torch.full((b,), 77, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fd.fdec_verify_drafts(target, draft, i32(tokens), None if parents is None else i32(parents), u.cuda(), path, lens, words,
                          node_counts=None if counts is None else i32(counts), device_errors=err)
    return path.cpu(), lens.cpu(), words.cpu(), int(err.item())


def check_verify(target, draft, tokens, parents, u, counts=None, flags=0, margin=1e-11):
    b, n, _ = target.shape
    path, lens, words, err = run_verify(target, draft, tokens, parents, u, counts)
    assert err == flags, hex(err)
    parents = [[i - 1 for i in range(n)]] * b if parents is None else parents
    lengths = []
    for i in range(b):
        want, want_words, near = verify_reference(
            target[i].float().cpu().numpy(), None if draft is None else draft[i].float().cpu().numpy(), tokens[i],
            parents[i], u[i].tolist(), n if counts is None else counts[i])
        assert near > margin, near  # (a case of the test's own making: no decision is that near)
        pad = lambda x: x + [-1] * (n - len(x))  # noqa: E731
        assert path[i].tolist() == pad(want) and lens[i] == len(want), (i, path[i].tolist(), want)
        assert words[i].tolist() == pad(want_words), (i, words[i].tolist(), want_words)
        lengths.append(len(want))
    return lengths


def drafts_of(g, rng, batch, nodes, vocab, dtype, kind, drafts, noise=0.7):
    """Probabilities, tokens and trees as a drafting step leaves them."""
    logits = torch.randn((batch, nodes, vocab), generator=g) * 3
    target = torch.softmax(logits, -1).to(PROB[dtype]).cuda()
    draft = torch.softmax(logits + noise * torch.randn((batch, nodes, vocab), generator=g), -1).to(PROB[dtype])
    parents = [random_parents(rng, nodes, kind) for _ in range(batch)]
    tokens = []
    for b in range(batch):
        rows = draft[b].double()
        best = rows.argsort(-1, descending=True)
        row, used = [0], {}
        for i in range(1, nodes):
            p = max(parents[b][i], 0)
            used[p] = used.get(p, -1) + 1
            if drafts:
                row.append(int(torch.multinomial(rows[p], 1, generator=g)) if rows[p].sum() > 0 else 0)
            else:
                row.append(int(best[p, used[p] % vocab]))
        tokens.append(row)
    return target, draft.cuda() if drafts else None, tokens, parents


VERIFY_TREES = [("chain", 1, False), ("chain", 5, True), ("tree", 12, True), ("star", 9, True), ("tree", 26, False),
                ("star", 64, False)]


@gpu
@pytest.mark.parametrize("vocab,kind,nodes,drafts", [
    (vocab, *tree) for vocab in (1, 2, 5, 127, 128, 1000, 4099, 50021, 131072) for tree in VERIFY_TREES
    if vocab * tree[1] <= 4_000_000])
def test_verify_drafts(vocab, kind, nodes, drafts):
    seed = vocab + nodes
    g, rng = torch.Generator().manual_seed(seed), random.Random(seed)
    batch = 4 if vocab > 10000 else 24
    for dtype in ("f32", "bf16", "f16") if vocab < 10000 else ("f32",):
        target, draft, tokens, parents = drafts_of(g, rng, batch, nodes, vocab, dtype, kind, drafts)
        u = torch.rand((batch, nodes), generator=g)
        check_verify(target, draft, tokens, parents, u)
        counts = [rng.randrange(0, nodes + 1) for _ in range(batch)]
        check_verify(target, draft, tokens, parents, u, counts=counts)


@gpu
def test_verify_drafts_goes_deep_and_tries_many_children():
    """Drafts of the target itself stand (a whole path is walked); drafts of another distribution fall (many residuals
    at one node)."""
    g, rng = torch.Generator().manual_seed(1), random.Random(1)
    target, draft, tokens, parents = drafts_of(g, rng, 16, 32, 500, "f32", "chain", True, noise=0.0)
    u = torch.rand((16, 32), generator=g)
    lens = check_verify(target, draft, tokens, None, u)
    assert min(lens) == 32
    target, draft, tokens, parents = drafts_of(g, rng, 16, 40, 500, "f32", "star", True, noise=6.0)
    lens = check_verify(target, draft, tokens, parents, torch.rand((16, 40), generator=g) * 0.2 + 0.8)
    assert 1 in lens and 2 in lens


@gpu
@pytest.mark.parametrize("vocab,dtype", [(300, "f32"), (4096, "bf16"), (4099, "f16"), (8192, "f32"), (8196, "f32"),
                                         (9001, "f32"), (8196, "bf16")])
def test_verify_drafts_of_many_sequences(vocab, dtype):
    g, rng = torch.Generator().manual_seed(2), random.Random(2)
    for drafts in (True, False):
        target, draft, tokens, parents = drafts_of(g, rng, 60, 7, vocab, dtype, "tree", drafts)
        check_verify(target, draft, tokens, parents, torch.rand((60, 7), generator=g))


@gpu
def test_weights_that_are_nearly_gone():
    """Children whose tokens take nearly all of the target's weight along: what is left is summed without them."""
    g = torch.Generator().manual_seed(8)
    batch, nodes, vocab = 16, 5, 3000
    rest = torch.softmax(torch.randn((batch, nodes, vocab), generator=g) * 2, -1)
    for left in (1e-2, 1e-5, 1e-8):
        p = rest * left
        p[:, :, 100:104] = (1 - left) / 4
        u = torch.ones((batch, nodes))
        u[:, 0] = torch.rand(batch, generator=g)
        tokens = [[0, 100, 101, 102, 103]] * batch
        # every child's number is above its chance: only the rest is left, where the fp32 numbers allow that
        lens = check_verify(p.float().cuda(), None, tokens, [[-1, 0, 0, 0, 0]] * batch, u * (1 - 2.0 ** -24))
        assert set(lens) <= {1, 2}


@gpu
def test_tokens_are_distributed_as_the_targets():
    """The first token of many sequences with the same probabilities, drafts drawn anew for each: its frequencies are the
    target's whatever the draft's.  40000 draws of 16 tokens: the chi-square statistic of 15 degrees of freedom is below 45
    but for a chance of 1e-4 (the seed is fixed)."""
    g = torch.Generator().manual_seed(3)
    n, vocab = 40000, 16
    p = torch.softmax(torch.randn(vocab, generator=g), -1)
    for children, noise in ((1, 1.0), (3, 1.5), (6, 3.0)):
        q = torch.softmax(p.log() + noise * torch.randn(vocab, generator=g), -1)
        nodes = children + 1
        tokens = torch.zeros(n, nodes, dtype=torch.int32)
        tokens[:, 1:] = torch.multinomial(q, n * children, replacement=True, generator=g).view(n, children)
        target = p.cuda().expand(n, nodes, vocab)
        draft = q.cuda().expand(n, nodes - 1, vocab)
        u = torch.rand((n, nodes), generator=g)
        path, lens, words, err = run_verify(target, draft, tokens, [random_parents(None, nodes, "star")] * n, u)
        assert err == 0 and target.stride(0) == 0
        seen = torch.bincount(words[:, 0].long(), minlength=vocab).double()
        want = n * p.double()
        assert ((seen - want) ** 2 / want).sum() < 45, (children, seen, want)
        assert 0 < (lens > 1).sum() < n


@gpu
def test_verify_drafts_of_special_probabilities():
    g, rng = torch.Generator().manual_seed(4), random.Random(4)
    target, draft, tokens, _ = drafts_of(g, rng, 8, 4, 700, "f32", "chain", True)
    u = torch.rand((8, 4), generator=g)
    # the draft equal to the target, and a child that it cannot have drawn: nothing is left, the target's row counts
    same = target[:, :3].clone()
    same[:, 0, 5] = target[:, 0, 5] = 0.0
    fallen = [list(t) for t in tokens]
    for t in fallen:
        t[1] = 5
    assert set(check_verify(target, same, fallen, None, u)) == {1}
    # uniforms at their ends
    for value in (0.0, 1.0, 2.0, -1.0, math.nan):
        check_verify(target, draft, tokens, None, torch.full((8, 4), value), margin=0)
    # rows of zeros give no token
    zero = target.clone()
    zero[3] = 0
    check_verify(zero, draft, tokens, None, u, flags=fd.DEVERR_PROB)
    # a row of one token, first and last
    for v in (0, 699):
        one = torch.zeros_like(target)
        one[:, :, v] = 1.0
        check_verify(one, draft, tokens, None, u, margin=0)
    # probabilities that are none count as 0 (NaN, below 0) or 2 (above)
    for bad in (math.nan, math.inf, -math.inf, -0.25, 17.0):
        odd = target.clone()
        odd[:, :, 11] = bad
        check_verify(odd, draft, tokens, None, u, flags=fd.DEVERR_PROB)


@gpu
def test_verify_drafts_of_odd_trees_and_tokens():
    g, rng = torch.Generator().manual_seed(5), random.Random(5)
    batch, nodes = 12, 14
    target, draft, tokens, parents = drafts_of(g, rng, batch, nodes, 300, "f32", "tree", False)
    u = torch.rand((batch, nodes), generator=g)
    # nodes that do not hang together with node 0
    loose = [[-1] + [p if rng.random() < 0.6 else -1 for p in row[1:]] for row in parents]
    check_verify(target, None, tokens, loose, u)
    # two children with one token: the second finds it without weight
    twice = [list(t) for t in tokens]
    for t in twice:
        t[2:6] = [t[1]] * 4
    star = [random_parents(rng, nodes, "star")] * batch
    check_verify(target, None, twice, star, u)
    # bad parents and tokens
    bad = [list(p) for p in parents]
    bad[2][4], bad[5][1], bad[6][0] = 4, -3, 2
    fixed = [list(p) for p in parents]
    fixed[2][4] = fixed[5][1] = fixed[6][0] = -1
    path, lens, words, err = run_verify(target, None, tokens, bad, u)
    want = run_verify(target, None, tokens, fixed, u)
    assert err == fd.DEVERR_TREE and want[3] == 0
    assert torch.equal(path, want[0]) and torch.equal(lens, want[1]) and torch.equal(words, want[2])
    wrong = [list(t) for t in tokens]
    for t in wrong:
        t[1], t[2] = 300, -1
    check_verify(target, None, wrong, star, u, flags=fd.DEVERR_TREE)
    path, lens, words, err = run_verify(target, None, tokens, parents, u, counts=[3, -1, 15] + [14] * 9)
    assert err == fd.DEVERR_SEQ_LEN and lens[1] == 0 and (path[1] == -1).all() and (words[1] == -1).all()


@gpu
def test_verify_drafts_takes_strided_probabilities():
    g, rng = torch.Generator().manual_seed(6), random.Random(6)
    for dtype, vocab, pad, shift in (("f32", 1000, 24, 0), ("f32", 1000, 25, 3), ("bf16", 777, 3, 1), ("f16", 512, 0, 2)):
        target, draft, tokens, _ = drafts_of(g, rng, 6, 5, vocab, dtype, "chain", True)
        u = torch.rand((6, 5), generator=g)
        want = run_verify(target, draft, tokens, None, u)
        wide = torch.full((6, 5, vocab + pad + shift), math.nan, dtype=target.dtype, device="cuda")
        wide[:, :, shift:shift + vocab] = target
        other = torch.full((4, 6, vocab + pad + shift), math.nan, dtype=target.dtype, device="cuda")
        other[:, :, shift:shift + vocab] = draft[:, :4].transpose(0, 1)
        got = run_verify(wide[:, :, shift:shift + vocab], other[:, :, shift:shift + vocab].transpose(0, 1), tokens, None, u)
        assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3])) and got[3] == 0
        check_verify(target, draft, tokens, None, u)


# --------------------------------------------------------------------------------------------------------- kept paths

def keep_reference(pools, table, prefix, path, lens, page):
    out = [bits(p).clone().view(p.dtype).view(p.shape) if p.is_contiguous() else p.clone() for p in pools]
    for x, p in zip(out, pools):
        for b, n in enumerate(lens):
            rows = [x[..., int(table[b, (prefix[b] + v) // page]), :, (prefix[b] + v) % page, :].clone()
                    for v in path[b][:n]]
            for i, r in enumerate(rows):
                x[..., int(table[b, (prefix[b] + i) // page]), :, (prefix[b] + i) % page, :] = r
    return out


def random_paths(rng, batch, nodes):
    paths, lens = np.full((batch, nodes), -1, dtype=np.int32), []
    for b in range(batch):
        n = rng.choice([0, 1, nodes, rng.randrange(0, nodes + 1), rng.randrange(0, nodes + 1)])
        paths[b, :n] = sorted(rng.sample(range(nodes), n))
        lens.append(n)
    return paths, lens


def keep_case(rng, batch, nodes, page):
    prefix = [rng.randrange(0, 4 * page) for _ in range(batch)]
    width = (4 * page + nodes) // page + 1
    order = list(range(batch * width + 3))
    rng.shuffle(order)
    table = np.array([[order.pop() for _ in range(width)] for _ in range(batch)], dtype=np.int32)
    return prefix, table, batch * width + 3


@gpu
@pytest.mark.parametrize("nodes,page,batch,hk,d,layers,dtype,layout", [
    (8, 16, 5, 2, 128, 3, "bf16", "hnd"), (64, 16, 3, 2, 64, 2, "f16", "nhd"), (16, 1, 4, 1, 64, 1, "bf16", "hnd"),
    (24, 8, 6, 4, 256, 2, "fp8", "interleaved"), (1, 64, 3, 2, 128, 2, "bf16", "hnd"), (33, 256, 2, 3, 192, 2, "bf16", "nhd"),
    (12, 16, 40, 8, 128, 5, "f16", "interleaved"), (5, 4, 3, 1, 512, 1, "f16", "hnd"),
])
def test_keep_path(nodes, page, batch, hk, d, layers, dtype, layout):
    rng = random.Random(nodes)
    for seed in range(3):
        prefix, table, pages = keep_case(rng, batch, nodes, page)
        k, v = make_pool(pages, hk, page, d, dtype, layout, seed, layers=layers)
        path, lens = random_paths(rng, batch, nodes)
        want = keep_reference([k, v], table, prefix, path.tolist(), lens, page)
        out = torch.full((batch,), -9, dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        fd.fdec_keep_path((k, v), i32(table), i32(prefix), i32(path), i32(lens), out, page, device_errors=err)
        assert int(err.item()) == 0
        assert torch.equal(bits(k), bits(want[0])) and torch.equal(bits(v), bits(want[1]))
        assert out.tolist() == [p + n for p, n in zip(prefix, lens)]


@gpu
def test_keep_path_of_caches_of_different_shapes():
    """Layers for themselves, another number of heads and types, rows of 8 bytes (block scales), a pool of more pages."""
    rng = random.Random(2)
    prefix, table, pages = keep_case(rng, 4, 20, 16)
    g = torch.Generator().manual_seed(2)
    pools = [torch.randn((pages + i, 1 + i % 3, 16, (64, 128, 4, 20, 256)[i % 5]), generator=g).half().cuda()
             for i in range(40)]
    path, lens = random_paths(rng, 4, 20)
    want = keep_reference(pools, table, prefix, path.tolist(), lens, 16)
    out = torch.empty(4, dtype=torch.int32, device="cuda")
    fd.fdec_keep_path(pools, i32(table), i32(prefix), i32(path), i32(lens), out, 16)
    for a, b in zip(pools, want):
        assert torch.equal(a, b)


@gpu
def test_keep_path_flags_bad_paths_pages_and_lengths():
    rng = random.Random(3)
    prefix, table, pages = keep_case(rng, 3, 10, 16)
    prefix = [5, 20, 40]

    def call(path, lens, prefix=prefix, table=table):
        k, v = make_pool(pages, 2, 16, 64, "bf16", "hnd", 1)
        out = torch.full((3,), -9, dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        fresh = k.clone(), v.clone()
        fd.fdec_keep_path([k, v], i32(table), i32(prefix), i32(path), i32(lens), out, 16, device_errors=err)
        return int(err.item()), k, v, out.tolist(), fresh

    good = [[0, 2, 5, 9] + [-1] * 6, [1, 3, 4] + [-1] * 7, [0, 1, 2, 7] + [-1] * 6]
    for row, bad, upto in ((0, [0, 2, 2, 9], 2), (1, [3, 1, 4], 1), (2, [0, 1, 2, 10], 3), (2, [-1, 1, 2, 3], 0),
                           (0, [0, 5, -1, 7], 2)):
        path = [list(p) for p in good]
        path[row] = bad + [-1] * (10 - len(bad))
        lens = [4, 3, 4]
        err, k, v, out, fresh = call(path, lens)
        assert err == fd.DEVERR_TREE
        lens[row] = upto
        want = keep_reference(fresh, table, prefix, path, lens, 16)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and out == [p + n for p, n in zip(prefix, lens)]
    full = [list(range(10))] * 3
    err, k, v, out, fresh = call(full, [-1, 11, 10])
    assert err == fd.DEVERR_SEQ_LEN and out == [5, 30, 50] and torch.equal(k, fresh[0])
    for page in (-1, pages):
        broken = table.copy()
        broken[2, 2] = page  # positions 32 .. 47 of sequence 2: nodes 0 .. 7
        err, k, v, out, fresh = call(good, [4, 3, 4], table=broken)
        want = keep_reference(fresh, table, prefix, good, [4, 3, 0], 16)
        assert err == fd.DEVERR_PAGE_ID and torch.equal(k, want[0]) and out == [9, 23, 44]


# -------------------------------------------------------------------------------------------------------------- pages

def reserve_reference(table, lens, new, sources, num_pages, page):
    """(table, granted, copies [(sequence, from page, to page, rows)])."""
    batch, width = table.shape
    table, granted, copies = table.copy(), list(lens), []
    old = table.copy()
    named = {}
    for b in range(batch):
        for p in old[b, :-(-lens[b] // page)]:
            if 0 <= p < num_pages:
                named[int(p)] = named.get(int(p), 0) + 1
    free = [p for p in range(num_pages) if p not in named]
    taken = 0
    for b in range(batch):
        a = b if sources is None or sources[b] < 0 else sources[b]
        kept = min(lens[a], new[b])
        want, part = -(-new[b] // page), 0
        if a != b:
            first, part = kept // page, kept % page
        elif new[b] <= lens[b]:
            granted[b] = new[b]
            continue
        else:
            first = -(-lens[b] // page)
            if lens[b] % page and named.get(int(old[b, lens[b] // page]), 0) > 1:
                first, part = lens[b] // page, lens[b] % page
        need = max(0, want - first)
        taken += need
        if need and taken > len(free):
            continue
        granted[b] = new[b]
        if a != b:
            table[b, :first] = old[a, :first]
        table[b, first:first + need] = free[taken - need:taken]
        if part:
            copies.append((b, int(old[a, first]), int(table[b, first]), part))
    return table, granted, copies


def run_reserve(table, lens, new, sources, num_pages, page, caches=()):
    t, granted = i32(table), torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((fd.fdec_reserve_pages_workspace(len(lens), num_pages),), 255, dtype=torch.uint8, device="cuda")
    fd.fdec_reserve_pages(t, i32(lens), i32(new), granted, num_pages, page, ws, sources=None if sources is None else i32(sources),
                          caches=caches, device_errors=err)
    return t.cpu().numpy(), granted.tolist(), int(err.item())


def reserve_case(rng, batch, width, page, spare, shared=False):
    """Random tables: sequences with pages of their own, and some that begin with another's."""
    room = width * page
    lens = [rng.choice([0, 1, page, rng.randrange(0, room // 2 + 1), rng.randrange(0, room // 2 + 1)]) for _ in range(batch)]
    used = sum(-(-n // page) for n in lens)
    num_pages = used + spare
    order = list(range(num_pages))
    rng.shuffle(order)
    table = np.full((batch, width), -3, dtype=np.int32)
    for b, n in enumerate(lens):
        table[b, :-(-n // page)] = [order.pop() for _ in range(-(-n // page))]
    if shared:
        for b in range(1, batch):
            if rng.random() < 0.5:  # the same pages as an earlier sequence, up to a shorter or equal length
                a = rng.randrange(b)
                lens[b] = rng.choice([lens[a], rng.randrange(lens[a] + 1)])
                table[b] = table[a]
                table[b, -(-lens[b] // page):] = -3
    return table, lens, num_pages


@gpu
@pytest.mark.parametrize("batch,width,page,spare", [(1, 4, 16, 5), (5, 9, 8, 40), (33, 70, 16, 900), (300, 12, 1, 2000),
                                                    (700, 3, 64, 1500), (64, 2048, 16, 3000), (3, 5, 256, 0)])
@pytest.mark.parametrize("shared", [False, True])
def test_reserve_pages(batch, width, page, spare, shared):
    rng = random.Random(batch)
    for _ in range(4):
        table, lens, num_pages = reserve_case(rng, batch, width, page, spare, shared)
        new = [min(width * page, max(0, n + rng.choice([0, 1, 7, page, 3 * page, -5]))) for n in lens]
        got, granted, err = run_reserve(table, lens, new, None, num_pages, page)
        want, want_granted, _ = reserve_reference(table, lens, new, None, num_pages, page)
        refused = any(g < n for g, n, l in zip(want_granted, new, lens) if n > l)
        assert err == (fd.DEVERR_NO_PAGES if refused else 0)
        assert granted == want_granted and np.array_equal(got, want)


@gpu
@pytest.mark.parametrize("dtype,layout,page,hk,d,layers", [("bf16", "hnd", 16, 2, 64, 3), ("fp8", "nhd", 8, 4, 128, 2),
                                                           ("f16", "interleaved", 64, 1, 192, 1), ("bf16", "hnd", 1, 2, 64, 2)])
def test_forks_and_shared_last_pages_are_copied(dtype, layout, page, hk, d, layers):
    rng = random.Random(page)
    for seed in range(6):
        n = rng.randrange(1, 6)
        table, lens, num_pages = reserve_case(rng, n, 9, page, 60, shared=True)
        forks = rng.randrange(0, 9)
        table = np.concatenate([table, np.full((forks, 9), -3, dtype=np.int32)])
        sources = [rng.choice([-1, i]) for i in range(n)] + [rng.randrange(n) for _ in range(forks)]
        lens = lens + [0] * forks
        new = [min(9 * page, max(0, lens[b if a < 0 else a] + rng.choice([0, 1, 5, page, -3]))) for b, a in enumerate(sources)]
        order = list(range(n + forks))
        if seed % 2:  # forks before their sources
            rng.shuffle(order)
        place = {b: i for i, b in enumerate(order)}
        table = table[order]
        lens, new = [lens[b] for b in order], [new[b] for b in order]
        sources = [-1 if sources[b] < 0 else place[sources[b]] for b in order]
        k, v = make_pool(num_pages, hk, page, d, dtype, layout, seed, layers=layers)
        want_k, want_v = k.clone(), v.clone()
        want, want_granted, copies = reserve_reference(table, lens, new, sources, num_pages, page)
        for _, of, to, rows in copies:
            for w, x in ((want_k, k), (want_v, v)):
                w[:, to, :, :rows] = x[:, of, :, :rows]
        got, granted, err = run_reserve(table, lens, new, sources, num_pages, page, caches=(k, v))
        assert err == 0 and granted == want_granted and np.array_equal(got, want)
        assert torch.equal(bits(k), bits(want_k)) and torch.equal(bits(v), bits(want_v))


@gpu
def test_reserve_pages_flags_what_it_leaves_alone():
    page, width = 16, 4
    table = np.array([[3, 4, -3, -3], [5, -3, -3, -3], [-3] * 4, [-3] * 4], dtype=np.int32)
    lens = [20, 16, 0, 0]

    def call(new, sources=None, lens=lens, table=table, pages=8):
        return run_reserve(table, lens, new, sources, pages, page)

    got, granted, err = call([33, 17, 0, 0])
    assert err == 0 and granted == [33, 17, 0, 0] and got[0, 2] == 0 and got[1, 1] == 1
    got, granted, err = call([65, 17, 0, 0])  # past the table
    assert err == fd.DEVERR_SEQ_LEN and granted == [20, 17, 0, 0] and got[1, 1] == 0 and got[0, 2] == -3
    got, granted, err = call([-1, 17, 0, 0])
    assert err == fd.DEVERR_SEQ_LEN and granted == [20, 17, 0, 0]
    got, granted, err = call([20, 16, 20, 20], [-1, -1, 2, 9])  # itself is no source; no such sequence
    assert err == fd.DEVERR_SEQ_LEN and granted == [20, 16, 20, 0] and got[2].tolist() == [0, 1, -3, -3]
    got, granted, err = call([20, 16, 20, 20], [-1, -1, 0, 2])  # a fork of a fork
    assert err == fd.DEVERR_SEQ_LEN and granted == [20, 16, 20, 0] and got[2].tolist() == [3, 0, -3, -3]
    got, granted, err = call([20, 40, 0, 0], [-1, 0, -1, -1])  # a fork that has a length
    assert err == fd.DEVERR_SEQ_LEN and granted == [20, 16, 0, 0]
    got, granted, err = call([20, 40, 16, 16], lens=[20, -2, 0, 70], sources=[-1, -1, 0, -1])
    assert err == fd.DEVERR_SEQ_LEN | fd.DEVERR_PAGE_ID and granted == [20, -2, 16, 70]
    broken = table.copy()
    broken[0, 0], broken[1, 0] = -1, 8
    got, granted, err = call([33, 17, 0, 0], table=broken)
    assert err == fd.DEVERR_PAGE_ID and got[0].tolist() == [-1, 4, 0, -3] and got[1].tolist() == [8, 1, -3, -3]
    got, granted, err = call([64, 64, 16, 0], pages=8)  # five free pages: 2 + 3, and none for the third
    assert err == fd.DEVERR_NO_PAGES and granted == [64, 64, 0, 0]
    assert got[0].tolist() == [3, 4, 0, 1] and got[1].tolist() == [5, 2, 6, 7] and got[2, 0] == -3


@gpu
@pytest.mark.parametrize("num_pages", [31, 32, 33, 8191, 8192, 8193, 300007])
def test_reserve_pages_of_odd_pools(num_pages):
    rng = random.Random(num_pages)
    width, page = min(num_pages, 40000), 1
    used = sorted(rng.sample(range(num_pages), min(num_pages - 3, width - 8)))
    rng.shuffle(used)
    table = np.full((2, width), -3, dtype=np.int32)
    table[0, :len(used)] = used
    lens, new = [len(used), 0], [len(used) + 2, min(width, num_pages - len(used) - 2)]
    got, granted, err = run_reserve(table, lens, new, None, num_pages, page)
    want, want_granted, _ = reserve_reference(table, lens, new, None, num_pages, page)
    assert err == 0 and granted == want_granted == new and np.array_equal(got, want)


@gpu
def test_offsets_past_32_bits():
    """Pools of more than 4 GB of which the last pages are used (2 x 4.6 GB)."""
    hk, page, d, pages = 2, 128, 128, 70000
    k, v = (torch.empty((pages, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    used = [pages - 1 - i for i in range(6)]
    g = torch.Generator().manual_seed(1)
    for x in (k, v):
        x[used] = torch.randn((6, hk, page, d), generator=g).bfloat16().cuda()
    c = Tree(d, 8, hk, 20, page, 2, seed=16, counts=[20, 20], prefix=[120, 250])
    c.k, c.v = k, v
    c.table = np.array([[used[0], used[1], -1], [-1, used[2], used[3]]], dtype=np.int32)
    c.check(*c.run())
    table = np.array([used[:2], used[2:4]], dtype=np.int32)
    path, lens = np.array([[0, 3, 9, 19] + [-1] * 16, [1, 2] + [-1] * 18], dtype=np.int32), [4, 2]
    small = [x[used].clone() for x in (k, v)]
    want = keep_reference(small, np.array([[0, 1], [2, 3]]), [120, 100], path.tolist(), lens, page)
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    fd.fdec_keep_path((k, v), i32(table), i32([120, 100]), i32(path), i32(lens), out, page)
    assert torch.equal(k[used], want[0]) and torch.equal(v[used], want[1])
    # a fork whose last page is the pool's last free one: all others but two are in use
    width = pages // 4
    table = np.full((5, width), -1, dtype=np.int32)
    order = [p for p in range(pages) if p != used[4]]
    for b in range(4):
        mine = order[b * width:(b + 1) * width]
        table[b, :len(mine)] = mine
    lens = [width * page] * 3 + [(len(order) - 3 * width) * page - 5, 0]
    table[3, len(order) - 3 * width - 1] = used[0]
    table[3, len(order) - 3 * width:] = -1
    first = [x[used[0], :, :page - 5].clone() for x in (k, v)]
    got, granted, err = run_reserve(table, lens, lens[:4] + [lens[3]], [-1, -1, -1, -1, 3], pages, page, caches=(k, v))
    want, want_granted, copies = reserve_reference(table, lens, lens[:4] + [lens[3]], [-1, -1, -1, -1, 3], pages, page)
    assert err == 0 and granted == want_granted and np.array_equal(got, want)
    (_, of, to, rows), = copies
    assert of == used[0] and rows == page - 5
    for x, w in zip((k, v), first):
        assert torch.equal(x[to, :, :rows], w)


# ------------------------------------------------------------------------------------------------------- a whole round

def causal_reference(q, k, v, scale, line):
    """q [Q, Hq, D], k / v [T, Hk, D] in 64 bits, line [Q, T] what each query sees."""
    group = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    z = torch.einsum("qhd,thd->hqt", q, k) * scale
    z = torch.where(line, z, -math.inf)
    return torch.einsum("hqt,thd->qhd", torch.softmax(z, -1), v)


@gpu
@pytest.mark.parametrize("graph", [False, True])
def test_rounds_of_speculative_decoding(graph):
    """Forks of prompts, then rounds of drafting, attention in two layers, verification and keeping, eager or replayed from
    one graph; after every round the caches hold what a plain list of the accepted rows holds, and the attention of
    the next round's nodes is that over these lists."""
    torch.manual_seed(0)
    batch, nodes, page, hq, hk, d, layers, vocab, pages = 4, 9, 16, 8, 2, 128, 2, 64, 96
    rng = random.Random(0)
    width = 24
    k = torch.randn(layers, pages, hk, page, d, device="cuda").bfloat16()
    v = torch.randn(layers, pages, hk, page, d, device="cuda").bfloat16()
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    tree = fd.TreeDecode([300] * batch, nodes, page, hq, hk, d, pages, "bf16")
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    # two prompts of 37 and 64 tokens, two forks of the first
    ws = torch.empty(fd.fdec_reserve_pages_workspace(batch, pages), dtype=torch.uint8, device="cuda")
    granted = torch.empty_like(lens)
    fd.fdec_reserve_pages(table, lens, i32([37, 64, 0, 0]), granted, pages, page, ws)
    assert granted.tolist() == [37, 64, 0, 0]
    lens.copy_(granted)
    fd.fdec_reserve_pages(table, lens, i32([37, 64, 37, 37]), granted, pages, page, ws, sources=i32([-1, -1, 0, 0]),
                          caches=(k, v))
    lens.copy_(granted)
    assert lens.tolist() == [37, 64, 37, 37] and table[2, :2].tolist() == table[0, :2].tolist()
    assert len(set(table[[0, 2, 3], 2].tolist())) == 3

    def rows_of(pool, b, n):
        at = torch.arange(n, device="cuda")
        return pool[:, table[b].long()[at // page], :, at % page]  # [n, layers, Hk, D]

    lists = [[rows_of(k, b, n).clone(), rows_of(v, b, n).clone()] for b, n in enumerate(lens.tolist())]
    half = d // 2
    angle = torch.arange(400, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(half, dtype=torch.float64, device="cuda") / half)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    qkv = torch.empty(layers, batch * nodes, hq + 2 * hk, d, device="cuda", dtype=torch.bfloat16)
    parents, depths = (torch.zeros(batch, nodes, dtype=torch.int32, device="cuda") for _ in range(2))
    target = torch.empty(batch, nodes, vocab, device="cuda")
    tokens = torch.zeros(batch, nodes, dtype=torch.int32, device="cuda")
    uniforms = torch.empty(batch, nodes, device="cuda")
    outs = [torch.empty(batch, nodes, hq, d, device="cuda") for _ in range(layers)]

    def step():
        tree.reserve(table, lens, caches=(k, v))
        for l in range(layers):
            tree.attend(qkv[l, :, :hq], qkv[l, :, hq:hq + hk], qkv[l, :, hq + hk:], None, None, cos_sin, k[l], v[l], table,
                        lens, parents, depths, outs[l])
        tree.verify(target, None, tokens, parents, uniforms)
        lens.copy_(tree.keep((k, v), table, lens))

    captured = None
    for turn in range(5):
        trees = [random_parents(rng, nodes, "tree") for _ in range(batch)]
        parents.copy_(i32(trees))
        depths.copy_(i32([[len(path_of(t, i)) - 1 for i in range(nodes)] for t in trees]))
        fresh = torch.randn(qkv.shape, device="cuda").bfloat16()
        target.copy_(torch.softmax(torch.randn(target.shape, device="cuda") * 3, -1))
        best = target.topk(nodes, -1)[1]
        for b in range(batch):
            used = {}
            for i in range(1, nodes):
                p = trees[b][i]
                tokens[b, i] = best[b, p, used.get(p, 0)]
                used[p] = used.get(p, 0) + 1
        uniforms.copy_(torch.rand(uniforms.shape, device="cuda"))
        before = lens.tolist()
        if graph and captured is None:
            qkv.copy_(fresh)
            saved = [x.clone() for x in (lens, table, k, v)]
            step()  # warm-up, undone
            for x, s in zip((lens, table, k, v), saved):
                x.copy_(s)
            torch.cuda.synchronize()
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
            for x, s in zip((lens, table, k, v), saved):
                x.copy_(s)
        qkv.copy_(fresh)
        if graph:
            captured.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert tree.device_errors() == 0
        path, path_lens = tree.path.tolist(), tree.path_lens.tolist()
        for b in range(batch):
            kept = path[b][:path_lens[b]]
            assert kept == path_of(trees[b], kept[-1]) and lens[b] == before[b] + len(kept)
            new_k = rows_of(k, b, int(lens[b]))
            assert torch.equal(new_k[:before[b]], lists[b][0])  # the prefix is as it was
            rows = torch.tensor(kept, device="cuda")
            v_rows = fresh[:, b * nodes + rows, hq + hk:].transpose(0, 1)  # [n, layers, Hk, D]
            lists[b][1] = torch.cat([lists[b][1], v_rows])
            assert torch.equal(rows_of(v, b, int(lens[b])), lists[b][1])
            # keys: the normed rows rotated by prefix + depth = the position they now have
            x = fresh[:, b * nodes + rows, hq:hq + hk].transpose(0, 1).double()
            x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            turn_by = cos_sin[before[b] + torch.arange(len(kept), device="cuda")].double()[:, None, None]
            c, s = turn_by[..., :half], turn_by[..., half:]
            want = torch.cat([x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s], -1)
            got = new_k[before[b]:].double()
            assert (got - want).abs().max() <= 2.0 ** -8 * want.abs().max() + 1e-6  # half a bf16 step
            # attention of the accepted nodes over the list itself: prefix and path, causally
            for l in range(layers):
                q = qkv[l, b * nodes + rows, :hq].double()  # normed and rotated in place
                total = before[b] + len(kept)
                line = torch.arange(total, device="cuda") <= before[b] + torch.arange(len(kept), device="cuda")[:, None]
                want = causal_reference(q, new_k[:, l].double(), lists[b][1][:, l].double(), 1 / math.sqrt(d), line)
                got = outs[l][b, rows].double()
                assert (got - want).abs().max() <= 2e-3 * want.abs().max()  # the prefix's own tolerance
            lists[b][0] = new_k.clone()
    assert max(lens.tolist()) > 64


@gpu
def test_chain_of_drafts_equals_the_causal_call():
    """prefix + chain, joined, against one causal call over the same cache."""
    batch, nodes, page, hq, hk, d = 3, 7, 16, 16, 4, 128
    prefix = [100, 1, 250]
    lens = [p + nodes for p in prefix]
    width = max(lens) // page + 1
    k, v = make_pool(batch * width, hk, page, d, "bf16", "hnd", 4)
    table = i32(np.random.default_rng(0).permutation(batch * width).reshape(batch, width))
    q = torch.randn(batch, nodes, hq, d).bfloat16().cuda()
    want, want_lse = torch.empty(batch, nodes, hq, d, device="cuda"), torch.empty(batch, nodes, hq, device="cuda")
    fd.PagedDecode(lens, nodes, page, hq, hk, d, "bf16", causal=True).run(q, k, v, table, i32(lens), want, want_lse)
    o, lse = torch.empty_like(want), torch.empty_like(want_lse)
    fd.PagedDecode(prefix, nodes, page, hq, hk, d, "bf16").run(q, k, v, table, i32(prefix), o, lse)
    fd.fdec_tree_attention(q, k, v, table, i32(prefix), None, o, lse, o, lse, page)
    assert (o - want).abs().max() <= 2 * 2e-3 * want.abs().max()
    assert (lse - want_lse).abs().max() <= 2e-4


@gpu
def test_calls_use_the_stream_they_are_given():
    """Inputs written on a stream just before the call, on that stream."""
    c = Tree(128, 8, 2, 10, 16, 3, seed=12)
    want, _ = c.run()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q, out, lse = torch.zeros_like(c.q), torch.full_like(want, 3.0), torch.empty(c.q.shape[:3], device="cuda")
    args = i32(c.table), i32(c.prefix), i32(c.parents)
    counts = i32(c.counts)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2_000_000)
        q.copy_(c.q)
        fd.fdec_tree_attention(q, c.k, c.v, *args, c.o_prefix, c.lse_prefix, out, lse, c.page, node_counts=counts)
    stream.synchronize()
    assert torch.equal(want, out)
    g, rng = torch.Generator().manual_seed(9), random.Random(9)
    target, draft, tokens, _ = drafts_of(g, rng, 6, 5, 1000, "f32", "chain", True)
    u = torch.rand((6, 5), generator=g)
    want = run_verify(target, draft, tokens, None, u)
    late = torch.zeros_like(target)
    path, words = (torch.empty((6, 5), dtype=torch.int32, device="cuda") for _ in range(2))
    lens, tok, u = torch.empty(6, dtype=torch.int32, device="cuda"), i32(tokens), u.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2_000_000)
        late.copy_(target)
        fd.fdec_verify_drafts(late, draft, tok, None, u, path, lens, words)
    stream.synchronize()
    assert torch.equal(path.cpu(), want[0]) and torch.equal(words.cpu(), want[2])
    # pages, then rows, on that stream, lengths written just before
    pool = torch.randn(12, 2, 16, 64).half().cuda()
    fresh, table = pool.clone(), i32(np.arange(12).reshape(2, 6))
    prefix, soon = i32([3, 20]), torch.zeros(2, dtype=torch.int32, device="cuda")
    kept, path_lens = i32([[0, 4, 9] + [-1] * 13, [2, 3, 15] + [-1] * 13]), i32([3, 2])  # of 16 nodes
    out, granted, table2 = torch.empty_like(soon), torch.empty_like(soon), i32(np.full((2, 6), -1))
    ws = torch.empty(fd.fdec_reserve_pages_workspace(2, 12), dtype=torch.uint8, device="cuda")
    more, none = i32([33, 17]), torch.full((2,), 7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2_000_000)
        soon.copy_(prefix)
        none.zero_()
        fd.fdec_keep_path([pool], table, soon, kept, path_lens, out, 16)
        fd.fdec_reserve_pages(table2, none, more, granted, 12, 16, ws)
    stream.synchronize()
    want = keep_reference([fresh], table.cpu().numpy(), [3, 20], kept.tolist(), [3, 2], 16)[0]
    assert torch.equal(pool, want) and out.tolist() == [6, 22]
    assert granted.tolist() == [33, 17] and table2[:, :3].tolist() == [[0, 1, 2], [3, 4, -1]]


@gpu
def test_two_captured_graphs_of_one_holder():
    """The rounds of two batches of one size, captured one after the other with the same workspaces, replayed in turns."""
    batch, nodes, page, pages, vocab = 3, 6, 16, 64, 200
    g, rng = torch.Generator().manual_seed(10), random.Random(10)
    tree = fd.TreeDecode([200] * batch, nodes, page, 8, 2, 64, pages, "f16")
    sides = []
    for _ in range(2):
        target, draft, tokens, parents = drafts_of(g, rng, batch, nodes, vocab, "f32", "tree", False)
        side = dict(target=target, tokens=i32(tokens), parents=i32(parents), u=torch.rand((batch, nodes), generator=g).cuda(),
                    table=torch.full((batch, 13), -1, dtype=torch.int32, device="cuda"),
                    lens=i32([0] * batch), pool=torch.randn(pages, 2, page, 64).half().cuda(),
                    out=[torch.zeros_like(tree.path), torch.zeros_like(tree.path_lens), torch.zeros_like(tree.path)])
        sides.append(side)

    def step(s):
        tree.reserve(s["table"], s["lens"])
        got = tree.verify(s["target"], None, s["tokens"], s["parents"], s["u"])
        for a, b in zip(s["out"], got):
            a.copy_(b)
        s["lens"].copy_(tree.keep([s["pool"]], s["table"], s["lens"]))

    graphs = []
    for s in sides:
        saved = {k: s[k].clone() for k in ("table", "lens", "pool")}
        step(s)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(s)
        for k, v in saved.items():
            s[k].copy_(v)
    want = [dict(table=s["table"].cpu().numpy(), lens=[0] * batch, pool=s["pool"].clone()) for s in sides]
    for turn in range(8):
        which = rng.randrange(2)
        s, w = sides[which], want[which]
        graphs[which].replay()
        torch.cuda.synchronize()
        w["table"], granted, _ = reserve_reference(w["table"], w["lens"], [n + nodes for n in w["lens"]], None, pages, page)
        paths = []
        for b in range(batch):
            path, words, _ = verify_reference(s["target"][b].cpu().numpy(), None, s["tokens"][b].tolist(),
                                              s["parents"][b].tolist(), s["u"][b].tolist(), nodes)
            paths.append(path)
            assert s["out"][0][b].tolist()[:len(path)] == path and s["out"][2][b].tolist()[:len(words)] == words
        w["pool"] = keep_reference([w["pool"]], w["table"], w["lens"], paths, [len(p) for p in paths], page)[0]
        w["lens"] = [n + len(p) for n, p in zip(w["lens"], paths)]
        assert s["lens"].tolist() == w["lens"] and np.array_equal(s["table"].cpu().numpy(), w["table"])
        assert torch.equal(s["pool"], w["pool"])
    assert tree.device_errors() == 0


@gpu
def test_a_sequence_without_pages_stands_still():
    """Its old entries name pages that are others' by now: no row is written there, and its length stays."""
    batch, nodes, page, hq, hk, d, vocab, pages = 3, 9, 16, 8, 2, 128, 64, 8
    torch.manual_seed(3)
    k = torch.randn(pages, hk, page, d, device="cuda").bfloat16()
    v = torch.randn(pages, hk, page, d, device="cuda").bfloat16()
    tree = fd.TreeDecode([60] * batch, nodes, page, hq, hk, d, pages, "bf16")
    lens = i32([30, 31, 32])
    table = i32([[0, 1, 2, 3], [2, 3, 0, 1], [4, 5, 0, 1]])  # entries past the lengths: another's pages
    qkv = torch.randn(batch * nodes, hq + 2 * hk, d, device="cuda").bfloat16()
    fresh = qkv.clone()
    cos_sin = torch.cat([torch.ones(200, d // 2), torch.zeros(200, d // 2)], 1).cuda()
    target = torch.softmax(torch.randn(batch, nodes, vocab, device="cuda"), -1)
    tokens, u = torch.zeros(batch, nodes, dtype=torch.int32, device="cuda"), torch.rand(batch, nodes, device="cuda")
    counts = i32([nodes, nodes - 2, nodes])
    out = torch.full((batch, nodes, hq, d), 7.0, device="cuda")

    def round_of():
        granted = tree.reserve(table, lens, (k, v)).tolist()
        tree.attend(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], None, None, cos_sin, k, v, table, lens, None, None,
                    out, node_counts=counts)
        path, path_lens, words = tree.verify(target, None, tokens, None, u, counts)
        return granted, path.tolist(), path_lens.tolist(), words.tolist(), tree.keep((k, v), table, lens).tolist()

    before_k, before_v = k.clone(), v.clone()
    granted, path, path_lens, words, kept = round_of()
    assert granted == [39, 40, 32]  # two pages were free
    assert tree.device_errors() == fd.DEVERR_NO_PAGES | fd.DEVERR_SEQ_LEN
    assert path[2] == [-1] * nodes and path_lens[2] == 0 and words[2] == [-1] * nodes and kept[2] == 32
    assert min(path_lens[:2]) >= 1 and kept[:2] == [30 + path_lens[0], 31 + path_lens[1]]
    assert torch.equal(qkv[2 * nodes:, :hq], fresh[2 * nodes:, :hq]) and (out[2] == 7).all()
    assert (out[0] != 7).all() and (out[1, :nodes - 2] != 7).all() and (out[1, nodes - 2:] == 7).all()
    for pool, before in ((k, before_k), (v, before_v)):
        changed = (pool != before).any(-1).any(1)  # [page, slot]
        assert not changed[[0, 2, 4, 5]].any()
        assert not changed[1, :14].any() and not changed[3, :15].any()
    for b in range(2):
        at = torch.arange(path_lens[b], device="cuda") + int(lens[b])
        rows = torch.tensor(path[b][:path_lens[b]], device="cuda") + b * nodes
        assert torch.equal(v[table[b].long()[at // page], :, at % page], fresh[rows, hq + hk:])
    lens.copy_(i32([0, kept[1], 32]))  # a sequence has ended: its pages are there for the third
    granted, path, path_lens, words, kept = round_of()
    assert granted[2] == 41 and path_lens[2] >= 1 and kept[2] == 32 + path_lens[2] and (out[2] != 7).all()
    assert tree.device_errors() == 0


@gpu
@pytest.mark.parametrize("default", [False, True])
@pytest.mark.parametrize("handle", [False, True])
def test_a_round_on_a_stream_of_its_own(handle, default):
    """The current stream is busy meanwhile: nothing of the round waits for it."""
    batch, nodes, page, hq, hk, d, vocab, pages = 2, 5, 16, 4, 2, 64, 32, 16
    torch.manual_seed(4)
    k = torch.randn(pages, hk, page, d, device="cuda").half()
    v = torch.randn(pages, hk, page, d, device="cuda").half()
    tree = fd.TreeDecode([60] * batch, nodes, page, hq, hk, d, pages, "f16")
    lens, table = i32([20, 16]), i32([[3, 1, 0, 0], [2, 0, 0, 0]])
    qkv = torch.randn(batch * nodes, hq + 2 * hk, d, device="cuda").half()
    cos_sin = torch.randn(100, d, device="cuda")
    parents, depths = i32([[-1, 0, 0, 1, 1]] * batch), i32([[0, 1, 1, 2, 2]] * batch)
    target = torch.softmax(torch.randn(batch, nodes, vocab, device="cuda"), -1)
    tokens, u = i32([[0, 1, 2, 3, 4]] * batch), torch.rand(batch, nodes, device="cuda")
    counts = i32([5, 4])

    def round_of(stream):
        state = [x.clone() for x in (k, v, table, qkv)]
        out = torch.zeros(batch, nodes, hq, d, device="cuda")
        torch.cuda.synchronize()
        if stream is not None:
            torch.cuda._sleep(200_000_000)
        kk, vv, tt, x = state
        tree.reserve(tt, lens, (kk, vv), stream=stream)
        tree.attend(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], None, None, cos_sin, kk, vv, tt, lens, parents, depths, out,
                    node_counts=counts, stream=stream)
        tree.verify(target, None, tokens, parents, u, counts, stream=stream)
        tree.keep((kk, vv), tt, lens, stream=stream)
        errors = tree.device_errors(stream=stream)
        busy = stream is not None and not torch.cuda.current_stream().query()
        torch.cuda.synchronize()
        return [*state, out, tree.path.clone(), tree.path_lens.clone(), tree.tokens.clone(), tree.seq_lens.clone()], errors, busy

    want, errors, _ = round_of(None)
    assert errors == 0
    side, main = torch.cuda.Stream(), torch.cuda.default_stream()
    own, current = (main, side) if default else (side, main)
    with torch.cuda.stream(current):
        got, errors, busy = round_of(own.cuda_stream if handle else own)
    assert errors == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
    assert busy  # (the round ended first)


# ------------------------------------------------------------------------------------------------------------ refusals

def cpu_tree(**kw):
    a = dict(q=torch.zeros(2, 4, 8, 128, dtype=torch.bfloat16), k=torch.zeros(6, 2, 16, 128, dtype=torch.bfloat16),
             v=torch.zeros(6, 2, 16, 128, dtype=torch.bfloat16), page_table=torch.zeros(2, 3, dtype=torch.int32),
             prefix_lens=torch.zeros(2, dtype=torch.int32), parents=torch.zeros(2, 4, dtype=torch.int32),
             o_prefix=torch.zeros(2, 4, 8, 128), lse_prefix=torch.zeros(2, 4, 8), out=torch.zeros(2, 4, 8, 128),
             lse=torch.zeros(2, 4, 8), page_size=16)
    a.update(kw)
    fd.fdec_tree_attention(**a)


def refused(status, call, **kw):
    with pytest.raises(fd.FdecError) as e:
        call(**kw)
    assert e.value.status_name == status, e.value


def test_tree_attention_refusals():
    with pytest.raises(ValueError, match="CUDA device"):
        cpu_tree()
    with pytest.raises(ValueError):
        cpu_tree(q=torch.zeros(2, 4, 8, 128))
    with pytest.raises(ValueError):
        cpu_tree(parents=torch.zeros(2, 5, dtype=torch.int32))
    with pytest.raises(ValueError):
        cpu_tree(parents=torch.zeros(2, 4, dtype=torch.int64))
    with pytest.raises(ValueError):
        cpu_tree(out=torch.zeros(2, 4, 8, 128, dtype=torch.float16))
    with pytest.raises(ValueError):
        cpu_tree(page_size=32)
    with pytest.raises(ValueError):
        cpu_tree(node_counts=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        cpu_tree(o_prefix=torch.zeros(2, 4, 8, 64))
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, o_prefix=None)
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, scale=math.inf)
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, v_scale=math.nan)
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, k=torch.zeros(6, 3, 16, 128, dtype=torch.bfloat16),
            v=torch.zeros(6, 3, 16, 128, dtype=torch.bfloat16))  # 8 heads over 3
    refused("FDEC_ERR_UNSUPPORTED", cpu_tree, q=torch.zeros(2, 65, 8, 128, dtype=torch.bfloat16), parents=None,
            o_prefix=None, lse_prefix=None, out=torch.zeros(2, 65, 8, 128), lse=None)
    refused("FDEC_ERR_UNSUPPORTED", cpu_tree, q=torch.zeros(2, 4, 8, 80, dtype=torch.bfloat16),
            k=torch.zeros(6, 2, 16, 80, dtype=torch.bfloat16), v=torch.zeros(6, 2, 16, 80, dtype=torch.bfloat16),
            o_prefix=None, lse_prefix=None, out=torch.zeros(2, 4, 8, 80))
    refused("FDEC_ERR_UNSUPPORTED", cpu_tree, k=torch.zeros(6, 2, 12, 128, dtype=torch.bfloat16),
            v=torch.zeros(6, 2, 12, 128, dtype=torch.bfloat16), page_size=12)
    refused("FDEC_ERR_LAYOUT", cpu_tree, q=torch.zeros(2 * 4 * 8 * 128 + 1, dtype=torch.bfloat16)[1:].view(2, 4, 8, 128))
    both = torch.zeros(2 * 2 * 4 * 8 * 128)
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, o_prefix=both[:8192].view(2, 4, 8, 128), out=both[4096:12288].view(2, 4, 8, 128))
    q = torch.zeros(2, 4, 8, 128, dtype=torch.bfloat16)
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, q=q, out=q)
    half = torch.zeros(2 * 8192, dtype=torch.bfloat16)
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, q=half[:8192].view(2, 4, 8, 128), out=half[8064:16256].view(2, 4, 8, 128))
    # (the last row of a strided q overlaps)
    wide = torch.zeros(8 * 3 * 1024 + 8192, dtype=torch.bfloat16)
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, q=wide[:8 * 3 * 1024].view(2, 4, 24, 128)[:, :, :8],
            out=wide[7 * 3 * 1024:][:8192].view(2, 4, 8, 128))
    f = torch.zeros(8192 + 64)
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, out=f[:8192].view(2, 4, 8, 128), lse=f[8160:8224].view(2, 4, 8))
    some = torch.zeros(8192)
    refused("FDEC_ERR_INVALID_ARG", cpu_tree, o_prefix=some.view(2, 4, 8, 128),
            out=some.view(torch.bfloat16)[:8192].view(2, 4, 8, 128))  # a 16-bit result over the fp32 state


def cpu_verify(**kw):
    a = dict(target_probs=torch.zeros(2, 4, 10), draft_probs=torch.zeros(2, 3, 10),
             tokens=torch.zeros(2, 4, dtype=torch.int32), parents=None, uniforms=torch.zeros(2, 4),
             path=torch.zeros(2, 4, dtype=torch.int32), path_lens=torch.zeros(2, dtype=torch.int32),
             out_tokens=torch.zeros(2, 4, dtype=torch.int32))
    a.update(kw)
    fd.fdec_verify_drafts(**a)


def test_verify_drafts_refusals():
    with pytest.raises(ValueError, match="CUDA device"):
        cpu_verify()
    with pytest.raises(ValueError):
        cpu_verify(target_probs=torch.zeros(2, 4, 10, dtype=torch.float64))
    with pytest.raises(ValueError):
        cpu_verify(draft_probs=torch.zeros(2, 2, 10))
    with pytest.raises(ValueError):
        cpu_verify(draft_probs=torch.zeros(2, 3, 10, dtype=torch.float16))
    with pytest.raises(ValueError):
        cpu_verify(target_probs=torch.zeros(2, 10, 4).transpose(1, 2))
    with pytest.raises(ValueError):
        cpu_verify(uniforms=torch.zeros(2, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        cpu_verify(tokens=torch.zeros(2, 4, dtype=torch.int64))
    with pytest.raises(ValueError):
        cpu_verify(path=torch.zeros(2, 5, dtype=torch.int32))
    refused("FDEC_ERR_INVALID_ARG", cpu_verify, target_probs=torch.zeros(2, 4, 0), draft_probs=None)
    big = torch.zeros(1, dtype=torch.float32).expand(1, 1, (1 << 24) + 1)
    one = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):  # (no unit stride)
        cpu_verify(target_probs=big, draft_probs=None, tokens=one, uniforms=torch.zeros(1, 1), path=one, out_tokens=one,
                   path_lens=torch.zeros(1, dtype=torch.int32))
    many = torch.zeros(2, 65, dtype=torch.int32)
    refused("FDEC_ERR_UNSUPPORTED", cpu_verify, target_probs=torch.zeros(2, 65, 10), draft_probs=None, tokens=many,
            uniforms=torch.zeros(2, 65), path=many, out_tokens=many)


def cpu_keep(**kw):
    a = dict(caches=[torch.zeros(6, 2, 16, 64, dtype=torch.float16)], page_table=torch.zeros(2, 3, dtype=torch.int32),
             prefix_lens=torch.zeros(2, dtype=torch.int32), path=torch.zeros(2, 4, dtype=torch.int32),
             path_lens=torch.zeros(2, dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32), page_size=16)
    a.update(kw)
    fd.fdec_keep_path(**a)


def test_keep_path_refusals():
    with pytest.raises(ValueError, match="CUDA device"):
        cpu_keep()
    with pytest.raises(ValueError):
        cpu_keep(caches=[torch.zeros(2, 16, 64)])
    with pytest.raises(ValueError):
        cpu_keep(caches=[torch.zeros(6, 2, 8, 64)])
    with pytest.raises(ValueError):
        cpu_keep(caches=[3])
    with pytest.raises(TypeError):
        cpu_keep(caches=3)
    refused("FDEC_ERR_INVALID_ARG", cpu_keep, caches=[])
    refused("FDEC_ERR_INVALID_ARG", cpu_keep, caches=[torch.zeros(6, 2, 16, 64)] * 129)
    refused("FDEC_ERR_LAYOUT", cpu_keep, caches=[torch.zeros(6, 2, 16, 3, dtype=torch.float16)])
    refused("FDEC_ERR_LAYOUT", cpu_keep, caches=[torch.zeros(6, 2, 16, 64, dtype=torch.float16)[..., 1:61]])
    same = torch.zeros(2, dtype=torch.int32)
    refused("FDEC_ERR_INVALID_ARG", cpu_keep, prefix_lens=same, seq_lens=same)
    path = torch.zeros(8, dtype=torch.int32)
    refused("FDEC_ERR_INVALID_ARG", cpu_keep, path=path.view(2, 4), seq_lens=path[3:5])
    pool = torch.zeros(6, 2, 16, 64)
    refused("FDEC_ERR_INVALID_ARG", cpu_keep, caches=[pool, pool])
    refused("FDEC_ERR_LAYOUT", cpu_keep, caches=[pool[:1].expand(6, 2, 16, 64)])
    refused("FDEC_ERR_LAYOUT", cpu_keep, caches=[pool[None].expand(3, 6, 2, 16, 64)])
    with pytest.raises(ValueError, match="CUDA device"):  # K and V in one tensor are two caches
        both = torch.zeros(6, 2, 2, 16, 64)
        cpu_keep(caches=[both[:, 0], both[:, 1]])
    refused("FDEC_ERR_UNSUPPORTED", cpu_keep, path=torch.zeros(2, 65, dtype=torch.int32))


def cpu_reserve(**kw):
    a = dict(page_table=torch.zeros(2, 3, dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32),
             new_lens=torch.zeros(2, dtype=torch.int32), granted=torch.zeros(2, dtype=torch.int32), num_pages=64, page_size=16,
             workspace=aligned_workspace(2, 64))
    a.update(kw)
    fd.fdec_reserve_pages(**a)


def aligned_workspace(batch, pages):
    n = fd.fdec_reserve_pages_workspace(batch, pages)
    raw = torch.zeros(n + 256, dtype=torch.uint8)
    at = -raw.data_ptr() % 256
    return raw[at:at + n]


def test_reserve_pages_refusals():
    with pytest.raises(ValueError, match="CUDA device"):
        cpu_reserve()
    with pytest.raises(ValueError):
        cpu_reserve(new_lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        cpu_reserve(seq_lens=torch.zeros(2, dtype=torch.int64))
    refused("FDEC_ERR_INVALID_ARG", cpu_reserve, num_pages=0)
    refused("FDEC_ERR_INVALID_ARG", cpu_reserve, num_pages=(1 << 26) + 1)
    refused("FDEC_ERR_UNSUPPORTED", cpu_reserve, page_size=24)
    refused("FDEC_ERR_WORKSPACE", cpu_reserve, workspace=aligned_workspace(2, 64)[:-1])
    refused("FDEC_ERR_WORKSPACE", cpu_reserve, workspace=torch.zeros(4096, dtype=torch.uint8)[1:])
    refused("FDEC_ERR_INVALID_ARG", cpu_reserve, caches=[torch.zeros(63, 2, 16, 64)])  # fewer pages than the pool's
    same = torch.zeros(2, dtype=torch.int32)
    for name in ("seq_lens", "new_lens", "sources"):
        refused("FDEC_ERR_INVALID_ARG", cpu_reserve, **{name: same, "granted": same})
    with pytest.raises(fd.FdecError):
        fd.fdec_reserve_pages_workspace(0, 64)


def test_workspace_is_at_most_what_is_said():
    for batch, pages in ((1, 1), (64, 65536), (300, 8193), (65536, 1 << 26)):
        assert fd.fdec_reserve_pages_workspace(batch, pages) <= 4 * pages + 256 * batch + 256


def test_a_round_makes_no_forks():
    """A fork's prefix would be the 0 that it has, and its nodes' rows would go into the pages it shares."""
    assert "sources" not in inspect.signature(fd.TreeDecode.reserve).parameters


def test_tree_decode_refuses_what_it_cannot_hold():
    with pytest.raises(ValueError):
        fd.TreeDecode([100], 65, 16, 8, 2, 128, 64)
    with pytest.raises(ValueError):
        fd.TreeDecode([100], 0, 16, 8, 2, 128, 64)
    with pytest.raises(ValueError):
        fd.TreeDecode([100], 8, 16, 8, 2, 128, 64, kv_dtype="q8_0")


def test_fresh_data_is_read_with_ordinary_loads():
    """These kernels are resident beside the ones that write their inputs: no read-only loads."""
    root = os.path.join(os.path.dirname(fd.__file__), "csrc")
    for name in ("tree_attention.cu", "verify_drafts.cu", "keep_path.cu", "reserve_pages.cu", "cache_rows.cuh"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(root, name)).read())
        assert "__ldg" not in text and ".nc." not in text, name
        for body in re.split(r"__global__", text)[1:]:
            wait = body.index("griddepcontrol.wait")
            assert "return" not in body[:wait], name  # no way out before the kernel before has completed
