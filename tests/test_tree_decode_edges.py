"""Drafting operators where they can go wrong: inputs that no test of the operators' ranges reaches."""
import ctypes
import math
import os
import random
import subprocess
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import paged_split_kv_gather_gb300 as fd
from test_tree_decode import (U, Tree, aligned_workspace, check_verify, cpu_keep, cpu_reserve, cpu_verify, drafts_of, i32,
                              path_of, refused, reserve_case, reserve_reference, run_reserve, run_verify)

HERE = os.path.dirname(os.path.abspath(__file__))
gpu = pytest.mark.gpu


# ------------------------------------------------------------------------------- verification: one decision for all

def chunk_of(vocab, runs=64):
    """Tokens of a warp's run: the launcher's."""
    return (-(-vocab // runs) + 127) // 128 * 128


@pytest.fixture(scope="module")
def host_sums(tmp_path_factory):
    out = tmp_path_factory.mktemp("pairs") / "libpair_sums.so"
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++20", "-O1", "-ffp-contract=off", "-shared", "-fPIC", "-pthread",
                    os.path.join(HERE, "csrc", "pair_sums_host.cpp"), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    at = lambda x: None if x is None else x.ctypes.data_as(ctypes.c_void_p)  # noqa: E731

    class Host:
        @staticmethod
        def row(vocab, seed):
            p = np.empty(vocab, np.float32)
            lib.seeded_row(vocab, seed, at(p))
            return p

        @staticmethod
        def run_sums(p, q=None, s=(0.0, 0.0)):
            sums = np.zeros((64, 32, 2), np.float32)
            lib.run_sums(at(p), at(q), len(p), chunk_of(len(p)), 64, ctypes.c_float(s[0]), ctypes.c_float(s[1]), at(sums))
            return sums

        @staticmethod
        def decisions(sums, gone, child, u):
            stands = np.zeros(8, np.int32)
            lib.decisions(at(sums), ctypes.c_float(gone), ctypes.c_float(child), ctypes.c_float(u), at(stands))
            return stands

    return Host


@pytest.mark.parametrize("vocab", [8193, 32768, 50021])
def test_every_lane_of_a_warp_has_one_sum(host_sums, vocab):
    """The CTAs of a cluster get a run's sum from as many lanes, and each walks for itself: the sums are the same bits."""
    p, q = host_sums.row(vocab, 2), host_sums.row(vocab, 3)
    for sums in (host_sums.run_sums(p), host_sums.run_sums(p, q, (1.0, 0.0)), host_sums.run_sums(p, q, (1.375, 3e-9))):
        bits = sums.view(np.uint32)
        assert (bits == bits[:, :1]).all()
    exact = p.astype(np.longdouble).sum()
    got = host_sums.run_sums(p)[:, 0].astype(np.longdouble).sum()
    assert abs(got - exact) <= 2.0 ** -44 * exact


def test_every_cta_decides_alike(host_sums):
    """A child so near to the border that two sums 2^-50 apart would differ about it."""
    p = host_sums.row(50021, 1)
    p[7] = 0.31
    p[40000], p[20000] = (np.float32(float.fromhex(x)) for x in ("0x1.b22d0ep-5", "0x1.772a6ap-7"))
    sums = host_sums.run_sums(p)
    assert len(set(host_sums.decisions(sums, 0.31, p[40000], float.fromhex("0x1.985344p-5")).tolist())) == 1


@gpu
@pytest.mark.parametrize("vocab", [8193, 20000, 50021])
def test_decisions_too_near_to_tell_are_one_path_and_its_token(vocab):
    """Second children whose two sides differ by less than 2^-46: either answer is as good, but path, length and tokens
    are those of one of them, the same every time."""
    g = np.random.default_rng(vocab)
    cases, first, second = 24, 7, vocab - 21
    target = np.zeros((cases, 3, vocab), np.float32)
    u = np.zeros((cases, 3), np.float32)
    for i in range(cases):
        p = np.exp(3 * g.standard_normal(vocab)).astype(np.float32)
        p /= p.sum()
        p[first], p[second] = 0.31, 0.0
        rest = p.astype(np.float64)
        rest[first] = 0.0
        rest = float(np.sum(rest))
        # u (rest + x) = x for x a value of fp32, but for 2^-46 of it
        while True:
            some = g.uniform(0.01, 0.5, 1 << 20).astype(np.float32)
            x = some.astype(np.float64) * rest / (1.0 - some.astype(np.float64))
            off = np.abs(x.astype(np.float32).astype(np.float64) / x - 1.0)
            best = int(off.argmin())
            if off[best] < 2.0 ** -46:
                break
        p[second] = np.float32(x[best])
        target[i] = p
        target[i, 2] = np.roll(p, 3)
        u[i] = g.random(), 0.9999, some[best]
    target, u = torch.from_numpy(target).cuda(), torch.from_numpy(u)
    tokens, parents = [[0, first, second]] * cases, [[-1, 0, 0]] * cases
    got = run_verify(target, None, tokens, parents, u)
    assert got[3] == 0
    sides = []
    for value in (0.0, 0.9999):
        near = u.clone()
        near[:, 2] = value
        sides.append(run_verify(target, None, tokens, parents, near))
    assert sides[0][0].tolist() == [[0, 2, -1]] * cases and sides[1][0].tolist() == [[0, -1, -1]] * cases
    for i in range(cases):
        side = sides[0 if got[1][i] == 2 else 1]
        assert all(torch.equal(a[i], b[i]) for a, b in zip(got[:3], side[:3])), i
    for _ in range(20):
        again = run_verify(target, None, tokens, parents, u)
        assert all(torch.equal(a, b) for a, b in zip(got[:3], again[:3]))


# ------------------------------------------------------------------------------------- tree attention: large and small

def check_every_value(c, out, lse):
    """As Tree.check, but each value within the tolerance of what it is the sum of itself: an error of a probability,
    relative to it, moves a column by that part of the column's own terms.  (Probabilities below 2^-125 may be 0.)"""
    group = c.hq // c.hk
    half, tiny = (0.0, 0.0) if out.dtype == torch.float32 else (torch.finfo(out.dtype).eps / 2, torch.finfo(out.dtype).tiny)
    for b in range(c.batch):
        for i in range(c.counts[b]):
            at = [c.prefix[b] + j for j in path_of(c.parents[b], i)]
            where = [(int(c.table[b, p // c.page]), p % c.page) for p in at]
            for kvh in range(c.hk):
                k, v = (torch.stack([x[pg, kvh, sl].double() for pg, sl in where]).cpu() for x in (c.k, c.v))
                rows = slice(kvh * group, (kvh + 1) * group)
                q = c.q[b, i, rows].double().cpu()
                z = q @ k.T * c.scale
                e = (2 * c.d + 4) * U * (q.abs() @ k.abs().T * abs(c.scale)).amax(-1)
                if c.lse_prefix is None:
                    before, o = torch.full((group,), -math.inf).double(), torch.zeros(group, c.d).double()
                else:
                    before, o = c.lse_prefix[b, i, rows].double().cpu(), c.o_prefix[b, i, rows].double().cpu()
                    o = torch.where(before[:, None] == -math.inf, 0.0, o)
                total = torch.logaddexp(torch.logsumexp(z, -1), before)
                p, w = torch.exp(z - total[:, None]), torch.exp(before - total)[:, None]
                want, size = p @ v + w * o, p @ v.abs() + w * o.abs()
                zmax = torch.maximum(z.abs().amax(-1), torch.where(before == -math.inf, 0.0, before).abs())
                tol = (2 * e + 8 * U * zmax + 200 * U)[:, None] * size + 2.0 ** -125 * v.abs().sum(0)
                limit = tol + half * torch.maximum(want.abs() + tol, torch.tensor(tiny).double())
                off = (out[b, i, rows].double().cpu() - want).abs()
                assert (off <= limit).all(), (b, i, kvh, (off / limit).max().item())
                near = e + 3 * U * zmax + 140 * U + U * total.abs()
                assert ((lse[b, i, rows].double().cpu() - total).abs() <= near).all()


def outlier(c, b, node, power, logit=None, columns=slice(None)):
    """Node's value row times 2^power; its key such that every query's logit is about `logit` (queries' first dim is 8)."""
    p = c.prefix[b] + node
    at = int(c.table[b, p // c.page]), slice(None), p % c.page
    row = c.v[at].double()
    row[:, columns] *= 2.0 ** power
    c.v[at] = row.to(c.v.dtype)
    if logit is not None:
        key = torch.zeros_like(c.k[at])
        key[:, 0] = logit / (c.scale * 8.0)
        c.k[at] = key


@gpu
@pytest.mark.parametrize("d,hq,hk,nodes", [(128, 8, 2, 13), (64, 4, 2, 40), (192, 4, 1, 20), (256, 4, 2, 64),
                                           (512, 2, 1, 33)])
@pytest.mark.parametrize("power", [9, 12, 30, 40, 100])
def test_large_rows_cost_the_others_nothing(d, hq, hk, nodes, power):
    """A value row far above the others: nodes that do not see it have their own rows' accuracy, those that do see it,
    with a weight near 0 among them, that of what it adds."""
    for state, out_type, logit in ((True, torch.float32, None), (False, torch.float32, -30.0),
                                   (True, torch.bfloat16, -70.0)):
        c = Tree(d, hq, hk, nodes, 16, 2, "bf16", seed=power + nodes, counts=[nodes, nodes - 1], state=state)
        c.q[..., 0] = 8.0
        outlier(c, 0, 2, power, logit)
        outlier(c, 1, nodes - 2, power, logit, columns=slice(5, 6))  # a leaf's, one column
        if nodes > 30:
            outlier(c, 1, 1, -power)
            outlier(c, 1, 0, 20, -25.0)
        if power >= 12:
            check_every_value(c, *c.run(out=torch.full(c.q.shape, 3.0, dtype=out_type, device="cuda")))
        else:  # (of one size: within the rows' tolerance)
            c.check(*c.run(out=torch.full(c.q.shape, 3.0, dtype=out_type, device="cuda")))


@gpu
def test_a_large_row_that_a_node_does_not_see_with_an_empty_prefix():
    """One sibling's value is 1e30, the other's 1: the result is 1, whatever the sibling's."""
    for nodes in (3, 20, 64):
        c = Tree(128, 4, 1, nodes, 16, 1, "bf16", seed=1, kind="star", counts=[nodes], prefix=[0])
        c.v.fill_(1.0)
        plain, lse = c.run()
        outlier(c, 0, 1, 100)
        out, lse2 = c.run()
        seen = torch.zeros(nodes, dtype=torch.bool)
        seen[1] = True
        assert (out[0, ~seen] - 1).abs().max() <= 200 * U and (out[0, 1] > 1e26).all()
        assert (out[0, ~seen] - plain[0, ~seen]).abs().max() <= 200 * U and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("d,dtype,kv", [(128, "bf16", ""), (128, "f16", ""), (256, "bf16", "fp8"), (512, "bf16", "")])
def test_infinite_values_of_hardly_any_weight_stay_infinite(d, dtype, kv):
    c = Tree(d, 6, 2, 22, 16, 2, dtype, kv, seed=9, counts=[22, 22])
    if kv:  # (E4M3 has no infinity)
        value = math.nan
    else:
        value = math.inf
    c.q[..., 0] = 8.0
    outlier(c, 1, 3, 0, -30.0)
    p = c.prefix[1] + 3
    c.v[int(c.table[1, p // 16]), 0, p % 16] = torch.tensor(value).to(c.v.dtype)
    out, lse = c.run()
    for i in range(22):
        rows = out[1, i, :3]
        if 3 in path_of(c.parents[1], i):
            assert (torch.isnan(rows) if kv else rows == math.inf).all(), i
        else:
            assert torch.isfinite(rows).all()
    assert torch.isfinite(out[1, :, 3:]).all() and torch.isfinite(lse[1]).all()


# ---------------------------------------------------------------------------------------- lengths that are none

@gpu
def test_keep_path_leaves_a_bad_length_as_it_is():
    pool = torch.randn(8, 2, 16, 64).half().cuda()
    before, out = pool.clone(), torch.full((3,), 9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    path = i32([[1, 3, -1, -1]] * 3)
    fd.fdec_keep_path([pool], i32(np.arange(6).reshape(3, 2)), i32([-7, 4, -(2 ** 31)]), path, i32([2, 2, 2]), out, 16,
                      device_errors=err)
    assert out.tolist() == [-7, 6, -(2 ** 31)] and int(err.item()) == fd.DEVERR_SEQ_LEN
    assert torch.equal(pool[[0, 1, 4, 5, 6, 7]], before[[0, 1, 4, 5, 6, 7]])
    assert torch.equal(pool[2, :, 4], before[2, :, 5]) and torch.equal(pool[2, :, 5], before[2, :, 7])


@gpu
def test_a_round_of_sequences_with_bad_lengths():
    """Negative, past the page table, and so near its end that the nodes have no room: no nodes, nothing written, the
    length stays; the other sequence's round is as ever."""
    batch, nodes, page, hq, hk, d, vocab, pages = 5, 6, 16, 4, 2, 64, 32, 40
    torch.manual_seed(5)
    k = torch.randn(pages, hk, page, d, device="cuda").half()
    v = torch.randn(pages, hk, page, d, device="cuda").half()
    tree = fd.TreeDecode([60] * batch, nodes, page, hq, hk, d, pages, "f16")
    lengths = [-1, 20, 65, 61, 2 ** 31 - 2]
    lens = i32(lengths)
    table = i32(np.arange(batch * 4).reshape(batch, 4))
    qkv = torch.randn(batch * nodes, hq + 2 * hk, d, device="cuda").half()
    fresh, cos_sin = qkv.clone(), torch.cat([torch.ones(100, d // 2), torch.zeros(100, d // 2)], 1).cuda()
    target = torch.softmax(torch.randn(batch, nodes, vocab, device="cuda"), -1)
    tokens, u = torch.zeros(batch, nodes, dtype=torch.int32, device="cuda"), torch.rand(batch, nodes, device="cuda")
    parents, depths = i32([[-1] + [0] * (nodes - 1)] * batch), i32([[0] + [1] * (nodes - 1)] * batch)
    out = torch.full((batch, nodes, hq, d), 7.0, device="cuda")
    for rotated in (cos_sin, None):
        before = k.clone(), v.clone()
        qkv.copy_(fresh)
        assert tree.reserve(table, lens, (k, v)).tolist() == [lengths[0], 26, *lengths[2:]]
        tree.attend(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], None, None, rotated, k, v, table, lens, parents,
                    depths, out)
        path, path_lens, words = tree.verify(target, None, tokens, parents, u)
        kept = tree.keep((k, v), table, lens).tolist()
        assert tree.device_errors() & fd.DEVERR_SEQ_LEN
        for b in (0, 2, 3, 4):
            assert (path[b] == -1).all() and path_lens[b] == 0 and (words[b] == -1).all() and kept[b] == lengths[b]
            assert (out[b] == 7).all() and torch.equal(qkv[b * nodes:(b + 1) * nodes, :hq],
                                                       fresh[b * nodes:(b + 1) * nodes, :hq])
        assert kept[1] == 20 + int(path_lens[1]) and path_lens[1] >= 1 and (out[1] != 7).all()
        mine = int(table[1, 1])
        for pool, old in zip((k, v), before):
            changed = (pool != old).any(-1).any(1)
            changed[mine] = False
            assert not changed.any()


# ------------------------------------------------------------------------------------------------ the holder's streams

@gpu
def test_a_new_holder_can_be_used_on_any_stream(monkeypatch):
    """What the constructor fills is there when it returns, however busy the stream that filled it."""
    plan = fd.PagedDecode.__init__

    def busy(self, *a, **kw):
        plan(self, *a, **kw)
        torch.cuda._sleep(200_000_000)

    monkeypatch.setattr(fd.PagedDecode, "__init__", busy)
    own, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(own):
        rubbish = [torch.full((n,), 99, dtype=torch.int32, device="cuda") for n in (1, 3, 6, 18)] * 4
        del rubbish  # (what the holder's tensors are made of)
        tree = fd.TreeDecode([60] * 3, 6, 16, 4, 2, 64, 32, "f16")
        assert own.query()
    with torch.cuda.stream(side):
        assert tree.counts.tolist() == [6] * 3 and tree.errors.tolist() == [0] and tree.nowhere.tolist() == [-2 ** 31]
        assert tree.offsets.tolist() == [list(range(6))] * 3 and tree.nodes.tolist() == list(range(6))
        assert tree.batch_indices.tolist() == [0] * 6 + [1] * 6 + [2] * 6


def test_a_holder_works_on_its_own_device(monkeypatch):
    """Whichever device is current: every call that goes by the current one is made with the holder's."""
    current, seen = ["cuda:0"], []

    class Device:
        def __init__(self, device):
            self.device = str(device)

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *_):
            current.pop()

    def call(name, result=None):
        def f(*_, **__):
            seen.append((name, current[-1]))
            return result
        return f

    monkeypatch.setattr(torch.cuda, "device", Device)
    for name in ("fdec_norm_rope_append", "fdec_tree_attention", "fdec_verify_drafts", "fdec_reserve_pages"):
        monkeypatch.setattr(fd, name, call(name))
    tree = fd.TreeDecode.__new__(fd.TreeDecode)
    tree.batch, tree.num_nodes, tree.page_size, tree.num_pages, tree.max_pages = 1, 2, 16, 8, 2
    tree.errors = SimpleNamespace(device=torch.device("cuda:1"), item=lambda: 0, zero_=lambda: None)
    tree.prefix = SimpleNamespace(run=call("run"), device_errors=call("device_errors", 0))
    tree.nodes, tree.nowhere = torch.arange(2, dtype=torch.int32), torch.full((1,), -1, dtype=torch.int32)
    tree.offsets, tree.counts = tree.nodes.repeat(1, 1), torch.full((1,), 2, dtype=torch.int32)
    tree.batch_indices = tree.o = tree.state_lse = tree.workspace = tree.path = tree.path_lens = tree.tokens = None
    tree.granted = lens = torch.zeros(1, dtype=torch.int32)
    rows, table = torch.zeros(2, 1, 64), torch.zeros(1, 2, dtype=torch.int32)
    tree.reserve(None, lens)
    tree.attend(rows, rows, rows, None, None, None, None, None, table, lens, None, None, None)
    tree.verify(None, None, None, None, None)
    assert tree.device_errors() == 0
    assert [name for name, _ in seen] == ["fdec_reserve_pages", "fdec_norm_rope_append", "run", "fdec_tree_attention",
                                          "fdec_verify_drafts", "device_errors"]
    assert {device for _, device in seen} == {"cuda:1"} and current == ["cuda:0"]


# ------------------------------------------------------------------------------- page tables that are views of columns

@gpu
def test_columns_that_are_not_the_views_are_neither_read_nor_written():
    """Tables within wider ones: a length past the view's columns is one past the page table, also in the last row."""
    page, width = 16, 3
    whole = i32(np.full((4, 8), 77))
    table = whole[1:3, 2:2 + width]
    table.copy_(i32([[0, 1, 2], [3, 4, 5]]))
    before = whole.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def flags():
        got = int(err.item())
        err.zero_()
        return got

    granted = torch.empty(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(fd.fdec_reserve_pages_workspace(2, 64), dtype=torch.uint8, device="cuda")

    def reserve(lens, new, sources=None):
        fd.fdec_reserve_pages(table, i32(lens), i32(new), granted, 64, page, ws, device_errors=err,
                              sources=None if sources is None else i32(sources))
        return granted.tolist()

    assert reserve([30, 20], [49, 49]) == [30, 20] and flags() == fd.DEVERR_SEQ_LEN and torch.equal(whole, before)
    assert reserve([49, 20], [49, 20]) == [49, 20] and flags() == fd.DEVERR_SEQ_LEN  # (marks its own columns only)
    assert reserve([0, 20], [49, 30], [1, -1])[0] == 0 and flags() == fd.DEVERR_SEQ_LEN
    assert torch.equal(whole, before)
    assert reserve([17, 20], [48, 48]) == [48, 48] and flags() == 0
    assert table.tolist() == [[0, 1, 2], [3, 4, 5]] and (whole[:, :2] == 77).all() and (whole[:, 5:] == 77).all()

    for path, upto, flag in (([0, 2, 5, 9], 2, fd.DEVERR_TREE),  # (of four nodes: it ends before the 5)
                             ([0, 2, 5, 9] + [-1] * 6, 3, fd.DEVERR_SEQ_LEN)):
        pool = torch.randn(6, 1, page, 64).half().cuda()
        kept, out = pool.clone(), torch.empty(2, dtype=torch.int32, device="cuda")
        fd.fdec_keep_path([pool], table, i32([44, 44]), i32([path] * 2), i32([3, 3]), out, page, device_errors=err)
        assert flags() == flag and out.tolist() == [44 + upto] * 2
        for b in range(2):
            last = kept[3 * b + 2]
            last[:, 13] = last[:, 14]  # (the third row lies past the view)
        assert torch.equal(pool, kept)

    c = Tree(64, 4, 2, 8, page, 2, "f16", seed=3, counts=[8, 8], prefix=[20, 40])
    wide = i32(np.full((3, 9), c.k.shape[0] - 1))
    view = wide[1:, 1:1 + 3]
    view.copy_(i32(c.table[:, :3]))
    out, lse = torch.zeros(c.q.shape, device="cuda"), torch.zeros(c.q.shape[:3], device="cuda")
    c.prefix = [20, 44]
    c.table = np.concatenate([c.table[:, :3], np.full((2, 1), -1, dtype=np.int32)], 1)
    fd.fdec_tree_attention(c.q, c.k, c.v, view, i32(c.prefix), i32(c.parents), c.o_prefix, c.lse_prefix, out, lse, page,
                           device_errors=err)
    assert flags() == fd.DEVERR_SEQ_LEN
    c.check(out, lse, unseen={(1, j) for j in range(4, 8)})


# ------------------------------------------------------------------------------------------- arrays that are one another's

def test_verify_drafts_refuses_results_on_one_another_or_on_inputs():
    with pytest.raises(ValueError, match="CUDA device"):  # each sequence's inputs are read first
        x, y, z = (torch.zeros(2, 4, dtype=torch.int32) for _ in range(3))
        n = torch.zeros(2, dtype=torch.int32)
        cpu_verify(tokens=x, out_tokens=x, parents=y, path=y, node_counts=n, path_lens=n)
    grid, line = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    many = torch.zeros(64, dtype=torch.int32)
    some = {"path": many[8:16].view(2, 4), "out_tokens": many[24:32].view(2, 4), "path_lens": many[40:42]}
    spans = {"path": (8, 16), "out_tokens": (24, 32), "path_lens": (40, 42)}
    refused("FDEC_ERR_INVALID_ARG", cpu_verify, path=grid, out_tokens=grid)
    for name, (a, b) in spans.items():
        for at in (a - 3, a + 1, b - 1):
            near = many[at:at + 8].view(2, 4)
            for other in ("tokens", "parents", "uniforms"):
                view = near.view(torch.float32) if other == "uniforms" else near
                refused("FDEC_ERR_INVALID_ARG", cpu_verify, **{**some, other: view})
            if name != "path_lens":
                refused("FDEC_ERR_INVALID_ARG", cpu_verify, **{**some, "path_lens": many[a + 2:a + 4]})
                refused("FDEC_ERR_INVALID_ARG", cpu_verify, **{**some, "node_counts": many[a:a + 2]})
        refused("FDEC_ERR_INVALID_ARG", cpu_verify, **{**some, "node_counts": many[b - 1:b + 1]})
        probs = many[a - 2:].view(torch.float32)[:8].view(2, 4, 1)
        refused("FDEC_ERR_INVALID_ARG", cpu_verify, **{**some, "target_probs": probs, "draft_probs": None})
        refused("FDEC_ERR_INVALID_ARG", cpu_verify, **{**some, "target_probs": torch.zeros(2, 4, 1), "draft_probs": probs})
    # the row behind the drafts' last is nobody's
    with pytest.raises(ValueError, match="CUDA device"):
        probs = torch.zeros(2 * 4 * 10 + 4)
        cpu_verify(draft_probs=probs[:80].view(2, 4, 10)[:, :3], path_lens=probs.view(torch.int32)[70:72])


def test_kept_lengths_and_granted_ones_have_arrays_of_their_own():
    table = torch.zeros(2, 3, dtype=torch.int32)
    refused("FDEC_ERR_INVALID_ARG", cpu_keep, page_table=table, seq_lens=table.view(-1)[4:6])
    refused("FDEC_ERR_INVALID_ARG", cpu_reserve, page_table=table, granted=table.view(-1)[:2])
    for name in ("seq_lens", "new_lens", "sources"):
        refused("FDEC_ERR_INVALID_ARG", cpu_reserve, page_table=table, **{name: table.view(-1)[3:5]})
    ws = aligned_workspace(2, 64)
    words = ws.view(torch.int32)
    for name in ("seq_lens", "new_lens", "sources", "granted"):
        refused("FDEC_ERR_INVALID_ARG", cpu_reserve, workspace=ws, **{name: words[3:5]})
    refused("FDEC_ERR_INVALID_ARG", cpu_reserve, workspace=ws, page_table=words[-6:].view(2, 3))
    # a row of a wider table, and what lies beside the view
    wide = torch.zeros(2, 8, dtype=torch.int32)
    refused("FDEC_ERR_INVALID_ARG", cpu_reserve, page_table=wide[:, 2:5], granted=wide[1, 4:6])
    with pytest.raises(ValueError, match="CUDA device"):
        cpu_reserve(page_table=wide[:, 2:5], granted=wide[1, 5:7])


@gpu
@pytest.mark.parametrize("vocab", [500, 9000])
def test_verify_drafts_in_place_of_what_it_reads(vocab):
    g, rng = torch.Generator().manual_seed(vocab), random.Random(vocab)
    target, draft, tokens, parents = drafts_of(g, rng, 9, 7, vocab, "f32", "tree", True)
    u, counts = torch.rand((9, 7), generator=g), [7, 0, 3, 7, 1, 6, 7, 7, 2]
    want = run_verify(target, draft, tokens, parents, u, counts)
    tok, par, n = i32(tokens), i32(parents), i32(counts)
    fd.fdec_verify_drafts(target, draft, tok, par, u.cuda(), par, n, tok, node_counts=n)
    assert torch.equal(par.cpu(), want[0]) and torch.equal(n.cpu(), want[1]) and torch.equal(tok.cpu(), want[2])


@gpu
@pytest.mark.parametrize("left,stands", [(1e-2, False), (1e-5, False), (1e-8, True)])
def test_heavy_tokens_fall_and_the_rest_is_drawn_from(left, stands):
    """Four children hold (1 - left) / 4 each.  The last is tried with W = (1 - left) / 4 + left, all numbers 1 - 2^-24: it
    falls where left > 2^-24 / 4 = 1.5e-8, and the next token is one of the rest; else it stands."""
    g = torch.Generator().manual_seed(8)
    batch, nodes, vocab = 16, 5, 3000
    p = torch.softmax(torch.randn((batch, nodes, vocab), generator=g) * 2, -1) * left
    p[:, :, 100:104] = (1 - left) / 4
    u = torch.ones((batch, nodes)) * (1 - 2.0 ** -24)
    u[:, 0] = torch.rand(batch, generator=g)
    tokens, parents = [[0, 100, 101, 102, 103]] * batch, [[-1, 0, 0, 0, 0]] * batch
    target = p.float().cuda()
    assert set(check_verify(target, None, tokens, parents, u)) == ({2} if stands else {1})
    path, _, words, _ = run_verify(target, None, tokens, parents, u)
    if stands:
        assert path[:, :2].tolist() == [[0, 4]] * batch and (words[:, 0] == 103).all()
    else:
        assert ((words[:, 0] < 100) | (words[:, 0] > 103)).all() and (words[:, 0] >= 0).all()


@gpu
@pytest.mark.parametrize("d,hq,hk,nodes,batch", [(192, 16, 4, 64, 80), (256, 12, 4, 35, 90), (512, 4, 2, 40, 80),
                                                 (512, 8, 2, 20, 160)])
def test_tree_attention_in_equal_shares_of_large_heads(d, hq, hk, nodes, batch):
    """More sequences' heads than CTAs are resident, where shared memory bounds those: shares span sequences."""
    c = Tree(d, hq, hk, nodes, 16, batch, "bf16", seed=17)
    out, lse = c.run()
    few = random.Random(2).sample(range(batch), 3) + [0, batch - 1]
    c.check(out, lse, counts=[n if b in few else 0 for b, n in enumerate(c.counts)])
    for b in range(0, batch, 8):  # the others against calls of few sequences, summed in another order
        part = slice(b, min(batch, b + 8))
        o, l2 = torch.full_like(out[part], 3.0), torch.full_like(lse[part], 5.0)
        fd.fdec_tree_attention(c.q[part], c.k, c.v, i32(c.table[part]), i32(c.prefix[part]), i32(c.parents[part]),
                               c.o_prefix[part], c.lse_prefix[part], o, l2, 16, node_counts=i32(c.counts[part]))
        # (sum |q_d k_d| is at most |q| |k|; twice the module's tolerance, for the two calls)
        most = c.scale * float((c.q[part].double().norm(dim=-1).max() * c.k.double().norm(dim=-1).max()).item())
        most, largest = max(most, 12.0), max(float(c.v.abs().max()), float(c.o_prefix.nan_to_num(0).abs().max()))
        e = (2 * d + 4) * U * most
        assert (o - out[part]).abs().nan_to_num(0).max() <= 2 * (2 * e + 8 * U * most + 200 * U) * largest
        assert torch.equal(torch.isnan(o), torch.isnan(out[part]))
        assert torch.equal((l2 == -math.inf), (lse[part] == -math.inf))
        assert (l2 - lse[part]).nan_to_num(0).abs().max() <= 2 * (e + 4 * U * (most + 8) + 140 * U)


# ------------------------------------------------------------------------------------------------------ large batches

@gpu
@pytest.mark.parametrize("batch,width,page,spare", [(4099, 6, 16, 3000), (65536, 3, 16, 40000)])
def test_reserve_pages_of_large_batches(batch, width, page, spare):
    rng = random.Random(batch)
    table, lens, num_pages = reserve_case(rng, batch, width, page, spare, True)
    new = [min(width * page, max(0, n + rng.choice([0, 1, 7, page, 3 * page, -5]))) for n in lens]
    got, granted, err = run_reserve(table, lens, new, None, num_pages, page)
    want, want_granted, _ = reserve_reference(table, lens, new, None, num_pages, page)
    short = any(g < n for g, n, l in zip(want_granted, new, lens) if n > l)
    assert err == (fd.DEVERR_NO_PAGES if short else 0)
    assert granted == want_granted and np.array_equal(got, want)


def test_reserve_pages_refuses_larger_batches():
    lens = [torch.zeros(65537, dtype=torch.int32) for _ in range(3)]
    refused("FDEC_ERR_UNSUPPORTED", cpu_reserve, page_table=torch.zeros(65537, 1, dtype=torch.int32), seq_lens=lens[0],
            new_lens=lens[1], granted=lens[2], workspace=aligned_workspace(65537, 64))


# ------------------------------------------------------------------------------------------- the holder and its operators

@gpu
@pytest.mark.parametrize("kv", ["fp8", ""])
@pytest.mark.parametrize("interleaved,chain,out_type", [(True, False, torch.bfloat16), (False, True, torch.float32)])
def test_a_layer_of_the_holder_is_its_operators(kv, interleaved, chain, out_type):
    """Weights, both rotations, E4M3 caches with scales, 16-bit results, lse, node counts: bit for bit the calls by hand."""
    batch, nodes, page, hq, hk, d, pages = 3, 7, 16, 8, 2, 128, 40
    g = torch.Generator().manual_seed(21)
    rand = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    kv_type = torch.float8_e4m3fn if kv else torch.bfloat16
    k, v = ((rand(pages, hk, page, d) * (8 if kv else 1)).to(kv_type) for _ in range(2))
    scales = dict(k_scale=0.04, v_scale=0.3) if kv else dict(k_scale=1.0, v_scale=1.0)
    qkv, weights = rand(batch * nodes, hq + 2 * hk, d).bfloat16(), [1 + 0.1 * rand(d).bfloat16() for _ in range(2)]
    cos_sin = rand(200, d)
    prefix, table = i32([50, 0, 33]), i32(np.arange(batch * 5).reshape(batch, 5))
    parents = None if chain else i32([[-1, 0, 0, 1, 1, 2, 5]] * batch)
    depths = None if chain else i32([[0, 1, 1, 2, 2, 2, 3]] * batch)
    counts = i32([7, 4, 0])
    tree = fd.TreeDecode([60] * batch, nodes, page, hq, hk, d, pages, "bf16", kv_dtype=kv)
    x, kk, vv = qkv.clone(), k.clone(), v.clone()
    out = torch.full((batch, nodes, hq, d), 5.0, dtype=out_type, device="cuda")
    lse = torch.full((batch, nodes, hq), 5.0, device="cuda")
    assert tree.reserve(table, prefix, (kk, vv)).tolist() == [57, 7, 40]
    tree.attend(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], *weights, cos_sin, kk, vv, table, prefix, parents, depths, out,
                lse, counts, interleaved=interleaved, **scales)
    assert tree.device_errors() == 0
    y, k2, v2 = qkv.clone(), k.clone(), v.clone()
    at = prefix[:, None] + torch.arange(nodes, dtype=torch.int32, device="cuda")
    turns = at if chain else prefix[:, None] + depths
    seqs = torch.arange(batch, dtype=torch.int32, device="cuda").repeat_interleave(nodes)
    fd.fdec_norm_rope_append(y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:], *weights, cos_sin, seqs, at.reshape(-1),
                             y[:, :hq], k2, v2, table, page, 1e-6, interleaved, turns.reshape(-1), **scales)
    rows = y[:, :hq].view(batch, nodes, hq, d)
    o, l = torch.empty((batch, nodes, hq, d), device="cuda"), torch.empty((batch, nodes, hq), device="cuda")
    plain = fd.PagedDecode([60] * batch, nodes, page, hq, hk, d, "bf16", kv_dtype=kv)
    plain.run(rows, k2, v2, table, prefix, o, l, **scales)
    want, want_lse = torch.full_like(out, 5.0), torch.full_like(lse, 5.0)
    fd.fdec_tree_attention(rows, k2, v2, table, prefix, parents, o, l, want, want_lse, page, node_counts=counts, **scales)
    for a, b in ((out, want), (lse, want_lse), (kk, k2), (vv, v2), (x, y)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert (out[2] == 5).all() and (out[1, 4:] == 5).all() and not (kk.view(torch.uint8) == k.view(torch.uint8)).all()


def test_a_holder_refuses_tables_of_fewer_columns_than_its_longest_prefix_needs():
    """A view of a wide table passes for one by its stride."""
    tree = fd.TreeDecode.__new__(fd.TreeDecode)
    tree.max_pages = 4
    wide = torch.zeros(2, 8, dtype=torch.int32)
    rows = torch.zeros(2, 1, 64)
    with pytest.raises(ValueError, match="columns"):
        tree.attend(rows, rows, rows, None, None, None, None, None, wide[:, 5:], torch.zeros(2, dtype=torch.int32), None, None,
                    None)
