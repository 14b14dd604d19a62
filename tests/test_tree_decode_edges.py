"""Drafting operators where they can go wrong: inputs that no test of the operators' ranges reaches."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest
import torch

import paged_split_kv_gather_gb300 as fd
from test_tree_decode import i32, run_verify

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
