"""The sizes that the GPU tests of the 8-bit products and of the backward from
checkpoints use reach every kernel that the plans can choose (CPU only): the
plans' own headers in a small program, asked about the tests' sizes and about
a wide sample of others."""
import math
import os
import random
import shutil
import subprocess

import pytest

import test_gpu_f8
import test_gpu_f8_edges
import test_gpu_f8_kernels
import test_gpu_qat_ckpt
import test_gpu_qat_ckpt_kernels

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "gemm_rbq_encode_amd", "csrc")
CXX = shutil.which("g++") or shutil.which("clang++")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if CXX is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("plans") / "plans")
    subprocess.run([CXX, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "plans", "plans.cpp"), "-o", exe], check=True)

    def ask(what, calls):
        text = "".join(f"{what} {' '.join(map(str, c))}\n" for c in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(calls)
        return got
    return ask


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def gemm_kernel(call, plan):
    out, _, M, f32 = call
    kind, whole, slices, tiles = plan
    if kind < 0:
        return f32, "few", out >= 12288, M > 16
    return f32, kind, "whole" if slices == 1 or whole == tiles else "all cut" if whole == 0 else "part cut"


def test_every_product_kernel_is_tested(plans):
    rng = random.Random(1)
    sample = [(log_uniform(rng, 1, 70000), 32 * log_uniform(rng, 1, 500), log_uniform(rng, 1, 5000), rng.randint(0, 1))
              for _ in range(40000)]
    tested = [(o, i, m, f) for o, m, i in test_gpu_f8.GEMM + test_gpu_f8.TILES for f in (0, 1)]
    tested += [(o, i, m, 0) for o, m, i in test_gpu_f8_edges.HEIGHTS]
    tested += test_gpu_f8_kernels.TILES + test_gpu_f8_kernels.FEW
    can = {gemm_kernel(c, p) for c, p in zip(sample, plans("gemm", sample))}
    have = {gemm_kernel(c, p) for c, p in zip(tested, plans("gemm", tested))}
    assert can - have == set()
    assert {k[:2] for k in can} == {(f, k) for f in (0, 1) for k in range(6) if f == 0 or k >= 3} | {(0, "few"), (1, "few")}


def test_non_finite_entries_meet_every_product_kernel(plans):
    calls = test_gpu_f8_kernels.NON_FINITE
    have = {gemm_kernel(c, p)[:2] for c, p in zip(calls, plans("gemm", calls))}
    assert {(0, k) for k in range(6)} | {(0, "few"), (1, 3), (1, 4), (1, 5), (1, "few")} == have


def backward_kernels(call, plan):
    M, _, _, K, ask = call
    dx_slices, large, dw_slices, both = plan
    tokens = next(t for t in (16, 32, 64, 128, 256) if M <= t or t == 256)
    cut = dx_slices > 1, dw_slices > 1
    if tokens <= 64:
        return [("few", tokens, K)]
    if both:
        return [("both", tokens, K, *cut)]
    return [("dx", tokens, K, cut[0])] * (ask & 1) + [("dw", large, cut[1])] * (ask >> 1)


def test_every_backward_kernel_is_tested(plans):
    rng = random.Random(2)
    sample = [(log_uniform(rng, 1, 5000), log_uniform(rng, 1, 15000), 32 * log_uniform(rng, 1, 400), rng.randint(1, 4),
               rng.randint(1, 3)) for _ in range(40000)]
    tested = [(M, o, i, K, 3) for o, i, K, _, M in test_gpu_qat_ckpt.BACKWARD + test_gpu_qat_ckpt.LARGE]
    one_by_one = [(600, 576, 2, 1100), (100, 160, 1, 70), (1030, 640, 4, 300), (257, 1056, 3, 130), (2050, 2048, 2, 128)]
    tested += [(M, o, i, K, ask) for o, i, K, M in one_by_one for ask in (1, 2, 3)]
    tested += [(M, o, i, K, ask) for M, o, i, K, _, ask in test_gpu_qat_ckpt_kernels.KERNELS]
    can = {k for c, p in zip(sample, plans("backward", sample)) for k in backward_kernels(c, p)}
    have = {k for c, p in zip(tested, plans("backward", tested)) for k in backward_kernels(c, p)}
    assert can - have == set()
