"""The sizes that the GPU tests of the products in 4 bits and of the operators on
logits use reach every kernel that the plans can choose (CPU only): the plans' own
headers in a small program, asked about the tests' sizes and a wide sample of
others."""
import math
import os
import random
import shutil
import subprocess

import pytest

import test_gpu_logits
import test_gpu_q4
import test_gpu_q4_kernels

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "gemm_rbq_encode_amd", "csrc")
CXX = shutil.which("g++") or shutil.which("clang++")


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if CXX is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("plans") / "q4_plans")
    subprocess.run([CXX, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "plans", "q4_plans.cpp"), "-o", exe], check=True)

    def plans(what, calls):
        text = "".join(f"{what} {' '.join(map(str, c))}\n" for c in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(calls)
        return got
    return plans


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def product(plan):
    tiled, slices, four, staged, row_tiles, _ = plan
    return ("tiled", slices > 1) if tiled else ("few", four, staged, row_tiles)


def test_every_product_kernel_is_reached(ask):
    rng = random.Random(1)
    sample = [(log_uniform(rng, 1, 200_000), 32 * log_uniform(rng, 1, 1024), log_uniform(rng, 1, 5000)) for _ in range(4000)]
    plans = ask("gemm", sample)
    for (out, inf, M), (tiled, slices, four, staged, row_tiles, lds) in zip(sample, plans):
        T = -(-inf // 128)
        assert 1 <= slices <= 16 and (slices == 1 or 2 * slices <= T + 1)
        assert tiled or (1 <= row_tiles <= 3 and lds + 32768 <= 65536 and (not four or M <= 4))
        assert M > 16 or not tiled
    used = [(out, inf, M) for out, inf in test_gpu_q4.SHAPES for M in test_gpu_q4.TOKENS]
    used += [(out, inf, M) for M, out, inf in test_gpu_q4.LARGER + test_gpu_q4_kernels.KERNELS]
    reached = {product(p) for p in ask("gemm", used)}
    assert {product(p) for p in plans} <= reached, {product(p) for p in plans} - reached
    assert sorted(reached) == sorted([("tiled", False), ("tiled", True), ("few", True, True, 1), ("few", True, False, 1),
                                      ("few", False, False, 1)] + [("few", False, True, n) for n in (1, 2, 3)])


def test_the_tiled_sizes_are_tiled(ask):
    calls = [(out, inf, M) for M, out, inf in test_gpu_q4_kernels.TILED]
    assert all(p[0] for p in ask("gemm", calls))
    # in so long that a tile's offsets would pass 32 bits: never tiled
    assert not any(p[0] for p in ask("gemm", [(100, 2 ** 23 + 32, 100), (2 ** 25, 2 ** 24, 2 ** 16)]))


def test_every_cut_of_logits_is_reached(ask):
    rng = random.Random(2)
    sample = [(log_uniform(rng, 1, 20_000), log_uniform(rng, 1, 2 ** 24), k) for k in (0, 20, 128) for _ in range(1500)]
    plans = ask("logits", sample)
    for (M, V, k), (slices, threads, need) in zip(sample, plans):
        vectors = -(-V // 8)
        assert 1 <= slices <= 256 and threads in (128, 256, 512)
        assert slices == 1 or -(-vectors // slices) >= 256          # every thread of the smallest workgroup has work
        assert need == (0 if slices == 1 else M * slices * (16 + 8 * k))
        assert k <= 64 or threads > 128
    kinds = {(s > 1, t, k) for (_, _, k), (s, t, _) in zip(sample, plans)}
    used = [(M, V, k) for M, V in test_gpu_logits.SHAPES + test_gpu_logits.CUT_SHAPES for k in (0, 20, 128)]
    reached = {(s > 1, t, k) for (_, _, k), (s, t, _) in zip(used, ask("logits", used))}
    assert kinds <= reached, kinds - reached
