"""Host code of the 4-bit linears and the operators on logits under AddressSanitizer
and UndefinedBehaviorSanitizer (CPU only): q4_logits_host.c with the sources whose
host code its calls run, the sanitizers on their host half, and the library's other
objects.  Any report aborts the driver, so a non-zero exit fails the test.
"""
import concurrent.futures
import os

import pytest

from gemm_rbq_encode_amd import build as libbuild
from test_sanitizers_cpu import HERE, ROOT, SAN_HIP, _run

CHECKED = ["api.hip", "gemm_q4.hip"]


@pytest.mark.skipif(not os.path.exists(libbuild.HIPCC), reason="hipcc not found")
def test_q4_and_logits_host_code_under_sanitizers(tmp_path):
    flags = [f for f in libbuild.FLAGS if f != "-O3"] + ["-O1"]

    def compiled(src):
        built = os.path.join(libbuild.BUILD, os.path.splitext(src)[0] + ".o")
        if src not in CHECKED and os.path.exists(built):
            return built
        obj = str(tmp_path / (src + ".o"))
        _run([libbuild.HIPCC, *flags, *(SAN_HIP if src in CHECKED else []), "-c", os.path.join(libbuild.CSRC, src), "-o", obj])
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        objs = list(ex.map(compiled, libbuild.SOURCES))
    exe = str(tmp_path / "q4_logits_host")
    _run([libbuild.HIPCC, "--offload-arch=gfx950", *SAN_HIP, "-I", os.path.join(ROOT, "include"),
          "-x", "c", os.path.join(HERE, "sanitize", "q4_logits_host.c"), "-x", "none", *objs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1")
    r = _run([exe], env=env)
    assert "4-bit and logits host checks passed" in r.stdout
