"""Host code of the 8-bit floating point and checkpoint calls under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): f8_host.c with
every library source, the sanitizers on the host half.  Any report aborts the
driver, so a non-zero exit fails the test.
"""
import concurrent.futures
import os

import pytest

from gemm_rbq_encode_amd import build as libbuild
from test_sanitizers_cpu import HERE, ROOT, SAN_HIP, _run


@pytest.mark.skipif(not os.path.exists(libbuild.HIPCC), reason="hipcc not found")
def test_8_bit_host_code_under_sanitizers(tmp_path):
    flags = [f for f in libbuild.FLAGS if f != "-O3"] + ["-O1"]

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        _run([libbuild.HIPCC, *flags, *SAN_HIP, "-c", os.path.join(libbuild.CSRC, src), "-o", obj])
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        objs = list(ex.map(compile_one, libbuild.SOURCES))
    exe = str(tmp_path / "f8_host")
    _run([libbuild.HIPCC, "--offload-arch=gfx950", *SAN_HIP, "-I", os.path.join(ROOT, "include"),
          "-x", "c", os.path.join(HERE, "sanitize", "f8_host.c"), "-x", "none", *objs, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1")
    r = _run([exe], env=env)
    assert "8-bit host checks passed" in r.stdout
