"""The host side of the router's and the products' entry points under host-only
address and undefined-behaviour sanitizers, with 300,000 random and extreme
descriptors and no device visible."""
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from combine_ep_get_amd import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all"]


@pytest.mark.skipif(shutil.which(libbuild.HIPCC) is None, reason="hipcc not available")
def test_host_code_under_address_and_ub_sanitizers(tmp_path):
    base = [libbuild.HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-fPIC", *SAN,
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", libbuild.INCLUDE]

    def run(cmd, **kw):
        r = subprocess.run(cmd, capture_output=True, text=True, **kw)
        assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
        return r.stdout

    def compiled(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        run([*base, "-c", src, "-o", obj])
        return obj

    with ThreadPoolExecutor(4) as pool:
        objs = list(pool.map(compiled, [libbuild.SRC, *libbuild.MORE_SRC]))
    driver = str(tmp_path / "driver.o")
    run(["/opt/rocm/llvm/bin/clang", "-O1", "-std=c11", "-fsanitize=address,undefined", "-I",
         libbuild.INCLUDE, "-c", os.path.join(HERE, "c", "products_host_driver.c"), "-o", driver])
    exe = str(tmp_path / "driver")
    run([libbuild.HIPCC, *SAN, *objs, driver, "-o", exe])
    # the HIP runtime itself is not built with the sanitizer: leaks it keeps until exit
    # are not this library's
    out = run([exe], timeout=600, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0",
                                           HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1"))
    assert "clean" in out
