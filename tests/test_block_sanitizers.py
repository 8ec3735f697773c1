"""The host side of the operators between the layers (ssd_block_api.cpp) under
AddressSanitizer and UndefinedBehaviorSanitizer, host-only, linked with stub
launchers that touch every byte the kernels would
(tests/host_sanitize/block_stubs.cpp) and driven with buffers of exactly the
documented sizes (block_driver.c).  CPU only."""
import os

import test_host_sanitizers as hs

pytestmark = hs.pytestmark


def test_block_host_code_under_asan_and_ubsan(tmp_path):
    api, stubs, drv = (str(tmp_path / n) for n in ("block_api.o", "block_stubs.o", "block_drv.o"))
    hs._hipcc_host(os.path.join(hs.CSRC, "ssd_block_api.cpp"), api)
    hs._hipcc_host(os.path.join(hs.HERE, "block_stubs.cpp"), stubs)
    hs._run([os.path.join(hs.LLVM, "clang"), "-std=c11", "-D_GNU_SOURCE", "-O1", "-g", *hs.SAN, "-I", hs.INCLUDE, "-c",
             os.path.join(hs.HERE, "block_driver.c"), "-o", drv])
    exe = str(tmp_path / "block_driver")
    hs._run([os.path.join(hs.LLVM, "clang++"), *hs.SAN, drv, api, stubs, "-o", exe])
    r = hs._run([exe], env=hs._env(), timeout=600)
    assert "all checks passed" in r.stdout, r.stdout + r.stderr
