"""The layer operators' binding on the host: the library without torch, and the
numbers that its argument structures cannot hold.  CPU only: no kernel is started."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_TORCH = """
import ctypes, sys
if {blocked}:
    sys.modules["torch"] = None          # any import of it raises ImportError
import ssd_chunked_scan_amd as ssd
from ssd_chunked_scan_amd import *       # names only: nothing is called
lib = ssd.load_library()
for name in ssd.EXPORTS:
    assert getattr(lib, name)
shape = ssd.GlrShape(1, 4096, 64, 0, 0, 0, 0, 1)
assert lib.ssd_glr_bwd_workspace_bytes(ctypes.byref(shape), 1) == 20 * 64 * 64
assert lib.ssd_glr_step(None, 1, *[None] * 7, None) == 1 and b"shape" in lib.ssd_last_error()
assert ssd.ssd_conv_step is ssd_conv_step and ssd.NormShape and ssd.ConvShape
if {blocked}:
    try:
        ssd.ssd_norm_fwd(None)
    except ImportError:
        pass
    else:
        raise AssertionError("a call without torch")
else:
    assert "torch" not in sys.modules
"""


@pytest.mark.parametrize("blocked", [True, False])
def test_the_library_loads_without_torch(blocked):
    """The C interface needs no torch: neither the package, its names nor the
    loaded library import it."""
    env = dict(os.environ, PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH.format(blocked=blocked)], capture_output=True, text=True,
                       env=env, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("block", [2 ** 32 + 128, 2 ** 32, 128 - 2 ** 32, 2 ** 64 + 128, 2 ** 31])
def test_a_block_is_not_cut_to_32_bits(block):
    """The structure's field has 32 bits and ctypes drops the others: 2^32 + 128
    would be scaled in blocks of 128 into scales allocated for one a row.  (The
    refusal comes before the one of tensors off the GPU.)"""
    import torch
    import ssd_chunked_scan_amd as ssd
    with pytest.raises(ValueError, match="block"):
        ssd.ssd_norm_quant_fwd(torch.zeros(2, 256), None, block=block)


@pytest.mark.parametrize("ngroups", [2 ** 64 + 2, 2 ** 63, 1 - 2 ** 64])
def test_ngroups_is_not_cut_to_64_bits(ngroups):
    import torch
    import ssd_chunked_scan_amd as ssd
    x = torch.zeros(2, 256)
    for call in (lambda: ssd.ssd_norm_fwd(x, None, ngroups=ngroups), lambda: ssd.ssd_norm_bwd(x, None, x, ngroups=ngroups),
                 lambda: ssd.ssd_norm_quant_fwd(x, None, ngroups=ngroups)):
        with pytest.raises(ValueError, match="ngroups"):
            call()


def test_the_sizes_at_the_documented_limits():
    """The largest sizes that include/ssd.h names get past the checks of the shape
    (to the NULL x), the next ones do not."""
    import ctypes
    import ssd_chunked_scan_amd as ssd
    lib = ssd.load_library()
    NULL, UNSUPPORTED = 1, 3

    def status(name, shape, pointers, workspace=()):
        return getattr(lib, name)(ctypes.byref(shape), 1, *[None] * pointers, *workspace, None)

    glr = lambda b, L, D: ssd.GlrShape(b, L, D, 0, 0, 0, 0, 1)
    for b, L, D, want in (((1 << 23) - 1, 1, 32, UNSUPPORTED), ((1 << 22) - 1, 1, 64, NULL), (1 << 22, 1, 64, UNSUPPORTED),
                          (1, 64 * ((1 << 23) - 1), 32, NULL), (1, 64 << 23, 32, UNSUPPORTED)):
        assert status("ssd_glr_fwd", glr(b, L, D), 9, (None, 0)) == want, (b, L, D)
        if L == 1:
            assert status("ssd_glr_step", glr(b, L, D), 7) == want
    conv = lambda b, L, D: ssd.ConvShape(b, L, D, 4, 0, 0, 1)
    for b, L, D, want in (((1 << 24) - 1, 64, 64, NULL), (1 << 24, 1, 64, UNSUPPORTED), (1, 64, 1 << 20, NULL)):
        assert status("ssd_conv_fwd", conv(b, L, D), 7) == want, (b, L, D)
    norm = lambda groups: ssd.NormShape(3, 4 * groups, groups, 0, 0, 0, 0, 0, 1e-5, 0)
    assert status("ssd_norm_fwd", norm(65535), 6) == NULL and status("ssd_norm_fwd", norm(65536), 6) == UNSUPPORTED
