"""A checkpoint has z exactly when there is a gate: one whose z is left over from
a call with a gate, or of which half is there, would give other gradients."""
import pytest
import torch

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_z_goes_with_a_gate():
    x = torch.randn(6, 300, device=DEV)
    _, _, kept = ssd.ssd_block_norm_fwd(x, x, z=x, checkpoint=True)
    without = {k: v for k, v in kept.items() if not k.startswith("z")}
    # to write into, without a gate: z's would keep what an earlier call left there
    for left in (("z_q",), ("z_scales",), ("z_q", "z_scales")):
        with pytest.raises(ValueError, match="without a gate"):
            ssd.ssd_block_norm_fwd(x, x, checkpoint=dict(without, **{k: kept[k] for k in left}))
    # with a gate, and backward: both or neither
    for missing in ("z_q", "z_scales"):
        half = {k: v for k, v in kept.items() if k != missing}
        with pytest.raises(ValueError, match="missing"):
            ssd.ssd_block_norm_fwd(x, x, z=x, checkpoint=half)
        with pytest.raises(ValueError, match="missing"):
            ssd.ssd_block_norm_bwd(None, None, None, None, x, checkpoint=half)
    _, _, plain = ssd.ssd_block_norm_fwd(x, x, checkpoint=dict(without, z_q=None))
    assert sorted(plain) == sorted(without)
    assert ssd.ssd_block_norm_bwd(None, None, None, None, x, checkpoint=plain)["dz"] is None
    assert ssd.ssd_block_norm_bwd(None, None, None, None, x, checkpoint=kept)["dz"] is not None
