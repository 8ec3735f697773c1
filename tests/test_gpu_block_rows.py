"""The block norm where a workgroup takes several rows of more columns than the
other cases have, and with outputs and checkpoints at any address."""
import math

import pytest
import torch

import block_reference as ref
import test_gpu_block_norm as norm
from test_gpu_block_norm import DEV, EPS, check_gradients, check_kept, cpu, forward, inputs, within

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu

# rows, columns, dtype, gate, which of post | pre | scale, alpha, pad (None: dense):
# three to four rows a workgroup on 256 compute units, the last round partial
CASES = [
    (900, 12288, "bf16", True, 7, 1.0, None), (900, 12288, "f32", True, 7, 1.0, None), (900, 12289, "bf16", True, 7, 1.0, None),
    (900, 12289, "f32", True, 7, 1.0, None), (900, 5001, "bf16", True, 7, 1.0, None), (900, 12290, "bf16", False, 7, 0.5, None),
    (900, 9001, "bf16", False, 7, 0.5, 1), (900, 9001, "f32", False, 7, 0.5, 1),
    # without a gate, in the widths that the other cases have with one only
    (40, 129, "bf16", False, 7, 1.0, None), (40, 510, "bf16", False, 7, 1.0, None), (1100, 1002, "bf16", False, 7, 1.0, None),
    (1100, 1003, "bf16", False, 7, 0.5, 1), (700, 5001, "bf16", False, 7, 1.0, None), (300, 6003, "f32", False, 7, 1.0, None),
    (600, 12288, "f32", False, 7, 1.0, None),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case):
    norm.test_forward_and_backward(case)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_checkpoints(case):
    norm.test_checkpoints(case)


def placed(like, off):
    """A dense tensor like `like` that begins `off` elements behind a 16-byte
    boundary, and the memory around it, filled with 0xff."""
    n, e = like.numel(), like.element_size()
    room = torch.full(((n + off + 32) * e,), 0xff, dtype=torch.uint8, device=DEV)
    return room[off * e:(off + n) * e].view(like.dtype).view(like.shape), room


def untouched(room, t, off):
    e = t.element_size()
    return bool((room[:off * e] == 0xff).all() and (room[(off + t.numel()) * e:] == 0xff).all())


# columns that are whole 16-byte pieces, whole words and neither; a wave a row
# and a workgroup a row, one to sixteen columns a thread
ADDRESSES = [(96, "bf16"), (96, "f32"), (2560, "bf16"), (2560, "f32"), (2562, "bf16"), (1003, "bf16"), (1003, "f32"), (4104, "bf16"),
             (4100, "f32"), (8200, "bf16"), (8200, "f32"), (12288, "bf16")]
OFFSETS = [(1, 0), (0, 1), (2, 3), (3, 2)]


@pytest.mark.parametrize("off,codes", OFFSETS)
@pytest.mark.parametrize("columns,dtype", ADDRESSES)
def test_outputs_and_checkpoints_at_any_address(columns, dtype, off, codes):
    """y, the stream and the gradients `off` elements behind a 16-byte boundary, a
    checkpoint's codes `codes` bytes behind one and its scales `off` of theirs."""
    p, io = inputs((21, columns, dtype, True, 7, 1.0, None))
    plain = forward(p, 1.0, True)
    c = {k: cpu(v) for k, v in p.items()}
    y, y_room = placed(plain[0], off)
    stream, stream_room = placed(plain[1], off)
    kept, rooms = {}, {}
    for k, v in plain[2].items():
        kept[k], rooms[k] = placed(v, codes if k.endswith("_q") else off)
    got = forward(p, 1.0, kept, y=y, residual_out=stream)
    assert got[0] is y and got[1] is stream
    within("stream", stream, ref.block_stream(c["x"], c["residual"], c["z"], c["post"], c["scale"], 1.0, EPS), io)
    within("y", y, ref.block_out(cpu(stream), c["pre"], EPS), io)
    for name in ("x", "z", "residual"):
        check_kept(kept, name, stream if name == "residual" else p[name])
    assert untouched(y_room, y, off) and untouched(stream_room, stream, off)
    assert all(untouched(rooms[k], kept[k], codes if k.endswith("_q") else off) for k in kept)
    held = {n: cpu(kept[n + "_q"].float()) * ref.per_column(cpu(kept[n + "_scales"]), columns) for n in ("x", "z", "residual")}
    for from_kept in (False, True):
        v = held if from_kept else dict(x=c["x"], z=c["z"], residual=cpu(stream))
        want = ref.block_backward(v["x"], v["residual"], v["z"], c["post"], c["pre"], c["scale"], c["dy"], c["dstream"], 1.0, EPS)
        # (from a checkpoint: code times scale rounds once more, twice the bound)
        want = {k: (t[0], t[1] * (2 if from_kept else 1)) for k, t in want.items()}
        like = dict(dx=p["dy"], dresidual=p["dy"], dz=p["dy"], dpost_weight=p["post"], dpre_weight=p["pre"], dscale=p["scale"])
        out, out_rooms = {}, {}
        for k, t in like.items():
            out[k], out_rooms[k] = placed(t, off)
        given = (None, None) if from_kept else (p["x"], stream)
        ssd.ssd_block_norm_bwd(*given, p["post"], p["pre"], p["dy"], z=None if from_kept else p["z"], scale=p["scale"],
                               dresidual_out=p["dstream"], eps=EPS, checkpoint=kept if from_kept else None, out=out)
        check_gradients(out, want, io)
        assert all(untouched(out_rooms[k], out[k], off) for k in out)
