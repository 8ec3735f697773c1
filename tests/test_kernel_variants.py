"""Every kernel that is built for the operators between the layers is reached by
a GPU test, and none is built that no call reaches: the launch rules, written
down again here, over the cases of the GPU tests on 256 compute units, against
the kernels' names in the library (CPU only)."""
import re

import torch

import ssd_chunked_scan_amd as ssd

CUS = 256
ceil = lambda a, b: -(-a // b)


def built(kernel):
    """Template arguments of a kernel's variants in the library."""
    ssd.load_library()
    with open(ssd.library_path(), "rb") as f:
        data = f.read()
    out = set()
    for args in re.findall(rb"_ZN3ssd\d+" + kernel.encode() + rb"I((?:DF16b|[fh]|L[ib]\d+E)+)EEv", data):
        parts = re.findall(r"DF16b|[fh]|L[ib]\d+E", args.decode())
        out.add(tuple({"DF16b": "bf16", "f": "f32", "h": "u8"}.get(p) or int(p[2:-1]) for p in parts))
    assert out, kernel
    return out


# --------------------------------------------------------- 4-bit products


def product(m, n, k, io, quantise, aligned=True):
    """The kernel of a product with outputs in `io`, from activations in `io` or in 4 bits."""
    kb = ceil(k, 128)
    if m <= 16 or (m <= 32 and ceil(n, 64) <= CUS // 2):
        source = io if quantise and m <= 16 else "u8"
        mt = 1 if m <= 16 else 2
        for nt in (4, 2):
            if 8 * ceil(n, 16 * nt) >= 5 * CUS:
                return "mx4_few_kernel", (source, io, mt, nt, 8)
        return "mx4_few_kernel", (source, io, mt, 1, 16 if source != "u8" and kb > 8 else 8)
    wide = int(aligned and n * (2 if io == "bf16" else 4) % 16 == 0)
    if kb <= 2 or ceil(m, 64) * ceil(n, 64) <= 2 * CUS:
        return "mx4_ring_kernel", (io, wide)
    if 8 * ceil(m, 256) * ceil(n, 256) >= 5 * CUS and kb > (32 if io == "f32" else 0 if wide else 16):
        return "mx4_tile_kernel", (io, 256, 256, 128, 64, 1, wide)
    return "mx4_tile_kernel", (io, 128, 128, 64, 64, 2, wide)


def product_cases():
    """(m, n, k, io, quantise) of the tests of whole results."""
    import test_gpu_mx4 as mx4
    import test_gpu_mx4_tiles as tiles
    name = {torch.bfloat16: "bf16", torch.float32: "f32"}
    for m, n, k in mx4.PRODUCTS:
        yield m, n, k, "f32", False
        if m * n * k < 3_000_000_000:
            for io in mx4.TYPES:
                for quantise in (False, True):
                    yield m, n, k, io, quantise
    for m, n, k, io in tiles.TILES + tiles.FEW:
        yield m, n, k, name[io], False
    for m, n, k, io in tiles.FEW_QUANTISED:
        yield m, n, k, name[io], True


def test_products():
    reached = {}
    for case in product_cases():
        kernel, variant = product(*case)
        reached.setdefault(kernel, set()).add(variant)
    assert sorted(reached) == ["mx4_few_kernel", "mx4_ring_kernel", "mx4_tile_kernel"]
    for kernel, variants in reached.items():
        assert built(kernel) == variants, (kernel, built(kernel) ^ variants)


# -------------------------------------------------------------- block norm


def block_variant(columns, io, gate, kept, wide, backward, code_words):
    single = (8, 8, 8, 16) if not backward else (4, 4, 8, 16)   # packs: a wave's lane, then a workgroup's thread
    V, packs = (1, single) if not wide else (8, (1, 1, 1, 2)) if io == "bf16" else (4, (2, 2, 2, 4))
    npack = ceil(columns, V)
    wave = npack <= 64 * packs[0]
    K = packs[0] if wave else next(k for k in packs[1:] if npack <= 1024 * k or k == packs[-1])
    how = int(kept) if backward else 0 if not kept else 1 if V == 1 or code_words else 2
    return io, V, int(wave), K, int(gate), how


def block(rows, columns, io, gate, pad=None, off=0, codes=0):
    """The kernels of a forward and a backward call without and with checkpoints:
    inputs `pad` elements inside wider rows, outputs `off` elements and codes
    `codes` bytes off a 16-byte boundary."""
    e = 2 if io == "bf16" else 4
    code_words = columns % 4 == 0 and codes % 4 == 0

    def fit(nbytes, *addresses):
        rows_in = (pad or 0) * e, (columns + 2 * (pad or 0)) * e
        return all(a % nbytes == 0 for a in (columns * e, *rows_in, *addresses))

    for kept in (False, True):
        wide = io == "f32" or fit(4, off * e)
        yield "block_fwd_kernel", block_variant(columns, io, gate, kept, wide, False, code_words)
        wide = (not kept or code_words) and fit(16 if columns <= 4096 else 4, off * e)
        yield "block_bwd_kernel", block_variant(columns, io, gate, kept, wide, True, code_words)


def block_cases():
    import test_gpu_block_norm as norm
    import test_gpu_block_rows as more
    for rows, columns, io, gate, _, _, pad in norm.CASES + more.CASES:
        yield rows, columns, io, gate, pad
    for columns, io in more.ADDRESSES:
        for off, codes in more.OFFSETS:
            yield 21, columns, io, True, None, off, codes


def test_block_norm():
    reached = {}
    for case in block_cases():
        for kernel, variant in block(*case):
            reached.setdefault(kernel, set()).add(variant)
    for kernel, variants in reached.items():
        made = built(kernel)
        assert made == variants, (kernel, "not reached", sorted(made - variants), "not built", sorted(variants - made))
