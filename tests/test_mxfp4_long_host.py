"""The GPU cases of long MXFP4 reductions reach what they are there for."""

from block_quantized_expert_amd import binding as B

# tile -> slots of scale words in its kernel; a word serves 512 inputs
SLOTS = {(256, 256): 2, (128, 256): 2, (64, 256): 2, (32, 256): 2, (128, 128): 3, (64, 64): 3}


def test_gpu_cases_use_every_tiled_forms_slots_again():
    """Every tile shape, plain and with SwiGLU, dense and grouped (each of those
    gathered and in expert order), more than twice around its slots of scale
    words within a tile, with an odd and an even number of words; and so across
    the tiles of a workgroup where a shape is chosen for several."""
    import test_gpu_mxfp4_long as G
    from test_gpu_mxfp4_tiles import counts_of

    reached, several = set(), set()

    def look(kind, e, rows, cols, counts, slots):
        words = -(-cols // 512)
        for swiglu in (False, True):
            r, c, workgroups = B.moe_mxfp4_form(e, rows, cols, slots, kind == "grouped", swiglu)
            form = (r, c * 2 if swiglu else c)
            if workgroups and words > 2 * SLOTS[form]:
                reached.add((kind, swiglu, form, words % 2))
                items = sum(-(-int(n) // r) for n in counts) * -(-rows // c)
                if items >= 2 * workgroups:
                    several.add((kind, swiglu, form, words % 2))

    for n, rows, cols in G.DENSE:
        look("dense", 1, rows, cols, [n], n)
    for e, slots, rows, cols in G.GROUPED:
        look("grouped", e, rows, cols, counts_of(e, slots), slots)
    want = {(kind, swiglu, form, odd) for kind in ("dense", "grouped") for swiglu in (False, True)
            for form in SLOTS for odd in (0, 1)}
    assert reached == want, (want - reached, reached - want)
    want = {(kind, swiglu, form, odd) for kind, swiglu, form, odd in want
            if kind == "grouped" or form in ((256, 256), (128, 256), (128, 128))}
    assert several >= want, want - several
