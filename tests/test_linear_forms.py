"""The choice of spec_linear's kernel (spec_linear_form), without a GPU: every form -- the few-token
stream, each tile width with each split of K, each width of the CTA pairs' tiles -- has sizes below
that reach it, in both input types and on devices that hold somewhat more or fewer clusters.  The GPU
tests run these sizes; a change of the rule that leaves a form without one fails here."""
import os
import shutil

import pytest
import torch

BF, E4 = torch.bfloat16, torch.float8_e4m3fn

# (kind, tokens of a tile, CTAs that share its K): rows, N, K in bf16 and in e4m3.  Rows end inside a
# tile, N inside a tile and off a group of four (N // 4 * 4 reaches the same form); pairs have seven
# slices of K or more (a ring of six) and more tiles than pairs.
FORMS = {
    ("few", 1, 1): ((1, 4099, 4096), (1, 301, 1040)),
    ("few", 2, 1): ((2, 101, 48), (2, 1003, 4112)),
    ("few", 3, 1): ((3, 999, 4096), (3, 18, 64)),
    ("few", 4, 1): ((4, 33, 12288), (4, 2001, 4096)),
    ("tiles", 16, 1): ((6, 65, 64), (6, 61, 64)),
    ("tiles", 16, 2): ((6, 5310, 1824), (6, 5145, 3664)),
    ("tiles", 16, 4): ((6, 69, 1280), (6, 61, 2736)),
    ("tiles", 16, 8): ((6, 61, 2224), (6, 65, 4336)),
    ("tiles", 32, 1): ((2095, 62, 96), (18, 9878, 64)),
    ("tiles", 32, 2): ((18, 5453, 2736), (18, 5346, 4976)),
    ("tiles", 32, 4): ((620, 66, 1440), (619, 69, 2912)),
    ("tiles", 32, 8): ((154, 133, 2208), (303, 61, 4688)),
    ("tiles", 64, 1): ((39, 9989, 64), (35, 10054, 64)),
    ("tiles", 64, 2): ((34, 5097, 3472), (1242, 138, 6288)),
    ("tiles", 64, 4): ((1287, 66, 2160), (1278, 62, 4208)),
    ("tiles", 64, 8): ((644, 61, 4096), (664, 61, 7936)),
    ("tiles", 128, 1): ((66, 7381, 96), (69, 7961, 160)),
    ("tiles", 128, 2): ((66, 5323, 6080), (71, 5185, 10192)),
    ("tiles", 128, 4): ((1279, 135, 4096), (1273, 135, 9600)),
    ("tiles", 128, 8): ((1258, 69, 7264), (1176, 62, 15024)),
    ("pairs", 96, 1): ((270, 12439, 464), (284, 12245, 784)),
    ("pairs", 128, 1): ((309, 12458, 400), (305, 12506, 864)),
    ("pairs", 160, 1): ((283, 13326, 416), (533, 7885, 784)),
    ("pairs", 192, 1): ((344, 13766, 400), (516, 10066, 784)),
    ("pairs", 224, 1): ((403, 14937, 400), (436, 13867, 784)),
    ("pairs", 256, 1): ((462, 13475, 464), (502, 13873, 832)),
}
CASES = [(form, size, dtype) for form, sizes in FORMS.items() for size, dtype in zip(sizes, (BF, E4))]
CASE_IDS = [f"{f[0]}-{f[1]}-{f[2]}-{'e4m3' if d is E4 else 'bf16'}" for f, _, d in CASES]
# three and more tiles for each pair: both accumulators used again
MANY_TILES = [((1100, 13003, 512), BF), ((1101, 13000, 1040), E4)]

SMS = 152
CLUSTERS = [(76, 36, 15), (76, 36, 16), (76, 38, 18), (74, 34, 14)]  # of 2, 4 and 8 CTAs; the first was measured


@pytest.fixture(scope="module")
def sv():
    if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from speculative_decoding_verification_31_gb300 import build
    build.build()
    import speculative_decoding_verification_31_gb300 as m
    m.load_library()
    return m


@pytest.mark.parametrize("form,size,dtype", CASES, ids=CASE_IDS)
def test_sizes_reach_their_form(sv, form, size, dtype):
    rows, N, K = size
    for held in CLUSTERS:
        assert sv.spec_linear_form(rows, N, K, dtype, SMS, held) == form
        if N >= 64 and form[0] != "few":
            assert sv.spec_linear_form(rows, N // 4 * 4, K, dtype, SMS, held) == form
    if form[0] == "pairs":
        assert K * (2 if dtype is BF else 1) > 6 * 128 and -(-rows // form[1]) * -(-N // 256) > SMS // 2


def test_every_form_has_sizes(sv):
    """Sizes over the whole range reach no other forms than those above (and pairs of 64 tokens)."""
    known = set(FORMS) | {("pairs", 64, 1)}
    seen = set()
    for dtype in (BF, E4):
        for rows in (1, 2, 3, 4, 5, 9, 16, 17, 31, 40, 64, 65, 100, 129, 200, 257, 300, 500, 777, 1024, 2000, 4096, 20000):
            for N in (1, 16, 100, 129, 300, 777, 1024, 2000, 4096, 5000, 8192, 12000, 20000, 50257, 152064):
                for K in (16, 48, 128, 512, 784, 1024, 2000, 4096, 8192, 16384):
                    seen.add(sv.spec_linear_form(rows, N, K, dtype, SMS, CLUSTERS[0]))
    assert seen <= known, seen - known
    assert len(seen) > 20  # (the sweep is not empty)


def test_many_tiles_take_pairs(sv):
    for (rows, N, K), dtype in MANY_TILES:
        for held in CLUSTERS:
            kind, bn, _ = sv.spec_linear_form(rows, N, K, dtype, SMS, held)
            assert kind == "pairs" and -(-rows // bn) * -(-N // 256) >= 3 * (SMS // 2)


def test_refusals(sv):
    E = sv.SpecVerifyError
    for args in ((0, 64, 64), (-1, 64, 64), (1, 0, 64), (1, 64, 12), (1, 64, 0), (1 << 20, 1 << 20, 64)):
        with pytest.raises(E):
            sv.spec_linear_form(*args, BF, SMS, CLUSTERS[0])
    with pytest.raises(E):
        sv.spec_linear_form(1, 64, 8, E4, SMS, CLUSTERS[0])
    with pytest.raises(E):
        sv.spec_linear_form(1, 64, 64, BF, 1, CLUSTERS[0])
    with pytest.raises(TypeError):
        sv.spec_linear_form(1, 64, 64, torch.float16, SMS, CLUSTERS[0])
    with pytest.raises(ValueError):
        sv.spec_linear_form(1, 64, 64, BF, SMS)
    lib = sv.load_library()
    assert lib.spec_linear_form(1, 64, 64, 1, SMS, None, None) == sv.SPEC_EINVAL
