"""spec_linear in every form of its kernel (marked gpu): the sizes of test_linear_forms.py, which a
test there ties to their forms, against the formula in 64 bits -- every tile width with every split
of K, CTA pairs whose ring of six slices wraps and whose accumulators are used again.

Beside the worst-case bound of test_gpu_linear.compare, fp32 outputs without an activation have to
hold a bound on their root mean square (of terms of random signs, so that the partial sum S_k of
k of n = K/16 additions has the root mean square sqrt(k/n) of the whole).  The tensor cores truncate:
an addition loses up to one step of S_k, 2^-23 |S_k| at most and half of that in the mean, always
towards zero, so the means add up: at most 2^-24 sum_k sqrt(k/n) <= 2^-24 (2n/3 + 1) in all (an
unsplit K of 9136 in bf16 reaches 1.0e-5 of a bound of 2.8e-5; the library's bf16 product is off by the
same amount).  What is left of each loss has no mean: sqrt(n + 16) such errors of 2^-23, twice.
Scales, bias and residual add 16 roundings 2^-24 of their magnitudes.
"""
import pytest
import torch

from test_gpu_linear import compare, problem
from test_linear_forms import CASE_IDS, CASES, MANY_TILES

pytestmark = pytest.mark.gpu

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ACTS = ["relu", "gelu", "gelu_tanh", "silu", "none"]
SPLIT = [c for c in CASES if c[0][2] > 1]
SPLIT_IDS = [i for c, i in zip(CASES, CASE_IDS) if c[0][2] > 1]
PAIRS = [c for c in CASES if c[0][0] == "pairs"]
PAIR_IDS = [i for c, i in zip(CASES, CASE_IDS) if c[0][0] == "pairs"]


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_31_gb300 as m
    m.load_library()
    return m


def rms(t):
    return float(t.double().square().mean().sqrt())


def near_in_the_mean(got, x, w, x_scale=None, w_scale=None, bias=None, residual=None, out_dtype=F32):
    x64, w64 = x.float().double(), w.float().double()
    if x_scale is not None:
        x64, w64 = x64 * x_scale.double()[:, None], w64 * w_scale.double()[:, None]
    v = x64 @ w64.T
    n = x.shape[1] / 16
    tol = ((2 * n / 3 + 1) * 2.0 ** -24 + 2 * (n + 16) ** 0.5 * 2.0 ** -23) * rms(v)
    parts = rms(v)
    for extra in (bias, residual):
        if extra is not None:
            v = v + extra.double()
            parts += rms(extra)
    off = rms(got.double() - v)
    assert off <= tol + 16 * 2.0 ** -24 * parts, (off, tol)


@pytest.mark.parametrize("form,size,dtype", CASES, ids=CASE_IDS)
def test_plain(sv, form, size, dtype):
    """fp32 out, nothing in the epilogue but the scales."""
    rows, N, K = size
    assert sv.spec_linear_form(rows, N, K, dtype) == form
    x, w, kw = problem(rows + N, rows, N, K, dtype is E4, F32, False, False)
    got = sv.spec_linear(x, w, **kw)
    compare(got, x, w, **kw)
    near_in_the_mean(got, x, w, **kw)
    assert sv.spec_verify_check() == sv.SPEC_OK


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("whole", [False, True], ids=["odd", "fours"])
@pytest.mark.parametrize("i", range(len(CASES)), ids=CASE_IDS)
def test_whole_epilogue(sv, i, whole, out):
    """Bias, activation and residual, channels off a group of four and on it."""
    form, (rows, N, K), dtype = CASES[i]
    N = N // 4 * 4 if whole else N
    act = ACTS[(i + whole) % 5]
    x, w, kw = problem(i, rows, N, K, dtype is E4, out, True, True)
    got = sv.spec_linear(x, w, activation=act, **kw)
    compare(got, x, w, act, **kw)
    if act == "none" and out is F32:
        near_in_the_mean(got, x, w, **kw)


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("i", range(len(MANY_TILES)))
def test_many_tiles_a_pair(sv, i, residual):
    (rows, N, K), dtype = MANY_TILES[i]
    assert sv.spec_linear_form(rows, N, K, dtype)[0] == "pairs"
    x, w, kw = problem(i, rows, N, K, dtype is E4, F32, True, residual)
    got = sv.spec_linear(x, w, **kw)
    compare(got, x, w, **kw)
    near_in_the_mean(got, x, w, **kw)


@pytest.mark.parametrize("form,size,dtype", SPLIT + PAIRS, ids=SPLIT_IDS + PAIR_IDS)
def test_in_place_guards_and_repeats(sv, form, size, dtype):
    """The same call gives the same bits (a split K is summed in a fixed order), also with out =
    residual; the rows around the result stay."""
    rows, N, K = size
    x, w, kw = problem(7, rows, N, K, dtype is E4, BF, True, True)
    want = sv.spec_linear(x, w, activation="silu", **kw)
    for _ in range(3):
        assert torch.equal(sv.spec_linear(x, w, activation="silu", **kw), want)
    buf = torch.full((rows + 2, N), 9.0, dtype=BF, device="cuda")
    buf[1:rows + 1] = kw["residual"]
    mid = buf[1:rows + 1]
    sv.spec_linear(x, w, activation="silu", out=mid, **{**kw, "residual": mid})
    assert torch.equal(mid, want) and bool((buf[0] == 9).all()) and bool((buf[-1] == 9).all())


@pytest.mark.parametrize("form,size,dtype", SPLIT + PAIRS, ids=SPLIT_IDS + PAIR_IDS)
def test_nan_stays_in_its_row_and_column(sv, form, size, dtype):
    rows, N, K = size
    x, w, kw = problem(8, rows, N, K, dtype is E4, F32, False, False)
    x[1, K - 1] = float("nan")
    w[N - 1, 3] = float("nan")
    got = sv.spec_linear(x, w, **kw)
    assert bool(got[1].isnan().all()) and bool(got[:, N - 1].isnan().all())
    keep = [r for r in range(rows) if r != 1]
    assert bool(got[keep][:, :N - 1].isfinite().all())


@pytest.mark.parametrize("form,size,dtype", SPLIT[::3] + PAIRS[::4], ids=SPLIT_IDS[::3] + PAIR_IDS[::4])
def test_captured_and_overlapping_calls(sv, form, size, dtype):
    rows, N, K = size
    x, w, kw = problem(9, rows, N, K, dtype is E4, BF, True, True)
    out = torch.empty(rows, N, dtype=BF, device="cuda")
    sv.spec_linear(x, w, activation="gelu", out=out, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_linear(x, w, activation="gelu", out=out, **kw)
    side = torch.cuda.Stream()
    for seed in range(2):
        x2 = problem(60 + seed, rows, N, K, dtype is E4, BF, False, False)[0]
        x.copy_(x2)
        torch.cuda.synchronize()
        graph.replay()
        other = [sv.spec_linear(x2, w, activation="gelu", stream=side, **kw) for _ in range(3)]
        torch.cuda.synchronize()
        compare(out, x2, w, "gelu", **kw)
        assert all(torch.equal(o, out) for o in other)
    assert sv.spec_verify_check() == sv.SPEC_OK
