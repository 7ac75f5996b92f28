"""The activations of spec_linear on a dense grid, fp32 output (marked gpu).

The product is zero and the bias holds the argument, so v is exact and the error is the
activation's own.  Bounds in units of e = 2^-24, from the operations of each form:

silu and gelu_tanh, v / (1 + e^-t): 2^x on the special-function unit 4 e, its argument's rounding
and the constant's 1.3 |t| e; the sum 1 e, the division (2 ulp) 4 e; the tanh form's t itself 4 e
relative, so 4 |t| e more.  A denominator past 2^126 gives 0 for |v| / (1 + e^|t|), which is then
below |v| 2^-126 (flush; 2^-119.5 for silu at v = -87.4, the largest).

gelu, max(v, 0) - s Q(s) e^{-a^2/2} with a = |v|: of the second term, s 4 e (reciprocal 1 ulp, two
roundings), Q's fit 0.5 e, its coefficients and Horner steps 3 cond e, where cond = sum |c_k| s^k
/ Q(s) <= 2 + 1.7 a, the power 4 e and its argument 1.2 a^2 e, two products 2 e: at most
(18 + 5 a + 1.2 a^2) e; the last subtraction 1 e of the result.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_31_gb300 as m
    m.load_library()
    return m


def expected(v, act):
    """The activation in 64 bits, and its bound."""
    flush = v.abs().clamp(min=1) * 2.0 ** -126
    if act == "gelu":
        a = v.abs()
        term = a * 0.5 * torch.special.erfc(a / math.sqrt(2))
        want = v.clamp(min=0) - term
        return want, (18 + 5 * a + 1.2 * a * a) * E * term + E * want.abs() + flush
    t = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    want = v * torch.sigmoid(t)
    slope = 1.3 if act == "silu" else 6.0
    return want, (10 + slope * t.abs()) * E * want.abs() + flush


@pytest.mark.parametrize("rows", [2, 40, 300])
@pytest.mark.parametrize("act,end", [("gelu", 13.0), ("gelu_tanh", 9.0), ("silu", 100.0)])
def test_dense_grid(sv, act, end, rows):
    N = 32768
    v = torch.linspace(-end, end, N, device="cuda", dtype=torch.float64).float()
    v[0], v[1], v[2] = 0.0, 1e-20, -1e-20
    x, w = torch.zeros(rows, 64, dtype=BF, device="cuda"), torch.zeros(N, 64, dtype=BF, device="cuda")
    got = sv.spec_linear(x, w, v, act, out_dtype=F32)
    assert torch.equal(got, got[:1].expand_as(got))
    want, tol = expected(v.double(), act)
    excess = (got[0].double() - want).abs() / tol
    assert float(excess.max()) <= 1.0, (float(excess.max()), float(v[excess.argmax()]))


@pytest.mark.parametrize("act,end", [("gelu", 8.0), ("gelu_tanh", 8.0), ("silu", 16.0)])
def test_bf16_output_is_the_rounded_value(sv, act, end):
    """In bf16 the activation's error is invisible: half a step of the type, widened by the bound."""
    N = 16384
    v = torch.linspace(-end, end, N, device="cuda").to(BF)
    x, w = torch.zeros(33, 64, dtype=BF, device="cuda"), torch.zeros(N, 64, dtype=BF, device="cuda")
    got = sv.spec_linear(x, w, v, act)
    want, tol = expected(v.double(), act)
    assert bool(((got.double() - want).abs() <= (1 + 2.0 ** -8) * tol + 2.0 ** -8 * want.abs()).all())
