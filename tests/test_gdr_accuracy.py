"""The accuracy that the rule's kernels claim, on results of 32 bits, where a bf16 rounding does
not hide it.

Bounds, from the roundings: an operand in fp16 is off by at most 2^-12 of itself, 2^-12 / sqrt 3 =
1.4e-4 in the mean; a product of two by 2.0e-4, independently from term to term.  A state is what
three products in a row make (R, X, and the update): 2.0e-4 sqrt 3 = 3.5e-4 of its norm where errors do
not add up over tokens, held to the 2^-10 that the kernels' comment claims.  Gradients go through the states and X (3.5e-4), the same
chain backwards (3.5e-4) and a product of both (2.0e-4): 5.3e-4, held to 1e-3; dg is a difference of
sums of that size, which cancel to a quarter in these draws or less: 4e-3.  bf16 results add the rounding
of the definition's own values."""
import pytest

torch = pytest.importorskip("torch")
import rule_reference as ref  # noqa: E402
import test_gdr_bwd as back  # noqa: E402
from test_gdr import SCALE, draw, kda, run_fwd  # noqa: E402,F401

CASES = [(1, 512, 2, 4, 0.05, 0.0), (1, 700, 1, 2, 0.3, 0.3), (3, 130, 2, 2, 0.01, 0.0), (1, 1000, 1, 1, 0.001, 0.2)]
STATES = 2.0 ** -10


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def bound(got, want, own):
    rounding = off(want.to(got.dtype), want)
    return 1.05 * (rounding ** 2 + own ** 2) ** 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_states_in_32_bits(kda, case):  # noqa: F811
    B, T, Hk, Hv, decay, mean = case
    *x, n = draw(B, T, Hk, Hv, 500 + T, decay=decay, mean=mean)
    S = 0.5 * n(B, Hv, 128, 128)
    out, fs = run_fwd(kda, x, S, "f32")
    for b in range(B):
        o, last, _ = ref.rule(*(t[b] for t in x), SCALE, S[b])
        assert off(fs[b], last) <= bound(fs, last, STATES), off(fs[b], last)
        assert off(out[b], o) <= bound(out, o, STATES), off(out[b], o)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradients_in_32_bits(kda, case):  # noqa: F811
    B, T, Hk, Hv, decay, mean = case
    *x, n = draw(B, T, Hk, Hv, 510 + T, decay=decay, mean=mean)
    dout, S, dS = n(B, T, Hv, 128).bfloat16(), 0.5 * n(B, Hv, 128, 128), 0.3 * n(B, Hv, 128, 128)
    r = back.run(kda, x, dout, S, dS)
    for b in range(B):
        want = ref.rule_bwd(*(t[b] for t in x), SCALE, S[b], dout[b], dS[b])
        for m, w in zip(back.NAMES + ("d_initial_state",), want):
            assert off(r[m][b], w) <= bound(r[m], w, 4e-3 if m == "dg" else 1e-3), (m, off(r[m][b], w))
