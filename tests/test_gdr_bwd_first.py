"""The decay of a sequence's first token has nothing to act on without an initial state: its
gradient is zero, exactly, not the rounding of sums that cancel."""
import pytest

torch = pytest.importorskip("torch")
import test_gdr_bwd as back  # noqa: E402
from test_gdr import draw, kda  # noqa: E402,F401


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hk,Hv", [([1], 3, 9), ([1, 1, 0, 1], 2, 2), ([5, 1, 64, 65, 130], 1, 4)])
def test_first_decay(kda, lens, Hk, Hv):  # noqa: F811
    T, ends = sum(lens), [sum(lens[:i]) for i in range(len(lens) + 1)]
    *x, n = draw(1, T, Hk, Hv, 600 + T, packed=True)
    dout, dS = n(1, T, Hv, 128).bfloat16(), n(len(lens), Hv, 128, 128)
    cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    r = back.run(kda, x, dout, None, dS, cu)
    for a, b in zip(ends[:-1], ends[1:]):
        if b > a:
            assert bool((r["dg"][0, a] == 0).all())
    back.check(r, x, dout, None, dS, list(zip([0] * len(lens), ends[:-1], ends[1:])))
    S = n(len(lens), Hv, 128, 128)
    r = back.run(kda, x, dout, S, dS, cu)
    assert bool((r["dg"][0, 0] != 0).all())


@pytest.mark.gpu
def test_first_decay_in_two_parts(kda):  # noqa: F811
    T, H = 2112, 32
    *x, n = draw(1, T, H, H, 610)
    dout = n(1, T, H, 128).bfloat16()
    r = back.run(kda, x, dout)
    assert bool((r["dg"][0, 0] == 0).all())
    assert bool((r["dg"][0, 1:] != 0).any(-1).all())
