"""Gradients of the rule where the kernels do not each take one piece of work: more (chunk, key
head) pairs than SMs, with one and with several value heads to a key head, against the
definition in 64 bits as in test_gdr_bwd; and one sequence long enough for two parts."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import test_gdr_bwd as base  # noqa: E402
from test_gdr import draw, kda  # noqa: E402,F401


@pytest.mark.gpu
def test_bwd_more_pairs_than_sms(kda):  # noqa: F811
    *x, n = draw(12, 130, 16, 16, 71, packed=True)
    dout, S = n(12, 130, 16, 128).bfloat16(), 0.5 * n(12, 16, 128, 128)
    base.check(base.run(kda, x, dout, S), x, dout, S, None, [(b, 0, 130) for b in range(12)])


@pytest.mark.gpu
def test_bwd_more_pairs_than_sms_packed(kda):  # noqa: F811
    lens = [int(a) for a in np.random.default_rng(5).integers(0, 140, size=24)]
    T, Hk, Hv = sum(lens), 8, 16
    *x, n = draw(1, T, Hk, Hv, 72, "bf16", packed=True)
    dout, dS = n(1, T, Hv, 128).bfloat16(), 0.3 * n(len(lens), Hv, 128, 128)
    ends = np.cumsum([0] + lens)
    cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    base.check(base.run(kda, x, dout, None, dS, cu), x, dout, None, dS,
               [(0, int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])])


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hk,Hv", [(2010, 16, 32), (4150, 5, 15)])
def test_bwd_in_two_parts_is_the_same_in_one(kda, T, Hk, Hv):  # noqa: F811
    """One long sequence of few heads is worked on in two parts, but not while the stream is being
    captured: the same bits both ways."""
    *x, n = draw(1, T, Hk, Hv, 73, packed=True)
    dout, S, dS = n(1, T, Hv, 128).bfloat16(), 0.5 * n(1, Hv, 128, 128), 0.3 * n(1, Hv, 128, 128)
    two = base.run(kda, x, dout, S, dS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = kda.kda_gdr_bwd(*x, base.SCALE, dout, initial_state=S, d_final_state=dS)
    graph.replay()
    torch.cuda.synchronize()
    assert kda.kda_fwd_get_error() == 0
    for m in two:
        assert torch.equal(one[m], two[m]), m
