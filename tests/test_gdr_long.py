"""One long sequence: its chunks are prepared in two parts, the second beside the first's
chains.  Results are those of shorter calls that hand the state on, bit for bit."""
import pytest

from test_gdr import kda  # noqa: F401  (the package, or a skip)


def draw(torch, T, Hk, Hv, gate):
    gen = torch.Generator(device="cuda").manual_seed(T + Hv)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    q, k = (torch.nn.functional.normalize(n(1, T, Hk, 128), dim=-1).bfloat16() for _ in range(2))
    # values as a view of a wider buffer
    v = n(1, T, Hv * 128 + 64).bfloat16()[..., :Hv * 128].view(1, T, Hv, 128)
    return q, k, v, (-0.3 * n(1, T, Hv).abs()).to(gate), torch.sigmoid(n(1, T, Hv)).to(gate)


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hk,Hv,gate,init", [(4097, 1, 2, "float32", None), (4200, 2, 2, "bfloat16", "float32"),
                                               (5000, 16, 32, "float32", "bfloat16"), (4500, 64, 128, "bfloat16", None)])
def test_parts_give_what_separate_calls_give(kda, T, Hk, Hv, gate, init):  # noqa: F811
    import torch
    x = draw(torch, T, Hk, Hv, getattr(torch, gate))
    S = None if init is None else (0.3 * torch.randn(1, Hv, 128, 128, device="cuda")).to(getattr(torch, init))

    def run(state):
        out, final = torch.full((1, T, Hv, 128), 7.0, device="cuda").bfloat16(), torch.empty(1, Hv, 128, 128, device="cuda")
        kda.kda_gdr_fwd(*x, 0.1, out, initial_state=state, final_state=final)
        return out, final

    out, final = run(S)
    state, pieces = S, []
    for a, b in ((0, 2048), (2048, 4096), (4096, T)):       # whole chunks; too short for two parts
        y, nxt = torch.empty(1, b - a, Hv, 128, device="cuda").bfloat16(), torch.empty(1, Hv, 128, 128, device="cuda")
        part = [t[:, a:b] if i < 3 else t[:, a:b].contiguous() for i, t in enumerate(x)]
        kda.kda_gdr_fwd(*part, 0.1, y, initial_state=state, final_state=nxt)
        state = nxt
        pieces.append(y)
    assert kda.kda_fwd_get_error() == 0
    assert torch.equal(out, torch.cat(pieces, 1))
    assert torch.equal(final, state)
    # on another stream, right after work that it depends on
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run(S)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again[0], out) and torch.equal(again[1], final)


@pytest.mark.gpu
def test_a_long_call_can_be_captured(kda):  # noqa: F811
    import torch
    T, Hv = 4300, 4
    x = draw(torch, T, 2, Hv, torch.float32)
    out, want = (torch.zeros(1, T, Hv, 128, device="cuda").bfloat16() for _ in range(2))
    kda.kda_gdr_fwd(*x, 0.1, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_gdr_fwd(*x, 0.1, out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hk,Hv,gate,init,dfinal", [(2100, 16, 32, "bfloat16", None, None),
                                                      (1990, 16, 48, "float32", "float32", "bfloat16")])
def test_backward_in_parts_gives_what_separate_calls_give(kda, T, Hk, Hv, gate, init, dfinal):  # noqa: F811
    """The gradient's chain in two parts: the same as three calls, last tokens first, that hand
    the gradient of the state back (fp32; a power of two scales each call's gradients, so that only
    gradients too small for fp16 may differ)."""
    import torch
    x = draw(torch, T, Hk, Hv, getattr(torch, gate))
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    d_out = n(1, T, Hv, 128).bfloat16()
    S = None if init is None else (0.3 * n(1, Hv, 128, 128)).to(getattr(torch, init))
    dS = None if dfinal is None else (0.3 * n(1, Hv, 128, 128)).to(getattr(torch, dfinal))
    got = kda.kda_gdr_bwd(*x, 0.1, d_out, initial_state=S, d_final_state=dS)
    cuts = [0, 768, 1280, T]
    states = [torch.zeros(1, Hv, 128, 128, device="cuda") if S is None else S.float()]
    piece = lambda t, a, b: t[:, a:b].contiguous()
    for a, b in zip(cuts[:-2], cuts[1:-1]):
        states.append(torch.empty(1, Hv, 128, 128, device="cuda"))
        kda.kda_gdr_fwd(*(piece(t, a, b) for t in x), 0.1, torch.empty_like(piece(d_out, a, b)),
                        initial_state=states[-2], final_state=states[-1])
    back, parts = dS, {k: [] for k in ("dq", "dk", "dv", "dg", "dbeta")}
    for i in (2, 1, 0):
        a, b = cuts[i], cuts[i + 1]
        r = kda.kda_gdr_bwd(*(piece(t, a, b) for t in x), 0.1, piece(d_out, a, b), initial_state=states[i], d_final_state=back)
        back = r["d_initial_state"]
        for k in parts:
            parts[k].insert(0, r[k])
    assert kda.kda_fwd_get_error() == 0
    for k in parts:
        want = torch.cat(parts[k], 1).float()
        # results of the same operations; what the scale's power of two changes is below fp16's
        # smallest normal numbers, 2^-14 of values scaled to 16 .. 32: far under a bf16 half unit
        assert ((got[k].float() - want).norm() <= 2.0 ** -8 * want.norm()), k
    if S is not None:
        assert (got["d_initial_state"].float() - back.float()).norm() <= 2.0 ** -8 * back.norm()
