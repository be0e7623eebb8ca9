"""The rule's calls by the path that their sizes choose, with the launches counted to show which one
ran: a few tokens for many (sequence, head) units token by token, one long sequence in two parts.
Bounds are those of test_gdr and test_gdr_bwd (fp32 arithmetic for the token-by-token path)."""
import pytest

torch = pytest.importorskip("torch")
import rule_reference as ref  # noqa: E402
import test_gdr as base  # noqa: E402
import test_gdr_bwd as back  # noqa: E402
from test_gdr import draw, kda  # noqa: E402,F401
from test_gdr_streams import launches  # noqa: E402

TYPES = base.TYPES


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 7, 8, 9])
@pytest.mark.parametrize("init,final,gate", [("f32", "bf16", "f32"), ("bf16", "f32", "bf16"), (None, "f32", "f32"), ("f32", None, "bf16")])
def test_fwd_a_few_tokens_for_many_units(kda, T, init, final, gate):  # noqa: F811
    """At most 8 tokens of fixed length for more units than SMs: the step's kernel and its
    accuracy; with 9 tokens the chunks."""
    B, Hk, Hv = 70, 2, 6
    *x, n = draw(B, max(T, 1), Hk, Hv, 300 + T, gate, packed=True)
    if T == 0:
        x = [t[:, :0] for t in x]
    S = None if init is None else (0.5 * n(B, Hv, 128, 128)).to(TYPES[init])
    done = []
    count = launches(kda, lambda: done.append(base.run_fwd(kda, x, S, final)))
    out, fs = done[0]
    few = T <= 8
    assert count["gdr_step_kernel"] == few and count["gdr_chain_kernel"] == (not few)
    if not few:
        return base.check_fwd(x, S, out, fs, [(b, 0, T) for b in range(B)])
    for b in range(0, B, 3):
        s = torch.zeros(Hv, 128, 128, device="cuda") if S is None else S[b]
        o, last, _ = ref.rule(*(t[b] for t in x), base.SCALE, s)
        base.check_out(out[b], o)
        if fs is not None:
            base.check_state(fs[b], last, T)
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,H,step", [(8, 8, 32, True), (4, 8, 38, False), (153, 1, 1, True), (152, 1, 1, False)])
def test_fwd_units_against_sms(kda, B, T, H, step):  # noqa: F811
    """The rule's other side (152 SMs), and a state that is updated in place on both."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("sizes for 152 SMs")
    *x, n = draw(B, T, H, H, 310)
    S = 0.5 * n(B, H, 128, 128)
    want = S.clone()
    out, out2 = torch.empty_like(x[2]), torch.empty_like(x[2])
    count = launches(kda, lambda: kda.kda_gdr_fwd(*x, base.SCALE, out, initial_state=S, final_state=S))
    assert count["gdr_step_kernel"] == step and count["gdr_chain_kernel"] == (not step)
    apart = torch.empty_like(S)
    kda.kda_gdr_fwd(*x, base.SCALE, out2, initial_state=want, final_state=apart)
    assert torch.equal(apart, S) and torch.equal(out, out2)
    base.check_fwd(x, want, out, S, [(b, 0, T) for b in range(B)])


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hk,Hv,gate,init,final", [(4096, 40, 40, "f32", "f32", "bf16"), (4200, 20, 60, "bf16", "bf16", "f32"),
                                                     (4111, 48, 96, "f32", None, "f32")])
def test_fwd_two_parts(kda, T, Hk, Hv, gate, init, final):  # noqa: F811
    """Two launches of both kernels; the bits of three calls that hand fp32 states on, and of the
    same call in one part while the stream is being captured."""
    *x, n = draw(1, T, Hk, Hv, 320, gate, packed=True)
    S = None if init is None else (0.5 * n(1, Hv, 128, 128)).to(TYPES[init])
    done = []
    count = launches(kda, lambda: done.append(base.run_fwd(kda, x, S, final)))
    out, fs = done[0]
    assert count["gdr_prep_kernel"] == count["gdr_chain_kernel"] == 2
    state, outs = S, []
    cuts = [0, 1536, 2880, T]
    for a, b in zip(cuts[:-1], cuts[1:]):
        y = [t[:, a:b] for t in x[:3]] + [t[:, a:b].contiguous() for t in x[3:]]
        part = []
        count = launches(kda, lambda: part.append(base.run_fwd(kda, y, state, "f32" if b < T else final)))
        assert count["gdr_chain_kernel"] == 1
        outs.append(part[0][0])
        state = part[0][1]
    assert torch.equal(out, torch.cat(outs, 1)) and torch.equal(fs, state)
    again, last = torch.zeros_like(out), torch.zeros_like(fs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_gdr_fwd(*x, base.SCALE, again, initial_state=S, final_state=last)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out) and torch.equal(last, fs)
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hk,Hv,gate,init", [(4300, 5, 15, "f32", "f32"), (2100, 38, 38, "bf16", "bf16"), (4180, 2, 16, "f32", None)])
def test_bwd_two_parts(kda, T, Hk, Hv, gate, init):  # noqa: F811
    """Two launches of the gradient's chain and of the chunk kernel; the same bits in one part."""
    *x, n = draw(1, T, Hk, Hv, 330, gate, packed=True)
    dout, dS = n(1, T, Hv, 128).bfloat16(), 0.3 * n(1, Hv, 128, 128)
    S = None if init is None else (0.5 * n(1, Hv, 128, 128)).to(TYPES[init])
    done = []
    count = launches(kda, lambda: done.append(back.run(kda, x, dout, S, dS)))
    assert count["gdr_bwd_chain_kernel"] == count["gdr_bwd_chunk_kernel"] == 2 * 2      # run() calls twice
    two = done[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = kda.kda_gdr_bwd(*x, back.SCALE, dout, initial_state=S, d_final_state=dS)
    graph.replay()
    torch.cuda.synchronize()
    for m in two:
        assert torch.equal(one[m], two[m]), m
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
def test_bwd_two_parts_match_the_definition(kda):  # noqa: F811
    """Two parts with three value heads to a key head, against the definition in 64 bits."""
    T, Hk, Hv = 2240, 10, 30
    *x, n = draw(1, T, Hk, Hv, 331, packed=True)
    dout, S = n(1, T, Hv, 128).bfloat16(), 0.5 * n(1, Hv, 128, 128)
    done = []
    count = launches(kda, lambda: done.append(back.run(kda, x, dout, S)))
    assert count["gdr_bwd_chunk_kernel"] == 2 * 2
    back.check(done[0], x, dout, S, None, [(0, 0, T)])
