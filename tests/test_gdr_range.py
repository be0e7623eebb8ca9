"""kda_gdr_fwd and kda_gdr_bwd on values, states and gradients of any size: the rule is linear in
values and initial states, its gradients in the incoming ones, and the results keep the accuracy
that they have at size 1.

Bounds.  The chunks' operands have fp16's 11 bits, and each of the few products that an element
goes through rounds its operands once: errors of 2^-12 each, random, over sums of 64 to 128
terms.  Held here, as a norm over a whole tensor beside the output's own rounding (2^-9 of its size
for bf16): 2^-9 = 0.002, four times one operand's largest rounding.  (An error that comes from
subnormal operands is larger: 0.5 % for values of size 1e-5, half of everything at 1e-7.)"""
import pytest

torch = pytest.importorskip("torch")
import rule_reference as ref  # noqa: E402
import test_gdr_bwd as back  # noqa: E402
from test_gdr import SCALE, TYPES, draw, kda, run_fwd  # noqa: E402,F401

OWN = {torch.bfloat16: 2.0 ** -9, torch.float32: 0.0}


def near(name, got, want, bound=2.0 ** -9):
    off, size = (got.double() - want).norm(), want.norm()
    assert bool(got.isfinite().all()), name
    assert float(off) <= (bound + OWN[got.dtype]) * float(size), (name, float(off / size))


def sequences(x, init, scale=SCALE):
    q, k, v, g, beta = x
    outs, last = [], []
    for b in range(v.shape[0]):
        S = init[b] if init is not None else torch.zeros(v.shape[2], 128, 128, device="cuda")
        o, s, _ = ref.rule(q[b], k[b], v[b], g[b], beta[b], scale, S)
        outs.append(o)
        last.append(s)
    return torch.stack(outs), torch.stack(last)


SIZES = [1e-30, 1e-12, 1e-8, 1e-7, 1e-6, 1e-5, 1.0, 300.0, 1e5, 1e12, 1e30]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("init,T", [(None, 512), ("f32", 200), ("bf16", 65)])
def test_fwd_values_and_states_of_any_size(kda, size, init, T):  # noqa: F811
    q, k, v, g, beta, n = draw(1, T, 2, 4, 400, decay=0.05)
    v = (size * v.float()).bfloat16()
    S = None if init is None else (0.5 * size * n(1, 4, 128, 128)).to(TYPES[init])
    out, fs = run_fwd(kda, (q, k, v, g, beta), S, "f32")
    o, last = sequences((q, k, v, g, beta), S)
    near("out", out, o)
    for h in range(4):
        near("state", fs[:, h], last[:, h])
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [(1e-8, 1.0), (1.0, 1e-8), (0.0, 1e-8), (1e8, 1e-8), (1e-8, 1e8), (1e20, 1e-12)], ids=str)
def test_fwd_sizes_that_change_on_the_way(kda, sizes):  # noqa: F811
    """The values' size changes between two chunks, and between two tokens of one; a decay that
    forgets what was before makes the new size the results' own.  A chunk's tokens and the state
    that it begins with share one scale: where the size falls, the tokens of that chunk and of the
    next are held to 2^-20 of the larger size, and what they leave in the state fades (e^-3.2 a
    chunk), so that three chunks on the new size's accuracy is there."""
    q, k, v, g, beta, n = draw(1, 640, 1, 2, 401, decay=0.05)
    for where in (256, 300):
        w = v.float()
        w = torch.cat([sizes[0] * w[:, :where], sizes[1] * w[:, where:]], 1).bfloat16()
        h = g.clone()
        h[:, where] = -float("inf")
        x = (q, k, w, h, beta)
        out, fs = run_fwd(kda, x, None, "f32")
        o, last = sequences(x, None)
        falls = sizes[1] < sizes[0]
        chunk = where // 64 * 64
        after = chunk + (256 if falls else 64)
        near("before", out[:, :chunk], o[:, :chunk])
        near("after", out[:, after:], o[:, after:])
        if falls:
            off = (out.double() - o)[:, where:].abs()
            assert bool((off <= 2.0 ** -20 * sizes[0] + 2.0 ** -8 * o[:, where:].abs()).all())
        near("state", fs, last)


@pytest.mark.gpu
def test_fwd_heads_and_sequences_of_different_sizes(kda):  # noqa: F811
    q, k, v, g, beta, n = draw(1, 500, 2, 4, 402, decay=0.05)
    size = torch.tensor([1e-9, 1.0, 1e6, 1e-20], device="cuda")
    v = (v.float() * size[:, None])
    v[:, 200:] *= 1e-6
    x = (q, k, v.bfloat16(), g, beta)
    cu = torch.tensor([0, 200, 500], dtype=torch.int32, device="cuda")
    out, fs = run_fwd(kda, x, None, "f32", cu, 2)
    for i, (a, b) in enumerate(((0, 200), (200, 500))):
        o, last = sequences([t[:, a:b] for t in x], None)
        for h in range(4):
            near("out", out[:, a:b, h], o[:, :, h])
            near("state", fs[i, h], last[0, h])


@pytest.mark.gpu
def test_fwd_an_initial_state_that_fades(kda):  # noqa: F811
    """A state of size 1 under strong decays, values of 1e-10: what remains is theirs."""
    q, k, v, g, beta, n = draw(1, 512, 1, 2, 403, decay=1.0)
    x = (q, k, (1e-10 * v.float()).bfloat16(), g, beta)
    S = n(1, 2, 128, 128)
    out, fs = run_fwd(kda, x, S, "f32")
    o, last = sequences(x, S)
    near("out", out[:, 192:], o[:, 192:])
    near("state", fs, last)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(4224, 40), (4096, 2)])
def test_fwd_long_sequences_of_small_values(kda, T, H):  # noqa: F811
    """In two parts and in one: the results of size 1, exactly, times a power of two."""
    q, k, v, g, beta, n = draw(1, T, H, H, 404, decay=0.05)
    S = 0.5 * n(1, H, 128, 128)
    out, fs = run_fwd(kda, (q, k, v, g, beta), S, "f32")
    small = 2.0 ** -40
    o2, f2 = run_fwd(kda, (q, k, (small * v.float()).bfloat16(), g, beta), small * S, "f32")
    near("out", o2 / small, out.double(), 2.0 ** -9)
    near("state", f2 / small, fs.double(), 2.0 ** -12)


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dsize", [1e-20, 1.0, 1e6])
def test_bwd_values_states_and_gradients_of_any_size(kda, size, dsize):  # noqa: F811
    if size * dsize < 1e-33:
        pytest.skip("gradients smaller than the types hold")
    q, k, v, g, beta, n = draw(1, 330, 2, 4, 410, decay=0.05)
    v = (size * v.float()).bfloat16()
    S = 0.5 * size * n(1, 4, 128, 128)
    dout, dS = (dsize * n(1, 330, 4, 128)).bfloat16(), 0.3 * dsize * n(1, 4, 128, 128)
    x = (q, k, v, g, beta)
    r = back.run(kda, x, dout, S, dS)
    want = ref.rule_bwd(*(t[0] for t in x), SCALE, S[0], dout[0], dS[0])
    for m, w in zip(back.NAMES, want):
        near(m, r[m][0], w, 2.0 ** -8)
    near("d_initial_state", r["d_initial_state"][0], want[5], 2.0 ** -8)


@pytest.mark.gpu
def test_bwd_heads_of_a_group_of_different_sizes(kda):  # noqa: F811
    """Value heads of one key head whose values and gradients differ in size: dq and dk are their
    sum, which the largest products dominate, in whatever order the heads come."""
    for order in ((1e-9, 1.0, 1e5), (1e5, 1.0, 1e-9), (1.0, 1e5, 1e-9)):
        for grads in ((1.0, 1.0, 1.0), (1e6, 1e-6, 1.0)):
            q, k, v, g, beta, n = draw(1, 200, 1, 3, 411, decay=0.05)
            a, b = (torch.tensor(t, device="cuda")[:, None] for t in (order, grads))
            x = (q, k, (v.float() * a).bfloat16(), g, beta)
            dout = (n(1, 200, 3, 128) * b).bfloat16()
            r = back.run(kda, x, dout)
            want = ref.rule_bwd(*(t[0] for t in x), SCALE, torch.zeros(3, 128, 128, device="cuda"), dout[0],
                                torch.zeros(3, 128, 128, device="cuda"))
            for m, w in zip(back.NAMES, want):
                if w.shape[1] == 1:
                    near(m, r[m][0], w, 2.0 ** -8)
                else:
                    for h in range(3):
                        near(m, r[m][0, :, h], w[:, h], 2.0 ** -8)


@pytest.mark.gpu
@pytest.mark.parametrize("T,strength", [(5000, 0.0), (5000, 1.0), (20000, 0.0)])
def test_bwd_gradients_that_add_up(kda, T, strength):  # noqa: F811
    """No decay, queries along one channel that the keys do not cover, gradients of one sign: the
    state's gradient grows with every token, far past the largest that comes in."""
    gen = torch.Generator(device="cuda").manual_seed(412)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q = torch.zeros(1, T, 1, 128, device="cuda")
    q[..., 0] = 1.0
    k = n(1, T, 1, 128)
    k[..., 0] = 0.0
    k = (k / k.norm(dim=-1, keepdim=True)).bfloat16()
    v, g = n(1, T, 1, 128).bfloat16(), torch.zeros(1, T, 1, device="cuda")
    beta = strength * torch.sigmoid(n(1, T, 1))
    dout = (1 + 0.1 * n(1, T, 1, 128).abs()).bfloat16()
    S = n(1, 1, 128, 128)
    x = (q.bfloat16(), k, v, g, beta)
    r = back.run(kda, x, dout, S)
    near("d_initial_state", r["d_initial_state"][0, :, 0], dout.double().sum(1)[0] * SCALE)
    assert all(bool(r[m].isfinite().all()) for m in r)
    if T > 5000:
        return
    want = ref.rule_bwd(*(t[0] for t in x), SCALE, S[0], dout[0], torch.zeros(1, 128, 128, device="cuda"))
    for m, w in zip(("dq", "dv"), (want[0], want[2])):
        near(m, r[m][0], w, 2.0 ** -8)


@pytest.mark.gpu
def test_bwd_gradients_that_fade(kda):  # noqa: F811
    """Only the last tokens have a gradient, and decays of 2^-18 a chunk take it away on the way to
    the first.  Within such a chunk the rows of Y are that far apart: with the largest held at
    2^3 .. 2^4 and a spacing of 2^-24, its first rows are rounded to 2^-8, twice, and every chunk
    adds to it.  Held to 2^-5, down to 1e-18 of the largest."""
    q, k, v, g, beta, n = draw(1, 512, 1, 2, 413, decay=0.2)
    dout = n(1, 512, 2, 128)
    dout[:, :448] = 0
    x, dout = (q, k, v, g, beta), dout.bfloat16()
    r = back.run(kda, x, dout)
    want = ref.rule_bwd(*(t[0] for t in x), SCALE, torch.zeros(2, 128, 128, device="cuda"), dout[0],
                        torch.zeros(2, 128, 128, device="cuda"))
    for lo in range(192, 512, 64):
        for m, w in (("dv", want[2]), ("dk", want[1])):
            near((m, lo), r[m][0, lo:lo + 64], w[lo:lo + 64], 2.0 ** -8 if lo >= 384 else 2.0 ** -5)
