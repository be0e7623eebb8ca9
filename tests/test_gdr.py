"""kda_gdr_fwd and kda_gdr_step (the delta rule with one decay per value head) against the
definition in 64 bits, token by token.

Tolerances.  kda_gdr_step computes in fp32: a state element is off by a few roundings per
token, so ||S - ref||_F <= 1e-6 sqrt(tokens + 1) ||ref||_F for fp32 states (2^-9 for bf16
ones), and the output by its own rounding and 1e-5 RMS.  kda_gdr_fwd has the package's
bounds for a prefill (parity.py): 2e-2 RMS beyond half a unit for outputs, 1e-2 in the
Frobenius norm for states.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import rule_reference as ref  # noqa: E402
from parity import bf16_half_ulp, out_error, state_error  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_39_gb300 as kda
    kda.load_library()
    return kda


def draw(B, T, Hk, Hv, seed, gate="f32", decay=0.3, packed=False, mean=0.0):
    """Inputs on the GPU: unit queries and keys (with a common part `mean`), decays up to
    2 * decay a token, strengths in (0, 1); packed: q, k, v as views of one buffer."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    common = mean * n(128)
    x = torch.cat([unit(n(B, T, 2 * Hk, 128) + common), n(B, T, Hv, 128)], 2).bfloat16()
    q, k, v = x[:, :, :Hk], x[:, :, Hk:2 * Hk], x[:, :, 2 * Hk:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    g = (-2 * decay * torch.rand(B, T, Hv, generator=gen, device="cuda")).to(TYPES[gate])
    beta = torch.sigmoid(n(B, T, Hv)).to(TYPES[gate])
    return q, k, v, g, beta, n


def f64(t):
    return t.detach().double().cpu().numpy()


def check_out(out, want):
    """fp32 arithmetic: half a unit of bf16 and 1e-5 of the tensor's size."""
    out, want = f64(out), f64(want)
    if want.size:
        rms = np.sqrt(np.mean(want ** 2))
        assert np.max(np.abs(out - want) - bf16_half_ulp(want) * 1.001) <= 1e-5 * rms


def check_state(S, want, tokens):
    own = 2.0 ** -9 if S.dtype == torch.bfloat16 else 0.0
    off = (S.double() - want).norm() / want.norm().clamp(min=1e-30)
    assert float(off) <= 1e-6 * (tokens + 1) ** 0.5 + own, float(off)


# ---- kda_gdr_step ---------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("N,T,Hk,Hv", [(1, 1, 1, 1), (3, 1, 2, 6), (2, 5, 3, 3), (7, 8, 1, 4), (1, 40, 2, 2)])
@pytest.mark.parametrize("typ,gate", [("f32", "f32"), ("bf16", "bf16")])
def test_step_matches_definition(kda, N, T, Hk, Hv, typ, gate):
    q, k, v, g, beta, n = draw(N, T, Hk, Hv, 11 * N + T, gate, packed=True)
    S = n(N, Hv, 128, 128).to(TYPES[typ])
    So = torch.full_like(S, float("nan"))
    out = torch.full(v.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    kda.kda_gdr_step(q, k, v, g, beta, SCALE, out=out, state_in=S, state_out=So)
    only = S.clone()
    kda.kda_gdr_step(q, k, v, g, beta, SCALE, state_in=only, state_out=only)   # in place, no outputs
    assert torch.equal(only, So)
    for i in range(N):
        o, last, _ = ref.rule(q[i], k[i], v[i], g[i], beta[i], SCALE, S[i])
        check_out(out[i], o)
        check_state(So[i], last, T)


@pytest.mark.gpu
def test_step_slots_and_lengths(kda):
    """States of a pool that is larger than the batch, in any order; a padding entry; the
    state after 0, some and all of the tokens; untouched slots stay as they are."""
    N, T, H = 6, 4, 2
    q, k, v, g, beta, n = draw(N, T, H, H, 21)
    pool = n(9, H, 128, 128)
    slots = torch.tensor([7, 0, -1, 3, 8, 2], dtype=torch.int32, device="cuda")
    keep = torch.tensor([0, 4, 2, 1, 3, 4], dtype=torch.int32, device="cuda")
    out = torch.full(v.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    after = pool.clone()
    kda.kda_gdr_step(q, k, v, g, beta, SCALE, out=out, state_in=pool, state_out=after, slots=slots, lengths=keep)
    advance = pool.clone()
    kda.kda_gdr_step(q, k, v, g, beta, SCALE, state_in=advance, state_out=advance, slots=slots, lengths=keep)
    assert torch.equal(after, advance)
    for s in (1, 4, 5, 6, 7):
        assert torch.equal(after[s], pool[s])
    assert bool((out[2] == 9).all())
    for i in (0, 1, 3, 4, 5):
        s, m = int(slots[i]), int(keep[i])
        check_out(out[i], ref.rule(q[i], k[i], v[i], g[i], beta[i], SCALE, pool[s])[0])
        check_state(after[s], ref.rule(q[i][:m], k[i][:m], v[i][:m], g[i][:m], beta[i][:m], SCALE, pool[s])[1], m)
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
def test_step_zero_state_no_tokens_and_extreme_gates(kda):
    q, k, v, g, beta, n = draw(2, 3, 1, 2, 22)
    g[:, 1] = -float("inf")                    # forgets everything before the second token
    g[0, 2], beta[1, 2] = 0.0, 0.0
    out = torch.empty(v.shape, dtype=torch.bfloat16, device="cuda")
    So = torch.empty(2, 2, 128, 128, device="cuda")
    kda.kda_gdr_step(q, k, v, g, beta, SCALE, out=out, state_out=So)
    zero = torch.zeros(2, 128, 128, device="cuda")
    for i in range(2):
        o, last, _ = ref.rule(q[i], k[i], v[i], g[i], beta[i], SCALE, zero)
        check_out(out[i], o)
        check_state(So[i], last, 3)
    S = n(2, 2, 128, 128)
    e = [x[:, :0] for x in (q, k, v, g, beta)]
    kda.kda_gdr_step(*[x.contiguous() for x in e], SCALE, state_in=S, state_out=So)
    assert torch.equal(S, So)
    e = [x[:0] for x in (q, k, v, g, beta)]
    kda.kda_gdr_step(*e, SCALE, state_in=S[:0], state_out=So[:0])


@pytest.mark.gpu
def test_step_indices_out_of_range(kda):
    q, k, v, g, beta, n = draw(4, 2, 1, 1, 23)
    S = n(4, 1, 128, 128)
    So, out = torch.full_like(S, 5.0), torch.full(v.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 4, -2, 3], dtype=torch.int32, device="cuda")
    keep = torch.tensor([2, 2, 2, 3], dtype=torch.int32, device="cuda")
    kda.kda_gdr_step(q, k, v, g, beta, SCALE, out=out, state_in=S, state_out=So, slots=slots, lengths=keep)
    assert kda.kda_fwd_get_error() == -16
    assert bool((out[1:] == 5).all()) and bool((So[1:] == 5).all()) and not bool((So[0] == 5).any())


@pytest.mark.gpu
def test_step_state_offsets_past_32_bits(kda):
    """A pool of bf16 states of more than 2^32 elements; the last slot."""
    H, pool = 4, 65537
    S = torch.zeros(pool, H, 128, 128, dtype=torch.bfloat16, device="cuda")
    q, k, v, g, beta, n = draw(1, 1, H, H, 24)
    S[-1] = n(H, 128, 128).bfloat16()
    before = S[-1].clone()
    out = torch.empty(v.shape, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([pool - 1], dtype=torch.int32, device="cuda")
    kda.kda_gdr_step(q, k, v, g, beta, SCALE, out=out, state_in=S, state_out=S, slots=slots)
    o, last, _ = ref.rule(q[0], k[0], v[0], g[0], beta[0], SCALE, before)
    check_out(out[0], o)
    check_state(S[-1], last, 1)
    assert bool((S[0] == 0).all()) and bool((S[-2] == 0).all())


# ---- kda_gdr_fwd ----------------------------------------------------------------------
def run_fwd(kda, x, init, final, cu=None, N=None):
    q, k, v, g, beta = x
    out = torch.full(v.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    fs = None
    if final is not None:
        fs = torch.full((N or q.shape[0], v.shape[2], 128, 128), float("nan"), dtype=TYPES[final], device="cuda")
    kda.kda_gdr_fwd(q, k, v, g, beta, SCALE, out, initial_state=init, final_state=fs, cu_seqlens=cu)
    return out, fs


def check_fwd(x, init, out, fs, spans):
    """spans: (batch, first token, last token + 1) of each sequence."""
    q, k, v, g, beta = x
    outs, wants, states = [], [], []
    for i, (b, lo, hi) in enumerate(spans):
        S = init[i] if init is not None else torch.zeros(v.shape[2], 128, 128, device="cuda")
        o, last, _ = ref.rule(q[b, lo:hi], k[b, lo:hi], v[b, lo:hi], g[b, lo:hi], beta[b, lo:hi], SCALE, S)
        outs.append(f64(out[b, lo:hi]))
        wants.append(f64(o))
        states.append(last)
    e = out_error(np.concatenate(outs), np.concatenate(wants))
    assert e["ok"], e
    if fs is not None:
        se = state_error(f64(fs), f64(torch.stack(states)))
        assert se["ok"], se


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hk,Hv", [(1, 1, 1, 1), (2, 15, 1, 2), (1, 63, 2, 2), (3, 64, 1, 3), (1, 65, 2, 4),
                                       (2, 130, 3, 3), (1, 200, 5, 10), (1, 1000, 1, 1)])
@pytest.mark.parametrize("init,final,gate", [(None, "f32", "f32"), ("f32", "bf16", "f32"), ("bf16", "f32", "bf16"),
                                             ("f32", None, "bf16")])
def test_fwd_matches_definition(kda, B, T, Hk, Hv, init, final, gate):
    *x, n = draw(B, T, Hk, Hv, 31 + T, gate, packed=True)
    S = None if init is None else (0.5 * n(B, Hv, 128, 128)).to(TYPES[init])
    out, fs = run_fwd(kda, x, S, final)
    check_fwd(x, S, out, fs, [(b, 0, T) for b in range(B)])
    again, fs2 = run_fwd(kda, x, S, final)
    assert torch.equal(out, again) and (fs is None or torch.equal(fs, fs2))


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[0, 1, 64, 65, 0, 127, 3], [200], [0, 0], [63, 1, 1, 300, 64], [5] * 40])
def test_fwd_packed_sequences(kda, lens):
    T, Hk, Hv = sum(lens), 2, 4
    *x, n = draw(1, T, Hk, Hv, 41, packed=True)
    S = 0.5 * n(len(lens), Hv, 128, 128)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    out, fs = run_fwd(kda, x, S, "f32", cu, len(lens))
    ends = np.cumsum([0] + lens)
    check_fwd(x, S, out, fs, [(0, int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])])
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
def test_fwd_neighbours_do_not_leak(kda):
    """A sequence next to one that is full of infinities and NaN keeps its results."""
    *x, _ = draw(1, 150, 1, 2, 42)
    cu = torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    out, fs = run_fwd(kda, x, None, "f32", cu, 2)
    y = [t.clone() for t in x]
    for t in y:
        t[:, 70:] = float("nan")
        t[:, 71] = float("inf")
    bad, bs = run_fwd(kda, y, None, "f32", cu, 2)
    assert torch.equal(out[:, :70], bad[:, :70]) and torch.equal(fs[0], bs[0])


@pytest.mark.gpu
@pytest.mark.parametrize("decay,mean", [(0.0, 0.0), (0.001, 0.7), (0.05, 0.3), (3.0, 0.0), (40.0, 0.0)])
def test_fwd_decays_and_related_keys(kda, decay, mean):
    *x, n = draw(1, 400, 1, 2, 43, decay=decay, mean=mean)
    S = 0.5 * n(1, 2, 128, 128)
    out, fs = run_fwd(kda, x, S, "f32")
    check_fwd(x, S, out, fs, [(0, 0, 400)])


@pytest.mark.gpu
def test_fwd_extreme_gates(kda):
    """Log decays of -inf and of the type's lowest value, strengths of 0, 1 and 2, one key
    throughout with strengths that alternate."""
    *x, n = draw(1, 200, 1, 4, 44)
    q, k, v, g, beta = x
    g[0, 5, 0] = g[0, 64, 0] = g[0, 100:103, 0] = -float("inf")
    g[0, 7, 1] = g[0, 130, 1] = torch.finfo(torch.float32).min
    beta[0, :, 2] = torch.arange(200, device="cuda") % 3
    beta[0, 50:, 3] = 0.0
    g[0, 50:, 3] = 0.0
    S = 0.5 * n(1, 4, 128, 128)
    out, fs = run_fwd(kda, x, S, "f32")
    check_fwd(x, S, out, fs, [(0, 0, 200)])


@pytest.mark.gpu
def test_fwd_state_carried_between_calls(kda):
    *x, n = draw(1, 333, 2, 2, 45)
    out, fs = run_fwd(kda, x, None, "f32")
    S = None
    parts = []
    for lo, hi in ((0, 100), (100, 101), (101, 333)):
        y = [t[:, lo:hi] for t in x[:3]] + [t[:, lo:hi].contiguous() for t in x[3:]]
        o, S = run_fwd(kda, y, S, "f32")
        parts.append(o)
    e = out_error(f64(torch.cat(parts, 1)), f64(out))
    assert e["ok"] and state_error(f64(S), f64(fs))["ok"]


@pytest.mark.gpu
def test_fwd_no_tokens_and_malformed_offsets(kda):
    *x, n = draw(2, 8, 1, 1, 46)
    S = n(2, 1, 128, 128)
    e = [t[:, :0].contiguous() for t in x]
    out, fs = run_fwd(kda, e, S, "f32")
    assert torch.equal(fs, S)
    y = [t[:1] for t in x]
    for cu in ([0, 9], [1, 8], [0, 5, 4, 8], [0, -1, 8]):
        t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, fs = run_fwd(kda, y, None, "f32", t, len(cu) - 1)
        assert kda.kda_fwd_get_error() == -8
        assert bool(out.isnan().all()) and bool(fs.isnan().all())


@pytest.mark.gpu
def test_fwd_on_another_stream(kda):
    *x, _ = draw(1, 256, 2, 4, 47)
    want, _ = run_fwd(kda, x, None, None)
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kda.kda_gdr_fwd(*x, SCALE, out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


# ---- refusals (host side, no GPU) -------------------------------------------------------
def _lib():
    from gated_delta_rule_39_gb300 import _build
    import gated_delta_rule_39_gb300 as kda
    _build.build()
    return kda.load_library()


def _p(i):
    return ctypes.c_void_p(0x10000000 * (i + 1))


def _rule_call(name, **over):
    a = dict(q=_p(0), k=_p(1), v=_p(2), g=_p(3), beta=_p(4), gate=1, scale=0.1, out=_p(5), s0=_p(6), d0=1,
             s1=_p(7), d1=1, slots=None, pool=0, lengths=None, cu=None, num=0, B=2, T=8, Hk=1, Hv=2, K=128,
             V=128, qs=128, ks=128, vs=256)
    a.update(over)
    front = [a[n] for n in ("q", "k", "v", "g", "beta", "gate", "scale", "out", "s0", "d0", "s1", "d1")]
    mid = [a["slots"], a["pool"], a["lengths"]] if name == "kda_gdr_step" else [a["cu"], a["num"]]
    end = [a[n] for n in ("B", "T", "Hk", "Hv", "K", "V", "qs", "ks", "vs")]
    return getattr(_lib(), name)(*front, *mid, *end, None)


@pytest.mark.parametrize("name", ["kda_gdr_fwd", "kda_gdr_step"])
@pytest.mark.parametrize("over,status", [
    ({"K": 64}, -3), ({"V": 256}, -3), ({"B": -1}, -2), ({"T": -1}, -2), ({"Hk": 0}, -2), ({"Hv": 0}, -2),
    ({"Hk": 2, "Hv": 3, "qs": 256, "ks": 256, "vs": 384}, -2), ({"qs": 120}, -2), ({"vs": 128}, -2),
    ({"qs": 132}, -4), ({"vs": 260}, -4), ({"q": None}, -1), ({"beta": None}, -1), ({"gate": 2}, -5),
    ({"d0": 3}, -5), ({"d1": -1}, -5), ({"scale": float("inf")}, -12), ({"k": ctypes.c_void_p(0x10000008)}, -4),
    ({"g": ctypes.c_void_p(0x10000002)}, -4), ({"out": ctypes.c_void_p(0x60000008)}, -4),
    ({"out": _p(2)}, -13), ({"s1": _p(5)}, -13), ({"s1": _p(6), "d1": 0}, -13),
    ({"T": 1 << 30, "B": 2}, -2),
], ids=str)
def test_rule_refusals(name, over, status):
    assert _rule_call(name, **over) == status


def test_fwd_and_step_refusals():
    assert _rule_call("kda_gdr_fwd", B=0) == -2
    assert _rule_call("kda_gdr_fwd", cu=_p(9), num=1) == -2            # packed sequences with B = 2
    assert _rule_call("kda_gdr_fwd", cu=_p(9), num=0, B=1) == -2
    assert _rule_call("kda_gdr_fwd", out=None) == -1
    assert _rule_call("kda_gdr_step", slots=_p(9), pool=0) == -2
    assert _rule_call("kda_gdr_step", lengths=ctypes.c_void_p(0x90000002)) == -4


def test_rule_binding_refusals():
    import gated_delta_rule_39_gb300 as kda
    from gated_delta_rule_39_gb300 import _operators as ops
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_gdr_fwd(x, x, x, x[..., 0], x[..., 0], 1.0, x)
    with pytest.raises(ValueError, match="equally spaced"):
        ops._token_stride(x.transpose(2, 3), "q")
    with pytest.raises(ValueError, match="equally spaced"):
        ops._token_stride(torch.zeros(3, 4, 2, 128)[:, :3], "q")
    assert ops._token_stride(torch.zeros(3, 4, 6, 128)[:, :, 1:3], "q") == 768
    assert ops._token_stride(torch.zeros(3, 1, 6, 128)[:, :, 1:3], "q") == 768
