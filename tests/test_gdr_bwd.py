"""kda_gdr_bwd (the backward pass of the delta rule with one decay per value head) against
the reversed token recurrence in 64 bits, and that formula against differences.

Tolerance: as for the prefill (parity.py), whose operands and sums have the same precision:
every gradient within 2e-2 of its RMS beyond half a bf16 unit at each element, and within
1e-2 in the Frobenius norm.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import rule_reference as ref  # noqa: E402
from parity import out_error  # noqa: E402
from test_gdr import SCALE, TYPES, draw, f64, kda  # noqa: E402,F401

NAMES = ("dq", "dk", "dv", "dg", "dbeta")


def run(kda, x, dout, init=None, dfinal=None, cu=None):
    q, k, v, g, beta = x
    r = kda.kda_gdr_bwd(q, k, v, g, beta, SCALE, dout, initial_state=init, d_final_state=dfinal, cu_seqlens=cu)
    again = kda.kda_gdr_bwd(q, k, v, g, beta, SCALE, dout, initial_state=init, d_final_state=dfinal, cu_seqlens=cu)
    assert all(torch.equal(r[n], again[n]) for n in r)
    assert kda.kda_fwd_get_error() == 0
    return r


def close(name, got, want):
    got, want = f64(got), f64(want)
    if want.size == 0:
        return
    e = out_error(got, want)
    assert e["ok"], (name, e)
    assert np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want), name


def check(r, x, dout, init, dfinal, spans):
    q, k, v, g, beta = x
    zero = torch.zeros(v.shape[2], 128, 128, device="cuda")
    want = {n: [] for n in NAMES + ("d_initial_state",)}
    for i, (b, lo, hi) in enumerate(spans):
        d = ref.rule_bwd(q[b, lo:hi], k[b, lo:hi], v[b, lo:hi], g[b, lo:hi], beta[b, lo:hi], SCALE,
                         zero if init is None else init[i], dout[b, lo:hi], zero if dfinal is None else dfinal[i])
        for n, y in zip(NAMES + ("d_initial_state",), d):
            want[n].append(y)
    for n in NAMES:
        close(n, torch.cat([r[n][b, lo:hi] for b, lo, hi in spans]), torch.cat(want[n]))
    if init is not None:
        close("d_initial_state", r["d_initial_state"], torch.stack(want["d_initial_state"]))


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hk,Hv", [(1, 1, 1, 1), (2, 17, 1, 3), (1, 64, 2, 2), (2, 65, 2, 4), (1, 200, 1, 2),
                                       (1, 700, 3, 3)])
@pytest.mark.parametrize("init,dfinal,gate", [(None, None, "f32"), ("f32", "f32", "f32"), ("bf16", "bf16", "bf16")])
def test_bwd_matches_definition(kda, B, T, Hk, Hv, init, dfinal, gate):  # noqa: F811
    *x, n = draw(B, T, Hk, Hv, 51 + T, gate, packed=True)
    dout = n(B, T, Hv, 128).bfloat16()
    S = None if init is None else (0.5 * n(B, Hv, 128, 128)).to(TYPES[init])
    dS = None if dfinal is None else (0.3 * n(B, Hv, 128, 128)).to(TYPES[dfinal])
    check(run(kda, x, dout, S, dS), x, dout, S, dS, [(b, 0, T) for b in range(B)])


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[0, 1, 64, 65, 0, 127, 3], [63, 1, 1, 300, 64]])
def test_bwd_packed_sequences(kda, lens):  # noqa: F811
    T, Hk, Hv = sum(lens), 2, 4
    *x, n = draw(1, T, Hk, Hv, 61, packed=True)
    dout, S, dS = n(1, T, Hv, 128).bfloat16(), 0.5 * n(len(lens), Hv, 128, 128), 0.3 * n(len(lens), Hv, 128, 128)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    ends = np.cumsum([0] + lens)
    r = run(kda, x, dout, S, dS, cu)
    check(r, x, dout, S, dS, [(0, int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])])


@pytest.mark.gpu
@pytest.mark.parametrize("decay,mean", [(0.0, 0.0), (0.01, 0.3), (0.3, 0.0), (3.0, 0.0)])
def test_bwd_decays_and_related_keys(kda, decay, mean):  # noqa: F811
    *x, n = draw(1, 400, 1, 2, 63, decay=decay, mean=mean)
    dout, S = n(1, 400, 2, 128).bfloat16(), 0.5 * n(1, 2, 128, 128)
    check(run(kda, x, dout, S), x, dout, S, None, [(0, 0, 400)])


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-30, 1e-7, 1e4, 1e30])
def test_bwd_gradients_of_any_size(kda, size):  # noqa: F811
    """Gradients far outside fp16's range: the results scale with them."""
    *x, n = draw(1, 130, 1, 2, 64, gate="bf16")
    dout = (size * n(1, 130, 2, 128)).bfloat16()
    dout[0, 40:80] = 0
    check(run(kda, x, dout), x, dout, None, None, [(0, 0, 130)])


@pytest.mark.gpu
def test_bwd_zero_gradients_and_extreme_gates(kda):  # noqa: F811
    *x, n = draw(1, 150, 1, 4, 65)
    q, k, v, g, beta = x
    zero = torch.zeros(1, 150, 4, 128, dtype=torch.bfloat16, device="cuda")
    r = run(kda, x, zero)
    assert all(bool((r[m] == 0).all()) for m in NAMES)
    g[0, 5, 0] = g[0, 64, 0] = -float("inf")
    g[0, 7, 1] = torch.finfo(torch.float32).min
    beta[0, ::3, 2] = 0.0
    g[0, :, 3], beta[0, :, 3] = 0.0, 1.0
    dout = n(1, 150, 4, 128).bfloat16()
    check(run(kda, x, dout), x, dout, None, None, [(0, 0, 150)])


@pytest.mark.gpu
def test_bwd_neighbours_do_not_leak(kda):  # noqa: F811
    *x, n = draw(1, 150, 1, 2, 66)
    dout = n(1, 150, 2, 128).bfloat16()
    cu = torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    r = run(kda, x, dout, cu=cu)
    y = [t.clone() for t in x] + [dout.clone()]
    for t in y:
        t[:, 70:] = float("nan")
        t[:, 71] = float("inf")
    bad = kda.kda_gdr_bwd(*y[:5], SCALE, y[5], cu_seqlens=cu)
    for m in NAMES:
        assert torch.equal(r[m][:, :70], bad[m][:, :70]), m


@pytest.mark.gpu
def test_bwd_no_tokens_malformed_offsets_and_other_stream(kda):  # noqa: F811
    *x, n = draw(1, 80, 1, 2, 67)
    dout, S, dS = n(1, 80, 2, 128).bfloat16(), n(1, 2, 128, 128), n(1, 2, 128, 128)
    e = [t[:, :0].contiguous() for t in x]
    r = kda.kda_gdr_bwd(*e, SCALE, dout[:, :0].contiguous(), initial_state=S, d_final_state=dS)
    assert torch.equal(r["d_initial_state"], dS)
    kda.kda_gdr_bwd(*x, SCALE, dout, cu_seqlens=torch.tensor([0, 81], dtype=torch.int32, device="cuda"))
    assert kda.kda_fwd_get_error() == -8
    want = run(kda, x, dout, S, dS)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.kda_gdr_bwd(*x, SCALE, dout, initial_state=S, d_final_state=dS, stream=s)
    s.synchronize()
    assert all(torch.equal(got[m], want[m]) for m in want)


def test_bwd_formula_against_differences():
    """The 64-bit reversed recurrence against central differences of the forward one (CPU)."""
    gen = torch.Generator().manual_seed(68)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    T, Hk, Hv, K = 9, 2, 4, 6
    x = [n(T, Hk, K) * 0.5, n(T, Hk, K) * 0.5, n(T, Hv, K), -n(T, Hv).abs(), torch.sigmoid(n(T, Hv)), n(Hv, K, K)]
    dout, dS = n(T, Hv, K), n(Hv, K, K)

    def loss(x):
        out, last, _ = ref.rule(*x[:5], 0.4, x[5])
        return (out * dout).sum() + (last * dS).sum()

    d = ref.rule_bwd(*x[:5], 0.4, x[5], dout, dS)
    for i in range(6):
        u, h = n(*x[i].shape), 1e-6
        up, down = ([y + s * h * u if j == i else y for j, y in enumerate(x)] for s in (1, -1))
        assert abs(float((loss(up) - loss(down)) / (2 * h) - (d[i] * u).sum())) < 1e-6, i


@pytest.mark.parametrize("over,status", [
    ({"K": 64}, -3), ({"B": 0}, -2), ({"T": -1}, -2), ({"Hv": 3, "Hk": 2}, -2), ({"cu": 9, "num": 1}, -2),
    ({"dout": None}, -1), ({"dq": None}, -1), ({"dbeta": None}, -1), ({"gate": 5}, -5), ({"df": 4}, -5),
    ({"di": 4}, -5), ({"scale": float("nan")}, -12), ({"dq": 0x100000008}, -4), ({"dg": 0x100000002}, -4),
    ({"dq": 0x10000000}, -13), ({"dk": 0xA0000000}, -13), ({"dinit": 0x70000000}, -13),
], ids=str)
def test_bwd_refusals(over, status):
    from gated_delta_rule_39_gb300 import _build
    import gated_delta_rule_39_gb300 as kda
    _build.build()
    p = [0x10000000 * (i + 1) for i in range(14)]
    a = dict(q=p[0], k=p[1], v=p[2], g=p[3], beta=p[4], gate=1, scale=0.1, s0=p[5], d0=1, dout=p[6], dfin=p[7],
             df=1, dq=p[9], dk=p[10], dv=p[11], dg=p[12], dbeta=p[13], dinit=p[8], di=1, cu=None, num=0, B=2, T=8,
             Hk=1, Hv=2, K=128, V=128, qs=128, ks=128, vs=256)
    a.update(over)
    wrap = lambda n, v: ctypes.c_void_p(v) if n in ("q", "k", "v", "g", "beta", "s0", "dout", "dfin", "dq", "dk", "dv", "dg", "dbeta", "dinit", "cu") else v  # noqa: E731
    assert kda.load_library().kda_gdr_bwd(*[wrap(n, v) for n, v in a.items()], None) == status


def test_bwd_workspace_bytes():
    import gated_delta_rule_39_gb300 as kda
    assert kda.kda_gdr_bwd_workspace_bytes(1, 0, 1, 1) < 4096
    per = kda.kda_gdr_bwd_workspace_bytes(1, 64000, 1, 2) / 128000
    assert 1850 < per < 2050
    assert kda.kda_gdr_bwd_workspace_bytes(1, 64, 1, 1, 7, True) >= 8 * 17680
