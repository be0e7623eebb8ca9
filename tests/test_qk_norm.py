"""kda_qk_norm and kda_qk_norm_bwd against the definition in 64 bits.

Tolerance: the kernels compute in fp32 and round once.  A result is off by a few fp32
roundings (2^-24 each; sums over at most 512 channels in a tree, so fewer than 16 of them in
a row) relative to the row's largest term, and by half a unit of its own type:
|y - ref| <= 2^-19 max|row of ref| + half a unit of ref (at most 2^-8 |ref| in bf16, which has
8 significant bits, and 2^-24 |ref| in fp32).
A weight's gradient is a sum over all rows in fp32: its error is held to 2^-18 times
the sum of its terms' magnitudes.
"""
import ctypes

import pytest

torch = pytest.importorskip("torch")
import rule_reference as ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_39_gb300 as kda
    kda.load_library()
    return kda


def _tables(rows, half, device="cuda"):
    angle = torch.arange(rows, device=device)[:, None] * 100.0 ** (-torch.arange(half, device=device) / max(half, 1))
    return angle.cos().float().contiguous(), angle.sin().float().contiguous()


def _close(got, want, typ):
    own = 2.0 ** -8 if typ == "bf16" else 2.0 ** -24
    limit = 2.0 ** -19 * want.abs().amax(-1, keepdim=True) + own * want.abs() + 1e-30
    off = (got.double() - want).abs()
    assert bool((off <= limit).all()), float((off / limit).max())


CASES = [
    # T, Hq, Hk, D, kind, rotary, interleaved, type
    (1, 1, 1, 128, "l2", 0, False, "bf16"),
    (5, 16, 2, 128, "rms", 128, False, "bf16"),
    (33, 3, 1, 64, "rms", 32, True, "f32"),
    (7, 5, 2, 256, "l2", 64, False, "f32"),
    (9, 2, 3, 96, "rms", 96, True, "bf16"),       # lanes that own no slot
    (11, 3, 1, 80, "rms", 20, False, "bf16"),     # half of the rotated part not a multiple of 8
    (4, 2, 2, 34, "l2", 6, True, "bf16"),         # rows that are not 16-byte aligned
    (3, 1, 1, 512, "rms", 512, False, "bf16"),
    (3, 2, 1, 512, "rms", 256, True, "f32"),
    (2, 1, 1, 510, "l2", 510, False, "f32"),
    (2, 3, 2, 2, "rms", 2, True, "f32"),
    (300, 40, 8, 128, "rms", 64, True, "bf16"),
]


def _inputs(case, seed=1):
    T, Hq, Hk, D, kind, rotary, inter, typ = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    packed = (n(T, Hq + Hk + 1, D) * 3).to(TYPES[typ])
    q, k = packed[:, :Hq], packed[:, Hq:Hq + Hk]
    x = {"norm": kind, "eps": 1e-5, "interleaved": inter}
    if kind == "rms":
        x |= {"q_weight": n(D), "k_weight": n(D)}
    if rotary:
        cos, sin = _tables(1000, rotary // 2)
        x |= {"cos": cos, "sin": sin,
              "positions": torch.randint(0, 1000, (T,), generator=gen, device="cuda", dtype=torch.int32)}
    return q, k, x, n


def _want(x, kw, which):
    pos = kw.get("positions")
    turn = {} if pos is None else {"cos": kw["cos"][pos.long()], "sin": kw["sin"][pos.long()],
                                   "interleaved": kw["interleaved"]}
    return dict(kind=kw["norm"], eps=kw["eps"], weight=kw.get(which + "_weight"), **turn)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_matches_definition(kda, case):
    q, k, kw, _ = _inputs(case)
    yq, yk = (torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda") for t in (q, k))
    kda.kda_qk_norm(q, k, yq, yk, **kw)
    _close(yq, ref.norm(q, **_want(q, kw, "q")), case[-1])
    _close(yk, ref.norm(k, **_want(k, kw, "k")), case[-1])
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_bwd_matches_definition(kda, case):
    q, k, kw, n = _inputs(case, 2)
    dzq, dzk = n(*q.shape).to(q.dtype), n(*k.shape).to(q.dtype)
    r = kda.kda_qk_norm_bwd(q, k, dzq, dzk, **kw)
    again = kda.kda_qk_norm_bwd(q, k, dzq, dzk, **kw)
    assert all(torch.equal(r[m], again[m]) for m in r)
    for which, x, dz in (("q", q, dzq), ("k", k, dzk)):
        w = _want(x, kw, which)
        dx, dw = ref.norm_bwd(x, dz, **w)
        # the two terms of dx may cancel: its error is relative to them
        term = (dz.double().abs().amax(-1, keepdim=True)
                * (1 if w["weight"] is None else w["weight"].double().abs().max())
                / (x.double().square().sum(-1, keepdim=True) / (x.shape[-1] if w["kind"] == "rms" else 1)
                   + w["eps"]).sqrt())
        own = 2.0 ** -8 if case[-1] == "bf16" else 2.0 ** -24
        off = (r["d" + which].double() - dx).abs()
        assert bool((off <= 2.0 ** -17 * term * x.shape[-1] ** 0.5 + own * dx.abs()).all())
        if w["weight"] is not None:
            terms = ref.norm_bwd(x, dz.abs(), **w)[1].abs() + ref.norm(x.abs(), w["kind"], w["eps"]).sum((0, 1)) * dz.double().abs().max()
            assert bool(((r[f"d{which}_weight"].double() - dw).abs() <= 2.0 ** -18 * terms).all())


def test_norm_bwd_formula_against_differences():
    """The 64-bit backward formula against central differences of the forward one (CPU)."""
    gen = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    for kind, rotary, inter in (("l2", 0, False), ("rms", 6, True), ("rms", 8, False)):
        x, w, dz = n(3, 2, 8), n(8), n(3, 2, 8)
        cos, sin = (None, None) if not rotary else (a[:3].double() for a in _tables(5, rotary // 2, "cpu"))
        f = lambda x, w: (ref.norm(x, kind, 1e-5, w, cos, sin, inter) * dz).sum()  # noqa: E731
        dx, dw = ref.norm_bwd(x, dz, kind, 1e-5, w, cos, sin, inter)
        ux, uw, h = n(3, 2, 8), n(8), 1e-6
        assert abs(float((f(x + h * ux, w) - f(x - h * ux, w)) / (2 * h) - (dx * ux).sum())) < 1e-7
        assert abs(float((f(x, w + h * uw) - f(x, w - h * uw)) / (2 * h) - (dw * uw).sum())) < 1e-7


@pytest.mark.gpu
def test_norm_in_place_empty_and_zero_rows(kda):
    x = torch.randn(6, 3, 128, device="cuda").bfloat16()
    x[2, 1] = 0
    q, k = x[:, :2].contiguous(), x[:, 2:].contiguous()
    want = ref.norm(q, "l2", 1e-6)
    kda.kda_qk_norm(q, k, q, k)
    _close(q, want, "bf16")
    assert bool((q[2, 1] == 0).all())
    e = torch.empty(0, 2, 128, device="cuda")
    kda.kda_qk_norm(e, e, torch.empty_like(e), torch.empty_like(e))
    w = torch.ones(128, device="cuda")
    r = kda.kda_qk_norm_bwd(e, e, e, e, q_weight=w, k_weight=w)
    assert bool((r["dq_weight"] == 0).all()) and bool((r["dk_weight"] == 0).all())


@pytest.mark.gpu
def test_norm_default_positions_batch_and_other_stream(kda):
    """[B, T, H, D] views, positions left out, on a stream that is not the current one."""
    x = torch.randn(2, 5, 6, 64, device="cuda")
    cos, sin = _tables(10, 16)
    q, k = x[:, :, :4], x[:, :, 4:]
    yq, yk = torch.empty(q.shape, device="cuda"), torch.empty(k.shape, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kda.kda_qk_norm(q, k, yq, yk, cos=cos, sin=sin, stream=s)
    s.synchronize()
    _close(yq, ref.norm(q.reshape(10, 4, 64), "l2", 1e-6, None, cos, sin).reshape(q.shape), "f32")


@pytest.mark.gpu
def test_norm_position_out_of_range(kda):
    """That token's rows are not written, the others are, and the error word says so."""
    x = torch.randn(4, 2, 64, device="cuda")
    cos, sin = _tables(8, 32)
    y = torch.full_like(x, 7.0)
    yk = torch.full_like(x, 7.0)
    pos = torch.tensor([1, 8, -1, 7], dtype=torch.int32, device="cuda")
    kda.kda_qk_norm(x, x, y, yk, cos=cos, sin=sin, positions=pos)
    assert kda.kda_fwd_get_error() == -16
    assert bool((y[1:3] == 7).all()) and bool((yk[1:3] == 7).all())
    good = torch.tensor([0, 3], device="cuda")
    _close(y[good], ref.norm(x[good], "l2", 1e-6, None, cos[pos.long()[good]], sin[pos.long()[good]]), "f32")


# ---- refusals (host side, no GPU) -------------------------------------------------------
def _c_call(name="kda_qk_norm", **over):
    from gated_delta_rule_39_gb300 import _build
    import gated_delta_rule_39_gb300 as kda
    _build.build()
    lib = kda.load_library()
    p = lambda i: ctypes.c_void_p(0x10000000 * (i + 1))  # noqa: E731
    a = dict(q=p(0), k=p(1), yq=p(2), yk=p(3), dx=p(8), dxk=p(9), dtype=0, norm=0, eps=1e-6, qw=None,
             kw=None, dqw=None, dkw=None, cos=p(4), sin=p(5), pos=p(6), rows=64, rotary=64, inter=0,
             T=4, Hq=2, Hk=1, D=64, qs=192, ks=192)
    a.update(over)
    mid = [a["dtype"], a["norm"], a["eps"], a["qw"], a["kw"]]
    end = [a[n] for n in ("cos", "sin", "pos", "rows", "rotary", "inter", "T", "Hq", "Hk", "D", "qs", "ks")]
    if name == "kda_qk_norm":
        return lib.kda_qk_norm(a["q"], a["k"], a["yq"], a["yk"], *mid, *end, None)
    return lib.kda_qk_norm_bwd(a["q"], a["k"], a["yq"], a["yk"], a["dx"], a["dxk"], *mid, a["dqw"], a["dkw"],
                               *end, None)


@pytest.mark.parametrize("name", ["kda_qk_norm", "kda_qk_norm_bwd"])
@pytest.mark.parametrize("over,status", [
    ({"D": 63, "rotary": 0}, -3), ({"D": 514, "rotary": 0, "qs": 2000, "ks": 2000}, -3), ({"D": 0, "rotary": 0}, -3),
    ({"T": -1}, -2), ({"Hq": 0}, -2), ({"Hk": -1}, -2), ({"qs": 127}, -2), ({"ks": 63}, -2),
    ({"pos": None, "rows": 3}, -2), ({"dtype": 2}, -5), ({"norm": 2}, -12), ({"eps": -1.0}, -12),
    ({"eps": float("nan")}, -12), ({"rotary": 3}, -12), ({"rotary": 66}, -12), ({"rotary": -2}, -12),
    ({"q": None}, -1), ({"yk": None}, -1), ({"cos": None}, -1), ({"q": ctypes.c_void_p(0x10000001)}, -4),
], ids=str)
def test_norm_refusals(name, over, status):
    assert _c_call(name, **over) == status


def test_norm_refuses_outputs_over_inputs():
    assert _c_call(yq=ctypes.c_void_p(0x20000000)) == -13
    assert _c_call(yq=ctypes.c_void_p(0x10000000)) == -13      # in place, but not contiguous
    assert _c_call(yk=ctypes.c_void_p(0x30000010)) == -13


def test_norm_bwd_refusals():
    w = ctypes.c_void_p(0xA0000000)
    assert _c_call("kda_qk_norm_bwd", qw=w) == -1
    assert _c_call("kda_qk_norm_bwd", dkw=w) == -1
    assert _c_call("kda_qk_norm_bwd", dx=ctypes.c_void_p(0x10000000)) == -13


def test_norm_binding_refusals():
    import gated_delta_rule_39_gb300 as kda
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_qk_norm(x, x, x, x)
