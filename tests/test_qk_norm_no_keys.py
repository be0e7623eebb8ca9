"""Queries alone (no key heads), with a weight for the keys all the same: both passes take it, and
its gradient, a sum over no rows, is zero."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
import test_qk_norm as base  # noqa: E402
from test_qk_norm import _c_call, kda, ref  # noqa: E402,F401


@pytest.mark.gpu
@pytest.mark.parametrize("typ,D", [("bf16", 128), ("f32", 64), ("bf16", 34)])
def test_no_keys(kda, typ, D):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(6)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k = n(50, 3, D).to(base.TYPES[typ]), n(50, 0, D).to(base.TYPES[typ])
    w, wk, dz = n(D), n(D), n(50, 3, D).to(base.TYPES[typ])
    y = torch.empty_like(q)
    kda.kda_qk_norm(q, k, y, torch.empty_like(k), norm="rms", q_weight=w, k_weight=wk)
    base._close(y, ref.norm(q, "rms", 1e-6, w), typ)
    r = kda.kda_qk_norm_bwd(q, k, dz, k, norm="rms", q_weight=w, k_weight=wk)
    alone = kda.kda_qk_norm_bwd(q, k, dz, k, norm="rms", q_weight=w)
    assert torch.equal(r["dq"], alone["dq"]) and torch.equal(r["dq_weight"], alone["dq_weight"])
    assert r["dk"].numel() == 0 and bool((r["dk_weight"] == 0).all())
    assert kda.kda_fwd_get_error() == 0


def test_a_weight_without_keys_is_not_refused_by_shape():
    w, dw = ctypes.c_void_p(0xA0000000), ctypes.c_void_p(0xB0000000)
    assert _c_call("kda_qk_norm_bwd", Hk=0, kw=w, dkw=dw) == _c_call("kda_qk_norm", Hk=0, kw=w) != -2
