"""The norms with weights, angles and rows that begin anywhere: slices of larger buffers, a
multiple of 4 bytes (fp32) or of the element's size from a 16- or 32-byte boundary.  Every
combination has to give, bit for bit, what copies on a boundary of their own give where the
same accesses serve both, and the definition's values in any case."""
import pytest

torch = pytest.importorskip("torch")
import test_qk_norm as base  # noqa: E402
from test_qk_norm import kda, ref  # noqa: E402,F401  (the package, or a skip)


def at(t, offset):
    """A copy of t that begins `offset` elements after a 256-byte boundary."""
    room = torch.empty(t.numel() + 256, dtype=t.dtype, device=t.device)
    assert room.data_ptr() % 256 == 0
    y = room[offset:offset + t.numel()].view(t.shape)
    y.copy_(t)
    return y


# elements after the boundary: 4 bytes, 16 bytes (not 32), 32 bytes
OFFSETS = [1, 4, 8]
CASES = [(70, 5, 3, 128, "rms", 128, False, "bf16"), (70, 5, 3, 128, "rms", 64, True, "bf16"),
         (70, 5, 3, 128, "rms", 0, False, "bf16"), (9, 2, 1, 512, "rms", 256, False, "bf16"),
         (70, 5, 3, 128, "rms", 64, True, "f32")]


@pytest.mark.gpu
@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_weights_and_angles_anywhere(kda, case, offset):  # noqa: F811
    q, k, kw, n = base._inputs(case, 4)
    moved = {m: at(t, offset) if m in ("q_weight", "k_weight", "cos", "sin") else t for m, t in kw.items()}
    yq, yk = (torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda") for t in (q, k))
    kda.kda_qk_norm(q, k, yq, yk, **moved)
    base._close(yq, ref.norm(q, **base._want(q, kw, "q")), case[-1])
    base._close(yk, ref.norm(k, **base._want(k, kw, "k")), case[-1])
    dzq, dzk = n(*q.shape).to(q.dtype), n(*k.shape).to(q.dtype)
    got, want = (kda.kda_qk_norm_bwd(q, k, dzq, dzk, **x) for x in (moved, kw))
    own = 2.0 ** -7 if case[-1] == "bf16" else 2.0 ** -16     # of one row's terms, other orders of fp32 sums
    for m in want:
        if offset % 4 == 0:                                   # 16 bytes: the same accesses
            assert torch.equal(got[m], want[m]), m
        else:
            assert (got[m].double() - want[m].double()).norm() <= own * want[m].double().norm(), m
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("offset", OFFSETS)
def test_rows_anywhere(kda, offset):  # noqa: F811
    case = (70, 5, 3, 128, "rms", 64, False, "bf16")
    q, k, kw, n = base._inputs(case, 5)
    q, k = at(q.contiguous(), offset), at(k.contiguous(), offset)
    yq, yk = at(torch.zeros_like(q), offset), at(torch.zeros_like(k), offset)
    kda.kda_qk_norm(q, k, yq, yk, **kw)
    base._close(yq, ref.norm(q, **base._want(q, kw, "q")), "bf16")
    base._close(yk, ref.norm(k, **base._want(k, kw, "k")), "bf16")
    assert kda.kda_fwd_get_error() == 0


def test_no_access_is_wider_than_the_checked_alignment():
    """The units that rows, weights and angles are read in promise 16 bytes at most; the
    entry points ask for no more (a wider promise would let the compiler use 32-byte loads)."""
    import os
    import re
    import gated_delta_rule_39_gb300 as package
    path = os.path.join(os.path.dirname(package.__file__), "csrc", "kda_qknorm.cu")
    with open(path) as f:
        source = f.read()
    unit = re.search(r"struct __align__\((.*?)\) Unit \{", source).group(1)
    for size, vec in ((4, 8), (2, 8), (4, 4), (4, 1), (2, 1)):
        promised = eval(unit.replace("sizeof(T)", str(size)).replace("VEC", str(vec)).replace(" ? ", " and ").replace(" : ", " or "))
        assert promised <= 16
