"""Long calls on two streams that do not depend on each other: one that is held up does not hold
up the other, though both give part of their work to a second stream."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from test_gdr import kda  # noqa: E402,F401  (the package, or a skip)
from test_gdr_long import draw  # noqa: E402


def launches(kda, call):  # noqa: F811
    """Kernel launches of a call, by name."""
    lib = kda.load_library()
    n = kda.KDA_NUM_KERNELS
    lib.kda_profile_enable(1)
    try:
        call()
        torch.cuda.synchronize()
        ms, count = (ctypes.c_double * n)(), (ctypes.c_longlong * n)()
        assert lib.kda_profile_read(ms, count) == 0
    finally:
        lib.kda_profile_enable(0)
    return dict(zip(kda.KERNEL_NAMES, count))


@pytest.mark.gpu
@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("priorities", [(0, 0), (0, -1)], ids=str)
def test_a_held_stream_does_not_hold_another(kda, backward, priorities):  # noqa: F811
    T, H = 4224, 40 if not backward else 16                # in two parts: checked below
    x = draw(torch, T, H, H, torch.float32)
    d_out = torch.randn(1, T, H, 128, device="cuda").bfloat16()

    def call():
        if backward:
            return kda.kda_gdr_bwd(*x, 0.1, d_out)["dv"]
        out = torch.empty(1, T, H, 128, dtype=torch.bfloat16, device="cuda")
        kda.kda_gdr_fwd(*x, 0.1, out)
        return out

    count = launches(kda, call)
    assert count["gdr_prep_kernel" if not backward else "gdr_bwd_chunk_kernel"] == 2
    want = call()
    a, b = (torch.cuda.Stream(priority=p) for p in priorities)
    for s in (a, b):                                       # both have been used before
        with torch.cuda.stream(s):
            call()
    torch.cuda.synchronize()
    held = torch.cuda.Event()
    with torch.cuda.stream(a):
        torch.cuda._sleep(2_000_000_000)                   # about a second
        held.record()
        first = call()
    with torch.cuda.stream(b):
        second = call()
    b.synchronize()
    free = not held.query()
    torch.cuda.synchronize()
    assert torch.equal(first, want) and torch.equal(second, want)
    assert free, "the call on the second stream ended only after the first stream's hold"
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
def test_more_streams_than_are_remembered(kda):  # noqa: F811
    x = draw(torch, 4224, 40, 40, torch.float32)
    rt = ctypes.CDLL("libcudart.so.13")
    handles, outs = [ctypes.c_void_p() for _ in range(40)], []     # torch's own streams are only a few
    for h in handles:
        assert rt.cudaStreamCreateWithFlags(ctypes.byref(h), 1) == 0
    want = torch.empty(1, 4224, 40, 128, dtype=torch.bfloat16, device="cuda")
    kda.kda_gdr_fwd(*x, 0.1, want)
    torch.cuda.synchronize()
    for h in handles * 2:
        outs.append(torch.zeros_like(want))
        torch.cuda.synchronize()
        kda.kda_gdr_fwd(*x, 0.1, outs[-1], stream=h.value)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    for h in handles:
        assert rt.cudaStreamDestroy(h) == 0
    assert kda.kda_fwd_get_error() == 0
