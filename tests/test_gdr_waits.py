"""The bounded waits of the gated delta rule's chunk chains, exercised without faulting
anything: in a variant of the library whose waits between warps give up at once
(-DKDA_WAIT_TRIES=0) every role leaves at its first hand-over, having waited for its own
copies and tensor-core operations.  The call must then report KDA_ERR_DEVICE_TIMEOUT
through the device error word, and the GPU must stay usable: a normal call right after it
gives what it gave before.
"""
import ctypes

import pytest

KDA_ERR_DEVICE_TIMEOUT = -7


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [None, [150, 0, 1, 64]])
@pytest.mark.parametrize("direction", ["forward", "backward"])
def test_waits_that_give_up_report_timeout_and_the_gpu_stays_usable(direction, lengths):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_39_gb300 as kda
    from gated_delta_rule_39_gb300 import _build
    kda.load_library()
    short = kda.declare(ctypes.CDLL(_build.build(lib="libkda_wait0.so", extra_flags=["-DKDA_WAIT_TRIES=0u"])))
    T, Hk, Hv = 215, 2, 4
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.nn.functional.normalize(torch.randn(1, T, Hk, 128, device="cuda", generator=gen), dim=-1).bfloat16()
            for _ in range(2))
    v, d_out = (torch.randn(1, T, Hv, 128, device="cuda", generator=gen).bfloat16() for _ in range(2))
    g = -torch.rand(1, T, Hv, device="cuda", generator=gen)
    beta = torch.rand(1, T, Hv, device="cuda", generator=gen)
    cu = None if lengths is None else torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")

    def run():
        if direction == "forward":
            out = torch.zeros(1, T, Hv, 128, dtype=torch.bfloat16, device="cuda")
            kda.kda_gdr_fwd(q, k, v, g, beta, 0.1, out, cu_seqlens=cu)
            return {"out": out}
        return kda.kda_gdr_bwd(q, k, v, g, beta, 0.1, d_out, cu_seqlens=cu)

    before = run()
    assert kda.kda_fwd_get_error() == 0
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    lib, kda._lib = kda._lib, short
    try:
        run()
        assert short.kda_fwd_get_error(stream) == KDA_ERR_DEVICE_TIMEOUT
        # the word is cleared by the read
        assert short.kda_fwd_get_error(stream) == 0
    finally:
        kda._lib = lib
    after = run()
    assert kda.kda_fwd_get_error() == 0
    for name, want in before.items():
        assert torch.equal(after[name], want), name
