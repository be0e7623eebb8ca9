"""Gradients are allocated in the memory of the stream that writes them.  A block that the current
stream's allocator has free may still be in use by work queued there, and memory of a result
that is dropped early must not go back there while the other stream still writes it."""
import pytest

torch = pytest.importorskip("torch")


def calls(kda):
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16()  # noqa: E731
    q, k, v = unit(n(1, 640, 4, 128)), unit(n(1, 640, 4, 128)), n(1, 640, 4, 128).bfloat16()
    g, beta, dout = -n(1, 640, 4).abs(), torch.sigmoid(n(1, 640, 4)), n(1, 640, 4, 128).bfloat16()
    S = n(1, 4, 128, 128)
    w = n(128)
    gk, bk, A, bias = n(1, 640, 4, 128).bfloat16(), beta.bfloat16(), n(4), n(4, 128)
    return {
        "kda_gdr_bwd": lambda s: kda.kda_gdr_bwd(q, k, v, g, beta, 0.1, dout, initial_state=S, stream=s),
        "kda_qk_norm_bwd": lambda s: kda.kda_qk_norm_bwd(q, k, dout, dout, norm="rms", q_weight=w, k_weight=w, stream=s),
        "kda_bwd": lambda s: kda.kda_bwd(q, k, v, gk, bk, 0.1, A, bias, -5.0, dout, initial_state=S, stream=s)}


def spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors]


def apart(a, b):
    return all(x[1] <= y[0] or y[1] <= x[0] for x in a for y in b)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["kda_gdr_bwd", "kda_qk_norm_bwd", "kda_bwd"])
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_results_come_from_the_launching_streams_memory(name, handle):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_39_gb300 as kda
    call = calls(kda)[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # blocks of the results' sizes, freed on the current stream with work queued on them
    held = [torch.empty_like(t) for t in want.values()]
    free = spans(held)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)
    for t in held:
        t.fill_(float("nan"))
    del held, t
    got = call(side.cuda_stream if handle else side)
    assert apart(spans(got.values()), free), name
    side.synchronize()
    torch.cuda.synchronize()
    for m in want:
        assert torch.equal(got[m], want[m]), m
    # dropped at once: nothing that the current stream allocates may lie there
    got = call(side)
    there = spans(got.values())
    del got
    taken = [torch.empty_like(t) for t in want.values()]
    assert apart(spans(taken), there)
    torch.cuda.synchronize()
    assert kda.kda_fwd_get_error() == 0


@pytest.mark.gpu
def test_the_current_stream_needs_no_detour():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_39_gb300._operators import results_on
    dev, made = torch.device("cuda:0"), []

    def make():
        made.append(torch.cuda.current_stream(dev).cuda_stream)
        return {"x": torch.empty(8, device=dev)}

    side = torch.cuda.Stream()
    for s in (None, torch.cuda.current_stream(), side, side.cuda_stream, 0):
        results_on(s, dev, make)
    with torch.cuda.stream(side):
        results_on(torch.cuda.default_stream(), dev, make)
    main = torch.cuda.current_stream().cuda_stream
    assert made == [main, main, side.cuda_stream, side.cuda_stream, main, torch.cuda.default_stream().cuda_stream]
