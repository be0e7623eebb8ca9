"""kda_verify_drafts: every result is a whole number and has to equal the definition's.

The definition is computed here in numpy with the same two fp32 operations whose rounding
can matter (uniform times q, p minus q, and the IEEE quotient by the noise)."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_39_gb300 as kda
    kda.load_library()
    return kda


def definition(target, draft, tokens, uniform, noise, count=None):
    N, D1, V = target.shape
    accepted, result = np.zeros(N, np.int32), np.full((N, D1), -1, np.int32)

    def race(rest, e):
        with np.errstate(all="ignore"):
            score = np.where(rest > 0, rest / e, np.float32(0))
        score = np.where(score > 0, score, np.float32(0))
        return int(score.argmax()) if score.max(initial=0) > 0 else -1

    for n in range(N):
        c = D1 - 1 if count is None else int(count[n])
        a = 0
        while a < c:
            x = tokens[n, a]
            q = draft[n, a, x] if draft is not None else np.float32(1)
            if not uniform[n, a] * q < target[n, a, x]:
                break
            a += 1
        row = target[n, a]
        best = -1
        if a < c:
            q = np.eye(1, V, tokens[n, a], dtype=np.float32)[0] if draft is None else draft[n, a]
            best = race(row - q, noise[n])
        if best < 0:
            best = race(row, noise[n])
        accepted[n] = a
        result[n, :a] = tokens[n, :a]
        result[n, a] = best
    return accepted, result


def _draw(N, D, V, seed, near=0.7, sharp=2.0):
    r = np.random.default_rng(seed)

    def soft(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)

    base = sharp * r.standard_normal((N, D + 1, V))
    target = soft(base)
    draft = soft(base[:, :D] + near * r.standard_normal((N, D, V)))
    tokens = np.zeros((N, D), np.int32)
    for n in range(N):
        for i in range(D):
            p = draft[n, i].astype(np.float64)
            tokens[n, i] = r.choice(V, p=p / p.sum())
    return (target, draft, tokens, r.random((N, D), dtype=np.float32),
            r.exponential(size=(N, V)).astype(np.float32))


def _run(kda, target, draft, tokens, uniform, noise, count=None, typ=torch.float32):
    up = lambda a, t=None: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(t or torch.from_numpy(a).dtype)  # noqa: E731
    N, D1, _ = target.shape
    accepted = torch.full((N,), -9, dtype=torch.int32, device="cuda")
    result = torch.full((N, D1), -9, dtype=torch.int32, device="cuda")
    kda.kda_verify_drafts(up(target, typ), up(draft, typ), up(tokens), up(uniform), up(noise), accepted,
                          result, num_drafts=up(count))
    return accepted.cpu().numpy(), result.cpu().numpy()


def _check(kda, args, count=None):
    got, want = _run(kda, *args, count), definition(*args, count)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), (got, want)
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("N,D,V", [(1, 1, 1), (1, 4, 50257), (3, 0, 100), (5, 3, 2), (40, 7, 1023),
                                   (2, 33, 65), (300, 2, 4097), (2, 5, 131072)])
def test_verify_matches_definition(kda, N, D, V):
    args = _draw(N, D, V, seed=N + D + V)
    _check(kda, args)
    count = np.random.default_rng(V).integers(0, D + 1, N).astype(np.int32)
    _check(kda, args, count)


@pytest.mark.gpu
def test_verify_bf16(kda):
    """bf16 probabilities are widened exactly: the definition on the rounded values."""
    target, draft, tokens, uniform, noise = _draw(20, 4, 999, 5)
    rounded = [torch.from_numpy(a).bfloat16().float().numpy() for a in (target, draft)]
    got = _run(kda, target, draft, tokens, uniform, noise, typ=torch.bfloat16)
    want = definition(rounded[0], rounded[1], tokens, uniform, noise)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.gpu
def test_verify_all_kept_and_none_kept(kda):
    target, draft, tokens, uniform, noise = _draw(6, 3, 500, 6)
    draft = target[:, :3].copy()                       # q = p: everything is kept
    acc, _ = _check(kda, (target, draft, tokens, uniform, noise))
    assert (acc == 3).all()
    for i in range(3):                                 # the target rules every draft out
        target[np.arange(6), i, tokens[:, i]] = 0
    acc, _ = _check(kda, (target, draft, tokens, uniform * 0, noise))
    assert (acc == 0).all()


@pytest.mark.gpu
def test_verify_certain_drafts(kda):
    """draft_probs = None: a draft is kept with probability p, redrawn from the others."""
    target, _, tokens, uniform, noise = _draw(50, 3, 40, 7)
    tokens = target[:, :3].argmax(-1).astype(np.int32)
    acc, res = _check(kda, (target, None, tokens, uniform, noise))
    assert 0 < (acc > 0).sum() < 50
    for n in range(50):
        assert acc[n] == 3 or res[n, acc[n]] != tokens[n, acc[n]]


@pytest.mark.gpu
def test_verify_rows_with_nothing_left_ties_and_strange_values(kda):
    V = 70
    target, draft, tokens, uniform, noise = _draw(6, 1, V, 8)
    uniform[:] = 0.999999
    noise[:] = 1.0
    draft[0, 0] = target[0, 0] * 2                     # p nowhere above q: drawn from p itself
    target[1] = 0.0                                    # an empty row: -1
    target[2, 0] = 0.0
    target[2, 0, [9, 33, 69]] = 0.25                   # a tie: the lowest index
    draft[2, 0] = 0.0
    tokens[2, 0] = 1
    target[3, 0] = np.nan                              # not a number anywhere: nothing to draw
    target[4, 0, 5] = np.inf                           # wins whatever the noise
    draft[4, 0, tokens[4, 0]] = 1.0
    noise[5, 3] = 0.0                                  # and so does a zero in the noise
    draft[5, 0] = 0.0
    draft[5, 0, tokens[5, 0]] = 1.0
    want = _check(kda, (target, draft, tokens, uniform, noise))
    assert want[1][1, 0] == -1 and want[1][2, 0] == 9 and want[1][3, 0] == -1


@pytest.mark.gpu
def test_verify_draws_from_the_target(kda):
    """20,000 sequences with the same rows: the first token's frequencies are the target's
    (each within 5 standard deviations, and there are 12 of them)."""
    r = np.random.default_rng(9)
    V, N = 12, 20000
    p, q = (r.dirichlet(np.ones(V)).astype(np.float32) for _ in range(2))
    target = np.broadcast_to(p, (N, 2, V)).copy()
    draft = np.broadcast_to(q, (N, 1, V)).copy()
    tokens = r.choice(V, size=(N, 1), p=q.astype(np.float64) / q.astype(np.float64).sum()).astype(np.int32)
    _, res = _run(kda, target, draft, tokens, r.random((N, 1), dtype=np.float32),
                  r.exponential(size=(N, V)).astype(np.float32))
    freq = np.bincount(res[:, 0], minlength=V) / N
    assert (np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / N)).all()


@pytest.mark.gpu
def test_verify_indices_out_of_range(kda):
    args = list(_draw(4, 2, 30, 10))
    args[2][1, 0] = 30
    args[2][2, 1] = -1
    count = np.array([2, 2, 2, 3], np.int32)
    args[3][:] = 0                                     # keeps what it can
    got = _run(kda, *args, count)
    assert kda.kda_fwd_get_error() == -16
    want = definition(*(a[:1] for a in args), count[:1])
    assert np.array_equal(got[0][:1], want[0]) and np.array_equal(got[1][:1], want[1])
    assert (got[0][1:] == -9).all() and (got[1][1:] == -9).all()


@pytest.mark.parametrize("over,status", [
    ({"N": -1}, -2), ({"D": -1}, -2), ({"V": 0}, -2), ({"dtype": 3}, -5), ({"target": None}, -1),
    ({"uniform": None}, -1), ({"noise": None}, -1), ({"result": None}, -1),
    ({"target": ctypes.c_void_p(0x10000002)}, -4), ({"tokens": ctypes.c_void_p(0x30000002)}, -4),
    ({"accepted": ctypes.c_void_p(0x80000000)}, -13), ({"result": ctypes.c_void_p(0x10000000)}, -13),
], ids=str)
def test_verify_refusals(over, status):
    from gated_delta_rule_39_gb300 import _build
    import gated_delta_rule_39_gb300 as kda
    _build.build()
    p = lambda i: ctypes.c_void_p(0x10000000 * (i + 1))  # noqa: E731
    a = dict(target=p(0), draft=p(1), dtype=1, tokens=p(2), uniform=p(3), noise=p(4), count=None,
             accepted=p(6), result=p(7), N=4, D=3, V=100)
    a.update(over)
    assert kda.load_library().kda_verify_drafts(*a.values(), None) == status
