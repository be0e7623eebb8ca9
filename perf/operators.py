"""Cases for the operators around the gated delta rule with one decay per head: the
norm and rotation of its queries and keys (forward and backward), the rule itself
(chunked forward, backward, and the step that applies a few new tokens to states in
memory), and the verification of drafted tokens.

Where ``own`` is false every operator is computed in its plain form, from elementary
torch operations in 32 bits, rounded once at the end; where it is true by the calls of
the package.  ``exact`` gives the same results from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DIM = 128      # key and value channels of a head in the delta rule
BLOCK = 64     # tokens per block of the plain chunked form
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a small batch: the norm alone, where the call's latency is all
        {"name": "norm_decode", "op": "norm", "tokens": 4, "hq": 16, "hk": 16, "dim": 128,
         "kind": "l2", "rot": 0, "inter": False, "type": "bf16"},
        # a long prompt of an attention layer with shared keys: weights and a full rotation
        {"name": "norm_prompt", "op": "norm", "tokens": 8192, "hq": 64, "hk": 8, "dim": 128,
         "kind": "rms", "rot": 128, "inter": False, "type": "bf16"},
        # training in 32 bits with odd sizes: half of each head rotated, neighbours as pairs
        {"name": "norm_bwd_odd", "op": "norm_bwd", "tokens": 1009, "hq": 12, "hk": 3, "dim": 64,
         "kind": "rms", "rot": 32, "inter": True, "type": "f32"},
        # a training batch of a delta-rule layer
        {"name": "norm_bwd_batch", "op": "norm_bwd", "tokens": 16384, "hq": 32, "hk": 32, "dim": 128,
         "kind": "l2", "rot": 0, "inter": False, "type": "bf16"},
        # several prompts of unequal length packed into one prefill, continued from states
        {"name": "rule_prompts", "op": "rule", "seqs": 9, "tokens": 2500, "hk": 16, "hv": 32,
         "init": "f32", "gate": "f32"},
        # the repository's headline size: one prompt of 8,192 tokens, 96 heads
        {"name": "rule_t8192_h96", "op": "rule", "seqs": 1, "tokens": 8192, "hk": 96, "hv": 96,
         "init": "bf16", "gate": "f32"},
        # fine-tuning on a few short samples packed together
        {"name": "rule_bwd_packed", "op": "rule_bwd", "seqs": 5, "tokens": 1300, "hk": 4, "hv": 8,
         "init": "none", "gate": "bf16"},
        # a training sequence, two value heads to a key head
        {"name": "rule_bwd_t4096", "op": "rule_bwd", "seqs": 1, "tokens": 4096, "hk": 16, "hv": 32,
         "init": "bf16", "gate": "bf16"},
        # a few sequences with five drafted tokens each: outputs for all of them, the state
        # after those that an earlier verification kept
        {"name": "step_drafts", "op": "step", "seqs": 16, "tokens": 5, "hk": 16, "hv": 32,
         "lengths": True, "state": "f32"},
        # one token for each of 256 sequences, 96 heads: the repository's decode step
        {"name": "step_n256_h96", "op": "step", "seqs": 256, "tokens": 1, "hk": 96, "hv": 96,
         "lengths": False, "state": "f32"},
        # one user, four drafted tokens, a vocabulary of odd size
        {"name": "verify_one", "op": "verify", "seqs": 1, "drafts": 4, "vocab": 50257,
         "ragged": False, "type": "f32"},
        # a batch of users, some with fewer drafts than others
        {"name": "verify_batch", "op": "verify", "seqs": 128, "drafts": 5, "vocab": 131072,
         "ragged": True, "type": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rule", "rule_bwd", "step", "verify"])
    if op in ("norm", "norm_bwd"):
        dim = rng.choice([64, 128, 256])
        hq, hk = rng.randint(1, 64), rng.randint(1, 32)
        top = 8192 * 72 * 128 if op == "norm" else 16384 * 64 * 128
        tokens = _log(rng, 1, min(20000, top // ((hq + hk) * dim)))
        rot = rng.choice([0, dim // 4, dim // 2, dim])
        return {"op": op, "tokens": tokens, "hq": hq, "hk": hk, "dim": dim,
                "kind": rng.choice(["l2", "rms"]), "rot": rot, "inter": rng.random() < 0.5,
                "type": rng.choice(["bf16", "bf16", "f32"])}
    if op in ("rule", "rule_bwd"):
        hk = _log(rng, 1, 32)
        hv = hk * rng.choice([1, 1, 2, 3])
        top = 8192 * 96 if op == "rule" else 4096 * 32
        tokens = _log(rng, 1, min(20000, top // hv))
        return {"op": op, "seqs": rng.randint(1, min(12, tokens)), "tokens": tokens, "hk": hk, "hv": hv,
                "init": rng.choice(["none", "bf16", "f32"]) if op == "rule" else rng.choice(["none", "bf16"]),
                "gate": rng.choice(["f32", "bf16"]) if op == "rule" else "bf16"}
    if op == "step":
        hk = _log(rng, 1, 96)
        hv = hk * rng.choice([1, 2]) if hk <= 48 else hk
        tokens = rng.randint(1, 8)
        return {"op": op, "seqs": _log(rng, 1, max(2, 256 * 96 // (hv * tokens))), "tokens": tokens,
                "hk": hk, "hv": hv, "lengths": rng.random() < 0.5, "state": rng.choice(["f32", "bf16"])}
    drafts, vocab = rng.randint(1, 8), _log(rng, 1000, 131072)
    return {"op": op, "seqs": _log(rng, 1, max(2, 128 * 6 * 131072 // (vocab * (drafts + 1)) // 4)),
            "drafts": drafts, "vocab": vocab, "ragged": rng.random() < 0.5,
            "type": rng.choice(["f32", "bf16"])}


def _lengths(case):
    """The lengths of a case's packed sequences: uneven ones that sum to its tokens."""
    n, total = case["seqs"], case["tokens"]
    r = random.Random(1000003 * total + n)
    cuts = sorted(r.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        size = 2 if case["type"] == "bf16" else 4
        n = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
        extra = case["tokens"] * (4 + 4 * case["rot"]) if case["rot"] else 0
        passes, ops = (2, 6) if op == "norm" else (3, 16)
        return {"bytes": passes * n * size + extra, "flops": ops * n}
    if op == "step":
        units = case["seqs"] * case["hv"]
        size = 4 if case["state"] == "f32" else 2
        tok = case["seqs"] * case["tokens"]
        return {"bytes": 2 * units * DIM * DIM * size + tok * (2 * case["hk"] + 2 * case["hv"]) * DIM * 2
                + tok * case["hv"] * 8, "flops": 7 * DIM * DIM * units * case["tokens"]}
    if op == "verify":
        size = 4 if case["type"] == "f32" else 2
        # the target's row and the noise; the draft's row is read only after a rejection
        return {"bytes": case["seqs"] * case["vocab"] * (size + 4), "flops": 2 * case["seqs"] * case["vocab"]}
    tok, gate = case["tokens"], 4 if case["gate"] == "f32" else 2
    states = {"none": 0, "bf16": 2, "f32": 4}[case["init"]]
    state = case["seqs"] * case["hv"] * DIM * DIM
    if op == "rule":
        return {"bytes": tok * (2 * case["hk"] + 2 * case["hv"]) * DIM * 2 + tok * case["hv"] * 2 * gate
                + state * (states + 2), "flops": 7 * DIM * DIM * tok * case["hv"]}
    return {"bytes": tok * (4 * case["hk"] + 3 * case["hv"]) * DIM * 2 + tok * case["hv"] * 4 * gate
            + state * (2 * states + 2), "flops": 18 * DIM * DIM * tok * case["hv"]}


# ---- inputs --------------------------------------------------------------------------
def _unit(x):
    return x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()


def _rule_inputs(gen, tok, hk, hv, gate):
    """Queries and keys as a layer has them (an activation with a positive mean, then unit
    length), values in a buffer that holds other things too, decays of short and long
    memory by head, write strengths around a half."""
    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    silu = torch.nn.functional.silu
    q = _unit(silu(normal(*tok, hk, DIM))).bfloat16()
    k = _unit(silu(normal(*tok, hk, DIM))).bfloat16()
    v = normal(*tok, hk + hv, DIM).bfloat16()[..., hk:, :]
    rate = torch.rand(hv, generator=gen, device="cuda") * 15 + 1
    dt = torch.exp(torch.rand(hv, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
    bias = dt + torch.log(-torch.expm1(-dt))
    g = (-rate * torch.nn.functional.softplus(normal(*tok, hv) + bias)).to(TYPES[gate])
    beta = torch.sigmoid(normal(*tok, hv)).to(TYPES[gate])
    return q, k, v, g, beta


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    op, s = case["op"], {"case": case}
    if op in ("norm", "norm_bwd"):
        t, hq, hk, d, typ = case["tokens"], case["hq"], case["hk"], case["dim"], TYPES[case["type"]]
        # queries and keys as views of the buffer that one projection writes: q, k and v
        packed = (normal(t, hq + 2 * hk, d) * torch.exp(normal(t, 1, 1))).to(typ)
        s["q"], s["k"] = packed[:, :hq], packed[:, hq:hq + hk]
        s["qw"] = s["kw"] = s["cos"] = s["sin"] = s["pos"] = None
        if case["kind"] == "rms":
            s["qw"], s["kw"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        if case["rot"]:
            rows = max(4096, t)
            freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda") / case["rot"])
            angle = torch.arange(rows, device="cuda")[:, None] * freq
            s["cos"], s["sin"] = angle.cos(), angle.sin()
            s["pos"] = torch.randint(0, rows, (t,), generator=gen, device="cuda", dtype=torch.int32)
        if op == "norm":
            s["yq"] = torch.empty(t, hq, d, dtype=typ, device="cuda")
            s["yk"] = torch.empty(t, hk, d, dtype=typ, device="cuda")
        else:
            s["dq"], s["dk"] = normal(t, hq, d).to(typ), normal(t, hk, d).to(typ)
    elif op in ("rule", "rule_bwd"):
        t, hk, hv = case["tokens"], case["hk"], case["hv"]
        s["q"], s["k"], s["v"], s["g"], s["beta"] = _rule_inputs(gen, (1, t), hk, hv, case["gate"])
        s["lengths"] = _lengths(case)
        ends = torch.tensor([0] + s["lengths"]).cumsum(0)
        s["cu"] = ends.to(torch.int32).cuda() if case["seqs"] > 1 else None
        n = case["seqs"]
        s["init"] = None
        if case["init"] != "none":
            s["init"] = (0.02 * normal(n, hv, DIM, DIM)).to(TYPES[case["init"]])
        if op == "rule":
            s["out"] = torch.empty(1, t, hv, DIM, dtype=torch.bfloat16, device="cuda")
            s["final"] = torch.empty(n, hv, DIM, DIM, dtype=torch.bfloat16, device="cuda")
        else:
            s["dout"] = normal(1, t, hv, DIM).bfloat16()
            s["dfinal"] = (0.1 * normal(n, hv, DIM, DIM)).bfloat16()
    elif op == "step":
        n, t, hk, hv = case["seqs"], case["tokens"], case["hk"], case["hv"]
        s["q"], s["k"], s["v"], s["g"], s["beta"] = _rule_inputs(gen, (n, t), hk, hv, "f32")
        s["state"] = (0.3 * normal(n, hv, DIM, DIM)).to(TYPES[case["state"]])
        s["state_out"] = torch.empty_like(s["state"])
        s["out"] = torch.empty(n, t, hv, DIM, dtype=torch.bfloat16, device="cuda")
        s["slots"] = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
        s["keep"] = None
        if case["lengths"]:
            s["keep"] = torch.randint(0, t + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    else:
        n, d, v, typ = case["seqs"], case["drafts"], case["vocab"], TYPES[case["type"]]

        def race(p):
            return (p / torch.empty(p.shape, device="cuda").exponential_(generator=gen)).argmax(-1)

        logits = 3.0 * normal(n, d + 1, v)
        draft = torch.softmax(logits[:, :d] + 0.7 * normal(n, d, v), -1)
        target = torch.softmax(logits, -1)
        del logits
        # a sampler's filter: what is less than a thousandth of the likeliest is struck out
        target = torch.where(target >= 1e-3 * target.amax(-1, keepdim=True), target, 0.0)
        s["target"] = (target / target.sum(-1, keepdim=True)).to(typ)
        del target
        s["draft"] = draft.to(typ)
        s["tokens"] = torch.stack([race(draft[:, i]) for i in range(d)], 1).to(torch.int32)
        s["uniform"] = torch.rand(n, d, generator=gen, device="cuda")
        s["noise"] = torch.empty(n, v, device="cuda").exponential_(generator=gen)
        s["count"] = None
        if case["ragged"]:
            s["count"] = torch.randint(0, d + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
        s["accepted"] = torch.empty(n, dtype=torch.int32, device="cuda")
        s["result"] = torch.empty(n, d + 1, dtype=torch.int32, device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    return (OWN if own else PLAIN)[op](state)


def _own_norm(s):
    import gated_delta_rule_39_gb300 as kda
    c = s["case"]
    kda.kda_qk_norm(s["q"], s["k"], s["yq"], s["yk"], norm=c["kind"], eps=1e-6, q_weight=s["qw"],
                    k_weight=s["kw"], cos=s["cos"], sin=s["sin"], positions=s["pos"],
                    interleaved=c["inter"])
    return s["yq"], s["yk"]


def _own_norm_bwd(s):
    import gated_delta_rule_39_gb300 as kda
    c = s["case"]
    r = kda.kda_qk_norm_bwd(s["q"], s["k"], s["dq"], s["dk"], norm=c["kind"], eps=1e-6,
                            q_weight=s["qw"], k_weight=s["kw"], cos=s["cos"], sin=s["sin"],
                            positions=s["pos"], interleaved=c["inter"])
    return [r[n] for n in ("dq", "dk", "dq_weight", "dk_weight") if n in r]


def _own_rule(s):
    import gated_delta_rule_39_gb300 as kda
    kda.kda_gdr_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], DIM ** -0.5, s["out"],
                    initial_state=s["init"], final_state=s["final"], cu_seqlens=s["cu"])
    return s["out"], s["final"]


def _own_rule_bwd(s):
    import gated_delta_rule_39_gb300 as kda
    r = kda.kda_gdr_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], DIM ** -0.5, s["dout"],
                        initial_state=s["init"], d_final_state=s["dfinal"], cu_seqlens=s["cu"])
    return [r[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state") if n in r]


def _own_step(s):
    import gated_delta_rule_39_gb300 as kda
    kda.kda_gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], DIM ** -0.5, out=s["out"],
                     state_in=s["state"], state_out=s["state_out"], slots=s["slots"],
                     lengths=s["keep"])
    return s["out"], s["state_out"]


def _own_verify(s):
    import gated_delta_rule_39_gb300 as kda
    kda.kda_verify_drafts(s["target"], s["draft"], s["tokens"], s["uniform"], s["noise"],
                          s["accepted"], s["result"], num_drafts=s["count"])
    return s["accepted"], s["result"]


# ---- plain forms ---------------------------------------------------------------------
def _turn(x, cos, sin, inter, back):
    """The leading channels of x [t, h, d] turned by each token's angles (or back)."""
    half = cos.shape[-1]
    cos, sin = cos[:, None], -sin[:, None] if back else sin[:, None]
    if inter:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_norm(s):
    c = s["case"]

    def one(x, w):
        x = x.float()
        squares = x.square()
        total = squares.mean(-1, keepdim=True) if c["kind"] == "rms" else squares.sum(-1, keepdim=True)
        y = x / (total + 1e-6).sqrt()
        y = y if w is None else y * w
        if c["rot"]:
            y = _turn(y, s["cos"][s["pos"].long()], s["sin"][s["pos"].long()], c["inter"], False)
        return y.to(TYPES[c["type"]])

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _plain_norm_bwd(s):
    c = s["case"]

    def one(x, dy, w):
        x, dy = x.float(), dy.float()
        if c["rot"]:
            dy = _turn(dy, s["cos"][s["pos"].long()], s["sin"][s["pos"].long()], c["inter"], True)
        share = 1.0 / c["dim"] if c["kind"] == "rms" else 1.0
        r = 1.0 / (share * x.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        dw = None if w is None else (dy * x * r).sum((0, 1))
        du = dy if w is None else dy * w
        dx = r * (du - x * (share * r * r * (x * du).sum(-1, keepdim=True)))
        return dx.to(TYPES[c["type"]]), dw

    (dq, dqw), (dk, dkw) = one(s["q"], s["dq"], s["qw"]), one(s["k"], s["dk"], s["kw"])
    return [x for x in (dq, dk, dqw, dkw) if x is not None]


def _unit_lower_inverse(a):
    """(I + a)^-1 for strictly lower a [..., 64, 64], from the inverses of its diagonal
    blocks of 1, 2, 4 .. tokens, two joined at a time."""
    d = torch.ones(a.shape[:-2] + (a.shape[-1], 1, 1), device=a.device, dtype=a.dtype)
    while d.shape[-1] < a.shape[-1]:
        m, n = d.shape[-1], d.shape[-3] // 2
        low = a.unflatten(-1, (n, 2 * m)).unflatten(-3, (n, 2 * m)).diagonal(dim1=-4, dim2=-2)
        low = low.movedim(-1, -3)[..., m:, :m]
        first, second = d[..., 0::2, :, :], d[..., 1::2, :, :]
        corner = -(second @ low @ first)
        d = torch.cat([torch.cat([first, torch.zeros_like(first)], -1),
                       torch.cat([corner, second], -1)], -2)
    return d.squeeze(-3)


def _rule(q, k, v, g, beta, state, lengths):
    """The chunked rule in 32 bits on [t, h, 128] rows of packed sequences (g, beta [t, h];
    state [n, h, 128, 128]); outputs [t, h, 128] and the last states."""
    n, width = len(lengths), max(1, -(-max(lengths) // BLOCK)) * BLOCK
    rows = torch.arange(width, device=q.device) < torch.tensor(lengths, device=q.device)[:, None]
    share = v.shape[1] // k.shape[1]

    def pad(x):   # [t, h, ...] -> [n, h, blocks, 64, ...], zeros after each sequence's end
        y = x.new_zeros((n, width) + x.shape[1:])
        y = y.masked_scatter(rows.reshape((n, width) + (1,) * (x.dim() - 1)), x)
        return y.unflatten(1, (-1, BLOCK)).movedim(3, 1)

    q, k = pad(q).repeat_interleave(share, 1), pad(k).repeat_interleave(share, 1)
    v, total, beta = pad(v), pad(g).cumsum(-1), pad(beta)
    lower = torch.ones(BLOCK, BLOCK, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((total[..., :, None] - total[..., None, :]).masked_fill(~lower, -torch.inf))
    solve = _unit_lower_inverse((beta[..., None] * decay * (k @ k.mT)).tril(-1))
    inside = decay * (q @ k.mT)
    begin, end = torch.exp(total)[..., None], torch.exp(total[..., -1:] - total)[..., None]
    outs = []
    for c in range(width // BLOCK):
        new = solve[:, :, c] @ (beta[:, :, c, :, None] * (v[:, :, c] - begin[:, :, c] * (k[:, :, c] @ state)))
        outs.append(DIM ** -0.5 * (begin[:, :, c] * (q[:, :, c] @ state) + inside[:, :, c] @ new))
        state = begin[:, :, c, -1:] * state + (end[:, :, c] * k[:, :, c]).mT @ new
    out = torch.stack(outs, 2).movedim(1, 3).flatten(1, 2)
    return out[rows], state


def _start(s):
    hv = s["case"]["hv"]
    if s["init"] is not None:
        return s["init"].float()
    return torch.zeros(s["case"]["seqs"], hv, DIM, DIM, device="cuda")


def _plain_rule(s):
    x = [s[n][0].float() for n in ("q", "k", "v", "g", "beta")]
    out, state = _rule(*x, _start(s), s["lengths"])
    return out[None].bfloat16(), state.bfloat16()


def _plain_rule_bwd(s):
    x = [s[n][0].float().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
    x.append(_start(s).requires_grad_())
    with torch.enable_grad():
        out, state = _rule(*x, s["lengths"])
        d = torch.autograd.grad([out, state], x, [s["dout"][0].float(), s["dfinal"].float()])
    grads = [y[None].to(s[n].dtype) for y, n in zip(d, ("q", "k", "v", "g", "beta"))]
    return grads + ([] if s["init"] is None else [d[5].to(s["init"].dtype)])


def _plain_step(s):
    share = s["case"]["hv"] // s["case"]["hk"]
    q, k = (s[n].float().repeat_interleave(share, 2) for n in ("q", "k"))
    v, decay, beta = s["v"].float(), s["g"].exp(), s["beta"]
    at = s["slots"].long()
    state = s["state"][at].float()
    t = s["case"]["tokens"]
    keep = s["keep"].long() if s["keep"] is not None else torch.full_like(at, t)
    kept, outs = state, []
    for i in range(t):
        state = decay[:, i, :, None, None] * state
        delta = beta[:, i, :, None] * (v[:, i] - (k[:, i, :, :, None] * state).sum(-2))
        state = state + k[:, i, :, :, None] * delta[:, :, None]
        outs.append(DIM ** -0.5 * (q[:, i, :, :, None] * state).sum(-2))
        kept = torch.where((keep > i)[:, None, None, None], state, kept)
    s["state_out"][at] = kept.to(s["state"].dtype)
    return torch.stack(outs, 1).bfloat16(), s["state_out"]


def _plain_verify(s):
    n, d = s["case"]["seqs"], s["case"]["drafts"]
    rows, steps = torch.arange(n, device="cuda"), torch.arange(d, device="cuda")
    token = s["tokens"].long()
    count = s["count"].long() if s["count"] is not None else torch.full_like(rows, d)
    p = s["target"][rows[:, None], steps, token].float()
    q = s["draft"][rows[:, None], steps, token].float()
    good = (s["uniform"] * q < p) & (steps < count[:, None])
    accepted = good.long().cumprod(1).sum(1)
    row = s["target"][rows, accepted].float()
    drafted = s["draft"][rows, accepted.clamp(max=d - 1)].float()
    rest = torch.where((accepted < count)[:, None], row - drafted, row).clamp(min=0)
    rest = torch.where(rest.amax(1, keepdim=True) > 0, rest, row)
    last = (rest / s["noise"]).argmax(1)
    places = torch.arange(d + 1, device="cuda")
    longer = torch.cat([token, torch.zeros_like(rows)[:, None]], 1)
    result = torch.where(places < accepted[:, None], longer, -1)
    result = torch.where(places == accepted[:, None], last[:, None], result)
    return accepted.to(torch.int32), result.to(torch.int32)


OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "rule": _own_rule, "rule_bwd": _own_rule_bwd,
       "step": _own_step, "verify": _own_verify}
PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "rule": _plain_rule,
         "rule_bwd": _plain_rule_bwd, "step": _plain_step, "verify": _plain_verify}


# ---- the definitions in 64 bits ------------------------------------------------------
def _exact_turn(s, x, back):
    """x [t, h, d] with its pairs of channels, as complex numbers, times e^(i angle)."""
    c = s["case"]
    if not c["rot"]:
        return x
    half = c["rot"] // 2
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + half)
    at = s["pos"].long()
    angle = torch.complex(s["cos"].double()[at], s["sin"].double()[at])[:, None]
    z = torch.complex(x[..., a], x[..., b]) * (angle.conj() if back else angle)
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_norm(s, backward):
    c = s["case"]
    outs, weights = [], []
    scale = c["dim"] if c["kind"] == "rms" else 1
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].double()
        root = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / scale + 1e-6)
        unit = x / root
        weight = torch.ones(c["dim"], dtype=torch.float64, device="cuda") if w is None else w.double()
        if not backward:
            outs.append(_exact_turn(s, unit * weight, False))
            continue
        dz = _exact_turn(s, s["d" + name].double(), True)
        weights += [] if w is None else [torch.einsum("thc,thc->c", dz, unit)]
        du = dz * weight
        outs.append(du / root - x * (x * du).sum(-1, keepdim=True) / (scale * root ** 3))
    return tuple(outs + weights)


def _exact_tokens(s, names):
    """A packed case's inputs as [n, longest, h, ...] in 64 bits, with zeros after a
    sequence's end (a zero key, strength and log decay leave the state as it is)."""
    c = s["case"]
    there = torch.arange(max(s["lengths"]), device="cuda") < torch.tensor(s["lengths"], device="cuda")[:, None]
    x = {}
    for name in names:
        y = s[name][0].double()
        if name in "qk":
            y = y.repeat_interleave(c["hv"] // c["hk"], 1)
        x[name] = torch.zeros(there.shape + y.shape[1:], dtype=torch.float64, device="cuda")
        x[name][there] = y
    return x, there


def _exact_token(S, k, v, a, b):
    """One token of the rule on states [n, h, 128, 128]."""
    held = S * a[..., None, None]
    read = torch.einsum("nhkv,nhk->nhv", held, k)
    return torch.baddbmm(held.flatten(0, 1), k.flatten(0, 1)[:, :, None],
                         (b[..., None] * (v - read)).flatten(0, 1)[:, None]).view_as(S)


def _exact_rule(s):
    x, there = _exact_tokens(s, ("q", "k", "v", "g", "beta"))
    S, out = _start(s).double(), torch.zeros_like(x["v"])
    for t in range(there.shape[1]):
        S = _exact_token(S, x["k"][:, t], x["v"][:, t], x["g"][:, t].exp(), x["beta"][:, t])
        out[:, t] = DIM ** -0.5 * torch.einsum("nhkv,nhk->nhv", S, x["q"][:, t])
    return out[there][None], S


def _exact_rule_bwd(s):
    c, span = s["case"], 64
    x, there = _exact_tokens(s, ("q", "k", "v", "g", "beta", "dout"))
    length = there.shape[1]
    S, saved = _start(s).double(), []

    def after(S, t):
        return _exact_token(S, x["k"][:, t], x["v"][:, t], x["g"][:, t].exp(), x["beta"][:, t])

    for t in range(length):
        if t % span == 0:
            saved.append(S)
        S = after(S, t)
    d = {n: torch.zeros_like(x[n]) for n in ("q", "k", "v", "g", "beta")}
    dS = s["dfinal"].double()
    for block in reversed(range(len(saved))):
        states = [saved[block]]
        last = min(length, (block + 1) * span)
        for t in range(block * span, last):
            states.append(after(states[-1], t))
        for t in reversed(range(block * span, last)):
            q, k, v, b, a, do = (x["q"][:, t], x["k"][:, t], x["v"][:, t], x["beta"][:, t],
                                 x["g"][:, t].exp(), x["dout"][:, t])
            old, new = states[t - block * span], states[t - block * span + 1]
            held = old * a[..., None, None]
            miss = v - torch.einsum("nhkv,nhk->nhv", held, k)
            D = dS + DIM ** -0.5 * q[..., None] * do[..., None, :]
            ddelta = torch.einsum("nhkv,nhk->nhv", D, k)
            dread = -b[..., None] * ddelta
            dheld = D + k[..., None] * dread[..., None, :]
            d["q"][:, t] = DIM ** -0.5 * torch.einsum("nhkv,nhv->nhk", new, do)
            d["k"][:, t] = (torch.einsum("nhkv,nhv->nhk", D, b[..., None] * miss)
                            + torch.einsum("nhkv,nhv->nhk", held, dread))
            d["v"][:, t] = b[..., None] * ddelta
            d["beta"][:, t] = (ddelta * miss).sum(-1)
            d["g"][:, t] = a * (dheld * old).sum((-2, -1))
            dS = a[..., None, None] * dheld
    grads = [d[n][there] for n in ("q", "k", "v", "g", "beta")]
    grads[:2] = [y.unflatten(1, (c["hk"], c["hv"] // c["hk"])).sum(2) for y in grads[:2]]
    return [y[None] for y in grads] + ([] if s["init"] is None else [dS])


def _exact_step(s):
    c = s["case"]
    t, share, at = c["tokens"], c["hv"] // c["hk"], s["slots"].long()
    S = s["state"].double()[at]
    k, q = (s[m].double().repeat_interleave(share, 2) for m in ("k", "q"))
    out, kept = torch.empty(s["v"].shape, dtype=torch.float64, device="cuda"), S.clone()
    for i in range(t):
        S = _exact_token(S, k[:, i], s["v"][:, i].double(), s["g"][:, i].double().exp(),
                         s["beta"][:, i].double())
        out[:, i] = DIM ** -0.5 * torch.einsum("nhkv,nhk->nhv", S, q[:, i])
        here = torch.ones_like(at) * t == i + 1 if s["keep"] is None else s["keep"] == i + 1
        kept[here] = S[here]
    final = torch.empty_like(kept)
    final[at] = kept
    return out, final


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return None   # whole numbers: the plain form's are the answer
    if op in ("norm", "norm_bwd"):
        return _exact_norm(s, op == "norm_bwd")
    return {"rule": _exact_rule, "rule_bwd": _exact_rule_bwd, "step": _exact_step}[op](s)
