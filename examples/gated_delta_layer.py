"""A token mixing layer on the delta rule with one decay per head, from training to
speculative decoding: the package's operators as a small language model uses them.

    training    kda_qk_norm -> kda_gdr_fwd;  kda_gdr_bwd -> kda_qk_norm_bwd
    a prompt    kda_qk_norm -> kda_gdr_fwd, packed sequences, final states into a pool
    decoding    kda_qk_norm -> kda_gdr_step (outputs of drafted tokens, states untouched)
                -> kda_verify_drafts -> kda_gdr_step (states after the kept tokens)

Run:  python examples/gated_delta_layer.py
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_39_gb300 as kda

DIM = 128                          # channels of a head


class Mix(torch.autograd.Function):
    """Norm of queries and keys, then the rule, with their gradients."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, scale):
        qn, kn = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k))
        kda.kda_qk_norm(q, k, qn, kn)
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        kda.kda_gdr_fwd(qn, kn, v, g, beta, scale, out)
        ctx.save_for_backward(q, k, qn, kn, v, g, beta)
        ctx.scale = scale
        return out

    @staticmethod
    def backward(ctx, d_out):
        q, k, qn, kn, v, g, beta = ctx.saved_tensors
        r = kda.kda_gdr_bwd(qn, kn, v, g, beta, ctx.scale, d_out.contiguous())
        n = kda.kda_qk_norm_bwd(q, k, r["dq"], r["dk"])
        return n["dq"], n["dk"], r["dv"], r["dg"], r["dbeta"], None


class Model(torch.nn.Module):
    """Embedding, one mixing layer with Hv value heads on Hk query and key heads, output."""

    def __init__(self, vocab=384, width=256, Hk=2, Hv=4):
        super().__init__()
        self.Hk, self.Hv, self.scale = Hk, Hv, DIM ** -0.5
        self.embed = torch.nn.Parameter(0.5 * torch.randn(vocab, width))
        self.head = torch.nn.Linear(width, vocab, bias=False)
        self.qkv = torch.nn.Linear(width, (2 * Hk + Hv) * DIM, bias=False)
        self.gates = torch.nn.Linear(width, 2 * Hv)
        self.out = torch.nn.Linear(Hv * DIM, width, bias=False)

    def heads(self, x):
        """Queries, keys and values as views of one projection's buffer, log decays, strengths."""
        y = self.qkv(x).bfloat16()
        lead, Hk = y.shape[:-1], self.Hk
        q, k, v = (part.view(*lead, -1, DIM) for part in y.split([Hk * DIM, Hk * DIM, self.Hv * DIM], -1))
        a, b = self.gates(x).float().chunk(2, -1)
        return F.silu(q), F.silu(k), v, -F.softplus(a - 2).contiguous(), torch.sigmoid(b).contiguous()

    def logits(self, x, mixed):
        return self.head(x + self.out(mixed.flatten(-2).float()))

    def loss(self, tokens):        # [B, T + 1]
        x = self.embed[tokens[:, :-1]]
        mixed = Mix.apply(*self.heads(x), self.scale)
        return F.cross_entropy(self.logits(x, mixed).flatten(0, 1), tokens[:, 1:].flatten().long())

    # ---- serving ------------------------------------------------------------------------
    def normed(self, tokens):
        x = self.embed[tokens]
        q, k, v, g, beta = self.heads(x)
        qn, kn = torch.empty_like(q), torch.empty_like(k)
        kda.kda_qk_norm(q, k, qn, kn)
        return x, (qn, kn, v, g, beta, self.scale)

    @torch.no_grad()
    def prompt(self, tokens, cu_seqlens):
        """Packed prompts [1, T]: logits of all tokens, states [N, Hv, 128, 128]."""
        x, rule = self.normed(tokens)
        mixed = torch.empty(rule[2].shape, dtype=torch.bfloat16, device=x.device)
        states = torch.empty(cu_seqlens.numel() - 1, self.Hv, DIM, DIM, device=x.device)
        kda.kda_gdr_fwd(*rule, mixed, final_state=states, cu_seqlens=cu_seqlens)
        return self.logits(x, mixed), states

    def draft(self, last, count, generator):
        """`count` tokens per sequence from the model without its mixing layer."""
        tokens, probs = [last], []
        for _ in range(count):
            x = self.embed[tokens[-1]]
            probs.append(torch.softmax(self.head(x), -1))
            tokens.append(torch.multinomial(probs[-1], 1, generator=generator)[:, 0].int())
        return torch.stack(tokens, 1), torch.stack(probs, 1)

    @torch.no_grad()
    def decode(self, pool, slots, last, drafts, generator):
        """One round: drafts, verifies, and moves the states past the kept tokens.  Returns the
        tokens [N, drafts + 1] (-1 after each sequence's last) and the number of kept drafts."""
        N = last.numel()
        fed, draft_probs = self.draft(last, drafts, generator)
        x, rule = self.normed(fed)
        mixed = torch.empty(rule[2].shape, dtype=torch.bfloat16, device=x.device)
        kda.kda_gdr_step(*rule, out=mixed, state_in=pool, slots=slots)
        target = torch.softmax(self.logits(x, mixed), -1)
        uniform = torch.rand(N, drafts, device=x.device, generator=generator)
        noise = torch.empty(N, target.shape[-1], device=x.device).exponential_(generator=generator)
        accepted = torch.empty(N, dtype=torch.int32, device=x.device)
        tokens = torch.empty(N, drafts + 1, dtype=torch.int32, device=x.device)
        kda.kda_verify_drafts(target, draft_probs, fed[:, 1:].contiguous(), uniform, noise, accepted, tokens)
        kda.kda_gdr_step(*rule, state_in=pool, state_out=pool, slots=slots, lengths=accepted + 1)
        return tokens, accepted


def train(model, steps=30, B=4, T=300):
    """Losses of a few steps on chains whose next token mostly follows from the last one."""
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    gen = torch.Generator(device="cuda").manual_seed(1)
    vocab = model.embed.shape[0]
    follows = torch.randperm(vocab, device="cuda", generator=gen)
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, vocab, (B, T + 1), device="cuda", generator=gen)
        stray = torch.rand(B, T + 1, device="cuda", generator=gen) < 0.1
        for t in range(1, T + 1):
            tokens[:, t] = torch.where(stray[:, t], tokens[:, t], follows[tokens[:, t - 1]])
        loss = model.loss(tokens)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


def serve(model, lengths=(70, 1, 130), rounds=8, drafts=4):
    """Prompts of the given lengths, then some rounds of decoding; returns each sequence's tokens
    that its state has seen, the last token (not yet fed), and the states."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    prompts = [torch.randint(0, model.embed.shape[0], (n,), device="cuda", generator=gen, dtype=torch.int32) for n in lengths]
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    logits, states = model.prompt(torch.cat(prompts)[None], cu)
    pool = torch.zeros(len(lengths) + 2, *states.shape[1:], device="cuda")     # a pool with room to spare
    slots = torch.arange(len(lengths), device="cuda", dtype=torch.int32) + 1
    pool[slots.long()] = states
    last = logits[0, cu[1:].long() - 1].argmax(-1).int()
    seen, kept = [p.tolist() for p in prompts], 0
    for _ in range(rounds):
        tokens, accepted = model.decode(pool, slots, last, drafts, gen)
        kept += int(accepted.sum())
        for n, (row, a) in enumerate(zip(tokens.tolist(), accepted.tolist())):
            seen[n] += [int(last[n])] + row[:a]
        last = tokens.gather(1, accepted[:, None].long())[:, 0].contiguous()
    return seen, last, pool[slots.long()], kept / (rounds * len(lengths))


def main():
    torch.manual_seed(0)
    model = Model().cuda()
    losses = train(model)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps")
    seen, last, states, kept = serve(model)
    print(f"drafted tokens kept per round and sequence: {kept:.2f} of 4; tokens now: {[len(s) + 1 for s in seen]}")
    for n, s in enumerate(seen):   # the states are those of the tokens from the start
        t = torch.tensor(s, dtype=torch.int32, device="cuda")
        want = model.prompt(t[None], torch.tensor([0, len(s)], dtype=torch.int32, device="cuda"))[1][0]
        print(f"sequence {n}: state against one prompt of all its tokens: "
              f"{((states[n] - want).norm() / want.norm()).item():.1e}")
    kda.kda_fwd_get_error()


if __name__ == "__main__":
    main()
