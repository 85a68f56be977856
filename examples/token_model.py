"""A small token model trained by SGD on this package's kernels, end to end.

    z_t   = h_t + W_{e(t)} h_t,   h_t = s E[token_t]      (an expert per token)
    logit = U z_t

One step looks the tokens up, multiplies the rows by their experts, forms the logits, takes
a loss on the logits with its gradient, and goes back: gradients of U, of the experts and
of the rows, and the table's update straight from embed_grad (accumulate, scale -eta s).
Two losses train it: pairs of sequences (preference_loss) and sampled tokens with a reward
(policy_loss).  Weights are kept in FP32 and multiplied in BF16.

    python -m examples.token_model
"""
from __future__ import annotations

import math

import torch

import communication_avoiding_step_gb300 as casgd

BF16 = torch.bfloat16


class TokenModel:
    """Weights, and the buffers and workspaces for batches of `rows` tokens."""

    def __init__(self, vocab: int, dim: int, experts: int, rows: int, pairs: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device="cuda") * std

        def rows_of(n, dtype=BF16):
            return torch.empty(rows, n, device="cuda", dtype=dtype)

        self.vocab, self.experts, self.scale = vocab, experts, math.sqrt(dim)
        self.table = normal(vocab, dim, std=dim ** -0.5)            # E, FP32
        self.w32 = normal(experts, dim, dim, std=0.5 * dim ** -0.5)
        self.u32 = normal(1, vocab, dim, std=dim ** -0.5)
        self.w, self.u = self.w32.to(BF16), self.u32.to(BF16)
        self.h, self.x, self.y, self.dx = (rows_of(dim) for _ in range(4))
        self.logits = rows_of(vocab)
        self.dw, self.du = torch.empty_like(self.w), torch.empty_like(self.u)
        self.all_rows = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        self.ws_embed = casgd.embed_workspace(rows, vocab, dim)
        self.ws_experts = casgd.group_workspace(self.x, self.w, self.y)
        self.ws_logits = casgd.group_workspace(self.y, self.u, self.logits)
        self.ws_pref = casgd.preference_workspace(rows, pairs)
        self.ws_policy = casgd.policy_workspace(rows)
        self.pref, self.policy = casgd.PreferenceOut.alloc(pairs), casgd.PolicyOut.alloc(rows)

    def forward(self, tokens: torch.Tensor) -> torch.Tensor:
        """Logits of the batch (in a buffer that the next forward reuses)."""
        self.tokens = tokens
        expert = tokens % self.experts
        self.order = torch.argsort(expert, stable=True)             # rows by expert
        self.offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device="cuda")
        self.offsets[1:] = torch.cumsum(torch.bincount(expert, minlength=self.experts), 0)
        casgd.embed(self.table, tokens, self.h, self.ws_embed, scale=self.scale)
        torch.index_select(self.h, 0, self.order, out=self.x)
        casgd.group_product(self.x, self.w, self.offsets, self.y, self.ws_experts)
        self.z = self.h.index_add(0, self.order, self.y)
        return casgd.group_product(self.z, self.u, self.all_rows, self.logits, self.ws_logits)

    def backward(self, dlogits: torch.Tensor, eta: float) -> None:
        """One SGD step on every weight from the gradient of the logits."""
        casgd.group_product_dw(dlogits, self.z, self.all_rows, self.du, self.ws_logits)
        dz = torch.empty_like(self.z)
        casgd.group_product_dx(dlogits, self.u, self.all_rows, dz, self.ws_logits)
        dy = dz[self.order]
        casgd.group_product_dw(dy, self.x, self.offsets, self.dw, self.ws_experts)
        casgd.group_product_dx(dy, self.w, self.offsets, self.dx, self.ws_experts)
        dh = dz.index_add(0, self.order, self.dx)
        casgd.embed_grad(dh, self.tokens, self.table, self.ws_embed, scale=-eta * self.scale,
                         accumulate=True)
        for w32, w, dw in ((self.w32, self.w, self.dw), (self.u32, self.u, self.du)):
            w32.add_(dw, alpha=-eta)
            w.copy_(w32)

    def preference_step(self, tokens, targets, seq_offsets, ref_logp, eta: float,
                        beta: float = 0.1) -> torch.Tensor:
        """One step on pairs of sequences; returns the loss (before the step)."""
        x = self.forward(tokens)
        casgd.preference_loss(x, targets, seq_offsets, ref_logp, x, self.pref, self.ws_pref,
                              beta=beta)                            # the gradient in place
        self.backward(x, eta)
        return self.pref.loss.clone()

    def policy_step(self, tokens, targets, old_logp, ref_logp, reward, eta: float,
                    kl: float = 0.01) -> torch.Tensor:
        """One step on sampled tokens; returns the loss (before the step)."""
        x = self.forward(tokens)
        n = tokens.numel()
        casgd.policy_loss(x, targets, torch.full((n,), 1.0 / n, device="cuda"), old_logp, reward,
                          x, self.policy, self.ws_policy, ref_logp=ref_logp, kl=kl)
        self.backward(x, eta)
        return self.policy.stats[:1].clone()

    def check(self) -> None:
        """Raises if a kernel reported a bad token, target or offset.  Blocks."""
        for ws in (self.ws_embed, self.ws_experts, self.ws_logits, self.ws_pref, self.ws_policy):
            code = casgd.get_status(ws)
            if code:
                raise RuntimeError(f"device status {code}")


def train(steps: int = 30, vocab: int = 1000, dim: int = 128, experts: int = 4, pairs: int = 16,
          length: int = 24, eta: float = 0.5, policy_eta: float = 8.0):
    """Preference steps, then policy steps.  Returns the preference losses, the pairs'
    margins after them, and the mean rewards of the sampled tokens."""
    rows = 2 * pairs * length
    m = TokenModel(vocab, dim, experts, rows, pairs)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    chosen = (torch.arange(rows, device="cuda") // length) % 2 == 0
    # chosen sequences follow a rule, rejected ones do not; a few targets are masked
    targets = torch.where(chosen, (3 * tokens + 1) % vocab,
                          torch.randint(0, vocab, (rows,), generator=g, device="cuda"))
    targets[::11] = -100
    seq = torch.arange(0, rows + 1, length, dtype=torch.int32, device="cuda")
    out = casgd.preference_loss(m.forward(tokens), targets, seq,
                                torch.zeros(2 * pairs, device="cuda"), None, m.pref, m.ws_pref)
    ref = out.logp.clone()                                          # the start is the reference
    losses = [m.preference_step(tokens, targets, seq, ref, eta) for _ in range(steps)]
    margins = m.pref.margin.clone()

    rewards, ref_logits = [], m.forward(tokens).float()
    ref_all = torch.log_softmax(ref_logits, 1)
    for _ in range(steps):
        logp = torch.log_softmax(m.forward(tokens).float(), 1)
        drawn = torch.multinomial(logp.exp(), 1, generator=g)
        reward = torch.where(drawn[:, 0] % 2 == 0, 1.0, -1.0)       # even tokens are wanted
        rewards.append(reward.mean())
        m.policy_step(tokens, drawn[:, 0], logp.gather(1, drawn)[:, 0],
                      ref_all.gather(1, drawn)[:, 0], reward, policy_eta)
    m.check()
    return torch.cat(losses).tolist(), margins.tolist(), torch.stack(rewards).tolist()


if __name__ == "__main__":
    losses, margins, rewards = train()
    print(f"preference loss {losses[0]:.4f} -> {losses[-1]:.4f}, "
          f"margins {min(margins):.2f} .. {max(margins):.2f}")
    print(f"mean reward {rewards[0]:+.3f} -> {rewards[-1]:+.3f}")
