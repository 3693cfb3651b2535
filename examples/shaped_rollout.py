"""A rollout and a training step of a policy that samples from shaped logits.

Requests bring their own low-rank adapter, penalties, biases, temperature and,
some of them, a grammar.  The rollout draws tokens from the shaped distribution
and keeps the shaped log-prob of each; the training step recomputes those
log-probs from the hidden states, forms the GSPO loss and takes its gradient
back to the raw logits.  Both sides shape with the same arithmetic, so before
the first update the ratio of the two policies is exactly 1.

    python examples/shaped_rollout.py

The "model" is a toy recurrence over token embeddings; the head and everything
after it is the library.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gspo_logprob_gb300 as g  # noqa: E402
from gspo_logprob_gb300 import ops  # noqa: E402


class Policy:
    def __init__(self, V=5000, D=256, adapters=3, rank=16, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen, device=device) * std).bfloat16()

        self.V, self.D = V, D
        self.embed = draw(V, D)
        self.W = draw(V, D, std=D ** -0.5)
        self.A = draw(adapters, rank, D, std=D ** -0.5)
        self.B = draw(adapters, V, rank, std=rank ** -0.5)
        self.scale = torch.ones(adapters, device=device)

    def step(self, h, token):
        return torch.tanh(0.5 * h.float() + self.embed[token].float()).bfloat16()

    def logits(self, H, adapter_id, status):
        return g.grpo_adapter_logits(H, self.W, self.A, self.B, self.scale, adapter_id, status=status)["logits"]


def request_shaping(requests, V, device, seed):
    """Per-request settings: what a server keeps for each request of a batch."""
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda lo, hi: lo + (hi - lo) * torch.rand(requests, generator=gen, device=device)  # noqa: E731
    few = torch.zeros((V + 31) // 32, dtype=torch.int32, device=device)
    few[:4] = -1                                          # a grammar that allows the first 128 tokens
    return dict(repetition=r(1.0, 1.3), presence=r(0.0, 0.4), frequency=r(0.0, 0.3), temperature=r(0.7, 1.1),
                bias_offsets=torch.tensor([0, 2], dtype=torch.int32, device=device),
                bias_tokens=torch.tensor([1, 7], dtype=torch.int32, device=device),
                bias_values=torch.tensor([-float("inf"), 1.5], device=device),   # token 1 is banned
                bias_set=(torch.arange(requests, device=device) % 2 - 1).to(torch.int32),
                allow_bits=few[None].contiguous(),
                allow_row=torch.where(torch.arange(requests, device=device) % 4 == 3, 0, -1).to(torch.int32))


def rollout(policy, prompts, settings, adapter_id, new_tokens, seed):
    """prompts [R, P] int32.  Returns tokens [R, P + new], hidden states of the sampled positions and their log-probs."""
    R, P = prompts.shape
    dev = prompts.device
    gen = torch.Generator(device=dev).manual_seed(seed)
    total = P + new_tokens
    tokens = torch.zeros(R, total, dtype=torch.int32, device=dev)
    tokens[:, :P] = prompts
    length = torch.full((R,), P, dtype=torch.int32, device=dev)
    # the histories live where the tokens are written: a step only raises `length`
    shaping = g.make_shaping(R, policy.V, tokens=tokens.view(-1),
                             hist_begin=torch.arange(R, device=dev, dtype=torch.int64) * total, hist_len=length,
                             prompt_len=torch.full((R,), P, dtype=torch.int32, device=dev), **settings)
    status = ops.new_status(dev)
    live = torch.ones(R, dtype=torch.uint8, device=dev)
    h = torch.zeros(R, policy.D, dtype=torch.bfloat16, device=dev)
    for t in range(P):
        h = policy.step(h, tokens[:, t].long())
    states, logps = [], []
    for t in range(P, total):
        states.append(h)
        z = policy.logits(h, adapter_id, status)
        shaped = g.grpo_shape_logits(z, shaping, out_dtype=torch.float32, status=status)["logits"]
        noise = -torch.log(-torch.log(torch.rand(shaped.shape, generator=gen, device=dev)))
        pick = (shaped + noise).argmax(1).to(torch.int32)          # a draw from softmax(shaped)
        logps.append(g.grpo_shaped_logp(z, pick, live, shaping, status=status)["logp"])
        tokens[:, t] = pick
        length += 1
        h = policy.step(h, pick.long())
    ops.raise_on_status(status)
    return tokens, torch.stack(states, 1), torch.stack(logps, 1)


def train_step(policy, tokens, P, states, old_logp, settings, adapter_id, advantages):
    """One GSPO step's loss, ratios and gradient with respect to the raw logits, over all sampled positions at once."""
    R, total = tokens.shape
    T = total - P
    n = R * T
    dev = tokens.device
    row = torch.arange(n, device=dev)
    seq, pos = row // T, P + row % T
    per_row = {k: (v[seq].contiguous() if v.shape[:1] == (R,) and k not in ("bias_tokens", "bias_values") else v)
               for k, v in settings.items()}
    shaping = g.make_shaping(n, policy.V, tokens=tokens.view(-1), hist_begin=seq * total,
                             hist_len=pos.to(torch.int32), prompt_len=torch.full((n,), P, dtype=torch.int32, device=dev),
                             **per_row)
    status = ops.new_status(dev)
    z = policy.logits(states.reshape(n, -1).contiguous(), adapter_id[seq].contiguous(), status)
    targets = tokens[:, P:].reshape(-1).contiguous()
    mask = torch.ones(n, dtype=torch.uint8, device=dev)
    f = g.grpo_shaped_logp(z, targets, mask, shaping, status=status)
    s = g.gspo_segment_loss(f["logp"], old_logp.reshape(-1).contiguous(), mask, seq.to(torch.int32), R, advantages,
                            eps_low=3e-4, eps_high=4e-4, divisor=float(R), status=status)
    b = g.grpo_shaped_logp_backward(z, targets, mask, shaping, f["lse"], s["coef"], status=status)
    ops.raise_on_status(status)
    return f["logp"].view(R, T), s, b["dlogits"]


def main(requests=8, prompt=12, new_tokens=24, V=5000):
    policy = Policy(V=V)
    dev = policy.W.device
    gen = torch.Generator(device=dev).manual_seed(5)
    prompts = torch.randint(0, V, (requests, prompt), generator=gen, device=dev, dtype=torch.int32)
    adapter_id = (torch.arange(requests, device=dev) % 4 - 1).to(torch.int32)
    settings = request_shaping(requests, V, dev, 6)
    tokens, states, old = rollout(policy, prompts, settings, adapter_id, new_tokens, 7)
    adv = g.grpo_group_advantage(torch.rand(requests, generator=gen, device=dev), requests // 2)
    logp, seam, dlogits = train_step(policy, tokens, prompt, states, old, settings, adapter_id, adv)
    print(f"{requests} requests x {new_tokens} tokens: mean log-prob {old.mean().item():.4f}, "
          f"largest |logp - old| {(logp - old).abs().max().item():.1e}, "
          f"ratios {seam['seg_ratio'].min().item():.6f} .. {seam['seg_ratio'].max().item():.6f}, "
          f"loss {seam['loss'].item():+.5f}, |dlogits| {dlogits.float().norm().item():.3e}")
    return tokens, old, logp, seam, dlogits, settings


if __name__ == "__main__":
    main()
