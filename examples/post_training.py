"""Post-training steps on one GPU, from logits to updated weights.

A small next-token model is trained first on a policy loss (sampled tokens,
a reward of 1 for the right one), then on a preference loss (right against
random continuations).  Two logical data-parallel ranks each bring a batch;
two owners hold the fp32 weights and 8-bit moments of their half of the
parameters, check, clip and step, and write the fp16 weights back:

    logits -> zero_token_logprobs (sampling policy, reference)
           -> zero_policy_loss / zero_preference_loss (loss, dlogits x loss scale)
           -> logits.backward(dlogits) -> each rank's flat gradient
           -> OwnerShard8.reduce_and_check -> zero_step_decision -> apply_update

Run: python examples/post_training.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

VOCAB, DIM, RANKS, SCALE = 96, 128, 2, 256.0
SHAPES = [(VOCAB, DIM), (DIM, 4 * DIM), (4 * DIM, DIM), (DIM,), (DIM, VOCAB)]
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.01, adamw=True)


class Trainer:
    """The model's flat fp16 weights, its owners, and the step counter."""

    def __init__(self, seed=0, device="cuda"):
        self.gen = torch.Generator(device).manual_seed(seed)
        numels = [torch.Size(s).numel() for s in SHAPES]
        self.owners = [zs.OwnerShard8(numels, RANKS, r, align=64, device=device) for r in range(RANKS)]
        sh = self.owners[0]
        self.flat = torch.zeros(sh.padded_total, dtype=torch.float16, device=device)
        self.slots = [(int(o), n) for o, n in zip(sh.offsets, numels)]
        self.weights = [self.flat[o:o + n].view(s).requires_grad_() for (o, n), s in zip(self.slots, SHAPES)]
        start = [torch.zeros(s, device=device) if len(s) == 1 else
                 torch.randn(s, generator=self.gen, device=device) * s[0] ** -0.5 for s in SHAPES]
        dense = torch.cat([w.reshape(-1) for w in start])
        for own in self.owners:
            own.alloc_state()
            own.from_dense(dense, own.master)
        with torch.no_grad():
            for w, x in zip(self.weights, start):
                w.copy_(x)
        self.grads = [torch.zeros_like(self.flat) for _ in range(RANKS)]
        self.step = 0

    def logits(self, tokens):
        emb, up, down, bias, head = self.weights
        h = emb[tokens] * DIM ** 0.5
        h = h + torch.nn.functional.gelu(h @ up) @ down + bias
        return h @ head

    def logprobs(self, tokens, targets):
        """Log-probabilities under the weights as they are."""
        with torch.no_grad():
            out = torch.empty(len(targets), device=self.flat.device)
            zs.zero_token_logprobs(self.logits(tokens), targets, out)
        return out

    def backward(self, rank, logits, dlogits):
        """This rank's flat gradient, its padding zero."""
        for w in self.weights:
            w.grad = None
        logits.backward(dlogits)
        for (o, n), w in zip(self.slots, self.weights):
            self.grads[rank][o:o + n].copy_(w.grad.reshape(-1))

    def update(self):
        """The owners' checked step from the ranks' gradients; False if it was skipped."""
        checks = [own.reduce_and_check(rank_grads=self.grads, divisor=RANKS * SCALE) for own in self.owners]
        go, coef = zs.zero_step_decision([c[0] for c in checks], [c[1] for c in checks], max_norm=1.0)
        if go:
            self.step += 1
            for own in self.owners:
                own.apply_update(step=self.step, hyper=HYPER, coef=coef, param16=self.flat)
        return go


def right(tokens):
    """The continuation that the rewards prefer."""
    return (tokens * 7 + 3) % VOCAB


def policy_phase(t: Trainer, steps: int, rows: int = 1024):
    """Mean reward of every step's samples."""
    dev, seen = t.flat.device, []
    workspace = zs.policy_workspace(rows, dev)
    stats, logp = torch.empty(4, device=dev), torch.empty(rows, device=dev)
    for _ in range(steps):
        reward_sum = 0.0
        for rank in range(RANKS):
            tokens = torch.randint(0, VOCAB, (rows,), generator=t.gen, device=dev)
            with torch.no_grad():
                probs = t.logits(tokens).float().softmax(1)
            actions = torch.multinomial(probs, 1, generator=t.gen)[:, 0]
            reward = (actions == right(tokens)).float()
            advantage = (reward - reward.mean()) / (reward.std() + 1e-3)
            old = t.logprobs(tokens, actions)
            logits = t.logits(tokens)
            dlogits = torch.empty_like(logits)
            zs.zero_policy_loss(logits.detach(), actions, old_logp=old, ref_logp=old, advantage=advantage,
                                divisor=float(rows), clip_low=0.2, clip_high=0.28, kl_coef=0.01, grad_scale=SCALE,
                                stats=stats, logp=logp, dlogits=dlogits, workspace=workspace)
            t.backward(rank, logits, dlogits)
            reward_sum += float(reward.mean())
        t.update()
        seen.append(reward_sum / RANKS)
    return seen


def preference_phase(t: Trainer, steps: int, pairs: int = 16, length: int = 8):
    """(loss, share of pairs in the right order) of every step, mean over ranks."""
    dev, seen = t.flat.device, []
    rows = 2 * pairs * length
    bounds = torch.arange(0, rows + 1, length, device=dev)
    workspace = zs.preference_workspace(rows, pairs, dev)
    f = lambda n: torch.empty(n, device=dev)  # noqa: E731
    stats, logp, seq, reward = f(2), f(rows), f(2 * pairs), f(2 * pairs)
    batches = []
    for _ in range(RANKS):  # one fixed set of pairs per rank, with the reference model's sums
        tokens = torch.randint(0, VOCAB, (rows,), generator=t.gen, device=dev)
        targets = torch.randint(0, VOCAB, (rows,), generator=t.gen, device=dev)
        chosen = (torch.arange(rows, device=dev) // length) % 2 == 0
        targets = torch.where(chosen, (tokens * 5 + 1) % VOCAB, targets)
        ref = t.logprobs(tokens, targets).view(-1, length).sum(1)
        batches.append((tokens, targets, ref))
    for _ in range(steps):
        total = torch.zeros(2)
        for rank, (tokens, targets, ref) in enumerate(batches):
            logits = t.logits(tokens)
            dlogits = torch.empty_like(logits)
            zs.zero_preference_loss(logits.detach(), targets, bounds, ref_logp=ref, beta=0.1, grad_scale=SCALE,
                                    stats=stats, logp=logp, seq_logp=seq, reward=reward, dlogits=dlogits,
                                    workspace=workspace)
            t.backward(rank, logits, dlogits)
            total += stats.cpu() / RANKS
        t.update()
        seen.append(tuple(total.tolist()))
    return seen


def main():
    t = Trainer()
    rewards = policy_phase(t, 60)
    print("policy:     mean reward %.3f at the start, %.3f after %d steps" % (rewards[0], rewards[-1], len(rewards)))
    seen = preference_phase(t, 30)
    print("preference: loss %.3f at the start, %.3f after %d steps; %.0f%% of pairs in order" % (
        seen[0][0], seen[-1][0], len(seen), 100 * seen[-1][1]))


if __name__ == "__main__":
    main()
