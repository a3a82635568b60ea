"""A rollout and a learner step on the same block, on synthetic data: each step
embeds the last tokens, runs the norm, the NVFP4 expert layer, the final norm and a
dense head, and draws the next tokens; the learner then scores the tokens of the
last step with the logits it computes itself, and the policy gradient goes back to
the embedding's table.

  python examples/rollout_step.py [--layer tiny|small] [--vocab V] [--steps N]

Every step but the dense products of router and head and the elementwise glue is
one of the package's entry points.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [p for p in (ROOT, os.path.join(ROOT, "examples")) if p not in sys.path]

import nvfp4_w4a4_moe_top_gb300 as M  # noqa: E402
import synth  # noqa: E402
from learner_step import BF16, I32, Block, new  # noqa: E402

SCALE = 4.0  # of the embedding


class Policy(Block):
    """The block with an embedding in front of it and a router of its own; one
    token per sequence and step."""

    def __init__(self, lay, vocab, seed=0):
        super().__init__(lay, vocab, seed)
        T, E, k, d, F = self.shape
        g = torch.Generator(device="cuda").manual_seed(seed + 100)
        self.vocab = vocab
        self.table = (torch.randn((vocab, d), generator=g, device="cuda") / SCALE).to(BF16)
        self.router = (torch.randn((E, d), generator=g, device="cuda") / d ** 0.5).to(BF16)
        self.ews = new(M.embed_tokens_backward_workspace_bytes(T, vocab, d), torch.uint8)

    def logits(self, tokens):
        """Logits [T][vocab] after `tokens`; tokens < 0 (sequences that have
        ended) have the embedding 0."""
        T, E, k, d, F = self.shape
        self.tokens, self.x = tokens, new((T, d), BF16)
        M.moe_embed_tokens(tokens, self.table, SCALE, self.x, self.status)
        return self.forward(self.x, None, (self.x @ self.router.t()).float())

    def table_gradient(self, dlogits):
        """Gradient of the table (FP32) and of the block's weights."""
        grads = self.backward(dlogits)
        grads["dtable"] = new(self.table.shape)
        M.moe_embed_tokens_backward(grads["dx"], self.tokens, SCALE, grads["dtable"], self.ews, status=self.status)
        return grads


def rollout(policy, tokens, steps, seed=1, temperature=0.8, top_k=50, top_p=0.95):
    """`steps` tokens of each sequence after `tokens`; returns the tokens fed to
    the last step, the tokens it drew and their log-probabilities under the policy
    at that temperature and as they were drawn."""
    T = len(tokens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = lambda v, t=torch.float32: torch.full((T,), v, dtype=t, device="cuda")  # noqa: E731
    inv_t, k, p = full(1.0 / temperature), full(top_k, I32), full(top_p)
    for _ in range(steps):
        fed, drawn = tokens, new(T, I32)
        logprob, kept = new(T), new(T)
        u = torch.rand(T, generator=g, device="cuda")
        logits = policy.logits(fed)
        M.moe_sample_tokens(logits, u, drawn, inv_t, k, p, None, logprob, kept, policy.status)
        tokens = torch.where(fed >= 0, drawn, fed)  # a sequence that has ended stays so
    return dict(fed=fed, drawn=drawn, logprob=logprob, kept_logprob=kept, u=u, logits=logits)


def learn(policy, fed, drawn, advantages, temperature=0.8):
    """The learner's pass over the last step: its log-probabilities of the drawn
    tokens, and the gradients of -mean(advantage * logprob)."""
    logits = policy.logits(fed)
    T, V = logits.shape
    n = (fed >= 0).sum().clamp(min=1)
    lp, ent, stats = new(T), new(T), new((T, 2))
    M.moe_token_logprobs(logits, drawn, 1.0 / temperature, 0, lp, ent, stats, status=policy.status)
    g = torch.where(fed >= 0, -advantages / n, 0.0)
    dlogits = torch.empty_like(logits)
    M.moe_token_logprobs_backward(logits, drawn, 1.0 / temperature, stats, None, g, None, dlogits, policy.status)
    return dict(logprob=lp, loss=(g * lp).sum(), dlogits=dlogits, grads=policy.table_gradient(dlogits))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layer", default="tiny", choices=["tiny", "small"])
    ap.add_argument("--vocab", type=int, default=4099)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args(argv)
    policy = Policy(synth.layer(a.layer), a.vocab)
    T = policy.shape[0]
    g = torch.Generator(device="cuda").manual_seed(7)
    first = torch.randint(0, a.vocab, (T,), generator=g, device="cuda", dtype=torch.int64).int()
    first[T - T // 16:] = -1  # sequences that have ended
    seen = rollout(policy, first, a.steps)
    step = learn(policy, seen["fed"], seen["drawn"], torch.randn(T, generator=g, device="cuda"))
    assert int(policy.status.item()) == 0, "device status %#x" % int(policy.status.item())
    print("loss %.5f  mean log-probability %.4f (as drawn %.4f)  learner against sampler %.1e  |dtable| %.3e"
          % (step["loss"].item(), step["logprob"].mean().item(), seen["kept_logprob"].mean().item(),
             (step["logprob"] - seen["logprob"]).abs().max().item(), step["grads"]["dtable"].norm().item()))
    return dict(policy=policy, seen=seen, step=step)


if __name__ == "__main__":
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()
    main()
