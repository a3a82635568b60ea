"""One learner step around the NVFP4 expert layer, on synthetic data: the
residual block in front of it, the layer, the final norm, a dense head, and a
loss of a policy gradient with an entropy bonus and of distillation from a BF16
teacher's top logits; then the gradients back to the block's input.

  python examples/learner_step.py [--layer tiny|small] [--vocab V]

Every step but the two dense products of the head and the elementwise glue (the
advantages, the sum of the two logit gradients, casts) is one of the package's
entry points.
"""
import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import nvfp4_w4a4_moe_top_gb300 as M  # noqa: E402
import synth  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPS = 1e-6


def dev_bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(BF16)


def new(shape, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="cuda")


class Block:
    """Norm, expert layer, final norm and head, with their weights, workspaces
    and the values the backward needs."""

    def __init__(self, lay, vocab, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        T, E, k, d, F = self.shape = lay.T, lay.E, lay.k, lay.d, lay.d_ff
        self.W1, self.W2 = dev_bf16(lay.w1()), dev_bf16(lay.w2())
        self.w1q, self.w2q = M.quantize_weights(self.W1), M.quantize_weights(self.W2)
        self.w_in = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(BF16)
        self.w_out = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(BF16)
        self.head = (torch.randn((vocab, d), generator=g, device="cuda") * 2 / d ** 0.5).to(BF16)
        mc = M.m_cap(T, E, k)
        self.ws = M.forward_workspace(T, E, k, d, F)
        self.save_u, self.save_h = new((mc, 2 * F), BF16), new((mc, F), BF16)
        self.bws = new(M.backward_workspace_bytes(T, E, k, d, F), torch.uint8)
        self.nws = new(M.add_rmsnorm_backward_workspace_bytes(T, d), torch.uint8)
        self.status = torch.zeros(1, dtype=I32, device="cuda")

    def forward(self, x, res, router_logits):
        """Logits [T][vocab] of the block on the sublayer output x and the
        residual stream res; the first norm's output also in 8 bits, as a dense
        block-scaled product beside the experts would take it."""
        T, E, k, d, F = self.shape
        self.h1, self.y1, self.r1 = new((T, d), BF16), new((T, d), BF16), new(T)
        self.y8, self.y8_sf = new((T, d), torch.uint8), new(M.mx8_sf_bytes(T, d), torch.uint8)
        M.moe_add_rmsnorm(x, res, self.w_in, EPS, self.h1, self.y1, self.y8, self.y8_sf, self.r1, self.status)
        out = new((T, d), BF16)
        M.moe_expert_forward_train(self.y1, router_logits, T, E, k, d, F, self.w1q["codes"], self.w1q["sf"],
                                   self.w1q["g"], self.w2q["codes"], self.w2q["sf"], self.w2q["g"], out, self.ws,
                                   self.save_u, self.save_h, self.status)
        self.h2, self.y2, self.r2 = new((T, d), BF16), new((T, d), BF16), new(T)
        M.moe_add_rmsnorm(out, self.h1, self.w_out, EPS, self.h2, self.y2, None, None, self.r2, self.status)
        return self.y2 @ self.head.t()

    def backward(self, dlogits):
        """Gradients of the block's input (x and res alike), of both norms'
        weights and of the experts' weights."""
        T, E, k, d, F = self.shape
        v = M.forward_views(self.ws, T, E, k, d, F)
        dw_in, dw_out = new(d), new(d)
        dh2 = new((T, d), BF16)  # of the experts' output and of h1 alike
        M.moe_add_rmsnorm_backward(dlogits @ self.head, None, self.h2, self.r2, self.w_out, dh2, dw_out, self.nws,
                                   self.status)
        dy1, dW1, dW2 = new((T, d)), new((E, 2 * F, d)), new((E, d, F))
        dw = new((T, k))
        M.moe_expert_backward(dh2, self.y1, T, E, k, d, F, self.W1, self.W2, self.w2q["codes"], self.w2q["sf"],
                              self.w2q["g"], v["topk_ids"], v["topk_w"], v["offsets"], v["row_to_token"],
                              v["token_slot_row"], self.save_u, self.save_h, v["h_codes"], v["h_sf"], v["h_g"], dy1,
                              dW1, dW2, None, dw, self.bws, self.status)
        dx = new((T, d), BF16)
        M.moe_add_rmsnorm_backward(dy1.to(BF16), dh2, self.h1, self.r1, self.w_in, dx, dw_in, self.nws, self.status)
        return dict(dx=dx, dw_in=dw_in, dw_out=dw_out, dW1=dW1, dW2=dW2)


def losses(logits, tokens, advantages, teacher, status, n_top=5, entropy_bonus=0.01, kl_weight=0.5):
    """Policy gradient with entropy bonus and distillation on the logits:
    (the scalars, the gradient of the logits, the reported values).  Rows with
    a negative token (prompt) count in neither mean of the policy loss."""
    T, V = logits.shape
    n = (tokens >= 0).sum().clamp(min=1)
    lp, ent, stats = new(T), new(T), new((T, 2))
    top_ids, top_lp = new((T, n_top), I32), new((T, n_top))
    M.moe_token_logprobs(logits, tokens, 1.0, n_top, lp, ent, stats, top_ids, top_lp, status)
    active = (tokens >= 0).float()
    g_lp, g_ent = -advantages * active / n, -entropy_bonus * active / n
    ids, values, lse = teacher
    kl, d_kl = new(T), torch.empty_like(logits)
    M.moe_distill_topk_train(logits, ids, values, lse, 1.0, torch.full_like(kl, kl_weight / T), kl, d_kl, status)
    dlogits = torch.empty_like(logits)
    M.moe_token_logprobs_backward(logits, tokens, 1.0, stats, ent, g_lp, g_ent, dlogits, status)
    dlogits += d_kl
    loss = (g_lp * lp + g_ent * ent).sum() + kl_weight * kl.mean()
    return loss, dlogits, dict(logprob=lp, entropy=ent, kl=kl, top_ids=top_ids, top_logprob=top_lp)


def inputs(lay, vocab, K=32, seed=1):
    """A batch: the sublayer output, the residual stream, router logits,
    sampled tokens with advantages, and a teacher's top logits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, d = lay.T, lay.d
    x, res = dev_bf16(lay.x()), torch.randn((T, d), generator=g, device="cuda").to(BF16)
    tokens = torch.randint(0, vocab, (T,), generator=g, device="cuda", dtype=torch.int64).int()
    tokens[: T // 8] = -1  # the prompt
    adv = torch.randn(T, generator=g, device="cuda")
    start = torch.randint(0, vocab, (T, 1), generator=g, device="cuda")
    ids = ((start + torch.arange(K, device="cuda") * 31) % vocab).int()
    values = 3 * torch.randn((T, K), generator=g, device="cuda")
    lse = torch.logsumexp(values, 1) + 0.1  # a tenth of the teacher's mass off its list
    return x, res, torch.from_numpy(lay.logits()).cuda(), tokens, adv, (ids, values, lse)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layer", default="tiny", choices=["tiny", "small"])
    ap.add_argument("--vocab", type=int, default=4099)
    a = ap.parse_args(argv)
    lay = synth.layer(a.layer)
    block = Block(lay, a.vocab)
    x, res, router, tokens, adv, teacher = inputs(lay, a.vocab)
    logits = block.forward(x, res, router)
    loss, dlogits, seen = losses(logits, tokens, adv, teacher, block.status)
    grads = block.backward(dlogits)
    assert int(block.status.item()) == 0, "device status %#x" % int(block.status.item())
    print("loss %.5f  mean entropy %.4f  mean KL %.4f  |dx| %.3e  |dw_in| %.3e  |dW1| %.3e"
          % (loss.item(), seen["entropy"].mean().item(), seen["kl"].mean().item(), grads["dx"].float().norm().item(),
             grads["dw_in"].norm().item(), grads["dW1"].norm().item()))
    print("first token's alternatives:", [(int(i), round(float(p), 3)) for i, p in
                                          zip(seen["top_ids"][0].tolist(), seen["top_logprob"][0].tolist())])
    return dict(loss=loss, logits=logits, dlogits=dlogits, block=block, grads=grads, seen=seen,
                inputs=(x, res, router, tokens, adv, teacher))


if __name__ == "__main__":
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()
    main()
