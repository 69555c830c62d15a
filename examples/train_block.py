"""One gated feed-forward block with several experts, trained with Muon on a GPU.

    python examples/train_block.py [--steps 60]

A small language model that predicts a fixed random successor of each token:
an embedding, the norm before the block, experts chosen by the token, the norm
after the block with a gate on the residual stream, the norm before the
logits, and the log probability of the successor.  Every step runs

    muon_block_norm -> muon_gated_ffn -> muon_block_norm -> logits -> muon_token_logprobs

and their backward calls; muon_step_batched then updates the experts' matrices
from the gradients as they are, and muon_adamw_update the other parameters.
Prints the mean log probability and entropy as it goes.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import muon_newton_schulz_expert_gb300 as mk  # noqa: E402


class Block:
    def __init__(self, vocab=512, hidden=256, ffn=512, experts=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

        ones = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        self.experts, self.vocab = experts, vocab
        # what AdamW trains, and what Muon trains: whole expert matrices
        self.p = {"embed": normal(vocab, hidden, std=1.0), "head": normal(vocab, hidden, std=hidden ** -0.5),
                  "w_in": ones.clone(), "w_post": ones.clone(), "w_out": ones.clone(), "gate": ones.clone()}
        self.w = {"w1": normal(experts, hidden, ffn, std=hidden ** -0.5),
                  "w3": normal(experts, hidden, ffn, std=hidden ** -0.5),
                  "w2": normal(experts, ffn, hidden, std=ffn ** -0.5)}
        self.momentum = {k: torch.zeros(v.shape, device="cuda") for k, v in self.w.items()}
        self.moments = {k: (torch.zeros(v.shape, device="cuda"), torch.zeros(v.shape, device="cuda"))
                        for k, v in self.p.items()}
        self.steps = 0

    def step(self, tokens, targets, lr=0.02, adam_lr=2e-3):
        """One training step; returns the mean log probability and entropy (tensors)."""
        p, w = self.p, self.w
        # rows sorted by expert (here the token decides), as the experts take them
        expert = tokens % self.experts
        order = torch.argsort(expert, stable=True)
        tokens, targets = tokens[order], targets[order]
        offsets = torch.zeros(self.experts + 1, dtype=torch.int64, device="cuda")
        offsets[1:] = torch.bincount(expert, minlength=self.experts).cumsum(0)

        stream = p["embed"][tokens].float()                          # residual stream in 32 bits
        _, x, _, r0 = mk.muon_block_norm(stream, w_pre=p["w_in"])
        y, g, u = mk.muon_gated_ffn(x, w["w1"], w["w3"], w["w2"], offsets, keep=True)
        stream2, out, q, r1 = mk.muon_block_norm(stream, y, w_post=p["w_post"], gate=p["gate"], w_pre=p["w_out"])
        logits = out @ p["head"].T
        score = mk.muon_token_logprobs(logits, targets)

        dlogp = torch.full_like(score.logp, -1.0 / len(tokens))      # loss: minus the mean log probability
        dlogits = mk.muon_token_logprobs_backward(logits, targets, score.lse, dlogp=dlogp, out=logits)
        d = {"head": dlogits.T @ out}
        n = mk.muon_block_norm_backward(None, dlogits @ p["head"], stream2, y, q, r1, w_post=p["w_post"],
                                        gate=p["gate"], w_pre=p["w_out"])
        d |= {"w_post": n.dw_post, "gate": n.dgate, "w_out": n.dw_pre}
        dx, dw1, dw3, dw2 = mk.muon_gated_ffn_backward(n.dblock, x, g, u, w["w1"], w["w3"], w["w2"], offsets)
        first = mk.muon_block_norm_backward(n.dresidual, dx, stream, None, None, r0, w_pre=p["w_in"])
        d["w_in"] = first.dw_pre
        d["embed"] = torch.zeros(p["embed"].shape, device="cuda").index_add_(0, tokens, first.dresidual).bfloat16()

        self.steps += 1
        for k, grad in (("w1", dw1), ("w3", dw3), ("w2", dw2)):
            mk.muon_step_batched(w[k], grad, self.momentum[k], lr=lr, weight_decay=0.01)
        for k, param in p.items():
            mk.muon_adamw_update(param, d[k], *self.moments[k], self.steps, lr=adam_lr, weight_decay=0.0)
        return score.logp.mean(), score.entropy.mean()


def main(steps=60, rows=4096, seed=1):
    block = Block()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    successor = torch.randperm(block.vocab, generator=gen, device="cuda")
    history = []
    for i in range(steps):
        tokens = torch.randint(0, block.vocab, (rows,), generator=gen, device="cuda")
        logp, entropy = block.step(tokens, successor[tokens])
        history.append((float(logp), float(entropy)))
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i:3d}  mean log probability {history[-1][0]:8.4f}  entropy {history[-1][1]:7.4f}")
    status = mk.muon_get_device_status()
    if status:
        raise RuntimeError(mk.muon_status_string(status))
    return history


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    parser.add_argument("--steps", type=int, default=60)
    main(parser.parse_args().steps)
