"""One mixture-of-experts block with a learned router, trained with Muon on a GPU.

    python examples/train_routed.py [--steps 60]

A small language model that predicts a fixed random successor of each token.
Every step runs

    muon_block_norm -> router's product -> muon_route -> muon_dispatch -> muon_gated_ffn -> muon_combine
    -> muon_block_norm -> muon_head_loss

and their backward calls: tokens go to the experts that the router chose and
come back with its weights, and the loss is taken straight from the last
hidden states, without logits.  muon_step_batched then updates the experts'
matrices, and muon_adamw_update the other parameters.  The router's bias is
moved against the experts' load, not by a gradient.  Prints the mean loss as it
goes.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import muon_newton_schulz_expert_gb300 as mk  # noqa: E402


class RoutedBlock:
    def __init__(self, vocab=512, hidden=256, ffn=256, experts=8, top=2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

        ones = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        self.experts, self.top, self.vocab = experts, top, vocab
        # what AdamW trains, and what Muon trains: whole expert matrices
        self.p = {"embed": normal(vocab, hidden, std=1.0), "head": normal(vocab, hidden, std=hidden ** -0.5),
                  "router": normal(experts, hidden, std=hidden ** -0.5), "w_in": ones.clone(), "w_post": ones.clone(),
                  "w_out": ones.clone()}
        self.w = {"w1": normal(experts, hidden, ffn, std=hidden ** -0.5),
                  "w3": normal(experts, hidden, ffn, std=hidden ** -0.5),
                  "w2": normal(experts, ffn, hidden, std=ffn ** -0.5)}
        self.bias = torch.zeros(experts, device="cuda")
        self.momentum = {k: torch.zeros(v.shape, device="cuda") for k, v in self.w.items()}
        self.moments = {k: (torch.zeros(v.shape, device="cuda"), torch.zeros(v.shape, device="cuda"))
                        for k, v in self.p.items()}
        self.steps = 0

    def gradients(self, tokens, targets):
        """(losses, gradients by parameter, the routes); a negative target is padding, which goes to no expert."""
        p, w = self.p, self.w
        padding = targets < 0
        scored = (~padding).sum().clamp(min=1)

        stream = p["embed"][tokens].float()                          # residual stream in 32 bits
        _, x, _, r0 = mk.muon_block_norm(stream, w_pre=p["w_in"])
        logits = (x @ p["router"].T).float()
        ids, weights = mk.muon_route(logits, self.top, bias=self.bias, score="sigmoid")
        ids = ids.masked_fill(padding[:, None], -1)
        rows, offsets, place = mk.muon_dispatch(x, ids, self.experts)
        y, g, u = mk.muon_gated_ffn(rows, w["w1"], w["w3"], w["w2"], offsets, keep=True)
        out = mk.muon_combine(y, place, weights)
        stream2, last, q, r1 = mk.muon_block_norm(stream, out, w_post=p["w_post"], w_pre=p["w_out"])
        loss, lse = mk.muon_head_loss(last, p["head"], targets)

        dloss = torch.ones_like(loss) / scored                       # the mean over what is scored
        dlast, dhead = mk.muon_head_loss_backward(dloss, last, p["head"], targets, lse)
        n = mk.muon_block_norm_backward(None, dlast, stream2, out, q, r1, w_post=p["w_post"], w_pre=p["w_out"])
        dy, dweights = mk.muon_combine_backward(n.dblock, y, place, weights)
        drows, dw1, dw3, dw2 = mk.muon_gated_ffn_backward(dy, rows, g, u, w["w1"], w["w3"], w["w2"], offsets)
        dlogits = mk.muon_route_backward(dweights, logits, ids, score="sigmoid").bfloat16()
        dx = mk.muon_dispatch_backward(drows, place) + dlogits @ p["router"]
        first = mk.muon_block_norm_backward(n.dresidual, dx, stream, None, None, r0, w_pre=p["w_in"])
        d = {"head": dhead, "router": dlogits.T @ x, "w_in": first.dw_pre, "w_post": n.dw_post, "w_out": n.dw_pre,
             "embed": torch.zeros(p["embed"].shape, device="cuda").index_add_(0, tokens, first.dresidual).bfloat16(),
             "w1": dw1, "w3": dw3, "w2": dw2}
        return loss, d, ids

    def step(self, tokens, targets, lr=0.02, adam_lr=2e-3, bias_lr=1e-3):
        """One training step; returns the mean loss (a tensor)."""
        loss, d, ids = self.gradients(tokens, targets)
        self.steps += 1
        for k, param in self.w.items():
            mk.muon_step_batched(param, d[k], self.momentum[k], lr=lr, weight_decay=0.01)
        for k, param in self.p.items():
            mk.muon_adamw_update(param, d[k], *self.moments[k], self.steps, lr=adam_lr, weight_decay=0.0)
        load = (ids.flatten()[:, None] == torch.arange(self.experts, device="cuda")).float().mean(0)
        self.bias += bias_lr * torch.sign(load.mean() - load)
        return loss.sum() / (targets >= 0).sum().clamp(min=1)


def main(steps=60, rows=4096, seed=1):
    block = RoutedBlock()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    successor = torch.randperm(block.vocab, generator=gen, device="cuda")
    history = []
    for i in range(steps):
        tokens = torch.randint(0, block.vocab, (rows,), generator=gen, device="cuda")
        targets = successor[tokens]
        targets[-rows // 50:] = -1                                   # a padded batch
        history.append(float(block.step(tokens, targets)))
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i:3d}  mean loss {history[-1]:8.4f}")
    status = mk.muon_get_device_status()
    if status:
        raise RuntimeError(mk.muon_status_string(status))
    return history


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    parser.add_argument("--steps", type=int, default=60)
    main(parser.parse_args().steps)
