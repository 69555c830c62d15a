"""The operators around the Muon step as measured cases: the gated feed-forward
block over whole expert matrices, the norms before and after a block, and the
log probabilities of given tokens, each forward and backward.

`run` computes a case in elementary torch operations in 32 bits (own = False)
or through the framework's entry points (own = True); `exact` computes it in
64 bits, separately.  Expert matrices are laid out as the Muon step takes them:
w1 and w3 [experts, hidden, ffn], w2 [experts, ffn, hidden].
"""

import math
import random

import torch

own = False

HIDDEN, EXPERT_HIDDEN = 6144, 1792   # the expert shape of the Muon workloads
EPS = 1e-6


def listed():
    return [
        # one token through one expert: the latency of a single decoding step
        {"name": "ffn_one_token", "op": "ffn", "rows": 1, "experts": 1, "hidden": HIDDEN, "ffn": EXPERT_HIDDEN,
         "act": "silu", "keep": False, "routing": 1},
        # eight decoding sequences, eight experts each, spread over the 32 experts that one rank owns
        {"name": "ffn_decode_routed", "op": "ffn", "rows": 64, "experts": 32, "hidden": HIDDEN, "ffn": EXPERT_HIDDEN,
         "act": "silu", "keep": False, "routing": 2},
        # a small model with odd group sizes and widths that end inside a tile, gate and up kept for the backward pass
        {"name": "ffn_train_ragged", "op": "ffn", "rows": 1777, "experts": 5, "hidden": 1000, "ffn": 328,
         "act": "gelu", "keep": True, "routing": 3},
        # a training step's rows over the 32 experts of one rank
        {"name": "ffn_train", "op": "ffn", "rows": 16384, "experts": 32, "hidden": HIDDEN, "ffn": EXPERT_HIDDEN,
         "act": "silu", "keep": True, "routing": 4},
        # the gradients of that step: rows, and all 96 expert matrices
        {"name": "ffn_backward", "op": "ffn_backward", "rows": 16384, "experts": 32, "hidden": HIDDEN,
         "ffn": EXPERT_HIDDEN, "act": "silu", "routing": 5},
        # decoding eight sequences: the norm after one block and before the next, one short call
        {"name": "norm_decode", "op": "norm", "rows": 8, "hidden": HIDDEN, "residual": "bf16", "branch": "bf16",
         "gate": "shared"},
        # a training step with a 32-bit residual stream and a gate of its own for each token
        {"name": "norm_train", "op": "norm", "rows": 16384, "hidden": HIDDEN, "residual": "f32", "branch": "bf16",
         "gate": "rows"},
        # its gradients with a 16-bit stream: rows, both weights and the shared gate
        {"name": "norm_backward", "op": "norm_backward", "rows": 16384, "hidden": HIDDEN, "residual": "bf16",
         "branch": "bf16", "gate": "shared"},
        # an odd width in 32 bits, as a small verification model has
        {"name": "norm_backward_odd", "op": "norm_backward", "rows": 1021, "hidden": 1001, "residual": "f32",
         "branch": "f32", "gate": "shared"},
        # scores of the tokens that four sequences sampled, with the alternatives that are shown beside them
        {"name": "logprobs_decode", "op": "logprobs", "rows": 4, "vocab": 256000, "type": "f32", "top": 20},
        # scores of a long packed batch, with entropy
        {"name": "logprobs_train", "op": "logprobs", "rows": 4096, "vocab": 256000, "type": "bf16", "top": 0},
        # the gradient that the loss sends into the logits, for an odd vocabulary
        {"name": "logprobs_backward", "op": "logprobs_backward", "rows": 8192, "vocab": 50003, "type": "bf16"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(("ffn", "ffn", "ffn_backward", "ffn_backward", "norm", "norm_backward", "logprobs",
                       "logprobs_backward"))
    if kind in ("ffn", "ffn_backward"):
        hidden, ffn = 8 * _spread(rng, 32, 768), 8 * _spread(rng, 16, 256)
        experts = _spread(rng, 1, 64)
        most = 16384 * HIDDEN * EXPERT_HIDDEN // (hidden * ffn)
        rows = _spread(rng, 1, min(32768, most))
        case = {"op": kind, "rows": rows, "experts": experts, "hidden": hidden, "ffn": ffn,
                "act": rng.choice(("silu", "gelu")), "routing": rng.randrange(1 << 20)}
        if kind == "ffn":
            case["keep"] = rows > 256 or rng.random() < 0.3
        return case
    if kind in ("norm", "norm_backward"):
        hidden = _spread(rng, 64, 8192)
        if rng.random() < 0.75:
            hidden = max(64, hidden // 8 * 8)
        rows = _spread(rng, 1, min(32768, 16384 * HIDDEN // hidden))
        residual, branch = rng.choice((("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")))
        return {"op": kind, "rows": rows, "hidden": hidden, "residual": residual, "branch": branch,
                "gate": rng.choice(("none", "shared", "rows"))}
    vocab = _spread(rng, 500, 256000)
    case = {"op": kind, "rows": _spread(rng, 1, min(16384, (400 << 20) // vocab)), "vocab": vocab,
            "type": rng.choice(("bf16", "f32"))}
    if kind == "logprobs":
        case["top"] = rng.choice((0, 0, 1, 5, 20, 32))
    return case


# ---------------------------------------------------------------------------- inputs
def group_sizes(case):
    """Rows of each expert: an uneven router's choice, some experts without rows."""
    rng = random.Random(case["routing"])
    weights = [rng.expovariate(1.0) ** 0.5 for _ in range(case["experts"])]
    picks = rng.choices(range(case["experts"]), weights, k=case["rows"])
    sizes = [0] * case["experts"]
    for e in picks:
        sizes[e] += 1
    return sizes


def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


class _Random:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(int(seed))

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=self.gen, device="cuda").mul_(std).to(dtype)

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.gen, device="cuda")


def prepare(case, seed):
    r = _Random(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("ffn", "ffn_backward"):
        E, H, F, T = case["experts"], case["hidden"], case["ffn"], case["rows"]
        bf = torch.bfloat16
        sizes = group_sizes(case)
        offsets = [0]
        for n in sizes:
            offsets.append(offsets[-1] + n)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int64, device="cuda")
        s["most"] = max(sizes)
        s["x"] = r.normal(T, H, dtype=bf)
        s["w1"] = r.normal(E, H, F, std=H ** -0.5, dtype=bf)
        s["w3"] = r.normal(E, H, F, std=H ** -0.5, dtype=bf)
        s["w2"] = r.normal(E, F, H, std=F ** -0.5, dtype=bf)
        if op == "ffn_backward":
            s["gate"] = r.normal(T, F, dtype=bf)
            s["up"] = r.normal(T, F, dtype=bf)
            s["dy"] = r.normal(T, H, std=1e-3, dtype=bf)
    elif op in ("norm", "norm_backward"):
        T, H = case["rows"], case["hidden"]
        rt, bt = _type(case["residual"]), _type(case["branch"])
        outlying = 1 + 9 * (r.uniform(H) < 0.01)   # a few channels far larger than the others, as streams have
        s["residual"] = (r.normal(T, H, std=3.0) * outlying).to(rt)
        s["block"] = r.normal(T, H, std=0.5, dtype=bt)
        s["w_post"] = (1 + 0.1 * r.normal(H)).to(bt)
        s["w_pre"] = (1 + 0.1 * r.normal(H)).to(bt)
        s["gate"] = None
        if case["gate"] != "none":
            shape = (H,) if case["gate"] == "shared" else (T, H)
            s["gate"] = (0.5 + 0.2 * r.normal(*shape)).to(bt)
        s["scale"] = 0.7
        if op == "norm_backward":
            b, n = s["block"].float(), s["residual"].float()
            s["rstd_post"] = torch.rsqrt(b.square().mean(1) + EPS)
            s["rstd_pre"] = torch.rsqrt(n.square().mean(1) + EPS)
            s["dresidual"] = r.normal(T, H, std=1e-2, dtype=rt)
            s["dnormed"] = r.normal(T, H, std=1e-2, dtype=bt)
    else:
        T, V = case["rows"], case["vocab"]
        logits = r.normal(T, V, std=2.5)
        tokens = (r.uniform(T) * (V - V // 50)).long()
        logits[torch.arange(T, device="cuda"), tokens] += 6.0   # a sampled token is mostly a likely one
        logits[:, V - V // 50:] = -math.inf                     # the vocabulary's padding is masked
        s["logits"] = logits.to(_type(case["type"]))
        tokens[(r.uniform(T) < 0.05) & (torch.arange(T, device="cuda") > 0)] = -1   # prompt and padding: no score
        s["tokens"] = tokens
        if op == "logprobs_backward":
            x = s["logits"].float()
            s["lse"] = torch.logsumexp(x, 1)
            p = torch.exp(x - s["lse"][:, None])
            s["entropy"] = s["lse"] - (p * torch.where(p > 0, x, 0.0)).sum(1)
            s["dlogp"] = r.normal(T, std=1.0 / T)
            s["dentropy"] = r.normal(T, std=1e-2 / T)
    return s


# ---------------------------------------------------------------------------- the plain form
def _act(g, kind):
    """(act(g), act'(g))"""
    if kind == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _places(s):
    """Each row's expert and its place among that expert's rows."""
    row = torch.arange(s["x"].shape[0], device="cuda")
    expert = torch.searchsorted(s["offsets"][1:].contiguous(), row, right=True)
    return expert, row - s["offsets"][expert]


def _by_expert(v, s, at):
    padded = torch.zeros(s["w1"].shape[0], s["most"], v.shape[1], dtype=torch.float32, device="cuda")
    padded[at] = v.float()
    return padded


def _plain_ffn(s):
    at = _places(s)
    x = _by_expert(s["x"], s, at)
    g, u = torch.bmm(x, s["w1"].float()), torch.bmm(x, s["w3"].float())
    y = torch.bmm(_act(g, s["case"]["act"])[0] * u, s["w2"].float())
    bf = torch.bfloat16
    out = {"y": y[at].to(bf)}
    if s["case"]["keep"]:
        out |= {"gate": g[at].to(bf), "up": u[at].to(bf)}
    return out


def _plain_ffn_backward(s):
    at = _places(s)
    x, g, u, dy = (_by_expert(s[k], s, at) for k in ("x", "gate", "up", "dy"))
    a, da = _act(g, s["case"]["act"])
    dh = torch.bmm(dy, s["w2"].float().mT)
    dg, du = dh * u * da, dh * a
    dx = torch.bmm(dg, s["w1"].float().mT) + torch.bmm(du, s["w3"].float().mT)
    bf = torch.bfloat16
    return {"dx": dx[at].to(bf), "dw1": torch.bmm(x.mT, dg).to(bf), "dw3": torch.bmm(x.mT, du).to(bf),
            "dw2": torch.bmm((a * u).mT, dy).to(bf)}


def _plain_norm(s):
    r, b = s["residual"].float(), s["block"].float()
    rstd_post = 1 / torch.sqrt((b * b).mean(1) + EPS)
    n = b * rstd_post[:, None] * s["w_post"].float()
    if s["gate"] is not None:
        n = n * s["gate"].float()
    r = r + s["scale"] * n
    rstd_pre = 1 / torch.sqrt((r * r).mean(1) + EPS)
    y = r * rstd_pre[:, None] * s["w_pre"].float()
    return {"residual": r.to(s["residual"].dtype), "normed": y.to(s["block"].dtype), "rstd_post": rstd_post,
            "rstd_pre": rstd_pre}


def _plain_norm_backward(s):
    xh = s["residual"].float() * s["rstd_pre"][:, None]
    bh = s["block"].float() * s["rstd_post"][:, None]
    dy, wp, wq = s["dnormed"].float(), s["w_pre"].float(), s["w_post"].float()
    t = dy * wp
    dr = s["dresidual"].float() + s["rstd_pre"][:, None] * (t - xh * (t * xh).mean(1, keepdim=True))
    dn = s["scale"] * dr
    out = {"dw_pre": (dy * xh).sum(0).to(wp_type(s))}
    if s["gate"] is not None:
        dgate = dn * bh * wq
        out["dgate"] = (dgate.sum(0) if s["gate"].dim() == 1 else dgate).to(s["gate"].dtype)
        dn = dn * s["gate"].float()
    out["dw_post"] = (dn * bh).sum(0).to(wp_type(s))
    t = dn * wq
    db = s["rstd_post"][:, None] * (t - bh * (t * bh).mean(1, keepdim=True))
    out["dresidual"], out["dblock"] = dr.to(s["residual"].dtype), db.to(s["block"].dtype)
    return out


def wp_type(s):
    return s["w_pre"].dtype


def _plain_logprobs(s):
    x, tokens, top = s["logits"].float(), s["tokens"], s["case"]["top"]
    most = x.amax(1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(1, keepdim=True)
    lse = (most + torch.log(total))[:, 0]
    entropy = lse - (e * torch.where(e > 0, x, 0.0)).sum(1) / total[:, 0]
    given = tokens >= 0
    logp = torch.where(given, x.gather(1, tokens.clamp(min=0)[:, None])[:, 0] - lse, 0.0)
    out = {"logp": logp, "entropy": entropy, "lse": lse}
    if top:
        values, ids = torch.sort(x, dim=1, descending=True, stable=True)   # stable: ties go to the lowest index
        out |= {"top_ids": ids[:, :top].contiguous(), "top_logp": values[:, :top] - lse[:, None]}
    return out


def _plain_logprobs_backward(s):
    x, tokens = s["logits"].float(), s["tokens"]
    logp = x - s["lse"][:, None]
    p = torch.exp(logp)
    given = tokens >= 0
    dlogp = torch.where(given, s["dlogp"], 0.0)[:, None]
    dent = s["dentropy"][:, None]
    d = -dlogp * p - dent * torch.where(p > 0, p * (logp + s["entropy"][:, None]), 0.0)
    d.scatter_add_(1, tokens.clamp(min=0)[:, None], dlogp)
    return {"dlogits": d.to(s["logits"].dtype)}


# ---------------------------------------------------------------------------- the framework's operators
def _kept(s, name, make):
    """A buffer that a user's program makes once and keeps."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own(s):
    import muon_newton_schulz_expert_gb300 as mk

    c = s["case"]
    op = c["op"]
    if op == "ffn":
        ws = _kept(s, "workspace", lambda: torch.empty(
            mk.muon_gated_ffn_workspace_bytes(c["rows"], c["experts"], c["hidden"], c["ffn"]), dtype=torch.uint8,
            device="cuda"))
        got = mk.muon_gated_ffn(s["x"], s["w1"], s["w3"], s["w2"], s["offsets"], act=c["act"], keep=c["keep"],
                                workspace=ws)
        return dict(zip(("y", "gate", "up"), got)) if c["keep"] else {"y": got}
    if op == "ffn_backward":
        ws = _kept(s, "workspace", lambda: torch.empty(
            mk.muon_gated_ffn_backward_workspace_bytes(c["rows"], c["experts"], c["hidden"], c["ffn"]),
            dtype=torch.uint8, device="cuda"))
        dw = _kept(s, "dw", lambda: tuple(torch.empty_like(s[k]) for k in ("w1", "w3", "w2")))
        dx, dw1, dw3, dw2 = mk.muon_gated_ffn_backward(
            s["dy"], s["x"], s["gate"], s["up"], s["w1"], s["w3"], s["w2"], s["offsets"], act=c["act"], dw=dw,
            workspace=ws)
        return {"dx": dx, "dw1": dw1, "dw3": dw3, "dw2": dw2}
    if op == "norm":
        residual, normed, rstd_post, rstd_pre = mk.muon_block_norm(
            s["residual"], s["block"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], scale=s["scale"],
            eps=EPS)
        return {"residual": residual, "normed": normed, "rstd_post": rstd_post, "rstd_pre": rstd_pre}
    if op == "norm_backward":
        ws = _kept(s, "workspace", lambda: torch.empty(
            mk.muon_block_norm_backward_workspace_bytes(c["rows"], c["hidden"]), dtype=torch.uint8, device="cuda"))
        g = mk.muon_block_norm_backward(
            s["dresidual"], s["dnormed"], s["residual"], s["block"], s["rstd_post"], s["rstd_pre"],
            w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], scale=s["scale"], workspace=ws)
        out = {"dresidual": g.dresidual, "dblock": g.dblock, "dw_post": g.dw_post, "dw_pre": g.dw_pre}
        if s["gate"] is not None:
            out["dgate"] = g.dgate
        return out
    if op == "logprobs":
        got = mk.muon_token_logprobs(s["logits"], s["tokens"], top=c["top"])
        out = {"logp": got.logp, "entropy": got.entropy, "lse": got.lse}
        if c["top"]:
            out |= {"top_ids": got.top_ids, "top_logp": got.top_logp}
        return out
    return {"dlogits": mk.muon_token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], s["dlogp"],
                                                       s["dentropy"])}


_PLAIN = {"ffn": _plain_ffn, "ffn_backward": _plain_ffn_backward, "norm": _plain_norm,
          "norm_backward": _plain_norm_backward, "logprobs": _plain_logprobs,
          "logprobs_backward": _plain_logprobs_backward}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("ffn", "ffn_backward"):
        T, E, H, F = case["rows"], case["experts"], case["hidden"], case["ffn"]
        used = sum(n > 0 for n in group_sizes(case))
        if op == "ffn":
            rows = 2 * H + (2 * F if case["keep"] else 0)                # x and y, gate and up
            return {"bytes": 2 * (T * rows + 3 * used * H * F) + 8 * (E + 1), "flops": 6 * T * H * F}
        rows = 3 * H + 2 * F                                             # dy, x, dx, gate and up
        return {"bytes": 2 * (T * rows + 3 * used * H * F + 3 * E * H * F) + 8 * (E + 1), "flops": 12 * T * H * F}
    if op in ("norm", "norm_backward"):
        T, H = case["rows"], case["hidden"]
        rb, bb = (2 if case[k] == "bf16" else 4 for k in ("residual", "branch"))
        gate = {"none": 0, "shared": bb * H, "rows": bb * T * H}[case["gate"]]
        if op == "norm":
            return {"bytes": T * H * (2 * rb + 2 * bb) + gate + 2 * H * bb + 8 * T, "flops": 10 * T * H}
        return {"bytes": T * H * (3 * rb + 3 * bb) + 2 * gate + 4 * H * bb + 8 * T, "flops": 24 * T * H}
    T, V = case["rows"], case["vocab"]
    size = 2 if case["type"] == "bf16" else 4
    if op == "logprobs":
        return {"bytes": T * V * size + 20 * T + 12 * T * case["top"], "flops": 5 * T * V}
    return {"bytes": 2 * T * V * size + 24 * T, "flops": 7 * T * V}


# ---------------------------------------------------------------------------- 64 bits
def _exact_act(g, kind):
    if kind == "silu":
        return torch.nn.functional.silu(g)
    return torch.nn.functional.gelu(g, approximate="tanh")


def _exact_ffn(s, backward):
    """Expert by expert, gradients by automatic differentiation of the definition."""
    c = s["case"]
    names = ("dx", "dw1", "dw3", "dw2") if backward else ("y", "gate", "up") if c["keep"] else ("y",)
    parts = {n: [] for n in names}
    start = 0
    for e, n in enumerate(group_sizes(c)):
        rows = slice(start, start + n)
        start += n
        x, w1, w3, w2 = s["x"][rows].double(), s["w1"][e].double(), s["w3"][e].double(), s["w2"][e].double()
        if not backward:
            g, u = x @ w1, x @ w3
            got = {"y": (_exact_act(g, c["act"]) * u) @ w2, "gate": g, "up": u}
        else:
            g = s["gate"][rows].double().requires_grad_()
            u = s["up"][rows].double().requires_grad_()
            with torch.enable_grad():
                h = _exact_act(g, c["act"]) * u
            dy = s["dy"][rows].double()
            dg, du = torch.autograd.grad(h, (g, u), dy @ w2.T)
            got = {"dx": dg @ w1.T + du @ w3.T, "dw1": x.T @ dg, "dw3": x.T @ du, "dw2": h.detach().T @ dy}
        for k in names:
            parts[k].append(got[k] if k in ("y", "gate", "up", "dx") else got[k].float()[None])
    return {k: torch.cat(v) for k, v in parts.items()}


def _rms(v, eps):
    return v / (v.square().mean(-1, keepdim=True) + eps).sqrt()


def _exact_norm(s):
    b, r = s["block"].double(), s["residual"].double()
    gate = 1.0 if s["gate"] is None else s["gate"].double()
    r = r + s["scale"] * gate * _rms(b, EPS) * s["w_post"].double()
    return {"residual": r, "normed": _rms(r, EPS) * s["w_pre"].double(),
            "rstd_post": (b.square().mean(1) + EPS).pow(-0.5), "rstd_pre": (r.square().mean(1) + EPS).pow(-0.5)}


def _exact_norm_backward(s):
    """The given reciprocal norms hold, so they enter the definition as what they are functions of."""
    H = s["block"].shape[1]
    r, b = s["residual"].double(), s["block"].double()
    p, q = s["rstd_pre"].double()[:, None], s["rstd_post"].double()[:, None]
    w_pre, w_post = s["w_pre"].double(), s["w_post"].double()
    dy = s["dnormed"].double()
    # d(r p)/dr with dp/dr = -p^3 r / H
    along = (dy * w_pre * r).sum(1, keepdim=True)
    dr = s["dresidual"].double() + dy * w_pre * p - p ** 3 * r * along / H
    gate = torch.ones_like(w_post) if s["gate"] is None else s["gate"].double()
    out = {"dresidual": dr, "dw_pre": torch.einsum("th,th,t->h", dy, r, p[:, 0])}
    per = s["scale"] * dr * b * q
    out["dw_post"] = (per * gate).sum(0)
    if s["gate"] is not None:
        out["dgate"] = per * w_post if s["gate"].dim() == 2 else (per * w_post).sum(0)
    up = s["scale"] * dr * gate * w_post
    out["dblock"] = q * up - q ** 3 * b * (up * b).sum(1, keepdim=True) / H
    return out


def _exact_logprobs(s):
    parts = []
    for rows in torch.arange(len(s["tokens"]), device="cuda").split(1024):
        x, tokens = s["logits"][rows].double(), s["tokens"][rows]
        logp = torch.log_softmax(x, 1)
        p = logp.exp()
        out = {"logp": torch.where(tokens >= 0, logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0], 0.0),
               "entropy": -torch.special.xlogy(p, p).sum(1), "lse": torch.logsumexp(x, 1)}
        if s["case"]["top"]:
            out |= {"top_ids": None, "top_logp": logp.topk(s["case"]["top"], 1).values}
        parts.append(out)
    return {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_logprobs_backward(s):
    parts = []
    for rows in torch.arange(len(s["tokens"]), device="cuda").split(1024):
        x, tokens = s["logits"][rows].double(), s["tokens"][rows]
        lse, ent = s["lse"][rows].double()[:, None], s["entropy"][rows].double()[:, None]
        dlogp = torch.where(tokens >= 0, s["dlogp"][rows], 0.0).double()[:, None]
        p = (x - lse).exp()
        hot = torch.zeros_like(x).scatter_(1, tokens.clamp(min=0)[:, None], 1.0)
        slope = torch.special.xlogy(p, p) + p * ent
        parts.append((dlogp * (hot - p) - s["dentropy"][rows].double()[:, None] * slope).float())
    return {"dlogits": torch.cat(parts)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("ffn", "ffn_backward"):
        return _exact_ffn(s, op == "ffn_backward")
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "logprobs": _exact_logprobs,
            "logprobs_backward": _exact_logprobs_backward}[op](s)
