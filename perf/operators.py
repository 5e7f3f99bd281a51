"""The draft-training operators: their plain forms, the library's calls, and
the cases they are timed on.

Three families over the same vocabularies as the verify step: the top logits
of target rows with the mass left outside them (`top`), the distillation loss
of draft rows against such a teacher with its gradient (`distill`), and the
cross entropy of a linear head with its gradients (`ce`)."""
import math

import torch

own = False


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def _top(name, B, K, V, M, dtype, T, view):
    return {"name": name, "op": "top", "B": B, "K": K, "V": V, "M": M, "dtype": dtype, "T": T, "view": view}


def _distill(name, B, K, V, M, dtype, T, tail, grad):
    return {"name": name, "op": "distill", "B": B, "K": K, "V": V, "M": M, "dtype": dtype, "T": T, "tail": tail,
            "grad": grad}


def _ce(name, N, D, V, keep, grad):
    return {"name": name, "op": "ce", "N": N, "D": D, "V": V, "keep": keep, "grad": grad}


def listed():
    return [
        # one request, four drafts and the bonus position: a single small fp32 batch, where latency counts
        _top("top_b1_k4_v1024_fp32", 1, 4, 1024, 8, "fp32", 1.0, False),
        # a serving batch at the verify step: the K draft positions of the target's [B, K+1, V] logits
        _top("top_b64_k6_v128256_bf16", 64, 6, 128256, 64, "bf16", 1.0, True),
        # a smaller vocabulary with an odd size (rows start at any element), temperature below one
        _top("top_b16_k5_v32003_fp32", 16, 5, 32003, 33, "fp32", 0.7, True),
        # the smallest distillation: one request, loss and gradient
        _distill("distill_b1_k4_v1024_fp32", 1, 4, 1024, 8, "fp32", 1.0, True, True),
        # online distillation on the drafts of one verify step: loss and gradient
        _distill("distill_b64_k6_v128256_bf16", 64, 6, 128256, 64, "bf16", 1.0, True, True),
        # evaluation of a draft: loss alone, odd vocabulary, renormalised top (no tail)
        _distill("distill_b16_k5_v32003_loss", 16, 5, 32003, 33, "bf16", 2.0, False, False),
        # the largest distillation batch
        _distill("distill_b256_k8_v151936_bf16", 256, 8, 151936, 128, "bf16", 1.0, True, True),
        # a draft head on one request's accepted tokens: few rows, odd sizes, loss and gradients
        _ce("ce_n5_d512_v5003", 5, 512, 5003, 0.8, True),
        # the accepted tokens of one verify step over the full vocabulary: the weight's bytes bound it
        _ce("ce_n64_d2048_v128256", 64, 2048, 128256, 0.7, True),
        # evaluation of a head: loss alone
        _ce("ce_n1000_d1024_v32000_loss", 1000, 1024, 32000, 1.0, False),
        # a training batch with prompts masked out
        _ce("ce_n1111_d1024_v32000", 1111, 1024, 32000, 0.6, True),
        # the largest training batch of a small draft's head
        _ce("ce_n4096_d2048_v128256", 4096, 2048, 128256, 1.0, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["top", "distill", "ce"])
    if op == "ce":
        N, V = _log_int(rng, 1, 4096), _log_int(rng, 1000, 128256)
        D = 8 * _log_int(rng, 32, 256)
        return {"op": "ce", "N": N, "D": D, "V": V, "keep": round(rng.uniform(0.5, 1.0), 2), "grad": rng.random() < 0.7}
    B, K, V = _log_int(rng, 1, 256), rng.randint(1, 8), _log_int(rng, 1000, 151936)
    M = min(_log_int(rng, 1, 128), V)
    case = {"op": op, "B": B, "K": K, "V": V, "M": M, "dtype": rng.choice(["bf16", "fp32"]),
            "T": rng.choice([0.6, 0.7, 1.0, 1.5])}
    if case["dtype"] == "fp32":
        case["B"] = max(1, B // 2)
    if op == "top":
        case["view"] = rng.random() < 0.5
    else:
        case["M"] = max(8, M)
        case["tail"], case["grad"] = rng.random() < 0.7, rng.random() < 0.7
    return case


def work(case):
    if case["op"] == "ce":
        n = max(1, round(case["N"] * case["keep"]))
        pair = 2.0 * n * case["V"] * case["D"]
        read = 2.0 * (n + case["V"]) * case["D"]
        if not case["grad"]:
            return {"bytes": read + 8.0 * case["N"], "flops": pair}
        return {"bytes": read + 2.0 * (case["N"] + case["V"]) * case["D"] + 8.0 * case["N"], "flops": 3 * pair}
    rows, s = case["B"] * case["K"], 2 if case["dtype"] == "bf16" else 4
    stream = float(rows) * case["V"] * s
    if case["op"] == "top":
        return {"bytes": stream + rows * (8.0 * case["M"] + 8), "flops": 4.0 * rows * case["V"]}
    passes = 2 if case["grad"] else 1
    return {"bytes": passes * stream + rows * (8.0 * case["M"] + 12), "flops": 4.0 * passes * rows * case["V"]}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _zipf_rows(shape, V, g):
    """Logits whose values fall like the logarithm of a rank, in random token order."""
    rank = torch.rand(*shape, V, generator=g, device="cuda").mul_(V).add_(1)
    return rank.log_().neg_().add_(torch.randn(*shape, V, generator=g, device="cuda"), alpha=0.3).add_(8.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "ce":
        N, D, V = case["N"], case["D"], case["V"]
        weight = (torch.randn(V, D, generator=g, device="cuda") * 0.02).bfloat16()
        target = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        # the hidden states lean towards their targets' rows, as those of a trained draft do
        hidden = torch.randn(N, D, generator=g, device="cuda")
        hidden += weight[target.long()].float() * torch.rand(N, 1, generator=g, device="cuda") * (250.0 / math.sqrt(D))
        order = torch.rand(N, generator=g, device="cuda").argsort()
        kept = max(1, round(N * case["keep"]))
        target[order[kept:]] = -1
        scale = torch.full((N,), 1.0 / kept, device="cuda")
        return {"case": case, "hidden": hidden.bfloat16(), "weight": weight, "target": target, "scale": scale}
    B, K, V, M = case["B"], case["K"], case["V"], case["M"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["op"] == "top":
        if case["view"]:
            logits = _zipf_rows((B, K + 1), V, g).to(dtype)[:, :K]
        else:
            logits = _zipf_rows((B, K), V, g).to(dtype)
        return {"case": case, "logits": logits}
    teacher = _zipf_rows((B, K), V, g)
    draft = (teacher + torch.randn(B, K, V, generator=g, device="cuda") * 0.77).to(dtype)
    values, tokens = teacher.topk(M, dim=-1)
    tail = teacher.double().div_(case["T"]).scatter_(-1, tokens, -math.inf).logsumexp(-1).float() if case["tail"] else None
    scale = torch.rand(B, K, generator=g, device="cuda") / (B * K)
    return {"case": case, "logits": draft, "tokens": tokens.int().contiguous(), "values": values.contiguous(),
            "tail": tail, "scale": scale}


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------
def _lse(x):
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    return (x - top).exp().sum(-1).log() + top.squeeze(-1)


def _plain_top(state):
    case, x = state["case"], state["logits"].float()
    ordered, index = x.sort(dim=-1, descending=True, stable=True)
    tokens = index[..., : case["M"]]
    scaled = x / case["T"]
    return {"tokens": tokens.int(), "values": ordered[..., : case["M"]].contiguous(), "lse": _lse(scaled),
            "tail": _lse(scaled.scatter(-1, tokens, -math.inf))}


def _lse64(x, T):
    """log sum exp(x / T): the exponentials in 32 bits, their sum and its logarithm in 64,
    since the loss below is a small difference of such logarithms."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    return ((x - top) / T).exp().sum(-1, dtype=torch.float64).log() + top.squeeze(-1).double() / T


def _plain_distill(state):
    case, T = state["case"], state["case"]["T"]
    z, tokens = state["logits"].float(), state["tokens"].long()
    atoms = state["values"].double() / T
    tail = state["tail"].double() if state["tail"] is not None else torch.full_like(atoms[..., 0], -math.inf)
    log_p = torch.cat([atoms, tail.unsqueeze(-1)], -1)
    log_p = log_p - _lse(log_p).unsqueeze(-1)
    total, rest = _lse64(z, T), _lse64(z.scatter(-1, tokens, -math.inf), T)
    log_q = torch.cat([z.gather(-1, tokens).double() / T, rest.unsqueeze(-1)], -1) - total.unsqueeze(-1)
    p = log_p.exp()
    loss = torch.where(p > 0, p * (log_p - log_q), torch.zeros_like(p)).sum(-1).float()
    if not case["grad"]:
        return {"loss": loss}
    weight = (state["scale"] / T).unsqueeze(-1)
    inside = (log_q[..., :-1].exp() - p[..., :-1]).float() * weight
    outside = (log_q[..., -1].exp() - p[..., -1]).float().unsqueeze(-1) * weight
    grad = ((z - T * rest.float().unsqueeze(-1)) / T).exp() * outside
    return {"loss": loss, "grad": grad.scatter(-1, tokens, inside).to(state["logits"].dtype)}


def _plain_ce(state):
    target = state["target"].long()
    kept, at = target >= 0, target.clamp(min=0).unsqueeze(-1)
    hidden, weight = state["hidden"].float(), state["weight"].float()
    logits = hidden @ weight.T
    lse = _lse(logits)
    zero = torch.zeros_like(lse)
    loss = torch.where(kept, lse - logits.gather(-1, at).squeeze(-1), zero)
    if not state["case"]["grad"]:
        return {"loss": loss}
    grad = (logits - lse.unsqueeze(-1)).exp()
    grad.scatter_add_(-1, at, torch.full_like(at, -1.0, dtype=torch.float32))
    grad *= torch.where(kept, state["scale"], zero).unsqueeze(-1)
    return {"loss": loss, "grad_hidden": (grad @ weight).bfloat16(), "grad_weight": (grad.T @ hidden).bfloat16()}


def run(state):
    op = state["case"]["op"]
    if own:
        from speculative_decoding_verify_ssd_b200 import binding as ssd

        if op == "top":
            r = ssd.ssd_teacher_top(state["logits"], state["case"]["M"], state["case"]["T"])
            return {"tokens": r.tokens, "values": r.values, "lse": r.lse, "tail": r.tail}
        if op == "distill":
            r = ssd.ssd_distill(state["logits"], state["tokens"], state["values"], state["tail"], state["case"]["T"],
                                row_scale=state["scale"], with_grad=state["case"]["grad"])
            return {"loss": r.loss, "grad": r.grad} if state["case"]["grad"] else {"loss": r.loss}
        r = ssd.ssd_linear_ce(state["hidden"], state["weight"], state["target"])
        if not state["case"]["grad"]:
            return {"loss": r.loss}
        grad_hidden, grad_weight = ssd.ssd_linear_ce_grad(state["hidden"], state["weight"], state["target"], r.lse,
                                                          row_scale=state["scale"])
        return {"loss": r.loss, "grad_hidden": grad_hidden, "grad_weight": grad_weight}
    return {"top": _plain_top, "distill": _plain_distill, "ce": _plain_ce}[op](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "ce":
        h, w, y = state["hidden"].double(), state["weight"].double(), state["target"].long()
        n = torch.arange(len(y), device="cuda")[y >= 0]
        log_q = torch.log_softmax(h[n] @ w.mT, dim=1)
        loss = torch.zeros(len(y), dtype=torch.float64, device="cuda")
        loss[n] = -log_q[torch.arange(len(n), device="cuda"), y[n]]
        if not case["grad"]:
            return {"loss": loss}
        G = log_q.exp_()
        G[torch.arange(len(n), device="cuda"), y[n]] -= 1
        G *= state["scale"].double()[n, None]
        dh = torch.zeros_like(h)
        dh[n] = G @ w
        return {"loss": loss, "grad_hidden": dh, "grad_weight": G.mT @ h[n]}
    z = state["logits"].double() / case["T"]
    if case["op"] == "top":
        kth = z.topk(case["M"], dim=-1).indices
        kept = state["logits"].double().topk(case["M"], dim=-1).values
        total = torch.logsumexp(z, -1)
        return {"tokens": None, "values": kept, "lse": total,
                "tail": torch.logsumexp(z.scatter(-1, kth, -math.inf), -1)}
    ids = state["tokens"].long()
    t = state["values"].double() / case["T"]
    if state["tail"] is not None:
        t = torch.cat([t, state["tail"].double()[..., None]], -1)
    p = torch.softmax(t, -1)
    q = torch.softmax(z, -1)
    inside = torch.zeros_like(q, dtype=torch.bool).scatter_(-1, ids, True)
    q_tail = q.masked_fill(inside, 0).sum(-1, keepdim=True)
    q_atoms = torch.cat([q.gather(-1, ids), q_tail], -1)[..., : p.shape[-1]]
    loss = torch.xlogy(p, p / q_atoms).sum(-1)
    if not case["grad"]:
        return {"loss": loss}
    d = q.scatter_add(-1, ids, -p[..., : case["M"]])
    if state["tail"] is not None:
        d -= torch.where(inside, 0.0, q / q_tail * p[..., case["M"]:])
    return {"loss": loss, "grad": d * (state["scale"].double() / case["T"])[..., None]}
