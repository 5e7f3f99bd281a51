"""Plain 64-bit forms of the draft-training calls and the error bounds that
their 32-bit evaluation allows, shared by the tests of those calls."""
import math

import torch

U32 = 2.0 ** -24  # half a step of fp32
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def top_ref(logits, M, T):
    """tokens, values, lse, tail of every row, in 64 bits (rows without NaN)."""
    x = logits.double()
    order = x.sort(dim=-1, descending=True, stable=True)
    tokens = order.indices[..., :M]
    z = x / T
    return tokens.int(), order.values[..., :M], torch.logsumexp(z, -1), \
        torch.logsumexp(z.scatter(-1, tokens, -math.inf), -1)


def teacher_weights(values, tail, T, absent=None):
    t = values.double() / T
    if absent is not None:
        t = t.masked_fill(absent, -math.inf)
    last = tail.double() if tail is not None else torch.full_like(t[..., 0], -math.inf)
    p = torch.softmax(torch.cat([t, last[..., None]], -1), -1)
    return p[..., :-1], p[..., -1]


def distill_ref(logits, tokens, values, tail, T, scale=None):
    """loss, gradient, and what the bounds need: q_tail, p_tail, softmax over the tail."""
    z = logits.double() / T
    absent = tokens < 0
    ids = tokens.long().clamp(min=0)
    p, p_tail = teacher_weights(values, tail, T, absent)
    q = torch.softmax(z, -1)
    hit = torch.zeros_like(z)
    hit.scatter_add_(-1, ids, (~absent).double())
    rest = torch.where(hit > 0, torch.zeros_like(q), q)
    q_tail = rest.sum(-1)
    log_q = torch.log_softmax(z, -1).gather(-1, ids)
    log_q_tail = torch.logsumexp(torch.where(hit > 0, torch.full_like(z, -math.inf), z), -1) - torch.logsumexp(z, -1)
    loss = torch.where(p > 0, p * (p.log() - log_q), torch.zeros_like(p)).sum(-1)
    loss = loss + torch.where(p_tail > 0, p_tail * (p_tail.log() - log_q_tail), torch.zeros_like(p_tail))
    target = torch.zeros_like(z).scatter_add_(-1, ids, torch.where(absent, torch.zeros_like(p), p))
    share = rest / q_tail[..., None].clamp(min=1e-300)
    grad = torch.where(hit > 0, q - target, share * (q_tail - p_tail)[..., None])
    w = (torch.ones_like(loss) if scale is None else scale.double()) / T
    return loss, grad * w[..., None], {"q": q, "q_tail": q_tail, "p_tail": p_tail, "share": share, "hit": hit > 0, "w": w}


def sum_error(V, dtype, depth=24.0):
    """Bound of the relative error of a sum of exponentials formed in 32 bits:
    a thread adds at most 13000 / 256 vectors of a slice one after the other (a
    slice is at most 200 KB; rows below 66 KB per slice give fewer), each term
    carries the rounding of its argument (at most `depth` * log2(e) in size
    where it matters, rounded twice) and two units of the exponential."""
    per_vec = 8 if dtype == torch.bfloat16 else 4
    size = 2 if dtype == torch.bfloat16 else 4
    slices = max(1, min(8, math.ceil(V * size / (66 * 1024))))
    chain = math.ceil(V / slices / per_vec / 256) * per_vec + 8
    return (chain + 2 * depth * 1.4427 + 8) * U32


def logits_like(shape, V, dtype, seed, spread=2.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(*shape, V, generator=g, device=device) * spread).to(dtype)


def linear_case(shape, D, V, seed, keep=1.0, device="cuda"):
    """hidden [*shape, D], weight [V, D] and targets, some of them left out."""
    g = torch.Generator(device=device).manual_seed(seed)
    weight = (torch.randn(V, D, generator=g, device=device) * (2.0 / math.sqrt(D))).bfloat16()
    hidden = torch.randn(*shape, D, generator=g, device=device).bfloat16()
    targets = torch.randint(0, V, shape, generator=g, device=device, dtype=torch.int32)
    if keep < 1.0:
        targets[torch.rand(*shape, generator=g, device=device) >= keep] = -1
    return hidden, weight, targets


def linear_ref(hidden, weight, targets, scale=None):
    """loss, lse, gradients in 64 bits, and bounds of each for products summed
    in 32 bits by matrix instructions of 16 k (every step truncated: 2^-23 of
    the running sum, at most D / 16 + 16 steps), G rounded to bf16, results
    rounded once."""
    lead = hidden.shape[:-1]
    h, w, y = hidden.reshape(-1, hidden.shape[-1]).double(), weight.double(), targets.reshape(-1).long()
    on = y >= 0
    s = on.double() if scale is None else scale.reshape(-1).double() * on
    on = on & (s != 0) if scale is not None else on
    h = torch.where(on[:, None], h, torch.zeros_like(h))
    z = h @ w.T
    D, V, N = h.shape[1], w.shape[0], h.shape[0]
    dz = ((D / 16 + 16) * 2.0 ** -23 * (h.abs() @ w.abs().T)).amax(1)
    lse = torch.logsumexp(z, 1)
    at = y.clamp(min=0)[:, None]
    zero = torch.zeros_like(lse)
    loss = torch.where(on, lse - z.gather(1, at)[:, 0], zero)
    # a tile's thread adds 8 sums of 8 terms; tiles are joined with one exponential each
    e = (2 * 24 * 1.4427 + 64) * U32
    lse_tol = dz + e + lse.abs() * U32
    loss_tol = 2 * dz + e + loss.abs() * U32
    p = (z - lse[:, None]).exp()
    G = p.scatter_add(1, at, torch.full_like(lse, -1.0)[:, None]) * s[:, None]
    # the exponent's argument carries z, lse and a rounding of each (|z| + |lse| below 2^7 here)
    dG = p * s.abs()[:, None] * (dz + lse_tol + 2.0 ** 7 * 2 * U32)[:, None] + (G.abs() + 1e-38) * 2.0 ** -8
    dh, dw = G @ w, G.T @ h
    acc_h = (V / 16 + 96) * 2.0 ** -23 * (G.abs() @ w.abs())
    acc_w = (N / 16 + 16) * 2.0 ** -23 * (G.abs().T @ h.abs())
    dh_tol = dG @ w.abs() + acc_h + dh.abs() * 2.0 ** -8 + 1e-38
    dw_tol = dG.T @ h.abs() + acc_w + dw.abs() * 2.0 ** -8 + 1e-38
    lse = torch.where(on, lse, zero)
    r = dict(loss=loss, lse=lse, loss_tol=loss_tol, lse_tol=lse_tol)
    r = {k: v.reshape(lead) for k, v in r.items()}
    r.update(dh=dh.reshape(hidden.shape), dw=dw, dh_tol=dh_tol.reshape(hidden.shape), dw_tol=dw_tol,
             on=on.reshape(lead))
    return r
