"""One training step of a draft next to one verify step: the drafts are
verified, the target's top logits kept, the draft's logits distilled on them
and its head trained on the verified tokens; the gradients against automatic
differentiation in 64 bits."""
import os
import subprocess
import sys

import pytest
import torch

from speculative_decoding_verify_ssd_b200 import binding as ssd

from train_testlib import linear_case, logits_like, sum_error

B, K, V, D, M = 6, 5, 8003, 256, 32


def step(target, hidden, weight, uniforms, drafts, alpha, scale):
    """The calls of one step; hidden [B, K, D] feeds the head that made the draft logits."""
    draft = (hidden.reshape(-1, D) @ weight.t()).view(B, K, V)
    r = ssd.ssd_verify(target, draft, drafts, uniforms, 1.0, alpha=alpha, C_coef=0.5, budget=16, cache=True)
    top = ssd.ssd_teacher_top(target[:, :K], M)
    dis = ssd.ssd_distill(draft, top.tokens, top.values, top.tail, row_scale=scale)
    y = r.out_tokens[:, :K].contiguous()          # accepted drafts, the bonus, then -1
    ce = ssd.ssd_linear_ce(hidden, weight, y)
    dh, dw = ssd.ssd_linear_ce_grad(hidden, weight, y, ce.lse, row_scale=scale)
    return draft, r, top, dis, y, ce, dh, dw


def inputs(seed):
    hidden, weight, _ = linear_case((B, K), D, V, seed)
    target = logits_like((B, K + 1), V, torch.bfloat16, seed + 1)
    near = (hidden.reshape(-1, D) @ weight.t()).view(B, K, V)
    target[:, :K] += near                          # a target that the draft resembles
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    drafts = torch.softmax(near.float(), -1).view(-1, V).multinomial(1, generator=g).view(B, K).int()
    return dict(target=target, hidden=hidden, weight=weight,
                uniforms=torch.rand(B, K + 1, generator=g, device="cuda") * 0.999, drafts=drafts,
                alpha=torch.full((B,), 0.6, device="cuda"),
                scale=torch.rand(B, K, generator=g, device="cuda") + 0.5)


@pytest.mark.gpu
def test_step_gradients():
    x = inputs(100)
    draft, r, top, dis, y, ce, dh, dw = step(**x)
    torch.cuda.synchronize()
    assert (r.status & ssd.ROW_INVALID == 0).all()
    for s in (top.status, dis.status, ce.status):
        assert (s & ssd.ROW_INVALID == 0).all()
    assert (y[:, 0] >= 0).all() and (y < 0).any()  # some rows end before K
    scale = x["scale"].double()

    # the divergence with the target's tail as one event, from the definition
    z = draft.double().requires_grad_(True)
    p = torch.softmax(x["target"][:, :K].double(), -1)
    q = torch.softmax(z, -1)
    ids = top.tokens.long()
    ps, qs = p.gather(-1, ids), q.gather(-1, ids)
    pt, qt = 1 - ps.sum(-1), 1 - qs.sum(-1)
    loss = (ps * (ps / qs).log()).sum(-1) + pt * (pt / qt).log()
    (loss * scale).sum().backward()
    e = sum_error(V, torch.bfloat16)
    # the kept values are the bf16 logits themselves; the tail's logarithm is rounded to fp32
    tol = 2 * e + 2 * 16 * 2.0 ** -24
    assert ((dis.loss.double() - loss).abs() <= tol + loss.abs() * 2.0 ** -24).all()
    err = (dis.grad.double() - z.grad).abs()
    assert (err <= z.grad.abs() * (2.0 ** -8 + 4 * tol) + 4 * tol * q.detach() * scale[..., None] + 1e-30).all()

    h = x["hidden"].double().requires_grad_(True)
    w = x["weight"].double().requires_grad_(True)
    on = y >= 0
    logp = torch.log_softmax(h[on] @ w.t(), -1)
    nll = -logp.gather(1, y[on].long()[:, None])[:, 0]
    (nll * scale[on]).sum().backward()
    # fp32 sums of 256 products of magnitude below 8 * 0.6: far below 1e-4
    assert ((ce.loss[on].double() - nll).abs() <= 1e-4).all() and (ce.loss[~on] == 0).all()
    assert (dh[~on] == 0).all()
    # G to bf16 (2^-8 of each term), then one rounding of the result
    p = logp.exp().detach()
    G = p.scatter_add(1, y[on].long()[:, None], -torch.ones_like(nll)[:, None]).abs() * scale[on][:, None]
    assert ((dh[on].double() - h.grad[on]).abs() <=
            1.1 * 2.0 ** -8 * (G @ w.detach().abs() + h.grad[on].abs()) + 1e-6).all()
    assert ((dw.double() - w.grad).abs() <=
            1.1 * 2.0 ** -8 * (G.t() @ h.detach()[on].abs() + w.grad.abs()) + 1e-6).all()


@pytest.mark.gpu
def test_step_captured():
    """The whole step as one graph, replayed on another batch: the bits of the eager step."""
    x = inputs(200)
    step(**x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(**x)
    for k, v in inputs(300).items():
        x[k].copy_(v)
    g.replay()
    torch.cuda.synchronize()
    again = step(**x)
    torch.cuda.synchronize()
    _, r, top, dis, y, ce, dh, dw = out
    _, r2, top2, dis2, y2, ce2, dh2, dw2 = again
    for a, b in ((r.out_tokens, r2.out_tokens), (top.tokens, top2.tokens), (top.tail, top2.tail),
                 (dis.loss, dis2.loss), (dis.grad, dis2.grad), (y, y2), (ce.loss, ce2.loss), (dh, dh2), (dw, dw2)):
        assert torch.equal(a, b)


FIRST = """
import sys, torch
sys.path[:0] = [%r, %r]
import test_train_together as t
from speculative_decoding_verify_ssd_b200 import binding as ssd
x = t.inputs(400)
draft = (x["hidden"].reshape(-1, t.D) @ x["weight"].t()).view(t.B, t.K, t.V)
y = x["drafts"]
torch.cuda.synchronize()
def calls():
    top = ssd.ssd_teacher_top(x["target"][:, :t.K], t.M)
    dis = ssd.ssd_distill(draft, top.tokens, top.values, top.tail, row_scale=x["scale"])
    ce = ssd.ssd_linear_ce(x["hidden"], x["weight"], y)
    return (top.tokens, dis.loss, dis.grad, ce.loss) + ssd.ssd_linear_ce_grad(x["hidden"], x["weight"], y, ce.lse)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = calls()
g.replay()
torch.cuda.synchronize()
for a, b in zip(out, calls()):
    assert torch.equal(a, b)
print("first calls captured")
"""


@pytest.mark.gpu
def test_first_calls_in_a_capture():
    """A process whose first training calls are captured."""
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST % (here, os.path.dirname(here))], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "first calls captured" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
