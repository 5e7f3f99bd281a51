"""ssd_linear_ce and ssd_linear_ce_grad against plain 64-bit forms: sizes from
one row on, odd vocabularies, pieces, left-out and void rows, strides, capture
and streams."""
import ctypes as C
import math

import pytest
import torch

from speculative_decoding_verify_ssd_b200 import binding as ssd

from train_testlib import linear_case, linear_ref

BF16 = torch.bfloat16


def _ce(L, **kw):
    a = dict(hidden=None, weight=None, dtype=1, nb=2, rpb=3, D=16, V=100, bs=48, rs=16, ws=16, work=None, n=0)
    a.update(kw)
    return L.ssd_linear_ce(a["hidden"], a["weight"], a["dtype"], a["nb"], a["rpb"], a["D"], a["V"], a["bs"], a["rs"],
                           a["ws"], a.get("y"), a.get("y"), a.get("y"), a.get("y"), a["work"], a["n"], None)


def _ce_grad(L, **kw):
    a = dict(hidden=None, weight=None, dtype=1, nb=2, rpb=3, D=16, V=100, bs=48, rs=16, ws=16, work=None, n=0)
    a.update(kw)
    return L.ssd_linear_ce_grad(a["hidden"], a["weight"], a["dtype"], a["nb"], a["rpb"], a["D"], a["V"], a["bs"],
                                a["rs"], a["ws"], a.get("y"), a.get("y"), None, a.get("y"), a.get("y", C.c_void_p(4096)),
                                None, a["work"], a["n"], None)


@pytest.mark.parametrize("call", [_ce, _ce_grad])
def test_host_refusals(call):
    L = ssd.load()
    assert call(L, dtype=0) == 2 and call(L, dtype=9) == 2
    for bad in (dict(nb=-1), dict(rpb=-1), dict(D=0), dict(D=12), dict(D=1 << 17), dict(V=0), dict(V=1 << 25),
                dict(nb=1 << 11, rpb=1 << 10), dict(bs=4), dict(rs=-8), dict(rs=12), dict(ws=8), dict(ws=20)):
        assert call(L, **bad) == 1, bad
    assert call(L) == 1                                                     # NULL arrays
    p, odd = C.c_void_p(4096), C.c_void_p(4098)
    assert call(L, hidden=odd, weight=p, y=p) == 3
    assert call(L, hidden=p, weight=odd, y=p) == 3
    assert call(L, hidden=p, weight=p, y=p, work=C.c_void_p(4096 + 16), n=1 << 30) == 3
    assert call(L, hidden=p, weight=p, y=p) == 4                            # no workspace
    assert call(L, hidden=p, weight=p, y=p, work=p, n=1000) == 4


def test_host_sizes():
    L = ssd.load()
    assert _ce(L, nb=0) == 0
    for bad in ((-1, 16, 10), (1, 12, 10), (1, 0, 10), (1, 16, 0), ((1 << 20) + 1, 16, 10)):
        assert L.ssd_linear_ce_workspace_bytes(*bad, 0) == 0 and L.ssd_linear_ce_workspace_bytes(*bad, 1) == 0
    # the logits of N rows are never kept: the forward call holds two words per row and 256 of them
    n, D, V = 4096, 2048, 128256
    assert L.ssd_linear_ce_workspace_bytes(n, D, V, 0) < n * (2 * D + 16) + n * V // 16
    assert L.ssd_linear_ce_workspace_bytes(n, D, V, 1) < n * V


def test_reference_gradient_against_differences():
    hidden, weight, targets = linear_case((3,), 8, 11, 1, device="cpu")
    targets[1] = -1
    scale = torch.tensor([0.5, 2.0, 1.5])
    r = linear_ref(hidden, weight, targets, scale)
    step = 2.0 ** -6      # exactly added to these bf16 values in 64 bits

    def total(h, w):
        return float((linear_ref(h, w, targets, scale)["loss"] * scale.double()).sum())

    h, w = hidden.double(), weight.double()
    # central differences: step^2 / 6 of a third derivative below 8 |w|^3 scale
    for (x, grad) in ((h, r["dh"]), (w, r["dw"])):
        for i in (0, 5, x.numel() - 1):
            d = torch.zeros_like(x).view(-1)
            d[i] = step
            d = d.view_as(x)
            up, down = (total(h + s * d, w) if x is h else total(h, w + s * d) for s in (1, -1))
            assert abs((up - down) / (2 * step) - float(grad.view(-1)[i])) < 100 * step * step


def check(hidden, weight, targets, scale=None, **kw):
    r = ssd.ssd_linear_ce(hidden, weight, targets)
    st = torch.full(targets.shape, 77, dtype=torch.int32, device="cuda")
    dh, dw = ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse, row_scale=scale, status=st, **kw)
    torch.cuda.synchronize()
    f = linear_ref(hidden, weight, targets)
    b = linear_ref(hidden, weight, targets, scale) if scale is not None else f
    assert (r.status == 0).all() and (st == 0).all()
    assert (r.loss[~f["on"]] == 0).all() and (r.lse[~f["on"]] == 0).all()
    for name, got in (("lse", r.lse), ("loss", r.loss)):
        d = (got.double() - f[name]).abs()
        assert (d <= f[name + "_tol"])[f["on"]].all(), (name, float(d.max()))
    for name, got in (("dh", dh), ("dw", dw)):
        d = (got.double() - b[name]).abs()
        assert (d <= b[name + "_tol"]).all(), (name, float((d - b[name + "_tol"]).max()))
    assert (dh[~b["on"]] == 0).all()
    return r, dh, dw


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 2, 31, 33, 127, 128, 129, 257, 300])
@pytest.mark.parametrize("D,V", [(8, 1), (8, 300), (72, 7), (64, 256), (136, 257), (512, 5003)])
def test_sizes(N, D, V):
    check(*linear_case((N,), D, V, N + D + V))


@pytest.mark.gpu
@pytest.mark.parametrize("N,D,V", [(5, 2048, 32003), (64, 1024, 128256), (1000, 256, 20011), (640, 2048, 4096),
                                    (3, 8192, 1025)])
def test_larger(N, D, V):
    hidden, weight, targets = linear_case((N,), D, V, N, keep=0.7)
    check(hidden, weight, targets, torch.rand(N, device="cuda") + 0.5)


@pytest.mark.gpu
def test_scales():
    """Signs, magnitudes far apart, and one scale for all: what is largest sets the common factor."""
    hidden, weight, targets = linear_case((150,), 72, 400, 19)
    g = torch.Generator(device="cuda").manual_seed(20)
    check(hidden, weight, targets, torch.randn(150, generator=g, device="cuda"))
    check(hidden, weight, targets, -torch.rand(150, generator=g, device="cuda") * 1e-6)
    check(hidden, weight, targets, 10.0 ** torch.randint(-12, 5, (150,), generator=g, device="cuda").float())
    same = torch.full((150,), 1.0 / 37, device="cuda")
    r = ssd.ssd_linear_ce(hidden, weight, targets)
    one, scaled = (ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse, row_scale=s) for s in (None, same))
    for a, b in zip(one, scaled):    # the same sums, times 1/37, rounded: a bf16 step of each at most
        assert ((a.double() / 37 - b.double()).abs() <= 2.0 ** -7 * b.double().abs() + 1e-38).all()


@pytest.mark.gpu
def test_pieces():
    """More rows than one piece of the vocabulary holds the logits of."""
    N, D, V = 5000, 64, 60001
    hidden, weight, targets = linear_case((N,), D, V, 3, keep=0.8)
    check(hidden, weight, targets, torch.rand(N, device="cuda") / N)


@pytest.mark.gpu
def test_left_out_rows():
    """Padding in every place, all rows left out, scale 0; what those rows hold does not matter."""
    hidden, weight, targets = linear_case((4, 70), 128, 1000, 5, keep=0.5)
    targets[1] = -1
    targets[3, 60:] = -100
    scale = torch.rand(4, 70, device="cuda")
    scale[0, ::3] = 0
    r, dh, dw = check(hidden, weight, targets, scale)
    dirty = hidden.clone()
    dirty[targets < 0] = math.nan
    r2 = ssd.ssd_linear_ce(dirty, weight, targets)
    dirty[scale == 0] = math.nan
    dh2, dw2 = ssd.ssd_linear_ce_grad(dirty, weight, targets, r.lse, row_scale=scale)
    assert torch.equal(r.loss, r2.loss) and torch.equal(dh, dh2) and torch.equal(dw, dw2)
    targets[:] = -1
    r = ssd.ssd_linear_ce(dirty, weight, targets)
    dh, dw = ssd.ssd_linear_ce_grad(dirty, weight, targets, r.lse)
    assert (r.loss == 0).all() and (dh == 0).all() and (dw == 0).all()


@pytest.mark.gpu
def test_void_rows():
    hidden, weight, targets = linear_case((200,), 64, 500, 7)
    good = torch.ones(200, dtype=torch.bool, device="cuda")
    hidden[3, 5] = math.nan
    hidden[150, 0] = math.inf
    targets[17] = 500
    targets[18] = 2 ** 31 - 1
    good[[3, 150, 17, 18]] = False
    r = ssd.ssd_linear_ce(hidden, weight, targets)
    st = torch.empty(200, dtype=torch.int32, device="cuda")
    dh, dw = ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse, status=st)
    want = torch.zeros(200, dtype=torch.int32, device="cuda")
    want[[3, 150]] = ssd.ROW_NONFINITE
    want[[17, 18]] = ssd.ROW_BAD_TOKEN
    assert torch.equal(r.status, want) and torch.equal(st, want)
    assert r.loss[~good].isnan().all() and r.lse[~good].isnan().all() and (dh[~good] == 0).all()
    only = torch.where(good, targets, torch.full_like(targets, -1))
    clean = torch.where(good[:, None], hidden, torch.zeros_like(hidden))
    f = linear_ref(clean, weight, only)
    assert ((r.loss.double() - f["loss"]).abs() <= f["loss_tol"])[good].all()
    assert ((dw.double() - f["dw"]).abs() <= f["dw_tol"]).all()
    assert ((dh.double() - f["dh"]).abs() <= f["dh_tol"]).all()


@pytest.mark.gpu
def test_same_target_everywhere_and_large_logits():
    hidden, weight, targets = linear_case((300,), 64, 777, 9)
    targets[:] = 776
    check(hidden, weight, targets)
    check(hidden * 4, weight * 4, targets)     # logits of some tens: most probabilities vanish


@pytest.mark.gpu
def test_views():
    """hidden without its last position, transposed batches, a weight that is a column slice."""
    hidden, weight, targets = linear_case((3, 50), 128, 600, 11)
    y = targets[:, 1:].contiguous()
    check(hidden[:, :-1], weight, y)
    check(hidden.transpose(0, 1), weight, targets.t().contiguous())
    check(hidden[:, :, 8:72], weight[:, 64:], targets)
    check(hidden[1, 4], weight, targets[1, 4])
    check(hidden[:1].expand(3, 50, 128), weight, targets)


@pytest.mark.gpu
def test_given_outputs_and_workspace():
    hidden, weight, targets = linear_case((65,), 136, 901, 13)
    n = max(ssd.linear_ce_workspace_bytes(65, 136, 901, g) for g in (False, True))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")     # NaN wherever it is read unwritten
    r = ssd.ssd_linear_ce(hidden, weight, targets, workspace=ws)
    ws.fill_(255)
    dh, dw = torch.full_like(hidden, 9.0), torch.full_like(weight, 9.0)
    out = ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse, grad_hidden=dh, grad_weight=dw, workspace=ws)
    assert out[0] is dh and out[1] is dw
    r2, dh2, dw2 = check(hidden, weight, targets)
    assert torch.equal(r.loss, r2.loss) and torch.equal(dh, dh2) and torch.equal(dw, dw2)


@pytest.mark.gpu
def test_binding_refusals():
    hidden, weight, targets = linear_case((6,), 16, 40, 15)
    lse = torch.zeros(6, device="cuda")
    for bad in (lambda: ssd.ssd_linear_ce(hidden.float(), weight, targets),
                lambda: ssd.ssd_linear_ce(hidden, weight[:, :8], targets),
                lambda: ssd.ssd_linear_ce(hidden, weight.t(), targets),
                lambda: ssd.ssd_linear_ce(hidden, weight, targets.long()),
                lambda: ssd.ssd_linear_ce(hidden, weight, targets[:5]),
                lambda: ssd.ssd_linear_ce(hidden.cpu(), weight, targets),
                lambda: ssd.ssd_linear_ce_grad(hidden, weight, targets, lse[:5]),
                lambda: ssd.ssd_linear_ce_grad(hidden, weight, targets, lse, row_scale=lse.double()),
                lambda: ssd.ssd_linear_ce_grad(hidden, weight, targets, lse, grad_weight=weight.float())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ssd.SsdError, match="workspace"):
        ssd.ssd_linear_ce(hidden, weight, targets, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ssd.SsdError):
        ssd.ssd_linear_ce(hidden[:, :12], weight[:, :12], targets)
    with pytest.raises(ssd.SsdError, match="misaligned"):
        ssd.ssd_linear_ce(hidden[:, 4:12], weight[:, :8], targets)
    e = ssd.ssd_linear_ce(hidden[:0], weight, targets[:0])
    assert e.loss.shape == (0,)
    dh, dw = ssd.ssd_linear_ce_grad(hidden[:0], weight, targets[:0], lse[:0])
    assert dh.shape == (0, 16) and (dw == 0).all()


@pytest.mark.gpu
def test_capture_and_streams():
    """Two graphs replayed at once on two streams, on new inputs, and an eager
    call on a third: all the bits of the eager call alone."""
    cases = [linear_case((90,), 256, 3001, 17 + i, keep=0.8) for i in range(2)]
    new = [linear_case((90,), 256, 3001, 27 + i, keep=0.8) for i in range(2)]
    graphs = []
    for h, w, y in cases:
        ssd.ssd_linear_ce(h, w, y)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = ssd.ssd_linear_ce(h, w, y)
            d = ssd.ssd_linear_ce_grad(h, w, y, r.lse)
        graphs.append((g, r, d))
    for old, fresh in zip(cases, new):
        for a, b in zip(old, fresh):
            a.copy_(b)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for (g, _, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    h, w, y = new[0]
    o = ssd.ssd_linear_ce(h, w, y, stream=streams[2])
    torch.cuda.synchronize()
    for (g, r, d), (h, w, y) in zip(graphs, new):
        e = ssd.ssd_linear_ce(h, w, y)
        dh, dw = ssd.ssd_linear_ce_grad(h, w, y, e.lse)
        assert torch.equal(r.loss, e.loss) and torch.equal(d[0], dh) and torch.equal(d[1], dw)
    assert torch.equal(o.loss, graphs[0][1].loss)
