"""ssd_teacher_top and ssd_distill against plain 64-bit forms: types, sizes,
strides, ties, masked and void rows, the gradient, capture and streams."""
import ctypes as C
import math

import pytest
import torch

from speculative_decoding_verify_ssd_b200 import binding as ssd

from train_testlib import HALF_STEP, U32, distill_ref, logits_like, sum_error, top_ref

BF16, FP32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------------------
# Without a GPU: refusals at the C entry, and the formulas.
# ---------------------------------------------------------------------------
def _top(L, **kw):
    a = dict(logits=None, dtype=1, nb=2, rpb=3, V=100, bs=300, rs=100, T=1.0, M=4)
    a.update(kw)
    return L.ssd_teacher_top(a["logits"], a["dtype"], a["nb"], a["rpb"], a["V"], a["bs"], a["rs"], a["T"], a["M"],
                             None, None, None, None, None, a.get("work"), a.get("n", 0), None)


def _distill(L, **kw):
    a = dict(logits=None, dtype=1, nb=2, rpb=3, V=100, bs=300, rs=100, T=1.0, M=4, grad=None, gbs=300, grs=100)
    a.update(kw)
    return L.ssd_distill(a["logits"], a["dtype"], a["nb"], a["rpb"], a["V"], a["bs"], a["rs"], a["T"], a["M"],
                         None, None, None, None, None, None, a["grad"], a["gbs"], a["grs"], None)


@pytest.mark.parametrize("call", [_top, _distill])
def test_host_refusals(call):
    L = ssd.load()
    assert call(L, dtype=7) == 2
    for bad in (dict(nb=-1), dict(rpb=-1), dict(V=0), dict(M=0), dict(M=257, V=1000), dict(M=101), dict(T=0.0),
                dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-5), dict(T=1e5), dict(bs=-1),
                dict(rs=-1), dict(nb=1 << 20, rpb=1 << 20)):
        assert call(L, **bad) == 1, bad
    assert call(L, nb=0) == 0 and call(L, rpb=0) == 0   # nothing to do
    assert call(L) == 1                                  # NULL arrays


def test_host_refuses_overlapping_gradient_rows():
    L = ssd.load()
    p = C.c_void_p(4096)
    assert _distill(L, grad=p, grs=99) == 1
    assert _distill(L, grad=p, gbs=0) == 1


def test_formula_gradient_against_differences():
    """The reference gradient is the derivative of the reference loss."""
    g = torch.Generator().manual_seed(3)
    V, M = 23, 5
    z = torch.randn(2, V, generator=g, dtype=torch.float64) * 2
    t = torch.randn(2, V, generator=g, dtype=torch.float64) * 2
    for T, use_tail in ((1.0, True), (0.7, False), (2.0, True)):
        values, tokens = t.topk(M, dim=-1)
        tail = torch.logsumexp((t / T).scatter(-1, tokens, -math.inf), -1) if use_tail else None
        tokens = tokens.int()
        tokens[1, 2] = -1
        _, grad, _ = distill_ref(z, tokens, values, tail, T)
        h = 1e-5
        for v in range(V):
            d = torch.zeros_like(z)
            d[:, v] = h
            up, down = (distill_ref(z + s * d, tokens, values, tail, T)[0] for s in (1, -1))
            # central differences: h^2 of the third derivative (below 10 / T^3) and 1e-16 / h of rounding
            torch.testing.assert_close((up - down) / (2 * h), grad[:, v], rtol=0, atol=30 * h * h + 1e-10)


# ---------------------------------------------------------------------------
# The top logits.
# ---------------------------------------------------------------------------
def check_top(logits, M, T):
    r = ssd.ssd_teacher_top(logits, M, T)
    torch.cuda.synchronize()
    tokens, values, lse, tail = top_ref(logits, M, T)
    assert torch.equal(r.status, torch.zeros_like(r.status))
    assert torch.equal(r.values.double(), values)
    assert torch.equal(r.tokens, tokens)
    e = sum_error(logits.shape[-1], logits.dtype)
    for got, want in ((r.lse, lse), (r.tail, tail)):
        fin = torch.isfinite(want)
        assert torch.equal(got.double()[~fin], want[~fin])
        err = (got.double() - want).abs()[fin]
        assert (err <= e + want.abs()[fin] * U32).all(), float(err.max())
    return r


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V,M", [(1, 1), (2, 2), (7, 3), (8, 8), (9, 1), (255, 255), (256, 256), (1023, 64),
                                 (5003, 200), (32003, 33), (66001, 256), (128256, 64), (262144, 128)])
def test_top_sizes(dtype, V, M):
    for rows, T in ((1, 1.0), (5, 0.7)):
        check_top(logits_like((rows,), V, dtype, V + M), M, T)


@pytest.mark.gpu
def test_top_many_rows():
    check_top(logits_like((100, 8), 4001, BF16, 5), 16, 1.0)
    check_top(logits_like((1500,), 1000, FP32, 6), 8, 1.3)
    check_top(logits_like((50, 6), 70001, BF16, 7), 100, 0.8)    # several slices each


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_top_views(dtype):
    """[B, K+1, V] without its last position, an odd V (rows at any element), a
    transposed batch, and a base pointer off the 16-byte grid."""
    x = logits_like((3, 5), 4099, dtype, 1)
    check_top(x[:, :4], 17, 1.0)
    check_top(x[:, 1:], 17, 1.0)
    check_top(x.transpose(0, 1), 17, 1.0)
    check_top(x[:, :, 3:4000], 17, 1.0)
    check_top(x[1, 2, 5:], 3, 1.0)
    check_top(x[:1].expand(4, 5, 4099), 9, 1.0)
    check_top(logits_like((2, 4), 210003, dtype, 2)[:, 1:], 17, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [3000, 70001, 140002])
def test_top_ties(dtype, V):
    """Quantised logits, constant rows, -0 against +0, and rows with fewer
    finite logits than M: equal logits in token order."""
    x = logits_like((4,), V, FP32, 9)
    check_top((x * 2).round().div(2).to(dtype), 64, 1.0)
    check_top(torch.zeros(2, V, device="cuda", dtype=dtype), 100, 1.0)
    z = torch.where(x > 0, torch.zeros_like(x), torch.full_like(x, -0.0)).to(dtype)
    check_top(z, 50, 1.0)
    check_top((-x.abs() * 2).round().to(dtype), 256, 1.0)
    few = torch.full((2, V), -math.inf, device="cuda", dtype=dtype)
    few[0, 77] = -3.0
    few[1, [5, 2999, V - 1]] = torch.tensor([1.0, 4.0, 1.0], device="cuda", dtype=dtype)
    check_top(few, 8, 1.0)
    asc = torch.arange(V, device="cuda").float().div(V / 200).to(dtype)
    check_top(torch.stack([asc, asc.flip(0)]), 200, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T", [1.0, 0.01, 100.0])
@pytest.mark.parametrize("V", [9001, 240007])
def test_top_tail_far_below(dtype, T, V):
    """The tail's logarithm stays exact when the top outweighs it by more than
    the exponent range of fp32, with and without ties at the threshold."""
    x = logits_like((3,), V, FP32, 11).clamp(-8, 8)
    x[:, [3, 500, 9000]] += 4000.0
    check_top(x.to(dtype), 3, T)
    x = torch.full((2, V), -5000.0, device="cuda")
    x[0, 100:4000] = 0.0
    x[1, :2000] = 0.0
    check_top(x.to(dtype), 256, T)
    x[:] = -5000.0
    x[:, 40:43] = 0.0
    check_top(x.to(dtype), 3, T)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [513, 140001])
def test_top_void_rows(dtype, V):
    x = logits_like((6,), V, dtype, 13)
    ref = ssd.ssd_teacher_top(x, 4, 1.0)
    bad = x.clone()
    bad[1, V - 1] = math.nan
    bad[2, 0] = math.inf
    bad[4] = -math.inf
    r = ssd.ssd_teacher_top(bad, 4, 1.0)
    assert r.status.tolist() == [0, ssd.ROW_NONFINITE, ssd.ROW_NONFINITE, 0, ssd.ROW_NONFINITE, 0]
    for b in (1, 2, 4):
        assert (r.tokens[b] == -1).all() and r.values[b].isnan().all() and r.lse[b].isnan() and r.tail[b].isnan()
    for b in (0, 3, 5):
        assert torch.equal(r.tokens[b], ref.tokens[b]) and r.lse[b] == ref.lse[b] and r.tail[b] == ref.tail[b]


# ---------------------------------------------------------------------------
# Distillation.
# ---------------------------------------------------------------------------
def teacher(shape, V, M, T, seed, use_tail, device="cuda"):
    t = logits_like(shape, V, FP32, seed, device=device)
    values, tokens = t.topk(M, dim=-1)
    tail = torch.logsumexp((t.double() / T).scatter(-1, tokens, -math.inf), -1).float() if use_tail else None
    return tokens.int().contiguous(), values.contiguous(), tail


def check_distill(logits, tokens, values, tail, T, scale=None, grad=None):
    before = logits.clone()
    alone = ssd.ssd_distill(logits, tokens, values, tail, T, row_scale=scale, with_grad=False)
    r = ssd.ssd_distill(logits, tokens, values, tail, T, row_scale=scale, grad=grad)
    torch.cuda.synchronize()
    loss, want, b = distill_ref(before, tokens, values, tail, T, scale)
    if scale is not None:
        loss = torch.where(scale == 0, torch.zeros_like(loss), loss)
    assert torch.equal(r.loss, alone.loss) and torch.equal(r.status, alone.status) and alone.grad is None
    assert (r.status & ssd.ROW_INVALID == 0).all()
    # log sums carry e; the loss holds at most two of them, and the rounding of its own value
    e = sum_error(before.shape[-1], before.dtype)
    fin = torch.isfinite(loss)
    assert torch.equal(r.loss.double()[~fin], loss[~fin])
    err = (r.loss.double() - loss).abs()[fin]
    assert (err <= 2 * e + loss.abs()[fin] * U32).all(), float(err.max())
    # a term's own error (at most e), q_tail's and an atom's q (2 e each), and one rounding of the result
    q = torch.where(b["hit"], b["q"], b["share"] * b["q_tail"][..., None])
    bound = b["w"].abs()[..., None] * 2 * e * q + 2 * e * want.abs() + (want.abs() + 1e-30) * HALF_STEP[before.dtype]
    # results below fp32's normal range are flushed
    bound = bound + 2.0 ** -126 * (b["w"].abs()[..., None] + 1)
    d = (r.grad.double() - want).abs()
    assert (d <= bound).all(), float((d - bound).max())
    return r


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V,M", [(1, 1), (2, 1), (7, 3), (8, 8), (9, 1), (257, 256), (1023, 64), (5003, 200),
                                 (32003, 33), (66001, 256), (128256, 64), (262144, 128)])
def test_distill_sizes(dtype, V, M):
    for rows, T, use_tail in ((1, 1.0, True), (5, 0.7, False), (3, 2.0, True)):
        z = logits_like((rows,), V, dtype, V + M)
        tokens, values, tail = teacher((rows,), V, M, T, V + M + 1, use_tail)
        scale = torch.rand(rows, device="cuda") + 0.5
        check_distill(z, tokens, values, tail, T, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_distill_views(dtype):
    """Strided logits, and gradients at other strides and alignments, in place too."""
    V, T = 4099, 1.0
    x = logits_like((3, 5), V, dtype, 1)
    tokens, values, tail = teacher((3, 4), V, 17, T, 2, True)
    r = check_distill(x[:, :4], tokens, values, tail, T)
    assert r.grad.is_contiguous()
    out = torch.full((3, 6, V + 5), 7.0, device="cuda", dtype=dtype)
    check_distill(x[:, 1:], tokens, values, tail, T, grad=out[:, 1:5, 3:V + 3])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[:, 1:5, 3:V + 3] = False
    assert (out[keep] == 7.0).all()      # nothing around the view was written
    out = torch.empty(4, 3, V, device="cuda", dtype=dtype)
    check_distill(x[:, :4], tokens, values, tail, T, grad=out.transpose(0, 1))
    y = x.clone()
    check_distill(y[:, :4], tokens, values, tail, T, grad=y[:, :4])
    assert torch.equal(y[:, 4], x[:, 4])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [600, 140001])
def test_distill_absent_and_left_out(dtype, V):
    """-1 atoms, -inf teacher logits, rows of scale 0 (whose contents do not matter), no atom at all."""
    T = 1.0
    z = logits_like((5,), V, dtype, 21)
    tokens, values, tail = teacher((5,), V, 12, T, 22, True)
    tokens[1, 3:] = -1
    tokens[2, :] = -1                # the tail is all there is: loss 0, gradient 0
    values[3, 5] = -math.inf
    scale = torch.tensor([1.0, 2.0, 1.0, 0.5, 0.0], device="cuda")
    r = check_distill(z, tokens, values, tail, T, scale)
    assert (r.grad[4] == 0).all() and r.loss[4] == 0
    assert (r.grad[2] == 0).all() and abs(float(r.loss[2])) <= 1e-6
    z2 = z.clone()
    z2[4] = math.nan
    tokens[4, 0] = V + 5
    r2 = ssd.ssd_distill(z2, tokens, values, tail, T, row_scale=scale)
    assert torch.equal(r2.loss, r.loss) and torch.equal(r2.grad, r.grad) and r2.status[4] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_distill_masked_logits(dtype):
    """-inf and the type's lowest value in the student's rows; atoms without student mass."""
    V, T = 3001, 1.0
    z = logits_like((4,), V, dtype, 31)
    tokens, values, tail = teacher((4,), V, 6, T, 32, True)
    z[0, ::2] = -math.inf
    z[1, 1::2] = torch.finfo(dtype).min
    for b in (0, 1):
        z[b, tokens[b].long()] = 0.5
    check_distill(z, tokens, values, tail, T)
    only = torch.full_like(z, -math.inf)           # no tail mass in the student
    only.scatter_(1, tokens.long(), 0.25)
    check_distill(only, tokens, values, None, T)
    r = ssd.ssd_distill(only, tokens, values, tail, T)
    assert (r.loss == math.inf).all() and (r.status == ssd.ROW_ZERO_Q).all() and r.grad.isfinite().all()
    none = z.clone()
    none[:] = 0
    none.scatter_(1, tokens.long(), -math.inf)     # no atom mass in the student
    r = ssd.ssd_distill(none, tokens, values, tail, T)
    assert (r.loss == math.inf).all() and (r.status == ssd.ROW_ZERO_Q).all()
    p = -r.grad.gather(1, tokens.long()).double()
    want = distill_ref(z, tokens, values, tail, T)[1] * 0
    q = torch.softmax(torch.cat([values.double(), tail.double()[:, None]], 1), 1)[:, :-1]
    assert ((p - q).abs() <= q * (HALF_STEP[dtype] + 4 * U32)).all() and want.abs().sum() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("V, M", [(513, 256), (40001, 256), (140001, 256), (140001, 67), (401, 5)])
def test_distill_token_twice_anywhere(V, M):
    # one row for each pair of places that hold one token; every third row has none
    pairs = [(i, j) for j in (1, 2, 3, 4, 31, 32, 63, 66, 127, 128, 131, 254, 255, M - 1) if j < M
             for i in (0, 1, 3, j // 2, j - 1) if i < j]
    rows = 3 * ((len(pairs) + 1) // 2)
    g = torch.Generator().manual_seed(V + M)
    tokens = torch.stack([torch.randperm(V, generator=g)[:M] for _ in range(rows)]).int()
    want = torch.zeros(rows, dtype=torch.int32)
    at = [r for r in range(rows) if r % 3 != 2][: len(pairs)]
    for r, (i, j) in zip(at, pairs):
        tokens[r, j] = tokens[r, i]
        want[r] = ssd.ROW_BAD_TOKEN
    z = torch.randn(rows, V, generator=g).bfloat16().cuda()
    values = torch.randn(rows, M, generator=g).cuda()
    r = ssd.ssd_distill(z, tokens.cuda(), values)
    bad = want.cuda() != 0
    assert torch.equal(r.status, want.cuda())
    assert torch.equal(r.loss.isnan(), bad) and torch.equal((r.grad == 0).all(-1), bad)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [513, 140001])
def test_distill_void_rows(dtype, V):
    T = 1.0
    z = logits_like((8,), V, dtype, 41)
    tokens, values, tail = teacher((8,), V, 9, T, 42, True)
    ref = ssd.ssd_distill(z, tokens, values, tail, T)
    z, tokens, values, tail = z.clone(), tokens.clone(), values.clone(), tail.clone()
    z[0, V - 1] = math.nan
    z[1, int(tokens[1, 0])] = math.inf
    z[2] = -math.inf
    tokens[3, 8] = tokens[3, 2]
    tokens[4, 1] = V
    values[5, 4] = math.nan
    tail[6] = math.inf
    r = ssd.ssd_distill(z, tokens, values, tail, T)
    N, B = ssd.ROW_NONFINITE, ssd.ROW_BAD_TOKEN
    assert r.status.tolist() == [N, N, N, B, B, N, N, 0]
    assert r.loss[:7].isnan().all() and (r.grad[:7] == 0).all()
    assert r.loss[7] == ref.loss[7] and torch.equal(r.grad[7], ref.grad[7])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_distill_offset_logits(dtype):
    """Logits far from zero: the exponentials' arguments are differences."""
    V = 3000
    z = (logits_like((3,), V, FP32, 55) + 5000.0).to(dtype)
    tokens, values, tail = teacher((3,), V, 5, 1.0, 56, True)
    check_distill(z, tokens, values, tail, 1.0)
    check_distill(z - 10000, tokens, values - 70, None, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_distill_extreme_temperatures(dtype):
    V = 2000
    for T in (1e-4, 0.05, 30.0, 1e4):
        z = logits_like((3,), V, dtype, 51, spread=min(2.0, 20 * T))
        tokens, values, tail = teacher((3,), V, 5, T, 52, True)
        check_distill(z, tokens, values * min(1.0, 10 * T), None, T)


@pytest.mark.gpu
def test_rows_binding_refusals():
    z = logits_like((2,), 50, BF16, 1)
    tokens, values, tail = teacher((2,), 50, 4, 1.0, 2, True)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_teacher_top(z, 51)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_teacher_top(z, 0)
    with pytest.raises(ValueError):
        ssd.ssd_teacher_top(z.half(), 4)
    with pytest.raises(ValueError):
        ssd.ssd_teacher_top(z.cpu(), 4)
    with pytest.raises(ValueError):
        ssd.ssd_teacher_top(z.t(), 1)
    with pytest.raises(ValueError):
        ssd.ssd_teacher_top(z[None, None], 1)
    with pytest.raises(ValueError):
        ssd.ssd_distill(z, tokens.long(), values, tail)
    with pytest.raises(ValueError):
        ssd.ssd_distill(z, tokens, values[:1], tail)
    with pytest.raises(ValueError):
        ssd.ssd_distill(z, tokens, values, tail, grad=torch.empty(2, 50, device="cuda"))
    with pytest.raises(ssd.SsdError):
        ssd.ssd_distill(z, tokens, values, tail, grad=torch.empty(1, 50, device="cuda", dtype=BF16).expand(2, 50))
    with pytest.raises(ssd.SsdError):
        ssd.ssd_distill(z, tokens, values, tail, T=0.0)
    with pytest.raises(ssd.SsdError, match="too large"):
        ssd.ssd_distill(torch.zeros(1, 1 << 20, device="cuda"), tokens[:1], values[:1])
    with pytest.raises(ssd.SsdError, match="too large"):
        ssd.ssd_teacher_top(torch.zeros(1, 1 << 22, device="cuda"), 1)
    with pytest.raises(ssd.SsdError, match="workspace"):
        ssd.ssd_teacher_top(logits_like((1,), 200001, BF16, 1), 4, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    e = ssd.ssd_teacher_top(z[:0], 4)
    assert e.tokens.shape == (0, 4) and ssd.ssd_distill(z[:0], tokens[:0], values[:0]).grad.shape == (0, 50)


@pytest.mark.gpu
def test_rows_capture_and_streams():
    """Captured and replayed on new inputs, and launched on a side stream: the
    same bits as the eager call."""
    V, T = 32003, 1.0
    z = logits_like((4, 3), V, BF16, 61)
    tokens, values, tail = teacher((4, 3), V, 16, T, 62, True)
    ssd.ssd_teacher_top(z, 16)
    ssd.ssd_distill(z, tokens, values, tail, T)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        top = ssd.ssd_teacher_top(z, 16)
        dis = ssd.ssd_distill(z, top.tokens, top.values, top.tail, T)
    z.copy_(logits_like((4, 3), V, BF16, 63))
    g.replay()
    torch.cuda.synchronize()
    e = ssd.ssd_teacher_top(z, 16)
    d = ssd.ssd_distill(z, e.tokens, e.values, e.tail, T)
    assert torch.equal(top.tokens, e.tokens) and torch.equal(top.tail, e.tail)
    assert torch.equal(dis.loss, d.loss) and torch.equal(dis.grad, d.grad)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = ssd.ssd_distill(z, e.tokens, e.values, e.tail, T, stream=s)
    s.synchronize()
    assert torch.equal(o.loss, d.loss) and torch.equal(o.grad, d.grad)
