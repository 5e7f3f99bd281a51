"""The training calls at the edges of what they allow: shared memory and
workspaces that earlier work left full, limits of sizes, scales and logits that
are not finite, waits that give up."""
import math
import os
import re

import pytest
import torch

from speculative_decoding_verify_ssd_b200 import _build
from speculative_decoding_verify_ssd_b200 import binding as ssd

from test_train_linear import check as check_linear
from test_train_rows import check_distill, check_top, teacher
from train_testlib import HALF_STEP, U32, distill_ref, linear_case, linear_ref, logits_like, sum_error, top_ref

BF16, FP32 = torch.bfloat16, torch.float32
TRAIN_CU = os.path.join(_build.CSRC, "ssd_train.cu")


# ---------------------------------------------------------------------------
# Workspaces.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("V,dtype", [(128256, 1), (151936, 1), (151936, 0), (32003, 0), (70001, 1), (400000, 0)])
def test_top_workspace_serves_fewer_rows(V, dtype):
    L = ssd.load()
    sizes = [L.ssd_teacher_top_workspace_bytes(n, V, dtype, 8) for n in range(1, 1200)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("D,V", [(8, 300), (64, 5003), (256, 20011), (1024, 32000), (2048, 128256), (64, 60001)])
@pytest.mark.parametrize("grad", [0, 1])
def test_linear_workspace_serves_fewer_rows(D, V, grad):
    L = ssd.load()
    sizes = [L.ssd_linear_ce_workspace_bytes(n, D, V, grad) for n in list(range(1, 2200)) + [5000, 70000, 1 << 18]]
    assert sizes == sorted(sizes)


@pytest.mark.gpu
def test_one_workspace_for_a_shrinking_batch():
    """Sized for the largest batch, dirty, used at sizes whose own plans need more than a larger one's."""
    V = 128256
    z = logits_like((64,), V, BF16, 76)
    ws = torch.empty(ssd.teacher_top_workspace_bytes(64, V, ssd.DTYPE_BF16, 16), dtype=torch.uint8, device="cuda")
    tokens, values, _, _ = top_ref(z, 16, 1.0)
    for n in (64, 59, 42, 29, 19, 1):
        ws.fill_(255)
        r = ssd.ssd_teacher_top(z[:n], 16, workspace=ws)
        assert (r.status == 0).all() and torch.equal(r.tokens, tokens[:n]) and torch.equal(r.values.double(), values[:n])
    hidden, weight, targets = linear_case((1030,), 256, 20011, 77)
    ws = torch.empty(ssd.linear_ce_workspace_bytes(1030, 256, 20011, True), dtype=torch.uint8, device="cuda")
    for n in (1030, 960, 640, 129, 3):
        h, y = hidden[:n], targets[:n]
        ws.fill_(255)
        r = ssd.ssd_linear_ce(h, weight, y, workspace=ws)
        ws.fill_(255)
        dh, dw = ssd.ssd_linear_ce_grad(h, weight, y, r.lse, workspace=ws)
        dh2, dw2 = ssd.ssd_linear_ce_grad(h, weight, y, r.lse)
        assert (r.status == 0).all() and torch.equal(dh, dh2) and torch.equal(dw, dw2)


@pytest.mark.gpu
def test_top_blocks_on_used_shared_memory():
    """Thousands of blocks one after the other on shared memory (their barriers'
    places too) that the blocks before them left full."""
    z = logits_like((3000,), 1500, BF16, 71)
    tokens, values, _, _ = top_ref(z, 8, 1.0)
    first = None
    for _ in range(20):
        ssd.ssd_distill(z, tokens, values.float())
        r = ssd.ssd_teacher_top(z, 8)
        assert (r.status == 0).all() and torch.equal(r.tokens, tokens) and torch.equal(r.values.double(), values)
        first = r if first is None else first
        assert torch.equal(r.lse, first.lse) and torch.equal(r.tail, first.tail)


# ---------------------------------------------------------------------------
# Limits.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("V,dtype", [(819197, 0), (1600000, 0), (1638393, 1), (3200000, 1)])
def test_longest_top_rows_have_a_workspace(V, dtype):
    L = ssd.load()
    assert L.ssd_teacher_top_workspace_bytes(1, V, dtype, 8) > 0
    assert L.ssd_teacher_top_workspace_bytes(1, 3300001 // (2 if dtype == 0 else 1), dtype, 8) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("V,dtype", [(819195, FP32), (819201, FP32), (1600000, FP32), (1638389, BF16), (3200000, BF16)])
def test_longest_top_rows(V, dtype):
    """16 slices of 200 KB, and more of them up to the documented 6.4 MB; at odd places too."""
    z = logits_like((2,), V + 1, dtype, 78)
    check_top(z[:, 1:], 256, 0.8)
    check_top(z[:, :V], 7, 1.0)
    check_top((z[:, :V] * 2).round(), 200, 1.0)     # slices full of equal logits


@pytest.mark.gpu
@pytest.mark.parametrize("V,dtype", [(400000, FP32), (800000, BF16)])
def test_longest_distill_rows(V, dtype):
    z = logits_like((2,), V + 1, dtype, 79)[:, 1:]
    tokens, values, tail = teacher((2,), V, 100, 1.0, 80, True)
    check_distill(z, tokens, values, tail, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [32768, 32769, 70001, 1 << 18])
def test_many_head_rows(N):
    """More rows than 1024 blocks of 32 hold, some of them left out, up to the limit."""
    hidden, weight, targets = linear_case((N,), 16, 70, 84, keep=0.7)
    check_linear(hidden, weight, targets, torch.rand(N, device="cuda") + 0.5)


@pytest.mark.parametrize("N", [1, 8192, 8193, 32769, 1 << 18])
def test_no_more_than_1024_blocks_read_all_targets(N):
    """The gather's blocks, each of which scans the N targets (its rule, from the source)."""
    rule = re.search(r"launch_prep\(PrepArgs& a.*?\n\}", open(TRAIN_CU).read(), re.S).group(0)
    rows = (N + 1023) // 1024
    assert "rows > 32" not in rule and "(a.N + 1023) / 1024" in rule
    assert -(-N // max(rows, 8)) <= 1024 and rows <= 256


# ---------------------------------------------------------------------------
# Scales and logits that are not finite.
# ---------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("N", [7, 300])
def test_linear_scales_that_are_not_finite(N):
    """Such a row is flagged and left out; the others' gradients are as if it were not there."""
    hidden, weight, targets = linear_case((N,), 72, 500, 81)
    scale = torch.rand(N, device="cuda") + 0.5
    for i, bad in ((1, math.nan), (3, math.inf), (6, -math.inf)):
        scale[i] = bad
    targets[0], targets[6] = 500, -1
    r = ssd.ssd_linear_ce(hidden, weight, targets)
    g = ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse, row_scale=scale)
    want = torch.zeros(N, dtype=torch.int32, device="cuda")
    want[0], want[1], want[3] = ssd.ROW_BAD_TOKEN, ssd.ROW_NONFINITE, ssd.ROW_NONFINITE
    assert torch.equal(g.status, want)
    only, without = targets.clone(), scale.clone()
    only[[0, 1, 3]] = -1
    without[[0, 1, 3, 6]] = 0
    f = linear_ref(hidden, weight, only, without)
    assert (g.grad_hidden[[0, 1, 3, 6]] == 0).all()
    assert ((g.grad_hidden.double() - f["dh"]).abs() <= f["dh_tol"]).all()
    assert ((g.grad_weight.double() - f["dw"]).abs() <= f["dw_tol"]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [6, 200])
def test_linear_logits_that_are_infinite(N):
    """-inf is a token of no mass, except at the target; +inf and NaN void the row."""
    hidden, weight, targets = linear_case((N,), 64, 300, 85)
    targets[targets == 17] = 18
    hidden[:, 0] = hidden[:, 0].abs() + 0.5
    hidden[1, 0], hidden[2, 0], targets[3] = -1.0, 0.0, 17     # +inf, NaN, -inf at the target
    masked = weight.clone()
    masked[17, 0] = -math.inf
    r = ssd.ssd_linear_ce(hidden, masked, targets)
    void = torch.zeros(N, dtype=torch.bool, device="cuda")
    void[1:4] = True
    assert torch.equal(r.status, torch.where(void, ssd.ROW_NONFINITE, 0).int())
    assert r.loss[void].isnan().all() and r.lse[void].isnan().all()
    keep = torch.arange(300, device="cuda") != 17
    small = torch.where(void, torch.full_like(targets, -1), targets - (targets > 17).int())
    f = linear_ref(hidden, weight[keep], small)
    assert ((r.loss.double() - f["loss"]).abs() <= f["loss_tol"])[~void].all()
    g = ssd.ssd_linear_ce_grad(hidden, masked, targets, r.lse)
    assert torch.equal(g.status, r.status)
    assert ((g.grad_weight[keep].double() - f["dw"]).abs() <= f["dw_tol"]).all() and (g.grad_weight[17] == 0).all()
    assert (g.grad_hidden[void] == 0).all()
    # (in the masked column G weight is 0 * -inf)
    d = (g.grad_hidden[:, 1:].double() - f["dh"][:, 1:]).abs()
    assert (d <= f["dh_tol"][:, 1:])[~void].all() and g.grad_hidden[~void, 0].isnan().all()
    none = weight.clone()
    none[:, 0] = -math.inf                                     # every logit -inf
    r = ssd.ssd_linear_ce(hidden[4:], none, targets[4:])
    assert (r.status == ssd.ROW_NONFINITE).all() and r.loss.isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_distill_scales_that_are_not_finite(dtype):
    z = logits_like((4,), 700, dtype, 82)
    tokens, values, tail = teacher((4,), 700, 9, 1.0, 83, True)
    scale = torch.tensor([1.0, math.nan, math.inf, 2.0], device="cuda")
    r = ssd.ssd_distill(z, tokens, values, tail, row_scale=scale)
    e = ssd.ssd_distill(z, tokens, values, tail, row_scale=torch.ones_like(scale) + (scale == 2.0))
    assert (r.status == 0).all() and torch.equal(r.loss, e.loss)
    assert not r.grad[1:3].isfinite().any()
    assert torch.equal(r.grad[[0, 3]], e.grad[[0, 3]])


@pytest.mark.gpu
def test_sizes_that_no_int_holds():
    """Refused, not taken modulo 2^32 (views of a few bytes: nothing of such a size is allocated)."""
    z = logits_like((1,), 8, BF16, 87)
    n = 2 ** 32 + 1
    for big in (z.expand(n, 8), z[None].expand(n, 1, 8), z[None].expand(1, n, 8)):
        with pytest.raises(ValueError, match="dimension above"):
            ssd.ssd_teacher_top(big, 1)
        with pytest.raises(ValueError, match="dimension above"):
            ssd.ssd_distill(big, z, z)
        with pytest.raises(ValueError, match="dimension above"):
            ssd.ssd_linear_ce(big, z, z)
    for M in (2 ** 32 + 1, 257, 2 ** 31):
        with pytest.raises(ssd.SsdError, match="invalid argument"):
            ssd.ssd_teacher_top(z, M)
    with pytest.raises(ValueError, match="weight must be"):
        ssd.ssd_linear_ce(z, z.expand(n, 8), torch.zeros(1, dtype=torch.int32, device="cuda"))


def test_stream_of_another_device():
    """Its launch would go to that device's default stream with this one's pointers."""
    class Stream:
        device = torch.device("cuda", 1)

    def never(raw):
        raise AssertionError("launched")

    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        ssd._launch(0, Stream(), never)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [3001, 140001])
def test_distill_rows_with_all_mass_on_one_side(dtype, V):
    """The whole gradient of rows whose atoms, or whose tail, have no student mass."""
    T = 1.0
    tokens, values, tail = teacher((4,), V, 6, T, 88, True)
    for use_tail in (tail, None):
        none = logits_like((4,), V, dtype, 89).scatter_(1, tokens.long(), -math.inf)
        r = check_distill(none, tokens, values, use_tail, T)
        assert (r.loss == math.inf).all() and (r.status == ssd.ROW_ZERO_Q).all()
        only = torch.full_like(none, -math.inf).scatter_(1, tokens.long(), 0.25)
        r = check_distill(only, tokens, values, use_tail, T)
        rest = torch.ones_like(only, dtype=torch.bool).scatter_(1, tokens.long(), False)
        assert (r.grad[rest] == 0).all()
        if use_tail is not None:
            assert (r.loss == math.inf).all() and (r.status == ssd.ROW_ZERO_Q).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_distill_weights_below_fp32(dtype):
    """Atoms and a tail of a weight that only 64 bits hold, where the student has
    none: infinite; without any weight (masked by the type's lowest value): not."""
    V = 40
    tokens = torch.arange(4, dtype=torch.int32, device="cuda").repeat(6, 1)
    values = torch.zeros(6, 4, device="cuda")
    tail = torch.zeros(6, device="cuda")
    z = logits_like((6,), V, dtype, 93)
    z[:3, 2] = -math.inf
    z[3:, 4:] = -math.inf
    for r, at in enumerate((-150.0, -2000.0, torch.finfo(FP32).min)):
        values[r, 2] = at
        tail[3 + r] = at
    r = ssd.ssd_distill(z, tokens, values, tail)
    f, grad, _ = distill_ref(z, tokens, values, tail, 1.0)
    assert torch.equal(f == math.inf, torch.tensor([1, 0, 0, 1, 0, 0], device="cuda").bool())
    assert torch.equal(r.loss == math.inf, f == math.inf)
    assert torch.equal(r.status, torch.where(f == math.inf, ssd.ROW_ZERO_Q, 0).int())
    fin = f.isfinite()
    assert ((r.loss.double() - f).abs()[fin] <= 2 * sum_error(V, dtype) + f[fin] * U32).all()
    assert ((r.grad.double() - grad).abs() <= 2 * sum_error(V, dtype) + grad.abs() * HALF_STEP[dtype]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_distill_small_weights_at_the_lowest_value(dtype):
    """p below 2^-126 times a logit of -3.4e38 is no small number: an atom's, and the tail's."""
    V, T = 40, 0.25
    tokens = torch.arange(4, dtype=torch.int32, device="cuda").repeat(4, 1)
    values = torch.zeros(4, 4, device="cuda")
    tail = torch.zeros(4, device="cuda")
    z = logits_like((4,), V, dtype, 95)
    z[:2, 2] = torch.finfo(dtype).min
    z[2:, 4:] = torch.finfo(dtype).min
    for r, log_p in enumerate((-88.0, -90.0)):
        values[r, 2] = log_p * T
        tail[2 + r] = log_p
    r = ssd.ssd_distill(z, tokens, values, tail, T)
    f, grad, _ = distill_ref(z, tokens, values, tail, T)
    assert (r.status == 0).all() and (f > 1.0).all()
    # the small weight's exponent, up to 2^8 in size, is rounded to 32 bits (2^-16), e^x adds 2^-22
    assert ((r.loss.double() - f).abs() <= 2 * sum_error(V, dtype) + f * (2.0 ** -16 + 2.0 ** -21)).all()
    assert ((r.grad.double() - grad).abs() <= 4 * sum_error(V, dtype) / T + grad.abs() * HALF_STEP[dtype]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V,M", [(2, 2), (40, 5), (3001, 70), (140001, 256)])
@pytest.mark.parametrize("T", [1.0, 0.25])
def test_distill_rows_of_nothing_but_the_lowest_value(dtype, V, M, T):
    """A mask of the type's lowest value that leaves nothing: the student is
    uniform, whatever the size of its logits; and logits of one large value."""
    tokens, values, tail = teacher((3,), V, M, T, 94, M < V)
    for at in (torch.finfo(dtype).min, -1e30, 2.0 ** 20):
        z = torch.full((3, V), at, device="cuda", dtype=dtype)
        r = ssd.ssd_distill(z, tokens, values, tail, T)
        f, grad, _ = distill_ref(torch.zeros_like(z), tokens, values, tail, T)
        e = sum_error(V, dtype)
        assert (r.status == 0).all()
        assert ((r.loss.double() - f).abs() <= 2 * e + f.abs() * U32).all()
        q = 1.0 / V      # an atom's q (2 e of it), then one rounding
        assert ((r.grad.double() - grad).abs() <= (4 * e * q + 2 * e * grad.abs() * T) / T + grad.abs() * HALF_STEP[dtype]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("V,dtype", [(262143, BF16), (131075, FP32)])
def test_distill_more_clusters_than_the_gpu_holds(V, dtype):
    """Rows of eight blocks each, several times what runs at once; loss and gradient, in place too."""
    z = logits_like((300,), V, dtype, 90)
    tokens, values, tail = teacher((300,), V, 33, 1.0, 91, True)
    r = check_distill(z, tokens, values, tail, 1.0)
    again = ssd.ssd_distill(z, tokens, values, tail, grad=z)
    assert torch.equal(again.loss, r.loss) and torch.equal(again.grad, r.grad)


@pytest.mark.gpu
@pytest.mark.parametrize("N,D,V", [(64, 1024, 32000), (700, 1024, 32003), (5000, 64, 60001)])
def test_linear_repeats_its_bits(N, D, V):
    hidden, weight, targets = linear_case((N,), D, V, 92, keep=0.8)
    first = None
    for _ in range(5):
        r = ssd.ssd_linear_ce(hidden, weight, targets)
        g = ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse)
        out = (r.loss, r.lse, g[0], g[1])
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


# ---------------------------------------------------------------------------
# Outputs over inputs.
# ---------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("N", [6, 200])
def test_linear_gradients_over_inputs(N):
    """Over the weight, one another, or parts of the hidden states: refused.  In
    the gaps of strided inputs, and over a dense hidden itself: allowed."""
    D, V = 64, 300
    hidden, weight, targets = linear_case((N,), D, V, 86, keep=0.6)
    targets[0] = 3
    r = ssd.ssd_linear_ce(hidden, weight, targets)
    want = ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse)
    big = torch.zeros(2 * (N + V), D, device="cuda", dtype=BF16)

    def refused(h, w, **out):
        with pytest.raises(ssd.SsdError, match="invalid argument"):
            ssd.ssd_linear_ce_grad(h, w, targets, r.lse, **out)

    refused(hidden, weight, grad_weight=weight)
    w = big[:V]
    w.copy_(weight)
    refused(hidden, w, grad_weight=big[V - 1:2 * V - 1])
    refused(hidden, w, grad_hidden=big[V - 1:V - 1 + N])
    refused(hidden, weight, grad_weight=big[:V], grad_hidden=big[V - 1:V - 1 + N])
    h = big[V:V + N]
    h.copy_(hidden)
    refused(h, weight, grad_hidden=big[V + 1:V + 1 + N])
    refused(h, weight, grad_hidden=big[V - N + 1:V + 1])
    pair = torch.zeros(V, 2, D, device="cuda", dtype=BF16)      # weight rows with a gap of one row between
    pair[:, 1] = weight
    refused(hidden, pair[:, 1], grad_weight=pair.view(2 * V, D)[:V])
    assert torch.equal(pair[:, 1], weight) and (pair[:, 0] == 0).all()
    # beside one another
    g = ssd.ssd_linear_ce_grad(h, w, targets, r.lse, grad_hidden=big[V + N:V + 2 * N],
                               grad_weight=big[V + 2 * N:2 * V + 2 * N])
    assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    # a gap of the hidden batches' stride holds the gradient
    gap = torch.zeros(4, N, D, device="cuda", dtype=BF16)
    gap[0], gap[3] = hidden, hidden
    both, two = gap[::3], torch.stack([targets, targets])
    lse = torch.stack([r.lse, r.lse])
    g = ssd.ssd_linear_ce_grad(both, weight, two, lse, grad_hidden=gap[1:3])
    assert torch.equal(g[0][0], want[0]) and torch.equal(g[0][1], want[0])
    # in place
    g = ssd.ssd_linear_ce_grad(h, weight, targets, r.lse, grad_hidden=h)
    assert torch.equal(h, want[0]) and torch.equal(g[1], want[1])


# ---------------------------------------------------------------------------
# Waits that give up: a build whose product kernel waits 200 ns past its first
# polls (of up to 100 us each) instead of 2 s.  The first tile of a head 65536
# wide takes longer than that, so its epilogue gives up; the copies and products
# that are under way still land, since a block that gave up stays 20 ms.
# ---------------------------------------------------------------------------
class Library:
    """Calls of the bindings go to another build inside the `with`."""

    def __init__(self, path):
        self.path = path

    def __enter__(self):
        self.saved = _build.LIB, ssd._lib
        _build.LIB, ssd._lib = self.path, None
        ssd.load(build_if_missing=False)

    def __exit__(self, *exc):
        _build.LIB, ssd._lib = self.saved


@pytest.fixture(scope="module")
def short_wait():
    return Library(_build.build_variant("shortgemm", ["SSD_GEMM_WAIT_NS=200ull"]))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [5, 200])          # single blocks, and pairs
def test_forward_that_gives_up_is_flagged(short_wait, N):
    hidden, weight, targets = linear_case((N,), 65536, 700, 73)
    targets[2] = -1
    with short_wait:
        r = ssd.ssd_linear_ce(hidden, weight, targets)
        torch.cuda.synchronize()
    on = targets >= 0
    # (what the products left may be no number besides)
    assert (r.status[on] & ssd.ROW_DEVICE_TIMEOUT != 0).all() and r.loss[on].isnan().all() and r.lse[on].isnan().all()
    assert r.status[2] == 0 and r.loss[2] == 0
    r = ssd.ssd_linear_ce(hidden, weight, targets)      # the usual limits: the answer
    f = linear_ref(hidden, weight, targets)
    assert (r.status == 0).all() and ((r.loss.double() - f["loss"]).abs() <= f["loss_tol"])[on].all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [5, 200])
def test_gradient_that_gives_up_is_flagged(short_wait, N):
    """Neither gradient holds a number, with or without a status array."""
    hidden, weight, targets = linear_case((N,), 65536, 700, 74)
    targets[2] = -1
    on = targets >= 0
    r = ssd.ssd_linear_ce(hidden, weight, targets)
    with short_wait:
        given = torch.full_like(targets, 77)
        outs = [ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse),
                ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse, status=given)]
        torch.cuda.synchronize()
    assert outs[1].status is given
    for g in outs:
        assert g.grad_weight.isnan().all() and g.grad_hidden[on].isnan().all() and (g.grad_hidden[2] == 0).all()
        assert (g.status[on] == ssd.ROW_DEVICE_TIMEOUT).all() and g.status[2] == 0
    dh, dw = g = ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse)
    f = linear_ref(hidden, weight, targets)
    assert (g.status == 0).all()
    assert ((dh.double() - f["dh"]).abs() <= f["dh_tol"]).all()
    assert ((dw.double() - f["dw"]).abs() <= f["dw_tol"]).all()


@pytest.mark.gpu
def test_gradient_status_without_being_asked():
    hidden, weight, targets = linear_case((9,), 64, 50, 75)
    targets[4] = 50
    r = ssd.ssd_linear_ce(hidden, weight, targets)
    r.lse[7] = math.inf
    g = ssd.ssd_linear_ce_grad(hidden, weight, targets, r.lse)
    want = torch.zeros(9, dtype=torch.int32, device="cuda")
    want[4], want[7] = ssd.ROW_BAD_TOKEN, ssd.ROW_NONFINITE
    assert isinstance(g, tuple) and len(g) == 2 and g[0] is g.grad_hidden and g[1] is g.grad_weight
    assert torch.equal(g.status, want)
