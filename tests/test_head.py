"""The head losses (qlora_head_xent, qlora_head_distill) against their definition
in 64 bits, and their refusals.

Tolerances.  u = 2^-24 is the fp32 rounding, b = 2^-8 the bf16 one.
 - A logit is an fp32 sum of exact bf16 products, taken 16 at a time by the
   tensor core, which may truncate (2 u) where it adds: at most K / 16 + 16
   such steps, so |dz| <= (K / 16 + 16) 2 u sum_k |x_k w_k| =: D per row (its
   largest over the vocabulary), divided by T with the logit.
 - lse and loss move by at most D and 2 D with the logits.  Their own fp32
   steps (reference, differences, exp2 with 2^-22, sums over 256 columns as
   trees of 32 and over the tiles, log2, the product with ln 2) are fewer than
   64 roundings of terms no larger than |z| + |lse| + 1, plus 72 relative
   roundings of a sum of positive terms; the tolerance allows 160 u of that.
 - p is rounded once to bf16 (as e), and so is a teacher's p - q (a label's p - 1
   and a row's largest p - q stay in fp32); both carry the logits' 2 D and the
   fp32 steps of the exponent.  Entries of e below 2^-126 are flushed to 0, and e
   is stored relative to a reference that is at most 2^64 above the row's sum (or
   factors of at least 2^-149 bring a value of at most 2^64 to one that is), so an
   entry of p loses at most 2^-62 by that.  The second product adds fp32 steps over
   the vocabulary (N / 16 + 16 truncations, and the pieces of a split tile), and dX
   is rounded once.
"""
import ctypes
import math

import pytest
import torch

from bit_nf4_quantized_24_b200 import binding as qb
from bit_nf4_quantized_24_b200 import workloads as wl

U, B16 = 2.0**-24, 2.0**-8
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_24_b200 import build
    build.build()
    return qb.lib()


# ------------------------------------------------------------ plain definition


def reference(W, X, T, q, idx, entropy, dloss, piece=256):
    """loss, lse, dX in 64 bits, and their tolerances.  W, X: values (any type);
    q, idx: the targets' weights and entries [M, k] (weight 0: none)."""
    W, X, q, entropy = W.double(), X.double(), q.double(), entropy.double()
    M, (N, K) = X.shape[0], W.shape
    out = {n: [] for n in ("loss", "lse", "dx", "tol_loss", "tol_lse", "tol_dx")}
    for a in range(0, M, piece):
        s = slice(a, min(M, a + piece))
        z = X[s] @ W.T / T
        lse = torch.logsumexp(z, 1)
        told = q[s].sum(1) > 0
        zt = z.gather(1, idx[s])
        loss = T * T * torch.where(told, entropy[s] + (q[s] * (lse[:, None] - zt)).sum(1), 0.0)
        D = (K / 16 + 16) * 2 * U * (X[s].abs() @ W.abs().T).amax(1) / T
        steps = 160 * U * (z.abs().amax(1) + lse.abs() + 1)
        out["lse"].append(lse)
        out["loss"].append(loss)
        out["tol_lse"].append(D + steps)
        out["tol_loss"].append(T * T * (2 * D + 2 * steps + 64 * U * entropy[s].abs()))
        if dloss is not None:
            p = (z - lse[:, None]).exp()
            t = torch.zeros_like(p).scatter_add_(1, idx[s], q[s])
            g = (T * dloss[s].double() * told)[:, None]
            dp = p * (1.02 * B16 + (3 * D + 2 * steps)[:, None]) + 2.0**-62  # of the entries that are no targets, and
            dt = (p - t).abs() * 1.01 * B16 + (p + t) * (3 * D + 2 * steps + 64 * U)[:, None]  # of those that are,
            dt = dt + 2.0**-62  # with what is flushed
            dp = torch.where(t > 0, dt, dp)
            rows = (N / 16 + 16 + 64) * 2 * U * ((p + t) @ W.abs())
            dx = g * ((p - t) @ W)
            out["dx"].append(dx)
            out["tol_dx"].append(g.abs() * (dp @ W.abs() + rows) * 1.01 + dx.abs() * 1.01 * B16 + 1e-38)
    return {n: torch.cat(v) if v else None for n, v in out.items()}


def xent_targets(labels, N):
    told = (labels >= 0) & (labels < N)
    return told[:, None].double(), labels.clamp(0, N - 1)[:, None], torch.zeros(len(labels), device=labels.device)


def distill_targets(idx, t, N, T):
    kept = (idx >= 0) & (idx < N) & (t.double() != -math.inf)
    lq = torch.where(kept, t.double() / T, -math.inf)
    lq = torch.where(kept, lq - torch.where(kept.any(1, keepdim=True), torch.logsumexp(lq, 1, keepdim=True), 0.0), 0.0)
    q = torch.where(kept, lq.exp(), 0.0)
    return q, idx.clamp(0, N - 1), (q * lq).sum(1)


def compare(got, ref):
    for name, g in zip(("loss", "lse", "dx"), got):
        if ref[name] is None:
            assert g is None
            continue
        err = (g.double() - ref[name]).abs()
        assert torch.isfinite(g).all(), name
        worst = (err / ref["tol_" + name]).max().item()
        assert worst <= 1, f"{name}: {worst:.3g} of the tolerance"
    if ref["dx"] is not None and ref["dx"].norm() > 0:
        assert ((got[2].double() - ref["dx"]).norm() / ref["dx"].norm()).item() <= 1e-2


# ------------------------------------------------------------ inputs


def make(seed, M, N, K, block=0, dq=256, w_std=0.05):
    """A head (bf16 or NF4 with its bf16 values), hidden states and labels on the GPU."""
    g = wl.generator(seed)
    W = torch.randn(N, K, generator=g) * w_std
    labels = torch.randint(0, N, (M,), generator=g)
    X = torch.randn(M, K, generator=g)
    X += W[labels] * (torch.rand(M, 1, generator=g) * 12 / W[labels].square().sum(1, keepdim=True))
    if block:
        head = qb.nf4_quantize(W.cuda(), block, dq)
        values = qb.nf4_dequantize(head)
    else:
        head = values = W.bfloat16().cuda()
    return head, values, X.bfloat16().cuda(), labels.cuda(), g


def teacher(g, M, N, k, bf16, empty=True):
    idx = torch.randint(0, N, (M, k), generator=g)
    t = torch.randn(M, k, generator=g) * 3
    if empty and M > 3:
        idx[1] = -1
        idx[2, k // 2:] = N
        t[3, : k - k // 2] = -math.inf
        if k > 1:
            idx[0, 1] = idx[0, 0]  # the same entry twice
        t[1] = math.nan  # marked empty by the index: not read as a number
    t = t.bfloat16() if bf16 else t
    return idx.cuda(), t.cuda()


SHAPES = [
    (1, 1, 64), (1, 7, 64), (2, 256, 64), (3, 65, 128), (16, 257, 192), (127, 1000, 64), (128, 255, 512),
    (129, 511, 128), (256, 2048, 256), (257, 513, 64), (300, 2049, 320), (600, 4099, 576), (1, 32003, 1024),
    (17, 9001, 2112), (60, 5000, 192), (64, 32003, 640), (40, 40001, 64), (65, 33333, 128),
    (90, 33333, 128), (128, 32003, 640),
    (2290, 4090, 8192),  # tiles of 512 in both products
]


@gpu
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_xent(L, M, N, K, grad):
    head, values, X, labels, g = make(M + N + K, M, N, K)
    if M > 4:
        labels[1], labels[2], labels[3] = -100, N, -1
    dloss = torch.randn(M, generator=g).cuda() if grad else None
    got = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    compare(got, reference(values, X, 1.0, *xent_targets(labels, N), dloss))
    assert (got[0][(labels < 0) | (labels >= N)] == 0).all()
    if grad:
        assert (got[2][(labels < 0) | (labels >= N)] == 0).all()
    assert qb.device_status() == 0


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 300, 256), (37, 9001, 512), (128, 1031, 768), (200, 1031, 512),
                                   (100, 32000, 2048), (128, 20001, 1280), (16, 32000, 1024)])
@pytest.mark.parametrize("block,dq", [(32, 0), (32, 256), (64, 256), (64, 0), (128, 0), (256, 256)])
def test_xent_nf4_head(L, block, dq, M, N, K):
    head, values, X, labels, g = make(block + dq, M, N, K, block, dq)
    dloss = torch.full((M,), 1.0 / M, device="cuda")
    ref = reference(values, X, 1.0, *xent_targets(labels, N), dloss)
    got = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    compare(got, ref)
    same = qb.qlora_head_xent(values, X, labels, dloss=dloss)  # the bf16 values as a head
    compare(same, ref)
    if M <= 64 or M > 128:  # the same sums in the same order (between, the two heads' stages differ in length)
        assert all(torch.equal(a, b) for a, b in zip(got, same))


@gpu
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,N,K,k,T,bf16", [
    (1, 1, 64, 1, 1.0, False), (5, 300, 64, 1, 2.0, False), (9, 65, 128, 7, 1.5, True), (130, 1000, 192, 64, 2.0, False),
    (257, 513, 64, 33, 4.0, True), (300, 2049, 320, 256, 0.5, False), (64, 40, 64, 100, 1.0, False),
    (520, 4099, 576, 128, 1.0, True), (70, 3000, 128, 12, 1e-4, False), (200, 3000, 128, 12, 1e4, True),
])
def test_distill(L, M, N, K, k, T, bf16, grad):
    head, values, X, _, g = make(M + N + K + k, M, N, K)
    idx, t = teacher(g, M, N, k, bf16)
    dloss = torch.randn(M, generator=g).cuda() if grad else None
    got = qb.qlora_head_distill(head, X, idx, t, T, dloss=dloss)
    compare(got, reference(values, X, T, *distill_targets(idx, t, N, T), dloss))
    assert qb.device_status() == 0


@gpu
@pytest.mark.parametrize("what", ["one_tile", "one_entry", "borders"])
def test_distill_crowded_targets(L, what):
    """All 256 slots of every row in one vocabulary tile, all on one entry, and on the tiles' first and last entries."""
    M, N, K, k = 140, 1300, 128, 256
    head, values, X, _, g = make(77, M, N, K)
    if what == "one_tile":
        idx = (256 + torch.stack([torch.randperm(256, generator=g) for _ in range(M)])).cuda()
    elif what == "one_entry":
        idx = torch.full((M, k), 700, device="cuda")
    else:
        idx = torch.tensor([0, 255, 256, 511, 512, 767, 1023, 1024, 1279, 1280, 1299]).repeat(M, 24)[:, :k].cuda()
    t = torch.randn(M, k, generator=g).cuda()
    dloss = torch.ones(M, device="cuda")
    got = qb.qlora_head_distill(head, X, idx, t, 1.0, dloss=dloss)
    compare(got, reference(values, X, 1.0, *distill_targets(idx, t, N, 1.0), dloss))


@gpu
def test_distill_of_one_slot_is_cross_entropy(L):
    M, N, K = 300, 1111, 256
    head, values, X, labels, g = make(5, M, N, K)
    labels[7] = -100
    dloss = torch.rand(M, generator=g).cuda()
    a = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    b = qb.qlora_head_distill(head, X, labels[:, None].contiguous(), torch.zeros(M, 1, device="cuda"), 1.0, dloss=dloss)
    ref = reference(values, X, 1.0, *xent_targets(labels, N), dloss)  # (the distillation rounds its p - q to bf16)
    compare(a, ref)
    compare(b, ref)


@gpu
def test_left_out_and_broken_rows(L):
    """A NaN in one row's hidden states stays in that row; a left-out row's loss and gradient are 0 even then; a
    zero dloss writes zeros; all rows left out is a loss of zeros."""
    M, N, K = 300, 700, 128
    head, values, X, labels, g = make(11, M, N, K)
    dloss = torch.rand(M, generator=g).cuda() + 0.1
    dloss[10] = 0.0
    good = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    assert (good[2][10] == 0).all()
    X2, lab2 = X.clone(), labels.clone()
    X2[4], X2[5, 3], X2[6, 0] = math.nan, math.nan, math.inf
    lab2[4] = -100
    loss, lse, dx = qb.qlora_head_xent(head, X2, lab2, dloss=dloss)
    assert loss[4] == 0 and (dx[4] == 0).all() and torch.isnan(lse[4])
    for r in (5, 6):
        assert torch.isnan(loss[r]) and torch.isnan(lse[r]) and torch.isnan(dx[r]).all()
    rest = [i for i in range(M) if i not in (4, 5, 6)]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(good, (loss, lse, dx)))
    loss, lse, dx = qb.qlora_head_xent(head, X, torch.full_like(labels, -100), dloss=dloss)
    assert (loss == 0).all() and (dx == 0).all()
    compare((loss, lse, None), reference(values, X, 1.0, *xent_targets(torch.full_like(labels, -100), N), None))
    idx, t = teacher(g, M, N, 5, False, empty=False)
    t[8, 2], idx[9] = math.nan, -1
    loss, _, dx = qb.qlora_head_distill(head, X, idx, t, 1.0, dloss=dloss)
    bad = torch.isnan(loss)
    assert bad[8] and bad.sum() == 1 and torch.isnan(dx[8]).all() and not torch.isnan(dx[:8]).any()
    assert loss[9] == 0 and (dx[9] == 0).all()


@gpu
def test_confident_tokens_keep_the_digits_of_their_gradient(L):
    """A label with p near 1: loss and p - 1 are small differences, held to their own size.  The loss is log1p of the
    others' sum over the label's exponential, so its relative error is that of the exponent: D and the fp32 steps of
    reference() times 2, and 64 roundings.  p - 1 is rounded in fp32 alone, e to bf16 once and dX once."""
    M, N, K = 64, 500, 256
    g = wl.generator(3)
    W = torch.randn(N, K, generator=g).sign() * 0.125
    labels = torch.randint(0, N, (M,), generator=g)
    X = (W[labels] * 4 * torch.linspace(0.7, 1.6, M)[:, None]).bfloat16()  # own logit 11 to 26, the others near 0
    head, X, labels = W.bfloat16().cuda(), X.cuda(), labels.cuda()
    dloss = torch.ones(M, device="cuda")
    ref = reference(head, X, 1.0, *xent_targets(labels, N), dloss)
    got = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    compare(got, ref)
    rel = (got[2].double() - ref["dx"]).norm(dim=1) / ref["dx"].norm(dim=1)
    assert ref["loss"].min() < 1e-6
    assert (rel <= 2 * ref["tol_loss"] + 64 * U + 3 * B16).all()
    assert ((got[0] - ref["loss"]).abs() <= (2 * ref["tol_loss"] + 64 * U) * ref["loss"]).all()


@gpu
@pytest.mark.parametrize("distill", [False, True])
def test_logits_of_any_size(L, distill):
    """Rows whose logits are far from 0: near +-45 (where the stored exponentials change their reference), in the
    hundreds, all far below 0, and some segments below with others above, next to ordinary rows."""
    M, N, K = 160, 1400, 256
    head, values, X, labels, g = make(81, M, N, K, w_std=0.06)
    W = values.float()
    W[:, 0] = 1.0                                  # a common offset: X[:, 0]
    W[:, 1] = (torch.arange(N) // 128 % 2).cuda()  # one of some segments: X[:, 1]
    head = W.bfloat16()
    X[:, :2] = 0
    X[10:40] *= torch.logspace(0, 2, 30).cuda()[:, None].bfloat16()
    X[40:70, 0] = torch.linspace(30, 300, 30).cuda().bfloat16()
    X[70:100, 0] = -torch.linspace(30, 300, 30).cuda().bfloat16()
    X[100:120, 0], X[100:120, 1] = -90, torch.linspace(20, 200, 20).cuda().bfloat16()
    X[120:140, 1] = torch.linspace(-200, 200, 20).cuda().bfloat16()
    dloss = torch.rand(M, generator=g).cuda()
    if distill:
        idx, t = teacher(g, M, N, 20, False)
        got = qb.qlora_head_distill(head, X, idx, t, 1.0, dloss=dloss)
        ref = reference(head, X, 1.0, *distill_targets(idx, t, N, 1.0), dloss)
    else:
        got = qb.qlora_head_xent(head, X, labels, dloss=dloss)
        ref = reference(head, X, 1.0, *xent_targets(labels, N), dloss)
    compare(got, ref)


@gpu
@pytest.mark.parametrize("piece", [256, 512])
def test_pieces_of_tokens(L, piece):
    """A smaller workspace takes fewer tokens at a time: the same results within their rounding (tile widths and split
    tiles follow the piece's size), the same bits when repeated, and the rows behind the last piece written once."""
    M, N, K = 900, 3001, 512
    head, values, X, labels, g = make(21, M, N, K)
    dloss = torch.rand(M, generator=g).cuda()
    ref = reference(values, X, 1.0, *xent_targets(labels, N), dloss)
    compare(qb.qlora_head_xent(head, X, labels, dloss=dloss), ref)
    nbytes = qb.head_workspace_bytes(M, N, K, piece=piece)  # M = 900: a last piece of 132, and of few tokens below
    assert nbytes < qb.head_workspace_bytes(M, N, K)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    outs = (torch.full((M,), 7.0, device="cuda"), torch.full((M,), 7.0, device="cuda"),
            torch.full((M, K), 7.0, device="cuda", dtype=torch.bfloat16))
    got = qb.qlora_head_xent(head, X, labels, dloss=dloss, outs=outs, workspace=ws)
    assert all(a is b for a, b in zip(got, outs))
    compare(got, ref)
    again = qb.qlora_head_xent(head, X, labels, dloss=dloss, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    idx, t = teacher(g, M, N, 9, False)
    for m in (M, 2 * piece + 1, 2 * piece + 128):
        nbytes = qb.head_workspace_bytes(m, N, K, 9, piece=piece)
        ws = torch.full((nbytes + 4096,), 171, dtype=torch.uint8, device="cuda")
        a = [x[:m].contiguous() if m <= M else torch.cat((x, x))[:m].contiguous() for x in (X, idx, t, dloss)]
        got = qb.qlora_head_distill(head, a[0], a[1], a[2], 2.0, dloss=a[3], workspace=ws[:nbytes])
        compare(got, reference(values, a[0], 2.0, *distill_targets(a[1], a[2], N, 2.0), a[3]))
        assert (ws[nbytes:] == 171).all()


@gpu
@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M", [1, 100, 128, 129, 256, 257, 640, 900])
def test_every_piece_that_can_be_asked_for(L, M, nf4):
    """A workspace of any piece is enough for its call, also where fewer tokens need more of it for partial sums."""
    N, K = 300, 1024
    head, values, X, labels, g = make(M, M, N, K, 64 if nf4 else 0)
    dloss = torch.rand(M, generator=g).cuda()
    ref = reference(values, X, 1.0, *xent_targets(labels, N), dloss)
    for piece in (1, 100, 256, 300, 512, 700, 0):
        nbytes = qb.head_workspace_bytes(M, N, K, nf4=nf4, piece=piece)
        ws = torch.full((nbytes + 4096,), 171, dtype=torch.uint8, device="cuda")
        compare(qb.qlora_head_xent(head, X, labels, dloss=dloss, workspace=ws[:nbytes]), ref)
        assert (ws[nbytes:] == 171).all()


@gpu
@pytest.mark.parametrize("M,N,grad", [(5000, 131072, True), (20000, 300, False)])
def test_several_pieces_of_the_librarys_choice(L, M, N, grad):
    """More tokens than the default workspace takes at once, with a gradient and without."""
    K = 64
    head, values, X, labels, g = make(M, M, N, K)
    dloss = torch.rand(M, generator=g).cuda() if grad else None
    got = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    compare(got, reference(values, X, 1.0, *xent_targets(labels, N), dloss))


@gpu
@pytest.mark.parametrize("M", [20, 300])
def test_gradient_without_weights_is_that_of_the_sum(L, M):
    """The C call with dX and a NULL dloss: weights of one."""
    N, K = 700, 128
    head, values, X, labels, g = make(M, M, N, K)
    want = qb.qlora_head_xent(head, X, labels, dloss=torch.ones(M, device="cuda"))
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dX = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(qb.head_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    assert L.qlora_head_xent(qb._ptr(head), None, None, None, 64, 256, N, K, qb._ptr(X), M, qb._ptr(labels), None,
                             qb._ptr(loss), qb._ptr(lse), qb._ptr(dX), qb._ptr(ws), ws.numel(), qb._stream()) == 0
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, dX), want))


@gpu
def test_outputs_stay_inside_their_rows(L):
    """Guard values around every output and behind the workspace are left as they were."""
    M, N, K = 131, 777, 192
    head, values, X, labels, g = make(31, M, N, K)
    f = torch.full((M + 64,), 5.0, device="cuda")
    f2 = f.clone()
    d = torch.full((M + 64, K), 5.0, device="cuda", dtype=torch.bfloat16)
    nbytes = qb.head_workspace_bytes(M, N, K)
    ws = torch.full((nbytes + 4096,), 171, dtype=torch.uint8, device="cuda")
    dloss = torch.ones(M, device="cuda")
    qb.qlora_head_xent(head, X, labels, dloss=dloss, outs=(f[:M], f2[:M], d[:M]), workspace=ws[:nbytes])
    assert (f[M:] == 5).all() and (f2[M:] == 5).all() and (d[M:] == 5).all() and (ws[nbytes:] == 171).all()
    compare((f[:M], f2[:M], d[:M]), reference(values, X, 1.0, *xent_targets(labels, N), dloss))


@gpu
def test_gradient_against_differences_of_the_loss(L):
    """The sum of the losses along a direction of X, by central differences of the op itself.  The step h d is exact
    in bf16 (X + h d and X - h d are representable), so the difference quotient is off by the losses' fp32 errors over
    2 h and by the third derivative, h^2 / 6 |d3|; |d3| <= 2 (max |W d|)^3 per token of a softmax's cumulant."""
    M, N, K, h = 64, 600, 128, 2.0**-5
    head, values, _, labels, g = make(41, M, N, K, w_std=0.1)
    X = torch.randint(-32, 33, (M, K), generator=g).float().div(32).cuda()
    d = torch.randint(-1, 2, (M, K), generator=g).float().cuda()
    up, down = (X + h * d).bfloat16(), (X - h * d).bfloat16()
    assert torch.equal(up.float(), X + h * d) and torch.equal(down.float(), X - h * d)
    idx, t = teacher(g, M, N, 11, False, empty=False)
    dloss = torch.ones(M, device="cuda")
    third = 2 * (d.double() @ values.double().T).abs().amax(1) ** 3
    for call, targets, T in (
            (lambda x, w: qb.qlora_head_xent(head, x, labels, dloss=w), xent_targets(labels, N), 1.0),
            (lambda x, w: qb.qlora_head_distill(head, x, idx, t, 2.0, dloss=w), distill_targets(idx, t, N, 2.0), 2.0)):
        slope = (call(up, None)[0].double() - call(down, None)[0].double()) / (2 * h)
        dx = call(X.bfloat16(), dloss)[2].double()
        ref = reference(values, X, T, *targets, dloss)
        tol = ref["tol_loss"] * 1.5 / h + T * T * h * h / 6 * third / T**3 + (ref["tol_dx"] * d.abs()).sum(1)
        assert ((slope - (dx * d).sum(1)).abs() <= tol).all()
        assert tol.max() < 0.5 * slope.abs().median()


@gpu
def test_captured_and_replayed_with_new_inputs(L):
    M, N, K, k = 300, 2100, 256, 6
    head, values, X, labels, g = make(51, M, N, K)
    idx, t = teacher(g, M, N, k, True)
    dloss = torch.rand(M, generator=g).cuda()
    qb.qlora_head_xent(head, X, labels, dloss=dloss)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = qb.qlora_head_xent(head, X, labels, dloss=dloss)
        b = qb.qlora_head_distill(head, X, idx, t, 2.0, dloss=dloss)
    X.copy_(torch.randn(M, K, generator=g))
    labels.copy_(torch.randint(0, N, (M,), generator=g))
    t.copy_(torch.randn(M, k, generator=g))
    for _ in range(2):
        graph.replay()
    want_a = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    want_b = qb.qlora_head_distill(head, X, idx, t, 2.0, dloss=dloss)
    assert all(torch.equal(x, y) for x, y in zip(a + b, want_a + want_b))


@gpu
def test_two_streams_at_once(L):
    """Two calls on two streams with no order between them, each with its own workspace."""
    cases = [make(61 + i, 500, 3000, 512) for i in range(2)]
    dloss = torch.rand(500, generator=wl.generator(1)).cuda()
    want = [qb.qlora_head_xent(c[0], c[2], c[3], dloss=dloss) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [qb.qlora_head_xent(c[0], c[2], c[3], dloss=dloss, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
def test_no_tokens(L):
    head = torch.zeros(100, 64, dtype=torch.bfloat16, device="cuda")
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse, dx = qb.qlora_head_xent(head, X, none, dloss=torch.empty(0, device="cuda"))
    assert loss.shape == lse.shape == (0,) and dx.shape == (0, 64)


@gpu
@pytest.mark.slow
def test_head_with_more_than_2_to_the_31_weights(L):
    """Offsets into the head that pass 32 bits, in the bf16 and the expanded NF4 head."""
    M, N, K = 5, 135001, 16384
    assert N * K > 2**31
    g = torch.Generator("cuda").manual_seed(9)
    codes = torch.randint(0, 256, (N * K // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.rand(N * K // 64, generator=g, device="cuda") * 0.02 + 0.01
    head = qb.NF4Weight(codes, torch.empty(0, dtype=torch.uint8, device="cuda"), scale, N, K, 64, 0)
    values = qb.nf4_dequantize(head)
    X = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    labels = torch.tensor([0, N - 1, N // 2, N - 2, 7], device="cuda")
    dloss = torch.ones(M, device="cuda")
    a = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    b = qb.qlora_head_xent(values, X, labels, dloss=dloss)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ref = {}
    z = torch.cat([X.double() @ values[i:i + 15000].double().T for i in range(0, N, 15000)], 1)
    lse = torch.logsumexp(z, 1)
    ref["loss"] = lse - z.gather(1, labels[:, None])[:, 0]
    p = (z - lse[:, None]).exp()
    p.scatter_add_(1, labels[:, None], torch.full((M, 1), -1.0, device="cuda", dtype=torch.float64))
    ref["dx"] = sum(p[:, i:i + 15000] @ values[i:i + 15000].double() for i in range(0, N, 15000))
    D = (K / 16 + 16) * 2 * U * X.double().abs().sum(1) * values.abs().max().double()
    assert ((a[0] - ref["loss"]).abs() <= 2 * D).all()
    assert ((a[2].double() - ref["dx"]).norm() / ref["dx"].norm()) <= 1e-2


@gpu
def test_training_step_of_a_layer_under_the_head(L, oracle):
    """The run a user makes: layer forward, head loss with its gradient, layer backward.  Against the chain in 64 bits
    on the values that the library rounds (Y, and dX of the head in bf16), with the layer's tolerance of 1e-2."""
    M, N, K, r, V = 384, 512, 256, 16, 3003
    p = wl.draw_small(71, M, N, K, r, 2.0 * r, b_std=0.05)
    q = qb.nf4_quantize(p["W"].cuda())
    X, A, Bl = (p[n].cuda() for n in ("X", "A", "B"))
    g = wl.generator(72)
    head = (torch.randn(V, N, generator=g) * 0.05).bfloat16().cuda()
    labels = torch.randint(0, V, (M,), generator=g).cuda()
    labels[::7] = -100
    dloss = torch.full((M,), 1.0, device="cuda") / (labels >= 0).sum()
    Y, H = qb.qlora_linear_fwd(q, X, A, Bl, p["scale"])
    loss, lse, dY = qb.qlora_head_xent(head, Y, labels, dloss=dloss)
    dX, dA, dB = qb.qlora_linear_bwd(q, X, dY, A, Bl, p["scale"], H=H)
    Wd = qb.nf4_dequantize(q).double()
    A64, B64, X64 = (t.double().requires_grad_() for t in (A, Bl, X))
    Y64 = X64 @ Wd.T + p["scale"] * (X64 @ A64.T) @ B64.T
    z = Y64 @ head.double().T
    keep = labels >= 0
    L64 = (torch.logsumexp(z, 1)[keep] - z[keep, labels[keep]]).mean()
    L64.backward()
    assert abs((loss * dloss).sum().item() - L64.item()) <= 1e-2 * L64.item()
    for name, got, want in (("dX", dX, X64.grad), ("dA", dA, A64.grad), ("dB", dB, B64.grad)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        assert rel <= 1e-2, (name, rel)


@gpu
@pytest.mark.parametrize("M", [32, 1024])
def test_chain_repeated_without_a_wait(L, M):
    """Layer forward, head loss, layer backward enqueued twenty times on one stream with nothing in between, each
    from other inputs: every kernel may be launched while the one before it still runs, and none may read what that
    one has yet to write.  Each result is the one of the same calls with a synchronisation after every call."""
    N, K, r, V = 1024, 512, 16, 3003
    p = wl.draw_small(91, M, N, K, r, 2.0 * r, b_std=0.05)
    q = qb.nf4_quantize(p["W"].cuda())
    A, Bl = p["A"].cuda(), p["B"].cuda()
    g = wl.generator(92)
    head = (torch.randn(V, N, generator=g) * 0.05).bfloat16().cuda()
    labels = torch.randint(0, V, (M,), generator=g).cuda()
    dloss = torch.full((M,), 1.0 / M, device="cuda")
    inputs = [torch.randn(M, K, generator=g).bfloat16().cuda() for _ in range(20)]

    def chain(X, wait):
        Y, H = qb.qlora_linear_fwd(q, X, A, Bl, p["scale"])
        wait()
        loss, lse, dY = qb.qlora_head_xent(head, Y, labels, dloss=dloss)
        wait()
        out = (loss, lse, dY, *qb.qlora_linear_bwd(q, X, dY, A, Bl, p["scale"], H=H))
        wait()
        return out

    want = [chain(X, torch.cuda.synchronize) for X in inputs]
    got = [chain(X, lambda: None) for X in inputs]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------ without a GPU


def test_reference_gradient_against_differences():
    """The 64-bit definition that the GPU tests compare with: its gradient against central differences."""
    g = wl.generator(1)
    M, N, K, T = 5, 40, 8, 1.7
    W, X = torch.randn(N, K, generator=g).double(), torch.randn(M, K, generator=g).double()
    idx = torch.randint(-1, N, (M, 6), generator=g)
    idx[2] = -1
    t = torch.randn(M, 6, generator=g).double()
    dloss = torch.rand(M, generator=g).double()
    for args in ((T, *distill_targets(idx, t, N, T)), (1.0, *xent_targets(torch.tensor([3, -100, 0, N - 1, N]), N))):
        dx = reference(W, X, *args, dloss)["dx"]
        h = 1e-5
        for i in range(M):
            for j in range(K):
                e = torch.zeros_like(X)
                e[i, j] = h
                up, down = (reference(W, X + s * e, *args, None)["loss"] for s in (1, -1))
                assert abs(((up - down) * dloss).sum() / (2 * h) - dx[i, j]) < 1e-8


def test_workspace_sizes(L):
    a = qb.head_workspace_bytes(4096, 32000, 4096)
    assert a % 256 == 0 and a >= 4096 * 32000 * 2
    assert qb.head_workspace_bytes(4096, 32000, 4096, want_dx=False) < a // 16  # no logits, no exponentials
    assert qb.head_workspace_bytes(4096, 32000, 4096, piece=256) < a // 8
    assert qb.head_workspace_bytes(1 << 20, 128000, 4096) < (3 << 29)  # bounded however many tokens there are
    assert qb.head_workspace_bytes(4096, 32000, 4096, nf4=True) >= a + 32000 * 4096 * 2
    assert qb.head_workspace_bytes(4096, 32000, 4096, k=64) > a
    assert qb.head_workspace_bytes(0, 32000, 4096) > 0
    # whatever piece is asked for, the bytes hold a call: whole tiles of tokens, one at least
    for M in (1, 100, 256, 257, 900, 5000):
        sizes = [qb.head_workspace_bytes(M, 1000, 512, piece=p) for p in (1, 100, 255, 256, 300, 512, 1000, 10**6)]
        assert sizes[0] == sizes[1] == sizes[2] == sizes[3] == sizes[4] and sizes[-1] == qb.head_workspace_bytes(M, 1000, 512)


def test_refusals(L):
    """Bad arguments come back as a status before anything is enqueued (no device is touched)."""
    n = ctypes.c_size_t()
    assert L.qlora_head_workspace(1, 10, 96, 0, 1, 0, 0, ctypes.byref(n)) == -2
    assert L.qlora_head_workspace(1, 0, 64, 0, 1, 0, 0, ctypes.byref(n)) == -1
    assert L.qlora_head_workspace(-1, 10, 64, 0, 1, 0, 0, ctypes.byref(n)) == -1
    assert L.qlora_head_workspace(1, 10, 64, -1, 1, 0, 0, ctypes.byref(n)) == -1
    assert L.qlora_head_workspace(1, 10, 64, 257, 1, 0, 0, ctypes.byref(n)) == -7
    assert L.qlora_head_workspace(1, 10, 64, 0, 1, 0, -1, ctypes.byref(n)) == -1
    assert L.qlora_head_workspace(1, 10, 64, 0, 1, 0, 0, None) == -1
    assert L.qlora_head_workspace(1, (1 << 24) + 1, 64, 0, 1, 0, 0, ctypes.byref(n)) == -2
    P = ctypes.c_void_p
    f, odd, big = P(0x10000), P(0x10008), 1 << 40

    def xent(W=f, codes=None, absmax=None, dq=None, block=64, dqb=256, N=100, K=64, X=f, M=4, labels=f, dloss=f, loss=f,
             lse=f, dX=f, ws=f, nbytes=big):
        return L.qlora_head_xent(W, codes, absmax, dq, block, dqb, N, K, X, M, labels, dloss, loss, lse, dX, ws, nbytes,
                                 None)

    assert xent(W=None) == -1 and xent(codes=f) == -1 and xent(W=None, codes=f) == -1
    assert xent(W=None, codes=f, dq=f) == -1  # double quantization without absmax_q
    assert xent(W=None, codes=f, absmax=f, dq=f, block=48) == -7
    assert xent(W=None, codes=f, absmax=f, dq=f, block=128) == -2
    assert xent(W=None, codes=P(0x10010), absmax=f, dq=f) == -2  # codes are read by 32 bytes
    assert xent(K=100) == -2 and xent(N=0) == -1 and xent(M=-1) == -1 and xent(M=(1 << 24) + 1) == -2
    assert xent(X=None) == -1 and xent(labels=None) == -1 and xent(loss=None) == -1 and xent(lse=None) == -1
    assert xent(dX=None) == -1  # a gradient's weights without a gradient
    assert xent(W=odd) == -2 and xent(X=odd) == -2 and xent(dX=odd) == -2
    assert xent(labels=P(0x10004)) == -2 and xent(loss=P(0x10002)) == -2 and xent(dloss=P(0x10002)) == -2
    assert xent(ws=None) == -4 and xent(ws=odd) == -4 and xent(nbytes=1000) == -4
    assert xent(M=0, X=None, labels=None, loss=None, lse=None, dX=None, dloss=None, ws=None) == 0

    def distill(idx=f, t=f, bf16=0, k=8, T=1.0, M=4, ws=f, nbytes=big):
        return L.qlora_head_distill(f, None, None, None, 64, 256, 100, 64, f, M, idx, t, bf16, k, ctypes.c_float(T), f,
                                    f, f, f, ws, nbytes, None)

    assert distill(idx=None) == -1 and distill(t=None) == -1 and distill(k=0) == -1 and distill(k=257) == -7
    for T in (0.0, -1.0, math.nan, math.inf, 1e-5, 1e5):
        assert distill(T=T) == -1
    assert distill(idx=P(0x10004)) == -2 and distill(t=P(0x10002)) == -2 and distill(t=P(0x10001), bf16=1) == -2
    assert distill(nbytes=1000) == -4 and distill(M=0, ws=None) == 0


def test_binding_refusals(L):
    W, X = torch.zeros(10, 64, dtype=torch.bfloat16), torch.zeros(3, 64, dtype=torch.bfloat16)
    labels = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        qb.qlora_head_xent(W, X, labels)
    with pytest.raises(TypeError, match="torch.Tensor"):
        qb.qlora_head_xent(None, X, labels)
    with pytest.raises(ValueError, match="teacher_idx"):
        qb.qlora_head_distill(W, X, labels, labels.float())
    with pytest.raises(TypeError, match="teacher_logits"):
        qb.qlora_head_distill(W, X, labels[:, None], labels[:, None])


@gpu
def test_binding_refusals_of_gpu_tensors(L):
    c = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    W, X, y = c(10, 64), c(3, 64), c(3, dt=torch.int64)
    for bad in (dict(X=c(3, 128)), dict(X=c(3)), dict(labels=c(4, dt=torch.int64)), dict(dloss=c(4, dt=torch.float32)),
                dict(X=c(64, 3).t()), dict(head=c(64)), dict(outs=(None, None, X.clone())),
                dict(workspace=c(1 << 20, 2, dt=torch.uint8)[:, 0]), dict(labels=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            qb.qlora_head_xent(**{**dict(head=W, X=X, labels=y), **bad})
    for bad in (dict(labels=y.int()), dict(X=X.float()), dict(head=W.half()), dict(dloss=c(3))):
        with pytest.raises(TypeError):
            qb.qlora_head_xent(**{**dict(head=W, X=X, labels=y), **bad})
    with pytest.raises(qb.QloraError) as e:
        qb.qlora_head_xent(W, X, y, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4
    with pytest.raises(qb.QloraError) as e:
        qb.qlora_head_xent(c(10, 96), c(3, 96), y)
    assert e.value.status == -2
    with pytest.raises(qb.QloraError) as e:
        qb.qlora_head_distill(W, X, c(3, 2, dt=torch.int64), c(3, 2), temperature=0.0)
    assert e.value.status == -1
