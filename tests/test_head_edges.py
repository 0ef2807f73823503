"""The head losses where they could go wrong.  Definition, inputs and tolerances: test_head.py."""
import ctypes
import math

import pytest
import torch
from test_head import B16, U, compare, distill_targets, make, reference, teacher, xent_targets

from bit_nf4_quantized_24_b200 import binding as qb
from bit_nf4_quantized_24_b200 import workloads as wl

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_24_b200 import build
    build.build()
    return qb.lib()


@gpu
@pytest.mark.parametrize("M", [20, 300])
def test_format_of_a_bf16_head_is_ignored(L, M):
    """block and dq_block mean nothing beside W: whatever they hold, the call is the same."""
    N, K = 700, 128
    head, _, X, labels, g = make(M, M, N, K)
    idx, t = teacher(g, M, N, 5, False)
    dloss = torch.rand(M, generator=g).cuda()
    want = qb.qlora_head_xent(head, X, labels, dloss=dloss) + qb.qlora_head_distill(head, X, idx, t, 2.0, dloss=dloss)
    ws = torch.empty(qb.head_workspace_bytes(M, N, K, 5), dtype=torch.uint8, device="cuda")
    out = [torch.empty(M, device="cuda") for _ in range(4)]
    dX = [torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    p, odd = qb._ptr, ctypes.c_void_p(0x10002)  # a scale that is not even aligned
    for block, dq in ((0, 0), (-1, -1), (2**31 - 1, 2**31 - 1), (-(2**31), 7), (48, 256), (1 << 30, 0), (32, 0)):
        for o in out + dX:
            o.zero_()
        assert L.qlora_head_xent(p(head), None, p(dloss), odd, block, dq, N, K, p(X), M, p(labels), p(dloss), p(out[0]),
                                 p(out[1]), p(dX[0]), p(ws), ws.numel(), qb._stream()) == 0
        assert L.qlora_head_distill(p(head), None, None, None, block, dq, N, K, p(X), M, p(idx), p(t), 0, 5,
                                    ctypes.c_float(2.0), p(dloss), p(out[2]), p(out[3]), p(dX[1]), p(ws), ws.numel(),
                                    qb._stream()) == 0
        got = (out[0], out[1], dX[0], out[2], out[3], dX[1])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_scales_beside_a_bf16_head_are_ignored(L):
    """No status comes from a pointer that a bf16 head does not use: the call gets as far as its workspace's size."""
    f = ctypes.c_void_p(0x10000)
    for absmax, scale in ((None, None), (f, f), (ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10002))):
        assert L.qlora_head_xent(f, None, absmax, scale, 48, 7, 100, 64, f, 4, f, f, f, f, f, f, 1000, None) == -4


def with_gone(W, X, gone, T, q, idx, entropy, dloss):
    """The definition in 64 bits where the logits in `gone` are -inf, with the tolerances of test_head.reference."""
    W, X, q, entropy, g = W.double(), X.double(), q.double(), entropy.double(), T * dloss.double()
    N, K = W.shape
    z = (X @ W.T / T).masked_fill(gone, -math.inf)
    lse = torch.logsumexp(z, 1)
    told = q.sum(1) > 0
    loss = torch.where(q > 0, q * (lse[:, None] - z.gather(1, idx)), 0.0).sum(1) + entropy
    loss = T * T * torch.where(told, loss, 0.0)
    D = (K / 16 + 16) * 2 * U * (X.abs() @ W.abs().T).masked_fill(gone, 0.0).amax(1) / T
    steps = 160 * U * (z.masked_fill(gone, 0.0).abs().amax(1) + lse.abs() + 1)
    p = (z - lse[:, None]).exp()
    t = torch.zeros_like(p).scatter_add_(1, idx, q)
    dt = (p - t).abs() * 1.01 * B16 + (p + t) * (3 * D + 2 * steps + 64 * U)[:, None] + 2.0**-62
    dp = p * (1.02 * B16 + (3 * D + 2 * steps)[:, None]) + 2.0**-62
    g = (g * told)[:, None]
    dx = g * ((p - t) @ W)
    tol = g.abs() * (torch.where(t > 0, dt, dp) @ W.abs() + (N / 16 + 80) * 2 * U * ((p + t) @ W.abs())) * 1.01
    return {"loss": loss, "lse": lse, "dx": dx, "tol_lse": D + steps,
            "tol_loss": T * T * (2 * D + 2 * steps + 64 * U * entropy.abs()),
            "tol_dx": tol + dx.abs() * 1.01 * B16 + 1e-38}


def compare_with_infinities(got, ref, rows, columns=slice(None)):
    """What is finite in fp32 within its tolerance, the rest the same infinity."""
    for name, have in zip(("loss", "lse", "dx"), got):
        want, tol, have = ref[name][rows], ref["tol_" + name][rows], have[rows]
        if name == "dx":
            want, tol, have = want[:, columns], tol[:, columns], have[:, columns]
        far = torch.isinf(want.float())
        assert torch.equal(have[far].float(), want[far].float()), name
        assert torch.isfinite(have[~far]).all(), name
        worst = ((have.double() - want).abs() / tol)[~far].max().item()
        assert worst <= 1, f"{name}: {worst:.3g} of the tolerance"


BIG = 2.0**100  # times -2^40: past fp32's range, from finite values


@gpu
@pytest.mark.parametrize("distill", [False, True])
@pytest.mark.parametrize("M,N,gone_at", [(20, 700, (300, 301)), (128, 700, (0, 1)), (300, 1400, (1399, 1400)),
                                         (20, 1400, (256, 700)), (300, 1400, (512, 1100))])
def test_logits_of_minus_infinity(L, distill, M, N, gone_at):
    """Every other token has logits of -inf at some entries (one, or whole segments of 128): they are its label, slots
    of its teacher, or neither."""
    K, T = 128, 2.0 if distill else 1.0
    _, values, X, labels, g = make(M + N, M, N, K)
    at = torch.arange(*gone_at)
    W = values.float()
    W[:, 0] = 0
    W[at.cuda(), 0] = -(2.0**40)
    X[:, 0] = 0
    X[::2, 0] = BIG
    head = W.bfloat16()
    gone = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    gone[::2, gone_at[0]:gone_at[1]] = True
    dloss = torch.rand(M, generator=g).cuda() + 0.5
    if distill:
        idx, t = teacher(g, M, N, 6, False)
        idx[4:, 0] = torch.where(torch.arange(4, M) % 4 < 2, at[0], 7 if at[0] > 7 else N - 1).cuda()
        targets = distill_targets(idx, t, N, T)
        got = qb.qlora_head_distill(head, X, idx, t, T, dloss=dloss)
    else:
        labels[6:12], labels[5], labels[4] = at[-1], -100, -100
        targets = xent_targets(labels, N)
        got = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    ref = with_gone(head, X, gone, T, *targets, dloss)
    assert torch.isinf(ref["loss"]).sum() >= 3
    compare_with_infinities(got, ref, slice(None))
    assert qb.device_status() == 0


@gpu
@pytest.mark.parametrize("M", [20, 300])
def test_an_infinite_weight(L, M):
    """An entry of W at -inf: that logit is -inf for every token whose value there is positive; the other columns of dX
    are those of a probability of 0."""
    N, K, j, c = 700, 128, 333, 5
    _, values, X, labels, g = make(M, M, N, K)
    labels[3], labels[4] = j, -100
    X[:, c] = X[:, c].abs() + 0.5
    dloss = torch.rand(M, generator=g).cuda() + 0.5
    finite = values.clone()
    finite[:, c] = 0
    gone = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    gone[:, j] = True
    head = finite.clone()
    head[j, c] = -math.inf
    got = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    compare_with_infinities(got, with_gone(finite, X, gone, 1.0, *xent_targets(labels, N), dloss), slice(None),
                            [k for k in range(K) if k != c])
    assert got[0][3] == math.inf and got[0][4] == 0 and (got[2][4] == 0).all()


@gpu
@pytest.mark.parametrize("M", [20, 300])
def test_all_logits_infinite_and_plus_infinity(L, M):
    N, K = 700, 128
    _, values, X, labels, g = make(M, M, N, K)
    W = values.float()
    W[:, 0] = -(2.0**20)
    X[:, 0] = 0
    head = W.bfloat16()
    labels[6] = -100
    idx, t = teacher(g, M, N, 6, False, empty=False)
    idx[6] = -1
    dloss = torch.rand(M, generator=g).cuda() + 0.5
    calls = (lambda x: qb.qlora_head_xent(head, x, labels, dloss=dloss),
             lambda x: qb.qlora_head_distill(head, x, idx, t, 2.0, dloss=dloss))
    for call in calls:
        good = call(X)
        X2 = X.clone()
        X2[5:7, 0] = 2.0**120   # every logit -inf
        X2[10:12, 0] = -(2.0**120)  # every logit +inf
        loss, lse, dx = call(X2)
        assert (lse[5:7] == -math.inf).all() and torch.isnan(loss[5]) and torch.isnan(dx[5]).all()
        assert loss[6] == 0 and (dx[6] == 0).all()
        assert torch.isnan(loss[10:12]).all() and torch.isnan(lse[10:12]).all() and torch.isnan(dx[10:12]).all()
        rest = [i for i in range(M) if i not in (5, 6, 10, 11)]
        assert all(torch.equal(a[rest], b[rest]) for a, b in zip(good, (loss, lse, dx)))


@gpu
@pytest.mark.parametrize("M", [20, 300])
def test_logits_that_the_temperature_makes_infinite(L, M):
    """Finite logits of -2^120 over T = 1e-4, in whole segments and as slots."""
    N, K, T = 1400, 128, 1e-4
    _, values, X, _, g = make(M, M, N, K)
    W = values.float()
    W[:, 0] = 0
    W[512:900, 0] = -(2.0**40)
    X[:, 0] = 0
    X[::2, 0] = 2.0**80
    head = W.bfloat16()
    gone = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    gone[::2, 512:900] = True
    idx, t = teacher(g, M, N, 6, False, empty=False)
    idx[:, 0] = torch.where(torch.arange(M) % 3 == 0, 600, 3).cuda()
    t[:, 0] = 20.0
    dloss = torch.rand(M, generator=g).cuda() + 0.5
    got = qb.qlora_head_distill(head, X, idx, t, T, dloss=dloss)
    ref = with_gone(head, X, gone, T, *distill_targets(idx, t, N, T), dloss)
    assert torch.isinf(ref["loss"]).sum() >= 3
    compare_with_infinities(got, ref, slice(None))


def test_workspace_of_large_vocabularies(L):
    """The default's bounds: 1 GB of exponentials with a gradient, of statistics and targets without, or what 256 tokens
    take.  Beside the exponentials (2 N bytes a token) lie the targets (16 k) and statistics (N / 8 at most): together at
    most a quarter of them where N >= 2^15 for k = 256."""
    GB = 1 << 30
    for lg in range(10, 25):
        N = 1 << lg
        for k in (0, 256):
            for M in (257, 16384, 1 << 20):
                few = qb.head_workspace_bytes(256, N, 512, k)
                if k == 0 or lg >= 15:
                    assert qb.head_workspace_bytes(M, N, 512, k) <= 1.25 * max(GB, few)
                few = qb.head_workspace_bytes(256, N, 512, k, want_dx=False)
                assert qb.head_workspace_bytes(M, N, 512, k, want_dx=False) <= 1.25 * max(GB, few)
    # an ordinary vocabulary still goes 16384 tokens at a time
    assert qb.head_workspace_bytes(1 << 20, 128000, 512, want_dx=False) == qb.head_workspace_bytes(
        16384, 128000, 512, want_dx=False) > qb.head_workspace_bytes(8192, 128000, 512, want_dx=False)


@gpu
def test_losses_of_a_large_vocabulary_in_several_pieces(L):
    """A vocabulary whose statistics bound the piece: 4609 tokens at 2 M entries go 2560 at a time."""
    M, N, K = 4609, (1 << 21) + 5, 64
    nbytes = qb.head_workspace_bytes(M, N, K, want_dx=False)
    assert nbytes == qb.head_workspace_bytes(M, N, K, want_dx=False, piece=2560) < M * (N / 128) * 8
    g = torch.Generator("cuda").manual_seed(3)
    W = (torch.randn(N, K, generator=g, device="cuda") * 0.05).bfloat16()
    X = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    labels = torch.randint(0, N, (M,), generator=g, device="cuda")
    labels[:3] = torch.tensor([0, N - 1, N])
    labels[-2:] = torch.tensor([N - 1, -100])
    loss, lse, _ = qb.qlora_head_xent(W, X, labels)
    rows = torch.tensor([0, 1, 2, 255, 256, 2559, 2560, 2561, 4607, 4608, M - 2, M - 1], device="cuda")
    ref = reference(W, X[rows], 1.0, *xent_targets(labels[rows], N), None, piece=4)
    compare((loss[rows], lse[rows], None), ref)
    again = qb.qlora_head_xent(W, X, labels)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse) and torch.isfinite(loss).all()


@gpu
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,N,K,k,T,bf16", [
    (1, 300, 256, 1, 1.0, False), (2, 9, 256, 5, 2.0, True), (37, 9001, 512, 33, 1.5, True), (16, 32000, 1024, 64, 2.0, False),
    (100, 1031, 256, 256, 0.5, False), (128, 2049, 768, 7, 4.0, True), (200, 1031, 512, 12, 1.0, False),
    (515, 4099, 256, 100, 2.0, True), (384, 600, 256, 3, 1e-3, False),
])
@pytest.mark.parametrize("block,dq", [(32, 0), (32, 256), (64, 256), (128, 0), (256, 256)])
def test_distill_nf4_head(L, block, dq, M, N, K, k, T, bf16, grad):
    head, values, X, _, g = make(block + dq + M, M, N, K, block, dq)
    idx, t = teacher(g, M, N, k, bf16)
    dloss = torch.randn(M, generator=g).cuda() if grad else None
    ref = reference(values, X, T, *distill_targets(idx, t, N, T), dloss)
    got = qb.qlora_head_distill(head, X, idx, t, T, dloss=dloss)
    compare(got, ref)
    same = qb.qlora_head_distill(values, X, idx, t, T, dloss=dloss)  # the bf16 values as a head
    compare(same, ref)
    if M <= 64 or M > 128:
        assert all(a is b or torch.equal(a, b) for a, b in zip(got, same))
    nbytes = qb.head_workspace_bytes(M, N, K, k, grad, True, piece=256)  # a last piece of few tokens on the expanded head
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    compare(qb.qlora_head_distill(head, X, idx, t, T, dloss=dloss, workspace=ws), ref)
    assert qb.device_status() == 0


def of_bytes(nbytes, value):
    """A workspace of `nbytes` bytes of one value, and a guard behind it."""
    ws = torch.full((nbytes + 4096,), value, dtype=torch.uint8, device="cuda")
    ws[nbytes:] = 171
    return ws


@gpu
@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M", [1, 16, 17, 100, 128, 129, 256, 257, 390, 700])
def test_nothing_is_read_that_was_not_written(L, M, nf4):
    """A workspace of NaNs (0xFF in bf16 and fp32, a label or slot of -1) and one of zeros: the same finite results, at
    vocabularies around the multiples of all that columns come in."""
    for N in (1, 31, 32, 33, 63, 64, 65, 111, 113, 127, 128, 129, 159, 161, 223, 225, 255, 256, 257, 500, 513, 895, 1025):
        for K in (64, 192, 576):
            head, values, X, labels, g = make(M + N + K, M, N, K, 64 if nf4 else 0)
            labels[M // 2] = -100 if M > 1 else labels[M // 2]
            idx, t = teacher(g, M, N, 3, False)
            dloss = torch.rand(M, generator=g).cuda() + 0.1
            for w in (None, dloss):
                for piece in (0, 256):
                    for k in (0, 3):
                        nbytes = qb.head_workspace_bytes(M, N, K, k, w is not None, nf4, piece)
                        got = []
                        for value in (255, 0):
                            ws = of_bytes(nbytes, value)
                            if k:
                                got.append(qb.qlora_head_distill(head, X, idx, t, 2.0, dloss=w, workspace=ws[:nbytes]))
                            else:
                                got.append(qb.qlora_head_xent(head, X, labels, dloss=w, workspace=ws[:nbytes]))
                            assert (ws[nbytes:] == 171).all(), (N, K, k)
                        for a, b in zip(*got):
                            assert a is b or (torch.equal(a, b) and torch.isfinite(a).all()), (N, K, k)
    assert qb.device_status() == 0


@gpu
@pytest.mark.parametrize("M,piece", [(700, 512), (900, 256), (384, 256)])
def test_pieces_of_a_workspace_of_nans(L, M, piece):
    """As in test_head.test_pieces_of_tokens, against the definition."""
    for N, K in ((1000, 192), (3001, 512), (4097, 64)):
        head, values, X, labels, g = make(M + N, M, N, K)
        idx, t = teacher(g, M, N, 9, False)
        dloss = torch.rand(M, generator=g).cuda()
        nbytes = qb.head_workspace_bytes(M, N, K, 9, piece=piece)
        ws = of_bytes(nbytes, 255)
        got = qb.qlora_head_distill(head, X, idx, t, 2.0, dloss=dloss, workspace=ws[:nbytes])
        compare(got, reference(values, X, 2.0, *distill_targets(idx, t, N, 2.0), dloss))
        assert (ws[nbytes:] == 171).all()
        nbytes = qb.head_workspace_bytes(M, N, K, piece=piece)
        ws = of_bytes(nbytes, 255)
        got = qb.qlora_head_xent(head, X, labels, dloss=dloss, workspace=ws[:nbytes])
        compare(got, reference(values, X, 1.0, *xent_targets(labels, N), dloss))
        assert (ws[nbytes:] == 171).all()


@gpu
@pytest.mark.slow
@pytest.mark.parametrize("M", [5, 200])
def test_offsets_into_a_head_past_32_bits(L, M):
    """More than 2^31 weights in bf16, in NF4, and (200 tokens) in the copy that an NF4 head is expanded to; entries at
    both ends are labels, slots, and what single tokens put all their probability on."""
    N, K, k = 135001, 16384, 3
    assert N * K > 2**31
    g = torch.Generator("cuda").manual_seed(9)
    codes = torch.randint(0, 256, (N * K // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.rand(N * K // 64, generator=g, device="cuda") * 0.02 + 0.01
    head = qb.NF4Weight(codes, torch.empty(0, dtype=torch.uint8, device="cuda"), scale, N, K, 64, 0)
    values = qb.nf4_dequantize(head)
    ends = torch.tensor([0, N - 1, N // 2, 131071, 131072, 131073, N - 2, 7], device="cuda")
    labels, liked = ends[torch.arange(M, device="cuda") % 8], ends[(torch.arange(M, device="cuda") + 1) % 8]
    X = torch.randn(M, K, generator=g, device="cuda") * 0.05
    X = (X + values[liked].float() * (30 / values[liked].float().square().sum(1, keepdim=True))).bfloat16()
    idx = torch.stack((labels, liked, torch.full_like(labels, -1)), 1)
    t = torch.randn(M, k, generator=g, device="cuda")
    dloss = torch.ones(M, device="cuda")
    z = torch.cat([X.double() @ values[i:i + 15000].double().T for i in range(0, N, 15000)], 1)
    assert (z.argmax(1) == liked).all()
    D = ((K / 16 + 16) * 2 * U * X.double().abs().sum(1) * values.abs().max().double())[:, None]
    for T, targets in ((1.0, xent_targets(labels, N)), (2.0, distill_targets(idx, t, N, 2.0))):
        call = ((lambda h: qb.qlora_head_xent(h, X, labels, dloss=dloss)) if T == 1.0 else
                (lambda h: qb.qlora_head_distill(h, X, idx, t, 2.0, dloss=dloss)))
        a, b = call(head), call(values)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        q, at, entropy = (v.double() if v.is_floating_point() else v for v in targets)
        lse = torch.logsumexp(z / T, 1)
        loss = T * T * (entropy + (q * (lse[:, None] - z.gather(1, at) / T)).sum(1))
        d = (z / T - lse[:, None]).exp().scatter_add_(1, at, -q)
        dx = T * sum(d[:, i:i + 15000] @ values[i:i + 15000].double() for i in range(0, N, 15000))
        assert ((a[1] - lse).abs() <= 2 * D[:, 0]).all() and ((a[0] - loss).abs() <= 4 * T * T * D[:, 0]).all()
        # a wrong row of W anywhere would be an error as large as the row's gradient itself
        assert ((a[2].double() - dx).norm(dim=1) <= 1e-2 * dx.norm(dim=1)).all()


@gpu
@pytest.mark.slow
def test_offsets_into_the_exponentials_past_32_bits(L):
    """A piece of 256 tokens times 8.4 M entries: more than 2^31 exponentials.  Each token puts nearly all its probability
    on an entry of its own, spread from the first to the last, which is not its label."""
    M, N, K = 256, (1 << 23) + 4099, 64
    assert M * N > 2**31
    g = torch.Generator("cuda").manual_seed(10)
    W = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    liked = (torch.arange(M, device="cuda") * (N - 1)) // (M - 1)
    labels = (liked + N // 2) % N
    X = (W[liked].float() * (40 / W[liked].float().square().sum(1, keepdim=True))).bfloat16()
    dloss = torch.ones(M, device="cuda")
    loss, lse, dx = qb.qlora_head_xent(W, X, labels, dloss=dloss)
    W64 = W.double()
    for a in range(0, M, 16):
        s = slice(a, a + 16)
        z = X[s].double() @ W64.T
        want = torch.logsumexp(z, 1)
        D = (K / 16 + 16) * 2 * U * (X[s].double().abs() @ W64.abs().T).amax(1) + 160 * U * (z.abs().amax(1) + want.abs() + 1)
        assert ((lse[s] - want).abs() <= D).all()
        assert ((loss[s] - (want - z.gather(1, labels[s, None])[:, 0])).abs() <= 2 * D + 2 * U * loss[s]).all()
        p = (z - want[:, None]).exp()
        assert (p.gather(1, liked[s, None]) > 0.9).all()
        grad = p @ W64 - W64[labels[s]]
        assert ((dx[s].double() - grad).norm(dim=1) <= 1e-2 * grad.norm(dim=1)).all()


@gpu
@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M", [1, 100, 128, 200, 2000])
def test_logit_of_the_label_is_summed_to_nearest(L, M, nf4):
    """A label's logit of about -20 out of 16384 products of one sign beside logits of 0, so that the loss is the logit
    and log(N - 128) alone.  Sums to nearest: a lane adds at most K / 32 products (every fp32 step is off by at most
    U of a partial sum, which grows evenly: K / 64 U of the whole), then 5 steps join the lanes, and 12 roundings of
    |loss| follow.  A sum that truncates, K / 16 steps in one to four parts, is off by more in the long run."""
    N, K = 400, 16384
    g = wl.generator(M)
    X = (torch.rand(M, K, generator=g) + 0.25).bfloat16().cuda()
    W = torch.zeros(N, K)
    W[:128] = -(torch.rand(128, K, generator=g) + 0.5) * (20 / (0.75 * K))
    labels = (torch.arange(M) % 128).cuda()
    head = qb.nf4_quantize(W.cuda()) if nf4 else W.bfloat16().cuda()
    values = (qb.nf4_dequantize(head) if nf4 else head).double()
    assert (values[128:] == 0).all()
    dloss = torch.ones(M, device="cuda")
    loss, lse, dx = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    z = X.double() @ values.T
    want = torch.logsumexp(z, 1) - z.gather(1, labels[:, None])[:, 0]
    assert (z.gather(1, labels[:, None]) < -15).all()
    tol = (K / 64 + 5) * U * z.gather(1, labels[:, None])[:, 0].abs() + 12 * U * want
    assert ((loss - want).abs() <= tol).all(), ((loss - want).abs() / tol).max()
    assert ((lse - torch.logsumexp(z, 1)).abs() <= 12 * U * 6).all()


def draw_lean(seed, M, N, K, lean):
    """Hidden states that lean towards their labels and an NF4 head of spread 0.03, as a trained one has."""
    g = torch.Generator("cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N * K // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scale = 0.052 * (0.7 + 0.6 * torch.rand(N * K // 64, generator=g, device="cuda"))
    head = qb.NF4Weight(codes, torch.empty(0, dtype=torch.uint8, device="cuda"), scale, N, K, 64, 0)
    values = qb.nf4_dequantize(head)
    labels = torch.randint(0, N, (M,), generator=g, device="cuda")
    rows = values[labels].float()
    X = torch.randn(M, K, generator=g, device="cuda")
    X += rows * (lean * torch.rand(M, 1, generator=g, device="cuda") / rows.square().sum(1, keepdim=True))
    return head, values, X.bfloat16(), labels, g


def six_digits(head, values, X, labels, idx, t, T):
    """Loss and lse of both operators hold six digits over the call: a relative 2-norm error of at most 1e-6."""
    N = values.shape[0]
    for got, targets, temp in ((qb.qlora_head_xent(head, X, labels), xent_targets(labels, N), 1.0),
                               (qb.qlora_head_distill(head, X, idx, t, T), distill_targets(idx, t, N, T), T)):
        ref = reference(values, X, temp, *targets, None)
        for name, g in zip(("loss", "lse"), got):
            err = ((g.double() - ref[name]).norm() / ref[name].norm()).item()
            assert err <= 1e-6, f"{name}: {err:.2g}"


@gpu
@pytest.mark.parametrize("K", [2048, 4096, 8192])
@pytest.mark.parametrize("M,N", [(200, 3000), (900, 1000), (300, 20001)])
def test_losses_hold_six_digits(L, M, N, K):
    """The promise of the documents, at the widths where the tensor core's truncating additions would break it: logits
    have a spread of 0.03 sqrt(K) and sums of K / 16 steps."""
    head, values, X, labels, g = draw_lean(M + K, M, N, K, 10.0)
    idx = torch.randint(0, N, (M, 20), generator=g, device="cuda")
    idx[:, 0] = labels
    t = 10.0 - 2.0 * torch.arange(1.0, 21.0, device="cuda").log().expand(M, 20).contiguous()
    six_digits(head, values, X, labels, idx, t, 1.0)


@gpu
@pytest.mark.parametrize("M,K", [(16, 8192), (33, 8192), (64, 4096), (64, 8192), (66, 4096), (96, 6080), (100, 8192),
                                 (113, 4096), (128, 2048), (128, 4096), (128, 8192), (128, 16384)])
@pytest.mark.parametrize("N", [1000, 20001])
def test_losses_of_few_tokens_hold_six_digits(L, N, M, K):
    head, values, X, labels, g = draw_lean(M + K, M, N, K, 10.0)
    idx = torch.randint(0, N, (M, 20), generator=g, device="cuda")
    idx[:, 0] = labels
    t = 10.0 - 2.0 * torch.arange(1.0, 21.0, device="cuda").log().expand(M, 20).contiguous()
    for h in (head, values):  # NF4 and bf16
        six_digits(h, values, X, labels, idx, t, 1.0)


@gpu
@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M,N,K", [(17, 300, 8256), (48, 5000, 4160), (48, 5000, 8192), (64, 300, 4160), (64, 40, 12352),
                                   (80, 700, 2112), (80, 19000, 4096), (97, 33333, 4160), (112, 1000, 8192), (113, 500, 2112),
                                   (128, 2000, 3136), (128, 20001, 4096), (128, 130, 16448)])
def test_contraction_in_rounds(L, M, N, K, nf4):
    """Few tokens whose contraction goes in rounds, several tiles per block among them, with the gradient."""
    head, values, X, labels, g = make(M + N + K, M, N, K, 64 if nf4 else 0, w_std=0.02)
    labels[1], labels[2] = -100, N
    idx, t = teacher(g, M, N, 7, False)
    dloss = torch.randn(M, generator=g).cuda()
    got = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    compare(got, reference(values, X, 1.0, *xent_targets(labels, N), dloss))
    again = qb.qlora_head_xent(head, X, labels, dloss=dloss)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    compare(qb.qlora_head_distill(head, X, idx, t, 2.0, dloss=dloss),
            reference(values, X, 2.0, *distill_targets(idx, t, N, 2.0), dloss))
    assert qb.device_status() == 0


@gpu
@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M", [1, 7, 15, 16])
@pytest.mark.parametrize("k", [3, 40, 200])
def test_gradient_of_a_flat_teacher(L, M, k, nf4):
    """Slots of one weight share a mantissa, so their p - q would round the same way: a token's dX off by up to 2^-9 of
    itself beside its own rounding.  Held to that rounding alone: at most 2^-9 of every value, so of a token's norm;
    the p of entries that are no slots round one by one, an error of 2^-9 sqrt(sum p^2) beside a gradient of
    sqrt(k) / k times a row of W, and the fp32 sums are far below: together under a sixth of 2^-9 here."""
    N, K, T = 20000, 512, 4.0
    head, values, X, _, g = make(M + k, M, N, K, 64 if nf4 else 0, w_std=0.02)
    idx = torch.stack([torch.randperm(N, generator=g)[:k] for _ in range(M)]).cuda()
    t = torch.full((M, k), 1.0, device="cuda")
    dloss = torch.rand(M, generator=g).cuda() + 0.5
    loss, lse, dx = qb.qlora_head_distill(head, X, idx, t, T, dloss=dloss)
    targets = distill_targets(idx, t, N, T)
    ref = reference(values, X, T, *targets, dloss)
    compare((loss, lse, dx), ref)
    p = torch.softmax(X.double() @ values.double().T / T, 1)
    assert (p.square().sum(1).sqrt() < k**-0.5 / 6).all()
    rel = (dx.double() - ref["dx"]).norm(dim=1) / ref["dx"].norm(dim=1)
    assert (rel <= 2.0**-9 * (1 + 1 / 6)).all(), rel.max()


@gpu
@pytest.mark.parametrize("M", [271, 272, 273, 513])
def test_last_piece_in_two_parts(L, M):
    """Pieces of 256 tokens and a last one of 1 to 17, in a workspace of exactly the size that the query returns."""
    for N, K, k in ((1000, 192, 5), (4097, 512, 30)):
        head, values, X, _, g = make(M + N, M, N, K)
        idx, t = teacher(g, M, N, k, False)
        dloss = torch.rand(M, generator=g).cuda()
        nbytes = qb.head_workspace_bytes(M, N, K, k, piece=256)
        ws = of_bytes(nbytes, 255)
        got = qb.qlora_head_distill(head, X, idx, t, 2.0, dloss=dloss, workspace=ws[:nbytes])
        compare(got, reference(values, X, 2.0, *distill_targets(idx, t, N, 2.0), dloss))
        assert (ws[nbytes:] == 171).all()
