"""The order of the kernels of layer calls that follow one another on a stream.

The fused GEMM and the decode kernels read their activations before they wait for the
kernel in front of them (programmatic dependent launch).  That is sound only behind a
kernel that lets its successor start after its own wait: all that precedes it, the last
layer's output among it, is then complete.
"""
import glob
import os
import re

import pytest
import torch

from bit_nf4_quantized_24_b200 import binding as qb
from bit_nf4_quantized_24_b200 import build
from bit_nf4_quantized_24_b200 import workloads as wl

gpu = pytest.mark.gpu
CSRC = os.path.join(build.HERE, "csrc")


@pytest.fixture(scope="module")
def L():
    build.build()
    return qb.lib()


def kernel_bodies(path):
    """name -> source from the kernel's __global__ to the next one (comments taken out)."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    parts = re.split(r"__global__", text)[1:]
    return {re.search(r"(k_\w+)\s*\(", p).group(1): p for p in parts}


def test_adapter_kernels_let_their_successor_start_after_their_own_wait():
    bodies = kernel_bodies(os.path.join(CSRC, "adapter.cu"))
    assert {"k_rows_small", "k_rows", "k_rows_tc", "k_rows_multi", "k_cols", "k_cols_tc"} <= set(bodies)
    for name, body in bodies.items():
        wait, trigger = body.find("pdl_wait();"), body.find("pdl_trigger();")
        assert 0 <= wait < trigger, name


def test_kernels_that_read_before_their_wait_are_the_known_ones():
    """Every other kernel that is launched early waits before anything else (but its trigger and what is its own)."""
    early = set()
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        for name, body in kernel_bodies(path).items():
            wait = body.find("pdl_wait();")
            if wait >= 0 and re.search(r"tma_load|__ldg|ldg_nc|wait_bounded", body[:wait]):
                early.add(name)
    assert early == {"k_nf4_gemm", "k_gemv"}  # and k_gemv_tiles, whose wait stands in front of its loads in the text


# Widths at which the layer's GEMM has whole tiles only and split ones, token counts of the decode kernels, of a
# partly filled tile and of many; rank 64 takes the tcgen05 adapter kernels.
CHAINS = [(1, 1024, 16), (16, 1024, 64), (32, 1024, 16), (300, 1024, 64), (1024, 2048, 16), (2048, 2048, 64)]


def layers(seed, n, D, r):
    out = []
    for i in range(n):
        p = wl.draw_small(seed + i, 16, D, D, r, float(r), b_std=0.05)
        out.append((qb.nf4_quantize(p["W"].cuda()), p["A"].cuda(), p["B"].cuda(), p["scale"]))
    return out


def repeat_without_a_wait(chain, inputs):
    """chain(x, wait) of every input, first with a synchronisation after each call, then with nothing in between: the
    same bits."""
    want = [chain(x, torch.cuda.synchronize) for x in inputs]
    for _ in range(3):
        got = [chain(x, lambda: None) for x in inputs]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert qb.device_status() == 0


@gpu
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("M,D,r", CHAINS)
def test_forward_after_forward(L, M, D, r, shared):
    """Four layers, each on the last one's output; shared: one workspace for all of them."""
    ls = layers(5, 4, D, r)
    ws = torch.empty(qb.fwd_workspace_bytes(M, D, D, r), dtype=torch.uint8, device="cuda") if shared else None
    g = wl.generator(6)

    def chain(x, wait):
        ys = []
        for q, A, B, s in ls:
            x, _ = qb.qlora_linear_fwd(q, x, A, B, s, workspace=ws)
            ys.append(x)
            wait()
        return ys

    repeat_without_a_wait(chain, [torch.randn(M, D, generator=g).bfloat16().cuda() for _ in range(8)])


@gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("M,D,r", CHAINS)
def test_backward_after_backward(L, M, D, r, given):
    """Three layers' backward calls, each on the last one's dX (given: with the forward's H), then without dX."""
    ls = layers(15, 3, D, r)
    ws = torch.empty(qb.bwd_workspace_bytes(M, D, D, r), dtype=torch.uint8, device="cuda")
    g = wl.generator(16)
    X = torch.randn(M, D, generator=g).bfloat16().cuda()
    Hs = [qb.qlora_linear_fwd(q, X, A, B, s)[1] if given else None for q, A, B, s in ls]

    def chain(dy, wait):
        out = []
        for (q, A, B, s), H in zip(ls, Hs):
            dx, da, db = qb.qlora_linear_bwd(q, X, dy, A, B, s, H=H, workspace=ws)
            wait()
            _, da2, db2 = qb.qlora_linear_bwd(q, X, dx, A, B, s, H=H, want_dx=False, workspace=ws)
            wait()
            out += [dx, da, db, da2, db2]
            dy = dx
        return out

    repeat_without_a_wait(chain, [torch.randn(M, D, generator=g).bfloat16().cuda() for _ in range(6)])


@gpu
@pytest.mark.parametrize("M", [1, 5, 16])
def test_decode_after_decode(L, M):
    """The decode forms: decode tiles, one adapter per token, the library's own scratch, row-major codes."""
    D, r = 1024, 16
    ls = layers(25, 4, D, r)
    tiles = [qb.nf4_decode_tiles(q) for q, *_ in ls]
    g = wl.generator(26)
    aidx = (torch.arange(M) % 3 - 1).int().cuda()
    stacks = [(torch.stack((A, A.flip(0))), torch.stack((B, B.flip(1)))) for _, A, B, _ in ls]
    scales = torch.tensor([1.0, 0.5], device="cuda")

    def chain(x, wait):
        ys = []
        for (q, A, B, s), t, (As, Bs) in zip(ls, tiles, stacks):
            for call in (lambda v: qb.qlora_linear_fwd_tiles(q, t, v, A, B, s)[0],
                         lambda v: qb.qlora_linear_fwd_multi(q, v, As, Bs, scales, aidx),
                         lambda v: qb.qlora_linear_fwd_noalloc(q, v, A, B, s)[0],
                         lambda v: qb.qlora_linear_fwd_multi_tiles(q, t, v, As, Bs, scales, aidx)):
                x = call(x)
                ys.append(x)
                wait()
        return ys

    repeat_without_a_wait(chain, [torch.randn(M, D, generator=g).bfloat16().cuda() for _ in range(8)])


@gpu
@pytest.mark.parametrize("M", [12, 200, 1024])
def test_dropout_after_dropout(L, M):
    D, r = 1024, 16
    ls = layers(35, 2, D, r)
    g = wl.generator(36)
    mask = (torch.rand(M, D, generator=g) > 0.1).to(torch.uint8).cuda()

    def chain(x, wait):
        out, xs = [], []
        for q, A, B, s in ls:
            xs.append(x)
            x, _ = qb.qlora_linear_fwd_dropout(q, x, A, B, s, mask, 1 / 0.9)
            wait()
            out.append(x)
        dy = x
        for (q, A, B, s), xi in zip(reversed(ls), reversed(xs)):
            dy, da, db = qb.qlora_linear_bwd_dropout(q, xi, dy, A, B, s, mask, 1 / 0.9)
            wait()
            out += [dy, da, db]
        return out

    repeat_without_a_wait(chain, [torch.randn(M, D, generator=g).bfloat16().cuda() for _ in range(6)])


@gpu
@pytest.mark.parametrize("M", [8, 512])
def test_captured_chain(L, M):
    """The forward chain and its head loss in a graph, replayed over new inputs."""
    D, r, V = 1024, 16, 3003
    ls = layers(45, 4, D, r)
    g = wl.generator(46)
    head = (torch.randn(V, D, generator=g) * 0.05).bfloat16().cuda()
    labels = torch.randint(0, V, (M,), generator=g).cuda()
    dloss = torch.full((M,), 1.0 / M, device="cuda")
    x0 = torch.randn(M, D, generator=g).bfloat16().cuda()

    def chain(x, wait):
        out, xs = [], []
        for q, A, B, s in ls:
            xs.append(x)
            x, _ = qb.qlora_linear_fwd(q, x, A, B, s)
            out.append(x)
            wait()
        loss, lse, dy = qb.qlora_head_xent(head, x, labels, dloss=dloss)
        out += [loss, lse, dy]
        wait()
        for (q, A, B, s), xi in zip(reversed(ls), reversed(xs)):
            dy, da, db = qb.qlora_linear_bwd(q, xi, dy, A, B, s)
            out += [dy, da, db]
            wait()
        return out

    chain(x0, torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(x0, lambda: None)
    for _ in range(5):
        x0.copy_(torch.randn(M, D, generator=g))
        want = chain(x0, torch.cuda.synchronize)
        for _ in range(4):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def stream_of(t):
    """The stream that the allocator holds t's memory for."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@gpu
@pytest.mark.parametrize("M", [4, 64])
def test_what_a_call_allocates_belongs_to_its_stream(L, M):
    """With stream= outputs and workspace come from that stream's memory, and memory whose last use on the caller's
    stream is still to run is not written."""
    D, r = 1024, 16
    (q, A, B, s), = layers(55, 1, D, r)
    g = wl.generator(56)
    X = torch.randn(M, D, generator=g).bfloat16().cuda()
    W = torch.randn(D, D, generator=g).cuda()
    mask = torch.ones(M, D, dtype=torch.uint8, device="cuda")
    tiles = qb.nf4_decode_tiles(q)
    aidx, scales = torch.zeros(M, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    calls = [lambda st: qb.qlora_linear_fwd(q, X, A, B, s, stream=st),
             lambda st: qb.qlora_linear_fwd(q, X, A, B, s, True, None, None, st),
             lambda st: qb.qlora_linear_bwd(q, X, X, A, B, s, stream=st),
             lambda st: qb.qlora_linear_fwd_dropout(q, X, A, B, s, mask, 1.0, stream=st),
             lambda st: qb.qlora_linear_bwd_dropout(q, X, X, A, B, s, mask, 1.0, stream=st),
             lambda st: qb.qlora_linear_fwd_noalloc(q, X, A, B, s, stream=st),
             lambda st: (qb.nf4_dequantize(q, stream=st), qb.nf4_decode_tiles(q, stream=st)),
             lambda st: [getattr(qb.nf4_quantize(W, stream=st), n) for n in ("codes", "absmax_q", "dq_scale")],
             lambda st: [getattr(qb.nf4_merge_lora(q, A, B, s, stream=st), n) for n in ("codes", "absmax_q")]]
    if M <= 16:
        calls += [lambda st: qb.qlora_linear_fwd_tiles(q, tiles, X, A, B, s, stream=st),
                  lambda st: (qb.qlora_linear_fwd_multi(q, X, A[None], B[None], scales, aidx, stream=st),
                              qb.qlora_linear_fwd_multi_tiles(q, tiles, X, A[None], B[None], scales, aidx, stream=st))]
    for call in calls:
        side = torch.cuda.Stream()
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        sums, blocks = [], [torch.full_like(t, 3) for t in want for _ in range(2)]
        torch.cuda._sleep(20_000_000)  # about 10 ms on the caller's stream
        for b in blocks:
            sums.append((b == 3).sum() == b.numel())
        del blocks, b
        got = call(side)
        assert all(stream_of(t) == side.cuda_stream for t in got)
        torch.cuda.synchronize()
        assert all(sums) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert qb.device_status() == 0
