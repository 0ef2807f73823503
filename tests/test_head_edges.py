"""The head losses where they could go wrong.  Definition, inputs and tolerances: test_head.py."""
import ctypes
import math

import pytest
import torch
from test_head import make, teacher

from bit_nf4_quantized_24_b200 import binding as qb

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
