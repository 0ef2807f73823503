"""Measured cases of the head losses: softmax cross entropy and distillation from a teacher's top logits,
both through a frozen output head [N, K] (bf16, or NF4 as the layer stores its weights), with the gradient
of the head's input.  `run` computes them in plain torch operations, or through the framework when `own`."""
import math

import torch

own = False

# The ascending NF4 levels of the weight format (nf4_codebook).
LEVELS = [-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976, -0.2844413220882416,
          -0.18477340042591095, -0.09104997664690018, 0.0, 0.07958031445741653, 0.16093014180660248,
          0.24611225724220276, 0.3379151225090027, 0.4407097399234772, 0.5626168847084045, 0.722956657409668, 1.0]
IGNORE = -100
LARGEST = 4 * 4096 * 128000 * 8192  # floating-point operations of the largest listed case


def _xent(name, M, N, K, grad, block=0, dq=0):
    return {"name": name, "op": "xent", "M": M, "N": N, "K": K, "grad": grad, "block": block, "dq": dq}


def _distill(name, M, N, K, grad, k, T, bf16_teacher, block=0, dq=0):
    return {"name": name, "op": "distill", "M": M, "N": N, "K": K, "grad": grad, "k": k, "T": T,
            "bf16_teacher": bf16_teacher, "block": block, "dq": dq}


def listed():
    """block 0: a bf16 head; otherwise an NF4 head with blocks of that many weights (dq 256: double quantization)."""
    return [
        # one answer's token scored by a small model: launch latency
        _xent("xent_score_1", 1, 8000, 512, False),
        # one token scored through an ordinary head: the head's bytes
        _xent("xent_score_1_wide", 1, 32000, 4096, False),
        # a handful of tokens scored through a head that is kept in NF4
        _xent("xent_score_nf4", 16, 32000, 4096, False, 64, 256),
        # perplexity of a held-out text: no gradient, ragged token count, a vocabulary of odd size
        _xent("xent_eval_odd", 2047, 50003, 2048, False),
        # the step of a short prompt: few tokens, with gradient
        _xent("xent_step_short", 128, 32000, 2048, True),
        # the ordinary fine-tuning step (the token count and width of the layer's own workloads)
        _xent("xent_step", 4096, 32000, 4096, True),
        # the same step with the head in NF4
        _xent("xent_step_nf4", 2048, 32000, 4096, True, 64, 256),
        # a long packed batch over a large vocabulary: where keeping the logits would cost gigabytes
        _xent("xent_step_large", 8192, 128000, 4096, True),
        # a teacher's stored answers scored by the student
        _distill("distill_score", 64, 32000, 4096, False, 16, 1.0, False),
        # the ordinary distillation step
        _distill("distill_step", 2048, 32000, 4096, True, 64, 2.0, False),
        # few stored logits in bf16, odd sizes
        _distill("distill_step_odd", 515, 50003, 2048, True, 7, 1.5, True),
        # the widest head of the workloads, large vocabulary, many stored logits
        _distill("distill_step_large", 4096, 128000, 8192, True, 128, 2.0, True),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    """Token counts 1 .. 8192, vocabularies 1000 .. 131072, widths 512 .. 8192, 1 .. 128 teacher logits."""
    while True:
        M, N = _log(rng, 1, 8192), _log(rng, 1000, 131072)
        K = 64 * _log(rng, 8, 128)
        grad = rng.random() < 0.65
        block = rng.choice([0, 0, 0, 32, 64, 128, 256])
        dq = rng.choice([0, 256])
        if block and K % block:
            block = 64
        if not block:
            dq = 0
        if (4 if grad else 2) * M * N * K > LARGEST:
            continue
        c = {"op": "xent", "M": M, "N": N, "K": K, "grad": grad, "block": block, "dq": dq}
        if rng.random() < 0.45:
            c.update(op="distill", k=_log(rng, 1, 128), T=rng.choice([1.0, 1.5, 2.0, 4.0]),
                     bf16_teacher=rng.random() < 0.5)
        return c


def _dequantize(head, N, K, block, dq):
    """bf16 [N, K] of an NF4 weight: level * absmax in fp32, rounded once to bf16."""
    codes, absmax_q, dq_scale = head
    levels = torch.tensor(LEVELS, dtype=torch.float32, device=codes.device)
    scale = dq_scale
    if dq:
        scale = absmax_q.float() * dq_scale.repeat_interleave(dq)[:absmax_q.numel()]
    pairs = torch.stack((codes & 15, codes >> 4), -1).view(-1, block).int()
    return (levels[pairs] * scale.view(-1, 1)).bfloat16().view(N, K)


def prepare(case, seed):
    """A head, hidden states behind a norm that lean towards their labels, labels with a tenth left out (prompt
    and padding), a mean's weights as the loss's gradient, and a teacher's distinct tokens with falling logits,
    fewer in some rows (index -1) and none in a few."""
    g = torch.Generator("cuda").manual_seed(seed)
    M, N, K = case["M"], case["N"], case["K"]
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if case["block"]:
        blocks = N * K // case["block"]
        codes = torch.randint(0, 256, (N * K // 2,), generator=g, device="cuda", dtype=torch.uint8)
        peak = 0.02 * 2.6 * (0.7 + 0.6 * rand(-(-blocks // 256) if case["dq"] else blocks))
        absmax_q = torch.empty(0, dtype=torch.uint8, device="cuda")
        if case["dq"]:
            absmax_q = torch.randint(120, 256, (blocks,), generator=g, device="cuda", dtype=torch.uint8)
            peak = peak / 200
        head = (codes, absmax_q, peak.float())
        w = None
    else:
        w = torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16).mul_(0.02)
        head = (w,)
    labels = torch.randint(0, N, (M,), generator=g, device="cuda")
    x = randn(M, K)
    if w is not None:
        rows = w[labels].float()
    else:
        rows = _dequantize(head, N, K, case["block"], case["dq"])[labels].float()
    x = (x + rows * (10.0 * rand(M, 1) / rows.square().sum(1, keepdim=True))).bfloat16()
    state = {"case": case, "head": head, "x": x, "dloss": None}
    left_out = rand(M) < 0.1
    left_out[0] = False
    if case["op"] == "xent":
        state["labels"] = torch.where(left_out, IGNORE, labels)
        if case["grad"]:
            state["dloss"] = torch.full((M,), 1.0, device="cuda") / (~left_out).sum()
    else:
        k = case["k"]
        gaps = 1 + ((N // k - 1) * rand(M, k) ** 4).long()
        idx = (labels[:, None] + torch.cumsum(gaps, 1) - gaps) % N
        idx = idx.gather(1, torch.cat((torch.zeros(M, 1, dtype=torch.long, device="cuda"),
                                       1 + torch.argsort(rand(M, k - 1), 1)), 1))
        t = 10.0 - 2.0 * torch.log1p(torch.arange(k, device="cuda").float()) + 0.3 * randn(M, k)
        t = t.sort(1, descending=True).values
        kept = 1 + (rand(M, 1) * 2 * k).long()
        idx = torch.where(torch.arange(k, device="cuda") < kept, idx, -1)
        idx[rand(M) < 0.03] = -1
        state["idx"] = idx
        state["t"] = t.bfloat16() if case["bf16_teacher"] else t
        if case["grad"]:
            state["dloss"] = torch.full((M,), 1.0 / M, device="cuda")
    return state


def run(state):
    """{"loss", "lse"} in fp32 and, where the case asks for it, the gradient "dx" in bf16."""
    case = state["case"]
    N, K = case["N"], case["K"]
    if own:
        from bit_nf4_quantized_24_b200 import binding as qb

        head = state["head"]
        head = qb.NF4Weight(*head, N, K, case["block"], case["dq"]) if case["block"] else head[0]
        if case["op"] == "xent":
            loss, lse, dx = qb.qlora_head_xent(head, state["x"], state["labels"], dloss=state["dloss"])
        else:
            loss, lse, dx = qb.qlora_head_distill(head, state["x"], state["idx"], state["t"], case["T"],
                                                  dloss=state["dloss"])
        return {"loss": loss, "lse": lse} if dx is None else {"loss": loss, "lse": lse, "dx": dx}
    w = _dequantize(state["head"], N, K, case["block"], case["dq"]) if case["block"] else state["head"][0]
    w = w.float()
    z = state["x"].float() @ w.T
    if case["op"] == "xent":
        T = 1.0
        labels = state["labels"][:, None]
        idx = labels.clamp(min=0)
        q = (labels >= 0).float()
        valid = labels >= 0
        log_q = torch.zeros_like(q)
    else:
        T = case["T"]
        valid = state["idx"] >= 0
        idx = state["idx"].clamp(min=0)
        t = torch.where(valid, state["t"].float() / T, -math.inf)
        top = t.amax(1, keepdim=True)
        t = t - torch.where(valid.any(1, keepdim=True), top, 0.0)
        total = t.exp().sum(1, keepdim=True)
        q = torch.where(valid, t.exp() / total, 0.0)
        log_q = torch.where(valid, t - total.log(), 0.0)
        z = z / T
    m = z.amax(1, keepdim=True)
    lse = m + (z - m).exp().sum(1, keepdim=True).log()
    picked = z.gather(1, idx)
    loss = T * T * (q * (log_q - (picked - lse))).sum(1)
    out = {"loss": loss, "lse": lse[:, 0]}
    if state["dloss"] is not None:
        p = z.sub_(lse).exp_()
        p *= valid.any(1, keepdim=True)
        p.scatter_add_(1, idx, -q)
        p *= (T * state["dloss"])[:, None]
        out["dx"] = (p @ w).bfloat16()
    return out


def exact(case, seed):
    """The definition in 64 bits, a piece of tokens at a time."""
    s = prepare(case, seed)
    M, N, K = case["M"], case["N"], case["K"]
    if case["block"]:  # the stored weight is the bf16 value that the format defines
        codes, absmax_q, dq_scale = s["head"]
        low, high = codes.long() % 16, codes.long() // 16
        level = torch.tensor(LEVELS, device="cuda", dtype=torch.float32)[torch.stack((low, high), 1).flatten()]
        of_block = torch.arange(N * K // case["block"], device="cuda")
        peak = absmax_q[of_block].float() * dq_scale[of_block // case["dq"]] if case["dq"] else dq_scale[of_block]
        w = (level.view(-1, case["block"]) * peak[:, None]).to(torch.bfloat16).reshape(N, K).double()
    else:
        w = s["head"][0].double()
    loss, lse = (torch.zeros(M, device="cuda", dtype=torch.float64) for _ in range(2))
    dx = torch.zeros(M, K, device="cuda", dtype=torch.float64) if case["grad"] else None
    for a in range(0, M, 1024):
        b = min(M, a + 1024)
        logits = torch.mm(s["x"][a:b].double(), w.t())
        target = torch.zeros_like(logits)  # the distribution that the student is held to
        if case["op"] == "xent":
            T, entropy = 1.0, 0.0
            here = torch.nonzero(s["labels"][a:b] >= 0)[:, 0]
            target[here, s["labels"][a:b][here]] = 1.0
        else:
            T = case["T"]
            row, slot = torch.nonzero(s["idx"][a:b] >= 0, as_tuple=True)
            teacher = torch.full((b - a, case["k"]), -math.inf, device="cuda", dtype=torch.float64)
            teacher[row, slot] = s["t"][a:b][row, slot].double() / T
            log_q = torch.log_softmax(teacher, 1)[row, slot]
            target[row, s["idx"][a:b][row, slot]] = log_q.exp()
            entropy = torch.zeros(b - a, device="cuda", dtype=torch.float64).index_add_(0, row, log_q.exp() * log_q)
        logits /= T
        lse[a:b] = torch.logsumexp(logits, 1)
        told = target.sum(1) > 0
        log_p = logits - lse[a:b, None]
        loss[a:b] = torch.where(told, T * T * (entropy - (target * log_p).sum(1)), 0.0)
        if dx is not None:
            dz = torch.where(told[:, None], T * (log_p.exp() - target), 0.0) * s["dloss"][a:b, None].double()
            dx[a:b] = torch.mm(dz, w)
    return {"loss": loss, "lse": lse} if dx is None else {"loss": loss, "lse": lse, "dx": dx}


def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    weight = 2 * N * K
    if case["block"]:
        blocks = N * K // case["block"]
        weight = N * K // 2 + (blocks + 4 * -(-blocks // 256) if case["dq"] else 4 * blocks)
    targets = 8 * M if case["op"] == "xent" else case["k"] * M * (8 + (2 if case["bf16_teacher"] else 4))
    grad = 4 * M + 2 * M * K if case["grad"] else 0
    return {"bytes": weight + 2 * M * K + targets + 8 * M + grad, "flops": (4 if case["grad"] else 2) * M * N * K}
