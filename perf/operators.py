"""Performance cases of the layer's scoring and softmax operators.

Three calls are covered, each in a plain form of elementary torch operations and
as a user calls it (``own``):

* ``logprob``  -- log probabilities of given labels, entropy and top alternatives
  of logits [B, N] (``haste_logprob``);
* ``grad``     -- its gradient with respect to the logits (``haste_logprob_backward``);
* ``i8``       -- the dense head's product in 8-bit integers with a scale for each
  sample and each label (``haste_head_forward_i8``); the weights are quantised once.
"""
import math

import torch

own = False

DEV = "cuda"
_LARGEST_LOGITS = 256 * 670_208         # B * N of the largest listed softmax case
_LARGEST_MACS = 512 * 131_072 * 1024    # B * H * d of the largest listed product


def listed():
    lp = lambda name, B, N, dtype, per_row, k, masked=False: dict(  # noqa: E731
        name=name, op="logprob", B=B, N=N, dtype=dtype, per_row=per_row, ragged=per_row > 1, k=k, masked=masked)
    gr = lambda name, B, N, dtype, per_row, entropy, masked=False: dict(  # noqa: E731
        name=name, op="grad", B=B, N=N, dtype=dtype, per_row=per_row, ragged=per_row > 1, entropy=entropy,
        masked=masked)
    i8 = lambda name, B, H, d, dtype, out: dict(name=name, op="i8", B=B, H=H, d=d, dtype=dtype, out=out)  # noqa: E731
    return [
        # one sample scored online against the 670K workload's head
        lp("logprob one sample", 1, 4096, "f32", 1, 8),
        # a batch against an odd number of labels, some of them filtered out
        lp("logprob odd masked", 64, 32_003, "bf16", 1, 20, masked=True),
        # a training batch of the 8.6M workload's head
        lp("logprob head 8.6m", 256, 16_384, "bf16", 8, 5),
        # a training batch over the whole tail of the 670K workload
        lp("logprob tail 670k", 256, 670_208, "bf16", 5, 5),
        # few samples over the sweep workloads' label count, many alternatives
        lp("logprob long rows", 3, 1_048_576, "f32", 2, 64),
        # softmax training of the 8.6M workload's head
        gr("grad head 8.6m", 256, 16_384, "bf16", 8, False),
        # a small odd batch with an entropy term, labels filtered out
        gr("grad odd entropy", 61, 10_007, "f32", 3, True, masked=True),
        # softmax training over the 670K workload's tail
        gr("grad tail 670k", 256, 670_208, "bf16", 5, False),
        # one sample scored online, 670K workload's head
        i8("i8 one sample", 1, 4096, 768, "bf16", "f32"),
        # a scoring batch of the 8.6M workload's head
        i8("i8 head 8.6m", 256, 16_384, 768, "bf16", "f32"),
        # a ragged batch, odd label and feature counts, fp32 features
        i8("i8 odd", 37, 10_007, 1000, "f32", "bf16"),
        # the largest batch over a large label set
        i8("i8 large", 512, 131_072, 1024, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprob", "logprob", "grad", "i8", "i8"])
    if op == "i8":
        while True:
            B, H, d = _log(rng, 1, 512), _log(rng, 16, 131_072), _log(rng, 16, 4096)
            if B * H * d <= _LARGEST_MACS and H * d <= 131_072 * 1024:
                break
        return dict(op=op, B=B, H=H, d=d, dtype=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
    while True:
        B, N = _log(rng, 1, 512), _log(rng, 100, 1_048_576)
        dtype = rng.choice(["bf16", "f32"])
        if B * N * (2 if dtype == "f32" else 1) <= _LARGEST_LOGITS:
            break
    per_row = _log(rng, 1, 16)
    c = dict(op=op, B=B, N=N, dtype=dtype, per_row=per_row, ragged=per_row > 1, masked=rng.random() < 0.3)
    if op == "logprob":
        c["k"] = _log(rng, 1, 64)
    else:
        c["entropy"] = rng.random() < 0.5
    return c


def _torch_dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _counts(case):
    """Given labels of each sample: per_row of them, or 0 .. per_row in turn when ragged."""
    m = min(case["per_row"], case["N"])
    return [(7 * b + 3) % (m + 1) if case["ragged"] else m for b in range(case["B"])]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = {"case": case}
    if case["op"] == "i8":
        B, H, d = case["B"], case["H"], case["d"]
        s["X"] = normal(B, d).to(_torch_dtype(case["dtype"]))
        # the quantised weights that a scoring program keeps: rows padded with zeros to 16 bytes
        W = normal(H, d) / math.sqrt(d)
        s["w_scale"] = W.abs().amax(1) / 127
        s["Wq"] = torch.zeros(H, (d + 15) // 16 * 16, dtype=torch.int8, device=DEV)
        s["Wq"][:, :d] = torch.round(W.div_(s["w_scale"][:, None])).clamp_(-127, 127).to(torch.int8)
        s["logits"] = torch.empty(B, H, dtype=_torch_dtype(case["out"]), device=DEV)
        return s
    B, N = case["B"], case["N"]
    z = normal(B, N).mul_(2)
    counts = torch.tensor(_counts(case), dtype=torch.int64)
    nnz = int(counts.sum())
    row_ptr = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    row = torch.repeat_interleave(torch.arange(B), counts).to(DEV)
    # a sample's labels: one from each of its equal stretches of the label range, so ascending and distinct
    i = torch.arange(nnz, device=DEV) - row_ptr.to(DEV)[row]
    m = counts.to(DEV)[row].clamp(min=1)
    lo, hi = i * N // m, (i + 1) * N // m
    ids = lo + (torch.rand(nnz, generator=g, device=DEV, dtype=torch.float64) * (hi - lo)).long()
    if case["masked"]:
        z.masked_fill_(torch.rand(B, N, generator=g, device=DEV) < 0.125, float("-inf"))
    z[row, ids] = normal(nnz) + 5    # the labels that a trained model expects
    s["logits"] = z.to(_torch_dtype(case["dtype"]))
    s["row_ptr"], s["ids"] = row_ptr.to(DEV, torch.int32), ids.to(torch.int32)
    if case["op"] == "logprob":
        out = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
        s["out"] = (out(nnz), out(B), out(B), out(B, case["k"]), out(B, case["k"], dtype=torch.int32))
        return s
    # what the forward pass left, and the loss's gradients: cross entropy averaged over the batch, an entropy bonus
    lse = [torch.logsumexp(r.double(), 1) for r in s["logits"].split(32)]
    s["lse"] = torch.cat(lse).float()
    s["d_logp"] = -(0.5 + torch.rand(nnz, generator=g, device=DEV)) / B
    s["entropy"] = s["d_entropy"] = None
    if case["entropy"]:
        H = []
        for r, l in zip(s["logits"].split(32), lse):
            lp = r.double() - l[:, None]
            H.append(-(lp.exp() * lp.clamp(min=-1e30)).sum(1))
        s["entropy"] = torch.cat(H).float()
        s["d_entropy"] = 0.01 * normal(B) / B
    s["d_logits"] = torch.empty_like(s["logits"])
    return s


def _rows_of(s):
    """The sample of each given label."""
    counts = (s["row_ptr"][1:] - s["row_ptr"][:-1]).long()
    return torch.repeat_interleave(torch.arange(len(counts), device=DEV), counts, output_size=len(s["ids"]))


def _plain_logprob(s):
    z = s["logits"].float() + 0.0                       # -0 ranks as 0
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    S = e.sum(1, keepdim=True)
    logp = (z - m) - torch.log(S)
    lse = (m + torch.log(S)).squeeze(1)
    entropy = -(e / S * torch.where(e > 0, logp, 0.0)).sum(1)
    given = logp[_rows_of(s), s["ids"].long()]
    # larger logit first, equal ones by the smaller id: one whole number that orders both
    bits = z.view(torch.int32)
    key = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long() * (1 << 32)
    key += (1 << 32) - 1 - torch.arange(z.shape[1], device=DEV)
    best = torch.topk(key, s["case"]["k"], dim=1).values
    top_id = (1 << 32) - 1 - (best & 0xFFFFFFFF)
    return given, lse, entropy, logp.gather(1, top_id), top_id.int()


def _plain_grad(s):
    z = s["logits"].float()
    logp = z - s["lse"][:, None]
    p = torch.exp(logp)
    row = _rows_of(s)
    G = torch.zeros(z.shape[0], device=DEV).index_add_(0, row, s["d_logp"])[:, None]
    if s["d_entropy"] is not None:
        G = G + s["d_entropy"][:, None] * (torch.where(p > 0, logp, 0.0) + s["entropy"][:, None])
    dz = -p * G
    dz.view(-1).index_add_(0, row * z.shape[1] + s["ids"].long(), s["d_logp"])
    return dz.to(s["logits"].dtype)


def _plain_i8(s):
    x = s["X"].float()
    # the scale rounds once, and next to a half the quotient is taken in 64 bits
    scale = (x.abs().amax(1, keepdim=True).double() / 127).float()
    q = torch.round(x.double() / scale.double()).clamp(-127, 127)
    w = s["Wq"][:, : x.shape[1]].float()
    return ((q.float() @ w.t()) * (scale * s["w_scale"])).to(s["logits"].dtype)


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"logprob": _plain_logprob, "grad": _plain_grad, "i8": _plain_i8}[op](state)
    from structured_sparse_output_b200 import haste as H

    s = state
    if op == "logprob":
        logp, lse, entropy, top_logp, top_id = s["out"]
        if "ws" not in s:                                # kept from step to step, as a training program does
            n = H.haste_logprob_workspace_size(*s["logits"].shape, H.dtype_code(s["logits"]), top_id.shape[1])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        H.haste_logprob(s["logits"], s["row_ptr"], s["ids"], logp, lse, entropy, top_logp, top_id, s["ws"])
        return s["out"]
    if op == "grad":
        H.haste_logprob_backward(s["logits"], s["lse"], s["entropy"], s["row_ptr"], s["ids"], s["d_logp"],
                                 s["d_entropy"], s["d_logits"])
        return s["d_logits"]
    if "ws" not in s:
        n = H.haste_head_i8_workspace_size(s["X"].shape[0], s["Wq"].shape[0], s["X"].shape[1])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    H.haste_head_forward_i8(s["X"], s["Wq"], s["w_scale"], s["logits"], s["ws"])
    return s["logits"]


def work(case):
    e = {"bf16": 2, "f32": 4}
    B = case["B"]
    if case["op"] == "i8":
        H, d = case["H"], case["d"]
        return {"bytes": B * d * e[case["dtype"]] + H * d + 4 * H + B * H * e[case["out"]], "flops": 2 * B * H * d}
    N, nnz = case["N"], sum(_counts(case))
    lists = 4 * (B + 1) + 4 * nnz
    if case["op"] == "logprob":
        return {"bytes": B * N * e[case["dtype"]] + lists + 4 * nnz + B * (8 + 8 * case["k"]), "flops": 6 * B * N}
    # lse, and with an entropy term the entropies and their gradients
    return {"bytes": 2 * B * N * e[case["dtype"]] + lists + 4 * nnz + B * (12 if case["entropy"] else 4),
            "flops": 6 * B * N}


def exact(case, seed):
    """The definitions in 64 bits, a few rows at a time."""
    s = prepare(case, seed)
    if case["op"] == "i8":
        x = s["X"].double()
        step = (x.abs().max(dim=1).values / 127).float().double()   # a scale is a 32-bit number
        q = (x / step[:, None]).round()
        w = s["Wq"].double()[:, : case["d"]]
        return torch.einsum("bd,hd->bh", q * step[:, None], w) * s["w_scale"].double()
    ptr = s["row_ptr"].tolist()
    per_row = []
    for b in range(case["B"]):
        z = s["logits"][b].double()
        ids = s["ids"][ptr[b]:ptr[b + 1]].long()
        lse = torch.logsumexp(z, 0)
        logp = z - lse
        p = torch.softmax(z, 0)
        H = -torch.special.xlogy(p, p).sum()
        if case["op"] == "logprob":
            top, top_id = torch.sort(s["logits"][b].float(), descending=True, stable=True)
            k = case["k"]
            per_row.append((logp[ids], lse, H, logp[top_id[:k]], top_id[:k].int()))
            continue
        g = s["d_logp"][ptr[b]:ptr[b + 1]].double()
        dz = -p * g.sum()
        dz[ids] += g
        if case["entropy"]:
            dz -= s["d_entropy"][b].double() * (torch.special.xlogy(p, p) + p * H)
        per_row.append(dz)
    if case["op"] == "grad":
        return torch.stack(per_row)
    logp, lse, H, top, top_id = zip(*per_row)
    return torch.cat(logp), torch.stack(lse), torch.stack(H), torch.stack(top), torch.stack(top_id)
