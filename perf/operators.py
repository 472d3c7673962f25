"""The vocabulary operators beside the sampler, the verify and the acceptance
statistics: the highest logits of a row, distillation from a teacher's highest
logits (loss and gradient), and a beam search's selection and reordering.

`run` computes them in elementary torch operations, or, where `own` is true,
calls the library.  Shapes follow the library's configurations (vocabulary
129280, draft blocks of 5 or 7 positions, 2048 training blocks) and generic
odd ones.  The vocabulary is summed in 32 bits; what 32 bits lose is held in
64: a beam candidate's score, which stands next to others, and the
distillation's few outcomes, whose probabilities of nearly 1 are subtracted.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
NEG = float("-inf")


# ---- cases ------------------------------------------------------------------


def listed():
    return [
        # one request's target row while decoding: the smallest call, latency counts
        dict(name="top_row", op="top", dtype="bf16", R=1, V=129280, K=8, T=1.0),
        # a small batch with float32 logits, a vocabulary that no vector width divides
        dict(name="top_odd", op="top", dtype="f32", R=33, V=50257, K=100, T=2.0),
        # a teacher pass over 2048 training blocks of 7 positions
        dict(name="top_train", op="top", dtype="bf16", R=14336, V=129280, K=64, T=1.0),
        # one small fine-tuning step's loss: the latency of the training call
        dict(name="distill_small", op="distill", dtype="f32", N=4, gamma=5, V=1024, K=16, T=1.0, rest=False, masked=False),
        # the training step's loss, the teacher's remaining mass as one more outcome
        dict(name="distill_train", op="distill", dtype="bf16", N=2048, gamma=7, V=129280, K=64, T=1.0, rest=True, masked=True),
        # gradient of a ragged batch: odd vocabulary, a softened teacher renormalised over its tokens
        dict(name="grad_odd", op="grad", dtype="bf16", N=61, gamma=5, V=32003, K=20, T=2.0, rest=False, masked=True),
        # the training step's gradient
        dict(name="grad_train", op="grad", dtype="bf16", N=2048, gamma=7, V=129280, K=64, T=1.0, rest=True, masked=True),
        # a single request's beam step
        dict(name="beam_one", op="beam", dtype="f32", B=1, W=4, V=32000, M=8, finished=False),
        # 64 requests of 4 beams, twice the picks so that ended hypotheses can be set aside
        dict(name="beam_batch", op="beam", dtype="bf16", B=64, W=4, V=129280, M=8, finished=False),
        # many beams late in the search, a quarter of them ended; an odd vocabulary
        dict(name="beam_wide", op="beam", dtype="bf16", B=24, W=16, V=50257, M=16, finished=True),
        # the beams' token history: a few KB, latency counts
        dict(name="reorder_tokens", op="reorder", dtype="i32", L=1, B=4, W=4, M=4, S=1, T=64, D=1, ragged=False),
        # keys and values of eight layers, each request at its own length
        dict(name="reorder_cache", op="reorder", dtype="bf16", L=16, B=16, W=4, M=4, S=8, T=1024, D=128, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["top", "distill", "grad", "beam", "reorder"])
    dtype = rng.choice(["bf16", "f32"])
    es = 2 if dtype == "bf16" else 4
    V = _log_int(rng, 1000, 200000)
    K = _log_int(rng, 1, 128)
    T = rng.choice([0.5, 1.0, 1.0, 2.0])
    most = 14336 * 129280 * 2 // (V * es)  # rows that cost what the largest listed case does
    if op == "top":
        return dict(op=op, dtype=dtype, R=_log_int(rng, 1, most), V=V, K=K, T=T)
    if op in ("distill", "grad"):
        gamma = rng.randint(1, 16)
        return dict(op=op, dtype=dtype, N=_log_int(rng, 1, max(1, min(2048, most // gamma))), gamma=gamma, V=V, K=K, T=T,
                    rest=rng.random() < 0.5, masked=rng.random() < 0.5)
    if op == "beam":
        W = rng.randint(1, 16)
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 128), W=W, V=V, M=rng.choice([W, 2 * W]), finished=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "f32", "i32"])
    W = rng.randint(2, 16)
    case = dict(op=op, dtype=dtype, L=_log_int(rng, 1, 16), B=_log_int(rng, 1, 16), W=W, M=W, S=rng.choice([1, 2, 5, 8]),
                T=_log_int(rng, 1, 1024), D=rng.choice([1, 3, 64, 80, 128]), ragged=rng.random() < 0.5)
    while work(case)["bytes"] > work(listed()[-1])["bytes"]:
        case["T"] = max(1, case["T"] // 2)
        case["L"] = max(1, case["L"] // 2)
    return case


# ---- inputs -----------------------------------------------------------------


def _dtype(case):
    return {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32}[case["dtype"]]


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _lse(z):
    """log of the sum of exponentials over the last axis: the exponentials and
    their sum in z's type, the logarithm in 64 bits; -inf for nothing."""
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == NEG, torch.zeros_like(m), m)
    return (m.double() + (z - m).exp().sum(-1, keepdim=True).double().log()).squeeze(-1)


def _distill_inputs(case, g):
    """Draft logits N(0, 3^2), a teacher that differs from them by N(0, 1) and its K highest logits."""
    N, G, V, K, T = (case[k] for k in ("N", "gamma", "V", "K", "T"))
    draft = _normal(g, (N, G, V), 3.0)
    teacher = _normal(g, (N, G, V), 1.0).add_(draft)
    values, ids = teacher.topk(K, dim=-1)
    rest = None
    if case["rest"]:
        rest = _lse(teacher.scatter_(-1, ids, NEG).div_(T)).float()
    mask = None
    if case["masked"]:  # one block in eight is padding
        mask = (torch.arange(N, device=DEV) % 8 != 7).to(torch.uint8)
    return dict(draft=draft.to(_dtype(case)), values=values.contiguous(), ids=ids.to(torch.int32), teacher_rest=rest, mask=mask)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op = case["op"]
    s = dict(case)

    def empty(dtype, *shape):
        return torch.empty(shape, dtype=dtype, device=DEV)

    if op == "top":
        R, V, K = case["R"], case["V"], case["K"]
        s["logits"] = _normal(g, (R, V), 3.0).to(_dtype(case))
        s["out"] = dict(top_values=empty(torch.float32, R, K), top_ids=empty(torch.int32, R, K), rest=empty(torch.float32, R),
                        lse=empty(torch.float32, R), flags=empty(torch.uint8, R))
    elif op == "distill":
        N, G = case["N"], case["gamma"]
        s |= _distill_inputs(case, g)
        s["out"] = dict(kl=empty(torch.float32, N, G), lse=empty(torch.float32, N, G), rest=empty(torch.float32, N, G),
                        flags=empty(torch.uint8, N, G), sums=empty(torch.float32, 4))
    elif op == "grad":
        s |= _distill_inputs(case, g)
        # what the loss call left: the draft's log mass outside the teacher's tokens
        z = s["draft"].float() / case["T"]
        s["draft_rest"] = _lse(z.scatter_(-1, s["ids"].long(), NEG)).float()
        s["scale"] = torch.rand((1,), generator=g, device=DEV) + 0.5  # the upstream gradient
        s["out"] = dict(grad_draft=torch.empty_like(s["draft"]))
    elif op == "beam":
        B, W, V, M = (case[k] for k in ("B", "W", "V", "M"))
        s["logits"] = _normal(g, (B, W, V), 3.0).to(_dtype(case))
        # cumulative log-probabilities of a search some steps old
        s["scores"] = _normal(g, (B, W), 0.7) - 20.0
        s["ended"] = None
        if case["finished"]:
            n = W // 4  # that many beams of each request, at places of their own
            place = torch.rand((B, W), generator=g, device=DEV).argsort(-1)
            s["ended"] = (place < n).to(torch.uint8)
        s["eos"] = 2
        s["out"] = dict(tokens=empty(torch.int32, B, M), parents=empty(torch.int32, B, M), scores=empty(torch.float32, B, M),
                        flags=empty(torch.uint8, B, W))
    else:
        L, B, W, M, S, T, D = (case[k] for k in ("L", "B", "W", "M", "S", "T", "D"))
        shape = (L, B, W, S, T, D)
        if case["dtype"] == "i32":
            s["state"] = torch.randint(0, 129280, shape, generator=g, device=DEV, dtype=torch.int32)
        else:
            s["state"] = _normal(g, shape, 1.0).to(_dtype(case))
        # the survivors: some beams have several children, others none
        n = _kept(W, M)
        keep = torch.rand((B, W), generator=g, device=DEV).argsort(-1)[:, :n]
        child = torch.randint(0, n, (B, M), generator=g, device=DEV)
        child[:, :n] = torch.arange(n, device=DEV)
        s["parents"] = keep.gather(1, child).to(torch.int32)
        s["lengths"] = None
        if case["ragged"]:
            order = torch.rand((B,), generator=g, device=DEV).argsort()
            s["lengths"] = torch.tensor(_lengths(B, T), dtype=torch.int32, device=DEV)[order]
        s["out"] = torch.zeros((L, B, M, S, T, D), dtype=_dtype(case), device=DEV)
    return s


def _kept(W, M):
    """Parents with a child after a selection."""
    return max(1, min(M, (5 * W + 4) // 8))


def _lengths(B, T):
    """The requests' lengths in a ragged batch, from half of the longest on."""
    return [max(1, T - (T // 2) * i // max(1, B)) for i in range(B)]


# ---- one pass ---------------------------------------------------------------


def run(s):
    return _RUN[s["op"]](s)


def _order_keys(x):
    """64-bit keys that order float32 values from the highest, equal ones by the lowest index."""
    bits = (x + 0.0).view(torch.int32).to(torch.int64)  # + 0.0: -0 and +0 are equal
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    return (bits << 32) | (0x7FFFFFFF - torch.arange(x.shape[-1], device=x.device, dtype=torch.int64))


def _highest(x, K):
    """The K highest values of each row and their indices; -inf and -1 for what is missing."""
    V = x.shape[-1]
    k = min(K, V)
    at = 0x7FFFFFFF - (_order_keys(x).topk(k, dim=-1).values & 0xFFFFFFFF)
    v = x.gather(-1, at)
    pad = x.shape[:-1] + (K - k,)
    at = torch.cat([torch.where(v == NEG, -1, at), torch.full(pad, -1, dtype=at.dtype, device=x.device)], -1)
    return torch.cat([v, torch.full(pad, NEG, device=x.device)], -1), at


def _without(z, at):
    """z with -inf at the indices `at` (-1: none)."""
    member = torch.zeros(z.shape[:-1] + (z.shape[-1] + 1,), dtype=torch.bool, device=z.device)
    member.scatter_(-1, torch.where(at < 0, z.shape[-1], at), True)
    return torch.where(member[..., :-1], NEG, z), member[..., :-1]


def _run_top(s):
    if own:
        import dspark_draft_sampling_amd as ds

        return ds.dspark_top_logits(s["logits"], s["K"], temperature=s["T"], out=s["out"])
    x = s["logits"].float()
    values, at = _highest(x, s["K"])
    z = x / s["T"]
    rest, _ = _without(z, at)
    flags = 2 * (x.isnan() | (x == math.inf)).any(-1) + 8 * (x == NEG).all(-1)
    return dict(top_values=values, top_ids=at.to(torch.int32), rest=_lse(rest).float(), lse=_lse(z).float(),
                flags=flags.to(torch.uint8))


def _outcomes(s, z, rest):
    """log-probabilities, in 64 bits, of the K + 1 outcomes under the teacher
    and under the draft: the teacher's tokens, then everything else."""
    zt = torch.where(s["ids"] < 0, NEG, s["values"].double() / s["T"])
    r = s["teacher_rest"]
    r = torch.full(zt.shape[:-1], NEG, device=zt.device) if r is None else r
    zt = torch.cat([zt, r.double()[..., None]], -1)
    zs = torch.where(s["ids"] < 0, NEG, z.gather(-1, s["ids"].long().clamp(min=0)).double())
    zs = torch.cat([zs, rest.double()[..., None]], -1)
    lse = _lse(zs)
    return zt - _lse(zt)[..., None], zs - lse[..., None], lse


def _weights(s, shape):
    """exp(-k / gamma) at position k = 1..gamma of every block that counts."""
    N, G = shape
    w = torch.exp(-torch.arange(1, G + 1, device=DEV, dtype=torch.float32) / G).expand(N, G)
    return w if s["mask"] is None else w * (s["mask"] != 0)[:, None]


def _run_distill(s):
    if own:
        import dspark_draft_sampling_amd as ds

        return ds.dspark_distill(s["draft"], s["values"], s["ids"], teacher_rest=s["teacher_rest"], block_mask=s["mask"],
                                 temperature=s["T"], out=s["out"])
    z = s["draft"].float() / s["T"]
    outside, _ = _without(z, s["ids"].long())
    rest = _lse(outside)
    lt, ls, lse = _outcomes(s, z, rest)
    t = lt.exp()
    kl = torch.where(t > 0, t * (lt - ls), 0.0).sum(-1)
    w = _weights(s, kl.shape)
    on = (w > 0).double()
    sums = torch.stack([(w * kl).sum(), on.sum(), (on * kl).sum(), on.sum()])
    return dict(kl=kl.float(), lse=lse.float(), rest=rest.float(), sums=sums.float(), flags=torch.zeros(kl.shape, dtype=torch.uint8, device=DEV))


def _run_grad(s):
    if own:
        import dspark_draft_sampling_amd as ds

        return ds.dspark_distill_backward(s["draft"], s["values"], s["ids"], s["draft_rest"], teacher_rest=s["teacher_rest"],
                                          block_mask=s["mask"], temperature=s["T"], grad_scale=s["scale"], out=s["out"])
    z = s["draft"].float() / s["T"]
    at = s["ids"].long()
    lt, ls, _ = _outcomes(s, z, s["draft_rest"])
    t, p = lt.exp(), ls.exp()
    _, member = _without(z, at)
    # at the teacher's tokens p - t, elsewhere the draft's share of (p - t) of everything else
    d = (z - s["draft_rest"][..., None]).exp() * (p - t)[..., -1:].float()
    d = torch.where(member, 0.0, d).scatter_add_(-1, at, (p - t)[..., :-1].float())
    w = s["scale"] * _weights(s, z.shape[:-1]) / s["T"]
    return dict(grad_draft=(w[..., None] * d).to(s["draft"].dtype))


def _run_beam(s):
    if own:
        import dspark_draft_sampling_amd as ds

        return ds.dspark_beam_select(s["logits"], s["scores"], s["M"], finished=s["ended"], eos_token=s["eos"], out=s["out"])
    x = s["logits"].float()
    B, W, V = x.shape
    M = s["M"]
    values, at = _highest(x, M)
    # 64 bits: the picks of two beams may stand closer than 32 bits tell apart
    x64 = x.double()
    m = x64.amax(-1, keepdim=True)
    lse = m + (x64 - m).exp().sum(-1, keepdim=True).log()
    score = s["scores"].double()[..., None] + (values.double() - lse)
    if s["ended"] is not None:  # an ended beam goes on with one candidate, as it is
        ended = (s["ended"] != 0)[..., None]
        first = torch.arange(M, device=DEV) == 0
        score = torch.where(ended, torch.where(first, s["scores"].double()[..., None], NEG), score)
        at = torch.where(ended, s["eos"], at)
    score, order = score.reshape(B, W * M).sort(dim=-1, descending=True, stable=True)
    score, order = score[:, :M], order[:, :M]
    token = at.reshape(B, W * M).gather(1, order)
    none = score == NEG
    return dict(tokens=torch.where(none, -1, token).to(torch.int32), parents=torch.where(none, -1, order // M).to(torch.int32),
                scores=score.float(), flags=torch.zeros((B, W), dtype=torch.uint8, device=DEV))


def _run_reorder(s):
    if own:
        import dspark_draft_sampling_amd as ds

        return ds.dspark_beam_reorder(s["state"], s["parents"], batch_dim=1, lengths=s["lengths"],
                                      length_dim=None if s["lengths"] is None else 4, out=s["out"])
    B = s["B"]
    got = s["state"][:, torch.arange(B, device=DEV)[:, None], s["parents"].long()]
    if s["lengths"] is None:
        return got
    inside = torch.arange(s["T"], device=DEV) < s["lengths"][:, None]
    return torch.where(inside[None, :, None, None, :, None], got, s["out"])


_RUN = dict(top=_run_top, distill=_run_distill, grad=_run_grad, beam=_run_beam, reorder=_run_reorder)


# ---- what a pass cannot do without -------------------------------------------


def work(case):
    op = case["op"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "top":
        R, V, K = case["R"], case["V"], case["K"]
        return dict(bytes=R * (V * es + 8 * K + 9), flops=4 * R * V)
    if op in ("distill", "grad"):
        N, R, V, K = case["N"], case["N"] * case["gamma"], case["V"], case["K"]
        live = (N - N // 8) * case["gamma"] if case["masked"] else R
        side = 8 * K + 4 * case["rest"]
        if op == "distill":  # every block's loss is an output, counted or not
            return dict(bytes=R * (V * es + side + 13) + 16 + N * case["masked"], flops=4 * R * V)
        return dict(bytes=live * (V * es + side + 8) + R * V * es + N * case["masked"], flops=4 * live * V)
    if op == "beam":
        B, W, V, M = (case[k] for k in ("B", "W", "V", "M"))
        live = W - W // 4 if case["finished"] else W
        return dict(bytes=B * (live * V * es + W * 6 + M * 12), flops=4 * B * live * V)
    L, B, W, M, S, T, D = (case[k] for k in ("L", "B", "W", "M", "S", "T", "D"))
    tokens = sum(_lengths(B, T)) if case["ragged"] else B * T
    return dict(bytes=L * tokens * S * D * es * (_kept(W, M) + M) + 4 * B * (M + 1), flops=0)


# ---- the same in 64 bits -------------------------------------------------------


def _rows_at_once(V):
    return max(1, (1 << 28) // V)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "reorder":
        st = s["state"]
        if not st.is_floating_point():
            return None
        out = s["out"].double()
        parents = s["parents"].tolist()
        lengths = [case["T"]] * case["B"] if s["lengths"] is None else s["lengths"].tolist()
        for b in range(case["B"]):
            for j, p in enumerate(parents[b]):
                out[:, b, j, :, :lengths[b]] = st[:, b, p, :, :lengths[b]].double()
        return out
    T = case.get("T", 1.0)
    if op == "top":
        parts = []
        for x in s["logits"].split(_rows_at_once(case["V"])):
            x = x.double()
            k = min(case["K"], x.shape[-1])
            v, at = torch.sort(x, dim=-1, descending=True, stable=True)
            v = torch.nn.functional.pad(v[:, :k], (0, case["K"] - k), value=NEG)
            z = x / T
            lse = torch.logsumexp(z, -1)
            z.scatter_(-1, at[:, :k], NEG)
            parts.append((v, torch.logsumexp(z, -1), lse))
        v, rest, lse = (torch.cat(p) for p in zip(*parts))
        return dict(top_values=v, top_ids=None, rest=rest, lse=lse, flags=None)
    if op == "beam":
        scores = []
        for b in range(case["B"]):
            lp = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double()[:, None]
            if s["ended"] is not None:
                e = s["ended"][b] != 0
                lp[e] = NEG
                lp[e, s["eos"]] = s["scores"][b].double()[e]
            top = lp.flatten().topk(min(case["M"], lp.numel())).values
            scores.append(torch.nn.functional.pad(top, (0, case["M"] - top.numel()), value=NEG))
        return dict(tokens=None, parents=None, scores=torch.stack(scores), flags=None)
    # distillation: the outcomes are the teacher's tokens and, where it is given, everything else
    N, G, V, K = (case[k] for k in ("N", "gamma", "V", "K"))
    R = N * G
    x, ids = s["draft"].view(R, V), s["ids"].view(R, K).long()
    logt = s["values"].view(R, K).double() / T
    if s["teacher_rest"] is not None:
        logt = torch.cat([logt, s["teacher_rest"].view(R, 1).double()], -1)
    t = torch.softmax(logt, -1)
    if op == "distill":
        kl, lses, rests = [], [], []
        for i in range(0, R, _rows_at_once(V)):
            rows = slice(i, i + _rows_at_once(V))
            z = x[rows].double() / T
            lse = torch.logsumexp(z, -1)
            q = z.gather(-1, ids[rows])
            rest = torch.logsumexp(z.scatter_(-1, ids[rows], NEG), -1)
            if s["teacher_rest"] is not None:
                q = torch.cat([q, rest[:, None]], -1)
            kl.append((torch.special.xlogy(t[rows], t[rows]) - t[rows] * (q - lse[:, None])).sum(-1))
            lses.append(lse)
            rests.append(rest)
        kl = torch.cat(kl).view(N, G)
        on = torch.ones(N, dtype=torch.float64, device=DEV) if s["mask"] is None else s["mask"].double()
        decay = torch.tensor([math.exp(-k / G) for k in range(1, G + 1)], dtype=torch.float64, device=DEV)
        count = on.sum() * G
        sums = torch.stack([(kl * decay).sum(-1) @ on, count, kl.sum(-1) @ on, count])
        return dict(kl=kl, lse=torch.cat(lses).view(N, G), rest=torch.cat(rests).view(N, G), flags=None, sums=sums)
    grad = torch.empty((R, V), dtype=torch.float64, device=DEV)
    for i in range(0, R, _rows_at_once(V)):
        rows = slice(i, i + _rows_at_once(V))
        z = x[rows].double() / T
        g = torch.softmax(z, -1)
        if s["teacher_rest"] is not None:
            tail = torch.softmax(z.scatter(-1, ids[rows], NEG), -1)
            g -= t[rows, -1:] * tail
        g.scatter_add_(-1, ids[rows], -t[rows, :K])
        k = torch.arange(i, min(R, i + _rows_at_once(V)), device=DEV)
        w = torch.exp(-((k % G) + 1).double() / G) * s["scale"].double() / T
        if s["mask"] is not None:
            w = w * s["mask"][k // G].double()
        grad[rows] = g * w[:, None]
    return dict(grad_draft=grad.view(N, G, V))
