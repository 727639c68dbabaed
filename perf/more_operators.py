"""Measured cases of training mixtures of experts with an outer step: the balance loss of a router with its
per-expert counts and its gradient, the norm of the merged outer gradient with its clipping factor, and the outer
step that takes that factor and weighs an expert's tensors by the tokens that each learner sent to it.

Layout of the outer gradient, as everywhere in the library: learner i owns row i of the [K][stride] codes, tensor t
occupies elements [lo, lo + n) of theta, of the momentum and of every row, lo a multiple of 64, with a codebook of
256 entries per (learner, tensor).  Elements between tensors, masked tokens and rows of absent learners hold values
in every case.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 64  # alignment of every tensor
BUCKETS = 256
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
IDS = {"int32": torch.int32, "int64": torch.int64}
COEF = 0.01  # of the balance loss
LR, BETA = 0.7, 0.9
MOST_LOGITS = 32768 * 256 * 8
MOST_CODES = 2_500_000_000


# --- cases -------------------------------------------------------------------------------------------------------

def listed():
    balance = {"op": "balance", "grad": True, "masked": False, "absent": False, "pad": 0}
    small = {"set": "vectors", "count": 4, "low": 4096, "high": 4096}
    ragged = {"set": "ragged", "count": 150, "low": 1, "high": 200_000}
    return [
        # a few tokens of one learner: the latency of one call
        {"name": "balance 64 tokens", **balance, "learners": 1, "tokens": 64, "experts": 8, "top": 2, "type": "fp32",
         "ids": "int64"},
        # one layer's micro-batch of four learners
        {"name": "balance 4096x64 K4", **balance, "learners": 4, "tokens": 4096, "experts": 64, "top": 6,
         "type": "bf16", "ids": "int64"},
        # padded batches, a number of experts that fills no load, dropped choices, one learner away
        {"name": "balance ragged K3", **balance, "learners": 3, "tokens": 5003, "experts": 60, "top": 4,
         "type": "fp16", "ids": "int32", "masked": True, "absent": True, "pad": 4},
        # the loss alone, for a report of how the experts are used
        {"name": "balance loss 16384x128 K8", **balance, "grad": False, "learners": 8, "tokens": 16384,
         "experts": 128, "top": 8, "type": "bf16", "ids": "int64"},
        # many small experts and long sequences on eight learners
        {"name": "balance 32768x256 K8", **balance, "learners": 8, "tokens": 32768, "experts": 256, "top": 8,
         "type": "bf16", "ids": "int32"},
        # the merged gradient's norm: four vectors, one of 24 fragments of the 135M set, the whole 1B set
        {"name": "norm 4 vectors K2", "op": "norm", **small, "learners": 2, "experts": 0, "absent": False},
        {"name": "norm 135M fragment K4", "op": "norm", "set": "fragment", "learners": 4, "experts": 0,
         "absent": False},
        {"name": "norm 1B K8", "op": "norm", "set": "1B", "learners": 8, "experts": 0, "absent": False},
        # the clipped step on the same, on odd sizes with an expert's weights and a learner away, and on a mixture of
        # experts whose every expert is three tensors
        {"name": "step 4 vectors K2", "op": "step", **small, "learners": 2, "experts": 0, "absent": False},
        {"name": "step 135M fragment K4", "op": "step", "set": "fragment", "learners": 4, "experts": 0,
         "absent": False},
        {"name": "step ragged K3", "op": "step", **ragged, "learners": 3, "experts": 9, "absent": True},
        {"name": "step experts K4", "op": "step", "set": "experts", "learners": 4, "experts": 128, "absent": False},
    ]


def draw(rng):
    """Routers of 2 to 512 experts and up to 32768 tokens a learner; tensor lists of 1 to 400 tensors, up to two and a
    half billion codes over one to fourteen learners."""
    def spread(low, high):
        return round(math.exp(rng.uniform(math.log(low), math.log(high))))

    op = rng.choice(("balance", "balance", "norm", "step", "step"))
    if op == "balance":
        experts, learners = spread(2, 512), rng.randint(1, 8)
        return {"op": op, "learners": learners, "experts": experts, "top": rng.randint(1, min(8, experts)),
                "tokens": spread(1, min(32768, MOST_LOGITS // (learners * experts))), "type": rng.choice(sorted(TYPES)),
                "ids": rng.choice(sorted(IDS)), "grad": rng.random() < 0.7, "masked": rng.random() < 0.5,
                "absent": learners > 1 and rng.random() < 0.3, "pad": rng.choice((0, 0, 1, 8))}
    learners, count = rng.randint(1, 14), spread(1, 400)
    high = spread(64, max(64, MOST_CODES // (count * learners)))
    return {"op": op, "set": rng.choice(("ragged", "vectors")), "count": count,
            "low": max(1, round(high * rng.random() ** 3)), "high": high, "learners": learners,
            "experts": rng.choice((0, 0, 1, 9, 64)), "absent": learners > 1 and rng.random() < 0.3}


def _sizes(case):
    """(elements, expert or -1) of each tensor."""
    kind = case["set"]
    if kind == "1B":
        d, kv, ffn = 2048, 512, 5632
        layer = [d, d * d, kv * d, kv * d, d * d, d, ffn * d, ffn * d, d * ffn]
        return [(n, -1) for n in [32000 * d] + layer * 16 + [d, 32000 * d]]
    if kind == "fragment":  # the median load of 24 fragments of the 135M set: whole tensors
        return [(n, -1) for n in [1536 * 576] * 5 + [192 * 576] * 2 + [576] * 2]
    if kind == "experts":  # eight layers of sixteen experts
        d, ffn = 1024, 1408
        out = [(32000 * d, -1)]
        for layer in range(8):
            out += [(n, -1) for n in (d, d * d, d * d // 4, d * d // 4, d * d, d, 16 * d)]
            out += [(ffn * d, layer * 16 + e) for e in range(16) for _ in range(3)]
        return out + [(d, -1)]
    r = random.Random(case["count"] * 1_000_003 + case["low"] * 101 + case["high"])
    if kind == "vectors":  # whole 64-element groups, as a model's own dimensions give
        sizes = [max(64, r.randint(case["low"], case["high"]) // 64 * 64) for _ in range(case["count"])]
    else:  # any size, spread over its logarithm
        lo, hi = math.log(case["low"]), math.log(case["high"])
        sizes = [min(case["high"], round(math.exp(r.uniform(lo, hi)))) for _ in range(case["count"])]
    return [(n, i % (case["experts"] + 1) - 1) for i, n in enumerate(sizes)]


def _tensors(case):
    """((offset, loffset, numel) of each tensor, expert of each, row length)."""
    sizes = _sizes(case)
    at, out = 0, []
    for n, _ in sizes:
        out.append((at, at, n))
        at += -(-n // BLOCK) * BLOCK
    return out, [e for _, e in sizes], at + BLOCK  # the row ends with a group of no tensor


def _present(case):
    return [int(not (case["absent"] and i == 1)) for i in range(case["learners"])]


def work(case):
    k = sum(_present(case))
    if case["op"] == "balance":
        n, size = k * case["tokens"] * case["experts"], 4 if case["type"] == "fp32" else 2
        ids = k * case["tokens"] * case["top"] * (4 if case["ids"] == "int32" else 8)
        rows = k * case["tokens"] if case["masked"] else 0
        return {"bytes": n * size * (2 if case["grad"] else 1) + ids + rows, "flops": n * (12 if case["grad"] else 6)}
    sizes = _sizes(case)
    n = sum(n for n, _ in sizes)
    books = len(sizes) * k * (BUCKETS * 4 + 8)
    if case["op"] == "norm":
        return {"bytes": n * k + books, "flops": n * (k + 2)}
    return {"bytes": n * (k + 16) + books, "flops": n * (k + 6)}


# --- inputs ------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    s = {"op": case["op"], "k": case["learners"], "present": _present(case), "experts": case["experts"]}
    s["on"] = torch.tensor(s["present"], dtype=torch.bool, device=DEV)
    (_prepare_balance if case["op"] == "balance" else _prepare_outer)(case, s, gen)
    return s


def _prepare_balance(case, s, gen):
    k, t, e, top = case["learners"], case["tokens"], case["experts"], case["top"]
    width = e + case["pad"]
    # a learned router: some experts are liked more, and every token has its favourites
    logits = torch.empty((k, t, width), device=DEV).normal_(generator=gen)
    logits += 0.5 * torch.empty((k, 1, width), device=DEV).normal_(generator=gen)
    s["logits"] = logits.to(TYPES[case["type"]])[:, :, :e]
    s["choices"] = torch.topk(s["logits"], top, dim=-1, sorted=False)[1]
    s["mask"] = None
    if case["masked"]:
        s["choices"][:, ::11, top - 1] = -1  # dropped: the expert was full
        length = torch.randint(t // 2, t + 1, (k, 1), device=DEV, generator=gen)  # sequences padded at their end
        s["mask"] = torch.arange(t, device=DEV) < length
        s["choices"] = torch.where(s["mask"][..., None], s["choices"], torch.full_like(s["choices"], e + 7))
        logits = s["logits"].masked_fill(~s["mask"][..., None], float("nan"))  # what padding holds is anybody's guess
        s["logits"] = torch.nn.functional.pad(logits, (0, case["pad"]))[:, :, :e]
    s["choices"] = s["choices"].to(IDS[case["ids"]])
    s["grad"] = torch.full((k, t, width), 2.0 ** -14, dtype=s["logits"].dtype, device=DEV) if case["grad"] else None
    # the loss scale, as half precision needs one
    s["upstream"] = torch.full((k,), 2.0 ** 16 if case["type"] == "fp16" else 1.0, dtype=torch.float64, device=DEV)
    s["loss"] = torch.full((k,), -COEF, device=DEV)
    s["means"] = torch.full((k, e), -1.0 / e, device=DEV)
    s["counts"] = torch.full((k, e), -1, dtype=torch.int64, device=DEV)
    s["totals"] = torch.randint(0, 1_000_000, (k, e), device=DEV, generator=gen)  # of the steps so far
    if own:
        import diloco_outer_step_amd as dlc
        s["workspace"] = dlc.alloc_expert_balance_workspace(k, t, e, DEV)


def _prepare_outer(case, s, gen):
    k, (tensors, expert_of, stride) = case["learners"], _tensors(case)
    nt = len(tensors)
    s["tensors"], s["expert_of"], s["stride"] = tensors, expert_of, stride
    blocks = torch.tensor([-(-n // BLOCK) for _, _, n in tensors])
    owner = torch.repeat_interleave(torch.arange(nt), blocks)
    s["owner"] = torch.cat([owner, owner[-1:]]).to(DEV)  # the tensor of each block
    count = torch.full((stride // BLOCK,), BLOCK, dtype=torch.int64)  # elements of each block that belong to a tensor
    count[blocks.cumsum(0) - 1] = torch.tensor([n for _, _, n in tensors]) - (blocks - 1) * BLOCK
    count[-1] = 0
    s["count"], s["whole"] = count.to(DEV), bool((count[:-1] == BLOCK).all())
    # 256 buckets over twelve standard deviations; an entry is its bucket's mean
    sigma = torch.exp(torch.empty((k, nt, 1), device=DEV).uniform_(math.log(1e-4), math.log(1e-2), generator=gen))
    place = torch.arange(BUCKETS, device=DEV) + 0.25 + 0.5 * torch.rand((k, nt, BUCKETS), device=DEV, generator=gen)
    s["codebook"] = sigma * (place * (12 / BUCKETS) - 6 + 0.1)
    s["codes"] = torch.empty((k, stride), dtype=torch.uint8, device=DEV)
    for row in s["codes"]:
        row.copy_(torch.empty(stride, device=DEV).normal_(128, BUCKETS / 12, generator=gen).clamp_(0, 255))
    s["weights"] = [(1.0 + 0.25 * i) * p for i, p in enumerate(s["present"])]  # tokens that each learner processed
    s["tokens"] = torch.tensor(s["weights"], dtype=torch.float64, device=DEV)
    s["expert_at"] = torch.tensor(expert_of, device=DEV)
    s["counts"] = None
    if case["experts"]:  # uneven, as routers are; the last expert got no token
        s["counts"] = torch.randint(1, 1 << 20, (k, case["experts"]), device=DEV, generator=gen)
        s["counts"][:, -1] = 0
    s["share"] = None if s["counts"] is None else torch.full((nt, k), -1.0, dtype=torch.float64, device=DEV)
    s["norm"] = torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
    s["scale"] = torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
    s["max_norm"] = 1e-3 * math.sqrt(sum(n for _, _, n in tensors))  # some draws are clipped, some are not
    if case["op"] == "step":
        s["theta"] = torch.empty(stride, device=DEV).normal_(0, 0.02, generator=gen)
        s["momentum"] = torch.empty(stride, device=DEV).normal_(0, 1e-3, generator=gen)
        s["clip"] = 0.25 + 0.75 * torch.rand(1, dtype=torch.float64, device=DEV, generator=gen)
    if s["share"] is not None and case["op"] == "norm":
        s["share"] = _plain_weights(s)
    if own:  # the tensor list as the library reads it, and the norm's workspace
        import diloco_outer_step_amd as dlc
        s["plan"] = dlc.TensorList(tensors)
        s["expert_ids"] = dlc.group_ids(expert_of)
        if case["op"] == "norm":
            s["workspace"] = dlc.alloc_outer_grad_norm_workspace(s["plan"], DEV)


# --- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _call(s)
    return {"balance": _plain_balance, "norm": _plain_norm, "step": _plain_step}[s["op"]](s)


def _call(s):
    import diloco_outer_step_amd as dlc
    if s["op"] == "balance":
        dlc.dlc_expert_balance(s["logits"], s["choices"], s["loss"], s["counts"], s["workspace"], coef=COEF,
                               mask=s["mask"], mean_probs=s["means"], totals=s["totals"],
                               grad_logits=None if s["grad"] is None else s["grad"][:, :, :s["experts"]],
                               grad_scale=s["upstream"], present=s["present"])
        return _balance_outputs(s)
    if s["op"] == "norm":
        dlc.dlc_outer_grad_norm(s["codes"], s["codebook"], s["weights"], s["plan"], s["norm"], s["scale"],
                                s["workspace"], max_norm=s["max_norm"], tensor_weights=s["share"])
        return {"norm": s["norm"], "scale": s["scale"]}
    if s["share"] is not None:
        dlc.dlc_expert_weights(s["counts"], s["weights"], s["expert_ids"], s["share"])
    dlc.dlc_merge_clipped_step(s["theta"], s["momentum"], s["codes"], s["codebook"], s["weights"], s["plan"],
                               grad_scale=s["clip"], tensor_weights=s["share"], lr=LR, beta=BETA)
    return _step_outputs(s)


def _balance_outputs(s):
    return {"loss": s["loss"], "means": s["means"], "counts": s["counts"], "totals": s["totals"], "grad": s["grad"]}


def _step_outputs(s):
    return {"theta": s["theta"], "momentum": s["momentum"], "share": s["share"]}


def _plain_balance(s):
    k, t, e = s["logits"].shape
    on = s["on"][:, None]
    live = torch.ones((k, t), dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
    tokens = live.sum(1)[:, None].float()
    ids = s["choices"].long()
    ids = torch.where(live[..., None] & (ids >= 0) & (ids < e), ids, e).view(k, -1)
    counts = torch.zeros((k, e + 1), dtype=torch.int64, device=DEV).scatter_add_(1, ids, torch.ones_like(ids))[:, :e]
    x = torch.where(live[..., None], s["logits"].float(), 0.0)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True) * live[..., None]
    means = p.sum(1) / tokens.clamp(min=1)
    # sum_e p_e = 1: the loss and its gradient see the counts' distances from their mean, and the mean itself
    mean = counts.double().mean(1, keepdim=True)
    apart = (counts - mean).float()
    rate = COEF * e / (tokens * s["choices"].shape[2]).clamp(min=1)
    loss = rate[:, 0] * ((apart * means).sum(1) + mean[:, 0].float() * means.sum(1))
    if s["grad"] is not None:
        size = rate / tokens.clamp(min=1) * s["upstream"].float()[:, None]
        c = apart[:, None]
        grad = size[..., None] * p * (c - (c * p).sum(-1, keepdim=True))
        old = s["grad"][:, :, :e]
        old.copy_(torch.where(on[..., None], grad.to(old.dtype), old))
    s["loss"].copy_(torch.where(on[:, 0], loss, s["loss"]))
    s["means"].copy_(torch.where(on, means, s["means"]))
    s["counts"].copy_(torch.where(on, counts, s["counts"]))
    s["totals"] += torch.where(on, counts, 0)
    return _balance_outputs(s)


def _plain_weights(s):
    """[T][K]: an expert's tensors by the tokens that it got from each learner, all others by the learners' own."""
    w = s["tokens"]
    shared = (w / w.sum()).expand(len(s["tensors"]), -1)
    if s["counts"] is None:
        return shared
    of = s["expert_at"][:, None]
    raw = (s["counts"].double() * (w > 0)[:, None])[:, of[:, 0].clamp(min=0)].T
    total = raw.sum(1, keepdim=True)
    return torch.where((of >= 0) & (total > 0), raw / total.clamp(min=1), shared)


def _plain_merge(s, share, dtype):
    """The merged outer gradient, [stride].  Learner by learner: the whole set's indices are eight bytes an element."""
    table = (share.T[..., None] * s["codebook"].double()).to(dtype).reshape(s["k"], -1)
    base = s["owner"][:, None] * BUCKETS
    g = torch.zeros(s["stride"], dtype=dtype, device=DEV)
    for i in range(s["k"]):
        if s["present"][i]:
            g += table[i][(s["codes"][i].view(-1, BLOCK) + base).view(-1)]
    return g


def _inside(s):
    """Which elements belong to a tensor, [stride]."""
    return (torch.arange(BLOCK, device=DEV) < s["count"][:, None]).view(-1)


def _plain_norm(s):
    share = _plain_weights(s) if s["share"] is None else s["share"]
    g = _plain_merge(s, share, torch.float64)  # a long sum: in 64 bits
    s["norm"].copy_(torch.where(_inside(s), g, 0.0).square().sum().sqrt())
    clip = torch.clamp(s["max_norm"] / s["norm"], max=1.0)
    s["scale"].copy_(torch.where(torch.isfinite(s["norm"]), clip, 0.0))
    return {"norm": s["norm"], "scale": s["scale"]}


def _plain_step(s):
    share = _plain_weights(s)
    if s["share"] is not None:
        s["share"].copy_(share)
    g = _plain_merge(s, share * s["clip"], torch.float32)
    v = BETA * s["momentum"] + g
    theta = s["theta"] - LR * (g + BETA * v)
    inside = _inside(s)
    s["theta"].copy_(torch.where(inside, theta, s["theta"]))
    s["momentum"].copy_(torch.where(inside, v, s["momentum"]))
    return _step_outputs(s)


# --- the definition in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    """Learner by learner and tensor by tensor, from the formulas."""
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(s)
    share = torch.empty((len(s["tensors"]), s["k"]), dtype=torch.float64, device=DEV)
    if s["counts"] is not None:  # tokens of each expert from each present learner, on the host
        sent = (s["counts"] * s["on"][:, None]).T.tolist()
    for t, e in enumerate(s["expert_of"]):
        raw = [float(w) for w in s["weights"]]
        if e >= 0 and sum(sent[e]) > 0:
            raw = sent[e]
        share[t] = torch.tensor([w / sum(raw) for w in raw], dtype=torch.float64)
    total = 0.0
    clip = float(s["clip"]) if case["op"] == "step" else 1.0
    out = {"theta": s["theta"].double(), "momentum": s["momentum"].double(),
           "share": None if s["share"] is None else share} if case["op"] == "step" else None
    for t, (off, lo, n) in enumerate(s["tensors"]):
        g = torch.zeros(n, dtype=torch.float64, device=DEV)
        for i in range(s["k"]):
            if s["present"][i]:
                g += share[t, i] * torch.index_select(s["codebook"][i, t].double(), 0, s["codes"][i, lo:lo + n].int())
        if out is None:
            total = total + torch.linalg.vector_norm(g) ** 2
            continue
        at = slice(off, off + n)
        out["momentum"][at] = out["momentum"][at] * BETA + clip * g
        out["theta"][at] -= LR * clip * g + LR * BETA * out["momentum"][at]
    if out is not None:
        return out
    norm = float(total) ** 0.5
    return {"norm": torch.tensor([norm], dtype=torch.float64),
            "scale": torch.tensor([min(1.0, s["max_norm"] / norm)], dtype=torch.float64)}


def _exact_balance(s):
    out = {name: s[name].clone() for name in ("loss", "means", "counts", "totals")}
    out["loss"], out["means"] = out["loss"].double(), out["means"].double()
    out["grad"] = None if s["grad"] is None else s["grad"].double()
    e, top = s["experts"], s["choices"].shape[2]
    for i in range(s["k"]):
        if not s["present"][i]:
            continue
        rows = slice(None) if s["mask"] is None else torch.nonzero(s["mask"][i])[:, 0]
        p = torch.softmax(s["logits"][i][rows].double(), -1)
        n = p.shape[0]
        ids = s["choices"][i][rows].reshape(-1).long()
        counts = torch.bincount(ids[(ids >= 0) & (ids < e)], minlength=e)
        out["counts"][i] = counts
        out["totals"][i] += counts
        out["means"][i] = p.sum(0) / max(n, 1)
        f = counts.double()
        f, apart = f / max(n * top, 1), (f - f.mean()) / max(n * top, 1)  # sum p = 1: the gradient sees no mean
        out["loss"][i] = COEF * e * torch.dot(f, out["means"][i])
        if out["grad"] is not None:
            out["grad"][i, :, :e] = 0
            g = p * (apart - (p @ apart)[:, None]) * (COEF * e / max(n, 1) * float(s["upstream"][i]))
            out["grad"][i, rows, :e] = g
    return out
