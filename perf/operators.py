"""Measured cases of the learner's inner step: the gradient norm with its clipping factor, AdamW with 32-bit
moments and AdamW with 8-bit coded moments, each over all tensors of all present learners in one pass.

Layout, as everywhere in the library: learner i owns row i of [K][stride] buffers, tensor t occupies elements
[lo, lo + n) of every row, lo a multiple of 64.  Elements between tensors and rows of absent learners are left as
they were, and every case's buffers hold values there.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 64  # elements that share a scale byte; also the alignment of every tensor
MASK = 0xFFFFFFFF
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# {lr, beta1, beta2, eps, weight_decay}: matrices, vectors without decay, embeddings with their own rate
GROUPS = ((1e-3, 0.9, 0.95, 1e-8, 0.1), (1e-3, 0.9, 0.95, 1e-8, 0.0), (2e-3, 0.9, 0.999, 1e-6, 0.01))
SEED = 20_11  # of the stochastic rounding


# --- cases -------------------------------------------------------------------------------------------------------

def listed():
    small = {"set": "vectors", "count": 4, "low": 4096, "high": 4096}
    ragged = {"set": "ragged", "count": 150, "low": 1, "high": 200_000}
    step = {"op": "adamw"}
    coded = {"op": "coded"}
    norm = {"op": "norm"}
    return [
        # a few scale vectors on their own: the latency of one call
        {"name": "adamw 4 vectors", **step, **small, "learners": 1, "grads": "fp32", "working": "", "absent": False},
        # one of 24 fragments of the 135M set, four replicas trained in fp32 on one card
        {"name": "adamw 135M fragment K4", **step, "set": "fragment", "learners": 4, "grads": "fp32", "working": "",
         "absent": False},
        # odd tensor sizes from one element up, fp16 training with a working copy, one learner away
        {"name": "adamw ragged K3", **step, **ragged, "learners": 3, "grads": "fp16", "working": "fp16", "absent": True},
        # the whole 1B set of one learner, the usual mixed-precision step
        {"name": "adamw 1B", **step, "set": "1B", "learners": 1, "grads": "bf16", "working": "bf16", "absent": False},
        # the same four uses with the moments in 8 bits; the largest is eight replicas of the 135M set
        {"name": "coded 4 vectors", **coded, **small, "learners": 1, "grads": "fp32", "working": "", "absent": False},
        {"name": "coded 135M fragment K4", **coded, "set": "fragment", "learners": 4, "grads": "fp32", "working": "",
         "absent": False},
        {"name": "coded ragged K3", **coded, **ragged, "learners": 3, "grads": "fp16", "working": "fp16", "absent": True},
        {"name": "coded 135M K8", **coded, "set": "135M", "learners": 8, "grads": "bf16", "working": "bf16",
         "absent": False},
        # the norm of the same gradients
        {"name": "norm 4 vectors", **norm, **small, "learners": 1, "grads": "fp32", "working": "", "absent": False},
        {"name": "norm 135M fragment K4", **norm, "set": "fragment", "learners": 4, "grads": "fp32", "working": "",
         "absent": False},
        {"name": "norm ragged K3", **norm, **ragged, "learners": 3, "grads": "fp16", "working": "", "absent": True},
        {"name": "norm 1B", **norm, "set": "1B", "learners": 1, "grads": "bf16", "working": "", "absent": False},
    ]


def draw(rng):
    """Tensor lists of 1 to 400 tensors, up to a quarter of a billion elements over one to eight learners."""
    learners = rng.randint(1, 8)
    count = round(math.exp(rng.uniform(0, math.log(400))))
    most = max(64, 250_000_000 // (count * learners))
    high = round(math.exp(rng.uniform(math.log(64), math.log(most))))
    op = rng.choice(("adamw", "adamw", "coded", "coded", "norm"))
    return {"op": op, "set": rng.choice(("ragged", "vectors")), "count": count,
            "low": max(1, round(high * rng.random() ** 3)), "high": high, "learners": learners,
            "grads": rng.choice(sorted(TYPES)), "working": "" if op == "norm" else rng.choice(("", "bf16", "fp16")),
            "absent": learners > 1 and rng.random() < 0.3}


def _llama(d, layers, ffn, kv, vocab, tied):
    """(sizes, group of each) of a Llama-style set: embedding, per layer the norms, projections and MLP, final norm, head."""
    layer = [(d, 1), (d * d, 0), (kv * d, 0), (kv * d, 0), (d * d, 0), (d, 1), (ffn * d, 0), (ffn * d, 0), (d * ffn, 0)]
    return [(vocab * d, 2)] + layer * layers + [(d, 1)] + ([] if tied else [(vocab * d, 2)])


def _sizes(case):
    kind = case["set"]
    if kind == "1B":
        return _llama(2048, 16, 5632, 512, 32000, False)
    if kind == "135M":
        return _llama(576, 30, 1536, 192, 49152, True)
    if kind == "fragment":  # the median load of 24 fragments of the 135M set: whole tensors
        return [(1536 * 576, 0)] * 5 + [(192 * 576, 0)] * 2 + [(576, 1)] * 2
    r = random.Random(case["count"] * 1_000_003 + case["low"] * 101 + case["high"])
    if kind == "vectors":  # whole 64-element groups, as a model's own dimensions give
        sizes = [max(64, r.randint(case["low"], case["high"]) // 64 * 64) for _ in range(case["count"])]
    else:  # any size, spread over its logarithm
        lo, hi = math.log(case["low"]), math.log(case["high"])
        sizes = [min(case["high"], round(math.exp(r.uniform(lo, hi)))) for _ in range(case["count"])]
    return [(n, i % 3) for i, n in enumerate(sizes)]


def _tensors(case):
    """((offset, loffset, numel) of each tensor, group of each, row length)."""
    sizes = _sizes(case)
    at, out = 0, []
    for n, _ in sizes:
        out.append((at, at, n))
        at += -(-n // BLOCK) * BLOCK
    return out, [g for _, g in sizes], at + BLOCK  # the row ends with a group of no tensor


def _elements(case):
    return sum(n for n, _ in _sizes(case)) * (case["learners"] - (1 if case["absent"] else 0))


def work(case):
    n = _elements(case)
    grad = 4 if case["grads"] == "fp32" else 2
    if case["op"] == "norm":
        return {"bytes": n * grad, "flops": 2 * n}
    state = 8 if case["op"] == "adamw" else 2 + 2 / BLOCK
    return {"bytes": n * (8 + grad + 2 * state + (2 if case["working"] else 0)), "flops": 15 * n}


# --- inputs ------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    tensors, group_of, stride = _tensors(case)
    k = case["learners"]
    shape = (k, stride)
    blocks = [(n + BLOCK - 1) // BLOCK for _, _, n in tensors]
    count = torch.full((stride // BLOCK,), BLOCK, dtype=torch.int64)  # elements of each block that belong to a tensor
    ends = torch.tensor(blocks).cumsum(0)
    count[ends - 1] = torch.tensor([n - (b - 1) * BLOCK for (_, _, n), b in zip(tensors, blocks)])
    count[-1] = 0
    sigma = torch.exp(torch.empty(len(tensors), device=DEV).uniform_(math.log(1e-5), math.log(1e-3), generator=gen))
    owner = torch.repeat_interleave(torch.arange(len(tensors)), torch.tensor(blocks))
    owner = torch.cat([owner, owner[-1:]]).to(DEV)  # the tensor of each block
    sigma = sigma[owner][None, :, None]

    def normal():
        return torch.empty(shape, device=DEV).normal_(generator=gen).view(k, -1, BLOCK)

    s = {"op": case["op"], "tensors": tensors, "group_of": group_of, "stride": stride, "k": k,
         "present": [int(not (case["absent"] and i == 1)) for i in range(k)], "count": count.to(DEV),
         "block_group": torch.tensor(group_of, device=DEV)[owner], "whole": bool((count[:-1] == BLOCK).all())}
    # gradients of rows that no token reached are zero, as an embedding's are
    s["grads"] = (normal() * sigma).to(TYPES[case["grads"]])
    s["grads"][:, ::37] = 0
    s["grads"] = s["grads"].view(shape)
    if case["op"] == "norm":
        s["norm"] = torch.zeros(k, dtype=torch.float64, device=DEV)
        s["scale"] = torch.ones(k, dtype=torch.float64, device=DEV)
        s["unscale"] = 0.5  # two accumulated micro-batches
        s["max_norm"] = 1e-3 * math.sqrt(stride) * 0.1  # some learners are clipped, some are not
    else:
        s["theta"] = (normal() * 0.02).view(shape)
        m = normal() * sigma * 0.3
        v = (sigma * (0.5 + torch.empty(shape, device=DEV).uniform_(generator=gen).view(k, -1, BLOCK))) ** 2
        s["steps"] = torch.randint(0, 2000, (k,), device=DEV, generator=gen)
        s["clip"] = None if case["set"] == "vectors" else 0.25 + 0.75 * torch.rand(
            k, device=DEV, dtype=torch.float64, generator=gen)
        s["lr_scale"] = torch.full((k,), 0.8, dtype=torch.float64, device=DEV)  # the schedule's factor
        s["working"] = s["theta"].to(TYPES[case["working"]]) if case["working"] else None
        if case["op"] == "adamw":
            s["m"], s["v"] = m.view(shape), v.view(shape)
        else:  # states that an earlier step left
            for name, x, to, top in (("m", m, torch.float8_e4m3fn, 7), ("v", v, torch.float8_e5m2, 14)):
                e = torch.clamp((x.abs().amax(-1).view(torch.int32) >> 23) - top, min=0)
                scale = ((254 - e) << 23).to(torch.int32).view(torch.float32)
                s[name] = (x * scale[..., None]).to(to).view(shape)
                s[name + "_scale"] = e.to(torch.uint8)
    if own:  # the tensor list as the library reads it, and the norm's workspace
        import diloco_outer_step_amd as dlc
        s["plan"] = dlc.TensorList(tensors)
        s["groups"] = [dlc.AdamWGroup(*g) for g in GROUPS]
        s["group_of"] = dlc.group_ids(group_of)
        if case["op"] == "norm":
            s["workspace"] = dlc.alloc_grad_norm_workspace(k, tensors, DEV)
    return s


# --- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _call(s)
    return {"norm": _plain_norm, "adamw": _plain_adamw, "coded": _plain_coded}[s["op"]](s)


def _call(s):
    import diloco_outer_step_amd as dlc
    if s["op"] == "norm":
        dlc.dlc_grad_norm(s["grads"], s["plan"], s["norm"], s["scale"], s["workspace"], max_norm=s["max_norm"],
                          unscale=s["unscale"], present=s["present"])
        return {"norm": s["norm"], "scale": s["scale"]}
    if s["op"] == "adamw":
        dlc.dlc_adamw_step(s["theta"], s["grads"], s["m"], s["v"], s["steps"], s["plan"], s["groups"],
                           group_of=s["group_of"], grad_scale=s["clip"], lr_scale=s["lr_scale"], working=s["working"],
                           present=s["present"])
    else:
        dlc.dlc_adamw_coded_step(s["theta"], s["grads"], s["m"], s["m_scale"], s["v"], s["v_scale"], s["steps"],
                                 s["plan"], s["groups"], group_of=s["group_of"], seed=SEED, grad_scale=s["clip"],
                                 lr_scale=s["lr_scale"], working=s["working"], present=s["present"])
    return _outputs(s)


def _outputs(s):
    out = {"theta": s["theta"], "working": s["working"], "steps": s["steps"], "m": s["m"], "v": s["v"]}
    if s["op"] == "coded":  # codes and scales as the numbers that they stand for
        out["m_scale"] = s["m_scale"].view(torch.float8_e8m0fnu)
        out["v_scale"] = s["v_scale"].view(torch.float8_e8m0fnu)
    return out


def _valid(s):
    """Which elements the pass owns, [K, blocks, 64]; None where that is every element of the tensors' blocks."""
    if s["whole"] and all(s["present"]):
        return None
    inside = torch.arange(BLOCK, device=DEV) < s["count"][:, None]
    return inside & torch.tensor(s["present"], dtype=torch.bool, device=DEV)[:, None, None]


def _put(s, name, new, keep):
    old = s[name].view(s["k"], -1, BLOCK)
    if keep is None:
        old[:, :-1].copy_(new[:, :-1])
    else:
        old.copy_(torch.where(keep, new.to(old.dtype), old))


def _plain_norm(s):
    g = s["grads"].view(s["k"], -1, BLOCK)[:, :-1]
    keep = _valid(s)
    g = g if keep is None else torch.where(keep[:, :-1], g, torch.zeros((), dtype=g.dtype, device=DEV))
    n = s["unscale"] * torch.sqrt(g.double().square().sum((1, 2)))  # a long sum: in 64 bits
    scale = s["unscale"] * torch.clamp(s["max_norm"] / n, max=1.0)
    scale = torch.where(torch.isfinite(n), scale, torch.zeros_like(scale))
    on = torch.tensor(s["present"], dtype=torch.bool, device=DEV)
    s["norm"].copy_(torch.where(on, n, s["norm"]))
    s["scale"].copy_(torch.where(on, scale, s["scale"]))
    return {"norm": s["norm"], "scale": s["scale"]}


def _moments(s, m, v):
    """The new moments, each computed in 64 bits and rounded once, and the step that they give (the subtrahend)."""
    k = s["k"]
    t = (s["steps"] + 1).double()[:, None]
    lr, b1, b2, eps, wd = torch.tensor(GROUPS, dtype=torch.float64, device=DEV).T
    rate = lr * s["lr_scale"][:, None]
    size = (rate / (1 - b1 ** t))[:, s["block_group"], None].float()
    root = torch.rsqrt(1 - b2 ** t)[:, s["block_group"], None].float()
    b1, b2 = b1[s["block_group"], None], b2[s["block_group"], None]
    g = s["grads"].view(k, -1, BLOCK).double()
    g = g if s["clip"] is None else g * s["clip"][:, None, None]
    m = (b1 * m + (1 - b1) * g).float()
    v = (b2 * v + (1 - b2) * g * g).float()
    step = size * m / (torch.sqrt(v) * root + eps[s["block_group"], None].float())
    decay = (1 - rate * wd)[:, s["block_group"], None].float()
    return m, v, s["theta"].view(k, -1, BLOCK) * decay - step


def _finish(s, theta, keep):
    _put(s, "theta", theta, keep)
    if s["working"] is not None:
        _put(s, "working", theta, keep)
    s["steps"] += torch.tensor(s["present"], device=DEV)


def _plain_adamw(s):
    keep = _valid(s)
    shape = (s["k"], -1, BLOCK)
    m, v, theta = _moments(s, s["m"].view(shape).double(), s["v"].view(shape).double())
    _put(s, "m", m, keep)
    _put(s, "v", v, keep)
    _finish(s, theta, keep)
    return _outputs(s)


def _mix(x):
    """A 32-bit mixing function on int64 tensors: multiply by odd constants (the golden ratio's and the root of two's
    first 32 bits), fold the high half in."""
    x = (x ^ (x >> 16)) * 0x9E3779B9 & MASK
    x = (x ^ (x >> 15)) * 0x6A09E667 & MASK
    return x ^ (x >> 16)


def _random(s):
    """32 random bits of each element: a function of (seed, step, learner, element) alone."""
    t = (s["steps"] + 1)[:, None]
    e = torch.arange(s["stride"], device=DEV)
    i = torch.arange(s["k"], device=DEV)[:, None]
    k1 = _mix(_mix((SEED + t) & MASK) + i + BLOCK * (e >> 32) & MASK)
    k2 = _mix(k1 + (SEED >> 32) + t & MASK)
    x = (e & MASK) + k1 & MASK
    x = (x ^ (x >> 16)) * 0x9E3779B9 + k2 & MASK
    x = (x ^ (x >> 15)) * 0x6A09E667 & MASK
    return (x ^ (x >> 16)).view(s["k"], -1, BLOCK)


def _encode(x, bits, inside, mantissa, bias, top):
    """(codes, scale bytes) of blocks: the scale puts the largest value's exponent at `top`; a code keeps `mantissa` bits,
    and 16 random bits (and a half) are added below them before the cut."""
    ok = torch.isfinite(x)
    largest = torch.where(ok & inside, x.abs(), torch.zeros_like(x)).amax(-1, keepdim=True)
    byte = torch.clamp((largest.view(torch.int32) >> 23) - top, min=0)
    y = x.abs() * ((254 - byte) << 23).view(torch.float32)
    least = 2.0 ** (1 - bias)  # the smallest normal number; below it a code counts units of its last bit
    small = y < least
    cut = 23 - mantissa
    b = torch.where(small, y + least, y).view(torch.int32) + (bits << (cut - 16)).int() + (1 << (cut - 17))
    code = (b >> cut) - torch.where(small, (128 - bias) << mantissa, (127 - bias) << mantissa)
    return torch.where(ok, code, 0x7F), byte[..., 0].to(torch.uint8)


def _plain_coded(s):
    k = s["k"]
    shape = (k, -1, BLOCK)
    keep = _valid(s)
    inside = torch.arange(BLOCK, device=DEV) < s["count"][:, None]
    bits = _random(s)

    def value(name):
        return s[name].view(shape).double() * torch.exp2(s[name + "_scale"].double() - 127)[..., None]

    m, v, theta = _moments(s, value("m"), value("v"))
    on = (s["count"] > 0) & torch.tensor(s["present"], dtype=torch.bool, device=DEV)[:, None]
    code, byte = _encode(m, bits & 0xFFFF, inside, 3, 7, 7)
    code = (code + 128 * torch.signbit(m)).to(torch.uint8).view(torch.float8_e4m3fn)
    _put_bytes(s, "m", code, keep)
    s["m_scale"].copy_(torch.where(on, byte, s["m_scale"]))
    code, byte = _encode(v, bits >> 16, inside, 2, 15, 14)
    code = torch.where((code == 0) & (v > 0), 1, code).to(torch.uint8).view(torch.float8_e5m2)
    _put_bytes(s, "v", code, keep)
    s["v_scale"].copy_(torch.where(on, byte, s["v_scale"]))
    _finish(s, theta, keep)
    return _outputs(s)


def _put_bytes(s, name, new, keep):
    old = s[name].view(torch.uint8).view(s["k"], -1, BLOCK)
    new = new.view(torch.uint8)
    if keep is None:
        old[:, :-1].copy_(new[:, :-1])
    else:
        old.copy_(torch.where(keep, new, old))


# --- the definition in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    """Tensor by tensor and learner by learner, from the formulas."""
    s = prepare(case, seed)
    rows = [i for i in range(s["k"]) if s["present"][i]]
    if s["op"] == "norm":
        norm, scale = s["norm"].clone(), s["scale"].clone()
        for i in rows:
            total = sum(torch.linalg.vector_norm(s["grads"][i, lo:lo + n].double()) ** 2 for _, lo, n in s["tensors"])
            norm[i] = s["unscale"] * total ** 0.5
            scale[i] = s["unscale"] * min(1.0, s["max_norm"] / float(norm[i]))
        return {"norm": norm, "scale": scale}
    coded = s["op"] == "coded"
    out = {"theta": s["theta"].double(), "working": None, "steps": s["steps"].clone(), "m": s["m"].double(),
           "v": s["v"].double()}
    if s["working"] is not None:
        out["working"] = s["working"].double()
    if coded:
        out["m_scale"] = s["m_scale"].view(torch.float8_e8m0fnu).double()
        out["v_scale"] = s["v_scale"].view(torch.float8_e8m0fnu).double()
    for i in rows:
        t = int(s["steps"][i]) + 1
        out["steps"][i] = t
        clip = 1.0 if s["clip"] is None else float(s["clip"][i])
        for (_, lo, n), q in zip(s["tensors"], s["group_of"]):
            lr, b1, b2, eps, wd = GROUPS[q]
            lr = lr * float(s["lr_scale"][i])
            at, blk = slice(lo, lo + n), slice(lo // BLOCK, -(-(lo + n) // BLOCK))
            g = s["grads"][i, at].double() * clip
            m, v = out["m"][i, at], out["v"][i, at]
            if coded:
                m = m * torch.repeat_interleave(out["m_scale"][i, blk], BLOCK)[:n]
                v = v * torch.repeat_interleave(out["v_scale"][i, blk], BLOCK)[:n]
            m = m * b1 + g * (1 - b1)
            v = v * b2 + g ** 2 * (1 - b2)
            if coded:  # the value that is coded is the 32-bit moment
                m, v = m.float().double(), v.float().double()
                r = _random_of(t, i, lo, n)
                out["m"][i, at], out["m_scale"][i, blk] = _exact_code(m, r % 65536, 3, -6, 7)
                code, out["v_scale"][i, blk] = _exact_code(v, r // 65536, 2, -14, 14)
                out["v"][i, at] = torch.where(v > 0, code.clamp(min=2.0 ** -16), code)
            else:
                out["m"][i, at], out["v"][i, at] = m, v
            update = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)) ** 0.5 + eps)
            new = out["theta"][i, at] - lr * wd * out["theta"][i, at] - lr * update
            out["theta"][i, at] = new
            if out["working"] is not None:
                out["working"][i, at] = new
    return out


def _random_of(t, i, lo, n):
    """The same 32 random bits as whole numbers, for elements lo .. lo + n of learner i at step t."""
    def mix(x):
        x = (x ^ (x >> 16)) * 0x9E3779B9 % 2 ** 32
        x = (x ^ (x >> 15)) * 0x6A09E667 % 2 ** 32
        return x ^ (x >> 16)

    k1 = mix((mix((SEED + t) % 2 ** 32) + i) % 2 ** 32)  # every listed and drawn row is shorter than 2^32
    k2 = mix((k1 + SEED // 2 ** 32 + t) % 2 ** 32)
    x = (torch.arange(lo, lo + n, device=DEV) + k1) % 2 ** 32
    x = ((x ^ (x >> 16)) * 0x9E3779B9 + k2) & MASK
    x = (x ^ (x >> 15)) * 0x6A09E667 & MASK
    return x ^ (x >> 16)


def _exact_code(x, r16, mantissa, least, top):
    """(values of the codes, values of the scales): floor to the code's grid after adding (r16 + 1/2) / 2^16 of its step."""
    n = x.numel()
    pad = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    big = pad.abs().amax(-1)
    e = torch.frexp(big)[1] - 1  # floor(log2)
    scale = torch.exp2(torch.where(big < 2.0 ** -126, -127, e.clamp(min=-127)).double() - top).clamp(min=2.0 ** -127)
    y = x.abs() / torch.repeat_interleave(scale, BLOCK)[:n]
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=least).double() - mantissa)
    q = torch.floor(y / step + (r16.double() + 0.5) / 65536) * step
    return torch.copysign(q, x), scale
