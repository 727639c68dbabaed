"""CPU oracle of the learners' inner step (gradient norm, AdamW, AdamW with 8-bit coded moments).

TEST INFRASTRUCTURE ONLY, like the rest of this package: numpy in fp64, one learner and
one tensor at a time, written from the definitions in include/dlc.h.  Each learner
takes AdamW steps between two outer steps (INTELLECT-1 reading notes, section 3.2
steps 2-3); the pages name the optimizer and give no formula, so the usual one with
decoupled weight decay and bias correction is taken.

Rows are [K][stride] numpy arrays (16-bit gradients already widened to float32);
tensors are (offset, loffset, numel) triples; every function updates in place.
"""
import numpy as np

CODE_BLOCK = 64
GROUP = (1e-3, 0.9, 0.999, 1e-8, 0.01)  # lr, beta1, beta2, eps, weight_decay


def grad_norm(grads, tensors, unscale=1.0, max_norm=np.inf):
    """One learner's (norm, gradient scale); grads is its row."""
    total = 0.0
    for _, lo, n in tensors:
        g = grads[lo:lo + n].astype(np.float64)
        total += float(np.sum(g * g))
    norm = unscale * float(np.sqrt(total))
    if not np.isfinite(norm):
        return norm, 0.0
    return norm, unscale * (max_norm / norm if norm > max_norm else 1.0)


def takes_step(scale):
    return bool(np.isfinite(scale) and scale > 0.0)


def moments(m, v, g, group):
    """New moments in fp64 (before any rounding)."""
    _, b1, b2, _, _ = group
    return b1 * m + (1.0 - b1) * g, b2 * v + (1.0 - b2) * g * g


def stepped(theta, m, v, t, group, lr_scale=1.0):
    """(new theta, the step subtracted) in fp64, from the new moments."""
    lr, b1, b2, eps, wd = group
    eta = lr * lr_scale
    step = eta / (1.0 - b1 ** t) * m / (np.sqrt(v) / np.sqrt(1.0 - b2 ** t) + eps)
    return (1.0 - eta * wd) * theta - step, step


def adamw(theta, grads, m, v, steps, tensors, groups=(GROUP,), group_of=None, grad_scale=None, lr_scale=None,
          present=None):
    """All present learners' step on fp32 rows, in place; the fp64 values are rounded once.
    Returns the absolute steps, [K][stride] fp64 (zeros where nothing was done)."""
    k = theta.shape[0]
    size = np.zeros(theta.shape)
    for i in range(k):
        c = 1.0 if grad_scale is None else float(grad_scale[i])
        if (present is not None and not present[i]) or not takes_step(c):
            continue
        t = int(steps[i]) + 1
        for j, (_, lo, n) in enumerate(tensors):
            q = groups[0 if group_of is None else group_of[j]]
            at = slice(lo, lo + n)
            g = grads[i, at].astype(np.float64) * c
            m64, v64 = moments(m[i, at].astype(np.float64), v[i, at].astype(np.float64), g, q)
            with np.errstate(over="ignore"):
                m[i, at], v[i, at] = m64, v64
            new, step = stepped(theta[i, at].astype(np.float64), m[i, at].astype(np.float64),
                                v[i, at].astype(np.float64), t, q, 1.0 if lr_scale is None else float(lr_scale[i]))
            theta[i, at] = new
            size[i, at] = np.abs(step)
        steps[i] = t
    return size


# --- coded moments ----------------------------------------------------------------

M32 = 0xFFFFFFFF


def mix(x, k1=0, k2=0):
    """The 32-bit mixing function of the random words (Python ints or uint64 arrays)."""
    x = (x + k1) & M32
    x = ((x ^ (x >> 16)) * 0x9E3779B9 + k2) & M32
    x = ((x ^ (x >> 15)) * 0x6A09E667) & M32
    return x ^ (x >> 16)


def random_words(seed, t, learner, lo, n):
    """The random words of row elements lo .. lo + n, uint64 holding 32 bits."""
    out = np.empty(n, np.uint64)
    for hi in range(lo >> 32, ((lo + n - 1) >> 32) + 1):
        a, b = max(lo, hi << 32), min(lo + n, (hi + 1) << 32)
        k1 = mix((mix((seed + t) & M32) + learner + 64 * hi) & M32)
        k2 = mix((k1 + (seed >> 32) + t) & M32)
        e = np.arange(a, b, dtype=np.uint64) & np.uint64(M32)
        out[a - lo:b - lo] = mix(e, k1, k2)
    return out


class Format:
    """An 8-bit float: mantissa bits, exponent of its smallest normal number, and the
    exponent its blocks' largest value is scaled to."""

    def __init__(self, mantissa, least, top):
        self.mantissa, self.least, self.top = mantissa, least, top
        codes = np.arange(128)
        e, f = codes >> mantissa, codes & ((1 << mantissa) - 1)
        unit = 2.0 ** (np.maximum(e, 1) - 1 + least - mantissa)
        self.value = np.where(e == 0, f, f + (1 << mantissa)) * unit  # of the codes 0 .. 126
        self.value[127] = np.nan
        if mantissa == 2:  # e5m2: exponent 31 is infinity and NaN
            self.value[124] = np.inf
            self.value[125:] = np.nan

    def decode(self, codes):
        x = self.value[codes & 127]
        return np.where(codes & 128, -x, x)


E4M3 = Format(3, -6, 7)
E5M2 = Format(2, -14, 14)


def scale_of(byte):
    return np.ldexp(1.0, byte.astype(np.int64) - 127)


def decode_blocks(fmt, codes, scales):
    """fp64 values of a tensor's codes, from its blocks' scale bytes."""
    return fmt.decode(codes) * np.repeat(scale_of(scales), CODE_BLOCK)[:len(codes)]


def encode_blocks(fmt, x, r16):
    """(codes, scale bytes) of fp32 values x, block by block from the first; r16: 16 random bits each."""
    n = len(x)
    pad = np.zeros(-(-n // CODE_BLOCK) * CODE_BLOCK, np.float32)
    pad[:n] = np.where(np.isfinite(x), np.abs(x), 0)
    largest = pad.reshape(-1, CODE_BLOCK).max(1)
    byte = np.maximum((largest.view(np.uint32) >> 23).astype(np.int64) - fmt.top, 0)
    y = np.where(np.isfinite(x), np.abs(x), 0).astype(np.float64) * np.repeat(np.ldexp(1.0, 127 - byte), CODE_BLOCK)[:n]
    e = np.maximum(np.frexp(y)[1] - 1, fmt.least)
    u = np.ldexp(1.0, e - fmt.mantissa)
    below = y < 2.0 ** fmt.least
    fine = u * 2.0 ** -(23 - fmt.mantissa)
    y = np.where(below, np.floor(y / fine) * fine, y)
    q = np.floor(y / u + (r16.astype(np.float64) + 0.5) / 65536).astype(np.int64)  # in units of u
    # a value's code: its exponent's first code plus how many steps it is above; the next binade follows on
    code = np.where(below, q, ((e - fmt.least + 1) << fmt.mantissa) + q - (1 << fmt.mantissa))
    code = np.where(np.isfinite(x), code, 127)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8), byte.astype(np.uint8)


def adamw_coded(theta, grads, mc, ms, vc, vs, steps, tensors, groups=(GROUP,), group_of=None, seed=0, grad_scale=None,
                lr_scale=None, present=None):
    """As adamw, with the moments in codes (mc e4m3, vc e5m2) and scale bytes, in place."""
    size = np.zeros(theta.shape)
    for i in range(theta.shape[0]):
        c = 1.0 if grad_scale is None else float(grad_scale[i])
        if (present is not None and not present[i]) or not takes_step(c):
            continue
        t = int(steps[i]) + 1
        for j, (_, lo, n) in enumerate(tensors):
            q = groups[0 if group_of is None else group_of[j]]
            at, blk = slice(lo, lo + n), slice(lo // CODE_BLOCK, -(-(lo + n) // CODE_BLOCK))
            g = grads[i, at].astype(np.float64) * c
            m64, v64 = moments(decode_blocks(E4M3, mc[i, at], ms[i, blk]), decode_blocks(E5M2, vc[i, at], vs[i, blk]),
                               g, q)
            with np.errstate(over="ignore"):
                m32, v32 = m64.astype(np.float32), v64.astype(np.float32)
            new, step = stepped(theta[i, at].astype(np.float64), m32.astype(np.float64), v32.astype(np.float64), t, q,
                                1.0 if lr_scale is None else float(lr_scale[i]))
            theta[i, at] = new
            size[i, at] = np.abs(step)
            r = random_words(seed, t, i, lo, n)
            mc[i, at], ms[i, blk] = encode_blocks(E4M3, m32, r & np.uint64(0xFFFF))
            code, vs[i, blk] = encode_blocks(E5M2, v32, r >> np.uint64(16))
            vc[i, at] = np.where((code == 0) & (v32 > 0), 1, code)
        steps[i] = t
    return size
