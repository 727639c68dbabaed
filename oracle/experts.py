"""CPU oracle of the mixture-of-experts calls (router balance loss, merge weights from counts, the merged
gradient's norm, the clipped step).

TEST INFRASTRUCTURE ONLY, like the rest of this package: numpy in fp64, one learner and one tensor at a time,
written from the definitions in include/dlc.h.  Learners that processed more tokens weigh more in the merge
(Decoupled DiLoCo digest, "fault tolerance" item 3); the pages give no formula.
"""
import numpy as np

from . import core


def softmax(row):
    """Probabilities of one token; all zero where nothing is possible."""
    with np.errstate(invalid="ignore"):
        m = np.max(row)
        if m == -np.inf:
            return np.zeros(len(row))
        w = np.exp(row - m)
        return w / np.sum(w)


def balance(logits, choices, mask=None, coef=1.0, grad_scale=1.0):
    """One learner: (loss, counts, mean probabilities, gradient [T][E]) of logits [T][E], choices [T][top]."""
    t, e = logits.shape
    top = choices.shape[1]
    kept = np.ones(t, bool) if mask is None else np.asarray(mask, bool)
    n = int(kept.sum())
    counts = np.zeros(e, np.int64)
    probs = np.zeros((t, e))
    for i in np.flatnonzero(kept):
        for j in choices[i]:
            if 0 <= j < e:
                counts[j] += 1
        probs[i] = softmax(np.asarray(logits[i], np.float64))
    if n == 0:
        return 0.0, counts, np.zeros(e), np.zeros((t, e))
    means = probs.sum(0) / n
    loss = coef * e * float(np.sum(counts / (n * top) * means))
    c = counts - counts.mean()
    size = grad_scale * coef * e / (n * n * top)
    grad = size * probs * (c[None] - (probs @ c)[:, None])
    grad[~kept] = 0.0
    return loss, counts, means, grad


def tensor_weights(counts, weights, expert_of, token_weight=None):
    """[T][K] merge weights."""
    k = len(weights)
    out = np.zeros((len(expert_of), k))
    for t, e in enumerate(expert_of):
        raw = [0.0] * k
        if e >= 0:
            raw = [0.0 if not weights[i] > 0 else (1.0 if token_weight is None else token_weight[i]) * max(int(counts[i][e]), 0)
                   for i in range(k)]
        total = 0.0
        for r in raw:
            total += r
        if not total > 0.0:
            raw = list(weights)
            total = 0.0
            for r in raw:
                total += r
        out[t] = [r / total for r in raw]
    return out


def _merged(codes, codebook, weights, tensors, t, share, scale=1.0):
    _, lo, n = tensors[t]
    w_hat = core.normalize_weights(weights) if share is None else share[t]
    rows = [i for i in range(len(weights)) if weights[i] > 0 and w_hat[i] != 0]
    if not rows:
        return np.zeros(n)
    return core.merge([codes[i, lo:lo + n] for i in rows], [codebook[i, t] for i in rows],
                      [np.float64(scale) * np.float64(w_hat[i]) for i in rows])


def outer_grad_norm(codes, codebook, weights, tensors, share=None, max_norm=np.inf):
    """(norm, factor) of the merged gradient over all tensors."""
    total = 0.0
    for t in range(len(tensors)):
        g = _merged(codes, codebook, weights, tensors, t, share)
        total += float(np.sum(g * g))
    norm = float(np.sqrt(total))
    if not np.isfinite(norm):
        return norm, 0.0
    return norm, max_norm / norm if norm > max_norm else 1.0


def clipped_step(theta, momentum, codes, codebook, weights, tensors, share=None, scale=None, lr=0.7, beta=0.9):
    """In place on fp32 arrays; a factor that is not finite and positive changes nothing."""
    s = 1.0 if scale is None else float(scale)
    if not (np.isfinite(s) and s > 0.0):
        return
    for t, (off, _, n) in enumerate(tensors):
        g = _merged(codes, codebook, weights, tensors, t, share, s)
        theta[off:off + n], momentum[off:off + n] = core.nesterov(theta[off:off + n], momentum[off:off + n], g, lr, beta)
