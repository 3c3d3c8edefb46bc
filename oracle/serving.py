"""The verify step of speculative decoding, in float64 from the definitions: the paged MXFP8 key/value cache, attention
of drafted tokens over it, and the verification of the drafts.

TEST INFRASTRUCTURE ONLY (see the package docstring). Written from the formulas in the library's header; shares no code
with the HIP library.
"""
import numpy as np

from . import formats as F

BLOCK = 32


def head_values(x, weight=None, eps=1e-6, cos=None, sin=None, interleaved=False):
    """x [R, H, D] float64: the root-mean-square norm over D (weight [D], or None for none), then the rotation of the
    first 2 * cos.shape[1] values by cos, sin [R, rot/2] (None for none): pairs (i, i + rot/2) or (2i, 2i + 1)."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if cos is not None:
        h = cos.shape[1]
        a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
        c, s = cos[:, None], sin[:, None]
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a] = xa * c - xb * s
        x[..., b] = xb * c + xa * s
    return x


def cache_values(codes, scales):
    """Codes [..., D] and scale bytes [..., D/32] -> the values they stand for (NaN for byte 255 and NaN codes)."""
    f = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return F.decode_e4m3(codes) * np.repeat(f, BLOCK, axis=-1)


def gather(pages, page, n_pages, length):
    """Slots of a sequence's positions 0..length-1 from its page table; -1 where the page does not exist."""
    j = np.arange(length)
    pg = np.asarray(pages, np.int64)[j // page]
    return np.where((pg >= 0) & (pg < n_pages), pg * page + j % page, -1)


def visible(T, length, here, mask=None):
    """[T, length]: what each node sees. mask: T integers (bit i: sees node i), or None for a chain."""
    see = np.zeros((T, length), bool)
    for t in range(min(T, here)):
        for j in range(length):
            i = j - (length - here)
            see[t, j] = i < 0 or ((int(mask[t]) >> i) & 1 if mask is not None else i <= t)
    return see


def attention(q, K, V, see, scale):
    """q [T, hq, D], K and V [length, hkv, D], see [T, length] -> (out [T, hq, D], sum of w |V| / sum of w, the largest
    sum |q k| scale): positions that a node does not see take no part at all; a node that sees none gives zeros."""
    T, hq, D = q.shape
    g = hq // K.shape[1] if K.shape[1] else 1
    out, mag, big = np.zeros((T, hq, D)), np.zeros((T, hq, D)), 0.0
    for t in range(T):
        at = np.nonzero(see[t])[0]
        if not len(at):
            continue
        for h in range(hq):
            k, v = K[at, h // g], V[at, h // g]
            x = k @ q[t, h] * scale
            w = np.exp(x - x.max())
            w /= w.sum()
            out[t, h], mag[t, h] = w @ v, w @ np.abs(v)
            big = max(big, (np.abs(k) @ np.abs(q[t, h])).max() * abs(scale))
    return out, mag, big


def probabilities(logits, t):
    """softmax(logits / t) of one row; t = 0: all on the lowest index of the largest. NaN counts as -inf, which has
    probability 0 at an infinite t too; logits of +inf share the row."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    p, top = np.zeros_like(x), x.max()
    if top == -np.inf:
        return p
    if not t > 0:
        p[int(x.argmax())] = 1.0
        return p
    live = x == top if top == np.inf else x > -np.inf
    p[live] = 1.0 if top == np.inf else np.exp((x[live] - top) / t)
    return p / p.sum()


def pick(w, u):
    """The first index whose running sum passes u times the total; 0 for no weight at all."""
    c = np.cumsum(w)
    if not c[-1] > 0:
        return 0
    past = np.nonzero((c > u * c[-1]) & (w > 0))[0]
    return int(past[0]) if len(past) else int(np.nonzero(w > 0)[0][-1])


def verify_chain(logits, draft, tokens, t, u, u_sample):
    """One sequence: logits [T, V], draft [T-1, V], tokens [T-1] -> (out_tokens [T], n)."""
    T, V = logits.shape
    n = 0
    while n < T - 1:
        x = int(tokens[n])
        p, q = probabilities(logits[n], t), probabilities(draft[n], t)
        if not 0 <= x < V or not (p[x] > 0 if not t > 0 else u[n] * q[x] < p[x]):
            break
        n += 1
    p = probabilities(logits[n], t)
    w = p
    if n < T - 1 and t > 0 and p.any():
        rest = np.maximum(p - probabilities(draft[n], t), 0)
        w = rest if rest.sum() > 0 else p
    out = np.full(T, -1, np.int32)
    out[:n] = tokens[:n]
    out[n] = pick(w, u_sample)
    return out, n


def verify_tree(logits, tokens, parents, t, u):
    """One sequence: logits [T, V], tokens and parents [T] -> (out_tokens [T], path [T], n)."""
    T = len(tokens)
    out, path = np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    cur, n = 0, 0
    while True:
        path[n], out[n] = cur, pick(probabilities(logits[cur], t), u[cur])
        nxt = [i for i in range(cur + 1, T) if parents[i] == cur and tokens[i] == out[n]]
        if not nxt:
            return out, path, n
        cur, n = nxt[0], n + 1
