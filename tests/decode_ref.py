"""Plain 64-bit forms of the decode-step operators, on the CPU, straight from
their definitions in include/vts.h (loops over requests and rows; small sizes)."""
import math

import numpy as np
import torch


def places(b, t, lens, table, page, num_pages, draft, mask, slots, prefix_only_slots=False):
    """[(position or None, slot)] that row (b, t) sees."""
    cap = table.shape[1] * page
    n = min(max(int(lens[b]), 0), cap)
    first = n - draft

    def slot_of(pos):
        entry = int(table[b, pos // page])
        return entry * page + pos % page if 0 <= entry < num_pages else None

    seen = []
    if slots is None:
        for pos in range(max(first, 0)):
            seen.append((pos, slot_of(pos)))
    else:
        for s in slots[b, t].tolist():
            seen.append((None, s if 0 <= s < num_pages * page else None))
    if slots is None or mask is not None:
        for i in range(draft):
            see = i <= t if mask is None else (int(mask[b, t]) >> i) & 1
            if see and first + i >= 0:
                seen.append((first + i, slot_of(first + i)))
    return [(p, s) for p, s in seen if s is not None]


def flat(cache):
    """[slots, kv_heads, dim] in float64."""
    c = cache.detach().cpu().double()
    return c.reshape(c.shape[0] * c.shape[1], c.shape[2], c.shape[3])


def attend(q, k, v, table, lens, mask=None, slots=None, scale=None):
    """out, lse, and the sum of p |v| and the largest sum of |q k| that bound errors."""
    q = q.detach().cpu().double()
    batch, draft, heads, dim = q.shape
    page, num_pages, kv = k.shape[1], k.shape[0], k.shape[2]
    scale = 1 / math.sqrt(dim) if scale is None else scale
    table, lens = table.cpu(), lens.cpu()
    mask = None if mask is None else mask.cpu()
    slots = None if slots is None else slots.cpu().view(batch, draft, -1)
    fk, fv = flat(k), flat(v)
    out = torch.zeros_like(q)
    mag = torch.zeros_like(q)
    lse = torch.full((batch, draft, heads), -math.inf, dtype=torch.float64)
    reach = torch.zeros(batch, draft, heads, dtype=torch.float64)
    for b in range(batch):
        for t in range(draft):
            at = [s for _, s in places(b, t, lens, table, page, num_pages, draft, mask, slots)]
            if not at:
                continue
            for h in range(heads):
                kk, vv = fk[at, h // (heads // kv)], fv[at, h // (heads // kv)]
                s = (kk @ q[b, t, h]) * scale
                reach[b, t, h] = (kk.abs() @ q[b, t, h].abs()).max() * abs(scale)
                lse[b, t, h] = torch.logsumexp(s, 0)
                if lse[b, t, h] == -math.inf:
                    continue
                p = torch.softmax(s, 0)
                out[b, t, h] = (p[:, None] * vv).sum(0)
                mag[b, t, h] = (p[:, None] * vv.abs()).sum(0)
    return out, lse, mag, reach


def attend_bounds(out, mag, reach, count, dim, dtype):
    """How far tree_attention may be from `out` and its lse from the true one.

    Scores: dim products summed in 32 bits, each sum off by at most 2^-24 of the
    sum of the magnitudes so far, and the scaling's and the exponent's roundings
    (2^-22 covers them and the exponential's last place).  Probabilities: that
    error, and a rounding to dtype (eps / 2; in fp16 at most 2^-25 below its
    normal range, against a sum of at least 1).  Sums over `count` places: 2^-24
    each.  The output: a rounding to dtype."""
    h = torch.finfo(dtype).eps / 2
    score = (dim + 8) * 2.0 ** -24 * reach + 2.0 ** -22
    rel = 2 * score + h + (count + 64) * 2.0 ** -24
    tiny = 2.0 ** -25 * count * 8 if dtype == torch.float16 else 0.0
    return (rel[..., None] * mag + h * out.abs() + tiny * 1.01 + 1e-30,
            2 * score + (count + 64) * 2.0 ** -24)


def weigh(weights, q, k, table, lens, lse, mask=None, keep=None, scale=None):
    w = weights.detach().cpu().double().clone()
    q, lse = q.detach().cpu().double(), lse.detach().cpu().double()
    batch, draft, heads, dim = q.shape
    page, num_pages, kv = k.shape[1], k.shape[0], k.shape[2]
    scale = 1 / math.sqrt(dim) if scale is None else scale
    table, lens = table.cpu(), lens.cpu()
    mask = None if mask is None else mask.cpu()
    fk = flat(k)
    bound = torch.zeros_like(w)
    for b in range(batch):
        for t in range(draft):
            if keep is not None and not bool(keep[b, t]):
                continue
            seen = places(b, t, lens, table, page, num_pages, draft, mask, None)
            seen = [(p, s) for p, s in seen if p < w.shape[2]]
            if not seen:
                continue
            pos = [p for p, _ in seen]
            at = [s for _, s in seen]
            for h in range(heads):
                if lse[b, t, h] == -math.inf:
                    continue
                kk = fk[at, h // (heads // kv)]
                s = (kk @ q[b, t, h]) * scale
                p = torch.exp(s - lse[b, t, h])
                w[b, h // (heads // kv), pos] += p
                reach = (kk.abs() @ q[b, t, h].abs()) * abs(scale)
                # the score's error, the exponent's at magnitudes up to reach + |lse|
                err = (dim + 8) * 2.0 ** -24 * reach + 2.0 ** -22 * (1 + s.abs() + lse[b, t, h].abs())
                bound[b, h // (heads // kv), pos] += p * err * 1.5
    rows = draft * heads // kv
    return w, bound + (rows + 2) * 2.0 ** -24 * w.abs() + 1e-30


def order_key(x):
    """Order of weights: -0 equals +0, NaN beyond the infinities by its sign."""
    if math.isnan(x):
        return (2 if math.copysign(1, x) > 0 else -2, 0.0)
    return (0, x + 0.0)


def evict(weights, lens, cap, keep, sinks, recent):
    """kept positions [batch][kv] and lengths."""
    w = weights.detach().cpu().numpy()
    kept, counts = [], []
    for b in range(w.shape[0]):
        n = min(max(int(lens[b]), 0), cap, w.shape[2])
        counts.append(min(n, keep))
        rows = []
        for h in range(w.shape[1]):
            if n <= keep:
                rows.append(list(range(n)))
                continue
            safe = list(range(sinks)) + list(range(n - recent, n))
            rest = range(sinks, n - recent)
            best = sorted(rest, key=lambda j: tuple(-x for x in order_key(float(w[b, h, j]))) + (j,))
            rows.append(sorted(safe + best[: keep - len(safe)]))
        kept.append(rows)
    return kept, counts


def verify(target, tokens, uniforms, draft=None, parents=None):
    """path [batch][..], next tokens; residuals formed one after the other."""
    target = np.nan_to_num(target.detach().cpu().double().numpy(), nan=0.0)
    target = np.maximum(target, 0)
    if draft is not None:
        draft = np.maximum(np.nan_to_num(draft.detach().cpu().double().numpy(), nan=0.0), 0)
    tokens, u = tokens.cpu().tolist(), uniforms.cpu().double().tolist()
    batch, n = len(tokens), len(tokens[0])
    vocab = target.shape[2]
    paths, nexts = [], []
    for b in range(batch):
        up = parents[b].tolist() if parents is not None else list(range(-1, n - 1))
        cur, path, r = -1, [], target[b, 0].copy()
        for t in range(n):
            if not -1 <= up[t] < t or up[t] != cur:
                continue
            x = tokens[b][t]
            ok = 0 <= x < vocab
            if draft is None:
                q = np.zeros(vocab)
                if ok:
                    q[x] = 1.0
            else:
                q = draft[b, cur + 1]
            if ok and r[x] > 0 and u[b][t] * q[x] < r[x]:
                path.append(t)
                cur = t
                r = target[b, t + 1].copy()
                continue
            if not ok and draft is None:
                continue
            rest = np.maximum(r - q, 0)
            if draft is None:  # r sums to what is left of 1
                left = 1.0 - r[x]
                r = np.where(q > 0, 0.0, r) / left if left > 0 else np.zeros(vocab)
            else:
                total = rest.sum()
                r = rest / total if total > 0 else rest
        if r.sum() == 0:
            r = target[b, cur + 1]
        if r.sum() == 0:
            nexts.append(-1)
        else:
            c = np.cumsum(r)
            hit = np.nonzero((c > u[b][n] * c[-1]) & (r > 0))[0]
            nexts.append(int(hit[0]) if len(hit) else int(np.nonzero(r > 0)[0][-1]))
        paths.append(path)
    return paths, nexts
