"""Plain 64-bit forms, on the CPU, of the operators that fill a paged cache, read it back and
attend prompts, straight from their definitions in include/vts.h."""
import math

import torch


def numbers(bits):
    """The format's magnitudes in order of their codes (the even code has the even mantissa)."""
    if bits == 4:
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    n = [m * 2.0 ** -9 for m in range(8)]
    n += [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return torch.tensor(n[:-1], dtype=torch.float64)  # the last code is NaN


def nearest(x, grid):
    """The code of the grid's number nearest to x >= 0, ties to the even code."""
    code = torch.zeros(x.shape, dtype=torch.int64)
    for i in range(len(grid) - 1):
        mid = (grid[i] + grid[i + 1]) / 2
        code = torch.where((x > mid) | ((x == mid) & (i % 2 == 1)), i + 1, code)
    return code


def quantise(x, bits):
    """(codes [.., D], scale bytes [.., D / 32]) of float64 rows, by trying every exponent."""
    grid = numbers(bits)
    blocks = x.unflatten(-1, (-1, 32))
    top = blocks.abs().amax(-1)
    finite = torch.isfinite(blocks).all(-1)
    # the next number past the largest, were there one: below their middle (and on it, if the
    # largest is even) a magnitude rounds to the largest
    past = 2 * grid[-1] - grid[-2]
    mid = (grid[-1] + past) / 2
    even = (len(grid) - 1) % 2 == 0
    e = torch.full(top.shape, -127, dtype=torch.int64)
    for cand in range(-127, 128):
        y = top / 2.0 ** cand
        fits = (y < mid) | ((y == mid) & even)
        e = torch.where(fits | (e != cand), e, cand + 1)  # goes up while it does not fit
    scale = torch.where(finite, e + 127, 255)
    y = torch.where(finite[..., None], blocks, 0.0) / torch.pow(2.0, e.double())[..., None]
    code = nearest(y.abs(), grid)
    sign = torch.signbit(y).long() << (3 if bits == 4 else 7)
    return (code | sign).flatten(-2), scale


def pack(codes, bits):
    codes = codes.to(torch.uint8)
    return codes if bits == 8 else codes[..., 0::2] | codes[..., 1::2] << 4


def unpack(data, bits):
    return data.long() if bits == 8 else torch.stack([data & 15, data >> 4], -1).flatten(-2).long()


def values(codes, scale, bits):
    """float64 values of codes [.., D] with scale bytes [.., D / 32]."""
    top = 8 if bits == 4 else 128
    grid = torch.cat([numbers(bits), torch.full((top - len(numbers(bits)),), math.nan, dtype=torch.float64)])
    x = grid[codes % top] * torch.where(codes >= top, -1.0, 1.0)
    x = x.unflatten(-1, (-1, 32)) * torch.pow(2.0, scale.double() - 127)[..., None]
    return torch.where((scale == 255)[..., None], math.nan, x).flatten(-2)


def ready(x, norm, eps, table, positions, interleaved):
    """(rows normalised and turned in float64, the sums of magnitudes that bound their errors)"""
    x = x.detach().cpu().double()
    mag = x.abs()
    if norm is not None:
        inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        x = x * inv * norm.detach().cpu().double()
        mag = x.abs()
    if table is None:
        return x, mag
    rot = table.shape[1]
    row = table.detach().cpu().double()[positions.cpu().long().clamp(0, table.shape[0] - 1)][:, None]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    out, m = x.clone(), mag.clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ci, si = c[..., i], s[..., i]
        out[..., a] = x[..., a] * ci - x[..., b] * si
        out[..., b] = x[..., b] * ci + x[..., a] * si
        m[..., a] = mag[..., a] * ci.abs() + mag[..., b] * si.abs()
        m[..., b] = mag[..., b] * ci.abs() + mag[..., a] * si.abs()
    outside = (positions.cpu() < 0) | (positions.cpu() >= table.shape[0])
    out[outside] = 0
    m[outside] = 0
    return out, m


def ready_bound(y, mag, dim, dtype):
    """How far a row computed in 32 bits may be from y: the sum of dim squares (2^-24 each; half of
    that in its root), its division and root, two products, a sum and the weights' product (2^-24
    each, 8 of them at most), each relative to the magnitudes added; then a rounding to dtype, in
    fp16 below its normal range by 2^-25 at most (bf16's subnormals: 2^-134)."""
    h = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133
    off = (dim / 2 + 8) * 2.0 ** -24 * mag
    return off + h * (y.abs() + off) + tiny


def prompt(q, k, v, cu_q, cu_k, causal=True, scale=None):
    """out, lse, and what bounds their errors, as decode_ref.attend."""
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    heads, dim, kv = q.shape[1], q.shape[2], k.shape[1]
    scale = 1 / math.sqrt(dim) if scale is None else scale
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    reach = torch.zeros(q.shape[:2], dtype=torch.float64)
    cu_q, cu_k = cu_q.tolist(), cu_k.tolist()
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(nq):
            seen = min(nk, i + nk - nq + 1) if causal else nk
            if seen <= 0:
                continue
            at = cu_q[b] + i
            keys = slice(cu_k[b], cu_k[b] + seen)
            kk = k[keys].repeat_interleave(heads // kv, 1)
            vv = v[keys].repeat_interleave(heads // kv, 1)
            s = torch.einsum("jhd,hd->hj", kk, q[at]) * scale
            reach[at] = torch.einsum("jhd,hd->hj", kk.abs(), q[at].abs()).amax(1) * abs(scale)
            lse[at] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            p = torch.where((lse[at] == -math.inf)[:, None], 0.0, p)
            for h in range(heads):
                if lse[at, h] == -math.inf:
                    continue
                out[at, h] = (p[h, :, None] * vv[:, h]).sum(0)
                mag[at, h] = (p[h, :, None] * vv[:, h].abs()).sum(0)
    return out, lse, mag, reach
