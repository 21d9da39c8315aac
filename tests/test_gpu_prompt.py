"""prompt_attention against plain 64-bit forms (tests/cache_ref.py): lengths from zero and one on,
sequences that end inside a tile, grouped heads, keys in front of the queries, fewer keys than
queries, infinities and NaN that are not seen, rows of no sequence, strides, streams, graphs."""
import math

import pytest
import torch

import varlen_top_select_amd as vts
from tests import cache_ref, decode_ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


def say(*a):
    print(*a, flush=True)


def cu(lens, first=0):
    return torch.tensor([first] + (first + torch.tensor(lens).cumsum(0)).tolist(), dtype=torch.int32, device=DEV)


def check(q, k, v, cu_q, cu_k=None, causal=True, scale=None, **kw):
    out, lse = vts.prompt_attention(q, k, v, cu_q, cu_seqlens_k=cu_k, causal=causal, scale=scale,
                                    return_lse=True, **kw)
    torch.cuda.synchronize()
    cu_k = cu_q if cu_k is None else cu_k
    o64, l64, mag, reach = cache_ref.prompt(q, k, v, cu_q, cu_k, causal, scale)
    count = int((cu_k[1:] - cu_k[:-1]).max()) + 1
    ob, lb = decode_ref.attend_bounds(o64, mag, reach, count, q.shape[2], q.dtype)
    got, gl = out.cpu().double(), lse.cpu().double()
    empty = l64 == -math.inf
    assert torch.equal(gl == -math.inf, empty)
    assert (got[empty] == 0).all()
    worst = ((got - o64).abs() / ob).max().item()
    assert worst <= 1, f"output {worst:.3g} times its bound"
    worst = ((gl - l64).abs()[~empty] / lb[~empty]).max().item() if (~empty).any() else 0
    assert worst <= 1, f"lse {worst:.3g} times its bound"
    return out, lse


CASES = [
    # query lengths, keys in front, heads, kv, dim, causal, dtype
    ([1], [0], 1, 1, 64, True, BF16),
    ([1, 1, 1], [0, 5, 70], 8, 1, 128, True, BF16),
    ([0, 1, 2, 0, 3, 31, 32, 33, 0], [0] * 9, 4, 2, 128, True, F16),
    ([63, 64, 65, 127, 128, 129], [0] * 6, 1, 1, 64, True, BF16),
    ([200, 7, 77], [0, 0, 0], 14, 2, 64, True, F16),
    ([150], [300], 6, 2, 128, True, BF16),
    ([40, 3, 100], [0, 500, 61], 12, 4, 128, True, BF16),
    ([33, 90], [10, -40], 3, 1, 64, True, F16),       # fewer keys than queries
    ([5, 64], [-5, -64], 2, 2, 128, True, BF16),      # no keys
    ([70, 1, 200], [0, 0, 0], 4, 4, 128, False, BF16),
    ([16, 130], [100, -129], 10, 2, 64, False, F16),
    ([1] * 150 + [40], [0] * 151, 7, 1, 64, True, BF16),  # more sequences than lanes
    ([300], [0], 32, 1, 64, True, BF16),              # a tile of four tokens
    ([20], [0], 130, 1, 128, True, F16),              # a token's heads over two tiles
]


def tensors(gen, lens, front, heads, kv, dim, dtype):
    lk = [a + b for a, b in zip(lens, front)]
    q = (1.5 * torch.randn(sum(lens), heads, dim, generator=gen)).to(dtype).to(DEV)
    k, v = (torch.randn(sum(lk), kv, dim, generator=gen).to(dtype).to(DEV) for _ in "kv")
    return q, k, v, cu(lens), cu(lk)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_prompts(i):
    lens, front, heads, kv, dim, causal, dtype = CASES[i]
    say("prompt", CASES[i])
    gen = torch.Generator().manual_seed(700 + i)
    q, k, v, cu_q, cu_k = tensors(gen, lens, front, heads, kv, dim, dtype)
    check(q, k, v, cu_q, cu_k, causal)
    if not any(front):
        check(q, k, v, cu_q, None, causal)


@pytest.mark.parametrize("dim", [64, 128])
def test_strides(dim):
    """Views of one projection, heads apart from each other in any order, padded rows."""
    gen = torch.Generator().manual_seed(70)
    x = torch.randn(90, 12, dim + 8, generator=gen).bfloat16().to(DEV)[:, :, :dim]
    check(x[:, :8], x[:, 8:10], x[:, 10:], cu([50, 40]))
    y = torch.randn(8, 90, dim, generator=gen).bfloat16().to(DEV).transpose(0, 1)
    check(y, y[:, :4], y[:, 4:], cu([89, 1]))
    one = torch.randn(90, 1, dim, generator=gen).bfloat16().to(DEV)
    check(one.expand(90, 4, dim), one, one, cu([90]))  # a broadcast head


@pytest.mark.parametrize("scale", [0.5, -0.3, 0.0, 4.0])
def test_scales(scale):
    gen = torch.Generator().manual_seed(71)
    q, k, v, cu_q, cu_k = tensors(gen, [70, 20], [9, 0], 4, 2, 64, BF16)
    check(q, k, v, cu_q, cu_k, scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_climbing_scores(dtype):
    """The maximum is passed again and again, and light keys stand next to a heavy one."""
    gen = torch.Generator().manual_seed(72)
    q, k, v, cu_q, _ = tensors(gen, [400], [0], 2, 1, 128, dtype)
    up = torch.linspace(-3, 3, 400, device=DEV)[:, None, None]
    k = (k * 0.1 + up * q[:1, :1].sign()).to(dtype)
    q = (q * 0.1 + q[:1, :1].sign() * 1.0).to(dtype)
    check(q, k, v, cu_q)
    check(q, k.flip(0), v, cu_q)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_not_finite_where_it_is_not_seen(dtype, bad):
    """Keys and values behind a row, of other sequences and of none."""
    gen = torch.Generator().manual_seed(73)
    lens = [100, 37, 64]
    q, k, v, cu_q, _ = tensors(gen, lens, [0] * 3, 4, 2, 128, dtype)
    q, k, v = (torch.cat([x, x[:40]]) for x in (q, k, v))  # rows behind the last sequence
    want, want_lse = vts.prompt_attention(q, k, v, cu_q, return_lse=True)
    k2, v2 = k.clone(), v.clone()
    spots = [50, 99, 130]  # keys of sequences 0, 0, 1
    for s in spots:
        k2[s, 0, 5] = bad
        v2[s, 1, 7] = bad
    k2[201:], v2[201:] = bad, bad
    got, lse = vts.prompt_attention(q, k2, v2, cu_q, return_lse=True)
    torch.cuda.synchronize()
    i = torch.arange(241)
    seq = torch.bucketize(i, torch.tensor(lens).cumsum(0), right=True)
    sees = torch.zeros(241, dtype=torch.bool)
    for s in spots:
        sees |= (i >= s) & (seq == seq[s])
    # heads 0, 1 belong to KV head 0, whose K is bad; 2, 3 to KV head 1, whose V is
    keep = ~sees[:201]
    got, want = got.cpu()[:201], want.cpu()[:201]
    assert torch.equal(got[keep], want[keep])
    assert torch.equal(lse.cpu()[:201][keep], want_lse.cpu()[:201][keep])
    assert torch.equal(lse.cpu()[:201, 2:], want_lse.cpu()[:201, 2:])
    part = got[~keep][:, 2:]
    assert not part[:, :, 7].isfinite().any()
    if not math.isnan(bad):
        assert (part[:, :, 7] == bad).all()
    others = torch.arange(128) != 7
    assert torch.equal(part[:, :, others], want[~keep][:, 2:][:, :, others])


def test_rows_without_weight():
    """Every score of a row -inf: zeros and -inf, whatever V holds."""
    gen = torch.Generator().manual_seed(74)
    q, k, v, cu_q, _ = tensors(gen, [70], [0], 2, 2, 64, BF16)
    q[:, 0] = q[:, 0].abs()
    k[:20, 0] = -math.inf
    v[3, 0, 1] = math.nan
    out, lse = vts.prompt_attention(q, k, v, cu_q, return_lse=True)
    assert (out[:20, 0] == 0).all() and (lse[:20, 0] == -math.inf).all()
    assert lse[20:].isfinite().all() and out[:, 1].isfinite().all()


def test_rows_of_no_sequence():
    gen = torch.Generator().manual_seed(75)
    q, k, v, _, _ = tensors(gen, [100], [0], 4, 2, 64, BF16)
    at = cu([30, 0, 40], first=10)
    alone = check(q[10:80], k[10:80], v[10:80], cu([30, 0, 40]))
    out = torch.full((100, 4, 64), 3.0, dtype=BF16, device=DEV)
    got, lse = vts.prompt_attention(q, k, v, at, out=out, return_lse=True)
    assert got is out and torch.equal(got[10:80], alone[0]) and torch.equal(lse[10:80], alone[1])
    assert (got[:10] == 3).all() and (got[80:] == 3).all()
    got, lse = vts.prompt_attention(q, k, v, at, return_lse=True)
    assert torch.equal(got[10:80], alone[0])
    for x, y in ((got, 0.0), (lse, -math.inf)):
        assert (x[:10] == y).all() and (x[80:] == y).all()
    for none in (torch.zeros(1, dtype=torch.int32, device=DEV), cu([0, 0], first=50)):
        got, lse = vts.prompt_attention(q, k, v, none, return_lse=True)
        assert (got == 0).all() and (lse == -math.inf).all()
    assert vts.prompt_attention(q[:0], k, v, cu([0]))[0].shape == (0, 4, 64)
    got, lse = vts.prompt_attention(q, k[:0], v[:0], cu([100]), cu_seqlens_k=cu([0]), return_lse=True)
    assert (got == 0).all() and (lse == -math.inf).all()


def test_bad_cu_seqlens_stay_inside():
    """Entries past the rows, negative ones, and ones that fall: nothing outside the outputs changes."""
    gen = torch.Generator().manual_seed(76)
    q, k, v, _, _ = tensors(gen, [100], [0], 4, 2, 64, BF16)
    room = torch.full((300, 4, 64), 3.0, dtype=BF16, device=DEV)
    out = room[100:200]
    for bad in ([-5, 40, 500], [0, 80, 20, 100], [90, 10], [2 ** 31 - 1, -2 ** 31, 7]):
        c = torch.tensor(bad, dtype=torch.int32, device=DEV)
        vts.prompt_attention(q, k, v, c, out=out)
        torch.cuda.synchronize()
        assert (room[:100] == 3).all() and (room[200:] == 3).all()
    c = torch.tensor([-5, 40, 500], dtype=torch.int32, device=DEV)  # clamped: 0, 40, 100
    assert torch.equal(vts.prompt_attention(q, k, v, c)[0], vts.prompt_attention(q, k, v, cu([40, 60]))[0])


def test_streams_and_graphs():
    gen = torch.Generator().manual_seed(77)
    q, k, v, cu_q, cu_k = tensors(gen, [300, 1, 77], [0, 200, 3], 8, 2, 128, BF16)
    kw = dict(cu_seqlens_k=cu_k, return_lse=True)
    want, lse = vts.prompt_attention(q, k, v, cu_q, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = vts.prompt_attention(q, k, v, cu_q, stream=side, **kw)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, out_lse = vts.prompt_attention(q, k, v, cu_q, **kw)
    for turn in range(4):
        if turn:
            q.mul_(-1.2)
            cu_q[1] -= 10  # other lengths in the same memory
        want, lse = vts.prompt_attention(q, k, v, cu_q, **kw)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out_lse, lse), turn


def test_long_prompt_and_its_parts():
    """A sequence of several thousand: the rows of its last chunk are the same, run as a chunk."""
    gen = torch.Generator().manual_seed(78)
    n = 4500
    q, k, v, cu_q, _ = tensors(gen, [n], [0], 4, 2, 128, BF16)
    out, lse = vts.prompt_attention(q, k, v, cu_q, return_lse=True)
    part, part_lse = vts.prompt_attention(q[-100:], k, v, cu([100]), cu_seqlens_k=cu([n]), return_lse=True)
    for rows, o, l in ((slice(n - 100, n), part, part_lse), (slice(n - 100, n), out[-100:], lse[-100:])):
        q1 = torch.zeros(100, 4, 128)
        o64, l64, mag, reach = cache_ref.prompt(q[rows], k, v, cu([100]), cu([n]))
        ob, lb = decode_ref.attend_bounds(o64, mag, reach, n, 128, BF16)
        assert ((o.cpu().double() - o64).abs() <= ob).all() and ((l.cpu().double() - l64).abs() <= lb).all()


def test_k_and_v_past_4_gib():
    """Key rows beyond 2^32 bytes and 2^31 elements, and query rows."""
    gen = torch.Generator().manual_seed(79)
    n = (5 << 30) // (8 * 128 * 2)
    big = torch.empty(n, 8, 128, dtype=BF16, device=DEV)
    x = torch.randn(200, 8, 128, generator=gen).bfloat16().to(DEV)
    big[-200:] = x
    # (the workgroups to a tile go by the rows of k there are, so the bits need not be those of
    # a call on x alone)
    o64, _, mag, reach = cache_ref.prompt(x, x, x, cu([200]), cu([200]))
    ob, _ = decode_ref.attend_bounds(o64, mag, reach, 201, 128, BF16)
    got = vts.prompt_attention(x, big, big, cu([200]), cu_seqlens_k=cu([200], first=n - 200))[0]
    assert ((got.cpu().double() - o64).abs() <= ob).all()
    out = torch.empty_like(big)
    vts.prompt_attention(big, big, big, cu([200], first=n - 200), out=out)
    assert ((out[-200:].cpu().double() - o64).abs() <= ob).all()


@pytest.mark.parametrize("lens,keys,dim", [([5, 3, 9], [5000, 4200, 6000], 64), ([2, 40], [4096, 4500], 128),
                                           ([1, 0, 2, 1], [9000, 0, 4096, 4096], 64)])
def test_few_queries_behind_long_contexts(lens, keys, dim):
    """Sequences taken in the order of their lengths, with ties and empty ones."""
    gen = torch.Generator().manual_seed(80)
    q = (1.5 * torch.randn(sum(lens), 4, dim, generator=gen)).bfloat16().to(DEV)
    k, v = (torch.randn(sum(keys), 2, dim, generator=gen).bfloat16().to(DEV) for _ in "kv")
    check(q, k, v, cu(lens), cu(keys))


def test_rows_far_apart():
    """Keys 2^25 bytes and more from each other."""
    gen = torch.Generator().manual_seed(81)
    n, step = 70, (1 << 24) + 8
    room = torch.empty(n * step, dtype=BF16, device=DEV)
    k, v = (room[at:at + n * step - 4096].as_strided((n, 2, 64), (step, 64, 1)) for at in (0, 2048))
    x = torch.randn(n, 8, 64, generator=gen).bfloat16().to(DEV)
    k.copy_(x[:, 4:6])
    v.copy_(x[:, 6:])
    want, _ = vts.prompt_attention(x[:, :4], x[:, 4:6], x[:, 6:], cu([n]))
    got, _ = vts.prompt_attention(x[:, :4], k, v, cu([n]))
    assert torch.equal(got, want)


SHARED = [
    # query lengths, keys, heads, kv, dim, causal, dtype: few tiles whose keys several workgroups share
    ([1], [5000], 8, 1, 128, True, BF16),
    ([16], [3333], 4, 2, 64, True, F16),
    ([16, 1, 40], [2500, 4100, 1100], 14, 2, 64, True, BF16),
    ([5, 0, 200], [4000, 0, 1500], 3, 3, 128, False, F16),
    ([100, 30], [7000, 10], 4, 1, 128, True, BF16),      # a sequence with fewer keys than queries
    ([1], [65536], 4, 4, 64, True, BF16),
]


@pytest.mark.parametrize("i", range(len(SHARED)))
def test_keys_shared_by_workgroups(i):
    lens, keys, heads, kv, dim, causal, dtype = SHARED[i]
    assert vts.library().vts_prompt_attention_workspace_bytes(len(lens), sum(lens), sum(keys), heads, kv, dim) > 0
    gen = torch.Generator().manual_seed(820 + i)
    q = (1.5 * torch.randn(sum(lens) + 3, heads, dim, generator=gen)).to(dtype).to(DEV)
    k, v = (torch.randn(sum(keys), kv, dim, generator=gen).to(dtype).to(DEV) for _ in "kv")
    n = sum(lens)
    out, lse = check(q[:n], k, v, cu(lens), cu(keys), causal)
    # what is not finite and not seen, in the last keys of a sequence
    if causal and lens[0] > 1:
        k2, v2 = k.clone(), v.clone()
        v2[keys[0] - 1] = math.inf
        v2[keys[0] - 2, 0, 3] = math.nan
        k2[keys[0] - 1, :, 5] = math.nan
        got, _ = vts.prompt_attention(q[:n], k2, v2, cu(lens), cu_seqlens_k=cu(keys))
        assert torch.equal(got[:lens[0] - 2], out[:lens[0] - 2]) and torch.equal(got[lens[0]:], out[lens[0]:])
        assert got[lens[0] - 2, 0, 3].isnan() and not got[lens[0] - 1].isfinite().any()
    # rows of no sequence, another stream, a captured graph
    room = torch.full_like(q, 3.0)
    vts.prompt_attention(q, k, v, cu(lens), cu_seqlens_k=cu(keys), out=room, causal=causal)
    assert torch.equal(room[:n], out) and (room[n:] == 3).all()
    at_q, at_k = cu(lens), cu(keys)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g, gl = vts.prompt_attention(q, k, v, at_q, cu_seqlens_k=at_k, return_lse=True, causal=causal)
    for turn in range(3):
        if turn:
            v.mul_(-1.5)
        want, _ = vts.prompt_attention(q, k, v, at_q, cu_seqlens_k=at_k, causal=causal)
        g.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(g, want) and torch.equal(gl[:n], lse), turn
