"""verify_draft against the rule as include/vts.h states it, residuals formed one
after the other and normalised by their own sums in 64 bits: nodes without a
draft, chosen siblings over rows whose sum is not 1."""
import numpy as np
import pytest
import torch

import varlen_top_select_amd as vts

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"


def definition(target, tokens, uniforms, drafts=None, parents=None):
    target = np.maximum(target.double().numpy(), 0)
    drafts = None if drafts is None else np.maximum(drafts.double().numpy(), 0)
    tokens, u = tokens.tolist(), uniforms.double().tolist()
    batch, n, vocab = len(tokens), len(tokens[0]), target.shape[2]
    paths, nexts = [], []
    for b in range(batch):
        up = list(range(-1, n - 1)) if parents is None else parents[b].tolist()
        cur, path, r = -1, [], target[b, 0].copy()
        for t in range(n):
            x = tokens[b][t]
            if up[t] != cur or not -1 <= up[t] < t or not 0 <= x < vocab:
                continue  # not a child, or no node
            if drafts is None:
                q = np.zeros(vocab)
                q[x] = 1
            else:
                q = drafts[b, cur + 1]
            if u[b][t] * q[x] < r[x]:
                path.append(t)
                cur = t
                r = target[b, t + 1].copy()
                continue
            r = np.maximum(r - q, 0)
            r = r / r.sum() if r.sum() > 0 else r
        if r.sum() == 0:
            r = target[b, cur + 1]
        c = np.cumsum(r)
        hit = np.nonzero((c > u[b][n] * c[-1]) & (r > 0))[0]
        nexts.append(int(hit[0]) if len(hit) else int(np.nonzero(r > 0)[0][-1]) if r.any() else -1)
        paths.append(path + [-1] * (n - len(path)))
    return paths, nexts


def check(target, tokens, u, drafts=None, parents=None):
    dev = [None if x is None else x.to(DEV) for x in (target, tokens, u, drafts, parents)]
    path, count, token = vts.verify_draft(dev[0], dev[1], dev[2], draft_probs=dev[3], parents=dev[4])
    torch.cuda.synchronize()
    paths, nexts = definition(target, tokens, u, drafts, parents)
    assert path.cpu().tolist() == paths
    assert count.cpu().tolist() == [sum(x >= 0 for x in p) for p in paths]
    assert token.cpu().tolist() == nexts
    return paths, nexts


def softmax(gen, *shape, scale=1.0, dtype=torch.float32):
    return torch.softmax(scale * torch.randn(*shape, generator=gen), -1).to(dtype)


# ---- nodes without a draft


@pytest.mark.parametrize("none", [-1, 2, 2 ** 31 - 1])
def test_no_draft_takes_nothing_from_the_target(none):
    """Nothing was drawn from q, so the next token is drawn from p itself."""
    u = torch.tensor([[0.5, x] for x in (0.0, 0.2, 0.49, 0.51, 0.9)])
    n = len(u)
    target = torch.tensor([0.5, 0.5]).expand(n, 2, 2).contiguous()
    drafts = torch.tensor([0.9, 0.1]).expand(n, 1, 2).contiguous()
    tokens = torch.full((n, 1), none, dtype=torch.int32)
    for parents in (None, torch.full((n, 1), -1, dtype=torch.int32)):
        paths, nexts = check(target, tokens, u, drafts, parents)
        assert nexts == [0, 0, 0, 1, 1] and paths == [[-1]] * n


@pytest.mark.parametrize("vocab", [50, 9001, 40000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_requests_with_fewer_drafts(vocab, dtype):
    """Chains cut short, and trees with holes among the siblings."""
    gen = torch.Generator().manual_seed(60 + vocab)
    batch, draft = 12, 6
    target = softmax(gen, batch, draft + 1, vocab, dtype=dtype)
    drafts = softmax(gen, batch, draft, vocab, dtype=dtype)
    for parents in (None, torch.tensor([-1, -1, -1, 0, 1, 1], dtype=torch.int32).repeat(batch, 1)):
        rows = torch.arange(draft).expand(batch, -1) if parents is None else parents.long() + 1
        dist = drafts.float().gather(1, rows[..., None].expand(-1, -1, vocab)).reshape(-1, vocab)
        tokens = torch.multinomial(dist, 1, generator=gen).view(batch, draft).int()
        for b in range(batch):
            if parents is None:
                tokens[b, b % (draft + 1):] = -1
            else:
                tokens[b, [0, 1, 2, 4][b % 4]] = -1
                tokens[b, b % draft] = vocab
        for _ in range(4):
            u = torch.rand(batch, draft + 1, generator=gen)
            check(target, tokens, u, drafts, parents)
            check(target, tokens, u, None, parents)


def test_nodes_that_are_not_there():
    """Tokens outside the vocabulary and parents that are no earlier node."""
    gen = torch.Generator().manual_seed(52)
    target = torch.softmax(torch.randn(2, 7, 50, generator=gen), -1)
    drafts = torch.softmax(torch.randn(2, 6, 50, generator=gen), -1)
    tokens = torch.tensor([[-1, 50, 3, 2 ** 31 - 1, 4, 5], [1, 2, 3, 4, 5, 6]], dtype=torch.int32)
    parents = torch.tensor([[-1, -1, -1, 2, 2, 4], [-2, 5, 2 ** 31 - 1, -2 ** 31, -1, 4]],
                           dtype=torch.int32)
    for u in (0.0, 0.1, 0.3, 0.7, 0.99):
        x = torch.full((2, 7), u)
        check(target, tokens, x, drafts, parents)
        check(target, tokens, x, None, parents)


@pytest.mark.parametrize("drawn", [True, False])
def test_distribution_with_holes(drawn):
    """The outcome's first token is distributed as the target, holes or not."""
    gen = torch.Generator().manual_seed(61)
    batch, vocab = 40000, 4
    p = torch.tensor([0.4, 0.3, 0.2, 0.1])
    q = torch.tensor([0.1, 0.2, 0.3, 0.4])
    parents = torch.full((batch, 4), -1, dtype=torch.int32)
    tokens = torch.multinomial(q.expand(batch * 4, vocab), 1, generator=gen).view(batch, 4).int()
    tokens[:, 0] = -1
    tokens[::2, 2] = vocab
    u = torch.rand(batch, 5, generator=gen)
    path, count, token = vts.verify_draft(p.expand(batch, 5, vocab).contiguous().to(DEV), tokens.to(DEV),
                                          u.to(DEV), parents=parents.to(DEV),
                                          draft_probs=q.expand(batch, 4, vocab).contiguous().to(DEV)
                                          if drawn else None)
    at = path.cpu()[:, :1].clamp(min=0).long()
    first = torch.where(count.cpu() > 0, tokens.gather(1, at)[:, 0], token.cpu())
    share = torch.bincount(first.long(), minlength=vocab).double() / batch
    # five standard deviations of a share
    assert ((share - p.double()).abs() <= 5 * (p.double() * (1 - p.double()) / batch).sqrt()).all()


# ---- chosen siblings


def best(target, parents):
    """Siblings are their parent's best tokens, in order."""
    batch, draft = parents.shape
    tokens = torch.zeros(batch, draft, dtype=torch.int32)
    for b in range(batch):
        used = {}
        for t in range(draft):
            row = int(parents[b, t]) + 1
            rank = used.get(row, 0)
            used[row] = rank + 1
            order = torch.argsort(target[b, row].float(), descending=True, stable=True)
            tokens[b, t] = order[min(rank, len(order) - 1)]
    return tokens


def test_rows_whose_sum_is_not_one():
    """After a rejection the rest counts by its own sum: (0.5, 0.4) is (1) without its first."""
    row = torch.tensor([[0.5, 0.4, 0.0, 0.0], [0.3, 0.2, 0.0, 0.0], [0.5, 0.4, 0.3, 0.2], [0.9, 0.9, 0.9, 0.9]])
    target = row[:, None].repeat(1, 4, 1)
    parents = torch.full((4, 3), -1, dtype=torch.int32)
    tokens = torch.tensor([[0, 1, 2]] * 4, dtype=torch.int32)
    u = torch.tensor([[0.95, 0.93, 0.9, 0.5]] * 4)
    paths, _ = check(target, tokens, u, None, parents)
    assert paths[0] == paths[1] == [1, -1, -1]
    for x in (0.2, 0.5, 0.8, 0.99):
        check(target, tokens, torch.full((4, 4), x), None, parents)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab,scale", [(37, 3.0), (4099, 6.0), (30011, 8.0)])
def test_sharp_targets(dtype, vocab, scale):
    """What two best tokens leave of a sharp row is far below a 16-bit row's error."""
    gen = torch.Generator().manual_seed(62 + vocab)
    batch, draft = 16, 9
    target = softmax(gen, batch, draft + 1, vocab, scale=scale, dtype=dtype)
    parents = torch.tensor([-1, -1, -1, -1, 2, 2, 3, 3, 5], dtype=torch.int32).repeat(batch, 1)
    tokens = best(target, parents)
    seen = set()
    for forced in (2, 3, 4, 0):
        for _ in range(3):
            u = torch.rand(batch, draft + 1, generator=gen)
            u[:, :forced] = 1 - 2.0 ** -24  # rejected unless the token has all there is
            paths, _ = check(target, tokens, u, None, parents)
            seen |= {p[0] for p in paths}
    assert len(seen) > 2


def test_chosen_deep_trees():
    """Rejections at many nodes of one path, and the same token among siblings."""
    gen = torch.Generator().manual_seed(63)
    batch, draft, vocab = 6, 63, 9001
    target = softmax(gen, batch, draft + 1, vocab, scale=4.0, dtype=torch.bfloat16)
    parents = torch.tensor([t // 3 * 3 - 1 for t in range(draft)], dtype=torch.int32).repeat(batch, 1)
    tokens = best(target, parents)
    tokens[:, 1::9] = tokens[:, 0::9]  # twice the same
    for _ in range(6):
        u = torch.rand(batch, draft + 1, generator=gen)
        u[:, 2::3] = 0  # the third sibling is taken where it can be
        check(target, tokens, u, None, parents)


def test_nothing_left_of_a_row():
    """All of the row's mass rejected: later siblings cannot be taken, p itself is drawn from."""
    target = torch.zeros(2, 4, 5000)
    target[:, :, 7], target[:, :, 4000] = 0.25, 0.25
    tokens = torch.tensor([[7, 4000, 9], [7, 7, 4000]], dtype=torch.int32)
    parents = torch.full((2, 3), -1, dtype=torch.int32)
    u = torch.tensor([[0.5, 0.999, 0.0, 0.6], [0.9, 0.0, 0.5, 0.6]])
    paths, _ = check(target, tokens, u, None, parents)
    assert paths == [[1, -1, -1], [2, -1, -1]]
    target[:, :, 4000] = 0
    paths, nexts = check(target, tokens, u, None, parents)
    assert paths == [[-1, -1, -1]] * 2 and nexts == [7, 7]
