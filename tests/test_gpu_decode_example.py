"""The decode example runs its operators together: lengths and counts fit, the
evicted cache keeps its budget, and a draft that equals the target is accepted."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

from varlen_top_select_amd.decode_example import PAGE, VOCAB, Decoder  # noqa: E402


def test_decode_loop():
    d = Decoder(batch=3, budget=64, top_k=20)
    total = torch.zeros(3, dtype=torch.int64, device="cuda")
    evicted = False
    for _ in range(250):  # a token a step at least: the budget is passed on the way
        count, tokens = d.step()
        assert ((count >= 0) & (count <= d.draft)).all()
        assert ((tokens[:, -1] >= 0) & (tokens[:, -1] < VOCAB)).all()
        total += 1 + count
        assert torch.equal(d.layers[1].lens.long(), total)
        evicted = evicted or (d.layers[0].lens.long() < total).any().item()
        assert int(d.layers[0].lens.max()) <= d.layers[0].width * PAGE
        # what is accumulated is one unit of weight per counted row and head
        assert torch.isfinite(d.layers[0].weights).all()
    assert evicted


def test_weights_add_up():
    """Before anything is evicted each counted row spreads a weight of 1 per head."""
    d = Decoder(batch=2)
    rows = torch.zeros(2, device="cuda")
    for _ in range(10):
        count, _ = d.step()
        rows += 1 + count
    per_head = d.layers[0].weights.sum(-1)
    want = rows[:, None] * 4  # query heads to a KV head
    # the score's and the exponential's errors, 2^-20 a row at these magnitudes
    assert torch.allclose(per_head, want.expand_as(per_head), rtol=1e-5)


def test_draft_equal_to_the_target_is_accepted():
    d = Decoder(batch=2)
    for p in d.proj:
        p.zero_()  # no attention: the target is the bigram itself
    for _ in range(5):
        count, _ = d.step()
        # (rows of x @ unembed may round differently by their number)
        assert (count >= d.draft - 1).all()
