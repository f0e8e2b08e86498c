"""Equal continuations of different beams stand in the order of their places, wherever the beams' rows
lie in memory."""
import pytest
import torch

from block_sparse_attention_slice_gb300 import attn_beam_select, attn_last_device_error
from test_gpu_beam import make, run

pytestmark = pytest.mark.gpu


def spread(logits, pad, skip):
    """The same rows `pad` more elements apart, the first `skip` behind a word."""
    rows, V = logits.shape
    wide = torch.full((rows, V + pad), float("inf"), dtype=logits.dtype, device="cuda")
    wide[:, skip:skip + V] = logits
    return wide[:, skip:skip + V]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [10, 6001, 6002, 6004, 30011, 100003])
@pytest.mark.parametrize("pad,skip", [(0, 0), (1, 1), (2, 1), (4, 3), (7, 5)])
def test_beams_alike(V, pad, skip, dtype):
    """All beams of a prompt have one row and one score: of each token the beams in their order."""
    for seed in range(3):
        logits, _ = make(4, 1, V, seed, dtype)
        beams = spread(logits.repeat_interleave(8, 0), pad, skip)
        got = run(beams, torch.full((4, 8), -1.5, device="cuda"), keep=20)
        assert dtype == torch.bfloat16 or torch.equal(got[1].cpu() % 8, (torch.arange(20) % 8).expand(4, 20).int())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [6001, 50257])
def test_pairs_of_beams_alike(V, dtype):
    """Two of five beams have one row, apart from one another, and equal scores."""
    for seed in range(4):
        logits, scores = make(3, 5, V, seed, dtype)
        logits[4::5], scores[:, 4] = logits[1::5], scores[:, 1]
        scores[:, 1] = scores[:, 4] = 0.0
        run(logits, scores, keep=16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 5, 100, 513, 2049, 20001])
@pytest.mark.parametrize("pad", [0, 1, 2, 3, 4, 8])
def test_rows_apart(V, pad, dtype):
    logits, scores = make(3, 4, V, V, dtype)
    for skip in range(pad + 1):
        run(spread(logits, pad, skip), scores, keep=min(9, 4 * V))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [50, 6001, 100003, 1 << 21])
@pytest.mark.parametrize("sigma", [0.01, 2.5])
def test_beams_as_near_as_their_sums_tell_apart(V, sigma, dtype):
    """Rows of the same logits in other orders: their sums differ by rounding alone, at most 2^-19 each, and
    scores 2^-18 apart and more decide."""
    gen = torch.Generator().manual_seed(V)
    row = (torch.randn(V, generator=gen) * sigma).to(dtype)
    row = row.clamp(max=7.5)
    row[0] = 8.0       # the best of each beam
    beams = torch.stack([row[torch.randperm(V, generator=gen)] for _ in range(8)]).cuda()
    order = torch.randperm(8, generator=gen)
    scores = torch.empty(8)
    scores[order] = -torch.arange(8).float() * 2.0 ** -18 * 1.0625
    got = attn_beam_select(beams, scores.view(1, 8).cuda())
    assert got[1].view(-1).tolist() == order.tolist()
    assert torch.equal(got[2].view(-1).cpu(), (beams == 8).int().argmax(1).int().cpu()[order])
    assert attn_last_device_error() == 0
