"""A beam search's step on a stream of its own, behind work that the current stream still has to do."""
import pytest
import torch

from block_sparse_attention_slice_gb300 import attn_beam_reorder, attn_beam_select, attn_last_device_error
from test_gpu_beam import make

pytestmark = pytest.mark.gpu


def test_another_stream_waits_for_the_current_one():
    logits, scores = make(6, 4, 5000, 4)
    want = attn_beam_select(logits, scores)
    first = torch.arange(24 * 9, device="cuda").view(24, 9)
    s = torch.cuda.Stream()
    late, state, parents = torch.zeros_like(logits), torch.zeros_like(first), torch.zeros_like(want[1]) + torch.arange(6, device="cuda").int()[:, None] * 4
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)       # about 50 ms
    late.copy_(logits), state.copy_(first), parents.copy_(want[1])
    got = attn_beam_select(late, scores, stream=s)
    attn_beam_reorder([state], parents, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(state, first[want[1].view(-1).long()])
    # and without a call before it that waits
    s = torch.cuda.Stream()
    state.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    state.copy_(first)
    attn_beam_reorder([state], parents, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(state, first[want[1].view(-1).long()])
    assert attn_last_device_error() == 0


def test_a_captured_step_on_the_capturing_stream():
    x = torch.arange(12, device="cuda").view(6, 2)
    parents = torch.tensor([[1, 1, 0], [5, 3, 4]], dtype=torch.int32, device="cuda")
    want = x[parents.view(-1).long()]
    attn_beam_reorder([x.clone()], parents)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        attn_beam_reorder([x], parents, stream=s)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want)
