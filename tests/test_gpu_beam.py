"""A beam search's choice and the reordering of its states against the oracle."""
import numpy as np
import pytest
import torch

import oracle
from block_sparse_attention_slice_gb300 import AttnError, attn_beam_reorder, attn_beam_select, attn_last_device_error
from block_sparse_attention_slice_gb300 import binding as B

pytestmark = pytest.mark.gpu
INF = float("inf")


def run(logits, scores, done=None, eos=-1, keep=None, **kw):
    """The call, held to the oracle: whole numbers exactly (where no two scores are as near as the sums'
    rounding), scores to 2^-24 of themselves and 2^-20 for the sum of exponentials (each off by 2^-22, f32 sums of
    32 terms and two trees: below 2^-21)."""
    want = oracle.oracle_beam_select(logits.double().cpu().numpy(), scores.cpu().numpy(), None if done is None else done.cpu().numpy(), eos, keep)
    got = attn_beam_select(logits, scores, done=done, eos=eos, keep=keep, **kw)
    assert attn_last_device_error() == 0
    s, w = got[0].double().cpu().numpy(), want[0]
    fin = np.isfinite(w)
    assert np.array_equal(np.isneginf(s), ~fin)
    assert np.all(np.abs(s[fin] - w[fin]) <= 2.0 ** -24 * np.abs(w[fin]) + 2.0 ** -20)
    r = want[4][:, :w.shape[1] + 1]
    with np.errstate(invalid="ignore"):
        gap = np.abs(np.diff(r, axis=1))
    assert not np.any((gap > 1e-12) & (gap < 4e-6)), "the inputs hold scores too near to tell apart"
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[2].cpu().numpy(), want[2])
    assert got[3].dtype == torch.bool and np.array_equal(got[3].cpu().numpy(), want[3])
    return got


def make(G, Bm, V, seed, dtype=torch.float32, sigma=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((G * Bm, V), generator=g) * sigma).to(dtype).cuda(), (-20 * torch.rand((G, Bm), generator=g)).cuda()


SIZES = [(1, 1, 1), (1, 1, 2), (3, 2, 5), (1, 4, 50), (7, 5, 1000), (2, 3, 2047), (2, 3, 2049), (1, 4, 32000), (40, 4, 8193), (3, 8, 100003), (1, 64, 700), (2, 16, 3000)]


@pytest.mark.parametrize("G,Bm,V", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sizes(G, Bm, V, dtype):
    logits, scores = make(G, Bm, V, G + V, dtype)
    if dtype == torch.bfloat16:       # few different logits: equal ones within a beam are many, and the lowest token stands first
        logits = (logits * 4).round() / 4
    run(logits, scores, keep=min(Bm, Bm * V))


@pytest.mark.parametrize("keep", [1, 2, 13, 64])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_keep(keep, dtype):
    logits, scores = make(3, 4, 9001, keep, dtype)
    run(logits, scores, keep=keep)
    logits, scores = make(2, 2, 32, keep + 5, torch.float32)
    run(logits, scores, keep=keep)


def test_rows_apart_and_unaligned():
    logits, scores = make(4, 3, 5003, 0)
    for skip, pad in ((0, 0), (1, 2), (3, 1), (2, 0)):
        wide = torch.full((12, 5003 + skip + pad), INF, device="cuda")
        wide[:, skip:skip + 5003] = logits
        run(wide[:, skip:skip + 5003], scores)
        b = torch.full((12, 5003 + skip + pad), INF, device="cuda", dtype=torch.bfloat16)
        b[:, skip:skip + 5003] = logits
        run(b[:, skip:skip + 5003], scores)


def test_equal_logits_and_equal_beams():
    scores = torch.zeros((2, 3), device="cuda")
    for V, keep in ((10, 5), (5000, 3), (40000, 64)):       # all equal: the lists overflow, places decide
        got = run(torch.full((6, V), 1.5, device="cuda"), scores, keep=keep)
        assert got[2][0].tolist() == ([0, 1, 2, 3, 4] if V == 10 else list(range(keep)))
    logits, _ = make(2, 1, 6000, 3)
    run(logits.repeat_interleave(3, 0), scores, keep=7)      # beams alike: the lowest beam first


@pytest.mark.parametrize("left", [0, 1, 3, 40])
def test_most_of_a_vocabulary_ruled_out(left):
    logits, scores = make(3, 4, 30000, left)
    allowed = torch.zeros_like(logits, dtype=torch.bool)
    for r in range(len(logits)):
        allowed[r, torch.randperm(30000, generator=torch.Generator().manual_seed(r))[:left].cuda()] = True
    logits.masked_fill_(~allowed, -INF)
    run(logits, scores, keep=16)
    low = torch.where(allowed, logits, torch.finfo(torch.float32).min)       # the type's lowest value instead
    if left:
        run(low, scores, keep=min(16, left))


def test_first_step_and_ended_beams():
    logits, scores = make(5, 4, 777, 1)
    first = torch.full_like(scores, -INF)
    first[:, 0] = 0
    run(logits, first)
    done = torch.tensor([[0, 0, 0, 0], [1, 0, 0, 0], [0, 1, 1, 0], [1, 1, 1, 1], [1, 1, 1, 0]], dtype=torch.bool, device="cuda")
    logits[done.view(-1)] = float("nan")      # of no use any more
    for eos in (0, 3, 776):
        got = run(logits, scores, done, eos)
        assert got[3][3].all() and torch.equal(got[0][3], scores[3].sort(descending=True).values)
        run(logits, scores, done, eos, keep=30)
    scores[3, 1], scores[1, 0] = -INF, float("nan")       # an ended beam without a score
    run(logits, scores, done, 5, keep=9)
    run(logits, scores, done.to(torch.uint8) * 3, 5, keep=9)


def test_beams_without_a_sum():
    logits, scores = make(4, 3, 4000, 2)
    logits[1, 17], logits[4, 3999], logits[8] = float("nan"), INF, -INF
    scores[3, 2] = INF
    run(logits, scores, keep=5)
    logits[:] = -INF       # nothing can be: the first places, at -inf
    got = run(logits, scores, keep=5)
    assert torch.isneginf(got[0]).all() and got[2][0].tolist() == [0, 1, 2, 3, 4] and not got[1][0].any()


def test_far_from_zero():
    logits, scores = make(3, 4, 5000, 9)
    for shift in (-1000.0, 300.0):
        run((logits + shift), scores - 1e4)


def test_slots_streams_and_graphs():
    logits, scores = make(6, 4, 20000, 4)
    done = torch.zeros((6, 4), dtype=torch.bool, device="cuda")
    slots = torch.randperm(24, generator=torch.Generator().manual_seed(0)).int().cuda() + 100
    want = attn_beam_select(logits, scores, done=done, eos=1, slots=slots)
    assert torch.equal(want[4], slots[want[1].long()])
    s = torch.cuda.Stream()
    got = attn_beam_select(logits, scores, done=done, eos=1, slots=slots, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    state, first = torch.arange(24 * 5, device="cuda").view(24, 5), torch.arange(24 * 5, device="cuda").view(24, 5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = attn_beam_select(logits, scores, done=done, eos=1, slots=slots)
        attn_beam_reorder([state], got[1])
    for _ in range(2):
        state.copy_(first)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(state, first[want[1].view(-1).long()])
    assert attn_last_device_error() == 0


def parents_of(G, Bm, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, Bm, (G, Bm), generator=g) + torch.arange(G)[:, None] * Bm).int().cuda()


@pytest.mark.parametrize("G,Bm", [(1, 1), (1, 2), (5, 4), (3, 5), (2, 8), (4, 13), (2, 16), (3, 17), (2, 64)])
def test_reorder(G, Bm):
    rows, g = G * Bm, torch.Generator().manual_seed(G)
    rand = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.int32)  # noqa: E731
    wide = rand(rows, 40).cuda()
    odd = rand(rows * 7 + 3).to(torch.uint8).cuda()
    states = [rand(rows, 3).cuda(), rand(rows, 4, 9).cuda().to(torch.bfloat16), rand(rows, 1001).to(torch.uint8).cuda(), rand(rows, 256).cuda(),
              rand(rows).cuda(), rand(rows, 0).cuda(), wide[:, 4:20], odd[3:].view(rows, 7), rand(rows, 70000).to(torch.uint8).cuda()]
    for seed in range(2):
        parents = parents_of(G, Bm, seed)
        want = [x.clone()[parents.view(-1).long()] for x in states]
        rest = wide[:, 20:].clone(), odd[:3].clone()
        attn_beam_reorder(states, parents)
        assert attn_last_device_error() == 0
        assert all(torch.equal(x, y) for x, y in zip(states, want))
        assert torch.equal(wide[:, 20:], rest[0]) and torch.equal(odd[:3], rest[1])
    attn_beam_reorder([], parents)
    attn_beam_reorder(states, torch.arange(rows, dtype=torch.int32, device="cuda").view(G, Bm))
    assert all(torch.equal(x, y) for x, y in zip(states, want))


def test_reorder_leaves_a_group_with_a_bad_parent():
    x = torch.arange(12, device="cuda").view(6, 2)
    for bad in (-1, 2, 6):
        y = x.clone()
        attn_beam_reorder([y], torch.tensor([[1, 0], [3, 2], [4, bad]], dtype=torch.int32, device="cuda"))
        assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
        assert torch.equal(y, x[[1, 0, 3, 2, 4, 5]])


def test_reorder_of_rows_past_four_gigabytes():
    n = 1 << 31
    x = torch.zeros((3, n), dtype=torch.uint8, device="cuda")
    x[:, -1] = torch.tensor([1, 2, 3], dtype=torch.uint8)
    x[:, n // 2 + 5] = torch.tensor([4, 5, 6], dtype=torch.uint8)
    attn_beam_reorder([x], torch.tensor([[2, 0, 0]], dtype=torch.int32, device="cuda"))
    assert attn_last_device_error() == 0
    assert x[:, -1].tolist() == [3, 1, 1] and x[:, n // 2 + 5].tolist() == [6, 4, 4]


@pytest.mark.parametrize("G,Bm,V,keep", [(1, 64, 5000, 64), (20000, 2, 40, 2), (3000, 5, 70, 7), (1, 1, 1 << 21, 64), (700, 3, 3001, 3)])
def test_the_most_beams_prompts_and_tokens(G, Bm, V, keep):
    logits, scores = make(G, Bm, V, 3)
    run(logits, scores, keep=keep)


def test_calls_at_once():
    logits, scores = make(9, 4, 30000, 6)
    want = attn_beam_select(logits, scores)
    states = [torch.arange(36 * 7, device="cuda").view(36, 7) + i for i in range(3)]
    first = [x.clone() for x in states]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for x, s in zip(states, streams):
        got.append(attn_beam_select(logits, scores, stream=s))
        attn_beam_reorder([x], got[-1][1], stream=s)
    torch.cuda.synchronize()
    for g, x, y in zip(got, states, first):
        assert all(torch.equal(a, b) for a, b in zip(g, want))
        assert torch.equal(x, y[want[1].view(-1).long()])
    assert attn_last_device_error() == 0


def test_refusals_of_tensors():
    logits, scores = make(2, 3, 100, 0)
    done = torch.zeros((2, 3), dtype=torch.bool, device="cuda")
    for bad in (dict(logits=logits.half()), dict(logits=logits.t().contiguous().t()), dict(logits=logits[:5]), dict(logits=logits[None]), dict(scores=scores.cpu()),
                dict(scores=scores.double()), dict(scores=scores.t()), dict(done=done.int()), dict(done=done[:1]), dict(done=done.cpu()), dict(slots=scores),
                dict(slots=torch.zeros(5, dtype=torch.int32, device="cuda")), dict(ws=torch.zeros(1 << 16))):
        with pytest.raises(ValueError):
            attn_beam_select(**{**dict(logits=logits, scores=scores, eos=1), **bad})
    for bad in (dict(keep=0), dict(keep=65), dict(eos=100), dict(done=done), dict(ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(AttnError):
            attn_beam_select(logits, scores, **bad)
    parents = parents_of(2, 3, 0)
    x = torch.zeros((6, 4, 5), device="cuda")
    for bad in ([x[:5]], [x.cpu()], [x.transpose(1, 2)], [x[0, 0, 0]], [x, x[:, :, ::2]]):
        with pytest.raises(ValueError):
            attn_beam_reorder(bad, parents)
    for bad in ([x, x], [x[:1].expand(6, -1, -1)], [x.clone() for _ in range(65)]):
        with pytest.raises(AttnError):
            attn_beam_reorder(bad, parents)
    for bad in (parents.long(), parents.view(-1), parents.cpu(), parents.t()):
        with pytest.raises(ValueError):
            attn_beam_reorder([x], bad)
    with pytest.raises(TypeError):
        attn_beam_reorder([x, 7], parents)
    attn_beam_reorder([], parents)
    attn_beam_reorder([x[:, :0], x], parents)
    assert attn_last_device_error() == 0


def test_states_side_by_side_in_one_tensor():
    """Columns of one tensor as states of their own."""
    x = torch.randint(0, 100, (12, 40), generator=torch.Generator().manual_seed(0)).cuda()
    parents = parents_of(3, 4, 1)
    want = x[parents.view(-1).long()]
    y = x.clone()
    attn_beam_reorder([y[:, :8], y[:, 8:17], y[:, 17:]], parents)
    assert torch.equal(y, want)
