"""The README's step of a beam search, run as it stands: every beam's row of the cache is its parent's."""
import os
import re

import pytest
import torch

import block_sparse_attention_slice_gb300 as attn
from conftest import ROOT
from test_gpu_cache8 import Pages, ints, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_the_beam_step_of_the_readme(fmt):
    with open(os.path.join(ROOT, "README.md")) as f:
        step = re.search(r"^# a beam search's step.*?(?=^```)", f.read(), re.S | re.M).group(0)
    G, Bm, page_size, V = 2, 3, 16, 40
    rows = G * Bm
    p = Pages(fmt, 60, page_size, 2, 64)
    k8, v8, ks, vs = p.k, p.v, p.ks, p.vs
    table = torch.full((rows, 6), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(60, dtype=torch.int32, device="cuda")
    slots, counts = ints(list(range(rows))), [21, 5, 40, 16, 33, 7]
    ptr, total = ints([0, 21, 26, 66, 82, 115, 122]), sum(counts)
    attn.attn_cache_extend(table, lens, refs, slots, ints(counts), page_size)
    attn.attn_cache_write(k8, v8, tokens(total, 2, 64, 1).cuda(), tokens(total, 2, 64, 2).cuda(), table, lens, ptr, k_scales=ks, v_scales=vs)
    read = lambda n, q: attn.attn_cache_read(k8, v8, table, lens, n, q_ptr=q, out_dtype=torch.float32, k_scales=ks, v_scales=vs)  # noqa: E731
    before = read(total, ptr)
    logits = torch.randn((rows, V), generator=torch.Generator().manual_seed(0)).cuda()
    scores = ints([[0, -1, -30], [-20, 0, -20]]).float()           # parents that have several children, and some that have none
    names = dict(attn=attn, k8=k8, v8=v8, ks=ks, vs=vs, table=table, lens=lens, refs=refs, page_size=page_size, slots=slots, logits=logits, scores=scores,
                 done=torch.zeros((G, Bm), dtype=torch.bool, device="cuda"), eos=1, history=torch.arange(rows * 4, device="cuda").view(rows, 4))
    exec(step, names)
    assert attn.attn_last_device_error() == 0
    parents = names["parents"].view(-1).tolist()
    assert len(set(parents)) < rows and lens.tolist() == [counts[a] for a in parents]
    assert names["history"][:, 0].tolist() == [4 * a for a in parents]
    ends = torch.cat([ints([0]), lens.cumsum(0).int()])
    for was, now in zip(before, read(int(lens.sum()), ends)):
        want = torch.cat([was[ptr[a]:ptr[a + 1]] for a in parents])
        assert torch.equal(want.nan_to_num(-7.0), now.nan_to_num(-7.0))
