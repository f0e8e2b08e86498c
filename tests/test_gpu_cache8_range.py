"""Attention over a cache in 8 bits where the scales of one sequence lie far apart: small ones before
large ones, none (0) beside large ones, and scores that grow from key to key.  Each case goes to every
kernel, many times the same sequence in one call, so that an item has several slabs of one warp."""
import numpy as np
import pytest
import torch

from block_sparse_attention_slice_gb300 import attn_last_device_error, attn_paged_fwd
from oracle import codes as C
import paged8_cases as P8
import paged_cases as P
from test_gpu_cache8 import FMTS, ints, prefix

pytestmark = pytest.mark.gpu
PAGE, G = 16, 4
FACTORS = (1.0, 0.75, 1.5, 0.875)        # of a token's heads: their queries

# tokens of a sequence and sequences of a call, by the kernel that they go to
KERNELS = {"up to 8 rows": (1, 900), "16 rows, 4 warps": (1, 80), "16 rows, 8 warps": (1, 250), "20 rows": (5, 500), "a row tile": (12, 300),
           "two row tiles": (60, 100)}


def tiny_then_huge(n, rng):
    return np.zeros(n), np.where(np.arange(n) < n // 2, 1.1e-24, 3e12)


def zeros_that_stand_above(n, rng):
    """A row of zeros whose score stands far above the others of its block; later ones reach it."""
    s, v = np.zeros(n), np.full(n, 1e-3)
    s[0], v[0] = 118.0, 0.0
    s[32:], v[32:] = 116.5, 8.0
    return s, v


def huge_then_tiny_rising(n, rng):
    b = np.arange(n) // 32
    return 9.0 * b, np.where(b % 3 == 0, 1e13, 1e-24)


def zeros_beside_huge(n, rng):
    return 4 * rng.random(n), np.where(rng.random(n) < 0.3, 0.0, 2.0 ** 70)


def all_sizes(n, rng):
    return 60 * rng.random(n), 10.0 ** rng.uniform(-24, 24, n)


def all_sizes_rising(n, rng):
    return 0.35 * np.arange(n) + 30 * rng.random(n), 10.0 ** rng.uniform(-24, 24, n)


def zeros_alone(n, rng):
    return rng.random(n), np.zeros(n)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("case", [tiny_then_huge, zeros_that_stand_above, huge_then_tiny_rising, zeros_beside_huge, all_sizes, all_sizes_rising, zeros_alone])
def test_scales_far_apart(case, kernel, d, fmt):
    """Bounds: u = 2^-24, N keys.  A score S (of d equal products and their scales) is off by r = (d + 12) u S + 2^-22,
    a weight by that, twice with the sum's; sums in f32 by N u, merges by 2^-21.  A weight times its
    value's scale is rounded to bf16 (h = 2^-8) or to f16, whose smallest step, 2^-24 where the row's largest such
    product W so far is 1 at least, adds half of it times the largest code: N 2^-25 max_j p_j |v_j|, doubled."""
    news, copies = KERNELS[kernel]
    n = 700
    rng = np.random.default_rng(3)
    logs, vs = case(n, rng)
    scale = 0.125
    # codes of keys are all ones: a key's score for a query of f everywhere is scale f d ks
    one = 1 if fmt == "int8" else 0x38
    ks = (logs * np.log(2.0) / (scale * d)).astype(np.float32)
    vs = vs.astype(np.float32)
    pages = -(-n // PAGE)
    k = torch.full((pages, PAGE, 1, d), one, dtype=torch.int8)
    vc = torch.from_numpy(rng.integers(-127, 128, (pages, PAGE, 1, d)).astype(np.int8))
    if fmt == "e4m3":
        vc[(vc & 127) == 127] = 0x7e
    v64 = C.values(vc.numpy(), fmt).reshape(-1, d)[:n] * vs[:, None].astype(np.float64)
    scales = [torch.full((pages * PAGE,), float("nan")) for _ in range(2)]
    for x, y in zip(scales, (ks, vs)):
        x[:n] = torch.from_numpy(y)
    scales = [x.view(pages, PAGE, 1).cuda() for x in scales]
    table = torch.arange(pages, dtype=torch.int32)[None].cuda()
    q = torch.tensor(FACTORS).bfloat16()[None, :, None].expand(copies * news, G, d).contiguous().cuda()
    out, lse = attn_paged_fwd(q, P8.typed(k.cuda(), fmt), P8.typed(vc.cuda(), fmt), table, ints([n]), scale, q_ptr=ints([news * i for i in range(copies + 1)]),
                              max_q=news, seqs=ints([0] * copies), out_dtype=torch.float32, k_scales=scales[0], v_scales=scales[1])
    assert attn_last_device_error() == 0
    out, lse = out.double().cpu().numpy().reshape(copies, news, G, d), lse.double().cpu().numpy().reshape(G, copies, news)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    u, h = 2.0 ** -24, 2.0 ** -8
    for t in range(news):
        m = n - news + t + 1
        for g, f in enumerate(FACTORS):
            s = scale * d * f * ks[:m].astype(np.float64)
            top = s.max()
            p = np.exp(s - top)
            L = top + np.log(p.sum())
            p /= p.sum()
            O, A, V = p @ v64[:m], p @ np.abs(v64[:m]), (p[:, None] * np.abs(v64[:m])).max()
            r = (d + 12) * u * top + 2.0 ** -22
            bound = A * (2 * r + (2 * m + 1) * u + 2.0 ** -21 + h) + m * u * V
            assert np.all(np.abs(out[:, t, g] - O) <= bound), (t, g, np.abs((out[:, t, g] - O) / bound).max())
            assert np.all(np.abs(lse[g, :, t] - L) <= r + m * u + 2.0 ** -21 + 2 * u * abs(L))


@pytest.mark.parametrize("fmt", FMTS)
def test_two_passes_that_share_the_sms(fmt):
    """Prefixes of many rows on the tiles and long sequences of a token each behind them on the kernel for few
    rows, side by side: the same bits every time."""
    lens = [(2600 + 91 * i) % 3000 for i in range(24)]
    c = P8.make(fmt, lens, [1] * 24, 64, 32, 8, 128, seed=11, plens=[3000, 900], first=[0, 16, 24], spread=0.3)
    want = prefix(c, max_q=1)
    assert attn_last_device_error() == 0
    P8.check(c, *want, P.reference(c))
    for _ in range(30):
        assert all(torch.equal(x, y) for x, y in zip(prefix(c, max_q=1), want))
