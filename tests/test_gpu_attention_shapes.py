"""beam_attention in the kernel shapes that the cases of test_gpu_attention.py do not
reach: two row tiles a unit without ancestors, units of two tiles and of one in turn
on a CTA, deep paths with more than one tile of rows, wide beams, and calls that the
header allows. The same oracle and tolerance."""
import numpy as np
import pytest

import oracle
from test_gpu_attention import Case, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tcb():
    import trie_constrained_beam_b200 as m
    from trie_constrained_beam_b200 import build
    build.build()
    return m


def _twice(tcb, c, **check):
    import torch
    first = c.run(tcb).clone()
    c.check(**check)
    assert torch.equal(first, c.run(tcb))


LENGTHS = [0, 1, 64, 100, 128, 129, 200, 256, 257, 300, 384, 500, 0, 1, 700]


@pytest.mark.parametrize("R,B,S,level", [(1, 200, 900, 0), (2, 130, 2500, 0), (3, 300, 257, 0),
                                         (1, 140, 1200, 3), (2, 300, 640, 8)])
@pytest.mark.parametrize("D,page", [(64, 0), (64, 16), (128, 64), (128, 0)])
def test_two_tiles_few_units(tcb, R, B, S, level, D, page):
    """More than 128 rows a key head and few units: the keys are split over clusters,
    with and without ancestors, whole and ragged second tiles."""
    c = Case(R, B, 2, 1, D, [max(S - 131 * r, 0) for r in range(R)], level=level, page=page,
             seed=S + D)
    _twice(tcb, c)


@pytest.mark.parametrize("R,B,H,Hkv,D,page", [(150, 140, 1, 1, 64, 0), (76, 67, 4, 2, 128, 16),
                                              (30, 256, 6, 6, 64, 64)])
def test_two_tiles_many_units_first_step(tcb, R, B, H, Hkv, D, page):
    """The same without ancestors, in persistent CTAs over ragged prompts of all lengths."""
    rng = np.random.default_rng(B)
    c = Case(R, B, H, Hkv, D, rng.choice(LENGTHS, size=R), page=page, seed=R)
    _twice(tcb, c)


@pytest.mark.parametrize("R,B,Hkv,level", [(75, 140, 1, 0), (75, 140, 1, 2), (151, 130, 1, 1),
                                           (151, 130, 1, 0), (67, 280, 1, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_units_of_two_tiles_and_of_one_in_turn(tcb, R, B, Hkv, level, D):
    """Units (256 and 24, 256 and 4, or 256, 256 and 48 rows of a request) whose number
    a CTA's stride does not share a factor with: on 148 SMs each CTA sees units of two
    row tiles before and behind units of one, with prompts of no, one and more tiles."""
    rng = np.random.default_rng(R + level)
    c = Case(R, B, 2 * Hkv, Hkv, D, rng.choice(LENGTHS, size=R), level=level, page=16,
             seed=R + level + D, dead=0.02)
    if B == 280:        # 3 units a request
        c = Case(R, B, 2, 1, D, rng.choice(LENGTHS, size=R), level=level, seed=R, dead=0.02)
    _twice(tcb, c)


@pytest.mark.parametrize("level", [9, 16])
@pytest.mark.parametrize("B,H,Hkv", [(65, 2, 1), (134, 3, 1), (200, 4, 2), (400, 1, 1)])
@pytest.mark.parametrize("D,lens", [(64, [70, 300]), (128, [0, 1000])])
def test_deep_paths_of_many_rows(tcb, level, B, H, Hkv, D, lens):
    """More than 8 levels with more than 128 rows a key head: one tile a unit, several
    tiles a request, beams whose heads lie in two tiles."""
    c = Case(2, B, H, Hkv, D, lens, level=level, seed=B + level, dead=0.005)
    _twice(tcb, c)


@pytest.mark.parametrize("B,H,Hkv,D,level", [(513, 2, 1, 64, 2), (1000, 2, 2, 128, 1),
                                             (4096, 1, 1, 64, 5), (2047, 2, 1, 128, 0),
                                             (1500, 1, 1, 64, 12)])
def test_wide_beams(tcb, B, H, Hkv, D, level):
    c = Case(2, B, H, Hkv, D, [150, 37], level=level, page=16, seed=B, dead=0.01)
    _twice(tcb, c)


@pytest.mark.parametrize("R,B,level", [(75, 140, 2), (2, 140, 0), (2, 200, 12)])
@pytest.mark.parametrize("scale", [-0.3, 0.0, -2.0 ** -10])
def test_scales(tcb, R, B, level, scale):
    """A negative scale flips the signs of q in place; zero weighs all tokens alike."""
    rng = np.random.default_rng(R)
    c = Case(R, B, 2, 1, 64, rng.choice(LENGTHS, size=R), level=level, seed=B, dead=0.01)
    c.run(tcb, scale=scale)
    c.check(scale=scale)


@pytest.mark.parametrize("level", [0, 2])
def test_scores_that_grow_along_the_prompt(tcb, level):
    """Two tiles of rows, several units a CTA: maxima that rise from tile to tile (and
    inside a tile by more than its second half's margin)."""
    import torch
    R, B = 75, 140
    rng = np.random.default_rng(level)
    c = Case(R, B, 2, 1, 64, rng.choice([129, 300, 500, 700], size=R), level=level, seed=9, sigma=20.0)
    ramp = torch.linspace(0.05, 6, c.k.shape[1], device="cuda")[None, :, None, None]
    c.k = torch.where(torch.isnan(c.k), c.k, (c.k * ramp).to(torch.bfloat16))
    c.prompts = [(_f64(c.k[r, :n]), _f64(c.v[r, :n])) for r, n in enumerate(c.lens)]
    _twice(tcb, c)


@pytest.mark.parametrize("R,B,H,Hkv,D,level", [(75, 140, 2, 1, 64, 3), (2, 70, 2, 1, 128, 10)])
def test_non_finite_values_stay_in_their_rows(tcb, R, B, H, Hkv, D, level):
    """As the test of one unit a CTA, with two tiles a unit and several units a CTA, and
    with paths of more than 8 levels: a NaN query reaches its row alone, NaN keys and
    infinite values a beam's descendants alone, a dead beam's nobody."""
    import torch
    rng = np.random.default_rng(R)
    c = Case(R, B, H, Hkv, D, rng.choice(LENGTHS, size=R), level=level, seed=B)
    last, r = level - 1, R - 1
    c.bp[last, 0, 5], c.bp[1, 1, 7] = -1, -1
    ref = c.run(tcb).clone()
    assert bool(torch.isfinite(ref.float()).all())
    paths = [[oracle.attention.ancestors(c.bp, level, i, b) for b in range(B)] for i in range(R)]
    c.kb[last, 5], c.vb[last, 5], c.q[5] = float("nan"), float("inf"), float("nan")
    assert torch.equal(c.run(tcb), ref)
    alive = [b for b in range(B) if paths[r][b] is not None]
    slot = paths[r][alive[-1]][1][1]              # level - 2, the last request
    c.vb[last, r * B + alive[3], :, 3] = float("inf")
    c.kb[last - 1, r * B + slot] = float("nan")
    c.q[B + 11] = float("nan")
    got = c.run(tcb).float()
    hit = {(1, 11), (r, alive[3])} | {(r, b) for b in alive if (last - 1, slot) in paths[r][b]}
    hit = {(i, b) for i, b in hit if paths[i][b] is not None}
    finite = torch.isfinite(got).all(dim=2).all(dim=1).tolist()
    assert finite == [(i // B, i % B) not in hit for i in range(R * B)]
    with np.errstate(invalid="ignore"):
        c.check(rows=[i for i in range(R * B) if (i // B, i % B) not in hit])


def test_shared_pages(tcb):
    """Requests whose tables name the same pages (a common prefix), one of them twice."""
    import torch
    c = Case(3, 4, 4, 2, 64, [100, 80, 64], level=1, page=16, seed=4, junk=False)
    table = c.table.clone()
    table[1, :4] = table[0, :4]
    table[2, :4] = table[0, 0]
    c.table = table
    flat = [c.k[table[r, :8].clamp_min(0).long()].reshape(-1, 2, 64) for r in range(3)]
    flat_v = [c.v[table[r, :8].clamp_min(0).long()].reshape(-1, 2, 64) for r in range(3)]
    c.prompts = [(_f64(k[:n]), _f64(v[:n])) for k, v, n in zip(flat, flat_v, c.lens)]
    _twice(tcb, c)
    assert torch.equal(c.table, table)


@pytest.mark.parametrize("cap,lens", [(1, [1, 0, 1]), (2, [2, 1, 0])])
def test_slabs_of_one_and_two_tokens(tcb, cap, lens):
    c = Case(3, 3, 2, 1, 64, lens, level=2, seed=cap)
    c.k, c.v = c.k[:, :cap].contiguous(), c.v[:, :cap].contiguous()
    _twice(tcb, c)


def test_large_pages_and_padded_tables(tcb):
    """Pages larger than every prompt, and table columns past the last page."""
    c = Case(2, 130, 2, 1, 64, [513, 1], level=1, page=4096, seed=6)
    _twice(tcb, c)


def test_two_graphs_share_a_workspace(tcb):
    """Two captured calls of different shapes with one status workspace, replayed on two
    streams at once, then each alone."""
    import torch
    a = Case(2, 140, 2, 1, 64, [300, 170], level=2, seed=1)
    b = Case(1, 1, 8, 8, 128, [2500], seed=2)
    ra, rb = a.run(tcb).clone(), b.run(tcb).clone()
    ka, kb = a.kwargs(), b.kwargs()
    graphs = []
    for c, kw in ((a, ka), (b, kb)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tcb.beam_attention(c.q, c.k, c.v, c.cache_len, c.out, a.ws, **kw)
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.out.fill_(7.0)
        b.out.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, ra) and torch.equal(b.out, rb)
    assert tcb.sidbeam_get_device_status(a.ws) == 0


@pytest.mark.parametrize("H,Hkv,D", [(1, 1, 64), (16, 8, 128), (128, 1, 64)])
@pytest.mark.parametrize("level", [1, 5, 16])
def test_greedy_paths(tcb, H, Hkv, D, level):
    """One beam a request: every level has one slot; a dead request among them."""
    c = Case(6, 1, H, Hkv, D, [130, 0, 1, 300, 64, 17], level=level, seed=level + H)
    c.bp[level - 1, 4, 0] = -1
    _twice(tcb, c)
    assert not c.out[4].any()


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("B", [1, 140])
def test_lengths_past_the_capacity_are_clamped(tcb, page, B):
    import torch
    c = Case(2, B, 2, 1, 64, [80, 64], page=page, seed=7, junk=False)
    if page:
        c.table = c.table[:, :5].contiguous()          # 80 tokens
    else:
        c.k, c.v = c.k[:, :80].contiguous(), c.v[:, :80].contiguous()
    good = c.run(tcb).clone()
    for n in (81, 1 << 30, 2 ** 31 - 1):
        lens = torch.tensor([n, 64], dtype=torch.int32, device="cuda")
        tcb.beam_attention(c.q, c.k, c.v, lens, c.out, c.ws, **c.kwargs())
        assert tcb.sidbeam_get_device_status(c.ws) == tcb.native.SIDBEAM_ERR_DEVICE_CHECK
        assert torch.equal(c.out, good)
