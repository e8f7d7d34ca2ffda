"""GPU parity of beam_attention against the float64 oracle.

Tolerance of an output element, from the roundings of the formula: the weights
are rounded to bf16 (2^-8 of each, so at most 2^-8 of the weighted mean of |v|),
a score is an fp32 sum of D products (off by at most (D + 4) 2^-24 of the sum of
their magnitudes; an error e of the scores moves a weight by a factor within
1 +- 2e of its share), 2^x, sums and the accumulation of the output stay in fp32
(together below 2^-16 of the weighted mean of |v|), and the result is rounded to
bf16 once (2^-8).
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tcb():
    import trie_constrained_beam_b200 as m
    from trie_constrained_beam_b200 import build
    build.build()
    return m


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _history(rng, level, R, B, dead=0.0):
    """Back-pointers as the steps write them; a share of dead slots."""
    bp = rng.integers(0, B, size=(max(level, 1), R, B)).astype(np.int32)
    bp[0] = 0
    if dead:
        bp[rng.random(bp.shape) < dead] = -1
    return bp


class Case:
    """Inputs of one call on the device and, for the oracle, on the host."""

    def __init__(self, R, B, H, Hkv, D, lens, level=0, page=0, seed=0, dead=0.0, sigma=1.5,
                 junk=True):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)

        def normal(*shape, s=1.0):
            return (s * torch.randn(shape, device="cuda", generator=g)).to(torch.bfloat16)
        self.R, self.B, self.H, self.Hkv, self.D, self.level = R, B, H, Hkv, D, level
        self.lens = [int(x) for x in lens]
        self.q = normal(R * B, H, D, s=sigma)
        self.cache_len = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        cap = max(max(self.lens), 1)
        nan = float("nan")
        self.table = None
        if page:
            per = -(-cap // page) + 1
            pages = R * per + 2
            order = rng.permutation(pages)[:R * per].reshape(R, per)
            self.k, self.v = normal(pages, page, Hkv, D), normal(pages, page, Hkv, D)
            table = order.copy()
            self.prompts = []
            for r, n in enumerate(self.lens):
                used = -(-n // page)
                idx = torch.from_numpy(order[r, :max(used, 1)].copy()).cuda()
                kk = self.k[idx].reshape(-1, Hkv, D)[:n]
                vv = self.v[idx].reshape(-1, Hkv, D)[:n]
                self.prompts.append((_f64(kk), _f64(vv)))
                table[r, used:] = -7          # never read
                if junk and n % page:         # rows past the end of the last page
                    self.k[order[r, used - 1], n % page:] = nan
                    self.v[order[r, used - 1], n % page:] = nan
            self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        else:
            self.k, self.v = normal(R, cap + 5, Hkv, D), normal(R, cap + 5, Hkv, D)
            self.prompts = []
            for r, n in enumerate(self.lens):
                self.prompts.append((_f64(self.k[r, :n]), _f64(self.v[r, :n])))
                if junk:
                    self.k[r, n:] = nan
                    self.v[r, n:] = float("inf")
        self.kb = normal(max(level, 1), R * B, Hkv, D)
        self.vb = normal(max(level, 1), R * B, Hkv, D)
        self.bp = _history(rng, level, R, B, dead)
        self.out = torch.full((R * B, H, D), 99.0, dtype=torch.bfloat16, device="cuda")
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def kwargs(self):
        import torch
        kw = dict(page_table=self.table, level=self.level)
        if self.level:
            kw.update(k_beam=self.kb, v_beam=self.vb, bp_parent=torch.from_numpy(self.bp).cuda())
        return kw

    def run(self, tcb, **more):
        tcb.beam_attention(self.q, self.k, self.v, self.cache_len, self.out, self.ws,
                           **{**self.kwargs(), **more})
        assert tcb.sidbeam_get_device_status(self.ws) == 0
        return self.out

    def check(self, out=None, scale=None, rows=slice(None)):
        ref, mean, terms = oracle.beam_attention(
            _f64(self.q), self.prompts, self.level, _f64(self.kb), _f64(self.vb), self.bp, scale)
        e = (self.D + 4) * 2.0 ** -24 * terms[:, :, None]
        tol = 2.0 ** -8 * np.abs(ref) + mean * (2.0 ** -8 + 2 * e + 2.0 ** -16) * (1 + 2.0 ** -7)
        err, tol = np.abs(_f64(self.out if out is None else out) - ref)[rows], tol[rows]
        assert np.all(err <= tol), (float((err - tol).max()), np.argwhere(err > tol)[:5].tolist())


HEADS = [(1, 1, 64), (2, 1, 128), (6, 2, 64), (8, 8, 128), (16, 2, 128), (5, 1, 128)]


@pytest.mark.parametrize("H,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [0, 16, 64, 128, 256])
def test_single_rows(tcb, H, Hkv, D, page):
    """The first step: one row per request, lengths around every tile and page
    edge, none and one token among them."""
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385, 700]
    c = Case(len(lens), 1, H, Hkv, D, lens, page=page, seed=H * 100 + D + page)
    c.run(tcb)
    c.check()
    assert not c.out[0].any()   # nothing to attend


@pytest.mark.parametrize("B", [2, 16, 33, 64, 65, 130, 200])
@pytest.mark.parametrize("H,Hkv,D", [(2, 1, 64), (4, 2, 128), (3, 1, 128)])
def test_beams(tcb, B, H, Hkv, D):
    """Beams with ancestors, one to three tiles of rows, ragged prompts."""
    c = Case(3, B, H, Hkv, D, [200, 0, 129], level=3, page=16, seed=B)
    c.run(tcb)
    c.check()


@pytest.mark.parametrize("level", [1, 2, 7, 16])
@pytest.mark.parametrize("lens", [[0, 0], [1, 130], [300, 5]])
def test_levels_and_dead_beams(tcb, level, lens):
    c = Case(2, 20, 4, 2, 64, lens, level=level, seed=level, dead=0.05)
    c.run(tcb)
    c.check()
    dead = [r * 20 + b for r in range(2) for b in range(20)
            if oracle.attention.ancestors(c.bp, level, r, b) is None]
    assert dead and not c.out[dead].any()


def test_bad_links_are_dead(tcb):
    """Links past the beam, at any level, give zero rows, and nothing is read."""
    c = Case(1, 8, 2, 1, 64, [40], level=3, seed=5)
    c.bp[2, 0, 3] = 8
    c.bp[1, 0, 4] = 1 << 30
    c.bp[0, 0, 5] = -1
    c.run(tcb)
    c.check()
    assert not c.out[3].any()


@pytest.mark.parametrize("R,B,S", [(1, 1, 6000), (2, 1, 20001), (1, 40, 3000), (1, 512, 700)])
def test_long_prompts_few_rows(tcb, R, B, S):
    """Few work items: the prompt is split over CTAs and the parts are joined.
    (One head pair; the largest case is checked on sampled rows.)"""
    c = Case(R, B, 2, 1, 128, [S - 3 * r for r in range(R)], level=2 if B > 1 else 0, seed=S)
    c.run(tcb)
    c.check()
    first = c.out.clone()
    c.run(tcb)
    import torch
    assert torch.equal(first, c.out)   # joined in a fixed order


@pytest.mark.parametrize("S", [256, 257, 384, 512, 900, 1024])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_split_over_few_tiles(tcb, S, D, page):
    """Two to eight key tiles over up to eight CTAs, some of which have none: the
    requests' own lengths are shorter than the capacity that the split goes by."""
    c = Case(4, 3, 2, 1, D, [S, 1, 130, 0], level=1, page=page, seed=S + D)
    c.run(tcb)
    c.check()


@pytest.mark.parametrize("R,B,H,Hkv,D,level,page", [(250, 1, 4, 2, 128, 0, 16), (330, 2, 1, 1, 64, 1, 0),
                                                    (80, 66, 4, 2, 64, 2, 0), (76, 67, 4, 2, 128, 1, 64)])
def test_many_units(tcb, R, B, H, Hkv, D, level, page):
    """More work items than SMs: every CTA runs several in a row, of all lengths
    (none, one tile, odd and even tiles, ragged or not), in both row shapes."""
    rng = np.random.default_rng(R)
    lens = rng.choice([0, 1, 64, 100, 128, 129, 200, 256, 300, 384, 500], size=R)
    c = Case(R, B, H, Hkv, D, lens, level=level, page=page, seed=R)
    first = c.run(tcb).clone()
    c.check()
    c.run(tcb)
    import torch
    assert torch.equal(first, c.out)


def test_group_of_128_heads(tcb):
    c = Case(2, 3, 128, 1, 64, [77, 300], level=1, seed=8)
    c.run(tcb)
    c.check()


def test_extreme_scores(tcb):
    """Scores far apart (one key takes all the weight, maxima that grow from tile
    to tile) and a negative scale."""
    import torch
    c = Case(2, 3, 2, 1, 64, [500, 390], level=2, seed=3, sigma=20.0)
    ramp = torch.linspace(0.05, 6, c.k.shape[1], device="cuda")[None, :, None, None]
    c.k = torch.where(torch.isnan(c.k), c.k, (c.k * ramp).to(torch.bfloat16))
    c.prompts = [(_f64(c.k[r, :n]), _f64(c.v[r, :n])) for r, n in enumerate(c.lens)]
    c.run(tcb)
    c.check()
    c.run(tcb, scale=-0.3)
    c.check(scale=-0.3)


@pytest.mark.parametrize("B,H,Hkv,D", [(40, 4, 2, 64), (70, 2, 1, 128)])
def test_non_finite_values_stay_where_they_belong(tcb, B, H, Hkv, D):
    """NaN and infinity in a beam's query reach that row alone; in a beam's keys or
    values, its descendants alone; whatever a dead beam holds reaches nobody."""
    import torch
    c = Case(2, B, H, Hkv, D, [150, 0], level=3, seed=B)
    c.bp[2, 0, 5], c.bp[1, 1, 7] = -1, -1      # dead beams
    ref = c.run(tcb).clone()
    assert bool(torch.isfinite(ref.float()).all())
    paths = [[oracle.attention.ancestors(c.bp, 3, r, b) for b in range(B)] for r in range(2)]
    # A dead beam's own token (slot 5 of the last level) and query.
    c.kb[2, 5], c.vb[2, 5] = float("nan"), float("inf")
    c.q[5] = float("nan")
    assert torch.equal(c.run(tcb), ref)
    # Live tokens: values of (level 2, slot 9), keys of (level 1, slot s) of request 0.
    s = paths[0][20][1][1]
    c.vb[2, 9, :, 3] = float("inf")
    c.kb[1, s] = float("nan")
    c.q[B + 11] = float("nan")                  # request 1, beam 11
    got = c.run(tcb)
    hit = {(0, 9), (1, 11)} | {(0, b) for b in range(B)
                               if paths[0][b] is not None and (1, s) in paths[0][b]}
    hit = {(r, b) for r, b in hit if paths[r][b] is not None}
    for r in range(2):
        for b in range(B):
            row = got[r * B + b].float()
            if (r, b) in hit:
                assert not bool(torch.isfinite(row).all()), (r, b)
            else:  # (a neighbour of an infinity is summed in another order)
                assert bool(torch.isfinite(row).all()), (r, b)
    with np.errstate(invalid="ignore"):
        c.check(rows=[r * B + b for r in range(2) for b in range(B) if (r, b) not in hit])
    assert bool(torch.isnan(got[20].float()).all())


def test_strided_query_cache_and_output(tcb):
    """q a slice of a fused projection, k and v interleaved in one cache array,
    out a slice of a wider buffer whose other columns stay."""
    import torch
    R, B, H, Hkv, D = 2, 5, 4, 2, 64
    c = Case(R, B, H, Hkv, D, [70, 33], level=0, seed=11, junk=False)
    wide = torch.zeros((R * B, H * D + 96), dtype=torch.bfloat16, device="cuda")
    wide[:, 32:32 + H * D] = c.q.view(R * B, H * D)
    c.q = wide[:, 32:32 + H * D].unflatten(1, (H, D))
    kv = torch.stack([c.k, c.v], dim=2)          # [R, cap, 2, Hkv, D]
    c.k, c.v = kv[:, :, 0], kv[:, :, 1]
    buf = torch.full((R * B, H * D + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    c.out = buf[:, :H * D].unflatten(1, (H, D))
    c.run(tcb)
    c.check()
    assert bool((buf[:, H * D:] == 5).all())


def test_offsets_past_32_bits(tcb):
    """A slab of 2^32 + elements: the last request's rows lie past 32-bit
    element offsets."""
    import torch
    R, cap, Hkv, D = 3, 1100, 8, 128
    big = (1 << 31) + 8 * 1024              # elements between two requests
    need = big * (R - 1) + cap * Hkv * D
    flat = torch.zeros(need, dtype=torch.bfloat16, device="cuda")
    k = torch.as_strided(flat, (R, cap, Hkv, D), (big, Hkv * D, D, 1))
    c = Case(R, 2, 8, 8, 128, [900, 64, 1001], level=0, seed=2, junk=False)
    for r in range(R):
        k[r, :c.lens[r]] = c.k[r, :c.lens[r]]
    c.prompts = [(kk, kk) for kk, _ in c.prompts]
    c.k, c.v = k, k
    c.run(tcb)
    c.check()


def test_bad_pages_and_lengths_set_status(tcb):
    """A page number outside the cache reads as zeros; a length outside the
    capacity is clamped; both set the status word and leave the others alone."""
    import torch
    c = Case(2, 1, 2, 1, 64, [100, 90], page=16, seed=6)
    good = c.run(tcb).clone()
    table = c.table.clone()
    table[0, 3] = 10 ** 6
    tcb.beam_attention(c.q, c.k, c.v, c.cache_len, c.out, c.ws, page_table=table)
    with pytest.raises(AssertionError):
        assert tcb.sidbeam_get_device_status(c.ws) == 0
    assert torch.equal(c.out[1], good[1]) and bool(torch.isfinite(c.out.float()).all())
    k0, v0 = c.prompts[0]
    k0, v0 = k0.copy(), v0.copy()
    k0[48:64], v0[48:64] = 0, 0
    c.prompts[0] = (k0, v0)
    c.check()
    lens = torch.tensor([-5, 90], dtype=torch.int32, device="cuda")
    tcb.beam_attention(c.q, c.k, c.v, lens, c.out, c.ws, page_table=c.table)
    assert tcb.sidbeam_get_device_status(c.ws) == -7
    assert not c.out[0].any() and torch.equal(c.out[1], good[1])


def test_captured_graph_side_stream_and_two_at_once(tcb):
    """One captured graph replayed on new inputs, and two calls of different
    shapes in flight on two streams with the same status workspace."""
    import torch
    a = Case(2, 24, 4, 2, 64, [300, 170], level=2, seed=1)
    b = Case(1, 1, 8, 8, 128, [2500], seed=2)
    ra, rb = a.run(tcb).clone(), b.run(tcb).clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ka, kb = a.kwargs(), b.kwargs()
    torch.cuda.synchronize()
    for _ in range(5):
        a.out.zero_()
        b.out.zero_()
        torch.cuda.synchronize()
        tcb.beam_attention(a.q, a.k, a.v, a.cache_len, a.out, a.ws, stream=s1, **ka)
        tcb.beam_attention(b.q, b.k, b.v, b.cache_len, b.out, a.ws, stream=s2, **kb)
        torch.cuda.synchronize()
        assert torch.equal(a.out, ra) and torch.equal(b.out, rb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tcb.beam_attention(a.q, a.k, a.v, a.cache_len, a.out, a.ws, **ka)
    q2 = torch.flip(a.q, [0])
    a.q.copy_(q2)
    a.cache_len.copy_(torch.tensor([17, 299], dtype=torch.int32))
    a.prompts = [(_f64(a.k[0, :17]), _f64(a.v[0, :17])), None]
    a.k[1, 170:299], a.v[1, 170:299] = 0.25, -1.0
    a.prompts[1] = (_f64(a.k[1, :299]), _f64(a.v[1, :299]))
    g.replay()
    torch.cuda.synchronize()
    a.check()


def test_argument_checks(tcb):
    import torch
    c = Case(2, 4, 4, 2, 64, [30, 20], level=2, seed=1)
    kw = c.kwargs()

    def call(q=c.q, k=c.k, v=c.v, n=c.cache_len, out=c.out, ws=c.ws, **more):
        tcb.beam_attention(q, k, v, n, out, ws, **{**kw, **more})
    with pytest.raises(TypeError):
        call(q=c.q.float())
    with pytest.raises(TypeError):
        call(n=c.cache_len.long())
    with pytest.raises(ValueError):
        call(v=c.v[:, :-1])
    with pytest.raises(ValueError):
        call(level=3)
    with pytest.raises(ValueError):
        call(k_beam=None)
    with pytest.raises(ValueError):
        call(q=c.q[:7], out=c.out[:7])
    with pytest.raises(ValueError):
        call(q=c.q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(tcb.SidbeamError) as e:
        call(scale=float("inf"))
    assert e.value.status == -1
    with pytest.raises(tcb.SidbeamError):
        call(ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tcb.SidbeamError):      # pages of 24 tokens
        p = torch.zeros((4, 24, 2, 64), dtype=torch.bfloat16, device="cuda")
        call(k=p, v=p, page_table=torch.zeros((2, 2), dtype=torch.int32, device="cuda"))
