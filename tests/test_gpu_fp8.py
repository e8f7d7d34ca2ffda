"""GPU parity of the 8-bit lm_head (residual_rmsnorm_fp8, lmhead_quantize_fp8,
lmhead_logits_fp8) against the float64 oracle.

Tolerances, all from roundings counted in the kernels' formulas:
* an e4m3 rounding is off by at most 2^-4 of the value, or by half the smallest
  step, 2^-10, below the normal range;
* the norm's factor comes from a sum of d squares in fp32 (relative error at
  most (d + 8) 2^-24), the rest of y and the scale from a few fp32 operations;
* a logit is an fp32 sum of exact products times a product of two scales: at most
  (d + nb + 4) 2^-24 of the sum of its terms' magnitudes; bf16 logits add 2^-8.
"""
import numpy as np
import pytest

from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu
BLOCK = 128


@pytest.fixture(scope="module")
def tcb():
    import trie_constrained_beam_b200 as m
    from trie_constrained_beam_b200 import build
    build.build()
    return m


def _bf16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _codes(t):
    import torch
    return t.detach().view(torch.uint8).cpu().numpy()


def _nb(d):
    return -(-d // BLOCK)


def _norm_out(M, d):
    import torch
    return (torch.full((M, d), 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.empty((M, d), dtype=torch.float8_e4m3fn, device="cuda"),
            torch.full((M, _nb(d)), -1.0, dtype=torch.float32, device="cuda"))


def _check_quantised(y, codes, scale, rows, rel):
    """codes, scale against float64 y whose device counterpart is off by `rel`."""
    ref = ofp8.blocks(y, rows)
    assert np.all(np.abs(scale - ref) <= (rel + 2.0 ** -23) * ref)
    s = ofp8.expand(scale.astype(np.float64), rows, y.shape)
    got = ofp8.e4m3_values()[codes] * s
    err = np.abs(got - y)
    bound = (2.0 ** -4 + 2 * rel + 2.0 ** -20) * np.abs(y) + (2.0 ** -10 * (1 + 1e-6)) * s
    assert np.all(err <= bound), float((err - bound).max())


@pytest.mark.parametrize("M,d", [(1, 16), (1, 2048), (3, 128), (5, 144), (2, 1040), (7, 4096),
                                 (3, 16384), (1184, 64), (1200, 2048), (1190, 1040), (1300, 2064)])
@pytest.mark.parametrize("residual", ["none", "given", "in_place"])
def test_residual_rmsnorm(tcb, M, d, residual):
    import torch
    rng = np.random.default_rng(M * 131 + d)
    x = _bf16(rng.standard_normal((M, d)) * np.exp(rng.uniform(-6, 6, size=(M, 1)))).cuda()
    r = None if residual == "none" else _bf16(3 * rng.standard_normal((M, d))).cuda()
    w = _bf16(1 + 0.3 * rng.standard_normal(d)).cuda()
    h64, y64 = ofp8.residual_rmsnorm(_f64(x), None if r is None else _f64(r), _f64(w), 1e-6)
    ro, q, s = _norm_out(M, d)
    if residual == "in_place":
        ro = r
    tcb.residual_rmsnorm_fp8(x, r, w, 1e-6, ro, q, s)
    assert np.all(np.abs(_f64(ro) - h64) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(h64))
    _check_quantised(y64, _codes(q), _f64(s), 1, (d + 16) * 2.0 ** -24)


def test_rmsnorm_extremes(tcb):
    """Rows of zeros, a row whose blocks differ by 2^60, an output not kept, and
    rows next to one that holds infinities and NaN."""
    import torch
    d = 384
    x = np.ones((5, d), np.float32)
    x[1] = 0
    x[2, :128], x[2, 128:256], x[2, 256:] = 2.0 ** -60, 1, 0
    x[3, 5], x[3, 6] = np.inf, np.nan
    xt = _bf16(x).cuda()
    w = _bf16(np.ones(d)).cuda()
    _, q, s = _norm_out(5, d)
    tcb.residual_rmsnorm_fp8(xt, None, w, 1e-6, None, q, s)
    codes, scale = _codes(q), _f64(s)
    assert np.all(codes[1] == 0) and np.all(scale[1] == 2.0 ** -100)
    assert np.all(codes[2, 256:] == 0) and scale[2, 2] == 2.0 ** -100
    keep = [0, 1, 2, 4]
    _, y = ofp8.residual_rmsnorm(_f64(xt)[keep], None, np.ones(d), 1e-6)
    _check_quantised(y, codes[keep], scale[keep], 1, (d + 16) * 2.0 ** -24)


def test_rmsnorm_no_rows(tcb):
    import torch
    ro, q, s = _norm_out(0, 256)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    tcb.residual_rmsnorm_fp8(x, None, torch.ones(256, dtype=torch.bfloat16, device="cuda"), 1e-6,
                             ro, q, s)


@pytest.mark.parametrize("V,d", [(1, 16), (128, 128), (129, 144), (500, 1040), (257, 2048),
                                 (8192, 256)])
def test_quantize_weight_is_exact(tcb, V, d):
    """Every operation of the weight's quantisation is a single fp32 rounding, so
    scales and codes are equal to the same operations done one by one."""
    import torch
    rng = np.random.default_rng(V + d)
    w = _bf16(0.02 * rng.standard_normal((V, d)) * np.exp(rng.uniform(-3, 3, size=(V, 1))))
    w[V // 2, :] = 0
    wq = torch.empty((V, d), dtype=torch.float8_e4m3fn, device="cuda")
    ws = torch.empty((-(-V // BLOCK), _nb(d)), dtype=torch.float32, device="cuda")
    tcb.lmhead_quantize_fp8(w.cuda(), wq, ws)
    f = w.float().numpy()
    amax = (ofp8.blocks(f.astype(np.float64), BLOCK) * 448.0).astype(np.float32)
    scale = amax / np.float32(448)
    assert np.array_equal(ws.cpu().numpy(), scale)
    inv = np.float32(1) / scale
    y = f * ofp8.expand(inv, BLOCK, f.shape)
    ref = torch.from_numpy(y).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert np.array_equal(_codes(wq), _codes(ref))
    _check_quantised(f.astype(np.float64), _codes(wq), _f64(ws), BLOCK, 2.0 ** -24)


def _operands(M, V, d, seed):
    """Random codes (no NaN) with scales that differ from block to block."""
    import torch
    rng = np.random.default_rng(seed)
    hq = torch.from_numpy((rng.standard_normal((M, d)) * 60).astype(np.float32)) \
        .clamp(-448, 448).to(torch.float8_e4m3fn)
    wq = torch.from_numpy((rng.standard_normal((V, d)) * 60).astype(np.float32)) \
        .clamp(-448, 448).to(torch.float8_e4m3fn)
    hs = np.exp(rng.uniform(-7, -3, size=(M, _nb(d)))).astype(np.float32)
    ws = np.exp(rng.uniform(-12, -8, size=(-(-V // BLOCK), _nb(d)))).astype(np.float32)
    return hq.cuda(), torch.from_numpy(hs).cuda(), wq.cuda(), torch.from_numpy(ws).cuda()


def _logits(tcb, ops, V, dtype, pad=0):
    import torch
    M = ops[0].shape[0]
    ld = -(-V // 8) * 8 + pad
    buf = torch.full((M, ld), float("nan"), dtype=dtype, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    tcb.lmhead_logits_fp8(*ops, buf[:, :V], ws)
    assert tcb.sidbeam_get_device_status(ws) == 0
    assert bool(torch.isnan(buf[:, V:].float()).all())   # columns past V are left alone
    return buf[:, :V]


def _check_logits(got, ops, d, dtype, rows=None, cols=None):
    import torch
    hq, hs, wq, ws = (_codes(ops[0]), ops[1].cpu().numpy(), _codes(ops[2]), ops[3].cpu().numpy())
    g = got.double().cpu().numpy()
    if rows is not None:
        hq, hs, g = hq[rows], hs[rows], g[rows]
    if cols is not None:  # whole blocks of 128 codes
        sel = np.concatenate([np.arange(c * BLOCK, min((c + 1) * BLOCK, wq.shape[0])) for c in cols])
        wq, ws, g = wq[sel], ws[cols], g[:, sel]
    ref, mag = ofp8.lmhead_logits(hq, hs, wq, ws)
    bound = (d + _nb(d) + 4) * 2.0 ** -24 * mag
    if dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(g - ref)
    assert np.all(err <= bound + 1e-30), float((err - bound).max())
    return err, mag


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("V,d", [(8, 16), (128, 128), (130, 144), (1001, 1040)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logits_shapes(tcb, M, V, d, dtype):
    """Every row variant with whole and ragged tiles on each side, a K tail, one
    block of d and several; fp32 and bf16 logits."""
    import torch
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    ops = _operands(M, V, d, M * 7 + V + d)
    _check_logits(_logits(tcb, ops, V, t, pad=8), ops, d, t)


@pytest.mark.parametrize("M,V,d", [(5, 300, 16384), (140, 300, 16384), (4, 32768, 256),
                                   (200, 32768, 256), (100, 300, 8192)])
def test_logits_long_sides(tcb, M, V, d):
    import torch
    ops = _operands(M, V, d, V + d)
    got = _logits(tcb, ops, V, torch.float32)
    cols = [0, (V - 1) // BLOCK] if V > 1000 else None
    _check_logits(got, ops, d, torch.float32, cols=cols)


def test_logits_workload_shape(tcb):
    """4,096 rows x 8,192 codes x d = 2,048 (several tiles per CTA): sampled rows,
    and the same bits from a second call."""
    import torch
    M, V, d = 4096, 8192, 2048
    ops = _operands(M, V, d, 3)
    got = _logits(tcb, ops, V, torch.float32)
    rows = np.r_[0:3, 127:130, 2047, 3000:3003, 4093:4096]
    err, mag = _check_logits(got, ops, d, torch.float32, rows=rows)
    # fp32 accumulation throughout: the typical error is far below the bound.
    assert np.median(err / mag) < 2.0 ** -22
    again = _logits(tcb, ops, V, torch.float32)
    assert torch.equal(got, again)


def test_logits_rows_do_not_depend_on_batch(tcb):
    """Infinite or NaN scales of one row stay in that row."""
    import torch
    ops = list(_operands(40, 256, 256, 9))
    ref = _logits(tcb, ops, 256, torch.float32).clone()
    ops[1] = ops[1].clone()
    ops[1][7, 0], ops[1][20, 1] = float("nan"), float("inf")
    got = _logits(tcb, ops, 256, torch.float32)
    keep = [i for i in range(40) if i not in (7, 20)]
    assert torch.equal(got[keep], ref[keep])
    assert bool(torch.isnan(got[7]).all())


def test_captured_graph_and_side_stream(tcb):
    """Norm and product captured into one graph, replayed on new inputs, and run
    on a stream other than the current one: the same bits as eager calls."""
    import torch
    M, V, d = 96, 700, 512
    rng = np.random.default_rng(4)
    w = _bf16(0.02 * rng.standard_normal((V, d))).cuda()
    g = _bf16(1 + 0.1 * rng.standard_normal(d)).cuda()
    head = tcb.LmheadFp8(w, g, M)
    xs = [_bf16(rng.standard_normal((M, d))).cuda() for _ in range(3)]
    eager = [head.logits(x).clone() for x in xs]
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = head.logits(x)
    for i in (1, 2):
        x.copy_(xs[i])
        graph.replay()
        assert torch.equal(out, eager[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = head.logits(xs[0], stream=side)
    side.synchronize()
    assert torch.equal(out, eager[0])


def test_argument_checks(tcb):
    import torch
    ops = _operands(4, 256, 256, 1)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.empty((4, 256), device="cuda")
    with pytest.raises(ValueError):      # scale of another shape
        tcb.lmhead_logits_fp8(ops[0], ops[1][:, :1], ops[2], ops[3], out, ws)
    with pytest.raises(TypeError):       # logits in fp16
        tcb.lmhead_logits_fp8(*ops, out.half(), ws)
    with pytest.raises(ValueError):      # transposed logits
        tcb.lmhead_logits_fp8(*ops, torch.empty((256, 4), device="cuda").t(), ws)
    with pytest.raises(tcb.SidbeamError) as e:   # rows not 16-byte aligned
        tcb.lmhead_logits_fp8(*ops, torch.empty((4, 258), device="cuda")[:, :256], ws)
    assert e.value.status == -3
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((4, 256), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((4, 2), device="cuda")
    with pytest.raises(TypeError):
        tcb.residual_rmsnorm_fp8(x.float(), None, x[0], 1e-6, None, q, s)
    with pytest.raises(ValueError):
        tcb.residual_rmsnorm_fp8(x.cpu(), None, x[0], 1e-6, None, q, s)
    with pytest.raises(tcb.SidbeamError):
        tcb.residual_rmsnorm_fp8(x, None, x[0], -1.0, None, q, s)


def test_head_made_on_a_side_stream(tcb):
    """A head made on a side stream while the current one is busy: weight, scales and
    status word are that stream's, none of them behind the current stream's work."""
    import torch
    V, d = 700, 512
    rng = np.random.default_rng(12)
    w = _bf16(0.02 * rng.standard_normal((V, d))).cuda()
    g = _bf16(1 + 0.1 * rng.standard_normal(d)).cuda()
    x = _bf16(rng.standard_normal((5, d))).cuda()
    want = tcb.LmheadFp8(w, g, 5)
    ref = want.logits(x).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device="cuda")
    junk = torch.full((64, 256), 255, dtype=torch.uint8, device="cuda")
    del junk                                  # freed, on the current stream
    for _ in range(20):
        busy = busy @ busy * 1e-4
    head = tcb.LmheadFp8(w, g, 5, stream=side)
    out = head.logits(x, stream=side)
    side.synchronize()
    assert tcb.sidbeam_get_device_status(head.workspace, stream=side) == 0
    assert np.array_equal(_codes(head.w_q), _codes(want.w_q))
    assert torch.equal(head.w_scale, want.w_scale) and torch.equal(out, ref)


@pytest.mark.parametrize("d", [272, 512, 528, 1024, 4112, 8192, 8208, 16368])
def test_residual_rmsnorm_row_shapes(tcb, d):
    """Hidden sizes at both ends of every count of threads and chunks a row."""
    rng = np.random.default_rng(d)
    M = 9
    x, r = _bf16(rng.standard_normal((M, d))).cuda(), _bf16(2 * rng.standard_normal((M, d))).cuda()
    w = _bf16(1 + 0.3 * rng.standard_normal(d)).cuda()
    h64, y64 = ofp8.residual_rmsnorm(_f64(x), _f64(r), _f64(w), 1e-6)
    ro, q, s = _norm_out(M, d)
    tcb.residual_rmsnorm_fp8(x, r, w, 1e-6, ro, q, s)
    assert np.all(np.abs(_f64(ro) - h64) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(h64))
    _check_quantised(y64, _codes(q), _f64(s), 1, (d + 16) * 2.0 ** -24)


@pytest.mark.parametrize("M,V,d", [(1300, 2050, 1040), (1300, 2177, 1040), (1281, 2303, 144),
                                   (9473, 255, 64), (1152, 2304, 16)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logits_wide_tiles_with_ragged_sides(tcb, M, V, d, dtype):
    """Tiles of 256 codes, both output types: a codebook that ends in a tile's first or
    second half (the other half has no column), rows and d that end inside a tile."""
    import torch
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    ops = _operands(M, V, d, M + V)
    got = _logits(tcb, ops, V, t, pad=8)
    _check_logits(got, ops, d, t)
    assert torch.equal(got, _logits(tcb, ops, V, t, pad=8))


@pytest.mark.parametrize("M,V,d", [(5, 256, 256), (20, 700, 2048), (16, 4096, 8192), (1300, 2050, 272)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logits_rows_are_isolated_in_every_kernel(tcb, M, V, d, dtype):
    """Infinite or NaN scales of a row stay in that row: few rows (their factors share a
    table, their parts meet across a cluster) and wide tiles."""
    import torch
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    ops = list(_operands(M, V, d, 9 + M))
    ref = _logits(tcb, ops, V, t).clone()
    assert bool(torch.isfinite(ref).all())
    ops[1] = ops[1].clone()
    ops[1][2, 0], ops[1][M - 1, 1] = float("nan"), float("inf")
    got = _logits(tcb, ops, V, t)
    keep = [i for i in range(M) if i not in (2, M - 1)]
    assert torch.equal(got[keep], ref[keep])
    assert bool(torch.isnan(got[2]).all()) and not bool(torch.isfinite(got[M - 1]).any())


def test_rmsnorm_in_place_of_x(tcb):
    """residual_out in x's place, and x as its own residual."""
    import torch
    rng = np.random.default_rng(8)
    x = _bf16(rng.standard_normal((6, 1040))).cuda()
    w = _bf16(1 + 0.3 * rng.standard_normal(1040)).cuda()
    h64, y64 = ofp8.residual_rmsnorm(_f64(x), _f64(x), _f64(w), 1e-6)
    _, q, s = _norm_out(6, 1040)
    tcb.residual_rmsnorm_fp8(x, x, w, 1e-6, x, q, s)
    assert np.array_equal(_f64(x), h64)                # twice a bf16 value: exact
    _check_quantised(y64, _codes(q), _f64(s), 1, (1040 + 16) * 2.0 ** -24)
