"""The operators of a decode step run together, as a serving loop would: attention
of the step's rows over the prompt and their ancestors, a residual RMS norm to 8
bits, the 8-bit lm_head, and the constrained step whose back-pointers the next
attention follows. Each stage is compared with the oracle on its own inputs."""
import numpy as np
import pytest

import oracle
from oracle import fp8 as ofp8
from sidgen import host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tcb():
    import trie_constrained_beam_b200 as m
    from trie_constrained_beam_b200 import build
    build.build()
    return m


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _search(tcb, dtype, captured):
    import torch
    from parity import TOL, compare_step
    R, n, depth, V, H, Hkv, D, page = 3, 24, 3, 200, 4, 2, 64, 16
    d = H * D
    lens = [150, 33, 64]
    cat = host.draw_catalog(77, 4000, [V] * depth)
    to = oracle.OracleTrie(cat, [V] * depth)
    trie = tcb.sid_trie_build(cat, [V] * depth)
    g = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape, s=1.0):
        return (s * torch.randn(shape, device="cuda", generator=g)).to(torch.bfloat16)
    search = tcb.BeamSearch(trie, R, n, V, depth=depth)
    w = normal(V, d, s=0.2)
    norm_w = (1 + normal(d, s=0.1).float()).to(torch.bfloat16)
    head = tcb.LmheadFp8(w, norm_w, R * n, dtype=dtype)
    kc, vc = normal(R * 10, page, Hkv, D), normal(R * 10, page, Hkv, D)
    table = torch.randperm(R * 10, device="cuda", generator=g).view(R, 10).to(torch.int32)
    cache_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    embed = normal(V, H, D, s=1.5)             # stands for the model's projections
    kv_embed = normal(2, V, Hkv, D)
    k_beam = torch.zeros((depth, R * n, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v_beam = torch.zeros_like(k_beam)
    start = normal(R, H, D, s=1.5)
    rows = [search.rows(t) for t in range(depth)]
    q = [torch.empty((m, H, D), dtype=torch.bfloat16, device="cuda") for m in rows]
    attn = [torch.empty_like(x) for x in q]
    resid = [torch.empty((m, d), dtype=torch.bfloat16, device="cuda") for m in rows]
    logits = [torch.empty((m, V), dtype=dtype, device="cuda") for m in rows]

    def decode():
        for t in range(depth):
            if t == 0:
                q[0].copy_(start)
            else:   # the chosen tokens' queries, keys and values (padding reads code 0)
                code = search.bp_code[t - 1].reshape(-1).clamp_min(0).long()
                q[t].copy_(embed[code])
                k_beam[t - 1].copy_(kv_embed[0][code])
                v_beam[t - 1].copy_(kv_embed[1][code])
            search.attention(t, q[t], kc, vc, cache_len, attn[t], k_beam=k_beam, v_beam=v_beam,
                             page_table=table)
            x = attn[t].view(rows[t], d)
            search.step_hidden(t, head, x, residual=q[t].view(rows[t], d), residual_out=resid[t])
            logits[t].copy_(head._logits[:rows[t], :V])
        return search.finalize()

    sids, leaf, scores = decode()
    if captured:
        torch.cuda.synchronize()
        eager = [x.clone() for x in (sids, leaf, scores)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            decode()
        start.copy_(torch.flip(start, [1]))
        graph.replay()
        start.copy_(torch.flip(start, [1]))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (sids, leaf, scores)):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    assert tcb.sidbeam_get_device_status(search.workspace) == 0
    assert tcb.sidbeam_get_device_status(head.workspace) == 0
    # ---- every stage against the oracle on that stage's inputs
    bp = search.bp_parent.cpu().numpy()
    tab = table.cpu().numpy()
    prompts = [tuple(_f64(c[torch.from_numpy(tab[r].astype(np.int64)).cuda()]).reshape(-1, Hkv, D)[:lens[r]]
                     for c in (kc, vc)) for r in range(R)]
    hq, ws = head.w_q.view(torch.uint8).cpu().numpy(), head.w_scale.cpu().numpy()
    w8 = ofp8.e4m3_values()[hq] * ofp8.expand(ws.astype(np.float64), 128, hq.shape)
    for t in range(depth):
        ref, mean, terms = oracle.beam_attention(_f64(q[t]), prompts, t, _f64(k_beam), _f64(v_beam),
                                                 bp)
        tol = 2.0 ** -8 * np.abs(ref) + mean * (2.0 ** -8 + 2 * (D + 4) * 2.0 ** -24 *
                                                terms[:, :, None] + 2.0 ** -16) * (1 + 2.0 ** -7)
        assert np.all(np.abs(_f64(attn[t]) - ref) <= tol)
        x = _f64(attn[t]).reshape(rows[t], d)
        h, y = ofp8.residual_rmsnorm(x, _f64(q[t]).reshape(rows[t], d), _f64(norm_w), head.eps)
        assert np.all(np.abs(_f64(resid[t]) - h) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(h))
        # Each e4m3 value is off by at most 2^-4 of y or half the smallest step
        # of its block (y's own error in fp32 is covered by the factor 1.01).
        step = ofp8.expand(ofp8.blocks(y, 1), 1, y.shape) * 2.0 ** -10
        z = y @ w8.T
        tol = 1.01 * ((2.0 ** -4 * np.abs(y) + step) @ np.abs(w8).T)
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(z) + tol)
        assert np.all(np.abs(_f64(logits[t]) - z) <= tol)
        ps, pn, B_in = search.parents(t)
        got = {"score": search.scores[t].view(R, n), "parent": search.bp_parent[t],
               "code": search.bp_code[t], "node": search.nodes[t].view(R, n)}
        compare_step({k: v.cpu().numpy() for k, v in got.items()}, to, t, _f64(logits[t]),
                     ps.cpu().numpy(), pn.cpu().numpy(), R, B_in, n, V, tol=TOL)
    catalog = {tuple(s) for s in to.leaves.tolist()}
    live = leaf.cpu().numpy().reshape(-1) >= 0
    assert live.any()
    for s in sids.cpu().numpy().reshape(-1, depth)[live].tolist():
        assert tuple(s) in catalog


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("captured", [False, True])
def test_decode_loop(tcb, dtype, captured):
    import torch
    _search(tcb, torch.bfloat16 if dtype == "bf16" else torch.float32, captured)


def test_step_hidden_status_reaches_the_search(tcb, monkeypatch):
    """A wait that gives up inside the 8-bit product (its bit set here behind the
    product, in the word that the product was handed) is what the search's status
    reads; the next step starts clean."""
    import torch
    from trie_constrained_beam_b200 import native
    R, n, depth, V, d = 2, 8, 2, 200, 256
    trie = tcb.sid_trie_build(host.draw_catalog(7, 1000, [V] * depth), [V] * depth)
    search = tcb.BeamSearch(trie, R, n, V, depth=depth)
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn((V, d), device="cuda", generator=g).to(torch.bfloat16)
    head = tcb.LmheadFp8(w, torch.ones(d, dtype=torch.bfloat16, device="cuda"), R * n)
    x = torch.randn((R, d), device="cuda", generator=g).to(torch.bfloat16)
    search.step_hidden(0, head, x)
    assert tcb.sidbeam_get_device_status(search.workspace) == 0
    product = native.lmhead_logits_fp8

    def gives_up(hq, hs, wq, ws, out, workspace, stream=None):
        product(hq, hs, wq, ws, out, workspace, stream=stream)
        workspace[:1].bitwise_or_(2)
    monkeypatch.setattr(native, "lmhead_logits_fp8", gives_up)
    search.step_hidden(0, head, x)
    assert tcb.sidbeam_get_device_status(search.workspace) == tcb.native.SIDBEAM_ERR_TIMEOUT
    assert tcb.sidbeam_get_device_status(search.workspace) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_decode_on_other_inputs(tcb, dtype):
    """A captured decode replayed on inputs that it was not captured on, over buffers
    filled with other values, gives every stage's bits of an eager decode on them."""
    import torch
    t16 = torch.bfloat16 if dtype == "bf16" else torch.float32
    R, n, depth, V, H, Hkv, D, page = 3, 24, 3, 200, 4, 2, 64, 16
    d = H * D
    trie = tcb.sid_trie_build(host.draw_catalog(78, 4000, [V] * depth), [V] * depth)
    g = torch.Generator(device="cuda").manual_seed(6)

    def normal(*shape, s=1.0):
        return (s * torch.randn(shape, device="cuda", generator=g)).to(torch.bfloat16)
    search = tcb.BeamSearch(trie, R, n, V, depth=depth)
    head = tcb.LmheadFp8(normal(V, d, s=0.2), 1 + normal(d, s=0.1), R * n, dtype=t16)
    kc, vc = normal(R * 10, page, Hkv, D), normal(R * 10, page, Hkv, D)
    table = torch.randperm(R * 10, device="cuda", generator=g).view(R, 10).to(torch.int32)
    cache_len = torch.tensor([150, 33, 64], dtype=torch.int32, device="cuda")
    embed, kv_embed = normal(V, H, D, s=1.5), normal(2, V, Hkv, D)
    kb = torch.zeros((depth, R * n, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vb = torch.zeros_like(kb)
    starts = [normal(R, H, D, s=1.5) for _ in range(2)]
    start = starts[0].clone()
    rows = [search.rows(t) for t in range(depth)]
    q = [torch.empty((m, H, D), dtype=torch.bfloat16, device="cuda") for m in rows]
    attn = [torch.empty_like(x) for x in q]
    resid = [torch.empty((m, d), dtype=torch.bfloat16, device="cuda") for m in rows]
    logits = [torch.empty((m, V), dtype=t16, device="cuda") for m in rows]

    def decode():
        q[0].copy_(start)
        for t in range(depth):
            if t:
                code = search.bp_code[t - 1].reshape(-1).clamp_min(0).long()
                q[t].copy_(embed[code])
                kb[t - 1].copy_(kv_embed[0][code])
                vb[t - 1].copy_(kv_embed[1][code])
            search.attention(t, q[t], kc, vc, cache_len, attn[t], k_beam=kb, v_beam=vb,
                             page_table=table)
            search.step_hidden(t, head, attn[t].view(rows[t], d), residual=q[t].view(rows[t], d),
                               residual_out=resid[t])
            logits[t].copy_(head._logits[:rows[t], :V])
        search.finalize()

    outputs = (q + attn + resid + logits + [search.scores, search.bp_parent, search.bp_code,
                                            search.nodes, search.sids, search.leaf])
    eager = []
    for s in starts:
        start.copy_(s)
        decode()
        eager.append([x.clone() for x in outputs])
    differ = [not torch.equal(a, b) for a, b in zip(*eager)]
    assert all(differ[:-6]) and any(differ[-6:])
    start.copy_(starts[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode()
    for which in (1, 0, 1):
        for x in outputs + [kb, vb, head._logits]:
            x.fill_(3)
        head.hidden_q.view(torch.uint8).fill_(0x38)
        head.hidden_scale.fill_(3)
        start.copy_(starts[which])
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(eager[which], outputs)):
            assert torch.equal(a, b), i
    assert tcb.sidbeam_get_device_status(search.workspace) == 0
