"""CPU checks of the attention and the 8-bit lm_head: the oracle's pins, and the
arguments that the library refuses on the host before any device call."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import fp8 as ofp8

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from trie_constrained_beam_b200 import build, native
    build.build()
    return native.load()


# ------------------------------------------------------------------ oracle pins
def test_oracle_e4m3_table_is_torchs():
    import torch
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).float().numpy()
    got = ofp8.e4m3_values()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.isnan(got).sum() == 2
    assert np.array_equal(got[~np.isnan(got)], ref[~np.isnan(ref)])
    assert np.nanmax(got) == ofp8.FP8_MAX


def test_oracle_logits_are_the_dequantised_product():
    rng = np.random.default_rng(0)
    M, V, d = 3, 130, 144
    hc, wc = rng.integers(0, 127, size=(M, d)), rng.integers(0, 127, size=(V, d))
    hs, ws = rng.random((M, 2)), rng.random((2, 2))
    val = ofp8.e4m3_values()
    z, _ = ofp8.lmhead_logits(hc, hs, wc, ws)
    for m, c in ((0, 0), (2, 127), (1, 128), (2, 129)):
        ref = sum(hs[m, k // 128] * ws[c // 128, k // 128] * val[hc[m, k]] * val[wc[c, k]]
                  for k in range(d))
        assert abs(z[m, c] - ref) <= 1e-12 * abs(ref) + 1e-9


def test_oracle_attention_equals_a_copied_prefix():
    """Following the back-pointers equals attention over a cache in which every
    beam has its own copy of prompt and ancestors (torch, float64)."""
    import torch
    rng = np.random.default_rng(1)
    R, B, H, Hkv, D, L = 2, 5, 4, 2, 16, 3
    lens = [7, 0]
    q = rng.standard_normal((R * B, H, D))
    prompts = [(rng.standard_normal((n, Hkv, D)), rng.standard_normal((n, Hkv, D))) for n in lens]
    kb, vb = rng.standard_normal((2, L, R * B, Hkv, D))
    bp = rng.integers(0, B, size=(L, R, B))
    bp[0] = 0
    bp[1, 1, 2] = -1
    out, mean, _ = oracle.beam_attention(q, prompts, L, kb, vb, bp)
    # Copies: level u's beams copy their parent's prefix and append their own token.
    for r in range(R):
        pre = [(prompts[r][0], prompts[r][1])]
        for u in range(L):
            nxt = []
            for s in range(B):
                p = bp[u, r, s]
                src = pre[p] if 0 <= p < len(pre) else None
                nxt.append(None if src is None else
                           (np.concatenate([src[0], kb[u, r * B + s][None]]),
                            np.concatenate([src[1], vb[u, r * B + s][None]])))
            pre = nxt
        for b in range(B):
            if pre[b] is None:
                assert not out[r * B + b].any()
                continue
            for h in range(H):
                k, v = (torch.from_numpy(t[:, h // 2]) for t in pre[b])
                w = torch.softmax(k @ torch.from_numpy(q[r * B + b, h]) / D ** 0.5, 0)
                assert np.allclose(out[r * B + b, h], (w @ v).numpy(), atol=1e-12)
    assert np.all(mean + 1e-12 >= np.abs(out))


# ------------------------------------------------------------------ refusals
def _norm(lib, x=0x1000, res=0x2000, w=0x3000, eps=1e-6, M=4, d=256, ro=0x4000, q=0x5000,
          s=0x6000):
    return lib.residual_rmsnorm_fp8(P(x), P(res), P(w), eps, M, d, P(ro), P(q), P(s), None)


def test_norm_refusals(lib):
    for bad in (dict(M=-1), dict(d=0), dict(d=8), dict(d=250), dict(d=16400), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x=0), dict(w=0), dict(q=0),
                dict(s=0)):
        assert _norm(lib, **bad) == -1, bad
    for bad in (dict(x=0x1008), dict(res=0x2004), dict(w=0x3002), dict(ro=0x4008), dict(q=0x5008),
                dict(s=0x6002)):
        assert _norm(lib, **bad) == -3, bad
    assert _norm(lib, M=0, x=0) == 0        # nothing to do, nothing launched


def test_quantize_refusals(lib):
    def quant(w=0x1000, V=128, d=256, q=0x2000, s=0x3000):
        return lib.lmhead_quantize_fp8(P(w), V, d, P(q), P(s), None)
    for bad in (dict(w=0), dict(q=0), dict(s=0), dict(V=0), dict(V=32769), dict(d=24),
                dict(d=32768)):
        assert quant(**bad) == -1, bad
    for bad in (dict(w=0x1008), dict(q=0x2008), dict(s=0x3001)):
        assert quant(**bad) == -3, bad


def test_logits_refusals(lib):
    def logits(hq=0x1000, hs=0x2000, wq=0x3000, ws=0x4000, M=4, V=256, d=256, out=0x5000, dt=0,
               ld=256, work=0x8000, size=256):
        return lib.lmhead_logits_fp8(P(hq), P(hs), P(wq), P(ws), M, V, d, P(out), dt, ld, P(work),
                                     size, None)
    for bad in (dict(hq=0), dict(hs=0), dict(wq=0), dict(ws=0), dict(out=0), dict(M=-1),
                dict(V=0), dict(V=40000), dict(d=0), dict(d=264), dict(dt=2), dict(ld=255)):
        assert logits(**bad) == -1, bad
    for bad in (dict(hq=0x1001), dict(wq=0x3008), dict(out=0x5004), dict(ld=258),
                dict(dt=1, ld=260), dict(hs=0x2001)):
        assert logits(**bad) == -3, bad
    for bad in (dict(work=0), dict(size=128), dict(work=0x8010)):
        assert logits(**bad) == -4, bad
    assert logits(M=0, out=0) == 0


def _attention(lib, **kw):
    a = dict(q=0x1000, qs=512, k=0x2000, v=0x3000, ps=4096, ts=256, pages=16, size=16, table=0x4000,
             per=4, lens=0x5000, level=2, bp=0x6000, kb=0x7000, vb=0x8000, R=2, B=4, H=4, Hkv=2,
             D=128, scale=0.1, out=0x9000, os=512, work=0xA000, wsize=256)
    a.update(kw)
    from trie_constrained_beam_b200 import native
    return lib.beam_attention(native._ATTENTION(
        a["q"], a["qs"], a["k"], a["v"], a["ps"], a["ts"], a["pages"], a["size"],
        a["table"] or 0, a["lens"], a["bp"], a["kb"], a["vb"], a["per"], a["level"], a["R"],
        a["B"], a["H"], a["Hkv"], a["D"], a["scale"], a["out"], a["os"], a["work"], a["wsize"]),
        None)


def test_attention_struct_layout(tmp_path):
    """The binding packs what a C compiler lays out."""
    import os
    import shutil
    import struct
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "sidbeam.h"\n#define O(f) '
                   '(int)offsetof(sidbeam_attention, f)\nint main(void) {\n'
                   '  printf("%d %d %d %d %d %d", (int)sizeof(sidbeam_attention), O(page_table),'
                   ' O(pages_per_request), O(scale), O(out), O(workspace_bytes)); return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    fields = "PqPPqqiiPPPPPiiiiiiifPqPN"
    ends = [struct.calcsize(fields[:k + 1]) for k in range(len(fields))]
    start = lambda k: ends[k] - struct.calcsize(fields[k])  # noqa: E731
    assert got == [struct.calcsize(fields), start(8), start(13), start(20), start(21), start(24)]
    from trie_constrained_beam_b200 import native
    assert len(native._ATTENTION(*([0] * 20 + [0.0] + [0] * 4))) == got[0]


def test_attention_refusals(lib):
    for bad in (dict(q=0), dict(k=0), dict(v=0), dict(lens=0), dict(out=0), dict(R=0), dict(B=0),
                dict(B=4097), dict(R=1 << 30, B=4), dict(D=96), dict(H=3), dict(H=0), dict(Hkv=0),
                dict(H=512, Hkv=2, qs=1 << 17, os=1 << 17), dict(level=-1), dict(level=17),
                dict(bp=0), dict(kb=0), dict(vb=0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(pages=0), dict(size=0), dict(size=8),
                dict(size=48), dict(size=1 << 17), dict(per=0), dict(per=1 << 30),
                dict(table=None), dict(qs=511), dict(os=504), dict(ts=248), dict(ps=128)):
        assert _attention(lib, **bad) == -1, bad
    for bad in (dict(q=0x1008), dict(k=0x2008), dict(v=0x3002), dict(out=0x9008), dict(kb=0x7008),
                dict(vb=0x8004), dict(qs=516), dict(os=516), dict(ts=260), dict(ps=4100)):
        assert _attention(lib, **bad) == -3, bad
    for bad in (dict(work=0), dict(wsize=255), dict(work=0xA010)):
        assert _attention(lib, **bad) == -4, bad


def test_python_checks_come_before_the_library():
    """Tensors of the wrong kind are refused by the binding, on the CPU."""
    import torch
    import trie_constrained_beam_b200 as tcb
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    q = torch.zeros((2, 256), dtype=torch.float8_e4m3fn)
    s = torch.zeros((2, 2))
    with pytest.raises(ValueError, match="CUDA"):
        tcb.residual_rmsnorm_fp8(x, None, x[0], 1e-6, None, q, s)
    with pytest.raises(TypeError):
        tcb.residual_rmsnorm_fp8(s, None, x[0], 1e-6, None, q, s)
    with pytest.raises(ValueError):
        tcb.lmhead_quantize_fp8(x, q, s)
    n = torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros((2, 8, 1, 64), dtype=torch.bfloat16)
    rows = torch.zeros((3, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rows"):
        tcb.beam_attention(rows, cache, cache, n, rows, torch.zeros(256, dtype=torch.uint8))


def test_import_without_torchs_cuda_bindings():
    """A torch built without CUDA has none of torch._C's CUDA functions: the package
    imports and answers host calls, and refuses CPU tensors as elsewhere."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import trie_constrained_beam_b200 as tcb
assert tcb.beam_step_workspace_size(2, 4, 4, 100) > 0
x = torch.zeros((2, 256), dtype=torch.bfloat16)
try:
    tcb.lmhead_quantize_fp8(x, x.to(torch.float8_e4m3fn), torch.zeros((1, 2)))
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise SystemExit("a CPU tensor was taken")
print("imported")
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert done.returncode == 0 and "imported" in done.stdout, done.stderr


def test_oracle_norm_and_blocks_are_torchs():
    """The norm against torch's own (float64), the block scales against the definition,
    element by element."""
    import torch
    rng = np.random.default_rng(2)
    x, res = rng.standard_normal((2, 5, 144)) * 3
    w = rng.standard_normal(144)
    for r in (None, res):
        h, y = ofp8.residual_rmsnorm(x, r, w, 1e-3)
        assert np.array_equal(h, x if r is None else x + r)
        ref = torch.nn.functional.rms_norm(torch.from_numpy(h), (144,), torch.from_numpy(w), 1e-3)
        assert np.allclose(y, ref.numpy(), rtol=1e-13, atol=0)
    m = rng.standard_normal((130, 144))
    m[128:] = 0
    for rows in (1, 128):
        s = ofp8.blocks(m, rows)
        assert s.shape == (-(-130 // rows), 2)
        full = ofp8.expand(s, rows, m.shape)
        for i, j in ((0, 0), (5, 127), (127, 128), (128, 3), (129, 143)):
            part = [abs(m[a, b]) for a in range(130) for b in range(144)
                    if a // rows == i // rows and b // 128 == j // 128]
            assert full[i, j] == max(max(part), 448 * 2.0 ** -100) / 448


def test_logits_refuse_rows_that_do_not_round_up(lib):
    """The last 127 row counts of an int do not round up to whole tiles."""
    def logits(M):
        return lib.lmhead_logits_fp8(P(0x1000), P(0x2000), P(0x3000), P(0x4000), M, 8, 16,
                                     P(0x5000), 0, 8, P(0x8000), 256, None)
    for M in ((1 << 31) - 1, (1 << 31) - 127):
        assert logits(M) == -1, M
