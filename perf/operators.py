"""Operator cases of the decode step around the constrained beam expansion: the
attention of beam rows over the prompt's cache and their own ancestors, the
residual RMS norm that leaves its rows in 8 bits, and the 8-bit SID-range
lm_head (its weight's quantisation and its matrix product).

``own`` chooses between elementary torch operations in 32 bits (False) and the
calls of this package (True). ``listed`` and ``draw`` give cases, ``prepare``
their seeded inputs, ``run`` one pass, ``work`` the bytes and operations a pass
cannot do without, ``exact`` the result in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128          # elements that share a scale
FP8_MAX = 448.0      # largest finite e4m3 value
MIN_AMAX = FP8_MAX * 2.0 ** -100  # blocks of smaller values share the scale 2^-100
EPS = 1e-6


def listed():
    # Hidden size 2,048, 8,192 codes, beams of 32 to 512 and 16 to 64 requests
    # are this repository's workloads; prompts of 1K and 5K tokens are the
    # lengths its notes quote.
    return [
        # First step of one request: one query row per head over a 1K prompt.
        dict(name="attention_one_row", op="attention", R=1, B=1, level=0, S=1000, H=16, Hkv=8, D=128, page=0),
        # First step of a whole batch over 5K prompts: reading the cache is all.
        dict(name="attention_rows_5k", op="attention", R=32, B=1, level=0, S=5000, H=16, Hkv=8, D=128, page=64),
        # Narrow beams (32) at the third step, smaller heads, paged cache.
        dict(name="attention_beam32", op="attention", R=32, B=32, level=2, S=1011, H=16, Hkv=4, D=64, page=16),
        # 64 requests x beam 128 at the third step, paged, ragged prompts.
        dict(name="attention_beam128", op="attention", R=64, B=128, level=2, S=2000, H=16, Hkv=8, D=128, page=64),
        # 16 requests x beam 512 at the fifth step, one slab per request.
        dict(name="attention_beam512", op="attention", R=16, B=512, level=4, S=1024, H=16, Hkv=8, D=128, page=0),
        # The final norm of one beam row, and of 16 x 512 rows.
        dict(name="norm_row", op="norm", M=1, d=2048),
        dict(name="norm_rows", op="norm", M=8192, d=2048),
        # The lm_head weight laid out once: a small odd codebook, the large one.
        dict(name="quantize_small", op="quantize", V=500, d=1040),
        dict(name="quantize_large", op="quantize", V=8192, d=2048),
        # lm_head products: step 0 of 32 requests, an odd shape, 32 x 128 rows.
        dict(name="lmhead_rows32", op="lmhead", M=32, V=8192, d=2048, out="bf16"),
        dict(name="lmhead_odd", op="lmhead", M=777, V=1001, d=1040, out="f32"),
        dict(name="lmhead_rows4096", op="lmhead", M=4096, V=8192, d=2048, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "norm", "quantize", "lmhead", "lmhead"])
    if op == "attention":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 3, 4, 8])
        B = _log_int(rng, 1, 512)
        level = 0 if B == 1 else rng.randint(0, 5)
        S = _log_int(rng, 1, 6000)
        # No more than the largest listed case's products or cache bytes.
        R = _log_int(rng, 1, 64)
        while R > 1 and (R * B * H * S * D > 16 * 512 * 16 * 1024 * 128 or R * S * Hkv * D > 32 * 5000 * 8 * 128):
            R //= 2
        while R * B * H * S * D > 16 * 512 * 16 * 1024 * 128:
            S //= 2
        return dict(op=op, R=R, B=B, level=level, S=S, H=H, Hkv=Hkv, D=D, page=rng.choice([0, 16, 64, 128]))
    d = 16 * _log_int(rng, 8, 256)
    if op == "norm":
        return dict(op=op, M=_log_int(rng, 1, 8192 * 2048 // max(d, 2048)), d=d)
    V = _log_int(rng, 8, 8192 * 2048 // max(d, 2048))
    if op == "quantize":
        return dict(op=op, V=V, d=d)
    return dict(op=op, M=_log_int(rng, 1, 4096), V=V, d=d, out=rng.choice(["f32", "bf16"]))


def _lens(case):
    """Prompt lengths: the longest first, the others spread over the upper half."""
    S, R = case["S"], case["R"]
    return [S - (r * 7919) % (S // 2 + 1) for r in range(R)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)

    def normal(*shape, sigma=1.0, dtype=torch.bfloat16):
        return torch.empty(shape, device="cuda", dtype=dtype).normal_(0, sigma, generator=g)

    s = dict(case)
    s["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    if case["op"] == "attention":
        R, B, S, H, Hkv, D, L = (case[k] for k in ("R", "B", "S", "H", "Hkv", "D", "level"))
        lens = _lens(case)
        s["cache_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = normal(R * B, H, D, sigma=1.5)
        if case["page"]:
            per = -(-S // case["page"])
            pages = R * per + 3
            s["page_table"] = torch.randperm(pages, device="cuda", generator=g)[:R * per].view(R, per).to(torch.int32)
            s["k_cache"] = normal(pages, case["page"], Hkv, D)
            s["v_cache"] = normal(pages, case["page"], Hkv, D)
        else:
            s["page_table"] = None
            s["k_cache"] = normal(R, S, Hkv, D)
            s["v_cache"] = normal(R, S, Hkv, D)
        s["k_beam"] = s["v_beam"] = s["bp_parent"] = None
        if L:
            s["k_beam"] = normal(L, R * B, Hkv, D)
            s["v_beam"] = normal(L, R * B, Hkv, D)
            # Back-pointers as the steps write them: step 0 has one parent row.
            s["bp_parent"] = torch.randint(0, B, (L, R, B), device="cuda", generator=g, dtype=torch.int32)
            s["bp_parent"][0] = 0
        s["out"] = torch.empty(R * B, H, D, dtype=torch.bfloat16, device="cuda")
        return s
    d = case["d"]
    nb = -(-d // BLOCK)
    if case["op"] == "norm":
        M = case["M"]
        s["x"], s["residual"] = normal(M, d), normal(M, d, sigma=3.0)
        s["weight"] = (1 + normal(d, sigma=0.1, dtype=torch.float32)).to(torch.bfloat16)
        s["residual_out"] = torch.empty_like(s["x"])
        s["hidden_q"] = torch.empty(M, d, dtype=torch.float8_e4m3fn, device="cuda")
        s["hidden_scale"] = torch.empty(M, nb, dtype=torch.float32, device="cuda")
        return s
    V = case["V"]
    w = normal(V, d, sigma=0.02)
    s["w_q"] = torch.empty(V, d, dtype=torch.float8_e4m3fn, device="cuda")
    s["w_scale"] = torch.empty(-(-V // BLOCK), nb, dtype=torch.float32, device="cuda")
    if case["op"] == "quantize":
        s["w"] = w
        return s
    M = case["M"]
    s["hidden_q"], s["hidden_scale"] = _plain_quantize(normal(M, d).float(), 1)
    s["w_q"], s["w_scale"] = _plain_quantize(w.float(), BLOCK)
    ld = -(-V // 8) * 8
    dtype = torch.float32 if case["out"] == "f32" else torch.bfloat16
    s["logits"] = torch.empty(M, ld, dtype=dtype, device="cuda")[:, :V]
    return s


def _blocks(t, rows):
    """[M, d] padded with zeros to whole blocks, as [mb, rows, nb, BLOCK]."""
    M, d = t.shape
    t = torch.nn.functional.pad(t, (0, -d % BLOCK, 0, -M % rows))
    return t.view(t.shape[0] // rows, rows, t.shape[1] // BLOCK, BLOCK)


def _plain_quantize(t, rows):
    """e4m3 values and fp32 scales of [M, d], a scale for each rows x BLOCK block."""
    M, d = t.shape
    b = _blocks(t, rows)
    scale = b.abs().amax(dim=(1, 3)).clamp_min(MIN_AMAX) / FP8_MAX
    q = b * (1.0 / scale)[:, None, :, None]
    q = q.view(q.shape[0] * rows, -1)[:M, :d].contiguous()
    return q.to(torch.float8_e4m3fn), scale


def _plain_attention(s):
    R, B, H, Hkv, D, L = (s[k] for k in ("R", "B", "H", "Hkv", "D", "level"))
    G = H // Hkv
    if s["page_table"] is not None:
        idx = s["page_table"].long()
        k, v = (s[n][idx].reshape(R, -1, Hkv, D).float() for n in ("k_cache", "v_cache"))
    else:
        k, v = s["k_cache"].float(), s["v_cache"].float()
    q = s["q"].view(R, B, Hkv, G, D).float() * (D ** -0.5)
    pos = torch.arange(k.shape[1], device=q.device)
    dead = pos[None, :] >= s["cache_len"][:, None]
    score = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(R, Hkv, B * G, D), k.permute(0, 2, 3, 1))
    score = score.masked_fill(dead[:, None, None, :], -math.inf).view(R, Hkv, B, G, -1)
    if L:
        # The slot of each beam's ancestor at every level, the last level first.
        slot = torch.arange(B, device=q.device).expand(R, B)
        base = torch.arange(R, device=q.device)[:, None] * B
        rows = [None] * L
        for u in range(L - 1, -1, -1):
            rows[u] = slot + base
            slot = s["bp_parent"][u].long().gather(1, slot)
        rows = torch.stack(rows)                                          # [L, R, B]
        lev = torch.arange(L, device=q.device)[:, None, None]
        kb, vb = s["k_beam"][lev, rows].float(), s["v_beam"][lev, rows].float()  # [L, R, B, Hkv, D]
        own_score = torch.einsum("rbhgd,lrbhd->rhbgl", q, kb)
        score = torch.cat([score, own_score], dim=-1)
    p = torch.exp(score - score.amax(dim=-1, keepdim=True))
    p = p / p.sum(dim=-1, keepdim=True)
    n = k.shape[1]
    o = torch.matmul(p[..., :n].reshape(R, Hkv, B * G, n), v.permute(0, 2, 1, 3)).view(R, Hkv, B, G, D)
    if L:
        o = o + torch.einsum("rhbgl,lrbhd->rhbgd", p[..., n:], vb)
    return o.permute(0, 2, 1, 3, 4).reshape(R * B, H, D).to(torch.bfloat16)


def run(state):
    s = state
    op = s["op"]
    if own:
        import trie_constrained_beam_b200 as tcb
        if op == "attention":
            tcb.beam_attention(s["q"], s["k_cache"], s["v_cache"], s["cache_len"], s["out"], s["workspace"],
                               page_table=s["page_table"], level=s["level"], k_beam=s["k_beam"],
                               v_beam=s["v_beam"], bp_parent=s["bp_parent"])
            return {"out": s["out"]}
        if op == "norm":
            tcb.residual_rmsnorm_fp8(s["x"], s["residual"], s["weight"], EPS, s["residual_out"], s["hidden_q"],
                                     s["hidden_scale"])
            return {"residual": s["residual_out"], "q": s["hidden_q"], "scale": s["hidden_scale"]}
        if op == "quantize":
            tcb.lmhead_quantize_fp8(s["w"], s["w_q"], s["w_scale"])
            return {"q": s["w_q"], "scale": s["w_scale"]}
        tcb.lmhead_logits_fp8(s["hidden_q"], s["hidden_scale"], s["w_q"], s["w_scale"], s["logits"], s["workspace"])
        return {"logits": s["logits"]}
    if op == "attention":
        return {"out": _plain_attention(s)}
    if op == "norm":
        h = s["x"].float() + s["residual"].float()
        y = h * torch.rsqrt(h.square().mean(dim=-1, keepdim=True) + EPS) * s["weight"].float()
        q, scale = _plain_quantize(y, 1)
        return {"residual": h.to(torch.bfloat16), "q": q, "scale": scale}
    if op == "quantize":
        q, scale = _plain_quantize(s["w"].float(), BLOCK)
        return {"q": q, "scale": scale}
    d, V = s["d"], s["V"]
    h = s["hidden_q"].float() * s["hidden_scale"].repeat_interleave(BLOCK, 1)[:, :d]
    w = s["w_q"].float() * s["w_scale"].repeat_interleave(BLOCK, 0)[:V].repeat_interleave(BLOCK, 1)[:, :d]
    return {"logits": torch.matmul(h, w.T).to(s["logits"].dtype)}


def work(case):
    op = case["op"]
    if op == "attention":
        R, B, H, Hkv, D, L = (case[k] for k in ("R", "B", "H", "Hkv", "D", "level"))
        tokens = sum(_lens(case))
        # Ancestors that are distinct: n draws with replacement out of B slots.
        rows, n = 0.0, float(B)
        for _ in range(L):
            rows += R * n
            n = B * (1 - (1 - 1 / B) ** n)
        kv = (tokens + rows) * Hkv * D * 2 * 2
        return {"bytes": kv + 2 * R * B * H * D * 2 + 4 * L * R * B + 4 * R,
                "flops": 4.0 * H * D * B * (tokens + R * L)}
    d = case["d"]
    nb = -(-d // BLOCK)
    if op == "norm":
        M = case["M"]
        return {"bytes": M * d * (2 + 2 + 2 + 1) + 2 * d + 4 * M * nb, "flops": 6.0 * M * d}
    V = case["V"]
    vb = -(-V // BLOCK)
    if op == "quantize":
        return {"bytes": 3 * V * d + 4 * vb * nb, "flops": 2.0 * V * d}
    M = case["M"]
    esize = 4 if case["out"] == "f32" else 2
    return {"bytes": (M + V) * d + 4 * (M + vb) * nb + M * V * esize, "flops": 2.0 * M * V * d}


def _exact_blocks(t, rows):
    """Unrounded e4m3 inputs and scales of a 64-bit matrix, block by block."""
    M, d = t.shape
    q = torch.empty_like(t)
    scale = torch.empty(-(-M // rows), -(-d // BLOCK), dtype=torch.float64, device=t.device)
    for j in range(scale.shape[1]):
        part = t[:, j * BLOCK:(j + 1) * BLOCK]
        a = part.abs().max(dim=1).values
        if rows > 1:
            a = torch.stack([c.max() for c in a.split(rows)])
        scale[:, j] = torch.clamp(a, min=MIN_AMAX) / FP8_MAX
        q[:, j * BLOCK:(j + 1) * BLOCK] = part / scale[:, j].repeat_interleave(rows)[:M, None]
    return q, scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + s["residual"].double()
        y = h / (h.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS).sqrt() * s["weight"].double()
        q, scale = _exact_blocks(y, 1)
        return {"residual": h, "q": q, "scale": scale}
    if op == "quantize":
        q, scale = _exact_blocks(s["w"].double(), BLOCK)
        return {"q": q, "scale": scale}
    if op == "lmhead":
        M, V, d = case["M"], case["V"], case["d"]
        z = torch.zeros(M, V, dtype=torch.float64, device="cuda")
        for j in range(0, d, BLOCK):
            part = s["hidden_q"][:, j:j + BLOCK].double() @ s["w_q"][:, j:j + BLOCK].double().T
            cols = s["w_scale"][:, j // BLOCK].double().repeat_interleave(BLOCK)[:V]
            z += part * s["hidden_scale"][:, j // BLOCK].double()[:, None] * cols[None, :]
        return {"logits": z}
    R, B, H, Hkv, D, L = (case[k] for k in ("R", "B", "H", "Hkv", "D", "level"))
    out = torch.zeros(R, B, H, D, dtype=torch.float64, device="cuda")
    lens = s["cache_len"].tolist()
    for r in range(R):
        n = lens[r]
        if s["page_table"] is not None:
            use = s["page_table"][r].long()
            k = s["k_cache"][use].reshape(-1, Hkv, D)[:n].double()
            v = s["v_cache"][use].reshape(-1, Hkv, D)[:n].double()
        else:
            k, v = s["k_cache"][r, :n].double(), s["v_cache"][r, :n].double()
        paths = []
        at = torch.arange(B, device="cuda")
        for u in reversed(range(L)):
            paths.append((u, at))
            at = s["bp_parent"][u, r].long()[at]
        for h in range(H):
            g = h * Hkv // H
            q = s["q"].view(R, B, H, D)[r, :, h].double() / math.sqrt(D)
            x = [q @ k[:, g].T] + [(q * s["k_beam"][u, r * B + a, g].double()).sum(1, keepdim=True) for u, a in paths]
            x = torch.softmax(torch.cat(x, dim=1), dim=1)
            o = x[:, :n] @ v[:, g]
            for i, (u, a) in enumerate(paths):
                o += x[:, n + i, None] * s["v_beam"][u, r * B + a, g].double()
            out[r, :, h] = o
    return {"out": out.view(R * B, H, D)}
