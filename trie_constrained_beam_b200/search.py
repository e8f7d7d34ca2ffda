"""Device buffers and the step loop of one constrained beam search.

Orchestration only: every step is one ``beam_step`` call, the end is one
``beam_finalize`` call. Step t reads the previous step's outputs as its parent
rows (B_in = 1 at step 0: the root of every request, score 0), and writes its
back-pointers straight into slice t of the [depth][R][n] history.
"""
from __future__ import annotations

import contextlib

import torch

from . import native


class LmheadFp8:
    """One level's lm_head in 8 bits with the norm before it: the weight laid out
    once (``lmhead_quantize_fp8``) and the row buffers of up to ``max_rows`` rows.

    w_sid bf16 [V, d], norm_weight bf16 [d]; logits in ``dtype`` (bf16 or f32).
    ``stream`` (default: the current one) quantises the weight and owns the
    buffers, which every call rewrites: one stream at a time, in the caller's order.
    ``workspace`` holds the status word of calls that are given no other.
    """

    def __init__(self, w_sid, norm_weight, max_rows: int, eps: float = 1e-6,
                 dtype=torch.bfloat16, stream=None):
        V, d = w_sid.shape
        dev = w_sid.device
        nb = -(-d // native.FP8_BLOCK)
        self.V, self.d, self.eps, self.max_rows = V, d, float(eps), int(max_rows)
        self.norm_weight = norm_weight
        # On `stream` as the quantisation is: memory that the current stream has freed
        # may still be in use there, and the status word has to be zero before its
        # first call.
        with torch.cuda.stream(stream):
            self.w_q = torch.empty((V, d), dtype=torch.float8_e4m3fn, device=dev)
            self.w_scale = torch.empty((-(-V // native.FP8_BLOCK), nb), dtype=torch.float32,
                                       device=dev)
            self.hidden_q = torch.empty((max_rows, d), dtype=torch.float8_e4m3fn, device=dev)
            self.hidden_scale = torch.empty((max_rows, nb), dtype=torch.float32, device=dev)
            # Rows of whole 16-byte units, as beam_step reads them.
            self._logits = torch.empty((max_rows, -(-V // 8) * 8), dtype=dtype, device=dev)
            self.workspace = torch.zeros(256, dtype=torch.uint8, device=dev)
        native.lmhead_quantize_fp8(w_sid, self.w_q, self.w_scale, stream=stream)

    def logits(self, x, residual=None, residual_out=None, stream=None, workspace=None):
        """Logits [rows, V] of rows x (+ residual), bf16 [rows, d]; a view of this
        object's buffer. ``workspace``: where the product reports a wait that gave
        up (the logits then hold an earlier call's), default this object's."""
        rows = x.shape[0]
        if rows > self.max_rows:
            raise ValueError(f"{rows} rows, room for {self.max_rows}")
        hq, hs = self.hidden_q[:rows], self.hidden_scale[:rows]
        native.residual_rmsnorm_fp8(x, residual, self.norm_weight, self.eps, residual_out, hq, hs,
                                    stream=stream)
        out = self._logits[:rows, :self.V]
        native.lmhead_logits_fp8(hq, hs, self.w_q, self.w_scale, out,
                                 self.workspace if workspace is None else workspace,
                                 stream=stream)
        return out


class BeamSearch:
    def __init__(self, trie, R: int, n: int, V, depth: int = None, device="cuda",
                 skip_rows: bool = False, temperature: float = 0.0, seed: int = 0,
                 widths=None):
        """widths: optional per-request beam widths (each <= n); request r keeps
        its widths[r] best beams at every step (the rest of its n slots are
        padding), so one launch per step and one captured graph serve requests
        of different widths."""
        self.trie = trie
        self.skip_rows = skip_rows  # beam_step_ex row skipping (same results)
        # temperature > 0: Gumbel top-k draws (beam_step_gumbel), Philox key `seed`
        self.temperature, self.seed = float(temperature), int(seed)
        self.depth = depth if depth is not None else trie.depth
        self.V = list(V) if isinstance(V, (list, tuple)) else [int(V)] * self.depth
        self.R, self.n = R, n
        dev = torch.device(device)
        self.root_scores = torch.zeros(R, dtype=torch.float32, device=dev)
        self.root_nodes = torch.zeros(R, dtype=torch.int32, device=dev)
        self.scores = torch.empty((self.depth, R * n), dtype=torch.float32, device=dev)
        self.nodes = torch.empty((self.depth, R * n), dtype=torch.int32, device=dev)
        self.bp_parent = torch.empty((self.depth, R, n), dtype=torch.int32, device=dev)
        self.bp_code = torch.empty((self.depth, R, n), dtype=torch.int32, device=dev)
        ws = 0
        for t in range(self.depth):
            size = (native.beam_step_gumbel_workspace_size if self.temperature > 0
                    else native.beam_step_workspace_size)
            ws = max(ws, size(R, 1 if t == 0 else n, n, self.V[t]))
        self.workspace = torch.zeros(ws, dtype=torch.uint8, device=dev)
        self.widths = None
        if widths is not None:
            w = [int(x) for x in widths]
            if len(w) != R or min(w) < 0 or max(w) > n:
                raise ValueError("widths: one value in [0, n] per request")
            if self.temperature > 0:
                raise ValueError("widths with temperature > 0 is not supported")
            self.widths = torch.tensor(w, dtype=torch.int32, device=dev)
        self.device_index = self.scores.get_device()
        self.sids = torch.empty((R, n, self.depth), dtype=torch.int32, device=dev)
        self.leaf = torch.empty((R, n), dtype=torch.int32, device=dev)

    def rows(self, t: int) -> int:
        return self.R * (1 if t == 0 else self.n)

    def parents(self, t: int):
        """(parent_scores, parent_nodes, B_in) of step t."""
        if t == 0:
            return self.root_scores, self.root_nodes, 1
        return self.scores[t - 1], self.nodes[t - 1], self.n

    def _on_device(self):
        """This search's device made current (the library launches there), as the calls
        that take their device from their tensors do by themselves."""
        if self.device_index < 0 or self.device_index == torch.cuda.current_device():
            return contextlib.nullcontext()
        return torch.cuda.device(self.device_index)

    def step(self, t: int, logits, stream=None):
        with self._on_device():
            self._step(t, logits, stream)

    def _step(self, t: int, logits, stream):
        ps, pn, B_in = self.parents(t)
        if self.temperature > 0:
            native.beam_step_gumbel(self.trie, t, logits, ps, pn, self.R, B_in, self.n,
                                    self.V[t], self.temperature, self.seed, self.scores[t],
                                    self.bp_parent[t], self.bp_code[t], self.nodes[t],
                                    self.workspace, stream=stream)
            return
        native.beam_step(self.trie, t, logits, ps, pn, self.R, B_in, self.n, self.V[t],
                         self.scores[t], self.bp_parent[t], self.bp_code[t], self.nodes[t],
                         self.workspace, stream=stream, skip_rows=self.skip_rows,
                         out_width=self.widths)

    def attention(self, t: int, q, k_cache, v_cache, cache_len, out, k_beam=None, v_beam=None,
                  page_table=None, scale=None, stream=None):
        """Attention of step t's rows (``beam_attention``): over their request's
        prompt and, from step 1, the beams' own tokens chosen at steps 0 .. t-1,
        found through this search's back-pointers. k_beam, v_beam bf16
        [>= t, R*n, Hkv, D]: slice u holds the tokens that step u chose."""
        native.beam_attention(q, k_cache, v_cache, cache_len, out, self.workspace,
                              page_table=page_table, level=t, k_beam=k_beam, v_beam=v_beam,
                              bp_parent=self.bp_parent, scale=scale, stream=stream)

    def step_hidden(self, t: int, head: LmheadFp8, x, residual=None, residual_out=None,
                    stream=None):
        """Step t from hidden states bf16 [rows(t), d]: residual RMS norm and
        lm_head in 8 bits (``head``), then the constrained step on its logits. All
        of them report in this search's workspace (``sidbeam_get_device_status``).
        Of more rows, or of a head with more codes, the step uses the first."""
        if x.shape[0] < self.rows(t) or head.V < self.V[t]:
            raise ValueError(f"step {t} takes {self.rows(t)} rows and {self.V[t]} codes, got "
                             f"{x.shape[0]} rows and a head of {head.V} codes")
        logits = head.logits(x, residual, residual_out, stream=stream, workspace=self.workspace)
        self.step(t, logits, stream=stream)

    def skipped_rows(self, stream=None) -> int:
        """Rows left unread by row skipping since the last call."""
        return native.beam_step_skipped_rows(self.workspace, stream=stream)

    def finalize(self, stream=None):
        with self._on_device():
            native.beam_finalize(self.depth, self.R, self.n, self.bp_parent, self.bp_code,
                                 self.nodes[self.depth - 1], self.sids, self.leaf, stream=stream)
        return self.sids, self.leaf, self.scores[self.depth - 1].view(self.R, self.n)

    def capture(self, logits_per_step, events=None):
        """A CUDA graph of the whole search (every beam_step, then beam_finalize)
        on fixed logits tensors; ``graph.replay()`` runs it on the current stream.

        Call the search once eagerly first (that sets the kernels' shared-memory
        limits outside the capture). ``events``: optional depth + 2 events made
        with ``enable_timing=True, external=True``, recorded before every step,
        before finalize and at the end (per-step device times of a replay).
        """
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            for t in range(self.depth):
                if events is not None:
                    events[t].record()
                self.step(t, logits_per_step[t])
            if events is not None:
                events[self.depth].record()
            self.finalize()
            if events is not None:
                events[self.depth + 1].record()
        torch.cuda.current_stream().wait_stream(side)
        return g

    def run(self, logits_for_step, stream=None):
        """logits_for_step(t, search) -> logits tensor [rows(t), ld] for step t."""
        for t in range(self.depth):
            self.step(t, logits_for_step(t, self), stream=stream)
        return self.finalize(stream=stream)
