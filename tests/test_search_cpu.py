"""CPU checks of the buffers and the plumbing of search.py: the library's entry
points are replaced by recorders, so no device is needed."""
import pytest
import torch

import trie_constrained_beam_b200 as tcb
from trie_constrained_beam_b200 import build, native

TIMEOUT_BIT = 2  # of the status word, the first 4 bytes of a workspace


@pytest.fixture
def calls(monkeypatch):
    """Every entry point that search.py calls, recorded; the 8-bit product gives up
    on a wait, as the kernel reports it, in the workspace that it was handed."""
    build.build()
    seen = []

    def product(hidden_q, hidden_scale, w_q, w_scale, out, workspace, stream=None):
        seen.append(("lmhead_logits_fp8", workspace))
        workspace[0] |= TIMEOUT_BIT

    def record(name):
        return lambda *args, **kw: seen.append((name, args, kw))
    monkeypatch.setattr(native, "lmhead_logits_fp8", product)
    for name in ("lmhead_quantize_fp8", "residual_rmsnorm_fp8", "beam_step", "beam_step_gumbel"):
        monkeypatch.setattr(native, name, record(name))
    return seen


def _search(R=2, n=4, V=200, depth=2, **kw):
    return tcb.BeamSearch(None, R, n, V, depth=depth, device="cpu", **kw)


def _head(V=200, d=256, max_rows=8, **kw):
    return tcb.LmheadFp8(torch.zeros((V, d), dtype=torch.bfloat16),
                         torch.ones(d, dtype=torch.bfloat16), max_rows, **kw)


def _rows(m, d=256):
    return torch.zeros((m, d), dtype=torch.bfloat16)


@pytest.mark.parametrize("temperature", [0.0, 0.7])
def test_step_hidden_reports_in_the_searchs_status_word(calls, temperature):
    """A product that gave up leaves logits of an earlier call: the status word that
    a user of the search reads has to say so."""
    search, head = _search(temperature=temperature), _head()
    search.step_hidden(0, head, _rows(2))
    assert int(search.workspace[0]) == TIMEOUT_BIT
    assert [c[0] for c in calls][-1] == ("beam_step_gumbel" if temperature else "beam_step")


def test_logits_alone_report_in_the_heads_status_word(calls):
    head = _head()
    head.logits(_rows(3))
    assert int(head.workspace[0]) == TIMEOUT_BIT
    own = torch.zeros(256, dtype=torch.uint8)
    head.workspace.zero_()
    head.logits(_rows(3), workspace=own)
    assert int(own[0]) == TIMEOUT_BIT and int(head.workspace[0]) == 0


def test_step_hidden_refuses_what_the_step_would_read_past(calls):
    """beam_step reads rows(t) rows of V[t] logits: fewer rows than that, or a head
    of fewer codes, would leave it with rows and columns that nothing has written
    (past the buffer's end, where max_rows is smaller too)."""
    search, head = _search(R=2, n=4, V=[200, 204]), _head(V=200, max_rows=8)
    done = len(calls)
    with pytest.raises(ValueError, match="rows"):
        search.step_hidden(0, head, _rows(1))
    with pytest.raises(ValueError, match="rows"):
        search.step_hidden(1, _head(V=204, max_rows=2), _rows(2))
    with pytest.raises(ValueError, match="codes"):
        search.step_hidden(1, head, _rows(8))
    assert all(c[0] == "lmhead_quantize_fp8" for c in calls[done:])   # nothing was launched
    # A padded batch and a head of more codes are fine: the step reads the first of them.
    search.step_hidden(0, head, _rows(5))
    search.step_hidden(1, _head(V=300), _rows(8))
    logits = calls[-1][1][2]
    assert logits.shape == (8, 300) and logits.stride() == (304, 1)


def test_head_allocates_on_the_stream_it_quantises_on(calls, monkeypatch):
    """Buffers made on the current stream and written by another one could be memory
    that work queued on the current stream still uses, and a status word that is not
    cleared yet: with a stream given, all of a head's buffers are that stream's."""
    import contextlib
    entered, made = [], []

    @contextlib.contextmanager
    def on(stream):
        entered.append(stream)
        yield
        entered.pop()
    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("empty", "zeros"):
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _make=make, **kw: (
            made.append(entered[-1] if entered else None), _make(*a, **kw))[1])
    w, norm = torch.ones((200, 256), dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    tcb.LmheadFp8(w, norm, 8, stream="side")
    assert len(made) == 6 and set(made) == {"side"}
    assert calls[-1][0] == "lmhead_quantize_fp8" and calls[-1][2]["stream"] == "side"
    made.clear()
    tcb.LmheadFp8(w, norm, 8)
    assert set(made) == {None}


def test_search_steps_on_its_own_device(calls, monkeypatch):
    """With another device current, attention and the 8-bit product run on the device of
    their tensors; the constrained step and the end must follow them there (on the
    current device they would read another device's memory, in no order)."""
    entered, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)

        def __exit__(self, *exc):
            entered.pop()
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: entered[-1])
    for name in ("beam_step", "beam_step_gumbel", "beam_finalize"):
        monkeypatch.setattr(native, name, lambda *a, _name=name, **kw: seen.append((_name, entered[-1])))
    for temperature, step in ((0.0, "beam_step"), (0.5, "beam_step_gumbel")):
        search, head = _search(temperature=temperature), _head()
        search.device_index = 1
        for t in range(2):
            search.step_hidden(t, head, _rows(search.rows(t)))
        search.step(1, head._logits)
        search.finalize()
        assert entered == [0]
        assert seen == [(step, 1)] * 3 + [("beam_finalize", 1)]
        seen.clear()
    seen.clear()
    search.device_index = 0     # already current: nothing is switched
    monkeypatch.setattr(Device, "__enter__", None)
    search.step(1, head._logits)
    search.finalize()
    assert [x[1] for x in seen] == [0, 0]
