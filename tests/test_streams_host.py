"""Buffers that a call allocates itself, when the call runs on another stream than the current one: they
must come from that stream's memory.  Taken from the current stream's, they could be memory that work
queued there still uses, and would go to its next allocation as soon as Python drops them -- a temporary
at the return, an LSE that the caller does not keep -- both while the call runs.  Results must be marked
as used on the current stream too, where the caller reads them.  Streams and allocations are stand-ins
here; nothing runs."""

import contextlib

import pytest
import torch

import context_long_sequence_non_b200 as cp
from context_long_sequence_non_b200 import _binding as B
from context_long_sequence_non_b200 import paths

MAIN, SIDE = "main", "side"


class Library:
    def __getattr__(self, name):
        return lambda *a: 1024 if "workspace" in name else 0


@pytest.fixture
def log(monkeypatch):
    """Allocations as (stream, tensor) and marks as (tensor, stream)."""
    current = [MAIN]
    made, marked = [], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream if stream is not None else current[-1])
        yield
        current.pop()

    def logged(fn):
        def alloc(*a, **kw):
            t = fn(*a, **kw)
            made.append((current[-1], t))
            return t
        return alloc

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    for name in ("empty", "empty_like", "empty_strided"):
        monkeypatch.setattr(torch, name, logged(getattr(torch, name)))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: marked.append((t, s)))
    monkeypatch.setattr(B, "lib", Library)
    monkeypatch.setattr(B, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(B, "_stream", lambda stream: stream)
    monkeypatch.setattr(B, "_same_device", lambda *ts: 0)
    monkeypatch.setattr(B, "_call", lambda *a: None)
    return made, marked


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


q, k = t(1, 6, 4, 64), t(1, 8, 4, 64)
s = t(2, 3, 4, 64)  # [P][S_l][H][D]
gam = torch.ones(64)
pos, freq = torch.arange(6, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
chunks = dict(k_chunks=[k, k, k], v_chunks=[k, k, k])
heads = lambda *ts: tuple(x[0] for x in ts)
f32 = torch.zeros(1, 4, 6)

CALLS = {
    "fwd": lambda **kw: B.fwd(q, k, k, **kw),
    "ulysses_fwd": lambda **kw: B.ulysses_fwd(s, s, s, 2, **kw),
    "ulysses_fwd_split": lambda **kw: B.ulysses_fwd_split(s, s, s, 2, **kw),
    "fwd_split": lambda **kw: B.fwd_split(q, k, k, n_split=2, **kw),
    "merge": lambda **kw: B.merge(q, f32, q, f32, **kw),
    "seq2head": lambda **kw: (B.seq2head(s, 2, **kw),),
    "seq2head_qkv": lambda **kw: B.seq2head_qkv(s, s, s, 2, **kw),
    "head2seq": lambda **kw: (B.head2seq(t(2, 6, 2, 64), 2, **kw),),
    "rmsnorm": lambda **kw: (B.rmsnorm(q, gam, **kw),),
    "seq2head_qkv_norm": lambda **kw: B.seq2head_qkv_norm(s, s, s, 2, gam, gam, **kw),
    "window_fwd": lambda **kw: B.window_fwd(q, k, k, left=2, **kw),
    "window_decode": lambda **kw: B.window_decode(q, k, k, left=2, **kw),
    "rope": lambda **kw: (B.rope(q, pos, freq, **kw),),
    "qk_norm_rope": lambda **kw: B.qk_norm_rope(q, q, gam, gam, pos, freq, **kw),
    "seq2head_qkv_norm_rope": lambda **kw: B.seq2head_qkv_norm_rope(s, s, s, 2, gam, gam, pos, freq, **kw),
    "selftest_exp2": lambda **kw: (B.selftest_exp2(f32, **kw),),
    "ring": lambda **kw: paths.ring_attention(q, **chunks, **kw),
    "ring, separate merges": lambda **kw: paths.ring_attention(q, **chunks, fused=False, **kw),
    "ring, keys in parts": lambda **kw: paths.ring_attention(q, **chunks, n_split=2, **kw),
    "ring, windowed": lambda **kw: paths.ring_attention(q, **chunks, left=2, **kw),
    "ulysses": lambda **kw: paths.ulysses_attention(s, s, s, 2, **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_belong_to_the_stream_of_the_call(log, name):
    made, marked = log
    res = CALLS[name](stream=SIDE)
    assert made and all(stream == SIDE for stream, _ in made)
    for r in res:
        assert any(r is x and stream == MAIN for x, stream in marked)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [None, MAIN])
def test_calls_on_the_current_stream_mark_nothing(log, name, stream):
    made, marked = log
    CALLS[name](stream=stream)
    assert made and all(st == MAIN for st, _ in made) and not marked


def test_a_split_ring_step_clears_its_accumulator_on_its_stream(log, monkeypatch):
    seen = []
    fill = torch.Tensor.fill_
    monkeypatch.setattr(torch.Tensor, "fill_", lambda x, v: (seen.append(torch.cuda.current_stream()), fill(x, v))[1])
    cp.ring_attention(q, **chunks, n_split=2, stream=SIDE)
    assert seen == [SIDE]
