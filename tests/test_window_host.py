"""Host-only checks of the windowed attention and rotary calls: argument errors are found before
any CUDA call, the frequency rules, and the binding's own checks."""

import ctypes
import math
import re

import numpy as np
import pytest
import torch

import context_long_sequence_non_b200 as cp
from context_long_sequence_non_b200 import _binding as B
from context_long_sequence_non_b200 import build as build_mod

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails validation
BIG = 1 << 24
bf = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


def window(L, q=FAKE, k=FAKE + BIG, v=FAKE + 2 * BIG, o=FAKE + 3 * BIG, lse=FAKE + 4 * BIG, kv_len=None, run=None,
           B_=1, H=4, Hkv=2, Sq=8, Skv=8, D=128, qs=0, ks=0, vs=0, scale=0.1, q_pos=0, k_pos=0, left=3,
           right=0, sinks=0, din=0, dout=0, acc=0):
    return L.cpattn_window_fwd(q, k, v, o, lse, kv_len, run, B_, H, Hkv, Sq, Skv, D, qs, ks, vs, scale, q_pos,
                               k_pos, left, right, sinks, din, dout, acc, None)


def decode(L, q=FAKE, k=FAKE + BIG, v=FAKE + 2 * BIG, kv_len=FAKE + 5 * BIG, o=FAKE + 3 * BIG,
           lse=FAKE + 4 * BIG, B_=1, H=4, Hkv=2, Sq=1, S=8, D=128, qs=0, ks=0, vs=0, scale=0.1, left=3,
           sinks=0, din=0, dout=0):
    return L.cpattn_window_decode(q, k, v, kv_len, o, lse, B_, H, Hkv, Sq, S, D, qs, ks, vs, scale, left,
                                  sinks, din, dout, None)


@pytest.mark.parametrize("call", [window, decode])
def test_window_argument_errors(L, call):
    assert call(L, B_=0) == B.ERR_SHAPE
    assert call(L, Sq=0) == B.ERR_SHAPE
    assert call(L, D=0) == B.ERR_SHAPE
    assert call(L, H=5) == B.ERR_SHAPE  # not a multiple of the key heads
    assert call(L, Hkv=0) == B.ERR_SHAPE
    assert call(L, B_=70000) == B.ERR_SHAPE
    assert call(L, Sq=1 << 30) == B.ERR_SHAPE
    assert call(L, B_=60000, Sq=60000) == B.ERR_SHAPE  # 32-bit row index
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(L, scale=scale) == B.ERR_SHAPE
    assert call(L, sinks=-1) == B.ERR_SHAPE
    assert call(L, din=7) == B.ERR_UNSUPPORTED
    assert call(L, dout=7) == B.ERR_UNSUPPORTED
    assert call(L, D=96) == B.ERR_UNSUPPORTED
    assert call(L, D=264, din=1, dout=1) == B.ERR_UNSUPPORTED
    assert call(L, q=None) == B.ERR_NULL
    assert call(L, k=None) == B.ERR_NULL
    assert call(L, v=None) == B.ERR_NULL
    assert call(L, o=None) == B.ERR_NULL
    assert call(L, q=FAKE + 8) == B.ERR_ALIGN
    assert call(L, k=FAKE + BIG + 2) == B.ERR_ALIGN
    assert call(L, lse=FAKE + 4 * BIG + 2) == B.ERR_ALIGN
    assert call(L, kv_len=FAKE + 5 * BIG + 1) == B.ERR_ALIGN
    assert call(L, qs=511) == B.ERR_SHAPE  # shorter than a token's heads
    assert call(L, ks=255) == B.ERR_SHAPE
    assert call(L, vs=1 << 40) == B.ERR_SHAPE
    for big in (1 << 39, 1 << 62):  # batches or tokens too far apart
        assert call(L, ks=big) == B.ERR_SHAPE
        assert call(L, qs=big, B_=2, Sq=3) == B.ERR_SHAPE
    assert call(L, vs=1 << 38, B_=2) == B.ERR_SHAPE
    assert call(L, qs=516) == B.ERR_ALIGN  # bf16 rows start on 16 bytes
    assert call(L, o=FAKE) == B.ERR_SHAPE  # out over q
    assert call(L, o=FAKE + BIG + 16) == B.ERR_SHAPE  # out over k
    assert call(L, lse=FAKE + 2 * BIG) == B.ERR_SHAPE  # lse over v
    assert call(L, lse=FAKE + 3 * BIG) == B.ERR_SHAPE  # lse over out
    assert call(L, kv_len=FAKE + 3 * BIG) == B.ERR_SHAPE  # out over the lengths


def test_window_position_errors(L):
    assert window(L, q_pos=-1) == B.ERR_SHAPE
    assert window(L, k_pos=-1) == B.ERR_SHAPE
    assert window(L, q_pos=(1 << 30) - 8) == B.ERR_SHAPE
    assert window(L, k_pos=(1 << 30) - 8) == B.ERR_SHAPE
    assert window(L, Skv=-1) == B.ERR_SHAPE
    assert window(L, acc=1, lse=None) == B.ERR_NULL
    assert window(L, acc=1, din=1, dout=1) == B.ERR_UNSUPPORTED
    assert decode(L, S=0) == B.ERR_SHAPE
    assert window(L, run=FAKE + 6 * BIG) == B.ERR_UNSUPPORTED  # not an accumulating call
    assert window(L, run=FAKE + 6 * BIG, acc=1, dout=1) == B.ERR_UNSUPPORTED
    assert window(L, run=FAKE + 6 * BIG + 4, acc=1) == B.ERR_ALIGN
    assert window(L, run=FAKE + 3 * BIG, acc=1) == B.ERR_SHAPE  # the running O over out
    assert window(L, run=FAKE + 4 * BIG, acc=1) == B.ERR_SHAPE  # and over lse
    # a chunk that no row sees leaves a running result alone: nothing is launched
    assert window(L, acc=1, q_pos=100, left=3, right=0) == B.OK
    assert window(L, acc=1, k_pos=100, left=3, right=0) == B.OK
    assert window(L, acc=1, Skv=0) == B.OK


def rope(L, x=FAKE, y=FAKE + BIG, pos=FAKE + 2 * BIG, freq=FAKE + 3 * BIG, T=8, rows=8, H=2, D=128, rot=128,
         axes=1, inter=0, factor=1.0, xs=0, ys=0, dt=0):
    return L.cpattn_rope(x, y, pos, freq, T, rows, H, D, rot, axes, inter, factor, xs, ys, dt, None)


def test_rope_argument_errors(L):
    assert rope(L, T=-1) == B.ERR_SHAPE
    assert rope(L, D=0) == B.ERR_SHAPE
    assert rope(L, D=258, rot=2) == B.ERR_SHAPE
    assert rope(L, rot=0) == B.ERR_SHAPE
    assert rope(L, rot=63) == B.ERR_SHAPE
    assert rope(L, rot=130) == B.ERR_SHAPE
    assert rope(L, axes=0) == B.ERR_SHAPE
    assert rope(L, axes=5) == B.ERR_SHAPE
    assert rope(L, factor=float("nan")) == B.ERR_SHAPE
    assert rope(L, dt=3) == B.ERR_UNSUPPORTED
    assert rope(L, H=0) == B.ERR_SHAPE
    assert rope(L, rows=3) == B.ERR_SHAPE
    assert rope(L, rows=0) == B.ERR_SHAPE
    assert rope(L, T=1 << 30, H=4) == B.ERR_SHAPE
    assert rope(L, xs=255) == B.ERR_SHAPE
    assert rope(L, ys=255) == B.ERR_SHAPE
    assert rope(L, xs=1 << 30) == B.ERR_SHAPE
    assert rope(L, ys=1 << 62) == B.ERR_SHAPE
    assert rope(L, x=None) == B.ERR_NULL
    assert rope(L, y=None) == B.ERR_NULL
    assert rope(L, pos=None) == B.ERR_NULL
    assert rope(L, freq=None) == B.ERR_NULL
    assert rope(L, x=FAKE + 8) == B.ERR_ALIGN
    assert rope(L, pos=FAKE + 2 * BIG + 2) == B.ERR_ALIGN
    assert rope(L, freq=FAKE + 3 * BIG + 4) == B.ERR_ALIGN
    assert rope(L, y=FAKE + 16) == B.ERR_SHAPE  # overlapping, not in place
    assert rope(L, y=FAKE, ys=512) == B.ERR_SHAPE  # in place with another stride
    assert rope(L, y=FAKE + 2 * BIG) == B.ERR_SHAPE  # over pos
    assert rope(L, y=FAKE + 3 * BIG) == B.ERR_SHAPE  # over freq
    assert rope(L, T=0, x=None, y=None, pos=None, freq=None) == B.OK


def qk(L, q=FAKE, k=FAKE + BIG, qo=FAKE + 2 * BIG, ko=FAKE + 3 * BIG, gq=FAKE + 4 * BIG, gk=FAKE + 5 * BIG,
       T=8, Hq=4, Hk=2, D=64, rot=64, eps=1e-6, out_scale=1.0, qs=0, ks=0, qos=0, kos=0):
    return L.cpattn_qk_norm_rope(q, k, qo, ko, gq, gk, FAKE + 6 * BIG, FAKE + 7 * BIG, T, T, Hq, Hk, D, rot, 1,
                                 0, eps, out_scale, 1.0, qs, ks, qos, kos, 0, None)


def test_qk_norm_rope_argument_errors(L):
    assert qk(L, eps=-1.0) == B.ERR_SHAPE
    assert qk(L, eps=float("inf")) == B.ERR_SHAPE
    assert qk(L, out_scale=float("nan")) == B.ERR_SHAPE
    assert qk(L, gq=None) == B.ERR_NULL
    assert qk(L, gk=None) == B.ERR_NULL
    assert qk(L, gk=FAKE + 5 * BIG + 4) == B.ERR_ALIGN
    assert qk(L, qo=FAKE + BIG) == B.ERR_SHAPE  # q's output over k
    assert qk(L, qo=FAKE + 3 * BIG) == B.ERR_SHAPE  # the two outputs together
    assert qk(L, qo=FAKE + 4 * BIG) == B.ERR_SHAPE  # over the weights
    # heads of one row: q's 4 and k's 2 heads of 64 in rows of 512; k's output one element into
    # q's heads
    row = 512
    assert qk(L, q=FAKE, k=FAKE + 512, qo=FAKE, ko=FAKE + 496, qs=row, ks=row, qos=row, kos=row) == B.ERR_SHAPE
    assert qk(L, q=FAKE, k=FAKE + 512, qo=FAKE + 512, ko=FAKE, qs=row, ks=row, qos=row, kos=row) == B.ERR_SHAPE


def s2h(L, q=FAKE, k=FAKE + BIG, v=FAKE + 2 * BIG, qh=FAKE + 3 * BIG, kh=FAKE + 4 * BIG, vh=FAKE + 5 * BIG,
        gq=FAKE + 6 * BIG, gk=FAKE + 7 * BIG, P=2, S=3, H=4, D=64, rot=64):
    return L.cpattn_seq2head_qkv_norm_rope(q, k, v, qh, kh, vh, gq, gk, FAKE + 8 * BIG, FAKE + 9 * BIG, P, S, H,
                                           D, rot, 1, 0, 1e-6, 1.0, 1.0, None)


def test_seq2head_norm_rope_argument_errors(L):
    assert s2h(L, P=0) == B.ERR_SHAPE
    assert s2h(L, P=3) == B.ERR_SHAPE
    assert s2h(L, S=0) == B.ERR_SHAPE
    assert s2h(L, D=4, rot=4, H=2) == B.ERR_SHAPE  # a run of 8 bytes
    assert s2h(L, gq=None) == B.ERR_NULL
    assert s2h(L, v=None) == B.ERR_NULL
    assert s2h(L, vh=FAKE) == B.ERR_SHAPE  # over an input
    assert s2h(L, kh=FAKE + 3 * BIG) == B.ERR_SHAPE  # over another output
    assert s2h(L, qh=FAKE + 3 * BIG + 2) == B.ERR_ALIGN


def test_frequencies(L):
    f, a = cp.rope_frequencies(8, base=100.0)
    assert f.dtype == torch.float64 and a == 1.0
    np.testing.assert_allclose(f, 100.0 ** (-np.arange(4) / 4), rtol=1e-15)
    f2, a = cp.rope_frequencies(8, base=100.0, scaling="linear", stretch=4.0)
    np.testing.assert_allclose(f2, f / 4, rtol=1e-15)
    f3, _ = cp.rope_frequencies(8, base=100.0, scaling="ntk", stretch=4.0)
    np.testing.assert_allclose(f3[0], f[0], rtol=1e-15)
    np.testing.assert_allclose(f3[-1], f[-1] / 4, rtol=1e-14)  # (100 * 4^(8/6))^(-6/8) = 100^(-6/8) / 4
    f4, a = cp.rope_frequencies(64, scaling="by_parts", stretch=8.0, train_len=4096)
    f0, _ = cp.rope_frequencies(64)
    turns = 4096 * f0 / (2 * math.pi)
    assert torch.equal(f4[turns >= 32], f0[turns >= 32])
    np.testing.assert_allclose(f4[turns <= 1], f0[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((f4 < f0) & (f4 > f0 / 8))[mid].all()
    assert a == pytest.approx(0.1 * math.log(8) + 1, rel=1e-7)
    ax = cp.rope_axes([f, f2[:2]])
    assert ax.shape == (2, 6) and torch.equal(ax[0, :4], f) and ax[0, 4:].sum() == 0 and torch.equal(ax[1, 4:], f2[:2])


def test_frequency_errors(L):
    for kw in (dict(rot=0), dict(rot=7), dict(rot=258), dict(base=1.0), dict(base=math.nan),
               dict(scaling="linear", stretch=0.5), dict(scaling="ntk", stretch=2.0, rot=2),
               dict(scaling="by_parts", stretch=2.0), dict(scaling="by_parts", stretch=2.0, train_len=10.0,
                                                           beta_fast=1.0, beta_slow=1.0)):
        kw = {"rot": 8, **kw}
        with pytest.raises(cp.CpattnError, match="SHAPE"):
            cp.rope_frequencies(**kw)
    with pytest.raises(ValueError, match="scaling"):
        cp.rope_frequencies(8, scaling="other")
    assert L.cpattn_rope_frequencies(None, None, 8, 100.0, 0, 1.0, 0.0, 0.0, 0.0) == B.ERR_NULL
    buf = (ctypes.c_double * 4)()
    assert L.cpattn_rope_frequencies(ctypes.addressof(buf), None, 8, 100.0, 4, 1.0, 0.0, 0.0, 0.0) == B.ERR_UNSUPPORTED


def t(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def test_window_binding_checks():
    q, k, v = t(2, 5, 4, 64), t(2, 9, 2, 64), t(2, 9, 2, 64)
    with pytest.raises(ValueError, match="k and v"):
        cp.window_fwd(q, k, t(2, 8, 2, 64))
    with pytest.raises(ValueError, match="one dtype"):
        cp.window_fwd(q, k, v.float())
    with pytest.raises(ValueError, match="out must have shape"):
        cp.window_fwd(q, k, v, out=t(2, 5, 4, 128))
    with pytest.raises(ValueError, match="lse must be"):
        cp.window_fwd(q, k, v, lse=t(2, 4, 5))
    with pytest.raises(ValueError, match="kv_len must be"):
        cp.window_fwd(q, k, v, kv_len=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="kv_len must have shape"):
        cp.window_decode(q, k, v, kv_len=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="running"):
        cp.window_fwd(q, k, v, accumulate=True)
    with pytest.raises(ValueError, match="accumulating"):
        cp.window_fwd(q, k, v, run=q.float())
    with pytest.raises(ValueError, match="run must be"):
        cp.window_fwd(q, k, v, run=q, accumulate=True, lse=t(2, 4, 5, dtype=torch.float32))
    with pytest.raises(ValueError, match="heads must be contiguous"):
        cp.window_fwd(t(2, 4, 5, 64).transpose(1, 2), k, v)
    with pytest.raises(ValueError, match="evenly spaced"):
        cp.window_fwd(q, t(2, 12, 2, 64)[:, :9], v)
    with pytest.raises(ValueError, match="out must be contiguous"):
        cp.window_fwd(q, k, v, out=t(2, 5, 8, 64)[:, :, :4])
    with pytest.raises(ValueError, match="CUDA"):
        cp.window_fwd(q, k, v)


def test_token_strides():
    ts = lambda x: B._token_stride(x, "x")
    assert ts(t(2, 5, 4, 64)) == 0  # packed
    assert ts(t(2, 5, 12, 64)[:, :, 4:8]) == 768
    assert ts(t(7, 12, 64)[:, :1]) == 768
    assert ts(t(1, 1, 12, 64)[:, :, :4]) == 0  # one token: any spacing will do
    assert ts(t(4, 9, 2, 64)[1:2, 3:]) == 0
    assert ts(t(0, 2, 64)) == 0
    assert ts(t(0, 12, 64)[:, :4]) == 0
    for bad in (t(2, 5, 64, 4).transpose(2, 3), t(1, 2, 64).expand(3, 2, 64), t(5, 2, 4, 64).transpose(0, 1),
                t(3, 6, 2, 64)[:, ::2].flip(0)[:, :2]):
        with pytest.raises(ValueError):
            ts(bad)


def test_rope_binding_checks():
    f = torch.ones(32, dtype=torch.float64)
    x = t(3, 5, 2, 64)
    with pytest.raises(ValueError, match="float64"):
        cp.rope(x, torch.zeros(5, dtype=torch.int32), f.float())
    with pytest.raises(ValueError, match="int32"):
        cp.rope(x, torch.zeros(5, dtype=torch.int64), f)
    with pytest.raises(ValueError, match="multiple"):
        cp.rope(x, torch.zeros(4, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="matching freq"):
        cp.rope(x, torch.zeros(5, 2, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="matching freq"):
        cp.rope(x, torch.zeros(10, dtype=torch.int32), f.repeat(2, 1))
    with pytest.raises(ValueError, match="out must have shape"):
        cp.rope(x, torch.zeros(5, dtype=torch.int32), f, out=t(3, 5, 2, 32))
    with pytest.raises(ValueError, match="same tokens"):
        cp.qk_norm_rope(x, t(3, 4, 2, 64), None, None, torch.zeros(5, dtype=torch.int32), f)
    g = torch.ones(64)
    with pytest.raises(ValueError, match="gamma"):
        cp.qk_norm_rope(x, x, g[:32], g, torch.zeros(5, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="go together"):
        cp.seq2head_qkv_norm_rope(x, x, x, 3, g, None, torch.zeros(15, dtype=torch.int32), f)
    s = t(2, 5, 4, 64)
    with pytest.raises(ValueError, match="every token"):
        cp.seq2head_qkv_norm_rope(s, s, s, 2, g, g, torch.zeros(5, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="ring step"):
        cp.ring_attention(s, [s], [s], left=3, fused=False)
    with pytest.raises(ValueError, match="needs chunks"):
        cp.ring_attention(s, [], [], left=3)
    with pytest.raises(ValueError, match="needs chunks"):
        cp.ring_attention(s, [s], [s], left=3, k_pos=[0, 5])


# ------------------------------------------------------------------ calls by number

def test_calls_by_number_reach_the_same_checks(L):
    w = [FAKE, FAKE + BIG, FAKE + 2 * BIG, FAKE + 3 * BIG, FAKE + 4 * BIG, 0, 0,
         1, 4, 2, 8, 8, 128, 0, 0, 0, 0.1, 0, 0, 3, 0, 0, 0, 0, 0, 0]
    good = B._WINDOW_FWD
    assert good.n == len(w) == len(L.cpattn_window_fwd.argtypes)
    for at, value, status in ((7, 0, B.ERR_SHAPE), (8, 5, B.ERR_SHAPE), (12, 96, B.ERR_UNSUPPORTED), (0, 0, B.ERR_NULL),
                              (1, FAKE + 8, B.ERR_ALIGN), (16, -1.0, B.ERR_SHAPE), (16, math.nan, B.ERR_SHAPE),
                              (10, (1 << 32) + 8, B.ERR_SHAPE),  # not cut to an int of 8
                              (19, -(1 << 40), B.ERR_SHAPE), (13, 1 << 62, B.ERR_SHAPE), (13, -1, B.ERR_SHAPE),
                              (22, 7, B.ERR_UNSUPPORTED)):
        bad = list(w)
        bad[at] = value
        assert L.cpattn_call(good.code, good.pack(*bad), good.n) == status, (at, value)
        if abs(value) < 1 << 31 or at == 13:
            assert L.cpattn_window_fwd(*bad[:5], None, None, *bad[7:25], None) == status, (at, value)


def test_calls_by_number_match_the_declared_arguments(L):
    kinds = {"P": ctypes.c_void_p, "d": ctypes.c_float}
    for e, layout in ((B._WINDOW_FWD, "7P9qd8qP"), (B._WINDOW_DECODE, "6P9qd4qP"), (B._ROPE, "4P7qd3qP"),
                      (B._QK_NORM_ROPE, "8P8q3d5qP"), (B._SEQ2HEAD_QKV_NORM_ROPE, "10P7q3dP")):
        flat = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([Pqd])", layout))
        declared = getattr(L, e.name).argtypes
        assert len(flat) == e.n == len(declared)
        for c, t in zip(flat, declared):
            assert t is kinds[c] if c in kinds else t in (ctypes.c_int, ctypes.c_longlong)
        zero = e.pack(*(0.0 if c == "d" else 0 for c in flat))
        assert L.cpattn_call(e.code, zero, e.n) == B.ERR_SHAPE  # no sizes
        assert L.cpattn_call(e.code, zero, e.n - 1) == B.ERR_SHAPE
        assert L.cpattn_call(e.code, zero, e.n + 1) == B.ERR_SHAPE
        assert L.cpattn_call(e.code, None, e.n) == B.ERR_NULL
    for code in (-1, 5, 1 << 30):
        assert L.cpattn_call(code, zero, 4) == B.ERR_SHAPE


# ------------------------------------------------------------------ ring step, float32

def test_float32_windowed_ring_step_folds_its_chunks_with_merge(monkeypatch):
    # the accumulating windowed call takes bf16 only: every chunk is a call of its own, then a merge
    calls = []
    monkeypatch.setattr(B, "window_fwd", lambda *a, **kw: calls.append(("window", kw["out"], kw.get("accumulate", False))))
    monkeypatch.setattr(B, "merge", lambda *a, **kw: calls.append(("merge", a[0], kw["out"])))
    q, k = t(1, 5, 4, 64, dtype=torch.float32), t(1, 6, 2, 64, dtype=torch.float32)
    for acc_dtype in (None, torch.float32, bf):
        calls.clear()
        out, _ = cp.ring_attention(q, [k, k, k], [k, k, k], left=3, acc_dtype=acc_dtype)
        assert out.dtype == (acc_dtype or torch.float32)
        assert [c[0] for c in calls] == ["window", "window", "merge", "window", "merge"]
        assert calls[0][1] is out and all(c[1] is out and c[2] is out for c in calls if c[0] == "merge")
        assert not any(c[2] for c in calls if c[0] == "window")
    calls.clear()
    cp.ring_attention(q, [k], [k], left=3)
    assert [c[0] for c in calls] == ["window"]


def test_float32_windowed_ring_step_refuses_rows_that_merge_does_not_take(monkeypatch):
    def launch(*a, **kw):
        raise AssertionError("launched")

    monkeypatch.setattr(B, "window_fwd", launch)
    for D, acc_dtype in ((30, None), (7, torch.float32), (44, bf)):
        q, k = t(1, 5, 4, D, dtype=torch.float32), t(1, 6, 2, D, dtype=torch.float32)
        with pytest.raises(ValueError, match="16 bytes"):
            cp.ring_attention(q, [k, k], [k, k], left=3, acc_dtype=acc_dtype)
