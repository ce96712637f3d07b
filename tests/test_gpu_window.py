"""GPU parity of the windowed attention (cpattn_window_fwd) and its single-token form
(cpattn_window_decode) against the fp64 oracle.

Bounds, from the arithmetic.  With A = sum_j w_j |v_j| (w the softmax weights): the kernel rounds
each weight to bf16, off by at most half a step, 2^-8 of it; its exponential is within 2e-5 of the
value; the logits are sums of D fp32 products, off by at most D 2^-24 sum_d |q_d k_d| scale =: S
each, which changes a weight by the factor e^(2S) at most.  So |O err| <= (2^-8 + 2e-5 + 2S) A in
fp32, and a bf16 O adds half a step, 2^-8 of its value; a running bf16 O adds another for each
merge, and each merge is off by the weights' own few fp32 steps.  |LSE err| <= S + 2e-5 + 2^-22 |LSE|.
The fp32 kernel has no rounding to bf16: |O err| <= (2e-6 + 2S + n 2^-24) A over n keys.
"""

import math
import warnings

import numpy as np
import pytest
import torch

import context_long_sequence_non_b200 as cp
from context_long_sequence_non_b200 import build as build_mod
from context_long_sequence_non_b200.paths import UlyssesPlan
from oracle import window as ow
from oracle.ref import _f64

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = 2.0 ** -8  # half a bf16 step, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build_mod.build()
    cp.lib()
    yield
    assert cp.device_error() == 0


def make(seed, B, H, Hkv, Sq, Skv, D, dtype=torch.bfloat16, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=g) * sigma).to(dtype)
    return r(B, Sq, H, D), r(B, Skv, Hkv, D), r(B, Skv, Hkv, D)


def logit_error(q, k, scale):
    """S: fp32 summation error of a logit, at most (|q|.|k| <= |q||k|)."""
    qn = np.sqrt((_f64(q) ** 2).sum(-1)).max(initial=0.0)
    kk = np.nan_to_num(_f64(k), nan=0.0, posinf=0.0, neginf=0.0)
    kn = np.sqrt((kk ** 2).sum(-1)).max(initial=0.0)
    return q.shape[-1] * 2.0 ** -24 * qn * kn * scale


def check(out, lse, ref, q, k, scale, merges=0, n=0):
    o_ref, l_ref, a = ref
    o, l = _f64(out), _f64(lse) if lse is not None else None
    S = logit_error(q, k, scale)
    if q.dtype == torch.float32:
        bound = (2e-6 + 2 * S + n * 2.0 ** -24) * a
    else:
        bound = (HALF + 2e-5 + 2 * S) * a + 1e-6 * merges * a
    if out.dtype == torch.bfloat16:
        bound = bound + HALF * (1 + merges) * (np.abs(o_ref) + bound)
    assert np.isfinite(o).all(), "non-finite output"
    err = np.abs(o - o_ref) - bound
    assert err.max() <= 1e-30, f"O off by {np.abs(o - o_ref).max():.3e}, bound exceeded by {err.max():.3e}"
    if l is not None:
        empty = np.isneginf(l_ref)
        assert np.array_equal(np.isneginf(l), empty)
        d = np.abs(l[~empty] - l_ref[~empty]) - (S + 2e-5 + 2.0 ** -22 * np.abs(l_ref[~empty])) * (1 + merges)
        assert d.size == 0 or d.max() <= 0, f"LSE bound exceeded by {d.max():.3e}"


def run_window(q, k, v, kv_len=None, out_dtype=None, **kw):
    scale = kw.pop("scale", 1 / math.sqrt(q.shape[-1]))
    kl = None if kv_len is None else torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    out, lse = cp.window_fwd(q.to(DEV), k.to(DEV), v.to(DEV), kv_len=kl, scale=scale, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    ref = ow.window_attention(q, k, v, scale, kv_len=kv_len, **kw)
    check(out, lse, ref, q, k, scale, n=k.shape[1])
    return out, lse


WINDOWS = [dict(left=-1, right=-1), dict(left=-1, right=0), dict(left=0, right=0), dict(left=100, right=0, sinks=4),
           dict(left=63, right=64), dict(left=300, right=17, sinks=130), dict(left=5, right=-1, sinks=1),
           dict(left=1 << 30, right=1 << 30, sinks=1 << 30), dict(left=127, right=0, sinks=128)]


@pytest.mark.parametrize("w", WINDOWS, ids=lambda w: "-".join(map(str, w.values())))
@pytest.mark.parametrize("D,H,Hkv", [(128, 2, 2), (64, 6, 2)])
def test_square(w, D, H, Hkv):
    q, k, v = make(D + len(w), 1, H, Hkv, 700, 700, D)
    run_window(q, k, v, **w)


@pytest.mark.parametrize("Sq,Skv,q_pos,k_pos,w", [
    (1, 1, 0, 0, dict(left=0, right=0)), (1, 1000, 999, 0, dict(left=77, right=0, sinks=3)),
    (129, 300, 171, 0, dict(left=64, right=0, sinks=5)), (255, 513, 300, 40, dict(left=90, right=33, sinks=50)),
    (256, 128, 0, 128, dict(left=-1, right=0)), (300, 200, 1000, 0, dict(left=850, right=10, sinks=2)),
    (200, 300, 0, 100, dict(left=20, right=30)), (100, 64, 0, 4000, dict(left=5, right=5)),
    (400, 640, 500000000, 499999800, dict(left=111, right=222, sinks=499999900)),
    (513, 1, 0, 0, dict(left=256, right=0)), (257, 900, 10, 0, dict(left=1, right=600, sinks=1)),
    (64, 2000, 1900, 0, dict(left=3, right=0, sinks=700))])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_slices_and_positions(Sq, Skv, q_pos, k_pos, w, out_dtype):
    q, k, v = make(Sq + Skv, 2, 4, 2, Sq, Skv, 128)
    run_window(q, k, v, q_pos=q_pos, k_pos=k_pos, out_dtype=out_dtype, **w)


def test_rows_without_keys():
    # rows 0..99 of the slice are behind every key; rows 140 on are past the window
    q, k, v = make(3, 1, 2, 1, 300, 60, 64)
    out, lse = run_window(q, k, v, left=40, right=0, q_pos=0, k_pos=100)
    assert torch.isneginf(lse[0, :, :100]).all() and (out[0, :100] == 0).all()
    assert torch.isneginf(lse[0, :, 200:]).all() and torch.isfinite(lse[0, :, 100:199]).all()
    # no keys at all
    out, lse = run_window(q, k[:, :0], v[:, :0], left=3, right=3)
    assert torch.isneginf(lse).all() and (out == 0).all()


def test_very_negative_and_large_logits():
    q, k, v = make(4, 1, 2, 2, 300, 300, 128)
    q[:, :, :, 0] = 60.0
    k[:, :, :, 0] = -60.0  # every logit near -318: far below any starting reference
    run_window(q, k, v, left=50, right=20, sinks=3)
    k[:, 150:, :, 0] = 60.0  # and a jump of 636 upwards half way
    run_window(q, k, v, left=120, right=0)
    k[:, :, :, 0] = torch.linspace(-60, 60, 300).view(1, 300, 1)
    run_window(q, k, v, left=-1, right=0)


@pytest.mark.parametrize("kv_len", [[400, 1, 0, 129], [399, 256, 500, -3]])
def test_padded_batch(kv_len):
    q, k, v = make(5, 4, 2, 2, 400, 400, 64)
    for b, n in enumerate(kv_len):  # whatever lies past a sequence's end
        k[b, max(n, 0):] = float("nan")
        v[b, max(n, 0):] = float("inf")
    run_window(q, k, v, kv_len=kv_len, left=90, right=90, sinks=10)
    run_window(q, k, v, kv_len=kv_len, left=-1, right=-1)
    run_window(q, k, v, kv_len=kv_len, left=33, right=0)


def test_unseen_rows_may_hold_anything():
    # 40 queries at 1000..1039 with 70 keys behind them and 5 sinks: rows 5..929 and 1040.. unseen
    q, k, v = make(6, 1, 2, 2, 40, 1200, 128)
    for t in (k, v):
        t[:, 5:930] = float("nan")
        t[:, 1040:] = float("inf")
    run_window(q, k, v, left=70, right=0, sinks=5, q_pos=1000)


def test_strided_heads_and_outputs_left_alone():
    # q, k, v out of one projection's rows; outputs inside larger buffers keep their margins
    B, S, H, Hkv, D = 2, 333, 4, 2, 64
    g = torch.Generator().manual_seed(7)
    row = torch.randn(B, S, H + 2 * Hkv, D, generator=g).bfloat16()
    q, k, v = row[:, :, :H], row[:, :, H:H + Hkv], row[:, :, H + Hkv:]
    rd = row.to(DEV)
    pad = 512
    ob = torch.full((B * S * H * D + 2 * pad,), 7.0, dtype=torch.bfloat16, device=DEV)
    lb = torch.full((B * H * S + 2 * pad,), 7.0, dtype=torch.float32, device=DEV)
    out, lse = ob[pad:-pad].view(B, S, H, D), lb[pad:-pad].view(B, H, S)
    cp.window_fwd(rd[:, :, :H], rd[:, :, H:H + Hkv], rd[:, :, H + Hkv:], left=64, right=0, sinks=4, out=out, lse=lse)
    torch.cuda.synchronize()
    check(out, lse, ow.window_attention(q, k, v, D ** -0.5, 64, 0, 4), q, k, D ** -0.5)
    for b in (ob, lb):
        assert (b[:pad] == 7).all() and (b[-pad:] == 7).all()


@pytest.mark.parametrize("D,sizes", [(64, (300, 300)), (128, (257, 131)), (40, (65, 70)), (256, (33, 200)), (1, (9, 9)),
                                     (7, (130, 64))])
@pytest.mark.parametrize("w", [dict(left=-1, right=-1), dict(left=50, right=0, sinks=3), dict(left=10, right=25)])
def test_f32(D, sizes, w):
    q, k, v = make(D, 2, 4, 2, *sizes, D, dtype=torch.float32)
    run_window(q, k, v, **w)
    run_window(q, k, v, kv_len=[sizes[1] // 2, 0], q_pos=20, k_pos=10, out_dtype=torch.bfloat16, **w)


@pytest.mark.parametrize("D", [64, 128])
def test_f32_many_rows(D):
    # enough 64-row blocks for two per SM: the wide form of the fp32 kernel
    q, k, v = make(21, 2, 8, 2, 1300, 1300, D, dtype=torch.float32)
    run_window(q, k, v, left=40, right=9, sinks=3)


@pytest.mark.parametrize("D", [64, 100, 128])
def test_f32_enough_rows_for_the_widest_tiles(D):
    q, k, v = make(25, 2, 8, 2, 1400, 1400, D, dtype=torch.float32)  # 468 blocks of 48 (token, head) rows
    run_window(q, k, v, left=40, right=9, sinks=3)


@pytest.mark.parametrize("B,H,Hkv,Sq,Skv,D", [(1, 1, 1, 20, 1500, 128), (1, 2, 1, 40, 700, 64), (2, 2, 2, 33, 300, 256),
                                              (1, 3, 3, 100, 2000, 64), (1, 6, 2, 7, 130, 33), (1, 7, 1, 1, 65, 128),
                                              (1, 12, 4, 300, 65, 64)])
@pytest.mark.parametrize("w", [dict(left=-1, right=-1), dict(left=-1, right=0), dict(left=150, right=0, sinks=70)])
def test_f32_keys_shared_out_to_a_cluster(B, H, Hkv, Sq, Skv, D, w):
    q, k, v = make(26 + D, B, H, Hkv, Sq, Skv, D, dtype=torch.float32)
    o, l = run_window(q, k, v, q_pos=max(Skv - Sq, 0), **w)
    again = run_window(q, k, v, q_pos=max(Skv - Sq, 0), **w)
    assert torch.equal(o, again[0]) and torch.equal(l, again[1])  # a fixed order of sums
    # blocks whose share of the keys is empty, and rows that see nothing
    run_window(q, k, v, kv_len=[Skv // 7] * B, q_pos=max(Skv - Sq, 0), out_dtype=torch.bfloat16, **w)
    run_window(q, k, v, kv_len=[Skv] + [0] * (B - 1), k_pos=Sq // 2, **w)


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    r = np.random.default_rng(1000 + seed)
    pick = lambda *a: a[int(r.integers(len(a)))]
    D, Hkv = pick(64, 128), pick(1, 2, 3)
    Sq, Skv = int(r.integers(1, 600)), int(r.integers(1, 900))
    q, k, v = make(seed, pick(1, 2), Hkv * pick(1, 2, 5), Hkv, Sq, Skv, D, sigma=pick(1.0, 1.0, 3.0))
    B = q.shape[0]
    w = dict(left=pick(-1, int(r.integers(0, 700))), right=pick(-1, 0, int(r.integers(0, 300))),
             sinks=pick(0, 4, int(r.integers(0, 500))), q_pos=int(r.integers(0, 900)), k_pos=int(r.integers(0, 300)))
    kv_len = [int(x) for x in r.integers(0, Skv + 1, B)] if pick(True, False) else None
    run_window(q, k, v, kv_len=kv_len, out_dtype=pick(torch.bfloat16, torch.float32), **w)
    q1 = q[:, :min(Sq, pick(1, 1, 2, 7))].contiguous()
    run_decode(q1, k, v, [int(x) for x in r.integers(0, Skv + 1, B)], left=w["left"], sinks=w["sinks"])


def test_without_lse():
    q, k, v = (x.to(DEV) for x in make(22, 1, 4, 2, 200, 200, 64))
    o, l = cp.window_fwd(q, k, v, left=30, right=0, want_lse=False)
    o2, _ = cp.window_fwd(q, k, v, left=30, right=0)
    d, l3 = cp.window_decode(q[:, -1:].contiguous(), k, v, left=30, want_lse=False)
    d2, _ = cp.window_decode(q[:, -1:].contiguous(), k, v, left=30)
    f, l4 = cp.window_fwd(q.float(), k.float(), v.float(), left=30, right=0, want_lse=False)
    torch.cuda.synchronize()
    assert l is None and l3 is None and l4 is None
    assert torch.equal(o, o2) and torch.equal(d, d2) and torch.isfinite(f).all()


@pytest.mark.parametrize("acc_dtype", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("w", [dict(left=150, right=100, sinks=6), dict(left=-1, right=0), dict(left=70, right=0)])
def test_ring_step(acc_dtype, w):
    B, Sq, H, Hkv, D = 1, 260, 4, 2, 128
    q, k, v = make(8, B, H, Hkv, Sq, 900, D)
    cuts = [0, 1, 200, 456, 900]
    order = [2, 0, 3, 1]
    ks = [k[:, a:b].contiguous().to(DEV) for a, b in zip(cuts, cuts[1:])]
    vs = [v[:, a:b].contiguous().to(DEV) for a, b in zip(cuts, cuts[1:])]
    out, lse = cp.ring_attention(q.to(DEV), [ks[i] for i in order], [vs[i] for i in order], acc_dtype=acc_dtype,
                                 q_pos=300, k_pos=[cuts[i] for i in order], **w)
    torch.cuda.synchronize()
    ref = ow.window_attention(q, k, v, D ** -0.5, q_pos=300, **w)
    if acc_dtype is None:  # rounded once: the bound of a single pass, but for the merges' fp32 steps
        o_ref, l_ref, a = ref
        assert out.dtype == torch.bfloat16
        S = logit_error(q, k, D ** -0.5)
        bound = (HALF + 2e-5 + 2 * S + 4e-6) * a
        assert (np.abs(_f64(out) - o_ref) <= bound + HALF * (np.abs(o_ref) + bound)).all()
    check(out, lse, ref, q, k, D ** -0.5, merges=4)


# Few tiles share their keys out to clusters of 2, 4 and 8; from 149 on (24 heads of 7) each has its own.
@pytest.mark.parametrize("B,H,Hkv,Sq,Skv,D", [(1, 1, 1, 1, 4000, 128), (1, 2, 1, 130, 2000, 64), (2, 3, 3, 300, 900, 128),
                                              (1, 10, 2, 128, 1500, 64), (1, 40, 8, 190, 1100, 128),
                                              (1, 24, 4, 800, 700, 128), (2, 12, 12, 890, 500, 64)])
@pytest.mark.parametrize("w", [dict(left=-1, right=-1), dict(left=300, right=0, sinks=70), dict(left=-1, right=0)])
def test_tiles_and_parts_in_every_form_of_result(B, H, Hkv, Sq, Skv, D, w):
    q, k, v = make(28 + Sq, B, H, Hkv, Sq, Skv, D)
    at = max(Skv - Sq, 0)
    o, l = run_window(q, k, v, q_pos=at, **w)
    again = run_window(q, k, v, q_pos=at, **w)
    assert torch.equal(o, again[0]) and torch.equal(l, again[1])  # sums in a fixed order
    run_window(q, k, v, q_pos=at, out_dtype=torch.float32, **w)
    run_window(q, k, v, kv_len=[Skv // 9] * B, q_pos=at, out_dtype=torch.float32, **w)  # parts without keys
    cuts = [0, Skv // 2 + 3, Skv - 5, Skv]
    ks = [k[:, a:b].contiguous().to(DEV) for a, b in zip(cuts, cuts[1:])]
    vs = [v[:, a:b].contiguous().to(DEV) for a, b in zip(cuts, cuts[1:])]
    ref = ow.window_attention(q, k, v, D ** -0.5, q_pos=at, **w)
    for acc_dtype in (None, torch.bfloat16, torch.float32):
        run = torch.empty(q.shape, dtype=acc_dtype or torch.float32, device=DEV)
        out, lse = run if acc_dtype else torch.empty_like(q, device=DEV), torch.empty((B, H, Sq), device=DEV)
        for c, (kc, vc) in enumerate(zip(ks, vs)):
            last = c == 2 and acc_dtype is None
            cp.window_fwd(q.to(DEV), kc, vc, out=out if last else run, run=run if last else None, lse=lse,
                          accumulate=c > 0, q_pos=at, k_pos=cuts[c], **w)
        torch.cuda.synchronize()
        check(out, lse, ref, q, k, D ** -0.5, merges=3)


@pytest.mark.parametrize("H,Hkv", [(2, 1), (8, 2), (12, 2), (24, 2), (64, 1), (128, 1), (256, 1), (20, 1), (27, 3)])
@pytest.mark.parametrize("B,Sq,Skv,D", [(1, 1, 300, 128), (2, 5, 700, 64), (1, 37, 90, 64), (1, 130, 260, 128)])
def test_heads_that_share_a_tile(H, Hkv, B, Sq, Skv, D):
    q, k, v = make(30 + H + Sq, B, H, Hkv, Sq, Skv, D)
    at, w = Skv - Sq, dict(left=60, right=2, sinks=3)
    kv_len = [Skv] + [Skv // 3] * (B - 1)
    for dt in (torch.bfloat16, torch.float32):
        run_window(q, k, v, q_pos=at, kv_len=kv_len, out_dtype=dt, **w)
    wide = torch.cat([torch.full_like(q[:, :, :1], float("nan")), q, torch.full_like(q[:, :, :1], float("nan"))], 2).to(DEV)
    cut = Skv // 2
    ref = ow.window_attention(q, k, v, D ** -0.5, q_pos=at, **w)
    pad = 8 * D
    for acc_dtype in (None, torch.bfloat16, torch.float32):  # guarded outputs, q inside a wider row
        n = q.numel()
        buf = torch.full((n + 2 * pad,), 7.0, dtype=torch.bfloat16 if acc_dtype is None else acc_dtype, device=DEV)
        out = buf[pad:-pad].view(q.shape)
        run = torch.empty(q.shape, device=DEV) if acc_dtype is None else out
        lse = torch.empty((B, H, Sq), device=DEV)
        qd, kd, vd = wide[:, :, 1:-1], k.to(DEV), v.to(DEV)
        cp.window_fwd(qd, kd[:, :cut].contiguous(), vd[:, :cut].contiguous(), out=run, lse=lse, q_pos=at, **w)
        cp.window_fwd(qd, kd[:, cut:].contiguous(), vd[:, cut:].contiguous(), out=out, lse=lse, accumulate=True,
                      run=run if acc_dtype is None else None, q_pos=at, k_pos=cut, **w)
        torch.cuda.synchronize()
        check(out, lse, ref, q, k, D ** -0.5, merges=2)
        assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()


def test_merge_into_rows_that_hold_anything():
    # running rows with LSE = -inf are never used, whatever they hold; rows that see nothing stay
    for B, H, Sq, Skv in ((1, 2, 200, 900), (2, 20, 500, 300)):
        q, k, v = make(29, B, H, H, Sq, Skv, 128)
        qd, kd, vd = (x.to(DEV) for x in (q, k, v))
        w = dict(left=150, right=0, q_pos=100, k_pos=200)
        ref = ow.window_attention(q, k, v, 128 ** -0.5, **w)
        sees = torch.from_numpy(~np.isneginf(ref[1])).transpose(1, 2)
        for dt in (torch.float32, torch.bfloat16):
            out = torch.full((B, Sq, H, 128), float("nan"), dtype=dt, device=DEV)
            lse = torch.full((B, H, Sq), -math.inf, device=DEV)
            cp.window_fwd(qd, kd, vd, out=out, lse=lse, accumulate=True, **w)
            torch.cuda.synchronize()
            assert torch.isnan(out.cpu()[~sees]).all() and (~sees).any()
            filled = torch.where(sees[..., None], out.cpu(), torch.zeros((), dtype=dt))
            check(filled, lse, ref, q, k, 128 ** -0.5, merges=1)


def test_last_chunk_out_of_a_float32_running_result():
    q, k, v = make(23, 1, 2, 2, 300, 100, 64)
    run = torch.full((1, 300, 2, 64), float("nan"), device=DEV)
    lse = torch.full((1, 2, 300), -math.inf, device=DEV)
    run[:, 250:] = 1.001
    lse[:, :, 250:] = 1.0
    out = torch.full((1, 300, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    qd, kd, vd = (x.to(DEV) for x in (q, k, v))
    cp.window_fwd(qd, kd, vd, left=20, right=0, q_pos=0, k_pos=60, out=out, lse=lse, run=run, accumulate=True)
    torch.cuda.synchronize()
    o, l, a = ow.window_attention(q, k, v, 0.125, 20, 0, 0, 0, 60)
    check(out[:, 60:180], lse[:, :, 60:180], (o[:, 60:180], l[:, :, 60:180], a[:, 60:180]), q, k, 0.125)
    assert (out[:, :60] == 0).all() and torch.isneginf(lse[:, :, :60]).all()  # empty before and after
    assert torch.equal(out[:, 250:], run[:, 250:].bfloat16()) and (lse[:, :, 250:] == 1).all()
    # a chunk that no row sees, and one without keys: the running result, rounded
    for kk in (kd, kd[:, :0]):
        out.fill_(9.0)
        cp.window_fwd(qd, kk, kk, left=20, right=0, q_pos=1000, k_pos=0, out=out, lse=lse, run=run, accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(out[:, 250:], run[:, 250:].bfloat16()) and (out[:, :60] == 0).all()


def test_accumulate_keeps_rows_that_see_nothing():
    q, k, v = make(9, 1, 2, 2, 300, 100, 64)
    out = torch.full((1, 300, 2, 64), float("nan"), dtype=torch.float32, device=DEV)
    lse = torch.full((1, 2, 300), -math.inf, device=DEV)
    out[:, 250:] = 3.0
    lse[:, :, 250:] = 1.0
    cp.window_fwd(q.to(DEV), k.to(DEV), v.to(DEV), left=20, right=0, q_pos=0, k_pos=60, out=out, lse=lse, accumulate=True)
    torch.cuda.synchronize()
    # rows 60..179 see keys and started empty: the result, whatever the row held
    ref = ow.window_attention(q, k, v, 0.125, 20, 0, 0, 0, 60)
    o, l, a = ref
    check(out[:, 60:180], lse[:, :, 60:180], (o[:, 60:180], l[:, :, 60:180], a[:, 60:180]), q, k, 0.125)
    assert torch.isnan(out[:, :60]).all() and torch.isneginf(lse[:, :, :60]).all()
    assert (out[:, 250:] == 3).all() and (lse[:, :, 250:] == 1).all()


# ------------------------------------------------------------------ single tokens

def run_decode(q, k, v, kv_len, out_dtype=None, **kw):
    scale = q.shape[-1] ** -0.5
    kl = None if kv_len is None else torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    out, lse = cp.window_decode(q.to(DEV), k.to(DEV), v.to(DEV), kl, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    check(out, lse, ow.decode_attention(q, k, v, scale, kv_len, **kw), q, k, scale, n=k.shape[1])
    return out, lse


@pytest.mark.parametrize("B,H,Hkv,Sq,S,D", [(1, 1, 1, 1, 1, 64), (3, 8, 2, 1, 700, 128), (2, 4, 4, 1, 2000, 64),
                                            (2, 16, 1, 1, 333, 128), (2, 6, 2, 5, 500, 128), (1, 40, 2, 3, 260, 64),
                                            (5, 3, 3, 17, 129, 64), (1, 8, 8, 2, 4097, 128), (2, 64, 1, 1, 97, 64)])
@pytest.mark.parametrize("w", [dict(left=-1), dict(left=0), dict(left=100, sinks=4), dict(left=31, sinks=33)])
def test_decode(B, H, Hkv, Sq, S, D, w):
    q, k, v = make(B + H + S, B, H, Hkv, Sq, S, D)
    r = np.random.default_rng(S)
    kv_len = [S] + [int(x) for x in r.integers(0, S + 1, B - 1)]
    for b, n in enumerate(kv_len):  # a cache holds anything past the newest token
        k[b, n:] = float("nan")
        v[b, n:] = float("inf")
    run_decode(q, k, v, kv_len, **w)
    run_decode(q, k, v, [max(n, 1) for n in kv_len[:1]] * B if B == 1 else kv_len, out_dtype=torch.float32, **w)


def test_decode_lengths_at_the_edges():
    q, k, v = make(11, 6, 4, 2, 4, 300, 128)
    kv_len = [0, -7, 1, 3, 300, 900]  # empty, below, shorter than the queries, past the cache
    for b, n in enumerate(kv_len):
        k[b, max(n, 0):] = float("nan")
        v[b, max(n, 0):] = float("nan")
    out, lse = run_decode(q, k, v, kv_len, left=50, sinks=2)
    assert torch.isneginf(lse[:2]).all() and (out[:2] == 0).all()
    assert torch.isneginf(lse[2, :, :3]).all() and torch.isfinite(lse[2, :, 3]).all()
    q, k, v = make(11, 6, 4, 2, 4, 100, 128)  # finite caches: these lengths see the first rows
    run_decode(q, k, v, [1, 2, 3, 4, 5, 6], left=-1)


def test_decode_unseen_cache_rows_may_hold_anything():
    q, k, v = make(12, 2, 8, 2, 1, 3000, 128)
    kv_len = [2900, 1500]
    for b, n in enumerate(kv_len):
        for t in (k, v):
            t[b, 7:n - 201] = float("nan")
            t[b, n:] = float("inf")
    run_decode(q, k, v, kv_len, left=200, sinks=7)


def test_decode_strided_cache():
    # keys and values of a token side by side in one cache
    B, S, Hkv, D = 2, 777, 2, 64
    g = torch.Generator().manual_seed(13)
    kv = torch.randn(B, S, 2 * Hkv, D, generator=g).bfloat16()
    q = torch.randn(B, 1, 3 * 8, D, generator=g).bfloat16()
    kd, qd = kv.to(DEV), q.to(DEV)
    kl = torch.tensor([777, 400], dtype=torch.int32, device=DEV)
    out, lse = cp.window_decode(qd[:, :, 8:16], kd[:, :, :Hkv], kd[:, :, Hkv:], kl, left=300, sinks=4)
    torch.cuda.synchronize()
    k, v, qs = kv[:, :, :Hkv], kv[:, :, Hkv:], q[:, :, 8:16]
    check(out, lse, ow.decode_attention(qs, k, v, D ** -0.5, [777, 400], 300, 4), qs, k, D ** -0.5)


@pytest.mark.parametrize("B,H,Hkv,Sq,S,D", [(4, 32, 8, 50, 600, 128), (9, 24, 24, 40, 300, 64), (2, 40, 8, 130, 500, 128)])
def test_decode_of_many_tokens(B, H, Hkv, Sq, S, D):
    # enough (token, head) rows for the tensor-core kernel, the lengths still on the device
    q, k, v = make(24, B, H, Hkv, Sq, S, D)
    kv_len = [S, 20, 0, Sq, 77, 299, 150, 41, 39][:B]
    for b, n in enumerate(kv_len):
        k[b, n:] = float("nan")
        v[b, n:] = float("inf")
    run_decode(q, k, v, kv_len, left=100, sinks=5)
    run_decode(q, k, v, kv_len, left=-1, out_dtype=torch.float32)


def test_decode_f32():
    q, k, v = make(14, 2, 4, 2, 2, 90, 48, dtype=torch.float32)
    run_decode(q, k, v, [90, 33], left=40, sinks=2)


@pytest.mark.parametrize("B,H,Hkv,Sq,S,D", [(1, 8, 8, 1, 3000, 128), (3, 8, 2, 1, 700, 64), (2, 16, 1, 1, 333, 256),
                                            (1, 40, 2, 3, 260, 64), (5, 3, 3, 17, 129, 48), (2, 5, 1, 1, 1, 7),
                                            (4, 32, 8, 2, 513, 128), (70, 10, 5, 1, 40, 64)])
@pytest.mark.parametrize("w", [dict(left=-1), dict(left=0), dict(left=100, sinks=4)])
def test_decode_f32_forms(B, H, Hkv, Sq, S, D, w):
    q, k, v = make(B + H + D, B, H, Hkv, Sq, S, D, dtype=torch.float32)
    r = np.random.default_rng(S)
    kv_len = [S] + [int(x) for x in r.integers(0, S + 1, B - 1)]
    for b, n in enumerate(kv_len):
        k[b, n:] = float("nan")
        v[b, n:] = float("inf")
    run_decode(q, k, v, kv_len, **w)
    run_decode(q, k, v, kv_len, out_dtype=torch.bfloat16, **w)


def test_decode_f32_strided_cache():
    B, S, Hkv, D = 2, 777, 2, 64
    g = torch.Generator().manual_seed(27)
    kv = torch.randn(B, S, 2 * Hkv, D, generator=g)
    q = torch.randn(B, 3, 3 * 8, D, generator=g)
    kd, qd = kv.to(DEV), q.to(DEV)
    kl = torch.tensor([777, 400], dtype=torch.int32, device=DEV)
    out, lse = cp.window_decode(qd[:, :, 8:16], kd[:, :, :Hkv], kd[:, :, Hkv:], kl, left=300, sinks=4)
    torch.cuda.synchronize()
    k, v, qs = kv[:, :, :Hkv], kv[:, :, Hkv:], q[:, :, 8:16]
    check(out, lse, ow.decode_attention(qs, k, v, D ** -0.5, [777, 400], 300, 4), qs, k, D ** -0.5, n=S)


def test_decode_far_offsets():
    # a cache whose last rows lie past 2^31 elements and past 2^32 bytes
    S, D = (1 << 31) // 128 + 1000, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 2 * S * D * 2 + (4 << 30):
        pytest.skip("needs 13 GB of device memory")
    k = torch.zeros(1, S, 1, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros(1, S, 1, D, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(15)
    tail = torch.randn(2, 600, D, generator=g).bfloat16()
    k[0, -600:, 0] = tail[0].to(DEV)
    v[0, -600:, 0] = tail[1].to(DEV)
    q = torch.randn(1, 2, 8, D, generator=g).bfloat16()
    out, lse = cp.window_decode(q.to(DEV), k, v, left=500)
    o2, l2 = cp.window_fwd(q.to(DEV), k, v, left=500, right=0, q_pos=S - 2)
    torch.cuda.synchronize()
    kt, vt = (tail[i].view(1, 600, 1, D) for i in range(2))
    ref = ow.decode_attention(q, kt, vt, D ** -0.5, None, 500, 0)
    check(out, lse, ref, q, kt, D ** -0.5)
    check(o2, l2, ref, q, kt, D ** -0.5)


# ------------------------------------------------------------------ together, streams, graphs

@pytest.mark.parametrize("P,S_l,H,D", [(2, 160, 4, 64), (4, 75, 8, 128)])
def test_ulysses_layer_with_norm_rotation_and_window(P, S_l, H, D):
    g = torch.Generator().manual_seed(P)
    q, k, v = ((torch.randn(P, S_l, H, D, generator=g) * 2).bfloat16() for _ in range(3))
    gq, gk = 1 + 0.1 * torch.randn(D, generator=g), 1 + 0.1 * torch.randn(D, generator=g)
    T = P * S_l
    pos = torch.stack((torch.arange(T) // 40, torch.arange(T) % 40), 1).int()
    f, _ = cp.rope_frequencies(D // 2)
    freq = cp.rope_axes([f, f])
    plan = UlyssesPlan(P, S_l, H, D, qk_norm=(gq.to(DEV), gk.to(DEV)), rope=(pos.to(DEV), freq.to(DEV)),
                       window=(100, 20, 8))
    out, lse = plan.run(q.to(DEV), k.to(DEV), v.to(DEV))
    torch.cuda.synchronize()
    full = lambda x: x.reshape(1, T, H, D)
    # the rotated heads are rounded to bf16 (half a step of each element) before the attention;
    # the oracle's attention runs on the kernel's own rounded heads, which are checked apart
    turn = lambda x, w: ow.rotate(ow.rms_norm(full(x), w), pos.numpy(), freq)
    heads = lambda x: x.cpu().reshape(P, T, H // P, D).permute(1, 0, 2, 3).reshape(1, T, H, D)
    for got, want in ((heads(plan.qh), turn(q, gq)), (heads(plan.kh), turn(k, gk))):
        assert (np.abs(_f64(got) - want) <= HALF * np.abs(want) + 1e-5).all()
    assert torch.equal(heads(plan.vh), full(v))
    qr, kr = heads(plan.qh), heads(plan.kh)
    ref = ow.window_attention(qr, kr, full(v), D ** -0.5, 100, 20, 8)
    check(out.cpu().reshape(1, T, H, D), lse.cpu().reshape(1, H, T), ref, qr, kr, D ** -0.5)


def test_prefill_then_decode_equals_one_pass():
    # a sequence written into a cache slice by slice, then token by token
    B, H, Hkv, D, S = 2, 4, 2, 128, 300
    q, k, v = (x.to(DEV) for x in make(16, B, H, Hkv, S, S, D))
    whole, lw = cp.window_fwd(q, k, v, left=60, right=0, sinks=3)
    cache_k, cache_v = torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    got, gl = torch.empty_like(whole), torch.empty_like(lw)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    for a, b in ((0, 100), (100, 290)):
        cache_k[:, a:b], cache_v[:, a:b] = k[:, a:b], v[:, a:b]
        lens.fill_(b)
        got[:, a:b], gl[:, :, a:b] = cp.window_fwd(q[:, a:b].contiguous(), cache_k, cache_v, left=60, right=0, sinks=3,
                                                   q_pos=a, kv_len=lens)
    for t in range(290, S):
        cache_k[:, t], cache_v[:, t] = k[:, t], v[:, t]
        lens.fill_(t + 1)
        got[:, t:t + 1], gl[:, :, t:t + 1] = cp.window_decode(q[:, t:t + 1].contiguous(), cache_k, cache_v, lens,
                                                              left=60, sinks=3)
    torch.cuda.synchronize()
    ref = ow.window_attention(q, k, v, D ** -0.5, 60, 0, 3)
    check(whole, lw, ref, q, k, D ** -0.5)
    check(got, gl, ref, q, k, D ** -0.5)


def test_side_stream_and_graph_replay():
    B, H, Hkv, D, S = 2, 8, 2, 128, 600
    q, k, v = (x.to(DEV) for x in make(17, B, H, Hkv, S, S, D))
    q1 = q[:, :1].contiguous()
    lens = torch.tensor([600, 100], dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(B, H, S, device=DEV)
    o1, l1 = torch.empty_like(q1), torch.empty(B, H, 1, device=DEV)
    pos = torch.arange(S, dtype=torch.int32, device=DEV)
    freq = cp.rope_frequencies(D, device=DEV)[0]
    gam = torch.ones(D, device=DEV)
    qr, kr = torch.empty_like(q), torch.empty_like(k)

    def step():
        cp.qk_norm_rope(q, k, gam, gam, pos, freq, out=(qr, kr))
        cp.window_fwd(qr, kr, v, left=200, right=0, sinks=4, out=out, lse=lse)
        cp.window_decode(q1, kr, v, lens, left=200, sinks=4, out=o1, lse=l1)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    want = [t.clone() for t in (qr, kr, out, lse, o1, l1)]
    for t in (qr, kr, out, lse, o1, l1):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (qr, kr, out, lse, o1, l1):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((qr, kr, out, lse, o1, l1), want):
        assert torch.equal(a, b)
    # the captured decode follows the lengths as they are at the replay
    lens.copy_(torch.tensor([37, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    eager = cp.window_decode(q1, kr, v, lens, left=200, sinks=4)
    torch.cuda.synchronize()
    assert torch.equal(o1, eager[0]) and torch.equal(l1, eager[1])
    assert torch.isneginf(l1[1]).all() and (o1[1] == 0).all()


def test_two_streams_at_once():
    a = [x.to(DEV) for x in make(18, 1, 8, 8, 1500, 1500, 128)]
    b = [x.to(DEV) for x in make(19, 4, 8, 2, 1, 3000, 128)]
    ra = cp.window_fwd(*a, left=300, right=300, sinks=8)
    rb = cp.window_decode(*b, left=1000, sinks=8)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        got.append((cp.window_fwd(*a, left=300, right=300, sinks=8, stream=s1), ra))
        got.append((cp.window_decode(*b, left=1000, sinks=8, stream=s2), rb))
    torch.cuda.synchronize()
    for (o, l), (ro, rl) in got:
        assert torch.equal(o, ro) and torch.equal(l, rl)


def _mixed_calls():
    """Calls that share tiles out to clusters, in every kernel, and ones that fill the GPU."""
    def call(fn, *shapes, dtype=torch.bfloat16, **kw):
        g = torch.Generator().manual_seed(31 + len(shapes[0]) + shapes[1][1])
        ts = [torch.randn(*s, generator=g).to(dtype).to(DEV) for s in shapes]
        return ts, lambda: fn(*ts, **kw)
    kv = lambda B, S, H, D: ((B, S, H, D), (B, S, H, D))
    return [call(cp.window_fwd, (1, 300, 2, 128), *kv(1, 3000, 2, 128), left=-1, right=-1),
            call(cp.window_fwd, (1, 200, 8, 64), *kv(1, 2100, 2, 64), left=1500, right=0, q_pos=1900, sinks=9),
            call(cp.window_fwd, (1, 90, 3, 96), *kv(1, 1000, 3, 96), dtype=torch.float32, left=-1, right=-1),
            call(cp.window_decode, (2, 1, 16, 128), *kv(2, 3100, 4, 128), left=2500),
            call(cp.window_decode, (1, 1, 4, 64), *kv(1, 2200, 4, 64), dtype=torch.float32),
            call(cp.window_decode, (2, 64, 8, 128), *kv(2, 2300, 4, 128), left=2000),
            call(cp.window_fwd, (1, 1300, 24, 128), *kv(1, 1400, 24, 128), left=300, right=20, q_pos=50),
            call(cp.fwd, (1, 700, 8, 128), *kv(1, 900, 8, 128))]


def test_clustered_calls_beside_one_another():
    calls = _mixed_calls()
    want = [f() for _, f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for turn in range(6):
        got = []
        for i in range(len(calls)):
            with torch.cuda.stream(streams[(i + turn) % len(streams)]):
                got.append([calls[i][1]() for _ in range(3)])
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for o, l in g:
                assert torch.equal(o, w[0]) and torch.equal(l, w[1])


def test_clustered_calls_in_two_graphs():
    calls = _mixed_calls()
    graphs, outs = [], []
    for order in (calls, calls[::-1]):  # captured twice, replayed beside one another
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([f() for _, f in order])
        graphs.append(g)
    for seed in range(2):
        for ts, _ in calls:
            for t in ts:
                t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)))
        want = [f() for _, f in calls]
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
        torch.cuda.synchronize()
        for got, ref in ((outs[0], want), (outs[1], want[::-1])):
            for (o, l), (ow_, lw) in zip(got, ref):
                assert torch.equal(o, ow_) and torch.equal(l, lw)


@pytest.mark.parametrize("H,Hkv,D", [(4, 2, 128), (3, 3, 40), (2, 1, 256)])
@pytest.mark.parametrize("acc_dtype", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("w", [dict(left=150, right=100, sinks=6), dict(left=-1, right=0), dict(left=70, right=0)])
def test_f32_ring_step(acc_dtype, H, Hkv, D, w):
    # Chunks folded by the merge kernel.  A merge's weights are e^(La - L) and e^(Lb - L): off by the LSEs'
    # own errors, S and a few 2^-23 of |LSE| <= 16 each (1e-5 in all, with the few fp32 steps of the
    # exponential, the quotient and the sum), so it adds (2 S + 1e-5) A; a bf16 result half a step besides.
    q, k, v = make(40 + D, 1, H, Hkv, 260, 900, D, dtype=torch.float32)
    cuts = [0, 1, 200, 456, 900]
    order = [2, 0, 3, 1]
    parts = [[x[:, a:b].contiguous().to(DEV) for a, b in zip(cuts, cuts[1:])] for x in (k, v)]
    ks, vs = ([p[i] for i in order] for p in parts)
    out, lse = cp.ring_attention(q.to(DEV), ks, vs, acc_dtype=acc_dtype, q_pos=300, k_pos=[cuts[i] for i in order], **w)
    torch.cuda.synchronize()
    assert out.dtype == (acc_dtype or torch.float32)
    o_ref, l_ref, a = ow.window_attention(q, k, v, D ** -0.5, q_pos=300, **w)
    S = logit_error(q, k, D ** -0.5)
    bound = (2e-6 + 2 * S + 900 * 2.0 ** -24 + 3 * (2 * S + 1e-5)) * a
    if acc_dtype == torch.bfloat16:
        bound = bound + 4 * HALF * (a + bound)
    assert (np.abs(_f64(out) - o_ref) <= bound + 2.0 ** -24 * np.abs(o_ref) + 1e-30).all()
    empty = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(_f64(lse)), empty)
    err = np.abs(_f64(lse) - np.where(empty, 0, l_ref))[~empty]
    assert (err <= 4 * (S + 2e-5 + 2.0 ** -22 * np.abs(l_ref[~empty]))).all()


# ------------------------------------------------------------------ which kernel serves a decode call

def kernel_of(call, tmp_path):
    """The windowed kernel that a call launches, by its captured graph's dump."""
    call()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    g.enable_debug_mode()
    with torch.cuda.graph(g):
        call()
    dump = tmp_path / "graph.dot"
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")  # it announces itself
        g.debug_dump(str(dump))
    text = dump.read_text()
    found = [n for n in ("window_sm100_kernel", "window_decode_kernel", "window_f32_kernel") if n in text]
    assert len(found) == 1, found
    return found[0]


def decode_served_by(kernel, tmp_path, B, H, Hkv, Sq, S, D, **w):
    q, k, v = make(B + Sq + S, B, H, Hkv, Sq, S, D)
    kv_len = [S, 20, 0, Sq, S // 2, 1, S - 7, Sq - 1, Sq + 1][:B]
    kv_len = [max(0, n) for n in kv_len] + [S - 31 * b for b in range(len(kv_len), B)]
    for b, n in enumerate(kv_len):
        k[b, n:] = float("nan")
        v[b, n:] = float("inf")
    lens = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    assert kernel_of(lambda: cp.window_decode(qd, kd, vd, lens, **w), tmp_path) == kernel
    o, l = run_decode(q, k, v, kv_len, **w)
    o2, l2 = run_decode(q, k, v, kv_len, **w)
    assert torch.equal(o, o2) and torch.equal(l, l2)
    run_decode(q, k, v, kv_len, out_dtype=torch.float32, **w)


# Sizes where the time to expect of the split kernel is 1.3 to 4 times that of the tiles: heads that share a
# tile (1, 4, 8 and 16 of them), tiles of their own and tiles in clusters, batches with empty sequences.
@pytest.mark.parametrize("B,H,Hkv,Sq,S,D", [(8, 32, 8, 32, 2000, 64), (8, 64, 4, 48, 2500, 64), (1, 128, 8, 64, 2500, 64),
                                            (16, 24, 24, 70, 1500, 64), (2, 8, 1, 300, 4000, 64), (4, 60, 12, 130, 1999, 64),
                                            (8, 32, 8, 32, 2000, 128), (3, 64, 4, 60, 1500, 128)])
@pytest.mark.parametrize("w", [dict(left=-1), dict(left=1200, sinks=70)])
def test_decode_on_the_tiles(B, H, Hkv, Sq, S, D, w, tmp_path):
    decode_served_by("window_sm100_kernel", tmp_path, B, H, Hkv, Sq, S, D, **w)


@pytest.mark.parametrize("B,H,Hkv,Sq,S,D", [(3, 8, 2, 1, 700, 128), (8, 16, 16, 4, 1990, 64), (16, 32, 8, 1, 900, 64),
                                            (1, 16, 16, 9, 3000, 128)])
@pytest.mark.parametrize("w", [dict(left=-1), dict(left=1200, sinks=70)])
def test_decode_on_the_split_kernel(B, H, Hkv, Sq, S, D, w, tmp_path):
    decode_served_by("window_decode_kernel", tmp_path, B, H, Hkv, Sq, S, D, **w)


# ------------------------------------------------------------------ a float32 running O, rounded once

def check_rounded_once(out, lse, ref, q, k, merges):
    """A single pass's bound plus the fp32 steps of the merges: O is off by the weights' error of each chunk
    (shares of A that sum to it), a few fp32 steps a merge, and one half-step of the result."""
    o_ref, l_ref, a = ref
    assert out.dtype == torch.bfloat16
    S = logit_error(q, k, q.shape[-1] ** -0.5)
    bound = (HALF + 2e-5 + 2 * S + merges * 1e-6) * a
    assert (np.abs(_f64(out) - o_ref) <= bound + HALF * (np.abs(o_ref) + bound) + 1e-30).all()
    empty = np.isneginf(l_ref)
    l = _f64(lse)
    assert np.array_equal(np.isneginf(l), empty)
    err = np.abs(l - np.where(empty, 0, l_ref))[~empty]
    assert (err <= S + 2e-5 + (1 + merges) * 2.0 ** -22 * np.abs(l_ref[~empty])).all()


@pytest.mark.parametrize("B,H,Hkv,Sq,Skv,D", [(1, 1, 1, 1, 4000, 128), (1, 2, 1, 130, 2000, 64), (2, 3, 3, 300, 900, 128),
                                              (1, 10, 2, 128, 1500, 64), (1, 40, 8, 190, 1100, 128),
                                              (1, 24, 4, 800, 700, 128), (2, 12, 12, 890, 500, 64),
                                              (2, 64, 1, 5, 700, 64), (1, 128, 1, 130, 260, 128), (1, 27, 3, 37, 90, 64)])
@pytest.mark.parametrize("w", [dict(left=-1, right=-1), dict(left=300, right=0, sinks=70), dict(left=60, right=2, sinks=3)])
def test_merges_of_a_float32_running_result_round_once(B, H, Hkv, Sq, Skv, D, w):
    q, k, v = make(50 + Sq, B, H, Hkv, Sq, Skv, D)
    at = max(Skv - Sq, 0)
    cuts = [0, Skv // 2 + 3, Skv - 5, Skv]
    run = torch.empty(q.shape, device=DEV)
    out, lse = torch.empty_like(q, device=DEV), torch.empty((B, H, Sq), device=DEV)
    for c in range(3):
        kc, vc = (x[:, cuts[c]:cuts[c + 1]].contiguous().to(DEV) for x in (k, v))
        last = c == 2
        cp.window_fwd(q.to(DEV), kc, vc, out=out if last else run, run=run if last else None, lse=lse,
                      accumulate=c > 0, q_pos=at, k_pos=cuts[c], **w)
    torch.cuda.synchronize()
    check_rounded_once(out, lse, ow.window_attention(q, k, v, D ** -0.5, q_pos=at, **w), q, k, 2)
