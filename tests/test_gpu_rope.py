"""GPU parity of the rotary positions and of the Q/K norm with rotation against the fp64 oracle.

Bound: the angle is reduced in 64 bits, so cos and sin are within 2^-22 of their values; a rotated
element is two fp32 products (2^-24 each of its parts) and the norm adds its sum and root, within
2^-20 in all: |err| <= 2e-6 (|x_a| + |x_b|) factor before the last rounding, which adds half a step
(bf16 2^-8, fp32 2^-24 of the value).
"""

import math

import numpy as np
import pytest
import torch

import context_long_sequence_non_b200 as cp
from context_long_sequence_non_b200 import build as build_mod
from oracle import ref as oref
from oracle import window as ow
from oracle.ref import _f64

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build_mod.build()
    cp.lib()
    yield
    assert cp.device_error() == 0


def randn(seed, *shape, dtype=torch.bfloat16, sigma=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * sigma).to(dtype)


def check(got, want, before, rot, interleaved, factor):
    """before: the values that were rotated (after the norm), fp64."""
    half = rot // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    size = np.abs(before).copy()
    both = size[..., a] + size[..., b]
    size[..., a], size[..., b] = both, both
    size[..., :rot] *= max(factor, 1.0)
    bound = 2e-6 * size + torch.finfo(got.dtype).eps / 2 * (np.abs(want) + 2e-6 * size)
    err = np.abs(_f64(got) - want)
    assert (err <= bound + 1e-37).all(), f"off by {err.max():.3e}, over the bound by {(err - bound).max():.3e}"


SHAPES = [((1, 1, 1), 128, 128), ((3, 37, 5), 64, 64), ((200, 3), 128, 64), ((2, 9, 4), 256, 256), ((50, 16), 128, 96),
          ((33, 7), 80, 48), ((19, 2), 96, 96), ((21, 3), 72, 72), ((13, 3), 128, 20), ((5, 3), 10, 6), ((9, 1), 2, 2),
          ((11, 5), 256, 32), ((6, 3), 250, 130), ((40, 2), 32, 32), ((40, 3), 16, 16), ((7, 2), 24, 8)]


@pytest.mark.parametrize("lead,D,rot", SHAPES, ids=lambda s: str(s).replace(" ", ""))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope(lead, D, rot, interleaved, dtype):
    x = randn(D + rot, *lead, D, dtype=dtype)
    tokens = lead[-2]
    pos = torch.randint(-500, 100000, (tokens,), generator=torch.Generator().manual_seed(rot)).int()
    freq, _ = cp.rope_frequencies(rot)
    want = ow.rotate(x, pos.numpy(), freq, interleaved, 1.25)
    xd, pd, fd = x.to(DEV), pos.to(DEV), freq.to(DEV)
    got = cp.rope(xd, pd, fd, interleaved=interleaved, factor=1.25)
    torch.cuda.synchronize()
    check(got, want, _f64(x), rot, interleaved, 1.25)
    assert torch.equal(got[..., rot:].cpu(), x[..., rot:])  # the rest of the head as it is
    same = cp.rope(xd, pd, fd, interleaved=interleaved, factor=1.25, out=xd)  # in place: the same bits
    torch.cuda.synchronize()
    assert same is xd and torch.equal(same, got)


@pytest.mark.parametrize("axes", [2, 3, 4])
def test_axes_and_far_positions(axes):
    x = randn(axes, 60, 2, 128, dtype=torch.float32)
    g = torch.Generator().manual_seed(axes)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (60, axes), generator=g).int()
    cut = [64 * a // axes for a in range(axes + 1)]
    freq = cp.rope_axes([cp.rope_frequencies(2 * (b - a))[0] for a, b in zip(cut, cut[1:])])
    got = cp.rope(x.to(DEV), pos.to(DEV), freq.to(DEV))
    torch.cuda.synchronize()
    # at 2^31 radians a double's angle is itself 2^-22 off (half a step, 2^-53 of it, and as much
    # again from each product and sum): a few 1e-6 more
    want = ow.rotate(x, pos.numpy(), freq)
    assert np.abs(_f64(got) - want).max() <= 8e-6 * np.abs(_f64(x)).max() * 2


def test_negated_positions_undo():
    x = randn(5, 100, 4, 64, dtype=torch.float32)
    pos = torch.arange(100, dtype=torch.int32) * 997
    freq, _ = cp.rope_frequencies(64)
    fd = freq.to(DEV)
    y = cp.rope(x.to(DEV), pos.to(DEV), fd)
    back = cp.rope(y, (-pos).to(DEV), fd)
    torch.cuda.synchronize()
    assert (back.cpu() - x).abs().max() <= 2 * 2 * 2e-6 * float(x.abs().max()) * 2


def test_empty_and_zero():
    freq = cp.rope_frequencies(64, device=DEV)[0]
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    assert cp.rope(e, torch.empty(0, dtype=torch.int32, device=DEV), freq).shape == e.shape
    z = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    g = torch.ones(64, device=DEV)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    for eps in (0.0, 1e-6):
        a, b = cp.qk_norm_rope(z, z.clone(), g, g, pos, freq, eps=eps)
        torch.cuda.synchronize()
        assert (a == 0).all() and (b == 0).all()


@pytest.mark.parametrize("T,Hq,Hk,D,rot,interleaved", [(1, 32, 8, 128, 128, False), (333, 6, 2, 128, 64, True),
                                                       (50, 3, 3, 64, 64, False), (41, 4, 1, 256, 64, False),
                                                       (29, 5, 2, 80, 48, True), (29, 2, 1, 72, 20, False),
                                                       (700, 1, 1, 32, 32, True), (17, 8, 2, 96, 96, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_qk_norm_rope(T, Hq, Hk, D, rot, interleaved, dtype):
    q, k = randn(T, T, Hq, D, dtype=dtype, sigma=3.0), randn(T + 1, T, Hk, D, dtype=dtype, sigma=0.1)
    gq, gk = 1 + 0.1 * randn(1, D, dtype=torch.float32), 1 + 0.1 * randn(2, D, dtype=torch.float32)
    pos = torch.arange(T, dtype=torch.int32) * 31
    freq, factor = cp.rope_frequencies(rot, scaling="by_parts", stretch=4.0, train_len=2048)
    out = cp.qk_norm_rope(q.to(DEV), k.to(DEV), gq.to(DEV), gk.to(DEV), pos.to(DEV), freq.to(DEV),
                          interleaved=interleaved, factor=factor, out_scale=0.5)
    # the same heads as slices of one row, in place: the same bits
    row = torch.cat((q, k, q), 1).to(DEV)
    rq, rk = row[:, :Hq], row[:, Hq:Hq + Hk]
    cp.qk_norm_rope(rq, rk, gq.to(DEV), gk.to(DEV), pos.to(DEV), freq.to(DEV), interleaved=interleaved,
                    factor=factor, out_scale=0.5, out=(rq, rk))
    torch.cuda.synchronize()
    for x, g, got in ((q, gq, out[0]), (k, gk, out[1])):
        n = ow.rms_norm(x, g, 1e-6, 0.5)
        check(got, ow.rotate(n, pos.numpy(), freq, interleaved, factor), n, rot, interleaved, factor)
    assert torch.equal(rq, out[0]) and torch.equal(rk, out[1])
    assert torch.equal(row[:, Hq + Hk:].cpu(), q)  # the other heads of the row are left alone


# a token's heads in 8, 4, 2 and 1 parts, uneven ones among them; three blocks of 32 pairs and a half one
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(150, 35, 5, 128, 128), (420, 32, 8, 64, 64), (900, 9, 3, 128, 96),
                                           (1100, 70, 1, 80, 80), (3000, 24, 8, 128, 128), (2500, 5, 3, 256, 224)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_parts_of_a_token(T, Hq, Hk, D, rot, interleaved):
    q, k = randn(T, T, Hq, D, sigma=3.0), randn(T + 1, T, Hk, D, sigma=0.1)
    gq, gk = 1 + 0.1 * randn(1, D, dtype=torch.float32), 1 + 0.1 * randn(2, D, dtype=torch.float32)
    pos = torch.arange(T, dtype=torch.int32) * 17 - 900
    freq, _ = cp.rope_frequencies(rot)
    out = cp.qk_norm_rope(q.to(DEV), k.to(DEV), gq.to(DEV), gk.to(DEV), pos.to(DEV), freq.to(DEV),
                          interleaved=interleaved)
    plain = cp.rope(q.to(DEV), pos.to(DEV), freq.to(DEV), interleaved=interleaved)
    torch.cuda.synchronize()
    for x, g, got in ((q, gq, out[0]), (k, gk, out[1])):
        n = ow.rms_norm(x, g, 1e-6, 1.0)
        check(got, ow.rotate(n, pos.numpy(), freq, interleaved, 1.0), n, rot, interleaved, 1.0)
    check(plain, ow.rotate(q, pos.numpy(), freq, interleaved, 1.0), _f64(q), rot, interleaved, 1.0)


@pytest.mark.parametrize("P,S_l,H,D,rot", [(2, 3, 4, 64, 64), (4, 33, 8, 128, 128), (8, 17, 16, 128, 64), (1, 9, 4, 256, 256),
                                           (3, 7, 6, 80, 48), (2, 11, 24, 72, 20), (2, 300, 4, 32, 32)])
@pytest.mark.parametrize("norm", [True, False])
def test_seq2head_norm_rope(P, S_l, H, D, rot, norm):
    q, k, v = (randn(P + i, P, S_l, H, D, sigma=2.0) for i in range(3))
    v.view(torch.int16).view(-1)[:7] = -1  # NaNs with a payload: V moves bit for bit
    g = 1 + 0.1 * randn(9, D, dtype=torch.float32)
    T = P * S_l
    pos = torch.randint(0, 5000, (T, 2), generator=torch.Generator().manual_seed(P)).int()
    n0 = rot // 4
    freq = cp.rope_axes([cp.rope_frequencies(2 * n0)[0], cp.rope_frequencies(2 * (rot // 2 - n0))[0]])
    gd = g.to(DEV) if norm else None
    qd, kd, vd = (x.to(DEV) for x in (q, k, v))
    qh, kh, vh = cp.seq2head_qkv_norm_rope(qd, kd, vd, P, gd, gd, pos.to(DEV), freq.to(DEV), interleaved=True)
    torch.cuda.synchronize()
    assert torch.equal(vh.cpu().view(torch.int16), torch.from_numpy(oref.seq2head(v.view(torch.int16).numpy(), P)))
    for x, got in ((q, qh), (k, kh)):
        n = ow.rms_norm(x, g) if norm else _f64(x)
        want = ow.rotate(n, pos.numpy(), freq, True)
        check(got, oref.seq2head(want, P), oref.seq2head(n, P), rot, True, 1.0)
    # the same bits as the separate calls
    full = lambda t: t.view(T, H, D)
    if norm:
        q2, k2 = cp.qk_norm_rope(full(qd), full(kd), gd, gd, pos.to(DEV), freq.to(DEV), interleaved=True)
    else:
        q2, k2 = (cp.rope(full(t), pos.to(DEV), freq.to(DEV), interleaved=True) for t in (qd, kd))
    q3, k3 = (cp.seq2head(t.view(P, S_l, H, D), P) for t in (q2, k2))
    torch.cuda.synchronize()
    assert torch.equal(qh, q3) and torch.equal(kh, k3)


@pytest.mark.parametrize("interleaved", [False, True])
def test_many_tokens_and_repeated_positions(interleaved):
    # more tokens than warps on the GPU, three sequences at the same positions
    x = randn(31, 3, 2500, 3, 64)
    pos = torch.randint(0, 1 << 20, (2500, 2), generator=torch.Generator().manual_seed(1)).int()
    freq = cp.rope_axes([cp.rope_frequencies(32)[0], cp.rope_frequencies(16)[0]])
    want = ow.rotate(x, pos.numpy(), freq, interleaved)
    got = cp.rope(x.to(DEV), pos.to(DEV), freq.to(DEV), interleaved=interleaved)
    torch.cuda.synchronize()
    check(got, want, _f64(x), 48, interleaved, 1.0)


def test_many_head_groups():
    P, S_l, H, D = 7, 3, 70, 32
    q, k, v = (randn(P + i, P, S_l, H, D) for i in range(3))
    g = torch.ones(D)
    T = P * S_l
    pos = torch.arange(T, dtype=torch.int32) * 11
    freq, _ = cp.rope_frequencies(D)
    qh, kh, vh = cp.seq2head_qkv_norm_rope(*(t.to(DEV) for t in (q, k, v)), P, g.to(DEV), g.to(DEV), pos.to(DEV),
                                           freq.to(DEV))
    torch.cuda.synchronize()
    n = ow.rms_norm(q, g)
    check(qh, oref.seq2head(ow.rotate(n, pos.numpy(), freq), P), oref.seq2head(n, P), D, False, 1.0)
    n = ow.rms_norm(k, g)
    check(kh, oref.seq2head(ow.rotate(n, pos.numpy(), freq), P), oref.seq2head(n, P), D, False, 1.0)
    assert torch.equal(vh.cpu().view(torch.int16), torch.from_numpy(oref.seq2head(v.view(torch.int16).numpy(), P)))


def test_margins_of_a_strided_output_are_left_alone():
    x = randn(3, 50, 2, 64)
    freq = cp.rope_frequencies(64, device=DEV)[0]
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    wide = torch.full((52, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    cp.rope(x.to(DEV), pos, freq, out=wide[1:51, 1:3])
    torch.cuda.synchronize()
    assert torch.equal(wide[1:51, 1:3], cp.rope(x.to(DEV), pos, freq))
    wide[1:51, 1:3] = 7.0
    assert (wide == 7).all()
    assert math.isfinite(float(wide.float().sum()))
