"""fp64 NumPy oracle of the windowed attention and of the rotary positions (test
infrastructure), written from their definitions.

Windowed attention: query row i is at position q_pos + i, key row j at k_pos + j; row i sees key
j when j is inside the sequence, not more than ``right`` ahead, and either not more than ``left``
behind or among the first ``sinks`` positions (a negative bound is no bound).  Softmax, O and LSE
run over the visible keys; a row that sees none has O = 0 and LSE = -inf.  Hidden keys are
dropped before any arithmetic, so whatever they hold cannot matter.

Rotation: every pair of the first ``rot`` elements of a head row, as a complex number, is
multiplied by factor * e^(i angle), angle = sum over axes of position times frequency.
"""

from __future__ import annotations

import numpy as np

from .ref import _f64


def visible(Sq, Skv, left, right, sinks, q_pos=0, k_pos=0, length=None):
    """bool [Sq][Skv]."""
    p = (q_pos + np.arange(Sq))[:, None]
    t = (k_pos + np.arange(Skv))[None, :]
    see = np.ones((Sq, Skv), dtype=bool)
    if right >= 0:
        see &= t <= p + right
    if left >= 0:
        see &= (t >= p - left) | (t < sinks)
    if length is not None:
        see &= np.arange(Skv)[None, :] < min(max(int(length), 0), Skv)
    return see


def window_attention(q, k, v, scale, left=-1, right=-1, sinks=0, q_pos=0, k_pos=0, kv_len=None):
    """q [B][Sq][H][D], k/v [B][Skv][Hkv][D] -> (O [B][Sq][H][D], LSE [B][H][Sq], A) in fp64, A
    the same average of |v| (what a relative error of the weights is a share of)."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Sq, H, D = q.shape
    Skv, Hkv = k.shape[1], k.shape[2]
    o, a = np.zeros((B, Sq, H, D)), np.zeros((B, Sq, H, D))
    lse = np.full((B, H, Sq), -np.inf)
    for b in range(B):
        off = q_pos
        see = visible(Sq, Skv, left, right, sinks, off, k_pos, None if kv_len is None else kv_len[b])
        any_row = see.any(0)  # keys that no row sees take no part
        for h in range(H):
            kh, vh = k[b, any_row, h // (H // Hkv)], v[b, any_row, h // (H // Hkv)]
            s = np.where(see[:, any_row], scale * (q[b, :, h] @ kh.T), -np.inf)
            if s.shape[1] == 0:
                continue
            m = s.max(1, keepdims=True)
            m[m == -np.inf] = 0.0
            e = np.exp(s - m)
            l = e.sum(1, keepdims=True)
            row = l[:, 0] > 0
            lse[b, h, row] = (m[:, 0] + np.log(np.where(l[:, 0] > 0, l[:, 0], 1.0)))[row]
            w = e / np.where(l > 0, l, 1.0)
            o[b, :, h] = w @ vh
            a[b, :, h] = w @ np.abs(vh)
    return o, lse, a


def decode_attention(q, k, v, scale, kv_len=None, left=-1, sinks=0):
    """The last Sq tokens of each sequence against its cache (causal)."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Sq, H, _ = q.shape
    outs = []
    for b in range(B):
        n = k.shape[1] if kv_len is None else min(max(int(kv_len[b]), 0), k.shape[1])
        outs.append(window_attention(q[b:b + 1], k[b:b + 1, :n], v[b:b + 1, :n], scale, left, 0, sinks,
                                     q_pos=n - Sq))
    return tuple(np.concatenate([o[i] for o in outs]) for i in range(3))


def angles(pos, freq):
    """pos [rows] or [rows][axes], freq [pairs] or [axes][pairs] -> radians [rows][pairs]."""
    freq = np.atleast_2d(_f64(freq))
    pos = np.asarray(pos, dtype=np.float64)
    pos = pos.reshape(-1, freq.shape[0])
    return pos @ freq


def rotate(x, pos, freq, interleaved=False, factor=1.0):
    """x [..., tokens, H, D] in fp64; the positions repeat over the leading axes."""
    x = _f64(x)
    a = angles(pos, freq)
    half = a.shape[1]
    tok = int(np.prod(x.shape[:-2]))
    y = x.reshape(tok, x.shape[-2], x.shape[-1]).copy()
    z = factor * np.exp(1j * np.tile(a, (tok // a.shape[0], 1)))[:, None, :]
    i = np.arange(half)
    re, im = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    w = (y[..., re] + 1j * y[..., im]) * z
    y[..., re], y[..., im] = w.real, w.imag
    return y.reshape(x.shape)


def rms_norm(x, gamma, eps=1e-6, out_scale=1.0):
    x = _f64(x)
    mean = (x * x).mean(-1, keepdims=True) + eps
    r = np.where(mean == 0, 0.0, 1.0 / np.sqrt(np.where(mean == 0, 1.0, mean)))  # NaN stays NaN
    return x * r * _f64(gamma) * out_scale
