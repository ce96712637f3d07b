"""Pins of the windowed-attention and rotation oracle: loop-only brute force, closed forms and
invariants (CPU)."""

import math

import numpy as np
import pytest

from oracle import ref
from oracle import window as ow


def brute(q, k, v, scale, left, right, sinks, q_pos, k_pos, kv_len):
    B, Sq, H, D = q.shape
    Skv, Hkv = k.shape[1:3]
    o, lse = np.zeros((B, Sq, H, D)), np.full((B, H, Sq), -np.inf)
    for b in range(B):
        for h in range(H):
            g = h * Hkv // H
            for i in range(Sq):
                p, keys = q_pos + i, []
                for j in range(Skv):
                    t = k_pos + j
                    if kv_len is not None and j >= kv_len[b]:
                        continue
                    if right >= 0 and t > p + right:
                        continue
                    if left >= 0 and t < p - left and t >= sinks:
                        continue
                    keys.append(j)
                if not keys:
                    continue
                e = [math.exp(scale * float(q[b, i, h] @ k[b, j, g])) for j in keys]
                lse[b, h, i] = math.log(sum(e))
                o[b, i, h] = sum(w * v[b, j, g] for w, j in zip(e, keys)) / sum(e)
    return o, lse


@pytest.mark.parametrize("left,right,sinks,q_pos,k_pos,kv_len", [
    (-1, -1, 0, 0, 0, None), (3, 0, 0, 0, 0, None), (2, 1, 2, 4, 0, None), (0, 0, 3, 9, 0, [7, 0]),
    (-1, 0, 0, 0, 5, None), (2, 2, 4, 20, 0, None), (2, -1, 3, 5, 2, [4, 11])])
def test_window_matches_brute_force(left, right, sinks, q_pos, k_pos, kv_len):
    r = np.random.default_rng(5 + left + 10 * sinks + q_pos)
    q, k, v = r.normal(size=(2, 7, 4, 3)), r.normal(size=(2, 11, 2, 3)), r.normal(size=(2, 11, 2, 3))
    o, l, _ = ow.window_attention(q, k, v, 0.7, left, right, sinks, q_pos, k_pos, kv_len)
    ob, lb = brute(q, k, v, 0.7, left, right, sinks, q_pos, k_pos, kv_len)
    np.testing.assert_allclose(o, ob, atol=1e-12)
    np.testing.assert_allclose(l, lb, atol=1e-12)


def test_no_bounds_is_the_plain_attention():
    r = np.random.default_rng(1)
    q, k, v = (r.normal(size=(1, 9, 2, 4)) for _ in range(3))
    o, l, _ = ow.window_attention(q, k, v, 0.5)
    o2, l2 = ref.attention(q, k, v, 0.5)
    np.testing.assert_allclose(o, o2, atol=1e-13)
    np.testing.assert_allclose(l, l2, atol=1e-13)


def test_hidden_keys_cannot_matter():
    r = np.random.default_rng(2)
    q, k, v = (r.normal(size=(1, 6, 1, 4)) for _ in range(3))
    k2, v2 = k.copy(), v.copy()
    k2[:, 2:4] = np.nan
    v2[:, 2:4] = np.inf
    q6 = q[:, 4:]  # rows at 5, 6: the window starts at 4, the sinks end at 1
    a = ow.window_attention(q6, k, v, 0.5, 1, 0, 2, q_pos=5)
    b = ow.window_attention(q6, k2, v2, 0.5, 1, 0, 2, q_pos=5)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_decode_rows_are_rows_of_the_whole_sequence():
    r = np.random.default_rng(3)
    S = 13
    q, k, v = (r.normal(size=(1, S, 2, 4)) for _ in range(3))
    o, l, _ = ow.window_attention(q, k, v, 0.5, 4, 0, 2)
    od, ld, _ = ow.decode_attention(q[:, 8:11], k, v, 0.5, [11], 4, 2)
    np.testing.assert_allclose(od, o[:, 8:11], atol=1e-13)
    np.testing.assert_allclose(ld, l[:, :, 8:11], atol=1e-13)


def test_rotation_closed_forms():
    x = np.array([[[1.0, 0.0, 0.0, 1.0, 5.0]]])  # one token, one head, rot 4 of 5
    half = ow.rotate(x, [1], [math.pi / 2, math.pi])
    np.testing.assert_allclose(half[0, 0], [0, 0, 1, -1, 5], atol=1e-15)
    inter = ow.rotate(x, [1], [math.pi / 2, math.pi], interleaved=True, factor=2.0)
    np.testing.assert_allclose(inter[0, 0], [0, 2, 0, -2, 5], atol=1e-15)
    axes = ow.rotate(x, [[3, 2]], [[math.pi / 2, 0], [0, math.pi / 4]])
    np.testing.assert_allclose(axes[0, 0], [0, -1, -1, 0, 5], atol=1e-15)


def test_rotated_products_depend_on_distance_only():
    r = np.random.default_rng(4)
    q, k = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8))
    f = 10000.0 ** (-np.arange(4) / 4)
    dot = [float((ow.rotate(q, [p + 7], f) * ow.rotate(k, [p], f)).sum()) for p in (0, 5, 100000)]
    np.testing.assert_allclose(dot, dot[0], atol=1e-9)
