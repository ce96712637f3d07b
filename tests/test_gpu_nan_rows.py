"""A NaN in a query row or a head row reaches the whole of that row's result, and no other row's.

0 and -inf say "this row saw no key" and 0 says "this row was all zeros": neither may stand for a row
whose arithmetic gave NaN.  Rows do not share arithmetic, so the others must keep their bits.
"""

import math

import pytest
import torch

import context_long_sequence_non_b200 as cp
from context_long_sequence_non_b200 import build as build_mod
from oracle import window as ow

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build_mod.build()
    cp.lib()
    yield
    assert cp.device_error() == 0


def make(seed, B, H, Hkv, Sq, Skv, D, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)
    return r(B, Sq, H, D), r(B, Skv, Hkv, D), r(B, Skv, Hkv, D)


def spoil(q, seed, value=NAN):
    """A copy of q with NaN rows (a whole one, or one element), and bool [B][Sq][H] of them."""
    B, Sq, H, D = q.shape
    g = torch.Generator().manual_seed(seed)
    bad = torch.rand(B, Sq, H, generator=g) < 0.1
    bad[0, 0, 0] = bad[-1, -1, -1] = True
    whole = torch.rand(B, Sq, H, generator=g) < 0.5
    at = torch.randint(0, D, (B, Sq, H), generator=g)
    hit = bad[..., None] & (whole[..., None] | (torch.arange(D) == at[..., None]))
    q = q.clone()
    q[hit.to(DEV)] = value
    return q, bad.to(DEV)


def check(got, want, bad, sees):
    """bad, sees: bool [B][Sq][H]."""
    torch.cuda.synchronize()
    (o, l), (wo, wl) = got, want
    l, wl = l.transpose(1, 2), wl.transpose(1, 2)
    hit = bad & sees
    assert hit.any()
    assert torch.isnan(l[hit]).all() and torch.isnan(o[hit]).all()
    assert torch.equal(o[~hit], wo[~hit]) and torch.equal(l[~hit], wl[~hit])
    assert torch.isneginf(l[~sees]).all() and (o[~sees] == 0).all()


def seen_by(q, Skv, kv_len=None, q_pos=0, k_pos=0, left=-1, right=-1, sinks=0):
    B, Sq, H, _ = q.shape
    rows = [torch.from_numpy(ow.visible(Sq, Skv, left, right, sinks, q_pos, k_pos,
                                        None if kv_len is None else kv_len[b]).any(1)) for b in range(B)]
    return torch.stack(rows)[..., None].expand(B, Sq, H).to(DEV)


WINDOWS = [dict(left=-1, right=-1), dict(left=-1, right=0), dict(left=90, right=20, sinks=5), dict(left=0, right=0)]
# tiles of their own, tiles whose keys are shared out to a cluster, one row, heads that share a tile; the
# fp32 kernel's three row counts and its clusters
WINDOW_SHAPES = [(1, 24, 24, 900, 900, 128, torch.bfloat16), (1, 24, 4, 900, 700, 64, torch.bfloat16),
                 (1, 2, 2, 300, 900, 128, torch.bfloat16), (2, 1, 1, 1, 2000, 64, torch.bfloat16),
                 (1, 16, 2, 200, 400, 128, torch.bfloat16), (2, 8, 2, 1400, 1400, 64, torch.float32),
                 (1, 3, 3, 200, 700, 128, torch.float32), (1, 2, 1, 3, 900, 256, torch.float32)]


@pytest.mark.parametrize("w", WINDOWS, ids=lambda w: "-".join(map(str, w.values())))
@pytest.mark.parametrize("B,H,Hkv,Sq,Skv,D,dtype", WINDOW_SHAPES)
def test_window_fwd(B, H, Hkv, Sq, Skv, D, dtype, w):
    q, k, v = make(Sq + D, B, H, Hkv, Sq, Skv, D, dtype)
    bad_q, bad = spoil(q, Sq)
    for out_dtype in (torch.bfloat16, torch.float32):
        for at in (dict(q_pos=Skv - min(Sq, Skv)), dict(q_pos=0, k_pos=min(70, Sq // 2))):
            a = {**w, **at}
            check(cp.window_fwd(bad_q, k, v, out_dtype=out_dtype, **a),
                  cp.window_fwd(q, k, v, out_dtype=out_dtype, **a), bad, seen_by(q, Skv, **a))


@pytest.mark.parametrize("B,H,Hkv,Sq,S,D,dtype", [
    (3, 8, 2, 1, 900, 128, torch.bfloat16), (2, 4, 4, 2, 2000, 64, torch.bfloat16), (1, 32, 1, 1, 64, 128, torch.bfloat16),
    (4, 32, 8, 50, 600, 128, torch.bfloat16), (8, 32, 8, 32, 2000, 64, torch.bfloat16),
    (3, 8, 2, 1, 700, 64, torch.float32), (1, 8, 8, 1, 3000, 128, torch.float32)])
@pytest.mark.parametrize("w", [dict(left=-1), dict(left=100, sinks=4)])
def test_window_decode(B, H, Hkv, Sq, S, D, dtype, w):
    q, k, v = make(B + S, B, H, Hkv, Sq, S, D, dtype)
    bad_q, bad = spoil(q, S)
    n = [S, 0, S // 3, 1, 40, 700, 1999, 3][:B]
    lens = torch.tensor(n, dtype=torch.int32, device=DEV)
    sees = torch.stack([torch.arange(Sq) + x - Sq >= 0 for x in n])[..., None].expand(B, Sq, H).to(DEV)
    for out_dtype in (torch.bfloat16, torch.float32):
        check(cp.window_decode(bad_q, k, v, lens, out_dtype=out_dtype, **w),
              cp.window_decode(q, k, v, lens, out_dtype=out_dtype, **w), bad, sees)


@pytest.mark.parametrize("B,H,Hkv,Sq,Skv,D", [(1, 24, 24, 900, 900, 128), (1, 2, 1, 300, 900, 64)])
@pytest.mark.parametrize("acc", [torch.bfloat16, torch.float32, "run"])
def test_merging_calls(B, H, Hkv, Sq, Skv, D, acc):
    # rows 0..99 see no key of this chunk, the rest do: a NaN query that sees one gives NaN, whatever ran before
    q, k, v = make(7 + Sq, B, H, Hkv, Sq, Skv, D)
    bad_q, bad = spoil(q, 3)
    w = dict(left=50, right=0, q_pos=100, k_pos=200)
    sees = seen_by(q, Skv, **w)
    dt = torch.float32 if acc == "run" else acc
    g = torch.Generator().manual_seed(5)
    o0 = torch.randn(q.shape, generator=g).to(dt).to(DEV)
    l0 = torch.randn(B, H, Sq, generator=g).to(DEV)
    l0[:, :, ::3] = -math.inf

    def step(x):
        o, l = o0.clone(), l0.clone()
        if acc == "run":
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
            return cp.window_fwd(x, k, v, out=out, run=o, lse=l, accumulate=True, **w)
        return cp.window_fwd(x, k, v, out=o, lse=l, accumulate=True, **w)

    got, want = step(bad_q), step(q)
    torch.cuda.synchronize()
    hit = bad & sees
    assert (bad & ~sees).any()
    assert torch.isnan(got[0][hit]).all() and torch.isnan(got[1].transpose(1, 2)[hit]).all()
    assert torch.equal(got[0][~hit], want[0][~hit])
    assert torch.equal(got[1].transpose(1, 2)[~hit], want[1].transpose(1, 2)[~hit])


@pytest.mark.parametrize("kw", [dict(), dict(acc_dtype=torch.bfloat16), dict(acc_dtype=torch.float32)])
def test_windowed_ring_step(kw):
    q, k, v = make(11, 1, 4, 2, 260, 900, 128)
    bad_q, bad = spoil(q, 8)
    cuts = [0, 1, 200, 456, 900]
    ks = [k[:, a:b].contiguous() for a, b in zip(cuts, cuts[1:])]
    vs = [v[:, a:b].contiguous() for a, b in zip(cuts, cuts[1:])]
    w = dict(left=150, right=100, sinks=6, q_pos=300, **kw)
    got, want = cp.ring_attention(bad_q, ks, vs, **w), cp.ring_attention(q, ks, vs, **w)
    check(got, want, bad, torch.ones_like(bad))


# ------------------------------------------------------------------ merges and folds

@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (128, torch.float32), (96, torch.float32), (512, torch.float32)])
def test_merge(D, dtype):
    B, S, H = 2, 70, 3
    g = torch.Generator().manual_seed(D)
    o = [torch.randn(B, S, H, D, generator=g).to(dtype).to(DEV) for _ in range(2)]
    l = [torch.randn(B, H, S, generator=g).to(DEV) for _ in range(2)]
    for t, part in enumerate((slice(0, 20), slice(20, 40))):  # NaN on one side, nothing on the other
        o[t][:, part], l[t][:, :, part] = NAN, NAN
        o[1 - t][:, part], l[1 - t][:, :, part] = 0, -math.inf
    o[0][:, 40:45], l[0][:, :, 40:45] = NAN, NAN  # beside an ordinary part
    for t in range(2):  # nothing on both
        o[t][:, 45:50], l[t][:, :, 45:50] = 0, -math.inf
    out, lse = cp.merge(o[0], l[0], o[1], l[1])
    torch.cuda.synchronize()
    assert torch.isnan(out[:, :45]).all() and torch.isnan(lse[:, :, :45]).all()
    assert (out[:, 45:50] == 0).all() and torch.isneginf(lse[:, :, 45:50]).all()
    assert torch.isfinite(out[:, 50:]).all() and torch.isfinite(lse[:, :, 50:]).all()


@pytest.mark.parametrize("n_split", [1, 2, 5, 0])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_fwd_split(n_split, accumulate, out_dtype):
    q, k, v = make(13, 1, 80, 80, 300, 700, 64)  # 160 items: with n_split = 0 the last 12 are shared out
    bad_q, bad = spoil(q, 2)

    def step(x):
        o = torch.zeros(q.shape, dtype=out_dtype, device=DEV)
        l = torch.full((1, 80, 300), -math.inf, device=DEV)  # an empty running result
        return cp.fwd_split(x, k, v, out=o, lse=l, accumulate=accumulate, n_split=n_split)

    check(step(bad_q), step(q), bad, torch.ones_like(bad))


# ------------------------------------------------------------------ norms

def spoil_rows(x, seed, value=NAN):
    flat = x.reshape(1, -1, 1, x.shape[-1])
    y, bad = spoil(flat, seed, value)
    return y.reshape(x.shape), bad.reshape(x.shape[:-1])


def check_rows(got, want, bad):
    torch.cuda.synchronize()
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("D", [8, 64, 128, 256])
def test_rmsnorm(D, value):
    x, _, _ = make(17, 1, 5, 1, 40, 1, D)
    y, bad = spoil_rows(x, D, value)
    g = torch.ones(D, device=DEV)
    check_rows(cp.rmsnorm(y, g), cp.rmsnorm(x, g), bad)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [NAN, math.inf])
@pytest.mark.parametrize("D,rot", [(128, 128), (256, 64), (64, 32), (72, 20)])
def test_qk_norm_rope(D, rot, value, dtype):
    q, k, _ = (t[0] for t in make(18, 1, 5, 2, 40, 40, D, dtype))
    q2, bad_q = spoil_rows(q, 1, value)
    k2, bad_k = spoil_rows(k, 2, value)
    g = torch.ones(D, device=DEV)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)
    freq = cp.rope_frequencies(rot, device=DEV)[0]
    for inter in (False, True):
        got, want = (cp.qk_norm_rope(a, b, g, g, pos, freq, interleaved=inter) for a, b in ((q2, k2), (q, k)))
        check_rows(got[0], want[0], bad_q)
        check_rows(got[1], want[1], bad_k)


@pytest.mark.parametrize("rope", [False, True])
def test_seq2head_norm(rope):
    P, S_l, H, D = 2, 21, 4, 64
    q, k, v = (t.reshape(P, S_l, H, D) for t in make(19, 1, H, H, P * S_l, P * S_l, D))
    q2, bad = spoil_rows(q, 4)
    g = torch.ones(D, device=DEV)
    pos = torch.arange(P * S_l, dtype=torch.int32, device=DEV)
    freq = cp.rope_frequencies(D, device=DEV)[0]
    step = lambda x: (cp.seq2head_qkv_norm_rope(x, k, v, P, g, g, pos, freq) if rope
                      else cp.seq2head_qkv_norm(x, k, v, P, g, g))
    got, want = step(q2), step(q)
    where = cp.seq2head(bad[..., None].expand(P, S_l, H, D).bfloat16().contiguous(), P)
    torch.cuda.synchronize()
    check_rows(got[0], want[0], where[..., 0] == 1)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
