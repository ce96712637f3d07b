"""Calls on another stream than the current one, while the current one allocates, writes and frees memory
of the sizes that the call allocates for itself: results must be those of a call on the current stream."""

import pytest
import torch

import context_long_sequence_non_b200 as cp
from context_long_sequence_non_b200 import build as build_mod
from context_long_sequence_non_b200.paths import ulysses_attention

pytestmark = pytest.mark.gpu

DEV = "cuda"
MS = 2_000_000  # about a millisecond of torch.cuda._sleep


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build_mod.build()
    cp.lib()
    yield
    assert cp.device_error() == 0


def make(seed, *shapes, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).to(dtype).to(DEV) for s in shapes]


def calls():
    q, k, v = make(1, (1, 300, 8, 128), (1, 900, 8, 128), (1, 900, 8, 128))
    s = make(2, *[(2, 150, 8, 128)] * 3)
    ks, vs = ([t[:, a:a + 300].contiguous() for a in (0, 300, 600)] for t in (k, v))
    q1 = q[:, :1].contiguous()
    pos = torch.arange(300, dtype=torch.int32, device=DEV)
    freq = cp.rope_frequencies(128, device=DEV)[0]
    gam = torch.ones(128, device=DEV)
    w = dict(left=200, right=50, sinks=4, q_pos=300)
    return {
        "ring windowed": lambda **kw: cp.ring_attention(q, ks, vs, **w, **kw),
        "ring in parts": lambda **kw: cp.ring_attention(q, ks, vs, n_split=2, **kw),
        "ring merged": lambda **kw: cp.ring_attention(q, ks, vs, fused=False, **kw),
        "fwd_split": lambda **kw: cp.fwd_split(q, k, v, n_split=3, **kw),
        "fwd": lambda **kw: cp.fwd(q, k, v, **kw),
        "ulysses": lambda **kw: ulysses_attention(*s, 2, **kw),
        "window_fwd": lambda **kw: cp.window_fwd(q, k, v, **w, **kw),
        "window_decode": lambda **kw: cp.window_decode(q1, k, v, left=200, **kw),
        "qk_norm_rope": lambda **kw: cp.qk_norm_rope(q, q, gam, gam, pos, freq, **kw),
    }


NAMES = ["ring windowed", "ring in parts", "ring merged", "fwd_split", "fwd", "ulysses", "window_fwd", "window_decode",
         "qk_norm_rope"]
SIZES = [1 << n for n in range(9, 23)] + [300 * 8 * 128 * 2, 300 * 8 * 128 * 4, 300 * 8 * 4, 8 * 128 * 2, 900 * 8 * 128 * 2]


def junk():
    """Blocks of the sizes that the calls allocate, filled on the current stream."""
    return [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in SIZES for _ in range(4)]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("keep", [0, 1])  # the result that the caller keeps; the other is dropped at once
def test_memory_taken_by_the_current_stream_meanwhile(name, keep):
    call = calls()[name]
    want = call()[keep].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10 * MS)
    got = call(stream=side)[keep]
    others = junk()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all((t == 0x7F).all() for t in others)


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_writes(name):
    call = calls()[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    blocks = junk()
    torch.cuda.synchronize()
    torch.cuda._sleep(10 * MS)
    for t in blocks:
        t.fill_(1)
    del blocks, t  # freed for the current stream, which has yet to write them
    got = call(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_results_dropped_while_the_current_stream_reads_them():
    call = calls()["window_fwd"]
    want = call()[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(10 * MS)
    copy = out.clone()
    del out
    with torch.cuda.stream(side):
        junk()
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def test_captured_compositions_follow_their_inputs():
    # ring steps with a window (their temporaries in the graph's memory) and a Ulysses layer with norm, rotation
    # and window, in two graphs replayed beside one another
    P, S_l, H, D = 2, 150, 8, 128
    q, k, v = make(5, *[(1, 300, H, D)] * 3)
    s = make(6, *[(P, S_l, H, D)] * 3)
    f = [t.float() for t in (q, k, v)]
    pos = torch.arange(P * S_l, dtype=torch.int32, device=DEV)
    gam = torch.ones(D, device=DEV)
    plans = [cp.UlyssesPlan(P, S_l, H, D, qk_norm=(gam, gam), rope=(pos, cp.rope_frequencies(D, device=DEV)[0]),
                            window=(60, 20, 4)) for _ in range(2)]

    def step(plan):
        ring = lambda a, b, c, **kw: cp.ring_attention(a, [b[:, :100], b[:, 100:]], [c[:, :100], c[:, 100:]], left=90,
                                                       right=30, sinks=3, **kw)
        return [*ring(q, k, v), *ring(q, k, v, acc_dtype=torch.float32), *ring(*f), *plan.run(*s)]

    graphs, outs = [], []
    step(plans[0])
    for plan in plans:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(plan))
        graphs.append(g)
    fresh = cp.UlyssesPlan(P, S_l, H, D, qk_norm=(gam, gam), rope=plans[0].rope, window=(60, 20, 4))
    for seed in range(2):
        for t in (q, k, v, *s, *f):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(seed + t.numel() % 7)))
        want = [t.clone() for t in step(fresh)]
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
        torch.cuda.synchronize()
        for got in outs:
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_calls_on_a_side_stream_of_a_capture():
    # the side stream joins the capture; what the calls allocate there is the graph's, dropped results among it
    q, k, v = make(9, (1, 300, 8, 128), (1, 900, 8, 128), (1, 900, 8, 128))
    ks, vs = ([t[:, a:a + 300].contiguous() for a in (0, 300, 600)] for t in (k, v))
    w = dict(left=200, right=50, sinks=4, q_pos=300)
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        a = cp.ring_attention(q, ks, vs, stream=side, **w)
        cp.window_fwd(q, k, v, stream=side, **w)
        b = cp.window_fwd(q, k, v, stream=side, **w)[0]
        here.wait_stream(side)
        c = cp.rmsnorm(b, torch.ones(128, device=DEV))
        return [*a, b, c]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(7)
        g.replay()
        junk()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
