"""Cases of the windowed-attention and rotary-position operators: inputs, the calls a user
makes of them, their plain forms in torch, and their values in 64 bits.

Four operators:

* ``window``  attention of a query slice over a key slice, limited to a window around each
  query's position and the first ``sinks`` positions, with its log-sum-exp; ``chunks`` > 1 runs
  it as one rank's ring step, chunk by chunk into a running (O, LSE)
* ``decode``  the last token(s) of each sequence against its key/value cache
* ``rope``    rotary positions of one tensor
* ``norm``    RMSNorm of query and key heads with the rotation in the same pass; ``P`` > 0 is
  the form fused into the Ulysses sequence -> head re-partition
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # image tokens of the joint image + text sequence, each looking 512 tokens to either
        # side and at the 512 text tokens in front
        window("window_image_4608", B=1, H=24, Hkv=24, Sq=4608, Skv=4608, D=128, left=512, right=512,
               sinks=512),
        # the video latent, causal over the last 4096 tokens with the first frame's tokens kept
        window("window_video_44160", B=1, H=16, Hkv=16, Sq=44160, Skv=44160, D=128, left=4096, right=0,
               sinks=64),
        # one rank's ring step: its 5520 queries against its own chunk and both neighbours
        window("window_ring_5520x3", B=1, H=16, Hkv=16, Sq=5520, Skv=16560, D=128, left=3000, right=3000,
               q_pos=5520, chunks=3),
        # a prefill slice of a padded batch after 444 tokens already in place, grouped heads
        window("window_prefill_gqa_333", B=3, H=8, Hkv=2, Sq=333, Skv=777, D=64, left=255, right=0, sinks=4,
               q_pos=444, padded=True),
        # the float32 form
        window("window_f32_1000", B=1, H=4, Hkv=4, Sq=1000, Skv=1000, D=64, left=200, right=100, sinks=8,
               dtype="f32"),
        # one token of one sequence: latency
        decode("decode_1x32", B=1, H=32, Hkv=8, Sq=1, S_max=8192, D=128, left=1023, sinks=4, least=5000),
        # a serving batch of ragged lengths
        decode("decode_64x32", B=64, H=32, Hkv=8, Sq=1, S_max=8192, D=128, left=4095, sinks=4, least=100),
        # four tokens a step (drafted ahead), one head per key head
        decode("decode_8x16_tokens4", B=8, H=16, Hkv=16, Sq=4, S_max=2992, D=64, left=1500, sinks=16,
               least=4),
        # the video latent's queries, rotated by frame, row and column
        rope("rope_video_44160", tokens=44160, H=16, D=128, rot=128, axes=3, interleaved=True),
        # a decode step's keys, part of the head, far positions of a stretched context
        rope("rope_decode_far", tokens=17, H=8, D=64, rot=32, axes=1, scaled=True, far=True),
        # the video shards of 8 ranks: norm, rotation and re-partition of Q and K (V moves along)
        norm("norm_ulysses_44160", tokens=44160, H=16, Hk=16, D=128, rot=128, axes=3, interleaved=True, P=8),
        # query and key heads out of a fused projection (strided), grouped heads
        norm("norm_image_4608", tokens=4608, H=24, Hk=8, D=128, rot=128, axes=1, fused=True),
    ]


def window(name=None, **kw):
    c = dict(op="window", B=1, left=-1, right=-1, sinks=0, q_pos=0, chunks=1, padded=False, dtype="bf16")
    return named(c, kw, name)


def decode(name=None, **kw):
    return named(dict(op="decode", dtype="bf16"), kw, name)


def rope(name=None, **kw):
    c = dict(op="rope", interleaved=False, scaled=False, far=False, dtype="bf16")
    return named(c, kw, name)


def norm(name=None, **kw):
    c = dict(op="norm", interleaved=False, scaled=False, far=False, fused=False, P=0, dtype="bf16")
    return named(c, kw, name)


def named(c, kw, name):
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("window", "window", "decode", "decode", "rope", "norm"))
    if kind == "window":
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        D = rng.choice((64, 128))
        Hkv = rng.choice((1, 2, 3, 4, 8, 16) if dtype == "bf16" else (1, 2, 3, 4))
        H = Hkv * (rng.choice((1, 2, 4)) if Hkv <= 8 else 1)
        Sq = log_int(rng, 200, 30000 if dtype == "bf16" else 3000)
        causal = rng.random() < 0.5
        chunks = rng.choice((1, 1, 1, 2, 4)) if dtype == "bf16" else 1
        before = log_int(rng, 1, 2000) if rng.random() < 0.5 else 0
        left = log_int(rng, 64, 8000)
        right = 0 if causal else log_int(rng, 1, 4000)
        B = 1 if Sq > 4000 else rng.randint(1, 3)
        # no more (row, key) pairs x width than the largest listed case
        most = 44160 * 4161 * 16 * 128 // 2
        while B * H * D * Sq * min(Sq + before, left + right + 1) > most:
            Sq = Sq // 2 + 1
        after = 0 if causal else rng.choice((0, 0, 37, 500))
        return window(B=B, H=H, Hkv=Hkv, Sq=Sq, Skv=before + Sq + after, D=D, left=left, right=right,
                      sinks=rng.choice((0, 4, 64, 300)), q_pos=before, chunks=chunks,
                      padded=causal and B > 1 and chunks == 1, dtype=dtype)
    if kind == "decode":
        Hkv = rng.choice((1, 2, 4, 8, 16))
        H = Hkv * rng.choice((1, 2, 4, 8))
        B = log_int(rng, 1, 64)
        S_max = log_int(rng, 300, 8192)
        return decode(B=B, H=H, Hkv=Hkv, Sq=rng.choice((1, 1, 1, 2, 5)), S_max=S_max, D=rng.choice((64, 128)),
                      left=log_int(rng, 100, 6000), sinks=rng.choice((0, 4, 32)), least=S_max // 3)
    rot_of = {64: (64, 32), 128: (128, 64, 96), 80: (80, 48), 256: (256, 64)}
    D = rng.choice(tuple(rot_of))
    common = dict(D=D, rot=rng.choice(rot_of[D]), interleaved=rng.random() < 0.5, scaled=rng.random() < 0.3,
                  far=rng.random() < 0.3, axes=rng.choice((1, 1, 2, 3)))
    if kind == "rope":
        return rope(tokens=log_int(rng, 1, 20000), H=rng.choice((1, 3, 8, 16)),
                    dtype=rng.choice(("bf16", "bf16", "f32")), **common)
    P = rng.choice((0, 0, 2, 4, 8))
    if P:
        return norm(tokens=P * log_int(rng, 3, 2500), H=16, Hk=16, P=P, **common)
    Hk = rng.choice((1, 2, 8))
    return norm(tokens=log_int(rng, 1, 20000), H=Hk * rng.choice((1, 3, 4)), Hk=Hk,
                fused=rng.random() < 0.5, **common)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=dt, sigma=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32) * sigma).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op == "window":
        B, H, Hkv, D = (case[n] for n in ("B", "H", "Hkv", "D"))
        s["q"] = randn(B, case["Sq"], H, D)
        s["k"] = randn(B, case["Skv"], Hkv, D)
        s["v"] = randn(B, case["Skv"], Hkv, D)
        s["kv_len"] = torch.tensor(lengths(case), dtype=torch.int32, device=DEV) if case["padded"] else None
        s["out"] = torch.empty(B, case["Sq"], H, D, dtype=dt, device=DEV)
        s["lse"] = torch.empty(B, H, case["Sq"], dtype=torch.float32, device=DEV)
        # a ring's chunks are buffers of their own
        at = chunk_starts(case)
        s["k_chunks"] = [s["k"][:, a:b].contiguous() for a, b in at] if len(at) > 1 else [s["k"]]
        s["v_chunks"] = [s["v"][:, a:b].contiguous() for a, b in at] if len(at) > 1 else [s["v"]]
        if len(at) > 1:
            del s["k"], s["v"]
    elif op == "decode":
        B, H, Hkv, D = (case[n] for n in ("B", "H", "Hkv", "D"))
        s["q"] = randn(B, case["Sq"], H, D)
        s["k"] = randn(B, case["S_max"], Hkv, D)
        s["v"] = randn(B, case["S_max"], Hkv, D)
        s["kv_len"] = torch.tensor(lengths(case), dtype=torch.int32, device=DEV)
        s["out"] = torch.empty(B, case["Sq"], H, D, dtype=dt, device=DEV)
        s["lse"] = torch.empty(B, H, case["Sq"], dtype=torch.float32, device=DEV)
    else:
        T, H, D = case["tokens"], case["H"], case["D"]
        s["freq"] = frequencies(case).to(DEV)
        s["factor"] = attention_factor(case)
        s["pos"] = positions(case, gen)
        if op == "rope":
            s["x"] = randn(T, H, D)
            s["out"] = torch.empty(T, H, D, dtype=dt, device=DEV)
        else:
            Hk = case["Hk"]
            for n in ("gamma_q", "gamma_k"):
                s[n] = 1.0 + 0.1 * torch.randn(D, generator=gen, device=DEV, dtype=torch.float32)
            if case["P"]:
                P = case["P"]
                for n in "qkv":
                    s[n] = randn(P, T // P, H, D, sigma=2.0)
                s["out"] = tuple(torch.empty(P, T, H // P, D, dtype=dt, device=DEV) for _ in range(3))
            else:
                if case["fused"]:  # one projection's output: query, key and value heads of a token together
                    qkv = randn(T, H + 2 * Hk, D, sigma=2.0)
                    s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + Hk]
                else:
                    s["q"], s["k"] = randn(T, H, D, sigma=2.0), randn(T, Hk, D, sigma=2.0)
                s["out"] = (torch.empty(T, H, D, dtype=dt, device=DEV),
                            torch.empty(T, Hk, D, dtype=dt, device=DEV))
    return s


def lengths(case):
    """Tokens of each sequence: the same for every seed, so that the work is known."""
    rng = random.Random(case["B"] * 1000 + case["D"])
    if case["op"] == "window":  # right-padded: the first sequence is whole
        return [case["Skv"] - (rng.randrange(case["Skv"] // 4) if b else 0) for b in range(case["B"])]
    return [rng.randint(min(case["least"], case["S_max"]), case["S_max"]) for _ in range(case["B"])]


def chunk_starts(case):
    n, size = case["chunks"], -(-case["Skv"] // case["chunks"])
    return [(c * size, min(case["Skv"], (c + 1) * size)) for c in range(n)]


def frequencies(case):
    """Radians per position of each rotated pair, [axes][rot/2] in 64 bits: an axis turns its own
    share of the pairs.  ``scaled`` stretches a context of 4096 eight times, by parts: fast pairs
    as they are, slow pairs at an eighth, a ramp between."""
    half, axes = case["rot"] // 2, case["axes"]
    f = torch.zeros(axes, half, dtype=torch.float64)
    cut = [half * a // axes for a in range(axes + 1)]
    for a in range(axes):
        n = cut[a + 1] - cut[a]
        w = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
        if case["scaled"]:
            turns = 4096 * w / (2 * math.pi)
            keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
            w = w / 8 * (1 - keep) + w * keep
        f[a, cut[a]:cut[a + 1]] = w
    return f


def attention_factor(case):
    return 0.1 * math.log(8.0) + 1.0 if case["scaled"] else 1.0


def positions(case, gen):
    """int32 [tokens][axes]: consecutive tokens (a grid in frame, row, column order), or, ``far``,
    tokens of a context of millions."""
    T, A = case["tokens"], case["axes"]
    t = torch.arange(T, device=DEV)
    if A == 1:
        pos = t[:, None]
    elif A == 2:
        pos = torch.stack((t // 64, t % 64), 1)
    else:
        pos = torch.stack((t // 1840, t // 46 % 40, t % 46), 1)
    off = torch.randint(0, 4000000 if case["far"] else 1000, (1, A), generator=gen, device=DEV)
    return (pos + off).to(torch.int32)


# ------------------------------------------------------------------ the calls

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import context_long_sequence_non_b200 as cp

        if op == "window":
            if case["chunks"] > 1:
                return cp.ring_attention(s["q"], s["k_chunks"], s["v_chunks"], left=case["left"],
                                         right=case["right"], sinks=case["sinks"], q_pos=case["q_pos"])
            return cp.window_fwd(s["q"], s["k"], s["v"], left=case["left"], right=case["right"],
                                 sinks=case["sinks"], q_pos=case["q_pos"], kv_len=s["kv_len"], out=s["out"],
                                 lse=s["lse"])
        if op == "decode":
            return cp.window_decode(s["q"], s["k"], s["v"], s["kv_len"], left=case["left"],
                                    sinks=case["sinks"], out=s["out"], lse=s["lse"])
        if op == "rope":
            return cp.rope(s["x"], s["pos"], s["freq"], interleaved=case["interleaved"], factor=s["factor"],
                           out=s["out"])
        if case["P"]:
            return cp.seq2head_qkv_norm_rope(s["q"], s["k"], s["v"], case["P"], s["gamma_q"], s["gamma_k"],
                                             s["pos"], s["freq"], interleaved=case["interleaved"],
                                             factor=s["factor"], out=s["out"])
        return cp.qk_norm_rope(s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["pos"], s["freq"],
                               interleaved=case["interleaved"], factor=s["factor"], out=s["out"])
    if op == "window":
        return plain_window(s)
    if op == "decode":
        return plain_decode(s)
    if op == "rope":
        cos, sin = plain_angles(s)
        return plain_rotate(s["x"].float(), cos, sin, case).to(s["x"].dtype)
    cos, sin = plain_angles(s)
    if case["P"]:
        P, T, H, D = case["P"], case["tokens"], case["H"], case["D"]

        def group(x):  # [P][S_l][H][D] shards -> [P][P*S_l][H/P][D] head groups
            return x.reshape(T, P, H // P, D).transpose(0, 1).contiguous()

        q, k = (plain_rotate(plain_norm(s[n].reshape(T, H, D), s["gamma_" + n]), cos, sin, case).to(s[n].dtype)
                for n in "qk")
        return group(q), group(k), group(s["v"])
    return tuple(plain_rotate(plain_norm(s[n], s["gamma_" + n]), cos, sin, case).to(s[n].dtype) for n in "qk")


# ------------------------------------------------------------------ plain forms

def row_blocks(case, keys):
    """Query rows at a time, so that a block's scores stay near 2^27 values."""
    step = max(64, min(case["Sq"], (1 << 27) // (case["B"] * case["H"] * max(keys, 1))))
    return [(i, min(case["Sq"], i + step)) for i in range(0, case["Sq"], step)]


def span(case, i0, i1):
    """Keys that rows i0 .. i1-1 can see beside the sinks: [lo, hi)."""
    lo = 0 if case["left"] < 0 else max(0, case["q_pos"] + i0 - case["left"])
    hi = case["Skv"] if case["right"] < 0 else min(case["Skv"], case["q_pos"] + i1 + case["right"])
    return lo, max(lo, hi)


def plain_window(s):
    case = s["case"]
    q = s["q"]
    k, v = torch.cat(s["k_chunks"], 1), torch.cat(s["v_chunks"], 1)
    B, H, Hkv, D = (case[n] for n in ("B", "H", "Hkv", "D"))
    G = H // Hkv
    out, lse = torch.empty_like(q), torch.empty(B, H, case["Sq"], dtype=torch.float32, device=q.device)
    width = case["Skv"] if case["left"] < 0 or case["right"] < 0 else case["left"] + case["right"] + case["sinks"]
    for i0, i1 in row_blocks(case, min(case["Skv"], width + 1024)):
        lo, hi = span(case, i0, i1)
        first = min(case["sinks"], lo)
        key = torch.cat((torch.arange(first, device=q.device), torch.arange(lo, hi, device=q.device)))
        qp = case["q_pos"] + torch.arange(i0, i1, device=q.device)[:, None]
        seen = torch.ones(i1 - i0, key.numel(), dtype=torch.bool, device=q.device)
        if case["right"] >= 0:
            seen &= key <= qp + case["right"]
        if case["left"] >= 0:
            seen &= (key >= qp - case["left"]) | (key < case["sinks"])
        seen = seen.expand(B, 1, 1, *seen.shape)
        if s["kv_len"] is not None:
            seen = seen & (key < s["kv_len"][:, None]).view(B, 1, 1, 1, -1)
        kf = torch.cat((k[:, :first], k[:, lo:hi]), 1).float().permute(0, 2, 1, 3).unsqueeze(2)
        vf = torch.cat((v[:, :first], v[:, lo:hi]), 1).float().permute(0, 2, 1, 3).unsqueeze(2)
        qf = q[:, i0:i1].float().reshape(B, i1 - i0, Hkv, G, D).permute(0, 2, 3, 1, 4)
        x = torch.matmul(qf, kf.transpose(-1, -2)) * (1.0 / math.sqrt(D))
        x = torch.where(seen, x, -math.inf)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        p = torch.exp(x - m)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, vf) / torch.where(total == 0, 1.0, total)
        out[:, i0:i1] = o.permute(0, 3, 1, 2, 4).reshape(B, i1 - i0, H, D).to(out.dtype)
        lse[:, :, i0:i1] = (m + torch.log(total)).reshape(B, H, i1 - i0)
    return out, lse


def decode_keys(case, kv_len):
    """Keys of each sequence that its last tokens can see: index [B][n], and whether [B][Sq][n]."""
    n_near, sinks = min(case["S_max"], case["left"] + case["Sq"]), min(case["sinks"], case["S_max"])
    L = kv_len.long()[:, None]
    near = L - n_near + torch.arange(n_near, device=L.device)
    early = torch.arange(sinks, device=L.device).expand(L.shape[0], sinks)
    key = torch.cat((early, near), 1)
    ok = torch.cat((early < torch.clamp(L - n_near, min=0), near >= 0), 1)  # each key once
    qp = L - case["Sq"] + torch.arange(case["Sq"], device=L.device)  # [B][Sq]
    key3, qp3 = key[:, None], qp[:, :, None]
    seen = ok[:, None] & (key3 <= qp3) & ((key3 >= qp3 - case["left"]) | (key3 < case["sinks"]))
    return key.clamp(0, case["S_max"] - 1), seen


def plain_decode(s):
    case = s["case"]
    q, k, v = s["q"], s["k"], s["v"]
    B, H, Hkv, D, Sq = (case[n] for n in ("B", "H", "Hkv", "D", "Sq"))
    G = H // Hkv
    index, seen = decode_keys(case, s["kv_len"])
    b = torch.arange(B, device=q.device)[:, None]
    kf = k[b, index].float().permute(0, 2, 1, 3)  # [B][Hkv][n][D]
    vf = v[b, index].float().permute(0, 2, 1, 3)
    qf = q.float().reshape(B, Sq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Sq, D)
    x = torch.matmul(qf, kf.transpose(-1, -2)).reshape(B, Hkv, G, Sq, -1) * (1.0 / math.sqrt(D))
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, G * Sq, -1), vf).reshape(B, Hkv, G, Sq, D)
    o = o / torch.where(total == 0, 1.0, total)
    out = o.permute(0, 3, 1, 2, 4).reshape(B, Sq, H, D).to(q.dtype)
    return out, (m + torch.log(total)).reshape(B, H, Sq)


def plain_angles(s):
    turn = s["pos"].double() @ s["freq"]  # [tokens][rot/2]: far positions lose their angle in 32 bits
    return (torch.cos(turn) * s["factor"]).float(), (torch.sin(turn) * s["factor"]).float()


def plain_norm(x, gamma):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma


def plain_rotate(x, cos, sin, case):
    """x [tokens][heads][D] in 32 bits; cos, sin [tokens][rot/2]."""
    rot = case["rot"]
    cos, sin = cos[:, None], sin[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


# ------------------------------------------------------------------ values in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "window":
        return exact_window(s)
    if op == "decode":
        return exact_decode(s)
    if op == "rope":
        return exact_rotation(s, s["x"].double())
    res = []
    for n in "qk":
        x = s[n].reshape(case["tokens"], -1, case["D"]).double()
        mean = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / case["D"]
        res.append(exact_rotation(s, x / torch.sqrt(mean + 1e-6) * s["gamma_" + n].double()))
    if case["P"]:
        P, T, D = case["P"], case["tokens"], case["D"]
        res.append(s["v"].reshape(T, -1, D).double())
        Hp = case["H"] // P
        res = [torch.stack([x[:, g * Hp:(g + 1) * Hp] for g in range(P)]) for x in res]
    return tuple(res)


def exact_rotation(s, x):
    """Each pair as a complex number, times e^(i angle)."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    angle = (s["pos"].double()[:, :, None] * s["freq"][None]).sum(1)
    z = torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]
    pair = torch.arange(half, device=x.device)
    re, im = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + half)
    w = torch.complex(x[..., re], x[..., im]) * z
    y = x.clone()
    y[..., re], y[..., im] = w.real, w.imag
    return y


def exact_window(s):
    """Head by head: softmax over the keys that a row's window and the sinks let it see."""
    case = s["case"]
    B, H, Hkv, D, Sq = (case[n] for n in ("B", "H", "Hkv", "D", "Sq"))
    q = s["q"]
    k, v = torch.cat(s["k_chunks"], 1), torch.cat(s["v_chunks"], 1)
    out = torch.empty(B, Sq, H, D, dtype=torch.float64, device=q.device)
    lse = torch.empty(B, H, Sq, dtype=torch.float64, device=q.device)
    have = [case["Skv"]] * B if s["kv_len"] is None else lengths(case)
    for b in range(B):
        for h in range(H):
            kh, vh = k[b, :have[b], h * Hkv // H].double(), v[b, :have[b], h * Hkv // H].double()
            for i0 in range(0, Sq, 2048):
                i1 = min(Sq, i0 + 2048)
                lo, hi = span(case, i0, i1)
                hi = min(hi, have[b])
                lo = min(lo, hi)
                j = torch.tensor([t for t in range(min(case["sinks"], lo))] + list(range(lo, hi)),
                                 device=q.device, dtype=torch.long)
                far = j[None] - (case["q_pos"] + torch.arange(i0, i1, device=q.device))[:, None]
                hide = torch.zeros_like(far, dtype=torch.bool)
                if case["left"] >= 0:
                    hide |= (far < -case["left"]) & (j >= case["sinks"])
                if case["right"] >= 0:
                    hide |= far > case["right"]
                x = (q[b, i0:i1, h].double() @ kh[j].T / math.sqrt(D)).masked_fill(hide, -math.inf)
                L = torch.logsumexp(x, -1)
                lse[b, h, i0:i1] = L
                out[b, i0:i1, h] = torch.nan_to_num(torch.exp(x - L[:, None])) @ vh[j]
    return out, lse


def exact_decode(s):
    """Sequence by sequence, over the part of the cache that its tokens see."""
    case = s["case"]
    B, H, Hkv, D, Sq = (case[n] for n in ("B", "H", "Hkv", "D", "Sq"))
    q = s["q"]
    out = torch.empty(B, Sq, H, D, dtype=torch.float64, device=q.device)
    lse = torch.empty(B, H, Sq, dtype=torch.float64, device=q.device)
    for b, L in enumerate(lengths(case)):
        for t in range(Sq):
            p = L - Sq + t
            j = [i for i in range(min(case["sinks"], p + 1))]
            j += list(range(max(len(j), p - case["left"]), p + 1))
            j = torch.tensor(j, device=q.device, dtype=torch.long)
            kj = s["k"][b, j].double().repeat_interleave(H // Hkv, 1)  # [n][H][D]
            vj = s["v"][b, j].double().repeat_interleave(H // Hkv, 1)
            x = torch.einsum("hd,nhd->hn", q[b, t].double(), kj) / math.sqrt(D)
            lse[b, :, t] = torch.logsumexp(x, -1)
            out[b, t] = torch.einsum("hn,nhd->hd", torch.softmax(x, -1), vj)
    return out, lse


# ------------------------------------------------------------------ work

def pairs_seen(case):
    """Visible (row, key) pairs of the batch, and the keys that some row sees."""
    pairs = keys = 0
    have = lengths(case) if case["padded"] else [case["Skv"]] * case["B"]
    for L in have:
        top = 0
        low = L
        for i in range(case["Sq"]):
            p = case["q_pos"] + i
            hi = L if case["right"] < 0 else min(L, p + case["right"] + 1)
            lo = 0 if case["left"] < 0 else max(0, p - case["left"])
            lo = min(lo, hi)
            pairs += hi - lo + min(case["sinks"], lo)
            if hi > lo:
                top, low = max(top, hi), min(low, lo)
        keys += max(0, top - low) + min(case["sinks"], low)
    return pairs, keys


def work(case):
    es = {"bf16": 2, "f32": 4}[case["dtype"]]
    op = case["op"]
    if op in ("window", "decode"):
        B, H, Hkv, D, Sq = (case[n] for n in ("B", "H", "Hkv", "D", "Sq"))
        if op == "window":
            pairs, keys = pairs_seen(case)
        else:
            pairs = keys = 0
            for L in lengths(case):
                for t in range(Sq):
                    lo = max(0, L - Sq + t - case["left"])
                    pairs += L - Sq + t + 1 - lo + min(case["sinks"], lo)
                lo = max(0, L - Sq - case["left"])
                keys += L - lo + min(case["sinks"], lo)
        return {"bytes": 2 * B * Sq * H * D * es + 2 * keys * Hkv * D * es + 4 * B * H * Sq,
                "flops": 4 * pairs * H * D}
    T, D, rot = case["tokens"], case["D"], case["rot"]
    small = 4 * T * case["axes"] + 4 * rot * case["axes"]
    if op == "rope":
        return {"bytes": 2 * T * case["H"] * D * es + small, "flops": 3 * T * case["H"] * rot}
    heads = case["H"] + case["Hk"]
    moved = heads + (case["H"] if case["P"] else 0)
    return {"bytes": 2 * T * moved * D * es + small + 8 * D, "flops": T * heads * (4 * D + 3 * rot)}
