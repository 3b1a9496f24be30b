"""The attention half of a diffusion transformer block beside the 4-bit linears: an 8-bit
integer linear, rotary positions with several axes, and block-sparse attention.

``listed()`` gives the measured cases, ``draw(rng)`` more of the same ranges, ``prepare`` the
inputs on the GPU, ``run`` one pass (``own`` false: elementary torch operations in 32 bits;
true: the library's calls), ``work`` the bytes and operations a pass cannot do without, and
``exact`` the outputs from the definitions in 64 bits.

Operators
  i8    Y = act((qa . qw) sa sw + bias): bf16 activations quantized to 8 bits per token
        (after an optional smoothing), int8 weights with one scale per output channel.
  rope  cos and sin tables [S, D/2] of tokens with several position axes.
  turn  [M, 3 H D] projections -> per-head RMS norm and rotary turn of Q and K -> Q, K, V in
        the attention layout [B, H, S, D].
  attn  attention of every block of 128 queries over the key blocks (64 keys) whose mean has
        the highest product with the query block's mean.
"""
import math

import torch

own = False

QUERY_BLOCK = 128
KEY_BLOCK = 64


# ------------------------------------------------------------------ cases

def listed():
    return [
        # --- 8-bit linear: one token through a modulation projection (latency and the weight
        # stream), a ragged text prompt, the fused QKV projection of 4096 image + 512 text
        # tokens, and the two halves of the MLP (GELU; smoothing; the long K).
        dict(name="i8_one_token", op="i8", M=1, K=4096, N=24576, act=0, bias=True, smooth=False),
        dict(name="i8_text", op="i8", M=333, K=4096, N=4096, act=0, bias=True, smooth=True),
        dict(name="i8_mlp_up", op="i8", M=4096, K=4096, N=16384, act=1, bias=True, smooth=True),
        dict(name="i8_mlp_down", op="i8", M=4608, K=12288, N=4096, act=0, bias=False, smooth=True),
        # --- rotary tables: an image of 64 x 64 patches behind 512 text tokens; a video clip
        # far into a long stream (time positions past 10^6).
        dict(name="rope_image", op="rope", text=512, t=1, h=64, w=64, far=0, dims="16,56,56",
             theta=10000.0),
        dict(name="rope_video", op="rope", text=0, t=33, h=45, w=80, far=1048576, dims="44,42,42",
             theta=10000.0),
        # --- norm and turn: one token (a new frame's first), the 4608 tokens of an image with
        # 24 heads of 128, a batch of odd lengths with heads of 64.
        dict(name="turn_one_token", op="turn", B=1, S=1, H=24, D=128, norm=True),
        dict(name="turn_image", op="turn", B=1, S=4608, H=24, D=128, norm=True),
        dict(name="turn_ragged", op="turn", B=3, S=3001, H=18, D=64, norm=True),
        # --- sparse attention: one query row over a long prefix, a padded batch of images with
        # their text blocks always taken, a video clip of 21 x 30 x 52 patches.
        dict(name="attn_one_query", op="attn", B=2, H=16, G=4, D=128, Sq=1, Sk=20000, keep=32,
             first=1, pad=777),
        dict(name="attn_image_batch", op="attn", B=2, H=24, G=24, D=128, Sq=4608, Sk=4608, keep=24,
             first=8, pad=300),
        dict(name="attn_video", op="attn", B=1, H=12, G=12, D=128, Sq=32760, Sk=32760, keep=64,
             first=0, pad=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["i8", "i8", "rope", "turn", "attn", "attn"])
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        if op == "i8":
            c = dict(op=op, M=_log_int(rng, 1, 8192), K=64 * _log_int(rng, 2, 256),
                     N=8 * _log_int(rng, 16, 4000), act=rng.randint(0, 1),
                     bias=rng.random() < 0.7, smooth=rng.random() < 0.5)
        elif op == "rope":
            c = dict(op=op, text=rng.choice([0, 1, rng.randint(2, 600)]), t=_log_int(rng, 1, 64),
                     h=_log_int(rng, 1, 128), w=_log_int(rng, 1, 128),
                     far=rng.choice([0, _log_int(rng, 1, 1 << 20)]),
                     dims=rng.choice(["16,56,56", "44,42,42", "64,64", "32,32,32,32", "8,28,28",
                                      "32,32", "64", "128"]),
                     theta=rng.choice([256.0, 10000.0, 1000000.0]))
        elif op == "turn":
            D = rng.choice([64, 128])
            c = dict(op=op, B=_log_int(rng, 1, 16), S=_log_int(rng, 1, 9000),
                     H=rng.randint(1, 32) * (128 // D), D=D, norm=rng.random() < 0.8)
        else:
            G = rng.randint(1, 16)
            Sk = _log_int(rng, 1, 33000)
            keep = _log_int(rng, 1, 128)
            c = dict(op=op, B=rng.randint(1, 4), H=G * rng.choice([1, 1, 1, 2, 4]), G=G,
                     D=rng.choice([64, 128]),
                     Sq=rng.choice([Sk, Sk, _log_int(rng, 1, 33000)]), Sk=Sk, keep=keep,
                     first=rng.choice([0, rng.randint(0, keep)]),
                     pad=rng.choice([0, _log_int(rng, 1, Sk)]))
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def _kv_lens(c):
    return [max(c["Sk"] - b * c["pad"], 0) for b in range(c["B"])]


def _tokens(c):
    return c["text"] + c["t"] * c["h"] * c["w"]


def work(c):
    if c["op"] == "i8":
        M, K, N = c["M"], c["K"], c["N"]
        b = 2 * M * K + N * K + 4 * N + 2 * M * N + (2 * N if c["bias"] else 0)
        return {"bytes": b + (4 * K if c["smooth"] else 0), "flops": 2 * M * K * N}
    if c["op"] == "rope":
        S, dims = _tokens(c), _dims(c)
        # an angle, its sine and cosine: counted as one operation each
        return {"bytes": 4 * S * len(dims) + 4 * S * sum(dims), "flops": 3 * S * sum(dims) // 2}
    if c["op"] == "turn":
        M, HD = c["B"] * c["S"], c["H"] * c["D"]
        b = 12 * M * HD + 4 * c["S"] * c["D"] + (4 * c["D"] if c["norm"] else 0)
        return {"bytes": b, "flops": 2 * M * HD * (3 + (4 if c["norm"] else 0))}
    B, H, G, D, Sq, Sk = (c[k] for k in ("B", "H", "G", "D", "Sq", "Sk"))
    nq = -(-Sq // QUERY_BLOCK)
    keys = sum(min(c["keep"] * KEY_BLOCK, n) for n in _kv_lens(c))
    # each key and value that some query block may take is read once
    read = G * D * sum(min(n, nq * (H // G) * c["keep"] * KEY_BLOCK) for n in _kv_lens(c))
    scored = G * D * sum(_kv_lens(c))
    return {"bytes": 2 * (B * H * Sq * D * 2 + scored + read) + 4 * B * H * nq * c["keep"],
            "flops": 4 * Sq * H * D * keys}


def _dims(c):
    return [int(x) for x in c["dims"].split(",")]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    if c["op"] == "i8":
        M, K, N = c["M"], c["K"], c["N"]
        X = normal(M, K)
        # a few loud channels, as the activations of these layers have
        loud = torch.rand(K, generator=g, device="cuda") < 0.01
        X = torch.where(loud, X * 20.0, X).to(torch.bfloat16)
        c["X"] = X
        W = normal(N, K) * (K ** -0.5)
        c["lam"] = None
        if c["smooth"]:
            c["lam"] = torch.where(loud, 4.0, 1.0) * (0.5 + torch.rand(K, generator=g, device="cuda"))
            W *= c["lam"]
        # what a checkpoint holds: int8 codes and one scale per output channel
        sw = (W.abs().amax(dim=1) * (1.0 / 127.0)).clamp_min(1e-12)
        c["qw"] = torch.round(W / sw[:, None]).clamp_(-127, 127).to(torch.int8)
        c["sw"] = sw
        c["b"] = (normal(N) * 0.1).to(torch.bfloat16) if c["bias"] else None
    elif c["op"] == "rope":
        c["pos"] = _positions(c, seed)
    elif c["op"] == "turn":
        M, HD, D = c["B"] * c["S"], c["H"] * c["D"], c["D"]
        gain = 0.5 + torch.rand(3 * HD, generator=g, device="cuda")
        c["qkv"] = (normal(M, 3 * HD) * gain).to(torch.bfloat16)
        c["gq"] = (1.0 + 0.2 * normal(D)).to(torch.bfloat16) if c["norm"] else None
        c["gk"] = (1.0 + 0.2 * normal(D)).to(torch.bfloat16) if c["norm"] else None
        angle = 50.0 * normal(c["S"], D // 2)
        c["cos"], c["sin"] = torch.cos(angle), torch.sin(angle)
    else:
        B, H, G, D, Sq, Sk = (c[k] for k in ("B", "H", "G", "D", "Sq", "Sk"))
        # neighbouring tokens are alike, and queries look for keys like themselves
        theme = normal(B, G, -(-max(Sq, Sk) // 48), D)

        def like(heads, S):
            x = theme.repeat_interleave(heads // G, dim=1)
            x = x.repeat_interleave(48, dim=2)[:, :, :S] + 1.2 * normal(B, heads, S, D)
            return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

        c["q"], c["k"] = like(H, Sq), like(G, Sk)
        c["v"] = normal(B, G, Sk, D).to(torch.bfloat16)
        c["kv_len"] = torch.tensor(_kv_lens(c), dtype=torch.int32, device="cuda")
    return c


def _positions(c, seed):
    """Token positions fp32 [S, axes]: text tokens count along the first axis, patches along
    (time, height, width); the clip starts `far` + seed % 97 frames into its stream."""
    n = len(_dims(c))
    t, h, w = torch.meshgrid(torch.arange(c["t"]), torch.arange(c["h"]), torch.arange(c["w"]),
                             indexing="ij")
    t = t + c["far"] + int(seed) % 97
    axes = [t, h, w]
    grid = torch.stack([axes[a % 3].reshape(-1) for a in range(n)], dim=1)
    text = torch.zeros(c["text"], n, dtype=torch.int64)
    text[:, 0] = torch.arange(c["text"]) + int(seed) % 97
    return torch.cat([text, grid]).to(torch.float32).cuda()


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"i8": _plain_i8, "rope": _plain_rope, "turn": _plain_turn,
            "attn": _plain_attn}[state["op"]](state)


def _run_own(s):
    import bit_diffusion_transformer_amd as bdt
    if s["op"] == "i8":
        return bdt.i8_linear(s["X"], s["lam"], s["qw"], s["sw"], s["b"], s["act"])
    if s["op"] == "rope":
        return bdt.rope_tables(s["pos"], _dims(s), s["theta"])
    if s["op"] == "turn":
        return bdt.qkv_norm_rope(s["qkv"], s["H"], s["D"], s["S"], s["gq"], s["gk"], 1e-6,
                                 s["cos"], s["sin"])
    return bdt.sparse_attention(s["q"], s["k"], s["v"], s["keep"], first=s["first"],
                                kv_len=s["kv_len"], return_blocks=True)


def _plain_i8(s):
    x = s["X"].float()
    if s["lam"] is not None:
        x = x * torch.reciprocal(s["lam"])
    amax = x.abs().amax(dim=1)
    scale = amax / torch.full_like(amax, 127.0)
    inv = torch.reciprocal(scale)
    inv = torch.where(torch.isfinite(inv), inv, 0.0)
    codes = torch.round(x * inv[:, None])
    y = codes @ s["qw"].float().t()
    y = y * (scale[:, None] * s["sw"][None, :])
    if s["b"] is not None:
        y = y + s["b"].float()
    if s["act"]:
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return y.to(torch.bfloat16)


def _plain_rope(s):
    pos = s["pos"].double()              # positions past 10^6: angles in 64 bits
    angle = torch.cat([pos[:, a:a + 1] * torch.exp(
        torch.arange(d // 2, dtype=torch.float64, device=pos.device) * (-2.0 * math.log(s["theta"]) / d))
        for a, d in enumerate(_dims(s))], dim=1)
    return torch.cos(angle).float(), torch.sin(angle).float()


def _plain_turn(s):
    B, S, H, D = s["B"], s["S"], s["H"], s["D"]
    x = s["qkv"].float().view(B, S, 3, H, D).permute(2, 0, 3, 1, 4)
    q, k, v = x[0], x[1], x[2]
    cos, sin = s["cos"], s["sin"]

    def turned(x, gamma):
        if gamma is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma.float()
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)

    bf = torch.bfloat16
    return (turned(q, s["gq"]).to(bf), turned(k, s["gk"]).to(bf), v.to(bf).contiguous())


def _plain_select(q, k, kv_len, keep, first):
    """Block numbers int32 [B, H, nq, keep], ascending, -1 behind the last one taken."""
    B, H, Sq, D = q.shape
    G, Sk = k.shape[1], k.shape[2]
    nq, nk = -(-Sq // QUERY_BLOCK), -(-Sk // KEY_BLOCK)
    pad = torch.nn.functional.pad
    qm = pad(q.double(), (0, 0, 0, nq * QUERY_BLOCK - Sq)).view(B, H, nq, QUERY_BLOCK, D).sum(3)
    rows = (Sq - torch.arange(nq, device=q.device) * QUERY_BLOCK).clamp(max=QUERY_BLOCK)
    qm = qm / rows[:, None]
    seen = torch.arange(Sk, device=q.device)[None, :] < kv_len[:, None]          # [B, Sk]
    km = torch.where(seen[:, None, :, None], k.double(), 0.0)
    km = pad(km, (0, 0, 0, nk * KEY_BLOCK - Sk)).view(B, G, nk, KEY_BLOCK, D).sum(3)
    keys = (kv_len[:, None] - torch.arange(nk, device=q.device) * KEY_BLOCK).clamp(0, KEY_BLOCK)
    km = km / keys.clamp(min=1)[:, None, :, None]
    km = km.repeat_interleave(H // G, dim=1)
    score = qm @ km.transpose(2, 3).contiguous()
    at = torch.arange(nk, device=q.device)
    score = torch.where(at < first, math.inf, score)
    score = torch.where((keys == 0)[:, None, None, :], -math.inf, score)
    order = torch.argsort(score, dim=-1, descending=True, stable=True)[..., :keep]
    taken = torch.gather(score, -1, order) > -math.inf
    order = torch.sort(torch.where(taken, order, nk), dim=-1).values
    blocks = torch.where(order < nk, order, -1)
    return pad(blocks, (0, keep - blocks.shape[-1]), value=-1).to(torch.int32)


def _plain_attn(s):
    q, k, v, kv_len = s["q"], s["k"], s["v"], s["kv_len"]
    B, H, Sq, D = q.shape
    G, Sk = k.shape[1], k.shape[2]
    nq, nk, keep = -(-Sq // QUERY_BLOCK), -(-Sk // KEY_BLOCK), s["keep"]
    blocks = _plain_select(q, k, kv_len, keep, s["first"])
    used = min(keep, nk)
    idx = blocks[..., :used].long()
    pad = torch.nn.functional.pad
    b = torch.arange(B, device=q.device)[:, None, None, None]
    h = (torch.arange(H, device=q.device) // (H // G))[None, :, None, None]
    at = idx.clamp(min=0)
    tail = (0, 0, 0, nk * KEY_BLOCK - Sk)
    kk = pad(k, tail).view(B, G, nk, KEY_BLOCK, D)[b, h, at].float()
    vv = pad(v, tail).view(B, G, nk, KEY_BLOCK, D)[b, h, at].float()
    key = at[..., None] * KEY_BLOCK + torch.arange(KEY_BLOCK, device=q.device)
    seen = ((idx >= 0)[..., None] & (key < kv_len[:, None, None, None, None])).flatten(3)
    kk, vv = kk.flatten(3, 4), vv.flatten(3, 4)
    vv = torch.where(seen[..., None], vv, 0.0)
    qq = pad(q.float(), (0, 0, 0, nq * QUERY_BLOCK - Sq)).view(B, H, nq, QUERY_BLOCK, D)
    score = (qq @ kk.transpose(3, 4).contiguous()) * (D ** -0.5)
    score = score.masked_fill(~seen[:, :, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = (p @ vv) / torch.where(total > 0, total, 1.0)
    out = out.view(B, H, nq * QUERY_BLOCK, D)[:, :, :Sq].permute(0, 2, 1, 3)
    return out.to(torch.bfloat16).contiguous(), blocks


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"i8": _exact_i8, "rope": _exact_rope, "turn": _exact_turn,
            "attn": _exact_attn}[s["op"]](s)


def _exact_i8(s):
    # The codes are part of the definition: scale, reciprocal and product are single fp32
    # operations, then the nearest integer.  Everything after them is exact or in 64 bits.
    x = s["X"].float()
    if s["lam"] is not None:
        x = x * (torch.ones_like(s["lam"]) / s["lam"])
    scale = x.abs().max(dim=1).values
    scale = scale / torch.full_like(scale, 127.0)
    inv = torch.ones_like(scale) / scale
    inv[~torch.isfinite(inv)] = 0.0
    codes = (x * inv.unsqueeze(1)).round().double()
    total = torch.matmul(codes, s["qw"].double().t())
    total *= scale.double().unsqueeze(1)
    total *= s["sw"].double()
    if s["b"] is not None:
        total += s["b"].double()
    if s["act"]:
        total = total * torch.special.erfc(-total / math.sqrt(2.0)) / 2.0
    return total


def _exact_rope(s):
    cols = []
    for a, d in enumerate(_dims(s)):
        for p in range(d // 2):
            cols.append(s["pos"][:, a].double() * s["theta"] ** (-2.0 * p / d))
    angle = torch.stack(cols, dim=1)
    return angle.cos(), angle.sin()


def _exact_turn(s):
    B, S, H, D = s["B"], s["S"], s["H"], s["D"]
    x = s["qkv"].double().view(B, S, 3, H, D)
    unit = torch.complex(s["cos"].double(), s["sin"].double())[None, :, None, :]
    out = []
    for sec, gamma in ((0, s["gq"]), (1, s["gk"])):
        y = x[:, :, sec]
        if gamma is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * gamma.double()
        z = torch.view_as_complex(y.reshape(B, S, H, D // 2, 2).contiguous()) * unit
        out.append(torch.view_as_real(z).reshape(B, S, H, D).transpose(1, 2).contiguous())
    return out[0], out[1], x[:, :, 2].transpose(1, 2).contiguous()


def _exact_attn(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, H, Sq, D = q.shape
    G, Sk = k.shape[1], k.shape[2]
    nq, keep = -(-Sq // QUERY_BLOCK), s["keep"]
    out = torch.zeros(B, Sq, H, D, dtype=torch.float64, device=q.device)
    blocks = torch.full((B, H, nq, keep), -1, dtype=torch.int32, device=q.device)
    for b, n in enumerate(_kv_lens(s)):
        if n == 0:
            continue
        nk = -(-n // KEY_BLOCK)
        for h in range(H):
            kd, vd = k[b, h // (H // G), :n].double(), v[b, h // (H // G), :n].double()
            km = torch.stack([kd[j * KEY_BLOCK:(j + 1) * KEY_BLOCK].mean(0) for j in range(nk)])
            for i0 in range(0, nq, 64):
                rows = q[b, h, i0 * QUERY_BLOCK:(i0 + 64) * QUERY_BLOCK].double()
                some = range(-(-rows.shape[0] // QUERY_BLOCK))
                qm = torch.stack([rows[i * QUERY_BLOCK:(i + 1) * QUERY_BLOCK].mean(0) for i in some])
                score = torch.mm(qm, km.t().contiguous())
                score[:, :s["first"]] = math.inf
                take = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :keep]
                mask = torch.zeros_like(score, dtype=torch.bool).scatter_(1, take, True)
                blocks[b, h, i0:i0 + len(some), :take.shape[1]] = \
                    take.sort(dim=1).values.to(torch.int32)
                mask = mask.repeat_interleave(KEY_BLOCK, 1)[:, :n]
                mask = mask.repeat_interleave(QUERY_BLOCK, 0)[:rows.shape[0]]
                logit = torch.mm(rows, kd.t().contiguous()) / math.sqrt(D)
                p = torch.softmax(logit.masked_fill_(~mask, -math.inf), dim=1)
                out[b, i0 * QUERY_BLOCK:i0 * QUERY_BLOCK + rows.shape[0], h] = torch.mm(p, vd)
    return out, blocks
