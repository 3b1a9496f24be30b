"""Attention over packed sequences and over a paged key/value cache, with what fills and plans
the cache: the text encoder (a decoder with grouped heads, prompts of different lengths) and
streaming generation (new frames or tokens over a kept cache) beside the quantized linears.

``listed()`` gives the measured cases, ``draw(rng)`` more of the same ranges, ``prepare`` the
inputs on the GPU, ``run`` one pass (``own`` false: elementary torch operations in 32 bits;
true: the library's calls), ``work`` the bytes and operations a pass cannot do without, and
``exact`` the outputs from the definitions in 64 bits.

Operators
  packed  attention of sequences packed one after another, q [T, H, D], k and v [T, G, D]:
          head h reads key head h / (H / G); causal or not.
  paged   attention of each request's new tokens over its cache pages [pages, G, page, D]
          (the new tokens' keys are in the cache already); causal or not.
  tables  from the lengths of the requests and a list of free pages: the pages of the new
          tokens, token starts, key counts, and every token's slot and position.
  cache   a projection [T, (H + 2 G) D] -> per-head RMS norm and rotary turn of Q and K
          (pairs interleaved or in halves, of the whole head or its first part), Q to
          [T, H, D], K and V to their slots of the cache.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases

def _text(numbers):
    return ",".join(str(int(n)) for n in numbers)


def _numbers(text):
    return [int(n) for n in text.split(",")] if text else []


def _spread(n, lo, hi, step):
    """n whole numbers from lo to hi, even over their logarithm, in a mixed order."""
    at = [(i * step) % n for i in range(n)]
    return [int(round(lo * (hi / lo) ** (i / max(n - 1, 1)))) for i in at]


def listed():
    return [
        # --- packed: one caption through a small text encoder (latency); a batch of prompts of
        # very different lengths; one long document; images of four resolutions side by side
        # (every token sees its whole image).
        dict(name="prompt_short", op="packed", H=12, G=12, D=64, causal=True, lens="77"),
        dict(name="prompt_batch", op="packed", H=32, G=8, D=128, causal=True,
             lens="129,1,17,2000,64,333,777,1024,512,0,63,1431"),
        dict(name="prompt_long", op="packed", H=32, G=8, D=128, causal=True, lens="16384"),
        dict(name="images_packed", op="packed", H=24, G=24, D=128, causal=False,
             lens="4096,1024,2304,777"),
        # --- paged: one token of one long request (its cache is read once); one token of each
        # of 64 requests of 9 to 8192 tokens; two streams that each add a frame of 30 x 52
        # patches to 20 frames; decoding requests beside a prompt that is taken in chunks.
        dict(name="decode_one", op="paged", H=32, G=8, D=128, page=64, causal=True,
             new="1", lens="65537"),
        dict(name="decode_batch", op="paged", H=32, G=8, D=128, page=16, causal=True,
             new=_text([1] * 64), lens=_text(_spread(64, 9, 8192, 27))),
        dict(name="stream_frames", op="paged", H=12, G=12, D=128, page=128, causal=False,
             new="1560,1560", lens="32760,29640"),
        dict(name="chunk_beside_decode", op="paged", H=28, G=4, D=64, page=32, causal=True,
             new=_text([1] * 20 + [512] + [1] * 11),
             lens=_text(_spread(20, 100, 6000, 7) + [4608] + _spread(11, 40, 3000, 4))),
        # --- tables: a step of 64 decoding requests; 512 requests that start or go on with
        # prompts of many lengths.
        dict(name="tables_decode", op="tables", page=16, width=512,
             cached=_text(_spread(64, 9, 8000, 27)), new=_text([1] * 64)),
        dict(name="tables_prompts", op="tables", page=64, width=128,
             cached=_text([0 if i % 3 else 37 * i % 4001 for i in range(512)]),
             new=_text([1 + (i * i * 7 + 13 * i) % 260 for i in range(512)])),
        # --- cache: 64 decoding tokens (pairs in halves); a prompt of 8000 tokens whose heads
        # turn a quarter only (neighbouring pairs).
        dict(name="cache_decode", op="cache", T=64, H=32, G=8, D=128, R=128, page=16, half=True,
             norm=True, far=8000),
        dict(name="cache_prompt", op="cache", T=8000, H=32, G=4, D=128, R=32, page=64, half=False,
             norm=True, far=30000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _heads(rng):
    G = rng.choice([1, 2, 3, 4, 5, 8, 10, 12, 16, 24])
    return G * rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8]), G


def draw(rng):
    op = rng.choice(["packed", "packed", "paged", "paged", "paged", "tables", "cache"])
    most = {"bytes": 0, "flops": 0}
    for c in listed():
        if c["op"] == op:
            w = work(c)
            most = {k: max(most[k], w[k]) for k in most}
    while True:
        c = dict(op=op)
        if op in ("packed", "paged"):
            c["H"], c["G"] = _heads(rng)
            c["D"] = rng.choice([64, 128, 128])
        if op == "packed":
            c["causal"] = rng.random() < 0.75
            n = _log_int(rng, 1, 48)
            top = _log_int(rng, 1, 16384)
            c["lens"] = _text(0 if rng.random() < 0.03 else _log_int(rng, 1, top) for _ in range(n))
            if sum(_numbers(c["lens"])) == 0:
                continue
        elif op == "paged":
            c["causal"] = rng.random() < 0.8
            c["page"] = rng.choice([16, 32, 64, 128, 256])
            n = _log_int(rng, 1, 128)
            kind = rng.choice(["one", "one", "few", "chunk", "mixed"])
            longest = _log_int(rng, 2, 2048)
            new = []
            for _ in range(n):
                new.append(1 if kind == "one" or (kind == "mixed" and rng.random() < 0.8)
                           else rng.randint(1, 8) if kind == "few" else _log_int(rng, 1, longest))
            top = _log_int(rng, 1, 65536)
            c["new"] = _text(new)
            c["lens"] = _text(q + _log_int(rng, 1, top) - 1 for q in new)
        elif op == "tables":
            c["page"] = rng.choice([16, 32, 64, 128, 256])
            n = _log_int(rng, 1, 512)
            top, more = _log_int(rng, 1, 20000), rng.choice([1, 1, _log_int(rng, 2, 600)])
            cached = [rng.choice([0, _log_int(rng, 1, top)]) for _ in range(n)]
            new = [rng.randint(0 if more > 1 else 1, more) for _ in range(n)]
            c["cached"], c["new"] = _text(cached), _text(new)
            c["width"] = max(-(-(a + b) // c["page"]) for a, b in zip(cached, new)) + rng.randint(0, 9)
            if sum(new) == 0 or c["width"] == 0:
                continue
        else:
            c["T"] = _log_int(rng, 1, 8000)
            c["H"], c["G"] = _heads(rng)
            c["D"] = rng.choice([64, 128])
            c["R"] = rng.choice([c["D"], c["D"], c["D"] // 2, c["D"] // 4, 16, 48])
            c["page"] = rng.choice([16, 32, 64, 128, 256])
            c["half"], c["norm"] = rng.random() < 0.6, rng.random() < 0.7
            c["far"] = rng.choice([0, _log_int(rng, 1, 60000)])
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _pairs(new, lens, causal):
    """Number of (query, key) pairs that see each other, all heads alike."""
    return sum(q * n - (q * (q - 1) // 2 if causal else 0) for q, n in zip(new, lens))


def work(c):
    if c["op"] == "packed":
        lens = _numbers(c["lens"])
        T = sum(lens)
        return {"bytes": 4 * T * (c["H"] + c["G"]) * c["D"],
                "flops": 4 * c["H"] * c["D"] * _pairs(lens, lens, c["causal"])}
    if c["op"] == "paged":
        new, lens = _numbers(c["new"]), _numbers(c["lens"])
        pages = sum(-(-n // c["page"]) for n in lens)
        return {"bytes": 4 * c["D"] * (sum(new) * c["H"] + sum(lens) * c["G"]) + 4 * pages,
                "flops": 4 * c["H"] * c["D"] * _pairs(new, lens, c["causal"])}
    if c["op"] == "tables":
        cached, new = _numbers(c["cached"]), _numbers(c["new"])
        B, T = len(new), sum(new)
        taken = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in zip(cached, new))
        # lengths in, starts and key counts out; pages read and put in the tables; a slot and
        # a position each token; a few whole-number operations a token and a page
        return {"bytes": 16 * B + 8 * taken + 8 * T, "flops": 4 * (T + taken + B)}
    T, H, G, D, R = (c[k] for k in ("T", "H", "G", "D", "R"))
    b = 4 * T * (H + 2 * G) * D + 4 * T * R + 8 * T + (4 * D if c["norm"] else 0)
    return {"bytes": b, "flops": T * (H + G) * (3 * R + (4 * D if c["norm"] else 0))}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    def bf16(*shape):
        return normal(*shape).to(torch.bfloat16)

    def ints(numbers):
        return torch.tensor(numbers, dtype=torch.int32, device="cuda")

    def starts(lens):
        out = [0]
        for n in lens:
            out.append(out[-1] + n)
        return out

    if c["op"] == "packed":
        lens = c["n"] = _numbers(c["lens"])
        T, H, G, D = sum(lens), c["H"], c["G"], c["D"]
        # the three parts of one projection, as a text encoder's layer has them
        qkv = (1.4 * normal(T, (H + 2 * G) * D)).to(torch.bfloat16)
        c["q"] = qkv[:, :H * D].view(T, H, D)
        c["k"] = qkv[:, H * D:(H + G) * D].view(T, G, D)
        c["v"] = qkv[:, (H + G) * D:].view(T, G, D)
        c["starts"] = ints(starts(lens))
    elif c["op"] == "paged":
        new, lens = c["m"], c["n"] = _numbers(c["new"]), _numbers(c["lens"])
        H, G, D, page = c["H"], c["G"], c["D"], c["page"]
        each = [-(-n // page) for n in lens]
        pages, width = sum(each) + 3, max(each) + 1
        c["k_cache"], c["v_cache"] = bf16(pages, G, page, D), bf16(pages, G, page, D)
        c["q"] = (1.4 * normal(sum(new), H, D)).to(torch.bfloat16)
        # pages in the order in which requests of different ages were given them: any
        order = torch.randperm(pages, generator=g, device="cuda").cpu().tolist()
        tables = torch.full((len(new), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(each):
            tables[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        c["tables"] = tables.cuda()
        c["starts"], c["kv_len"] = ints(starts(new)), ints(lens)
        c["most"] = max(new)
    elif c["op"] == "tables":
        cached, new = c["a"], c["m"] = _numbers(c["cached"]), _numbers(c["new"])
        page, width = c["page"], c["width"]
        held = [-(-a // page) for a in cached]
        taken = [-(-(a + b) // page) - h for a, b, h in zip(cached, new, held)]
        c["pages"] = sum(held) + sum(taken) + 5
        order = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)
        tables = torch.full((len(new), width), -1, dtype=torch.int32)
        at, given = 0, order.cpu()
        for b, n in enumerate(held):
            tables[b, :n] = given[at:at + n]
            at += n
        c["tables"], c["free"] = tables.cuda(), order[at:].contiguous()
        c["cached_len"], c["new_len"], c["T"] = ints(cached), ints(new), sum(new)
    else:
        T, H, G, D, R, page = (c[k] for k in ("T", "H", "G", "D", "R", "page"))
        gain = 0.5 + torch.rand((H + 2 * G) * D, generator=g, device="cuda")
        c["qkv"] = (normal(T, (H + 2 * G) * D) * gain).to(torch.bfloat16)
        c["gq"] = (1.0 + 0.2 * normal(D)).to(torch.bfloat16) if c["norm"] else None
        c["gk"] = (1.0 + 0.2 * normal(D)).to(torch.bfloat16) if c["norm"] else None
        P = T + c["far"]
        angle = torch.outer(torch.arange(P, device="cuda", dtype=torch.float64), torch.exp(
            torch.arange(R // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(1e6) / R)))
        c["cos"], c["sin"] = angle.cos().float(), angle.sin().float()
        c["pos"] = torch.randperm(P, generator=g, device="cuda")[:T].to(torch.int32)
        pages = -(-T // page) + 2
        c["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
        if T >= 256:                     # a prompt: its tokens fill page after page
            c["slots"] = torch.randperm(pages, generator=g, device="cuda")[
                torch.arange(T, device="cuda") // page] * page
            c["slots"] = (c["slots"] + torch.arange(T, device="cuda") % page).to(torch.int32)
            c["pos"] = (torch.arange(T, device="cuda") + int(seed) % (c["far"] + 1)).to(torch.int32)
        c["k_cache"], c["v_cache"] = bf16(pages, G, page, D), bf16(pages, G, page, D)
    return c


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"packed": _plain_packed, "paged": _plain_paged, "tables": _plain_tables,
            "cache": _plain_cache}[state["op"]](state)


def _run_own(s):
    import bit_diffusion_transformer_amd as bdt
    if s["op"] == "packed":
        return bdt.packed_attention(s["q"], s["k"], s["v"], s["starts"], causal=s["causal"])
    if s["op"] == "paged":
        return bdt.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["starts"],
                                   s["kv_len"], max_new=s["most"], causal=s["causal"])
    if s["op"] == "tables":
        return (s["tables"],) + tuple(bdt.page_tables(s["cached_len"], s["new_len"], s["free"],
                                                      s["tables"], s["page"], s["pages"], s["T"]))
    q = bdt.qkv_norm_rope_cache(s["qkv"], s["H"], s["G"], s["gq"], s["gk"], EPS, s["cos"], s["sin"],
                                s["pos"], s["slots"], s["k_cache"], s["v_cache"], half=s["half"])
    return q, s["k_cache"], s["v_cache"]


def _rows(q, k, v, sees, scale):
    """q fp32 [G, n, D], k and v fp32 [G, m, D], sees [n, m] (None: all) -> [G, n, D]."""
    score = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(scale)
    if sees is not None:
        score.masked_fill_(~sees, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.bmm(p, v) / torch.where(total > 0, total, 1.0)


def _one(q, k, v, causal, scale):
    """Attention of one sequence: q [n, H, D] over k, v [G, m, D] -> fp32 [n, H, D]."""
    n, H, D = q.shape
    G, m = k.shape[:2]
    kf, vf = k.float(), v.float()
    out = torch.empty(n, H, D, dtype=torch.float32, device=q.device)
    step = max(1, (1 << 28) // max(H * m, 1))       # scores of 1 GB at a time
    for i in range(0, n, step):
        j = min(i + step, n)
        seen = m - n + j if causal else m
        rows = q[i:j].float().view(j - i, G, H // G, D).permute(1, 0, 2, 3).reshape(G, -1, D)
        sees = None
        if causal:
            at = torch.arange(i, j, device=q.device).repeat_interleave(H // G) + (m - n)
            sees = torch.arange(seen, device=q.device)[None, :] <= at[:, None]
        o = _rows(rows, kf[:, :seen], vf[:, :seen], sees, scale)
        out[i:j] = o.view(G, j - i, H // G, D).permute(1, 0, 2, 3).reshape(j - i, H, D)
    return out


def _plain_packed(s):
    at, out = 0, torch.empty(s["q"].shape, dtype=torch.bfloat16, device=s["q"].device)
    for n in s["n"]:
        part = slice(at, at + n)
        if n:
            out[part] = _one(s["q"][part], s["k"][part].transpose(0, 1), s["v"][part].transpose(0, 1),
                             s["causal"], s["D"] ** -0.5)
        at += n
    return out


def _plain_paged(s):
    q, D, page = s["q"], s["D"], s["page"]
    H, G, scale = s["H"], s["G"], s["D"] ** -0.5
    if s["most"] == 1 and len(s["n"]) > 1 and min(s["m"]) == 1:
        # a token each: requests side by side, padded to the longest of some
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        step = max(1, (1 << 28) // (G * D * max(s["n"])))
        for i in range(0, len(s["n"]), step):
            j = min(i + step, len(s["n"]))
            width = -(-max(s["n"][i:j]) // page)
            at = s["tables"][i:j, :width].clamp(min=0)
            k = s["k_cache"][at].float().permute(0, 2, 1, 3, 4).reshape((j - i) * G, -1, D)
            v = s["v_cache"][at].float().permute(0, 2, 1, 3, 4).reshape((j - i) * G, -1, D)
            sees = torch.arange(width * page, device=q.device) < s["kv_len"][i:j, None]
            sees = sees.repeat_interleave(G, 0)[:, None, :]
            rows = q[i:j].float().view((j - i) * G, H // G, D)
            out[i:j] = _rows(rows, k, v, sees, scale).view(j - i, H, D)
        return out
    at, out = 0, torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    for b, (m, n) in enumerate(zip(s["m"], s["n"])):
        pages = s["tables"][b, :-(-n // page)]
        k = s["k_cache"][pages].transpose(0, 1).reshape(G, -1, D)[:, :n]
        v = s["v_cache"][pages].transpose(0, 1).reshape(G, -1, D)[:, :n]
        out[at:at + m] = _one(q[at:at + m], k, v, s["causal"], scale)
        at += m
    return out


def _plain_tables(s):
    cached, new, tables, page, T = s["cached_len"], s["new_len"], s["tables"], s["page"], s["T"]
    dev, B = cached.device, cached.shape[0]
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    starts = torch.cat([zero, torch.cumsum(new, 0)])
    held = (cached + (page - 1)) // page
    taken = (cached + new + (page - 1)) // page - held
    first = torch.cat([zero, torch.cumsum(taken, 0)])
    column = torch.arange(tables.shape[1], device=dev)[None, :]
    mine = (column >= held[:, None]) & (column < (held + taken)[:, None])
    at = (first[:B, None] + column - held[:, None]).clamp(0, max(s["free"].shape[0] - 1, 0))
    tables.copy_(torch.where(mine, s["free"][at], tables))
    request = torch.repeat_interleave(torch.arange(B, device=dev), new, output_size=T)
    position = cached[request] + torch.arange(T, device=dev) - starts[request]
    slot = tables[request, position // page] * page + position % page
    count = torch.stack([first[B], zero[0]])
    i32 = torch.int32
    return (tables, starts.to(i32), (cached + new).to(i32), slot.to(i32), position.to(i32),
            count.to(i32))


def _plain_cache(s):
    T, H, G, D, R, page = (s[k] for k in ("T", "H", "G", "D", "R", "page"))
    x = s["qkv"].float()
    pos = s["pos"].long()
    cos, sin = s["cos"][pos][:, None, :], s["sin"][pos][:, None, :]

    def turned(x, gamma):
        if gamma is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()
        y, rest = x[..., :R], x[..., R:]
        if s["half"]:
            a, b = y[..., :R // 2], y[..., R // 2:]
            return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], dim=-1)
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        return torch.cat([y, rest], dim=-1)

    bf = torch.bfloat16
    q = turned(x[:, :H * D].view(T, H, D), s["gq"]).to(bf)
    k = turned(x[:, H * D:(H + G) * D].view(T, G, D), s["gk"]).to(bf)
    v = s["qkv"][:, (H + G) * D:].view(T, G, D)
    slot = s["slots"].long()
    s["k_cache"][slot // page, :, slot % page] = k
    s["v_cache"][slot // page, :, slot % page] = v
    return q, s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"packed": _exact_packed, "paged": _exact_paged, "tables": _exact_tables,
            "cache": _exact_cache}[s["op"]](s)


def _exact_heads(q, k, v, causal):
    """One sequence, head by head: q [n, H, D], k and v [m, G, D] -> fp64 [n, H, D]."""
    n, H, D = q.shape
    m, G = k.shape[:2]
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    key = torch.arange(m, device=q.device)
    for h in range(H):
        kd, vd = k[:, h * G // H].double(), v[:, h * G // H].double()
        for i in range(0, n, 4096):
            logit = torch.mm(q[i:i + 4096, h].double(), kd.t().contiguous()) / math.sqrt(D)
            if causal:
                last = torch.arange(i, min(i + 4096, n), device=q.device) + m - n
                logit[key[None, :] > last[:, None]] = -math.inf
            out[i:i + 4096, h] = torch.mm(torch.softmax(logit, dim=1), vd)
    return out


def _exact_packed(s):
    edges = s["starts"].tolist()
    return torch.cat([_exact_heads(s["q"][a:b], s["k"][a:b], s["v"][a:b], s["causal"])
                      for a, b in zip(edges[:-1], edges[1:])])


def _exact_paged(s):
    edges, page, out = s["starts"].tolist(), s["page"], []
    for b, n in enumerate(s["kv_len"].tolist()):
        key = torch.arange(n, device=s["q"].device)
        at = s["tables"][b].long()[key // page]
        k, v = s["k_cache"][at, :, key % page], s["v_cache"][at, :, key % page]
        out.append(_exact_heads(s["q"][edges[b]:edges[b + 1]], k, v, s["causal"]))
    return torch.cat(out)


def _exact_tables(s):
    free, rows = iter(s["free"].tolist()), s["tables"].tolist()
    page, starts, lens, slots, positions, taken = s["page"], [0], [], [], [], 0
    for row, a, m in zip(rows, s["a"], s["m"]):
        for p in range(a, a + m):
            if p % page == 0:
                row[p // page] = next(free)
                taken += 1
            slots.append(row[p // page] * page + p % page)
            positions.append(p)
        starts.append(starts[-1] + m)
        lens.append(a + m)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    return tuple(ints(x) for x in (rows, starts, lens, slots, positions, [taken, 0]))


def _exact_cache(s):
    T, H, G, D, R, page = (s[k] for k in ("T", "H", "G", "D", "R", "page"))
    unit = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()].unsqueeze(1)
    q, k, v = s["qkv"].double().split([H * D, G * D, G * D], dim=1)

    def turned(x, gamma):
        x = x.reshape(T, -1, D)
        if gamma is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * gamma.double()
        x = x.clone()
        if s["half"]:
            z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * unit
            x[..., :R // 2], x[..., R // 2:R] = z.real, z.imag
        else:
            z = torch.view_as_complex(x[..., :R].reshape(T, -1, R // 2, 2).contiguous()) * unit
            x[..., :R] = torch.view_as_real(z).reshape(T, -1, R)
        return x

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k, v = turned(k, s["gk"]), v.reshape(T, G, D)
    page_of, at = torch.div(s["slots"].long(), page, rounding_mode="floor"), s["slots"].long() % page
    k_cache[page_of, :, at] = k
    v_cache[page_of, :, at] = v
    return turned(q, s["gq"]), k_cache, v_cache
