"""Inputs and checks of attention over many keys, made so that one block, page or key that is lost,
counted twice or seen in spite of a mask passes the bound by far (a bound from sum p |v| alone
grows to the size of the output, which shrinks like the root of the number of keys).

All run on any device.  q [n, H, D], k, v [m, G, D] of one sequence, bf16; sees [n, m]."""
import math

import torch

BF = torch.bfloat16
LN2 = float(torch.tensor(math.log(2.0), dtype=torch.float32))
THIRD = float(torch.tensor(math.log(2.0) / 3, dtype=torch.float32))


def visible(n, m, causal, dead=None, device="cpu"):
    row, key = torch.arange(n, device=device), torch.arange(m, device=device)
    sees = key[None, :] <= row[:, None] + (m - n) if causal else torch.ones(n, m, dtype=torch.bool, device=device)
    return sees if dead is None else sees & ~dead[None, :]


def exact(q, k, v, scale, sees):
    """(sum p v, sum p |v|) in 64 bits [n, H, D]; a row that sees no key gives zeros."""
    H, G = q.shape[1], k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(out)
    some = sees.any(1, keepdim=True)
    used = sees.any(0)[:, None]
    for h in range(H):
        kd = torch.where(used, k[:, h // (H // G)].double(), 0.0)
        vd = torch.where(used, v[:, h // (H // G)].double(), 0.0)
        s = scale * (q[:, h].double() @ kd.t().contiguous())
        s = s.masked_fill(~sees, -math.inf)
        p = torch.softmax(torch.where(some, s, 0.0), dim=1)
        p = torch.where(some & sees, p, 0.0)
        out[:, h], size[:, h] = p @ vd, p @ vd.abs()
    return out, size


def normal(seed, *shape, device="cpu"):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.randn(shape, generator=g, device=device).to(BF)


# ------------------------------------------------------------------ random values

def check_rms(out, ref, what=""):
    """Normal values over many keys.  Each weight's rounding to bf16 is off by at most 2^-8 of it, in
    the root of the mean square by 2^-8 / sqrt 3, independently for each key, so sum p v by as much
    of its own size (values without a mean: both add like roots of squares); the result's
    rounding again: 2^-8 sqrt(2 / 3) = 0.0032 together.  0.004 leaves a quarter for the spread of a
    mean over a hundred values and more and for sums in fp32 (2^-24 sqrt m).  One lost key of m is
    off by 1 / sqrt m: 0.007 at 20000 keys, a lost block of 64 by 0.057."""
    err = float((out.double() - ref).square().mean().sqrt() / ref.square().mean().sqrt())
    assert err <= 0.004, "%s: off by %.5f in the root of the mean square" % (what, err)


# ------------------------------------------------------------------ counted keys

def counted(n, m, H, G, D, device="cpu"):
    """Queries of zero, so that every key that a row sees weighs the same; v counts units of 16 keys,
    unit u in column u % D: out[:, d] = keys of column d / keys, sums of ones, exact in fp32."""
    q = torch.zeros(n, H, D, dtype=BF, device=device)
    k = normal(1, m, G, D, device=device)
    unit = torch.arange(m, device=device) // 16 % D
    v = torch.nn.functional.one_hot(unit, D).to(BF)[:, None, :].expand(m, G, D).contiguous()
    return q, k, v


def check_counted(out, v, sees, what=""):
    """One rounding of the quotient to bf16 (2^-8), one of the reciprocal and one of the product in
    fp32 (2^-22 is more).  A unit lost of the U of its column is off by 1 / U: at 65537 keys and
    D = 128 1 / 33."""
    n = sees.sum(1, keepdim=True).double()
    ref = torch.where(n > 0, (sees.double() @ v[:, 0].double()) / n.clamp(min=1), 0.0)[:, None, :]
    err = (out.double() - ref).abs() - ref * (2.0 ** -8 + 2.0 ** -22)
    assert bool((err <= 0).all()), "%s: a count is off by %.3g of its column" % (
        what, float(((out.double() - ref).abs() / ref.clamp(min=1e-30)).max()))


# ------------------------------------------------------------------ weights of powers of two

def check_powers(out, ref, size, what=""):
    """Scores whose weights are whole powers of two times 1 +- 2^-14 (the offset's rounding where it
    is at most 2^10, common to a row; otherwise less; c = scale log2 e is off by 2^-23 of the few
    tens of steps that count), so their rounding to bf16 puts them right: 2^-13 of sum p |v| is
    what the weights of several parts and the sums in fp32 leave, and one rounding of the result to
    bf16, 2^-8 of it.  With v in 1 .. 2 that is 0.4 % of the output."""
    err = (out.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -13 * size
    assert bool((err <= tol).all()), "%s: worst %.3g of the bound" % (what, float((err / (tol + 1e-30)).max()))


def positive(seed, *shape, device="cpu"):
    """Values in 1 .. 2."""
    g = torch.Generator(device=device).manual_seed(seed)
    return (1 + torch.rand(shape, generator=g, device=device)).to(BF)


def peaked(n, m, H, G, D, peaks, device="cpu"):
    """Key head g: the score of key i is -|i - peaks[g]| times log 2 (scale LN2), so the weights
    halve with every key away from the peak."""
    q = torch.zeros(n, H, D, dtype=BF, device=device)
    q[..., 0], q[..., 1] = -256.0, -1.0
    k = torch.zeros(m, G, D, dtype=BF, device=device)
    at = torch.arange(m, device=device)
    for g in range(G):
        away = (at - peaks[g]).abs()
        k[:, g, 0], k[:, g, 1] = (away // 256).to(BF), (away % 256).to(BF)
    return q, k, positive(5, m, G, D, device=device)


def far(n, m, H, G, D, seed, device="cpu"):
    """Scores of 3 a 2^22 + j, a = 1, -1 or 0 from row to row and j = 0 .. -120 from key to key, exact in
    fp32, scale log 2 / 3 (THIRD): exponents in the millions in steps of a third.  In each block of
    64 keys the largest j is another one (0 .. -4), so that partial results have other maxima, and v
    is 1 or 2 for a whole block and column, so that a wrong weight of a part shows."""
    g = torch.Generator().manual_seed(seed)
    q = torch.zeros(n, H, D, dtype=BF, device=device)
    a = torch.tensor([1.0, -1.0, 0.0])[torch.randint(0, 3, (n, H), generator=g)]
    q[..., 0], q[..., 1] = (192 * a).to(device).to(BF), 1.0
    k = torch.zeros(m, G, D, dtype=BF, device=device)
    blocks = -(-m // 64)
    j = torch.randint(-120, 1, (m, G), generator=g)
    least = torch.randint(0, 5, (blocks, G), generator=g).repeat_interleave(64, 0)[:m]
    k[..., 0], k[..., 1] = 65536.0, (j - least).clamp(min=-120).to(device).to(BF)
    v = torch.randint(1, 3, (blocks, G, D), generator=g).repeat_interleave(64, 0)[:m].to(device).to(BF)
    return q, k, v


def check_thirds(out, ref, size, what=""):
    """Weights of 2^(i / 3): each rounded to bf16 (2^-8 of sum p |v|), otherwise as check_powers.  An
    offset of 2^22 rounded to fp32 is off by up to a quarter: by 19 % of a part."""
    err = (out.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -13) * size
    assert bool((err <= tol).all()), "%s: worst %.3g of the bound" % (what, float((err / (tol + 1e-30)).max()))


# ------------------------------------------------------------------ pages

def in_pages(ks, vs, page, seed, spare=3):
    """(k_cache, v_cache, tables on the host): the sequences' keys in pages in a mixed order; what no
    key fills is NaN or infinite."""
    device, (_, G, D) = ks[0].device, ks[0].shape
    each = [-(-k.shape[0] // page) for k in ks]
    pages, width = sum(each) + spare, max(each + [0]) + 1
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    tables = torch.full((len(ks), width), -1, dtype=torch.int32)
    kc = torch.full((pages, G, page, D), float("nan"), dtype=BF, device=device)
    vc = torch.full((pages, G, page, D), float("inf"), dtype=BF, device=device)
    at = 0
    for b, (k, v) in enumerate(zip(ks, vs)):
        mine = order[at:at + each[b]]
        tables[b, :each[b]] = mine.to(torch.int32)
        at += each[b]
        i = torch.arange(k.shape[0])
        p, r = mine[i // page].to(device), (i % page).to(device)
        kc[p, :, r], vc[p, :, r] = k, v
    return kc, vc, tables
