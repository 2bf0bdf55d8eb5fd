"""Caches in 8 bits: plain 64-bit forms and inputs that their tests share."""
import math

import torch

from state_cached_causal_gb300 import synth

DEV = torch.device("cuda")
F8 = torch.float8_e4m3fn


def scale_byte(m):
    """The byte of the least power of two 2^e with m <= 448 * 2^e, e >= -126."""
    if m == 0:
        return 1
    f, x = math.frexp(m)                       # m = f 2^x, 1/2 <= f < 1; 448 = 0.875 * 2^9
    return max(x - 9 + (f > 0.875), -126) + 127


def values(cache, scale):
    """What bytes and scales stand for, in 64 bits."""
    return cache.double() * torch.exp2(scale.view(torch.uint8).double() - 127)[..., None]


def quantised(x):
    """Rows of x (CPU, double) as (e4m3, scale bytes)."""
    m = x.abs().amax(-1)
    byte = torch.tensor([scale_byte(v) for v in m.flatten().tolist()], dtype=torch.uint8).view(m.shape)
    # (no value is exactly between two of e4m3, so that rounding to fp32 on the way changes nothing)
    return (x * torch.exp2(127 - byte.double())[..., None]).float().to(F8), byte


def cache_pair(g, shape, heads_first=False, spread=3, device=DEV):
    """Two caches [pages, page, heads, D] with rows of several sizes, and their scales; `heads_first`: the
    storage of both is [pages, heads, page, ..]."""
    out = []
    for _ in range(2):
        x = torch.randn(*shape, generator=g, device=device)
        e = torch.randint(-spread, spread + 1, shape[:3], generator=g, device=device)
        m = x.abs().amax(-1, keepdim=True)
        c = (x / m * 440).to(F8)               # the scale is free: any byte stands for a row
        s = (e + 119).to(torch.uint8)          # 440 * 2^-8 and thereabouts
        if heads_first:
            c = c.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(F8)
            s = s.transpose(1, 2).contiguous().transpose(1, 2)
        out.append((c, s))
    (kc, ks), (vc, vs) = out
    return kc, vc, ks, vs


def case(seed, lens, hq, hkv, D, page, n, dtype, heads_first=False, big=1.0, spread=3):
    """As tests.test_attn_decode.case, over a cache in 8 bits: q, k, v, scales, table, lengths. Rows that no
    request holds are NaN with a scale of 255."""
    g = synth.generator(seed, DEV)
    used = [(x + page - 1) // page for x in lens]
    pages = sum(used) + 2
    kc, vc, ks, vs = cache_pair(g, (pages, page, hkv, D), heads_first, spread)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(used + [1]) + 2), 2 ** 30, dtype=torch.int32, device=DEV)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
        tail = used[b] * page - lens[b]
        if tail:
            for c in (kc, vc):
                c.view(torch.uint8)[int(table[b, u - 1]), page - tail:] = 0x7f
            for s in (ks, vs):
                s[int(table[b, u - 1]), page - tail:] = 255
    q = (big * torch.randn(len(lens) * n, hq * D + 16, generator=g, device=DEV)).to(dtype)
    return (q[:, :hq * D].unflatten(1, (hq, D)), kc, vc, ks, vs, table,
            torch.tensor(lens, dtype=torch.int32, device=DEV))


def in_64_bits(kc, vc, ks, vs):
    """The caches' values on the CPU; scales of rows that hold NaN do not matter."""
    fix = lambda s: torch.where(s == 255, 127, s)      # noqa: E731
    return values(kc.cpu(), fix(ks.cpu())), values(vc.cpu(), fix(vs.cpu()))
