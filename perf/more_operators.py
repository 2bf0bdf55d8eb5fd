"""Measured cases of the paged cache in 8 bits and of attention over a prefix that requests share: the head
norm, rotation and write into a cache of 8-bit floats (``norm rope q8``), that cache's rows read back
(``read q8``), the attention of new tokens over it (``attention q8``), and the attention of requests whose
first positions are the same, over a cache of either type (``shared``).

``run`` computes an operator in plain torch (32-bit arithmetic, one rounding at the end) where ``own`` is
false, and calls ``state_cached_causal_gb300.ops`` where it is true. ``exact`` is the operators' definition in
64 bits. Caches are updated in place, as a serving loop does, and returned whole.

A cache in 8 bits holds, for each position and kv head, the ``dim`` values of a row as e4m3 floats and the
power of two they are multiplied by, the least one that brings the row's largest value to 448 or below.
"""
import math
import random

import torch

own = False

NORM_EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F8, F8_SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # the tokens of a batch of 256 decodes and 8 prefills of 4096, 16 + 4 heads of 128
        dict(name="norm rope q8 batch", op="norm", hq=16, hkv=4, dim=128, rot=128, tokens=33024,
             page=16, pairs=False, dtype="bf16"),
        # a decode step of an odd number of requests, rotation of half a head, neighbouring pairs, 32-bit type
        dict(name="norm rope q8 decode", op="norm", hq=16, hkv=4, dim=64, rot=32, tokens=61,
             page=16, pairs=True, dtype="f32"),
        # a batch's contexts read back for a prompt that continues them
        dict(name="read q8 batch", op="read", hkv=4, dim=128, tokens=65536, page=16, dtype="bf16"),
        # one short context of a small model: latency
        dict(name="read q8 short", op="read", hkv=2, dim=64, tokens=333, page=16, dtype="f32"),
        # 256 requests decode over contexts of 1 to 8192 tokens
        dict(name="attention q8 batch", op="attn", hq=16, hkv=4, dim=128, batch=256, n_spec=0,
             max_len=8192, ragged=3, page=16, dtype="bf16"),
        # one request with a long context: the length has to be split
        dict(name="attention q8 long", op="attn", hq=16, hkv=4, dim=128, batch=1, n_spec=0,
             max_len=131072, ragged=0, page=64, dtype="bf16"),
        # speculative decode over ragged contexts
        dict(name="attention q8 spec", op="attn", hq=16, hkv=4, dim=128, batch=64, n_spec=3,
             max_len=4096, ragged=5, page=16, dtype="bf16"),
        # a small model's single request in 32 bits: latency
        dict(name="attention q8 short", op="attn", hq=8, hkv=2, dim=64, batch=1, n_spec=0,
             max_len=333, ragged=0, page=16, dtype="f32"),
        # 256 requests behind one document of 32768 tokens, each with up to 1024 of its own
        dict(name="shared batch", op="shared", hq=16, hkv=4, dim=128, groups=1, batch=256, n_spec=0,
             prefix=32768, most_own=1024, ragged=7, page=16, cache="bf16"),
        # eight samples of one long context: few rows, the prefix's bytes count
        dict(name="shared long", op="shared", hq=16, hkv=4, dim=128, groups=1, batch=8, n_spec=0,
             prefix=131072, most_own=256, ragged=8, page=64, cache="bf16"),
        # speculative decode of several groups of requests, each behind its own instructions, cache in 8 bits
        dict(name="shared groups spec q8", op="shared", hq=16, hkv=4, dim=128, groups=7, batch=96,
             n_spec=3, prefix=4096, most_own=2048, ragged=9, page=16, cache="q8"),
        # a small model's four samples: latency
        dict(name="shared short", op="shared", hq=8, hkv=2, dim=64, groups=1, batch=4, n_spec=0,
             prefix=333, most_own=60, ragged=10, page=16, cache="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "read", "attn", "attn", "shared", "shared", "shared"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8] if hkv < 4 else [1, 2, 4])
    page = rng.choice([16, 32, 64])
    if op == "norm":
        dim = rng.choice([64, 128, 256])
        top = 33024 * 16 * 128 // (max(hq, 16) * dim) // (2 if dtype == "f32" else 1)
        return dict(op=op, hq=hq, hkv=hkv, dim=dim, rot=rng.choice([dim, dim // 2, dim // 4]),
                    tokens=_log(rng, 1, top), page=page, pairs=rng.choice([False, True]), dtype=dtype)
    if op == "read":
        dim = rng.choice([64, 128, 256])
        top = 65536 * 4 * 128 // (hkv * dim) // (2 if dtype == "f32" else 1)
        return dict(op=op, hkv=hkv, dim=dim, tokens=_log(rng, 1, min(top, 131072)), page=page, dtype=dtype)
    if op == "attn":
        dim, batch = rng.choice([64, 128, 128, 256]), _log(rng, 1, 200)
        top = 256 * 4096 * 4 * 128 // (hkv * dim * batch) // (2 if dtype == "f32" else 1)
        return dict(op=op, hq=hq, hkv=hkv, dim=dim, batch=batch, n_spec=rng.choice([0, 0, 1, 3]),
                    max_len=_log(rng, 16, min(131072, top)), ragged=rng.randint(1, 9999),
                    page=page, dtype=dtype)
    dim, batch, n_spec = rng.choice([64, 128, 128, 256]), _log(rng, 1, 200), rng.choice([0, 0, 1, 3])
    groups = min(batch, rng.choice([1, 1, _log(rng, 2, 24)]))
    top = min(4096 * 32768 * 128 // (batch * (1 + n_spec) * hq * dim), 131072 * 4 * 128 // (groups * hkv * dim))
    return dict(op=op, hq=hq, hkv=hkv, dim=dim, groups=groups, batch=batch, n_spec=n_spec,
                prefix=_log(rng, 16, min(131072, top)), most_own=_log(rng, 8, 1024),
                ragged=rng.randint(1, 9999), page=page, cache=rng.choice(["bf16", "bf16", "q8"]))


def _lens(case):
    """Context lengths: all of max_len where ragged is 0."""
    n = case["batch"]
    if case["ragged"] == 0:
        lens = [case["max_len"]] * n
    else:
        r = random.Random(case["ragged"])
        lens = [r.randint(1, case["max_len"]) for _ in range(n)]
    return [max(x, 1 + case["n_spec"]) for x in lens]


def _groups(case):
    """Requests of each group, the groups' prefix lengths (one of them the longest), and the positions
    that each request has behind its prefix, its new tokens among them."""
    r = random.Random(case["ragged"])
    cut = sorted(r.sample(range(1, case["batch"]), case["groups"] - 1))
    sizes = [b - a for a, b in zip([0] + cut, cut + [case["batch"]])]
    prefix = [r.randint((case["prefix"] + 1) // 2, case["prefix"]) for _ in sizes]
    prefix[0] = case["prefix"]
    return sizes, prefix, [r.randint(1, case["most_own"]) + case["n_spec"] for _ in range(case["batch"])]


# ---- inputs ----------------------------------------------------------------

def _to_q8(x):
    """Rows of x as e4m3 values and the biased exponents of their powers of two."""
    m, e = torch.frexp(x.float().abs().amax(-1))          # largest value m 2^e, 1/2 <= m < 1
    e = (e - 9 + (m > 0.875).int()).clamp(-126, 127)      # 448 = 0.875 2^9
    y = torch.ldexp(x.float(), -e[..., None])
    return y.to(F8), (e + 127).to(torch.uint8)


def _from_q8(values, scales):
    return values.float() * torch.exp2(scales.float() - 127)[..., None]


def _rows(x, at):
    """Entries `at` of a tensor's first dimension; 8-bit floats are indexed as bytes."""
    return x.view(torch.uint8)[at].view(x.dtype) if x.dtype == F8 else x[at]


def _cache(s, shape, kind, g):
    for name in ("k", "v"):
        x = torch.randn(*shape, generator=g, device="cuda")
        if kind == "q8":
            # rows of several sizes, as keys and values of trained heads are
            x *= torch.exp2(torch.randint(-3, 4, shape[:3], generator=g, device="cuda").float())[..., None]
            s[name + "_cache"], s[name + "_scale"] = _to_q8(x * 0.5)
        else:
            s[name + "_cache"] = x.to(TYPES[kind])


def _tables(s, used, page, g):
    """A block table over shuffled pages: row b has used[b] of them. Returns the number of pages."""
    dev = torch.device("cuda")
    pages = sum(used) + 2
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    n_used = torch.tensor(used, device=dev)
    col = torch.arange(max(used), device=dev)
    at = (n_used.cumsum(0) - n_used)[:, None] + col
    s["block_table"] = torch.where(col < n_used[:, None], perm[at.clamp(max=pages - 1)], -1)
    return pages


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev, op = torch.device("cuda"), case["op"]
    hkv, d, page = case["hkv"], case["dim"], case["page"]
    s = dict(op=op)
    if op in ("norm", "read"):
        T, dtype = case["tokens"], TYPES[case["dtype"]]
        pages = (T + page - 1) // page + 3
        _cache(s, (pages, page, hkv, d), "q8", g)
        s["slots"] = torch.randperm(pages * page, generator=g, device=dev)[:T].to(torch.int32)
        if op == "read":
            # positions lie in runs of a page, pages anywhere
            order = torch.randperm(pages, generator=g, device=dev)
            at = torch.arange(T, device=dev)
            s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
            s["k_out"], s["v_out"] = (torch.zeros(T, hkv, d, device=dev, dtype=dtype) for _ in range(2))
        if T > 8:
            s["slots"][T // 2] = -1         # a padding row
        if op == "read":
            return s
        hq = case["hq"]
        x = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device=dev).to(dtype)
        q, k, v = x.split([hq * d, hkv * d, hkv * d], dim=1)
        s["q"], s["k"], s["v"] = (q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)),
                                  v.unflatten(1, (hkv, d)))
        s["qw"] = (1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(dtype)
        s["kw"] = (1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(dtype)
        rot, most = case["rot"], 8192
        inv = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        ang = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["pairs"] = case["pairs"]
        s["positions"] = torch.randint(0, most, (T,), generator=g, device=dev, dtype=torch.int32)
        s["q_out"] = torch.zeros(T, hq, d, device=dev, dtype=dtype)
        return s
    B, n, hq = case["batch"], 1 + case["n_spec"], case["hq"]
    dtype = TYPES[case.get("dtype", "bf16")]
    s["n_spec"], s["scale"] = case["n_spec"], d ** -0.5
    s["q"] = torch.randn(B * n, hq, d, generator=g, device=dev).to(dtype)
    s["out"] = torch.zeros(B * n, hq, d, device=dev, dtype=dtype)
    if op == "attn":
        lens = _lens(case)
        pages = _tables(s, [(x + page - 1) // page for x in lens], page, g)
        _cache(s, (pages, page, hkv, d), "q8", g)
    else:
        sizes, prefix, owns = _groups(case)
        of = [i for i, m in enumerate(sizes) for _ in range(m)]
        lens = [prefix[i] + x for i, x in zip(of, owns)]
        # whole pages of the prefix are the group's first request's, for all of the group
        pages = _tables(s, [(x + page - 1) // page for x in lens], page, g)
        first = torch.tensor([sum(sizes[:i]) for i in of], device=dev)
        whole = torch.tensor([prefix[i] // page for i in of], device=dev)
        col = torch.arange(s["block_table"].shape[1], device=dev)
        s["block_table"] = torch.where(col < whole[:, None], s["block_table"][first], s["block_table"])
        # a page that the prefix ends in is each request's own, with the same rows before the end
        _cache(s, (pages, page, hkv, d), case["cache"], g)
        last = torch.tensor([prefix[i] // page for i in of], device=dev)
        theirs = s["block_table"].gather(1, last[:, None])[:, 0].long()
        source = s["block_table"][first].gather(1, last[:, None])[:, 0].long()
        held = torch.arange(page, device=dev) < torch.tensor([prefix[i] % page for i in of], device=dev)[:, None]
        for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
            if name in s:
                c = s[name].view(torch.uint8) if s[name].dtype == F8 else s[name]
                c[theirs] = torch.where(held[(...,) + (None,) * (c.dim() - 2)], c[source], c[theirs])
        cu = [0]
        for m in sizes:
            cu.append(cu[-1] + m)
        s["cu_groups"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device=dev)
        # (what the plain form pads to, known on the host as the lengths are)
        s["most"] = max(sizes), max(prefix), max(owns)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    return s


# ---- one pass --------------------------------------------------------------

def run(state):
    return {"norm": _norm, "read": _read, "attn": _attn, "shared": _shared}[state["op"]](state)


def _norm(s):
    if own:
        from state_cached_causal_gb300 import ops
        ops.attn_norm_rope_cache_q8(s["q"], s["k"], s["v"], s["qw"], s["kw"], NORM_EPS, s["cos_sin"],
                                    s["positions"], s["pairs"], s["k_cache"], s["v_cache"],
                                    s["k_scale"], s["v_scale"], s["slots"], s["q_out"])
    else:
        _plain_norm(s)
    return (s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"].view(F8_SCALE),
            s["v_scale"].view(F8_SCALE))


def _read(s):
    if own:
        from state_cached_causal_gb300 import ops
        ops.kv_cache_read_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"],
                             s["k_out"], s["v_out"])
    else:
        _plain_read(s)
    return s["k_out"], s["v_out"]


def _attn(s):
    if own:
        from state_cached_causal_gb300 import ops
        ops.attn_decode_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                           s["block_table"], s["seq_lens"], s["n_spec"], s["scale"], s["out"])
    else:
        _plain_attn(s)
    return s["out"]


def _shared(s):
    if own:
        from state_cached_causal_gb300 import ops
        if "k_scale" in s:
            ops.attn_decode_shared_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                      s["block_table"], s["seq_lens"], s["cu_groups"],
                                      s["prefix_lens"], s["n_spec"], s["scale"], s["out"])
        else:
            ops.attn_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["block_table"],
                                   s["seq_lens"], s["cu_groups"], s["prefix_lens"], s["n_spec"],
                                   s["scale"], s["out"])
    else:
        _plain_shared(s)
    return s["out"]


# ---- plain forms -----------------------------------------------------------

def _plain_norm(s):
    def turn(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * w.float()
        cos, sin = s["cos_sin"][s["positions"].long()][:, None, :].chunk(2, -1)
        rot = s["cos_sin"].shape[1]
        head, rest = x[..., :rot], x[..., rot:]
        if s["pairs"]:
            x0, x1 = head[..., 0::2], head[..., 1::2]
            y = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
        else:
            x0, x1 = head.chunk(2, -1)
            y = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
        return torch.cat([y, rest], -1)

    s["q_out"].copy_(turn(s["q"], s["qw"]))
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    for name, rows in (("k", turn(s["k"], s["kw"])), ("v", s["v"])):
        values, scales = _to_q8(rows[keep])
        s[name + "_cache"].view(torch.uint8).flatten(0, 1)[at] = values.view(torch.uint8)
        s[name + "_scale"].flatten(0, 1)[at] = scales


def _plain_read(s):
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    for name in ("k", "v"):
        rows = _from_q8(_rows(s[name + "_cache"].flatten(0, 1), at), s[name + "_scale"].flatten(0, 1)[at])
        s[name + "_out"][keep] = rows.to(s[name + "_out"].dtype)


def _gather(s, name, pages, tokens=None):
    """Rows of a cache in 32 bits: whole pages, or one token of each."""
    at = pages if tokens is None else (pages, tokens)
    rows = _rows(s[name + "_cache"], at)
    return _from_q8(rows, s[name + "_scale"][at]) if name + "_scale" in s else rows.float()


def _plain_attn(s):
    B, page = s["seq_lens"].shape[0], s["k_cache"].shape[1]
    n, hq, d = 1 + s["n_spec"], s["q"].shape[1], s["q"].shape[2]
    hkv = s["k_cache"].shape[2]
    table = s["block_table"].long().clamp(min=0)
    k = _gather(s, "k", table).flatten(1, 2).transpose(1, 2)              # [B, hkv, length, d]
    v = _gather(s, "v", table).flatten(1, 2).transpose(1, 2)
    q = s["q"].float().reshape(B, n, hkv, hq // hkv, d).transpose(1, 2).flatten(2, 3)
    x = (q @ k.transpose(-1, -2)) * s["scale"]                            # [B, hkv, n * group, length]
    last = s["seq_lens"].long()[:, None] - n + 1 + torch.arange(n, device=q.device)
    seen = torch.arange(table.shape[1] * page, device=q.device) < last[..., None]
    x = x.masked_fill(~seen.repeat_interleave(hq // hkv, 1)[:, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p @ v) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.unflatten(2, (n, hq // hkv)).transpose(1, 2).reshape(B * n, hq, d))


def _plain_shared(s):
    """The prefixes' products once a group, for all rows of its requests (groups padded to the largest),
    the rest by request, and both under one softmax."""
    B, page = s["seq_lens"].shape[0], s["k_cache"].shape[1]
    n, hq, d, hkv = 1 + s["n_spec"], s["q"].shape[1], s["q"].shape[2], s["k_cache"].shape[2]
    dev, table, cu = s["q"].device, s["block_table"].long().clamp(min=0), s["cu_groups"].long()
    q = s["q"].float().reshape(B, n, hkv, hq // hkv, d).transpose(1, 2).flatten(2, 3)   # [B, hkv, r, d]
    r = q.shape[2]
    # prefixes
    P = s["prefix_lens"].long()
    size = cu[1:] - cu[:-1]
    most_members, most_prefix, most_own = s["most"]
    member = torch.arange(most_members, device=dev)
    rows = q[(cu[:-1, None] + member).clamp(max=B - 1)].transpose(1, 2).flatten(2, 3)   # [G, hkv, m r, d]
    width = (most_prefix + page - 1) // page
    pages = table[cu[:-1]][:, :width]
    k = _gather(s, "k", pages).flatten(1, 2).transpose(1, 2)              # [G, hkv, length, d]
    x = (rows @ k.transpose(-1, -2)) * s["scale"]
    x = x.masked_fill((torch.arange(width * page, device=dev) >= P[:, None])[:, None, None], -math.inf)
    mp = x.amax(-1, keepdim=True)
    p = torch.exp(x - mp)
    del x, k
    lp = p.sum(-1, keepdim=True)
    op = p @ _gather(s, "v", pages).flatten(1, 2).transpose(1, 2)
    del p
    of = torch.repeat_interleave(torch.arange(cu.shape[0] - 1, device=dev), size, output_size=B)
    back = lambda t: t.unflatten(2, (-1, r)).transpose(1, 2)[of, torch.arange(B, device=dev) - cu[of]]  # noqa: E731
    mp, lp, op = back(mp), back(lp), back(op)                             # [B, hkv, r, 1 or d]
    # each request's own positions
    rest = s["seq_lens"].long() - P[of]
    at = torch.arange(most_own, device=dev)
    pos = P[of, None] + at
    own_page = table.gather(1, (pos // page).clamp(max=table.shape[1] - 1))
    k = _gather(s, "k", own_page, pos % page).transpose(1, 2)             # [B, hkv, own, d]
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    last = rest[:, None] - n + 1 + torch.arange(n, device=dev)
    x = x.masked_fill(~(at < last[..., None]).repeat_interleave(hq // hkv, 1)[:, None], -math.inf)
    m = torch.maximum(x.amax(-1, keepdim=True), mp)
    p = torch.exp(x - m)
    o = p @ _gather(s, "v", own_page, pos % page).transpose(1, 2) + op * torch.exp(mp - m)
    o = o / (p.sum(-1, keepdim=True) + lp * torch.exp(mp - m))
    s["out"].copy_(o.unflatten(2, (n, hq // hkv)).transpose(1, 2).reshape(B * n, hq, d))


# ---- work ------------------------------------------------------------------

def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}
    hkv, d = case["hkv"], case["dim"]
    row = 2 * hkv * (d + 1)                        # k and v of a position in 8 bits, with their scales
    if op == "norm":
        T, hq, e = case["tokens"], case["hq"], size[case["dtype"]]
        return {"bytes": T * ((2 * hq + 2 * hkv) * d * e + row + 4 * case["rot"]),
                "flops": 12.0 * T * (hq + 2 * hkv) * d}
    if op == "read":
        T = case["tokens"]
        return {"bytes": T * (row + 2 * hkv * d * size[case["dtype"]]), "flops": 2.0 * T * hkv * d}
    n, hq = 1 + case["n_spec"], case["hq"]
    io = 2 * case["batch"] * n * hq * d * size[case.get("dtype", "bf16")]
    if op == "attn":
        total = sum(_lens(case))
        return {"bytes": total * row + io, "flops": 4.0 * total * n * hq * d}
    sizes, prefix, owns = _groups(case)
    if case["cache"] != "q8":
        row = 2 * hkv * d * size[case["cache"]]
    seen = sum(m * p for m, p in zip(sizes, prefix)) + sum(owns)
    return {"bytes": (sum(prefix) + sum(owns)) * row + io, "flops": 4.0 * seen * n * hq * d}


# ---- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "read":
        return _exact_read(s)
    return _exact_attn(s)


def _values(s, name):
    """A cache's values in 64 bits."""
    c = s[name + "_cache"].to(torch.float64)
    if name + "_scale" in s:
        c = torch.ldexp(c, s[name + "_scale"].int()[..., None] - 127)
    return c


def _exact_norm(s):
    """Written rows as they are before they are rounded to 8 bits, in units of their power of two."""
    d64 = torch.float64
    cs = s["cos_sin"].to(d64)[s["positions"].long()]
    half = cs.shape[1] // 2
    phase = torch.complex(cs[:, :half], cs[:, half:])[:, None, :]

    def one(x, w):
        x = x.to(d64)
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + NORM_EPS) * w.to(d64)
        z = x[..., :2 * half]
        z = z.unflatten(-1, (half, 2)) if s["pairs"] else z.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * phase)
        z = z if s["pairs"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., 2 * half:]], -1)

    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"].long()[rows]
    page = s["k_cache"].shape[1]
    out = []
    for name, x in (("k", one(s["k"], s["kw"])), ("v", s["v"].to(d64))):
        c = s[name + "_cache"].to(d64)
        x = x[rows]
        e = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 448))
        c[at // page, at % page] = x / torch.exp2(e)
        out.append(c)
    # (the powers of two are whole numbers, without a value between)
    return one(s["q"], s["qw"]), out[0], out[1], None, None


def _exact_read(s):
    keep = s["slots"] >= 0
    at = s["slots"].long()[keep]
    page, out = s["k_cache"].shape[1], []
    for name in ("k", "v"):
        o = s[name + "_out"].to(torch.float64)
        o[keep] = _values(s, name)[at // page, at % page]
        out.append(o)
    return tuple(out)


def _exact_attn(s):
    """A request at a time, each over its own block table: the prefix too where it shares one."""
    d64 = torch.float64
    page, n, hq = s["k_cache"].shape[1], 1 + s["n_spec"], s["q"].shape[1]
    group = hq // s["k_cache"].shape[2]
    out = torch.zeros_like(s["q"], dtype=d64)
    for b, length in enumerate(s["seq_lens"].tolist()):
        pages = s["block_table"][b, :(length + page - 1) // page].long()
        part = {x: _rows(s[x], pages) for x in ("k_cache", "v_cache", "k_scale", "v_scale") if x in s}
        k = _values(part, "k").flatten(0, 1)[:length]
        v = _values(part, "v").flatten(0, 1)[:length]
        for i in range(n):
            see = length - (n - 1 - i)
            q = s["q"][b * n + i].to(d64).unflatten(0, (-1, group))
            w = torch.softmax(torch.einsum("hgd,lhd->hgl", q, k[:see]) * s["scale"], -1)
            out[b * n + i] = torch.einsum("hgl,lhd->hgd", w, v[:see]).flatten(0, 1)
    return out
