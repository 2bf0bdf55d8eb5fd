"""Measured cases of the mixer operators that follow the short convolutions: the gated delta rule over a
packed varlen batch (``delta prefill``) and for decode and speculative decode (``delta update``), the
per-head norm and rotation of q and k with the write into a paged cache (``norm rope``), and the attention
of new tokens over that cache (``attention``).

``run`` computes an operator in plain torch (32-bit arithmetic, one rounding at the end) where ``own`` is
false, and calls ``state_cached_causal_gb300.ops`` where it is true. ``exact`` is the operators' definition in
64 bits, token by token. State pools and caches are updated in place, as a serving loop does, and returned whole.
"""
import math
import random

import torch

own = False

CHUNK = 64
L2_EPS = 1e-6
NORM_EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # a mixed continuous batch: 128 one-token decodes, then 16 prefills of up to 2048 tokens; the 8192
        # q/k/v channels are 16 + 16 heads of q and k and 32 of v, the state pool holds 512 slots
        dict(name="delta prefill mixed", op="prefill", hk=16, hv=32, decodes=128, prefills=16,
             max_len=2048, ragged=1, slots=512, state="f32"),
        # one long prompt alone: the chain of its chunks is what counts
        dict(name="delta prefill long", op="prefill", hk=16, hv=32, decodes=0, prefills=1,
             max_len=16384, ragged=0, slots=4, state="bf16"),
        # a short odd prompt of a small model: latency
        dict(name="delta prefill short", op="prefill", hk=4, hv=8, decodes=0, prefills=1,
             max_len=77, ragged=0, slots=4, state="f32"),
        # 64 requests decode one token each, out of a pool of 256
        dict(name="delta decode", op="update", hk=16, hv=32, batch=64, n_spec=0, slots=256,
             dim=128, dtype="bf16", state="f32"),
        # one request decodes: latency
        dict(name="delta decode one", op="update", hk=16, hv=32, batch=1, n_spec=0, slots=8,
             dim=128, dtype="bf16", state="bf16"),
        # speculative decode: 1 + 3 tokens a request, each token's state in a slot of its own
        dict(name="delta spec", op="update", hk=16, hv=32, batch=128, n_spec=3, slots=520,
             dim=128, dtype="bf16", state="f32"),
        # the tokens of a batch of 256 decodes and 8 prefills of 4096, 16 + 4 heads of 128
        dict(name="norm rope batch", op="norm", hq=16, hkv=4, dim=128, rot=128, tokens=33024,
             page=16, pairs=False, dtype="bf16"),
        # a decode step of an odd number of requests, rotation of half a head, neighbouring pairs, 32-bit type
        dict(name="norm rope decode", op="norm", hq=16, hkv=4, dim=64, rot=32, tokens=61,
             page=16, pairs=True, dtype="f32"),
        # 256 requests decode over contexts of 1 to 8192 tokens
        dict(name="attention batch", op="attn", hq=16, hkv=4, dim=128, batch=256, n_spec=0,
             max_len=8192, ragged=3, page=16, dtype="bf16"),
        # one request with a long context: the length has to be split
        dict(name="attention long", op="attn", hq=16, hkv=4, dim=128, batch=1, n_spec=0,
             max_len=131072, ragged=0, page=64, dtype="bf16"),
        # speculative decode over ragged contexts
        dict(name="attention spec", op="attn", hq=16, hkv=4, dim=128, batch=64, n_spec=3,
             max_len=4096, ragged=5, page=16, dtype="bf16"),
        # a small model's single request in 32 bits: latency
        dict(name="attention short", op="attn", hq=8, hkv=2, dim=64, batch=1, n_spec=0,
             max_len=333, ragged=0, page=16, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prefill", "update", "norm", "attn"])
    if op == "prefill":
        hk = rng.choice([2, 4, 8, 16])
        prefills = _log(rng, 1, 24)
        decodes = rng.choice([0, 0, _log(rng, 1, 100)])
        return dict(op=op, hk=hk, hv=hk * rng.choice([1, 2]), decodes=decodes, prefills=prefills,
                    max_len=_log(rng, 2, 16384 // prefills), ragged=rng.randint(1, 9999),
                    slots=prefills + decodes + rng.randint(1, 40), state=rng.choice(["f32", "bf16"]))
    if op == "update":
        hk, batch, n_spec = rng.choice([2, 4, 8, 16]), _log(rng, 1, 100), rng.choice([0, 0, 1, 2, 3])
        return dict(op=op, hk=hk, hv=hk * rng.choice([1, 2]), batch=batch, n_spec=n_spec,
                    slots=batch * (1 + n_spec) + rng.randint(1, 40), dim=rng.choice([64, 128, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), state=rng.choice(["f32", "bf16"]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8] if hkv < 4 else [1, 2, 4])
    if op == "norm":
        dim = rng.choice([64, 128, 256])
        top = 33024 * 16 * 128 // (max(hq, 16) * dim) // (2 if dtype == "f32" else 1)
        return dict(op=op, hq=hq, hkv=hkv, dim=dim, rot=rng.choice([dim, dim // 2, dim // 4]),
                    tokens=_log(rng, 1, top), page=rng.choice([16, 32, 64]),
                    pairs=rng.choice([False, True]), dtype=dtype)
    dim, batch = rng.choice([64, 128, 128, 256]), _log(rng, 1, 200)
    top = 256 * 4096 * 4 * 128 // (hkv * dim * batch) // (2 if dtype == "f32" else 1)
    return dict(op=op, hq=hq, hkv=hkv, dim=dim, batch=batch, n_spec=rng.choice([0, 0, 1, 3]),
                max_len=_log(rng, 16, min(131072, top)), ragged=rng.randint(1, 9999),
                page=rng.choice([16, 32, 64]), dtype=dtype)


def _lens(case):
    """Sequence (or context) lengths: decodes of one token first; all of max_len where ragged is 0."""
    n = case["prefills"] if "prefills" in case else case["batch"]
    if case["ragged"] == 0:
        tail = [case["max_len"]] * n
    else:
        r = random.Random(case["ragged"])
        tail = [r.randint(1, case["max_len"]) for _ in range(n)]
    return [1] * case.get("decodes", 0) + tail


# ---- inputs ----------------------------------------------------------------

def _gate_inputs(T, hv, dtype, g):
    """Raw gate projections, and A in [1, 16], dt in [1e-3, 1e-1] as such layers are initialised."""
    dev = torch.device("cuda")
    a = torch.randn(T, hv, generator=g, device=dev).to(dtype)
    b = torch.randn(T, hv, generator=g, device=dev).to(dtype)
    A_log = torch.log(1 + 15 * torch.rand(hv, generator=g, device=dev))
    dt = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(hv, generator=g, device=dev))
    return a, b, A_log, dt + torch.log(-torch.expm1(-dt))


def _qkv_rows(T, hk, hv, d, dtype, g):
    """One row of q, k, v channels a token, SiLU of a convolution's output, and its three views."""
    x = torch.randn(T, (2 * hk + hv) * d, generator=g, device="cuda")
    x = (x * torch.sigmoid(x)).to(dtype)
    q, k, v = x.split([hk * d, hk * d, hv * d], dim=1)
    return q.unflatten(1, (hk, d)), k.unflatten(1, (hk, d)), v.unflatten(1, (hv, d))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev, op = torch.device("cuda"), case["op"]
    s = dict(op=op)
    if op in ("prefill", "update"):
        hk, hv, d = case["hk"], case["hv"], case.get("dim", 128)
        dtype = TYPES[case.get("dtype", "bf16")]
        lens = _lens(case) if op == "prefill" else [1 + case["n_spec"]] * case["batch"]
        T = sum(lens)
        s["q"], s["k"], s["v"] = _qkv_rows(T, hk, hv, d, dtype, g)
        s["a"], s["b"], s["A_log"], s["dt_bias"] = _gate_inputs(T, hv, dtype, g)
        pool = torch.randn(case["slots"], hv, d, d, generator=g, device=dev)
        s["states"] = pool.mul_(0.2).to(TYPES[case["state"]])
        perm = torch.randperm(case["slots"], generator=g, device=dev).to(torch.int32)
        s["scale"] = d ** -0.5
        s["out"] = torch.zeros(T, hv, d, device=dev, dtype=dtype)
        if op == "prefill":
            s["lens"] = lens
            s["state_idx"] = perm[:len(lens)].contiguous()
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
            hi = (torch.rand(len(lens), generator=g, device=dev) < 0.5).to(torch.uint8)
            hi[:case["decodes"]] = 1
            s["has_init"] = hi
        else:
            B, ns = case["batch"], case["n_spec"]
            s["n_spec"] = ns
            s["state_idx"] = perm[:B * (1 + ns)].reshape(B, 1 + ns).contiguous()
            s["num_accepted"] = torch.randint(1, 2 + ns, (B,), generator=g, device=dev,
                                              dtype=torch.int32)
        return s
    hq, hkv, d, page, dtype = case["hq"], case["hkv"], case["dim"], case["page"], TYPES[case["dtype"]]
    if op == "norm":
        T = case["tokens"]
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
        pages = (T + page - 1) // page + 3
        s["k_cache"] = torch.randn(pages, page, hkv, d, generator=g, device=dev).to(dtype)
        s["v_cache"] = torch.randn(pages, page, hkv, d, generator=g, device=dev).to(dtype)
        s["slots"] = torch.randperm(pages * page, generator=g, device=dev)[:T].to(torch.int32)
        if T > 8:
            s["slots"][T // 2] = -1         # a padding row
        s["q_out"] = torch.zeros(T, hq, d, device=dev, dtype=dtype)
        return s
    B, q_len = case["batch"], 1 + case["n_spec"]
    lens = [max(n, q_len) for n in _lens(case)]
    width = max((n + page - 1) // page for n in lens)
    used = [(n + page - 1) // page for n in lens]
    pages = sum(used) + 2
    s["q"] = torch.randn(B * q_len, hq, d, generator=g, device=dev).to(dtype)
    s["k_cache"] = torch.randn(pages, page, hkv, d, generator=g, device=dev).to(dtype)
    s["v_cache"] = torch.randn(pages, page, hkv, d, generator=g, device=dev).to(dtype)
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    n_used = torch.tensor(used, device=dev)
    col = torch.arange(width, device=dev)
    at = (n_used.cumsum(0) - n_used)[:, None] + col
    s["block_table"] = torch.where(col < n_used[:, None], perm[at.clamp(max=pages - 1)], -1)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["n_spec"], s["scale"] = case["n_spec"], d ** -0.5
    s["out"] = torch.zeros(B * q_len, hq, d, device=dev, dtype=dtype)
    return s


# ---- one pass --------------------------------------------------------------

def run(state):
    return {"prefill": _prefill, "update": _update, "norm": _norm, "attn": _attn}[state["op"]](state)


def _prefill(s):
    if own:
        from state_cached_causal_gb300 import ops
        ops.gdn_fwd_varlen(s["q"], s["k"], s["v"], s["a"], s["b"], s["A_log"], s["dt_bias"],
                           s["states"], s["state_idx"], s["cu_seqlens"], s["has_init"],
                           s["scale"], s["out"])
    else:
        _plain_prefill(s)
    return s["out"], s["states"]


def _update(s):
    if own:
        from state_cached_causal_gb300 import ops
        ops.gdn_update(s["q"], s["k"], s["v"], s["a"], s["b"], s["A_log"], s["dt_bias"],
                       s["states"], s["state_idx"], s["n_spec"], s["num_accepted"], None,
                       s["scale"], s["out"])
    else:
        _plain_update(s)
    return s["out"], s["states"]


def _norm(s):
    if own:
        from state_cached_causal_gb300 import ops
        ops.attn_norm_rope_cache(s["q"], s["k"], s["v"], s["qw"], s["kw"], NORM_EPS, s["cos_sin"],
                                 s["positions"], s["pairs"], s["k_cache"], s["v_cache"],
                                 s["slots"], s["q_out"])
    else:
        _plain_norm(s)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _attn(s):
    if own:
        from state_cached_causal_gb300 import ops
        ops.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                        s["n_spec"], s["scale"], s["out"])
    else:
        _plain_attn(s)
    return s["out"]


# ---- plain forms -----------------------------------------------------------

def _heads(s):
    """q and k normalised and repeated for every v head, v, log decay and beta, in 32 bits."""
    rep = s["v"].shape[1] // s["k"].shape[1]
    q, k = s["q"].float(), s["k"].float()
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + L2_EPS) * s["scale"]
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + L2_EPS)
    x = s["a"].float() + s["dt_bias"]
    softplus = torch.log1p(torch.exp(-x.abs())) + x.clamp(min=0)
    return (q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1), s["v"].float(),
            -torch.exp(s["A_log"]) * softplus, torch.sigmoid(s["b"].float()))


def _plain_prefill(s):
    """Chunks of 64 tokens of every sequence: the products inside them at once, then chunk by chunk
    with the sequences in order of falling length, so that those still running are the first ones."""
    q, k, v, g, beta = _heads(s)
    dev, lens = q.device, s["lens"]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    count = [(lens[i] + CHUNK - 1) // CHUNK for i in order]
    alive = [sum(c > n for c in count) for n in range(count[0])]
    at = torch.cat([torch.full((m,), n, device=dev) for n, m in enumerate(alive)]) * CHUNK
    seq = torch.tensor(order, device=dev)[torch.cat([torch.arange(m, device=dev) for m in alive])]
    start, length = s["cu_seqlens"][:-1].long()[seq], torch.tensor(lens, device=dev)[seq]
    pos = at[:, None] + torch.arange(CHUNK, device=dev)
    valid = pos < length[:, None]
    row = torch.where(valid, start[:, None] + pos, 0)
    take = lambda x: (x[row] * valid[(...,) + (None,) * (x.dim() - 1)]).transpose(1, 2)  # noqa: E731
    q, k, v, g, beta = take(q), take(k), take(v), take(g), take(beta)      # [chunks, head, 64, ..]
    G = g.cumsum(-1)
    i = torch.arange(CHUNK, device=dev)
    low = i[:, None] >= i
    decay = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf))
    A = torch.where(i[:, None] > i, beta[..., None] * decay * (k @ k.transpose(-1, -2)), 0)
    T = torch.eye(CHUNK, device=dev).expand_as(A).clone()
    for r in range(1, CHUNK):
        T[..., r, :r] = -(A[..., r, None, :r] @ T[..., :r, :r])[..., 0, :]
    P = decay * (q @ k.transpose(-1, -2))
    U, W = T @ (beta[..., None] * v), T @ ((beta * G.exp())[..., None] * k)
    qg, kg = q * G.exp()[..., None], k * torch.exp(G[..., -1:] - G)[..., None]
    slot = s["state_idx"].long()[torch.tensor(order, device=dev)]
    init = s["has_init"][torch.tensor(order, device=dev)].bool()
    S = torch.where(init[:, None, None, None], s["states"][slot].float(), 0)
    o, first = torch.empty_like(v), 0
    for m in alive:
        c = slice(first, first + m)
        vn = U[c] - W[c] @ S[:m]
        o[c] = qg[c] @ S[:m] + P[c] @ vn
        S[:m] = G[c, :, -1, None, None].exp() * S[:m] + kg[c].transpose(-1, -2) @ vn
        first += m
    s["out"][row[valid]] = o.transpose(1, 2)[valid].to(s["out"].dtype)
    s["states"][slot] = S.to(s["states"].dtype)


def _plain_update(s):
    q, k, v, g, beta = _heads(s)
    B, n = s["state_idx"].shape
    q, k, v, g, beta = (x.unflatten(0, (B, n)) for x in (q, k, v, g, beta))
    slots = s["state_idx"].long()
    S = s["states"][slots.gather(1, s["num_accepted"].long()[:, None] - 1)[:, 0]].float()
    o = torch.empty_like(v)
    for t in range(n):
        S = S * g[:, t].exp()[..., None, None]
        r = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, None, :] @ S)[..., 0, :])
        S = S + k[:, t, :, :, None] * r[..., None, :]
        o[:, t] = (q[:, t, :, None, :] @ S)[..., 0, :]
        s["states"][slots[:, t]] = S.to(s["states"].dtype)
    s["out"].copy_(o.flatten(0, 1))


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
    s["k_cache"].flatten(0, 1)[at] = turn(s["k"], s["kw"])[keep].to(s["k_cache"].dtype)
    s["v_cache"].flatten(0, 1)[at] = s["v"][keep]


def _plain_attn(s):
    B, page = s["seq_lens"].shape[0], s["k_cache"].shape[1]
    n, hq, d = 1 + s["n_spec"], s["q"].shape[1], s["q"].shape[2]
    hkv = s["k_cache"].shape[2]
    table = s["block_table"].long().clamp(min=0)
    k = s["k_cache"][table].flatten(1, 2).float().transpose(1, 2)         # [B, hkv, length, d]
    v = s["v_cache"][table].flatten(1, 2).float().transpose(1, 2)
    q = s["q"].float().reshape(B, n, hkv, hq // hkv, d).transpose(1, 2).flatten(2, 3)
    x = (q @ k.transpose(-1, -2)) * s["scale"]                            # [B, hkv, n * group, length]
    last = s["seq_lens"].long()[:, None] - n + 1 + torch.arange(n, device=q.device)
    seen = torch.arange(table.shape[1] * page, device=q.device) < last[..., None]
    x = x.masked_fill(~seen.repeat_interleave(hq // hkv, 1)[:, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p @ v) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.unflatten(2, (n, hq // hkv)).transpose(1, 2).reshape(B * n, hq, d))


# ---- work ------------------------------------------------------------------

def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}
    if op in ("prefill", "update"):
        hk, hv, d, e = case["hk"], case["hv"], case.get("dim", 128), size[case.get("dtype", "bf16")]
        one = hv * d * d * size[case["state"]]
        if op == "prefill":
            lens = _lens(case)
            T = sum(lens)
            # every sequence's state is written, those of about half the prefills are read
            moved = one * (2 * case["decodes"] + 1.5 * case["prefills"])
        else:
            T = case["batch"] * (1 + case["n_spec"])
            moved = one * (case["batch"] + T)
        return {"bytes": T * e * ((2 * hk + 2 * hv) * d + 2 * hv) + moved, "flops": 6.0 * T * hv * d * d}
    hq, hkv, d, e = case["hq"], case["hkv"], case["dim"], size[case["dtype"]]
    if op == "norm":
        T = case["tokens"]
        return {"bytes": T * (2 * (hq + 2 * hkv) * d * e + 4 * case["rot"]), "flops": 10.0 * T * (hq + hkv) * d}
    n = 1 + case["n_spec"]
    total = sum(max(x, n) for x in _lens(case))
    return {"bytes": total * 2 * hkv * d * e + 2 * case["batch"] * n * hq * d * e,
            "flops": 4.0 * total * n * hq * d}


# ---- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("prefill", "update"):
        return _exact_delta(s)
    return _exact_norm(s) if case["op"] == "norm" else _exact_attn(s)


def _exact_delta(s):
    """The recurrence, a token of every sequence at a time."""
    d64 = torch.float64
    hk, hv = s["k"].shape[1], s["v"].shape[1]
    of = torch.arange(hv, device="cuda") // (hv // hk)
    q, k, v = s["q"].to(d64), s["k"].to(d64), s["v"].to(d64)
    q = (q / torch.sqrt(q.pow(2).sum(-1, keepdim=True) + L2_EPS))[:, of]
    k = (k / torch.sqrt(k.pow(2).sum(-1, keepdim=True) + L2_EPS))[:, of]
    rate = torch.exp(s["A_log"].to(d64))
    alpha = torch.exp(-rate * torch.nn.functional.softplus(s["a"].to(d64) + s["dt_bias"].to(d64),
                                                           threshold=700))
    beta = 1 / (1 + torch.exp(-s["b"].to(d64)))
    pool = s["states"].to(d64)
    out = torch.zeros_like(v)
    prefill = s["op"] == "prefill"
    if prefill:
        order = torch.argsort(torch.tensor(s["lens"], device="cuda"), descending=True)
        first, slot = s["cu_seqlens"].long()[order], s["state_idx"].long()[order]
        S = pool[slot] * s["has_init"].to(d64)[order][:, None, None, None]
        sizes = sorted(s["lens"], reverse=True)     # how many still run at each token
        m, running = len(sizes), []
        for t in range(sizes[0]):
            while sizes[m - 1] <= t:
                m -= 1
            running.append(m)
    else:
        B, n = s["state_idx"].shape
        first = torch.arange(B, device="cuda") * n
        slots = s["state_idx"].long()
        S = pool[slots[torch.arange(B, device="cuda"), s["num_accepted"].long() - 1]]
        running = [B] * n
    for t, m in enumerate(running):
        at = first[:m] + t
        now = S[:m]
        now *= alpha[at][..., None, None]
        err = v[at] - torch.einsum("bhk,bhkv->bhv", k[at], now)
        now += torch.einsum("bhk,bhv->bhkv", k[at], beta[at][..., None] * err)
        out[at] = torch.einsum("bhk,bhkv->bhv", q[at], now) * s["scale"]
        if not prefill:
            pool[slots[:, t]] = now
    if prefill:
        pool[slot] = S
    return out, pool


def _exact_norm(s):
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

    kc, vc = s["k_cache"].to(d64), s["v_cache"].to(d64)
    page = kc.shape[1]
    k = one(s["k"], s["kw"])
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"].long()[rows]
    kc[at // page, at % page] = k[rows]
    vc[at // page, at % page] = s["v"].to(d64)[rows]
    return one(s["q"], s["qw"]), kc, vc


def _exact_attn(s):
    """A request at a time."""
    d64 = torch.float64
    page, n, hq = s["k_cache"].shape[1], 1 + s["n_spec"], s["q"].shape[1]
    group = hq // s["k_cache"].shape[2]
    out = torch.zeros_like(s["q"], dtype=d64)
    for b, length in enumerate(s["seq_lens"].tolist()):
        pages = s["block_table"][b, :(length + page - 1) // page].long()
        k = s["k_cache"][pages].flatten(0, 1)[:length].to(d64)
        v = s["v_cache"][pages].flatten(0, 1)[:length].to(d64)
        for i in range(n):
            see = length - (n - 1 - i)
            q = s["q"][b * n + i].to(d64).unflatten(0, (-1, group))
            w = torch.softmax(torch.einsum("hgd,lhd->hgl", q, k[:see]) * s["scale"], -1)
            out[b * n + i] = torch.einsum("hgl,lhd->hgd", w, v[:see]).flatten(0, 1)
    return out
