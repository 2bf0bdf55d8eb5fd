"""Plain 64-bit CPU forms of the operators behind the convolutions, and what their tests share.

Tolerances (2-norm of the error over the 2-norm of the result, and the largest error over
max(rms, |value|)), from the arithmetic the kernels state:
* fp32 results: sums of up to a few thousand fp32 terms are off by sqrt(n) 2^-24 (4e-6 at n = 4096), and
  a sum of two bf16 terms stands for an fp32 factor to 2^-17; three such factors in a row stay under
  1e-5 in norm; a single element may be 100 times further off than the norm (cancellation).
* bf16 results: one rounding is 2^-9 at most; operands that the kernel rounds to bf16 once (softmax
  weights, the factors of an output product) add the same again twice: 2^-7 in norm, and 2^-4 for a
  single element, whose terms may cancel.
"""
import math

import torch

TOL = {torch.float32: (1e-5, 1e-3), torch.bfloat16: (2.0 ** -7, 2.0 ** -4)}


def assert_close(got, want, what):
    g, w = got.detach().double().cpu(), want.double()
    assert g.shape == w.shape, what
    if not w.numel():
        return
    assert torch.equal(torch.isfinite(g), torch.isfinite(w)), f"{what}: finite elsewhere"
    fin = torch.isfinite(w)
    assert torch.equal(g[~fin], w[~fin]), what
    g, w = g[fin], w[fin]
    if not w.numel():
        return
    rel, big = TOL[got.dtype]
    norm, rms = w.norm().item(), w.pow(2).mean().sqrt().item()
    err = (g - w)
    assert err.norm().item() <= rel * norm + 1e-12, f"{what}: rel {err.norm().item() / max(norm, 1e-30):.3g}"
    worst = (err.abs() / w.abs().clamp(min=max(rms, 1e-30))).max().item()
    assert worst <= big, f"{what}: max {worst:.3g}"


def gdn_ref(q, k, v, a, b, A_log, dt_bias, S, scale, l2norm=True):
    """One sequence: q, k [L, Hk, dk], v [L, Hv, dv], S [Hv, dk, dv] (all double). Returns the
    outputs and the state after every token (the first entry is S)."""
    L, hv = v.shape[:2]
    rep = hv // k.shape[1]
    if l2norm:
        q = q / torch.sqrt(q.pow(2).sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt(k.pow(2).sum(-1, keepdim=True) + 1e-6)
    x = a + dt_bias
    alpha = torch.exp(-torch.exp(A_log) * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))))
    beta = 1 / (1 + torch.exp(-b))
    out, states = torch.zeros(L, hv, v.shape[2], dtype=torch.float64), [S]
    for t in range(L):
        kt, qt = k[t].repeat_interleave(rep, 0), q[t].repeat_interleave(rep, 0)
        S = alpha[t][:, None, None] * S
        r = beta[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", kt, S))
        S = S + kt[:, :, None] * r[:, None, :]
        out[t] = scale * torch.einsum("hk,hkv->hv", qt, S)
        states.append(S)
    return out, states


def norm_rope_ref(x, w, eps, cos_sin, positions, pairs):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w.double()
    half = cos_sin.shape[1] // 2
    y = x.clone()
    for t in range(x.shape[0]):
        for i in range(half):
            c, s = cos_sin[positions[t], i].double(), cos_sin[positions[t], half + i].double()
            i0, i1 = (2 * i, 2 * i + 1) if pairs else (i, i + half)
            y[t, :, i0] = x[t, :, i0] * c - x[t, :, i1] * s
            y[t, :, i1] = x[t, :, i1] * c + x[t, :, i0] * s
    return y


def attn_ref(q, k_cache, v_cache, table, lens, n, scale):
    """q [B*n, Hq, D], caches [pages, page, Hkv, D]; pages out of range hold nothing."""
    hq, d = q.shape[1:]
    pages, page, hkv = k_cache.shape[:3]
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    for b, length in enumerate(lens):
        for i in range(n):
            at = [(int(table[b, j // page]), j % page) for j in range(length - (n - 1 - i))]
            at = [p for p in at if 0 <= p[0] < pages]
            if not at:
                continue
            p, o = torch.tensor(at).T
            k = k_cache[p, o].double().repeat_interleave(hq // hkv, 1)
            v = v_cache[p, o].double().repeat_interleave(hq // hkv, 1)
            x = torch.einsum("hd,lhd->hl", q[b * n + i].double(), k) * scale
            out[b * n + i] = torch.einsum("hl,lhd->hd", torch.softmax(x, -1), v)
            lse[b * n + i] = torch.logsumexp(x, -1)
    return out, lse
