"""A hybrid model's two kinds of mixer served together: prompts first, then a token at a time.

One gated-delta-rule layer and one attention layer share a batch of requests. Each keeps what its
kind remembers: the delta-rule layer a convolution window and a [dk, dv] state a head, in slots of
two pools; the attention layer the CCA convolution's window and delayed value, and keys and values
in a paged cache. A prompt goes through

    cconv_fwd_varlen -> gdn_fwd_varlen
    cca_qk_conv_fused -> attn_norm_rope_cache

and a decode step through

    cconv_update -> gdn_update
    cca_qk_conv_fused -> attn_norm_rope_cache -> attn_decode

The attention of a prompt's tokens over each other is not part of the library: a prompt fills the cache
here, and the tokens after it attend.

Weights and inputs are random (seeded). Run it on a GPU: python examples/hybrid_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from state_cached_causal_gb300 import ops  # noqa: E402

HIDDEN = 256
GDN_HK, GDN_HV, DIM = 2, 4, 128
ATT_HQ, ATT_HKV = 8, 2
PAGE, MAX_POS = 16, 512
EPS = 1e-6


class HybridMixers:
    """The weights and the memory of both layers, for up to `requests` requests."""

    def __init__(self, requests, seed=0, device="cuda", dtype=torch.bfloat16):
        g = torch.Generator(device=device).manual_seed(seed)
        self.dev, self.dtype, self.requests = torch.device(device), dtype, requests

        def normal(*shape, std=None, like=dtype):
            std = shape[0] ** -0.5 if std is None else std
            return (torch.randn(*shape, generator=g, device=device) * std).to(like)

        f32 = torch.float32
        # gated delta rule: channels of q, k, v behind one convolution, and its gates
        self.C = (2 * GDN_HK + GDN_HV) * DIM
        self.w_qkv, self.w_ab = normal(HIDDEN, self.C), normal(HIDDEN, 2 * GDN_HV)
        self.conv_w, self.conv_b = normal(self.C, 4, std=0.5), normal(self.C, std=0.02)
        self.A_log = torch.log(1 + 15 * torch.rand(GDN_HV, generator=g, device=device))
        self.dt_bias = normal(GDN_HV, std=0.5, like=f32) - 3
        self.conv_pool = torch.zeros(requests, self.C, 3, device=device, dtype=dtype)
        self.states = torch.zeros(requests, GDN_HV, DIM, DIM, device=device)
        # attention behind the CCA convolution
        self.Cqk, self.groups = (ATT_HQ + ATT_HKV) * DIM, ATT_HQ + ATT_HKV
        self.Dv = ATT_HKV * DIM // 2
        self.w_qk, self.w_v = normal(HIDDEN, self.Cqk), normal(HIDDEN, 2 * self.Dv)
        self.w_dw, self.b_dw = normal(self.Cqk, 2, std=0.7), normal(self.Cqk, std=0.02)
        self.w_gr = normal(self.Cqk, DIM, 2, std=(2 * DIM) ** -0.5)
        self.b_gr = normal(self.Cqk, std=0.02)
        self.delayed_init = normal(self.Dv, std=0.02)
        self.cca_pool = torch.zeros(requests, self.Cqk, 2, device=device, dtype=dtype)
        self.delayed = torch.zeros(requests, self.Dv, device=device, dtype=dtype)
        self.q_norm, self.k_norm = 1 + normal(DIM, std=0.1), 1 + normal(DIM, std=0.1)
        freq = 10000.0 ** (-torch.arange(0, DIM, 2, device=device, dtype=f32) / DIM)
        angle = torch.arange(MAX_POS, device=device, dtype=f32)[:, None] * freq
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
        # a request's pages lie anywhere in the cache
        width = MAX_POS // PAGE
        pages = requests * width
        self.table = torch.randperm(pages, generator=g, device=device).to(torch.int32).view(
            requests, width)
        self.k_cache = torch.zeros(pages, PAGE, ATT_HKV, DIM, device=device, dtype=dtype)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.lens = torch.zeros(requests, device=device, dtype=torch.int32)
        self.slots = torch.arange(requests, device=device, dtype=torch.int32)
        # the kernels report bad indices here
        self.err = torch.zeros(1, device=device, dtype=torch.int32)
        self.workspace = torch.empty(ops.attn_decode_workspace_bytes(
            requests, 0, ATT_HQ, ATT_HKV, DIM), device=device, dtype=torch.uint8)

    def _delta(self, x, mixed):
        """q, k, v of the delta rule as views of the convolution's rows, and the raw gates."""
        q, k, v = mixed.split([GDN_HK * DIM, GDN_HK * DIM, GDN_HV * DIM], 1)
        gates = x @ self.w_ab
        return (q.unflatten(1, (GDN_HK, DIM)), k.unflatten(1, (GDN_HK, DIM)),
                v.unflatten(1, (GDN_HV, DIM)), gates[:, :GDN_HV], gates[:, GDN_HV:])

    def _keys(self, x, cu, has_init, positions, owner):
        """The attention layer's queries; its keys and values go to the cache."""
        v = x @ self.w_v
        rows = torch.empty(x.shape[0], self.Cqk + 2 * self.Dv, device=self.dev, dtype=self.dtype)
        ops.cca_qk_conv_fused(x @ self.w_qk, self.w_dw, self.b_dw, self.w_gr, self.b_gr,
                              self.groups, ATT_HQ, 2, 2, v[:, self.Dv:], self.delayed_init,
                              v[:, :self.Dv], self.cca_pool, self.delayed, self.slots, cu,
                              has_init, rows, self.err)
        q, k, v = rows.split([ATT_HQ * DIM, ATT_HKV * DIM, ATT_HKV * DIM], 1)
        page = self.table[owner, positions // PAGE]
        slot = page * PAGE + (positions % PAGE).to(torch.int32)
        heads = [t.unflatten(1, (-1, DIM)) for t in (q, k, v)]
        q_out = torch.empty(x.shape[0], ATT_HQ, DIM, device=self.dev, dtype=self.dtype)
        ops.attn_norm_rope_cache(*heads, self.q_norm, self.k_norm, EPS, self.cos_sin,
                                 positions.to(torch.int32), False, self.k_cache, self.v_cache,
                                 slot, q_out, self.err)
        return heads, q_out

    def prefill(self, x, lens):
        """Prompts of all requests, packed: x [sum(lens), HIDDEN]. Returns the tensors passed on."""
        n = torch.tensor(lens, device=self.dev)
        cu = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        owner = torch.repeat_interleave(torch.arange(len(lens), device=self.dev), n)
        positions = torch.arange(x.shape[0], device=self.dev) - cu[owner]
        mixed = torch.empty(x.shape[0], self.C, device=self.dev, dtype=self.dtype)
        new = torch.zeros(len(lens), device=self.dev, dtype=torch.uint8)
        ops.cconv_fwd_varlen(x @ self.w_qkv, self.conv_w, self.conv_b, self.conv_pool, self.slots,
                             cu, new, 4, 1, ops.ACT_SILU, mixed, dev_err=self.err)
        args = self._delta(x, mixed)
        delta = torch.empty(x.shape[0], GDN_HV, DIM, device=self.dev, dtype=self.dtype)
        ops.gdn_fwd_varlen(*args, self.A_log, self.dt_bias, self.states, self.slots, cu, new,
                           DIM ** -0.5, delta, True, self.err)
        heads, q = self._keys(x, cu, new, positions, owner)
        self.lens = n.to(torch.int32)
        return dict(delta_in=args, delta=delta, heads=heads, q=q, positions=positions)

    def decode(self, x):
        """One more token of every request: x [requests, HIDDEN]."""
        B = self.requests
        mixed = torch.empty(B, self.C, device=self.dev, dtype=self.dtype)
        ops.cconv_update(x @ self.w_qkv, self.conv_pool, self.conv_w, self.conv_b, self.slots, 0,
                         None, None, 4, 1, ops.ACT_SILU, mixed, dev_err=self.err)
        args = self._delta(x, mixed)
        delta = torch.empty(B, GDN_HV, DIM, device=self.dev, dtype=self.dtype)
        ops.gdn_update(*args, self.A_log, self.dt_bias, self.states, self.slots, 0, None, None,
                       DIM ** -0.5, delta, True, self.err)
        cu = torch.arange(B + 1, device=self.dev, dtype=torch.int32)
        old = torch.ones(B, device=self.dev, dtype=torch.uint8)
        heads, q = self._keys(x, cu, old, self.lens.long(), torch.arange(B, device=self.dev))
        self.lens = self.lens + 1
        attn = torch.empty(B, ATT_HQ, DIM, device=self.dev, dtype=self.dtype)
        ops.attn_decode(q, self.k_cache, self.v_cache, self.table, self.lens, 0, DIM ** -0.5, attn,
                        workspace=self.workspace, dev_err=self.err)
        return dict(delta_in=args, delta=delta, heads=heads, q=q, attn=attn)


def serve(lens, steps, seed=0, split=0):
    """Prompts of `lens` tokens, then `steps` tokens each. With `split` > 0 the first `split` of
    those come with the prompts instead: the same tokens by the other path. Returns the mixers, the
    prompts' tensors and those of the last step."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    tokens = [torch.randn(n + steps, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
              for n in lens]
    m = HybridMixers(len(lens), seed)
    first = [n + split for n in lens]
    prompt = m.prefill(torch.cat([t[:n] for t, n in zip(tokens, first)]), first)
    step = None
    for i in range(split, steps):
        step = m.decode(torch.stack([t[n + i] for t, n in zip(tokens, lens)]))
    return m, prompt, step


def main():
    lens, steps = [37, 200, 5, 64], 6
    one = serve(lens, steps)
    two = serve(lens, steps, split=steps - 1)      # all but the last token with the prompts
    torch.cuda.synchronize()
    for what in ("delta", "attn"):
        a, b = one[2][what].float(), two[2][what].float()
        rel = ((a - b).norm() / b.norm()).item()
        print(f"{what}: {steps} single tokens against one after longer prompts: {rel:.2g} apart")
        # bf16 rounds each result and what feeds it by 2^-9, along another order of sums
        assert rel < 2e-2, what
    assert int(one[0].err) == 0 and int(two[0].err) == 0
    print("hybrid step ok")


if __name__ == "__main__":
    main()
