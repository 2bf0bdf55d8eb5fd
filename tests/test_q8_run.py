"""The operators of the 8-bit cache together, as a server runs them: a prompt written once, its pages shared by
several samples, which then decode token by token; against 64 bits over the rows that kv_cache_read_q8 gives back,
and those against what was written."""
import pytest
import torch

from state_cached_causal_gb300 import ops, synth
from tests._mixers import assert_close, attn_ref, norm_rope_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("prompt,samples,n_spec", [(70, 3, 0), (128, 5, 2), (333, 9, 0)])
def test_samples_of_one_prompt(prompt, samples, n_spec, q8):
    hq, hkv, D, page, steps, n = 8, 2, 128, 16, 4, 1 + n_spec
    g = synth.generator(prompt, DEV)
    width = (prompt + steps * n + page - 1) // page
    pages = (samples + 1) * width + 1
    shape = (pages, page, hkv, D)
    if q8:
        kc, vc = (torch.full(shape, 0x7f, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
        ks, vs = (torch.full(shape[:3], 255, dtype=torch.uint8, device=DEV) for _ in range(2))
        scales = (ks, vs)
    else:
        kc, vc = (torch.full(shape, float("nan"), dtype=BF16, device=DEV) for _ in range(2))
        scales = ()
    table = torch.randperm(pages, generator=g, device=DEV)[:samples * width].view(samples, width).to(torch.int32)
    whole = prompt // page
    table[1:, :whole] = table[0, :whole]                # whole pages of the prompt are shared
    cs = torch.randn(prompt + steps * n, D, generator=g, device=DEV)
    qw, kw = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(BF16), None
    err = i32([0])
    rows = {}                                           # (sample, position) -> k, v as they were given

    def write(x, owner, pos):
        """Heads of rows x of these samples at these positions into the cache; the queries."""
        q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([hq * D, hkv * D, hkv * D], 1))
        at = torch.tensor(pos, device=DEV)
        slot = table[torch.tensor(owner, device=DEV), at // page] * page + (at % page).to(torch.int32)
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        fn = ops.attn_norm_rope_cache_q8 if q8 else ops.attn_norm_rope_cache
        fn(q, k, v, qw, kw, 1e-6, cs, i32(pos), False, kc, vc, *scales, slot.contiguous(), q_out, dev_err=err)
        want_k = norm_rope_ref(k.cpu(), None, 1e-6, cs.cpu(), pos, False)
        for i, (b, p) in enumerate(zip(owner, pos)):
            rows[b, p] = want_k[i], v[i].cpu().double()
        want_q = norm_rope_ref(q.cpu(), qw.cpu(), 1e-6, cs.cpu(), pos, False)
        assert_close(q_out, want_q, "queries")
        return q_out

    draw = lambda t: torch.randn(t, (hq + 2 * hkv) * D, generator=g, device=DEV).to(BF16)   # noqa: E731
    x = draw(prompt)
    write(x, [0] * prompt, list(range(prompt)))
    tail = list(range(whole * page, prompt))            # the page that it ends in is each sample's own
    for b in range(1, samples):
        if tail:
            write(x[tail], [b] * len(tail), tail)
    cu, prefix = i32([0, samples]), i32([prompt])
    for step in range(steps):
        first = prompt + step * n
        owner = [b for b in range(samples) for _ in range(n)]
        q = write(draw(samples * n), owner, [first + i for _ in range(samples) for i in range(n)])
        lens = i32([first + n] * samples)
        out, plain = torch.zeros_like(q), torch.zeros_like(q)
        shared = ops.attn_decode_shared_q8 if q8 else ops.attn_decode_shared
        shared(q, kc, vc, *scales, table, lens, cu, prefix, n_spec, D ** -0.5, out, dev_err=err)
        decode = ops.attn_decode_q8 if q8 else ops.attn_decode
        decode(q, kc, vc, *scales, table, lens, n_spec, D ** -0.5, plain, dev_err=err)
        if q8:
            back = [torch.zeros(pages * page, hkv, D, device=DEV) for _ in range(2)]
            ops.kv_cache_read_q8(kc, vc, ks, vs, torch.arange(pages * page, dtype=torch.int32, device=DEV), *back,
                                 dev_err=err)
            kd, vd = (t.cpu().view(shape).double() for t in back)
        else:
            kd, vd = kc.cpu().double(), vc.cpu().double()
        torch.cuda.synchronize()
        assert err.item() == 0
        want, _ = attn_ref(q.cpu(), kd, vd, table.cpu(), lens.tolist(), n, D ** -0.5)
        assert_close(out, want, f"step {step}, shared")
        assert_close(plain, want, f"step {step}, each alone")
    for (b, p), (k, v) in rows.items():
        page_of = int(table[b, p // page])
        for got, w in ((kd, k), (vd, v)):
            m = w.abs().amax(-1, keepdim=True)
            # half a step of e4m3 (2^-4), or of values below its normal ones; bf16: half a step, 2^-8
            off = (got[page_of, p % page] - w).abs()
            assert (off <= (w.abs() * 2.0 ** -4 + m * 2.0 ** -17 if q8 else w.abs() * 2.0 ** -8) * 1.001
                    + m * 2.0 ** -20).all()
