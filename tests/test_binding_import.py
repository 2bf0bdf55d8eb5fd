"""Types that the binding takes: on a PyTorch without the 8-bit scales' one everything loads, and a cache in 8 bits takes
its scales as uint8; the C module refuses what Python refuses."""
import subprocess
import sys

import pytest
import torch

from state_cached_causal_gb300 import build as cbuild
from state_cached_causal_gb300 import ops
from tests.test_mixer_abi import _Placed, _two, no_gpu
from tests.test_q8_abi import _calls

SCRIPT = r'''
import torch
for name in %r:
    delattr(torch, name)
from state_cached_causal_gb300 import ops
ops.load()
assert ops._fast is not None
u8 = torch.zeros(5, 16, 2, 64, dtype=torch.uint8)
scale, out = u8[..., 0].contiguous(), torch.zeros(4, 2, 64)
args = (scale, scale, torch.zeros(4, dtype=torch.int32), out, out)
try:
    if hasattr(torch, "float8_e4m3fn"):
        f8 = u8.view(torch.float8_e4m3fn)
        ops.kv_cache_read_q8(f8, f8, *args)
except ValueError as e:
    assert "must live on the GPU" in str(e), e
else:
    assert not hasattr(torch, "float8_e4m3fn")
try:
    ops.kv_cache_read_q8(u8, u8, *args)
except TypeError as e:
    assert "float8_e4m3fn" in str(e)
else:
    raise AssertionError("bytes of no type were taken")
'''


def test_without_the_types_of_8_bits():
    cbuild.build()
    for names in (["float8_e8m0fnu"], ["float8_e8m0fnu", "float8_e4m3fn"]):
        r = subprocess.run([sys.executable, "-c", SCRIPT % (names,)], cwd=cbuild.ROOT, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]


@no_gpu
def test_types_that_python_refuses_are_refused_in_c(monkeypatch):
    """Truth values are no scales, and scales are no flags."""
    lib = ops.load()
    if ops._fast is None:
        pytest.skip("the C module is not built")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(ops, "_raw_stream", lambda stream: None)
    ops._fast.init(lib._handle, (torch.float32, torch.bfloat16, torch.int32, torch.uint8, torch.bool, ops._F8,
                                 ops._F8_SCALE), lambda d: 0, None, lambda: 0)
    placed = lambda call: {n: _Placed(t) if torch.is_tensor(t) else t for n, t in call.items()}     # noqa: E731
    norm, read, attn, q8, i = _calls()
    attn = dict(attn, workspace=torch.zeros(1 << 26, dtype=torch.uint8))
    try:
        for fn, call in (("attn_norm_rope_cache_q8", norm), ("kv_cache_read_q8", read), ("attn_decode_q8", attn)):
            with pytest.raises(ops.CConvError, match=fn):            # (there is no GPU)
                getattr(ops, fn)(**placed(call))
            for name in ("k_scale", "v_scale"):
                with pytest.raises(TypeError, match=name):
                    getattr(ops, fn)(**placed({**call, name: call[name].bool()}))
        gdn, _, _, _ = _two()
        for fn, call in (("gdn_fwd_varlen", gdn),):
            call = dict(call, state_idx=i(2), cu_seqlens=i(3), has_init=torch.zeros(2, dtype=torch.bool))
            with pytest.raises(ops.CConvError, match=fn):
                getattr(ops, fn)(**placed(call))
            with pytest.raises(TypeError, match="has_init"):
                getattr(ops, fn)(**placed(dict(call, has_init=call["has_init"].to(torch.uint8).view(ops._F8_SCALE))))
    finally:
        ops._load_fast(lib)
