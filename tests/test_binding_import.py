"""The binding on a PyTorch without the 8-bit scales' type: everything loads, and a cache in 8 bits takes its scales as
uint8."""
import subprocess
import sys

from state_cached_causal_gb300 import build as cbuild

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
