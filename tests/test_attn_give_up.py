"""What a given-up wait of the attention kernel must not do: leave a barrier without a limit short, end the
block under copies in flight, or send the join to parts that were never written. A wait that runs out needs a
copy that never comes, which no call can make, so the rules are held to the source and to a host build here.
"""
import os
import re
import shutil
import subprocess

import pytest

from state_cached_causal_gb300 import build as cbuild


def source(name):
    with open(os.path.join(cbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernel(text, name):
    """The kernel's body, from the braces."""
    at = text.index("{", text.index(f"{name}(const AttnArgs a"))
    depth, i = 0, at
    while True:
        depth += (text[i] == "{") - (text[i] == "}")
        i += 1
        if depth == 0:
            return text[at:i]


def test_no_barrier_without_a_limit_behind_the_first_wait():
    text = source("attn_mma.cu")
    body = kernel(text, "attn_mma_kernel")
    behind = body[body.index("attn_split<"):].split("\n", 1)[1]      # (the split's own come before any wait)
    assert "wait_bar(" in behind
    for call in set(re.findall(r"\b([A-Za-z_]\w*)\s*\(", behind)):
        callee = re.search(rf"void {call}\([^)]*\) \{{(.*?)\n\}}", text, re.S)
        assert "sync" not in call or call in ("__syncwarp", "__any_sync", "__shfl_xor_sync", "fence_proxy_async"), call
        assert not callee or not re.search(r"bar(rier)?\.(cta\.)?sync|__syncthreads", callee.group(1)), call
    assert text.count("mbar_try(") == 1                               # the one in wait_bar


def test_a_warp_that_gives_up_waits_for_the_copies():
    text = source("attn_mma.cu")
    body = kernel(text, "attn_mma_kernel")
    behind = body[body.index("attn_split<"):].split("\n", 1)[1]
    assert behind.count("return;") == 1, "the loading warp's usual end"
    given_up = re.findall(r"if \([^;]*!(wait_bar|meet)\([^;]*?\)\)\s*return settle\(full, stages, (\w+), (\w+),", behind)
    assert given_up == [("wait_bar", "st", "ph"), ("wait_bar", "stage", "phase")] + 3 * [("meet", "stage", "phase")]
    assert len(re.findall(r"\b(?:wait_bar|meet)\(", behind)) == len(given_up) + 1      # (and meet's own wait)
    settle = re.search(r"void settle\([^)]*\) \{(.*?)\n\}", text, re.S).group(1)
    assert re.search(r"for \(int i = 0; i < stages; \+\+i\) wait_bar\(&full\[i\], i < st \? ph \^ 1 : ph, err\);", settle)


@pytest.mark.parametrize("stages", [2, 3, 4])
def test_phases_that_the_loading_warp_ends_on(stages):
    """Place i is waited for in parity `i < st ? ph ^ 1 : ph`: for the loading warp (places from 0, ph from 1)
    that of its last tile, or, where none came, the one in which a fresh barrier counts as done; for one that
    reads (ph from 0) that of the next tile it would come to."""
    st, ph, last = 0, 1, [-1] * stages                                # round of each place's last tile
    for tile in range(4 * stages + 1):
        for i in range(stages):
            assert (ph ^ 1 if i < st else ph) == last[i] % 2
            assert (ph if i < st else ph ^ 1) == (last[i] + 1) % 2
        last[st] = tile // stages
        st += 1
        if st == stages:
            st, ph = 0, ph ^ 1


def test_joins_of_notes_that_were_not_written(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    text = source("attn_decode.cu")
    assert text.count("attn_joins(c0, c1, a.grid)) return;") == 2     # both joins, before any part is read
    src = tmp_path / "joins.cu"
    src.write_text('#include "attn_decode.cuh"\n#include <stdio.h>\nint main() {\n  const int v[] = {'
                   '-2147483647 - 1, -1, 0, 1, 303, 304, 305, 2147483647};\n  for (int a : v)\n    for (int b : v)'
                   '\n      printf("%d %d %d\\n", a, b, (int)cconv::attn_joins(a, b, 304));\n}\n')
    exe = tmp_path / "joins"
    subprocess.run([nvcc, "-std=c++17", "-I", cbuild.CSRC, "-I", cbuild.INCLUDE, str(src), "-o", str(exe)], check=True)
    rows = [tuple(map(int, r.split())) for r in subprocess.run([exe], check=True, capture_output=True,
                                                               text=True).stdout.splitlines()]
    assert len(rows) == 64
    for a, b, joins in rows:
        assert joins == (0 <= a <= b < 304), (a, b)
