"""What a given-up wait of the newer attention kernels must not do, as tests/test_attn_give_up.py holds it for the
first one: wait without a limit, end the block under copies or products in flight, or leave parts that the join
reads unwritten. A wait that runs out needs a copy or a product that never ends, which no call can make, so the
rules are held to the source, and the shared kernel's split of its work to a plain restatement."""
import os
import random
import re

import pytest

from state_cached_causal_gb300 import build as cbuild


def source(name):
    with open(os.path.join(cbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body_of(text, start):
    at = text.index("{", text.index(start))
    depth, i = 0, at
    while True:
        depth += (text[i] == "{") - (text[i] == "}")
        i += 1
        if depth == 0:
            return text[at:i]


def test_the_8_bit_kernel():
    text = source("attn_mma_q8.cu")
    body = body_of(text, "attn_mma_q8_kernel(const AttnArgs a")
    behind = body[body.index("attn_split<"):].split("\n", 1)[1]
    assert "__syncthreads" not in behind and "bar.sync" not in behind
    assert text.count("mbar_try(") == 1                               # the one in wait_bar
    assert behind.count("return;") == 2, "the usual ends of the copying warp and of the scales' one"
    given_up = re.findall(r"if \([^;]*!(wait_bar|meet)\([^;]*?\)\)\s*return settle\(full, stages, (\w+), (\w+),", behind)
    assert given_up == 2 * [("wait_bar", "st", "ph")] + [("wait_bar", "stage", "phase")] + 3 * [
        ("meet", "stage", "phase")]
    assert len(re.findall(r"\b(?:wait_bar|meet)\(", behind)) == len(given_up) + 1      # (and meet's own wait)
    settle = re.search(r"void settle\([^)]*\) \{(.*?)\n\}", text, re.S).group(1)
    assert re.search(r"for \(int i = 0; i < stages; \+\+i\) wait_bar\(&full\[i\], i < st \? ph \^ 1 : ph, err\);", settle)


def test_the_shared_kernel():
    text = source("attn_shared.cu")
    body = body_of(text, "attn_prefix_kernel(const PrefixArgs x")
    roles = body[body.index("const Wait wait"):]
    # two waits in all: Wait, which has a limit, and that for the last products, which has one too
    assert text.count("mbar_try(") == 2 and "kWaitClocks" in roles
    for role in ("copy_role(", "mma_role(", "soft_role("):
        inside = body_of(text, role)
        assert "__syncthreads" not in inside and "bar.sync" not in inside and "mbar_try" not in inside
        for call in re.findall(r"(\S*)\s*\bwait\(&c", inside):
            assert call in ("(!", "return", "&&", "if", "!"), call
    # copies in flight and products issued have ended, or run out of their limit, before tensor memory goes
    assert roles.index("cp.async.wait_all") < roles.index("tc::commit(&c.fin)") < roles.index("__syncthreads()") \
        < roles.index("tcgen05.dealloc")
    # every segment of a stream ends with its part's statistics, given up or not
    soft = body_of(text, "soft_role(")
    assert soft.count("empty_part<D>(x, s, stream);") == 2 and soft.count("x.ps[row0 + lane] =") == 1


def split(groups, hkv, streams, grid, K, pair):
    """(rows of a kv head, tiles) of each group -> the tiles that each block takes, and their parts' places."""
    R, unit, base, info = 128 * streams, 0, 0, []
    for rows, tiles in groups:
        blocks = -(-rows // R)
        units = blocks * hkv if tiles > 0 else 0
        full = units - hkv if streams == 2 and units > 0 else 0
        wide = pair if streams == 2 and rows - (blocks - 1) * R > 128 else 1
        per, per_full = wide * tiles + K, pair * tiles + K
        info.append((base, unit, units, full, wide, per, per_full, tiles))
        base += full * per_full + (units - full) * per
        unit += units
    total, runs = base, min(grid, base // 2)
    taken, places = {}, set()
    for block in range(runs):
        p, end, g = block * total // runs, (block + 1) * total // runs, 0
        while p < end:
            while g + 1 < len(info) and p >= info[g + 1][0]:
                g += 1
            b, u0, units, full, wide, per, per_full, tiles = info[g]
            rel = p - b
            whole = rel < full * per_full
            rel -= 0 if whole else full * per_full
            one, w = (per_full, pair) if whole else (per, wide)
            u, off = rel // one, rel % one
            take = min(one - off, end - p)
            p += take
            j0, j1 = (max(x - K + w - 1, 0) >> (w - 1) for x in (off, off + take))
            if j1 <= j0:
                continue
            u += 0 if whole else full
            assert u0 + u + block not in places, "two parts in one place"
            places.add(u0 + u + block)
            assert u0 + u + block < unit + runs
            first = b + K + (u * per_full if u < full else full * per_full + (u - full) * per)
            for j in range(j0, j1):
                assert j < tiles and (g, u, j) not in taken
                taken[g, u, j] = block
                assert ((first + j * w + 1) * runs - 1) // total == block, "the join looks elsewhere"
    return taken, info


@pytest.mark.parametrize("streams,start,pair", [(1, 8, 2), (2, 8, 2), (2, 3, 1)])
def test_every_tile_of_a_prefix_is_taken_once(streams, start, pair):
    """And the parts of a unit are those of neighbouring blocks, each of which has tiles of it."""
    r = random.Random(streams + start)
    for _ in range(1500):
        groups = [(r.choice([0, 1, 4, 100, 128, 129, 256, 257, 600, 1000]), r.choice([0, 0, 1, 2, 3, 8, 30, 200]))
                  for _ in range(r.randint(1, 9))]
        taken, info = split(groups, r.choice([1, 2, 4]), streams, r.choice([3, 10, 152]), start, pair)
        assert len(taken) == sum(i[2] * i[7] for i in info)
        for g, i in enumerate(info):
            for u in range(i[2]):
                blocks = sorted({taken[g, u, j] for j in range(i[7])})
                assert blocks == list(range(blocks[0], blocks[-1] + 1))
