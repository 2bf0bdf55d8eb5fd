"""The example that serves both mixers together, against the plain 64-bit forms of their inputs."""
import importlib.util
import os

import pytest
import torch

from _mixers import assert_close, attn_ref, gdn_ref, norm_rope_ref

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                     "hybrid_step.py")


@pytest.fixture(scope="module")
def hybrid():
    spec = importlib.util.spec_from_file_location("hybrid_step", _PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_paths_agree(hybrid, capsys):
    hybrid.main()
    assert "ok" in capsys.readouterr().out


def test_against_plain_forms(hybrid):
    lens = [9, 70, 1, 130]
    m, prompt, step = hybrid.serve(lens, 1)
    d64 = lambda ts: [t.double().cpu() for t in ts]  # noqa: E731
    A, dt = m.A_log.double().cpu(), m.dt_bias.double().cpu()
    pin, sin = d64(prompt["delta_in"]), d64(step["delta_in"])
    scale, at = hybrid.DIM ** -0.5, 0
    states = []
    for r, n in enumerate(lens):
        S = torch.zeros(m.states.shape[1:], dtype=torch.float64)
        out, st = gdn_ref(*[t[at:at + n] for t in pin], A, dt, S, scale)
        assert_close(prompt["delta"][at:at + n], out, f"prompt {r}")
        out, st = gdn_ref(*[t[r:r + 1] for t in sin], A, dt, st[-1], scale)
        assert_close(step["delta"][r:r + 1], out, f"token {r}")
        states.append(st[-1])
        at += n
    assert_close(m.states, torch.stack(states), "states")
    cs = m.cos_sin.cpu()
    for got, heads, pos in ((prompt["q"], prompt["heads"], prompt["positions"].tolist()),
                            (step["q"], step["heads"], lens)):
        want = norm_rope_ref(heads[0].cpu(), m.q_norm.cpu(), hybrid.EPS, cs, pos, False)
        assert_close(got, want, "queries")
    want, _ = attn_ref(step["q"].cpu(), m.k_cache.cpu(), m.v_cache.cpu(), m.table.cpu(),
                       [n + 1 for n in lens], 1, scale)
    assert_close(step["attn"], want, "attention")
    assert int(m.err) == 0
