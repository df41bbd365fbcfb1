"""Waits of the recurrence's kernels that run out, without a GPU fault.

The kernels bound every wait for their copies (KDA_WAIT_LIMIT_MS).  With KDA_DEBUG_SKIP_SCAN_COPIES
set before the library's first scan, the copies are not made, so every wait runs out: the kernels
return, everything that depends on the copies is NaN, and the context stays usable.  The calls run
in a child process, so that the switches stay there.
"""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

CHILD = r"""
import torch
from linear_attention_layer_kda_b200 import operators as K
from test_operators_gpu import grads, inputs, norm_inputs, run_forward

# one group of four warps; two groups; one warp to 16 columns
for lens, nh, ragged in (([70, 200], 2, True), ([40] * 6, 16, True), ([70] * 6, 16, False)):
    for dk, dv in ((128, 128), (64, 128)):
        for dt in (torch.float32, torch.bfloat16):
            x, e = inputs(lens, nh, dk, dv, dt)
            o, S = run_forward(K, x, e, lens, ragged)
            g = grads(K, x, e, lens, ragged)
            torch.cuda.synchronize()
            bad = [m for m, t in dict(g, o=o, state=S).items() if not torch.isnan(t).all()]
            print("WAITED", bad)
x, r, w = norm_inputs(4, 256, torch.float32, torch.float32)
print("USABLE", bool(torch.isfinite(K.residual_norm(x, r, w).y).all()))
lens = [1, 5, 0, 20]   # token by token: no copies
x, e = inputs(lens, 2, 64, 64, torch.float32)
print("TOKENS", bool(torch.isfinite(run_forward(K, x, e, lens)[0]).all()))
"""


def run(**env):
    env = dict(os.environ, **env)
    env["PYTHONPATH"] = os.pathsep.join([ROOT, os.path.join(ROOT, "tests")] +
                                        ([env["PYTHONPATH"]] if env.get("PYTHONPATH") else []))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    return r.stdout.splitlines()


def test_waits_that_run_out_make_everything_nan():
    lines = run(KDA_WAIT_LIMIT_MS="2", KDA_DEBUG_SKIP_SCAN_COPIES="1")
    assert [x for x in lines if x.startswith("WAITED")] == ["WAITED []"] * 12, lines
    assert "USABLE True" in lines and "TOKENS True" in lines


def test_a_short_limit_does_not_matter_while_the_copies_arrive():
    lines = run(KDA_WAIT_LIMIT_MS="500")
    waited = [x for x in lines if x.startswith("WAITED")]
    assert len(waited) == 12 and not any(x == "WAITED []" for x in waited)
