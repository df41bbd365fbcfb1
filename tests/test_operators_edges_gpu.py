"""The operators around the decode step where they are easiest to get wrong: calls that overlap, values
and gates of very different sizes, widths between the tested ones, and waits that run out.

Tolerances are those of test_operators_gpu.py (derived there) unless a test says otherwise.
"""
import pytest
import torch

from test_operators_gpu import K, check_backward, check_forward, grads, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,nh", [([500, 40, 64], 2), ([200] * 9, 16)], ids=["one_group", "two_groups"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64)])
def test_fp32_gradients_on_streams_at_once(K, dk, dv, lens, nh):
    """fp32 keeps the gradient of the states where (g q)^T do was: with the memory busy from other streams,
    every call still gives the bits of a call that had the GPU for itself."""
    work = [inputs(lens, nh, dk, dv, torch.float32, seed=s) for s in range(4)]
    want = [grads(K, x, e, lens) for x, e in work]
    check_backward(K, *work[0], lens)
    big = [torch.empty(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in work]
    traffic = torch.cuda.Stream()
    for _ in range(6):
        torch.cuda.synchronize()
        with torch.cuda.stream(traffic):
            for _ in range(8):
                big[0].copy_(big[1])
        got = []
        for st, (x, e) in zip(streams, work):
            with torch.cuda.stream(st):
                got.append([grads(K, x, e, lens) for _ in range(3)])
        torch.cuda.synchronize()
        for w, gs in zip(want, got):
            for g in gs:
                assert all(torch.equal(w[m], g[m]) for m in w)


# ------------------------------------------------------------------ gates and values of very different sizes

DTYPES = pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])


@DTYPES
@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 128)])
@pytest.mark.parametrize("b", [-14.0, -20.0, -30.0])
def test_scan_of_small_betas(K, b, dk, dv, dt):
    """All of a sequence's betas are small: nothing larger hides what their rounding loses."""
    lens = [100, 64, 70]
    for state in (False, True):
        x, e = inputs(lens, 2, dk, dv, dt, state=state)
        x["b"] += b
        if not state:
            e["dstate"] = e["dstate"] * 0.01
        check_forward(K, x, e, lens)
        check_backward(K, x, e, lens)
