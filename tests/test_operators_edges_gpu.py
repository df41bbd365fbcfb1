"""The operators around the decode step where they are easiest to get wrong: calls that overlap, values
and gates of very different sizes, widths between the tested ones, and waits that run out.

Tolerances are those of test_operators_gpu.py (derived there) unless a test says otherwise.
"""
import pytest
import torch

from test_operators_gpu import (HALF, TYPES, K, check_backward, check_forward, check_norm, grads, inputs,  # noqa: F401
                                norm_inputs, run_forward)

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
@pytest.mark.parametrize("b", [-14.0, -20.0, -30.0, 8.0, 20.0])
def test_scan_of_betas_near_zero_and_one(K, b, dk, dv, dt):
    """All of a sequence's betas are small, or near 1: nothing larger hides what their rounding loses."""
    lens = [100, 64, 70]
    for state in (False, True):
        x, e = inputs(lens, 2, dk, dv, dt, state=state)
        x["b"] += b
        if not state:
            e["dstate"] = e["dstate"] * 0.01
        check_forward(K, x, e, lens)
        check_backward(K, x, e, lens)


def exponents(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp2(torch.randint(-30, 31, (n,), generator=g, device="cuda").float())


@DTYPES
@pytest.mark.parametrize("lens", [[5, 20], [70, 140]], ids=["tokens", "chunks"])
def test_scan_of_value_columns_of_different_sizes(K, lens, dt):
    """Value columns do not meet: a power of two in one comes out as it went in, to the bit."""
    x, e = inputs(lens, 2, 128, 64, dt)
    c = exponents(64, 1)
    o, S = run_forward(K, x, e, lens)
    y, f = dict(x, v=x["v"] * c.to(dt)), dict(e, state0=e["state0"] * c)
    o2, S2 = run_forward(K, y, f, lens)
    assert torch.equal(o2, o * c.to(dt)) and torch.equal(S2, S * c)
    g = grads(K, x, e, lens)
    g2 = grads(K, x, dict(e, do=e["do"] * c.to(dt), dstate=e["dstate"] * c), lens)
    assert torch.equal(g2["dv"], g["dv"] * c.to(dt)) and torch.equal(g2["dstate0"], g["dstate0"] * c)


@DTYPES
@pytest.mark.parametrize("lens", [[5, 20], [70, 140]], ids=["tokens", "chunks"])
def test_scan_of_queries_of_different_sizes(K, lens, dt):
    """A power of two in a token's query shows in its output only; with the inverse in that output's
    gradient, in the query's gradient only."""
    x, e = inputs(lens, 2, 64, 128, dt)
    c = exponents(sum(lens), 2).to(dt)[:, None, None]
    o, S = run_forward(K, x, e, lens)
    y = dict(x, q=x["q"] * c)
    o2, S2 = run_forward(K, y, e, lens)
    assert torch.equal(o2, o * c) and torch.equal(S2, S)
    g, g2 = grads(K, x, e, lens), grads(K, y, dict(e, do=e["do"] / c), lens)
    assert torch.equal(g2["dq"], g["dq"] / c)
    for m in ("dk", "dv", "dz", "db", "dstate0"):
        assert torch.equal(g[m], g2[m]), m


def same_where_finite(got, want):
    ok = torch.isfinite(got)
    assert torch.equal(got[ok], want[ok])


@DTYPES
@pytest.mark.parametrize("t", [3, 40, 100])
def test_scan_with_one_infinity(K, t, dt):
    """What an infinity does not reach keeps its bits, and what it reaches is not finite: no value in between."""
    lens, nh = [150], 2
    x, e = inputs(lens, nh, 128, 64, dt)
    (o, S), g = run_forward(K, x, e, lens), grads(K, x, e, lens)
    rest = [j for j in range(64) if j != 5]

    y = dict(x, v=x["v"].clone())
    y["v"][t, 0, 5] = float("inf")
    o2, S2 = run_forward(K, y, e, lens)
    assert torch.equal(o2[:, 1], o[:, 1]) and torch.equal(o2[:, 0, rest], o[:, 0, rest])
    assert torch.equal(S2[:, 1], S[:, 1]) and torch.equal(S2[:, 0, :, rest], S[:, 0, :, rest])
    assert not torch.isfinite(o2[t:, 0, 5]).any() and not torch.isfinite(S2[:, 0, :, 5]).any()
    same_where_finite(o2, o)
    for m, got in grads(K, y, e, lens).items():
        same_where_finite(got, g[m])

    y = dict(x, q=x["q"].clone())
    y["q"][t, 0, 5] = float("inf")
    o2, S2 = run_forward(K, y, e, lens)
    others = [i for i in range(150) if i != t]
    assert torch.equal(S2, S) and torch.equal(o2[others], o[others]) and torch.equal(o2[:, 1], o[:, 1])
    assert not torch.isfinite(o2[t, 0]).any()
    for m, got in grads(K, y, e, lens).items():
        same_where_finite(got, g[m])

    do = e["do"].clone()
    do[t, 0, 5] = float("inf")
    g2 = grads(K, x, dict(e, do=do), lens)
    assert torch.equal(g2["dv"][:, 0, rest], g["dv"][:, 0, rest])
    assert torch.equal(g2["dstate0"][:, 0, :, rest], g["dstate0"][:, 0, :, rest])
    assert not torch.isfinite(g2["dstate0"][:, 0, :, 5]).any()
    for m in g:
        assert torch.equal(g2[m][:, 1], g[m][:, 1])
        same_where_finite(g2[m], g[m])


@DTYPES
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_scan_of_a_padded_batch(K, dk, dv, dt):
    """Sequences padded with zeros to one length: the padding's gates halve the state at every token, and
    what is left of it, and the gradient that passes back through it, keep their accuracy."""
    real, T = [24, 1, 40], 84
    lens = [T] * 3
    for only_state in (False, True):
        x, e = inputs(lens, 2, dk, dv, dt)
        for i, n in enumerate(real):
            for m in x:
                x[m][i * T + n:(i + 1) * T] = 0
            e["do"][i * T + n:(i + 1) * T] = 0
        if only_state:
            e["do"].zero_()
        check_forward(K, x, e, lens, ragged=False)
        check_backward(K, x, e, lens, ragged=False)


# ------------------------------------------------------------------ the residual norm

WIDTHS = [2176, 4096, 4224, 6144, 6272, 8192]   # two, three and four 16-byte pieces to a thread, whole and part-filled


@pytest.mark.parametrize("xdt,rdt", TYPES)
@pytest.mark.parametrize("hidden", WIDTHS)
def test_residual_norm_of_many_wide_rows(K, hidden, xdt, rdt):
    x, r, w = norm_inputs(600, hidden, xdt, rdt)
    check_norm(K, x, r, w)
    check_norm(K, x, None, w)


@pytest.mark.parametrize("rdt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_residual_norm_gradient_of_many_wide_rows(K, hidden, rdt):
    from test_operators_gpu import test_residual_norm_gradient as one
    for with_dres in (True, False):
        one(K, 700, hidden, rdt, with_dres)


@pytest.mark.parametrize("whole", [True, False], ids=["ties", "sizes"])
def test_residual_norm_codes_are_those_of_the_division(K, whole):
    """y8 is E4M3(y / scale), scale max |y| / 448, both divisions rounded once: the codes of torch's division
    of the same fp32 numbers, at ties and at groups of any size."""
    g = torch.Generator(device="cuda").manual_seed(11)
    rows, hidden = 3000, 1024
    if whole:    # whole numbers up to the largest code: every second quotient is a code or a tie of two
        r = torch.randint(-448, 449, (rows, hidden), generator=g, device="cuda").float()
        r[:, ::128] = 448.0
    else:
        r = torch.randn(rows, hidden // 128, 128, generator=g, device="cuda")
        r = (r * torch.exp2(torch.randint(-120, 30, (rows, hidden // 128, 1), generator=g, device="cuda").float())).view(rows, hidden)
    got = K.residual_norm(r, None, torch.ones(hidden, device="cuda", dtype=torch.bfloat16), fp8=True)
    y = (r * got.rstd[:, None]).view(rows, hidden // 128, 128)
    m = y.abs().amax(-1)     # (by a tensor: torch multiplies by the inverse of a number)
    scale = torch.where(m > 0, (m / torch.full_like(m, 448.0)).clamp_min(2.0 ** -126), torch.ones_like(m))
    assert torch.equal(got.scale, scale)
    want = (y / scale[..., None]).to(torch.float8_e4m3fn).view(rows, hidden)
    assert torch.equal(got.y8.view(torch.uint8), want.view(torch.uint8))


# ------------------------------------------------------------------ calls

def test_a_call_that_loses_a_gradient_says_so(K):
    """Inputs that require a gradient give detached outputs: with a warning, but not inside an
    autograd.Function or under no_grad, where the gradient is the caller's."""
    import warnings
    x, e = inputs([40], 2, 64, 64, torch.float32)
    h, r, w = norm_inputs(4, 256, torch.float32, torch.float32)
    w = torch.nn.Parameter(w)
    x["v"].requires_grad_()
    with pytest.warns(UserWarning, match="scan_forward records no graph"):
        o, _ = run_forward(K, x, e, [40])
    assert not o.requires_grad
    with pytest.warns(UserWarning, match="residual_norm records no graph"):
        K.residual_norm(h, r, w)

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, h, r, w):
            f = K.residual_norm(h, r, w)
            ctx.save_for_backward(f.residual, w, f.rstd)
            return f.y

        @staticmethod
        def backward(ctx, dy):
            residual, w, rstd = ctx.saved_tensors
            dr, dw = K.residual_norm_backward(dy.contiguous(), residual, w, rstd)
            return dr, dr, dw.to(w.dtype)

    with warnings.catch_warnings():
        warnings.simplefilter("error")
        Norm.apply(h, r, w).float().sum().backward()
        with torch.no_grad():
            run_forward(K, x, e, [40])
            K.residual_norm(h, r, w)
    rr, ww = (h + r).double(), w.detach().double().requires_grad_()
    y = rr / torch.sqrt((rr * rr).mean(1, keepdim=True) + 1e-6) * ww
    c, = torch.autograd.grad(y.sum(), ww)
    # a bf16 gradient of sums over 4 rows (the tolerances of test_residual_norm_gradient)
    assert ((w.grad.double() - c).abs() <= HALF[torch.bfloat16] * c.abs() + 2.0 ** -17 * max(1.0, float(c.abs().max()))).all()


def test_arguments_of_another_kind(K):
    """What is no tensor is refused by name; bytes are numbers of rows, not their memory."""
    x, e = inputs([20, 20], 2, 64, 64, torch.float32)
    for over, text in ((dict(cu_seqlens=[0, 20, 40]), "cu_seqlens must be a CUDA"), (dict(cu_seqlens=e["cu"].cpu()), "cu_seqlens must be a CUDA"),
                       (dict(cu_seqlens=e["cu"][0]), "cu_seqlens must be int32"), (dict(cu_seqlens=e["cu"][:1]), "cu_seqlens must be int32"),
                       (dict(state0=[0.0]), "state0 must be a CUDA"), (dict(state0=e["state0"].sum()), "state0 must have"),
                       (dict(nseq=0), "give cu_seqlens"), (dict(nseq=-1), "give cu_seqlens")):
        with pytest.raises(ValueError, match=text):
            K.scan_forward(*(x[m] for m in "qkvzb"), **over)
    pool = torch.arange(8.0, device="cuda")[:, None].repeat(1, 4)
    want = pool.clone()
    want[0], want[5] = pool[2], pool[1]
    K.state_rows(pool, bytes([2, 1]), bytearray([0, 5]))
    assert torch.equal(pool, want)
    K.state_rows(pool, torch.tensor([3]), torch.tensor([4]))   # whatever yields whole numbers
    assert (pool[4] == 3).all()


FIRST_CALLS = r"""
import torch
from linear_attention_layer_kda_b200 import operators as K
from test_operators_gpu import grads, inputs, norm_inputs, run_forward

made = []
for lens, ragged in (([70, 200, 1], True), ([70, 70], False), ([1, 1], False)):
    x, e = inputs(lens, 2, 64, 64, torch.bfloat16)
    made.append((x, e, lens, ragged))
h, r, w = norm_inputs(4, 256, torch.float32, torch.float32)
dy = h.bfloat16()
pool = torch.arange(8.0, device="cuda")[:, None].repeat(1, 4)
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    got = [(run_forward(K, x, e, lens, ragged), grads(K, x, e, lens, ragged)) for x, e, lens, ragged in made]
    f = K.residual_norm(h, r, w, fp8=True)
    d = K.residual_norm_backward(dy, f.residual, w, f.rstd)
    K.state_rows(pool, [1, 0, -1], [0, 1, 5])
gr.replay()
torch.cuda.synchronize()
for (x, e, lens, ragged), ((o, S), g) in zip(made, got):
    o2, S2 = run_forward(K, x, e, lens, ragged)
    g2 = grads(K, x, e, lens, ragged)
    assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(g[m], g2[m]) for m in g)
f2 = K.residual_norm(h, r, w, fp8=True)
assert all(torch.equal(a.float(), c.float()) for a, c in zip(f, f2))
assert all(torch.equal(a, c) for a, c in zip(d, K.residual_norm_backward(dy, f2.residual, w, f2.rstd)))
assert pool[:, 0].tolist() == [1, 0, 2, 3, 4, 0, 6, 7]
print("CAPTURED")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """Every call can be captured, the first ones of a process included (kernels are loaded on the way)."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ)
    env["PYTHONPATH"] = os.pathsep.join([root, os.path.join(root, "tests")] +
                                        ([env["PYTHONPATH"]] if env.get("PYTHONPATH") else []))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "CAPTURED" in r.stdout, (r.stdout + r.stderr)[-4000:]


def test_calls_from_two_threads(K):
    """Threads with streams of their own share nothing."""
    import threading
    lens = [70, 3, 130]
    work = [inputs(lens, 2, 64, 128, dt, seed=s) for s, dt in enumerate((torch.float32, torch.bfloat16))]
    want = [(run_forward(K, x, e, lens), grads(K, x, e, lens)) for x, e in work]
    torch.cuda.synchronize()
    failed = []

    def run(i):
        try:
            x, e = work[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    (o, S), g = run_forward(K, x, e, lens), grads(K, x, e, lens)
                    torch.cuda.current_stream().synchronize()
                    (o2, S2), g2 = want[i]
                    assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(g[m], g2[m]) for m in g)
        except BaseException as ex:  # noqa: BLE001
            failed.append(ex)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
