"""The operators around the decode step (operators.py) against their definitions in fp64.

Tolerances.  A product of fp32 values over K terms is off by at most about K 2^-24 of the sum of
its terms' sizes; with K <= 128 and errors of random sign that is about sqrt(128) 2^-24 < 2^-20 of
the largest result.  A chunk of 64 tokens puts some eight products one behind another (2^-17), and
a state passes through one chunk after another by a map of norm <= 1, so that the chunks' errors
add up, again with random signs: 2^-17 sqrt(chunks), relative to the head's largest value.  The
backward pass runs the forward's products first and adds as many: twice that.  dz is a sum over
the tokens of a chunk of differences of terms that may be 8 times the sum: eight times that.  A
bf16 result is off by another half step, 2^-8 of itself.
"""
import math
import random

import pytest
import torch

import scan_ref as R

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def K():
    from linear_attention_layer_kda_b200 import operators
    return operators


def inputs(lens, nh, dk, dv, dt, seed=1, zmean=-2.0, zscale=1.0, state=True, pad=0, first=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = first + sum(lens) + pad

    def r(*s, scale=1.0, mean=0.0):
        return torch.randn(*s, generator=g, device="cuda") * scale + mean
    x = dict(q=r(n, nh, dk), k=r(n, nh, dk), v=r(n, nh, dv), z=r(n, nh, dk, scale=zscale, mean=zmean), b=r(n, nh))
    x = {m: t.to(dt) for m, t in x.items()}
    cu = [first]
    for m in lens:
        cu.append(cu[-1] + m)
    extra = dict(state0=r(len(lens), nh, dk, dv, scale=0.1) if state else None,
                 cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                 do=r(n, nh, dv).to(dt), dstate=r(len(lens), nh, dk, dv, scale=0.1))
    return x, extra


def close(got, ref, tol, what, dims=None):
    """|got - ref| <= tol * (largest |ref| of the head) + half a step of got's type."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    g, head = got.double(), 1 if dims is None else dims
    assert torch.isfinite(g).all(), what
    d = [i for i in range(ref.dim()) if i != head]
    size = ref.abs().amax(d, keepdim=True)
    over = (g - ref).abs() - tol * size - HALF[got.dtype] * ref.abs()
    worst = ((g - ref).abs() / size.clamp_min(1e-300)).max()
    assert (over <= 0).all(), f"{what}: error {float(worst):.2e} of the head's largest, allowed {tol:.2e}"


def tol_forward(lens):
    return 2.0 ** -17 * math.sqrt(max(1, -(-max(lens) // 64)))


def run_forward(K, x, e, lens, ragged=True, **kw):
    return K.scan_forward(x["q"], x["k"], x["v"], x["z"], x["b"], state0=e["state0"],
                          cu_seqlens=e["cu"] if ragged else None, nseq=len(lens), **kw)


def check_forward(K, x, e, lens, ragged=True, first=0):
    o, S = run_forward(K, x, e, lens, ragged)
    ro, rS = R.scan(x["q"], x["k"], x["v"], x["z"], x["b"], lens, e["state0"], first)
    t = tol_forward(lens)
    close(o[first:first + sum(lens)], ro, t, "o")
    close(S, rS, t, "state")


SHAPES = [(64, 64), (64, 128), (128, 64), (128, 128)]
LENS = [[1], [2], [16], [17], [63], [64], [65], [200], [1, 0, 63, 64, 65, 5], [0, 0, 3], [129, 15, 16, 48, 33, 31]]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_scan_matches_the_recurrence(K, dk, dv, dt):
    for i, lens in enumerate(LENS):
        x, e = inputs(lens, 3, dk, dv, dt, seed=i, state=i % 3 != 0)
        check_forward(K, x, e, lens)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("nseq,T", [(1, 1), (7, 1), (3, 16), (2, 17), (3, 64), (2, 300), (300, 1)])
def test_scan_of_equal_lengths(K, nseq, T, dt):
    x, e = inputs([T] * nseq, 2, 128, 64, dt, seed=nseq)
    check_forward(K, x, e, [T] * nseq, ragged=False)


def test_scan_of_long_sequences_among_short_ones(K):
    """Those of up to 32 tokens go token by token, the others by chunks, in any order and number."""
    rng = random.Random(8)
    for dt in (torch.float32, torch.bfloat16):
        for n, long in ((1, 33), (40, 33), (1500, 200)):
            lens = [rng.choice([0, 1, 2, 31, 32]) if rng.random() < 0.9 else rng.randint(33, long) for _ in range(n)] + [33, 1]
            x, e = inputs(lens, 1, 64, 64, dt, seed=n)
            check_forward(K, x, e, lens)
    lens = [1] * 400 + [90] + [0] * 700 + [34]
    x, e = inputs(lens, 2, 128, 128, torch.bfloat16)
    check_forward(K, x, e, lens)
    check_backward(K, x, e, lens)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_scan_of_many_heads(K, dk, dv, dt):
    """Enough heads and sequences for the forms of the pass over the chunks that large batches take."""
    lens = [65, 130, 0, 7]
    x, e = inputs(lens, 40, dk, dv, dt, seed=6)
    check_forward(K, x, e, lens)
    check_backward(K, x, e, lens)
    lens = [70] * 3
    x, e = inputs(lens, 40, dk, dv, dt, seed=7)
    check_forward(K, x, e, lens, ragged=False)
    check_backward(K, x, e, lens, ragged=False)


@pytest.mark.parametrize("dk,dv,dt", [(64, 64, torch.float32), (128, 128, torch.bfloat16)], ids=["fp32", "bf16"])
def test_scan_of_many_heads_and_lengths(K, dk, dv, dt):
    rng = random.Random(dk)
    lens = [rng.choice([0, 1, 33, 64, 65, rng.randint(33, 130)]) for _ in range(40)]
    x, e = inputs(lens, 32, dk, dv, dt, seed=dk)
    check_forward(K, x, e, lens)
    check_backward(K, x, e, lens)


def test_scan_of_a_long_sequence(K):
    x, e = inputs([1500], 2, 128, 128, torch.float32, zmean=-6.0)
    check_forward(K, x, e, [1500])


def test_scan_of_many_short_sequences(K):
    rng = random.Random(3)
    lens = [rng.choice([0, 1, 1, 2, 3]) for _ in range(1300)]
    x, e = inputs(lens, 1, 64, 64, torch.bfloat16)
    check_forward(K, x, e, lens)
    lens = [rng.choice([0, 1, 5, 20, 70]) for _ in range(1100)]
    x, e = inputs(lens, 1, 64, 64, torch.float32)
    check_forward(K, x, e, lens)


def extreme(x, lens):
    """Zero keys, tiny and huge keys, gates open and shut, in every position of a chunk."""
    n = x["q"].shape[0]
    x["k"][::7] = 0
    x["k"][1::11] *= 1e-12
    x["k"][2::13] *= 1e12
    x["b"][::5] = 30.0
    x["b"][1::5] = -200.0
    x["z"][3::17] = 200.0
    x["z"][4::19] = -200.0
    x["z"][5::23, :, ::2] = 25.0
    assert n > 23


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("zmean,zscale", [(30.0, 1.0), (0.0, 15.0), (8.0, 1.0), (-20.0, 1.0)])
def test_scan_with_strong_and_weak_decay(K, zmean, zscale, dt):
    lens = [100, 70]
    x, e = inputs(lens, 2, 128, 64, dt, zmean=zmean, zscale=zscale)
    check_forward(K, x, e, lens)
    check_backward(K, x, e, lens)
    x, e = inputs(lens, 2, 64, 128, dt)
    extreme(x, lens)
    check_forward(K, x, e, lens)
    check_backward(K, x, e, lens)


def grads(K, x, e, lens, ragged=True, dstate=True):
    return K.scan_backward(x["q"], x["k"], x["v"], x["z"], x["b"], e["do"], dstate=e["dstate"] if dstate else None,
                           state0=e["state0"], cu_seqlens=e["cu"] if ragged else None, nseq=len(lens))


def check_backward(K, x, e, lens, ragged=True, first=0, dstate=True):
    got = grads(K, x, e, lens, ragged, dstate)
    ref = R.scan_grads(x["q"], x["k"], x["v"], x["z"], x["b"], lens, e["do"], e["dstate"] if dstate else None,
                       e["state0"], first)
    assert got.keys() == ref.keys()
    t = 2 * tol_forward(lens)
    for m in ref:
        if m == "dk":  # in units of 1 / |k|, which scales a row's gradient
            size = x["k"].double().norm(dim=-1, keepdim=True)
            close((got[m].double() * size).to(torch.float32) if got[m].dtype == torch.float32
                  else (got[m].double() * size).float().to(got[m].dtype), ref[m] * size, t + 2 * HALF[got[m].dtype], m)
        else:
            close(got[m], ref[m], 8 * t if m == "dz" else t, m)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("dk,dv", SHAPES)
def test_scan_gradients(K, dk, dv, dt):
    for i, lens in enumerate(LENS):
        x, e = inputs(lens, 2, dk, dv, dt, seed=20 + i, state=i % 3 != 1)
        check_backward(K, x, e, lens, dstate=i % 2 == 0)


@pytest.mark.parametrize("nseq,T", [(2, 1), (3, 64), (2, 130)])
def test_scan_gradients_of_equal_lengths(K, nseq, T):
    x, e = inputs([T] * nseq, 2, 128, 128, torch.float32, seed=T)
    check_backward(K, x, e, [T] * nseq, ragged=False)


def test_scan_gradients_of_a_long_sequence(K):
    x, e = inputs([900], 2, 64, 64, torch.float32, zmean=-6.0)
    check_backward(K, x, e, [900])


@pytest.mark.parametrize("name", ["q", "k", "v", "z", "b", "state0"])
def test_scan_gradients_against_differences(K, name):
    """(f(x + h d) - f(x - h d)) / 2h of the fp64 recurrence, h = 1e-5 (its own error is about h^2
    = 1e-10), against the kernel's gradient along d: a sum over N entries each off by the
    gradient's tolerance with random sign."""
    lens = [70, 20]
    x, e = inputs(lens, 2, 64, 64, torch.float32, seed=77)
    got = grads(K, x, e, lens)["d" + name].double()
    base = {m: t.double() for m, t in x.items()}
    s0 = e["state0"].double()
    d = torch.randn(got.shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda", dtype=torch.float64)

    def f(h):
        y = dict(base)
        s = s0
        if name == "state0":
            s = s0 + h * d
        else:
            y[name] = base[name] + h * d
        o, S = R.scan(y["q"], y["k"], y["v"], y["z"], y["b"], lens, s)
        return ((o * e["do"].double()).sum() + (S * e["dstate"].double()).sum()).item()
    h = 1e-5
    want = (f(h) - f(-h)) / (2 * h)
    t = 16 * tol_forward(lens) * float(got.abs().max()) * math.sqrt(d.numel()) + 1e-6 * abs(want)
    assert abs(float((got * d).sum()) - want) <= t


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_scan_leaves_rows_of_no_sequence(K, dt):
    for lens in ([70, 3], [1, 1, 0, 1]):
        x, e = inputs(lens, 2, 64, 128, dt, pad=9, first=5)
        for m in x:  # nothing of them is read into a result
            x[m][:5] = float("nan")
            x[m][5 + sum(lens):] = float("inf")
        e["do"][:5] = float("nan")
        e["do"][5 + sum(lens):] = float("nan")
        out = torch.full_like(x["v"], 7.0)
        o, _ = run_forward(K, x, e, lens, out=out)
        assert o is out and (out[:5] == 7).all() and (out[5 + sum(lens):] == 7).all()
        check_forward(K, x, e, lens, first=5)
        got = grads(K, x, e, lens)
        for m in "qkvzb":
            g = got["d" + m]
            assert (g[:5] == 0).all() and (g[5 + sum(lens):] == 0).all()
            x[m][:5] = 0
            x[m][5 + sum(lens):] = 0
        e["do"][:5] = 0
        e["do"][5 + sum(lens):] = 0
        check_backward(K, x, e, lens, first=5)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T", [3, 90])
def test_scan_of_columns_of_one_projection(K, T, dt):
    nh, dk, dv = 2, 64, 128
    lens = [T, T]
    x, e = inputs(lens, nh, dk, dv, dt)
    wide = torch.full((2 * T, nh * (3 * dk + dv) + 8), float("nan"), dtype=dt, device="cuda")
    view, at = {}, 0
    for m, w in (("q", dk), ("k", dk), ("v", dv), ("z", dk)):
        view[m] = wide[:, at:at + nh * w].view(2 * T, nh, w)
        view[m].copy_(x[m])
        at += nh * w
    view["b"] = wide[:, at + 1:at + 1 + nh]  # odd offset
    view["b"].copy_(x["b"])
    for a, c in zip(run_forward(K, x, e, lens), run_forward(K, view, e, lens)):
        assert torch.equal(a, c)
    a, c = grads(K, x, e, lens), grads(K, view, e, lens)
    assert all(torch.equal(a[m], c[m]) for m in a)


@pytest.mark.parametrize("T", [20, 130])
def test_scan_of_rows_past_32_bits(K, T):
    """Rows 2^24 elements apart, so that the last ones start behind element 2^31."""
    nh, dk, dv, dt = 2, 64, 128, torch.bfloat16
    gap = 1 << 24 if T > 100 else 1 << 27
    wide = torch.empty(T, gap, dtype=dt, device="cuda")
    x, e = inputs([T], nh, dk, dv, dt)
    view, at = {}, 0
    for m, w in (("q", dk), ("k", dk), ("v", dv), ("z", dk)):
        view[m] = wide[:, at:at + nh * w].unflatten(1, (nh, w))
        at += nh * w
    view["b"] = wide[:, at:at + nh]
    for m in view:
        view[m].copy_(x[m])
    assert (T - 1) * gap > 2 ** 31
    for a, c in zip(run_forward(K, x, e, [T]), run_forward(K, view, e, [T])):
        assert torch.equal(a, c)
    a, c = grads(K, x, e, [T]), grads(K, view, e, [T])
    assert all(torch.equal(a[m], c[m]) for m in a)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("lens", [[5, 20], [70, 140]], ids=["tokens", "chunks"])
def test_scan_of_any_size_of_values(K, lens, dt):
    """Powers of two in v and the states, q, k and the gradients come out as they went in, to the bit."""
    x, e = inputs(lens, 2, 128, 64, dt)
    o, S = run_forward(K, x, e, lens)
    g = grads(K, x, e, lens)
    y, f = dict(x), dict(e)
    y["v"], f["state0"] = x["v"] * 2.0 ** -60, e["state0"] * 2.0 ** -60
    y["q"], y["k"] = x["q"] * 2.0 ** 20, x["k"] * 2.0 ** -30
    o2, S2 = run_forward(K, y, f, lens)
    assert torch.equal(o2.float(), o.float() * 2.0 ** -40) and torch.equal(S2, S * 2.0 ** -60)
    y, f = dict(x), dict(e)
    f["do"], f["dstate"] = e["do"] * 2.0 ** -40, e["dstate"] * 2.0 ** -40
    g2 = grads(K, y, f, lens)
    for m in g:
        assert torch.equal(g2[m].float(), g[m].float() * 2.0 ** -40), m


def test_scan_same_call_same_bits(K):
    lens = [300, 1, 90]
    x, e = inputs(lens, 4, 128, 128, torch.float32)
    o, S = run_forward(K, x, e, lens)
    g = grads(K, x, e, lens)
    for _ in range(5):
        o2, S2 = run_forward(K, x, e, lens)
        assert torch.equal(o, o2) and torch.equal(S, S2)
        g2 = grads(K, x, e, lens)
        assert all(torch.equal(g[m], g2[m]) for m in g)


@pytest.mark.parametrize("T", [1, 5, 70])
def test_scan_state_in_place(K, T):
    lens = [T, T, T]
    x, e = inputs(lens, 2, 128, 64, torch.bfloat16)
    o, S = run_forward(K, x, e, lens, ragged=False)
    s = e["state0"]
    o2, S2 = run_forward(K, x, e, lens, ragged=False, state_out=s)
    assert S2 is s and torch.equal(S, s) and torch.equal(o, o2)


def test_scan_split_over_calls(K):
    """A prompt, then its continuation token by token, through the state."""
    lens = [150]
    x, e = inputs(lens, 2, 128, 128, torch.float32)
    _, S = run_forward(K, x, e, lens)
    s = e["state0"]
    for a, c in ((0, 100), (100, 133)) + tuple((t, t + 1) for t in range(133, 150)):
        _, s = K.scan_forward(*(x[m][a:c] for m in "qkvzb"), state0=s)
    close(s, S.double(), 2 * tol_forward(lens), "state")


def test_scan_captured_and_replayed(K):
    """Two graphs of different shapes, replayed in turn and with new inputs, equal eager calls."""
    made = []
    for lens, dt in (([130, 7], torch.bfloat16), ([33, 64, 2], torch.float32)):
        x, e = inputs(lens, 2, 64, 64, dt)
        run_forward(K, x, e, lens), grads(K, x, e, lens)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o, S = run_forward(K, x, e, lens)
            d = grads(K, x, e, lens)
        made.append((x, e, lens, gr, o, S, d))
    for seed in (31, 32, 33):
        for x, e, lens, gr, o, S, d in made:
            y, f = inputs(lens, 2, 64, 64, x["q"].dtype, seed=seed)
            for m in x:
                x[m].copy_(y[m])
            for m in ("state0", "do", "dstate"):
                e[m].copy_(f[m])
        for _, _, _, gr, *_ in made:
            gr.replay()
        for x, e, lens, gr, o, S, d in made:
            o2, S2 = run_forward(K, x, e, lens)
            d2 = grads(K, x, e, lens)
            assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(d[m], d2[m]) for m in d)


def test_scan_on_two_streams_at_once(K):
    lens = [500, 40]
    work = [inputs(lens, 4, 128, 128, torch.bfloat16, seed=s) for s in range(4)]
    want = [(run_forward(K, x, e, lens), grads(K, x, e, lens)) for x, e in work]
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(3):
        got = []
        for st, (x, e) in zip(streams, work):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append((run_forward(K, x, e, lens), grads(K, x, e, lens)))
        torch.cuda.synchronize()
        for (f, g), (f2, g2) in zip(want, got):
            assert all(torch.equal(a, c) for a, c in zip(f, f2)) and all(torch.equal(g[m], g2[m]) for m in g)


def test_scan_lengths_that_break_the_rule_stay_inside(K):
    """Starts that are negative, decreasing or too large: any result, but none outside the buffers, and
    correct calls afterwards."""
    lens = [100, 30, 70]
    x, e = inputs(lens, 2, 64, 64, torch.float32)
    good = e["cu"].clone()
    for bad in ([0, 10 ** 9, 5, 200], [-7, 100, 50, 200], [200, 150, 100, 0], [0, 200, 0, 200], [0, 0, 0, 2 ** 31 - 1]):
        e["cu"].copy_(torch.tensor(bad, dtype=torch.int32))
        run_forward(K, x, e, lens)
        grads(K, x, e, lens)
        torch.cuda.synchronize()
    e["cu"].copy_(good)
    check_forward(K, x, e, lens)


def test_scan_keeps_sequences_apart(K):
    """NaN and infinities of one sequence reach no other one."""
    lens = [70, 66, 3, 130]
    for dt in (torch.float32, torch.bfloat16):
        x, e = inputs(lens, 2, 64, 64, dt)
        want, wg = run_forward(K, x, e, lens), grads(K, x, e, lens)
        for i, m in enumerate("qkvzb"):
            x[m][71 + 13 * i] = (float("nan"), float("inf"))[i % 2]
        e["state0"][1, 0, 0, 0] = float("inf")
        got, gg = run_forward(K, x, e, lens), grads(K, x, e, lens)
        rows = torch.tensor([i for i in range(269) if not 70 <= i < 136], device="cuda")
        assert torch.equal(got[0][rows], want[0][rows])
        for s in (0, 2, 3):
            assert torch.equal(got[1][s], want[1][s]) and torch.equal(gg["dstate0"][s], wg["dstate0"][s])
        for m in "qkvzb":
            assert torch.equal(gg["d" + m][rows], wg["d" + m][rows])
        assert not torch.isfinite(got[1][1].sum()) and not torch.isfinite(got[0][135].float().sum())


def test_scan_of_nothing(K):
    x, e = inputs([0, 0], 2, 64, 64, torch.bfloat16)
    o, S = run_forward(K, x, e, [0, 0])
    assert o.shape[0] == 0 and torch.equal(S, e["state0"])
    g = grads(K, x, e, [0, 0])
    assert torch.equal(g["dstate0"], e["dstate"])
    o, S = run_forward(K, x, e, [0, 0], ragged=False)
    assert torch.equal(S, e["state0"])
    g = grads(K, x, e, [0, 0], ragged=False)
    assert torch.equal(g["dstate0"], e["dstate"])


def test_scan_refusals(K):
    x, e = inputs([20, 20], 2, 64, 64, torch.float32)
    q, k, v, z, b = (x[m] for m in "qkvzb")
    bad = [
        (dict(q=q.half()), "q must be float32 or bfloat16"), (dict(k=k.bfloat16()), "k must be"),
        (dict(q=q.cpu()), "q must be a CUDA"), (dict(v=v.cpu()), "v must be a CUDA"), (dict(z=z[:39]), "z must have"),
        (dict(b=b[:, :1]), "b must have"), (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), "dense"),
        (dict(k=k[:1].expand(40, 2, 64)), "not overlap"), (dict(state0=e["state0"].bfloat16()), "state0 must be"),
        (dict(state0=e["state0"][:1], nseq=2), "state0 must have"), (dict(cu_seqlens=e["cu"].long()), "cu_seqlens must be"),
        (dict(cu_seqlens=e["cu"], nseq=3), "does not agree"), (dict(nseq=3), "give cu_seqlens"),
        (dict(out=torch.empty(40, 2, 64, device="cuda", dtype=torch.bfloat16)), "out must be"),
        (dict(state_out=torch.empty(1, 2, 64, 64, device="cuda"), nseq=2), "state_out must have"),
    ]
    for over, text in bad:
        kw = dict(q=q, k=k, v=v, z=z, b=b, state0=None)
        kw.update(over)
        with pytest.raises(ValueError, match=text):
            K.scan_forward(**kw)
    from linear_attention_layer_kda_b200.binding import KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED_SHAPE, KdaError
    one = torch.empty(41 * 2 * 64 + 1, device="cuda")[1:]
    status = [
        (dict(q=one[:40 * 128].view(40, 2, 64)), KDA_ERR_INVALID_ARG),         # 4-byte aligned
        (dict(out=v), KDA_ERR_INVALID_ARG),                                     # output over an input
        (dict(state0=e["state0"], out=e["state0"].view(-1)[:40 * 128].view(40, 2, 64)), KDA_ERR_INVALID_ARG),
    ]
    for over, want in status:
        kw = dict(q=q, k=k, v=v, z=z, b=b)
        kw.update(over)
        with pytest.raises(KdaError) as ei:
            K.scan_forward(**kw)
        assert ei.value.status == want
    w = torch.zeros(40, 2, 32, device="cuda")
    with pytest.raises(KdaError) as ei:
        K.scan_forward(w, w, v, w, b)
    assert ei.value.status == KDA_ERR_UNSUPPORTED_SHAPE
    with pytest.raises(ValueError, match="do must"):
        K.scan_backward(q, k, v, z, b, e["do"][:3])
    with pytest.raises(ValueError, match="dstate must"):
        K.scan_backward(q, k, v, z, b, e["do"], dstate=e["dstate"][:1], nseq=2)


# ------------------------------------------------------------------ the residual norm
# A row's sum of squares has up to 65536 positive terms, summed in fp32 by threads of up to 64 terms,
# then pairwise: (64 + 10 + 32) 2^-24 at most.  rstd is half of that off (its square root), plus a
# few roundings: 64 2^-24 = 2^-18.

def norm_inputs(rows, hidden, xdt, rdt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, hidden, generator=g, device="cuda").to(xdt)
    r = (torch.randn(rows, hidden, generator=g, device="cuda") * 3).to(rdt)
    w = (torch.randn(hidden, generator=g, device="cuda") * 0.2 + 1).to(torch.bfloat16)
    return x, r, w


TYPES = [(a, b) for a in (torch.float32, torch.bfloat16) for b in (torch.float32, torch.bfloat16)]
E4M3_STEP = 2.0 ** -4  # half a step of a normal value


def check_norm(K, x, r, w, eps=1e-6, **kw):
    keep = None if r is None else r.clone()
    got = K.residual_norm(x, r, w, eps=eps, fp8=True, **kw)
    rr, y, scale, rstd = R.residual_norm(x, keep, w, eps)
    assert torch.equal(got.residual.double(), rr)
    t = 2.0 ** -18
    assert ((got.rstd.double() - rstd).abs() <= t * rstd).all()
    assert ((got.y.double() - y).abs() <= (2.0 ** -8 + 2 * t) * y.abs() + 1e-38).all()
    assert ((got.scale.double() - scale).abs() <= 2 * t * scale).all()
    back = got.y8.float().double().view(y.shape[0], -1, 128) * got.scale.double()[..., None]
    yg = y.view_as(back)
    # half a step: 2^-4 of a normal value, half of 2^-9 units of the scale below that
    lim = (E4M3_STEP + 4 * t) * yg.abs() + (2.0 ** -10 + 4 * t) * got.scale.double()[..., None]
    assert ((back - yg).abs() <= lim).all()
    return got


@pytest.mark.parametrize("xdt,rdt", TYPES)
@pytest.mark.parametrize("rows,hidden", [(1, 128), (3, 384), (8, 4096), (5, 6144), (2, 8192), (2, 8320), (1, 65536), (700, 256)])
def test_residual_norm(K, rows, hidden, xdt, rdt):
    check_norm(K, *norm_inputs(rows, hidden, xdt, rdt))


def test_residual_norm_edges(K):
    x, r, w = norm_inputs(6, 512, torch.float32, torch.float32)
    x[0], r[0] = 0, 0                 # a row of zeros
    x[1] = -r[1]                      # that cancels
    x[2, 128:256], r[2, 128:256] = 0, 0   # a group of zeros
    x[3], r[3] = 1e-30, 0             # far below eps
    x[4] *= 1e15
    got = check_norm(K, x, r, w)
    assert (got.y[0] == 0).all() and (got.scale[0] == 1).all() and got.scale[2, 1] == 1
    got = K.residual_norm(x[:2], r[:2], w, eps=0.0, fp8=True)   # 0 / 0 of a zero row
    assert not torch.isfinite(got.y[0].float()).any()
    x[5, 3] = float("nan")
    got = K.residual_norm(x, r, w, fp8=True)
    assert torch.isnan(got.y[5].float()).all() and torch.isnan(got.y8[5].float()).all()
    assert torch.isfinite(got.y[:5].float()).all()
    empty = K.residual_norm(x[:0], r[:0], w, fp8=True)
    assert empty.y.shape == (0, 512) and empty.rstd.shape == (0,)


def test_residual_norm_without_residual_and_in_place(K):
    x, r, w = norm_inputs(9, 1024, torch.bfloat16, torch.bfloat16)
    check_norm(K, x, None, w)
    want = K.residual_norm(x, r, w, fp8=True)
    keep = r.clone()
    got = K.residual_norm(x, r, w, fp8=True, residual_out=r)
    assert got.residual is r and all(torch.equal(a, c) for a, c in zip(got[:2], want[:2]))
    got = K.residual_norm(x, keep, w, residual_out=x)
    assert torch.equal(x, want.residual) and torch.equal(got.y, want.y) and got.y8 is None and got.scale is None
    got = K.residual_norm(x, None, w, bf16=False, fp8=True)
    assert got.y is None


@pytest.mark.parametrize("rdt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(1, 128), (5, 384), (8, 4096), (1300, 1024), (3, 8320), (2, 65536), (0, 256)])
@pytest.mark.parametrize("with_dres", [True, False])
def test_residual_norm_gradient(K, rows, hidden, rdt, with_dres):
    x, r, w = norm_inputs(rows, hidden, torch.float32, rdt)
    g = torch.Generator(device="cuda").manual_seed(9)
    dy = torch.randn(rows, hidden, generator=g, device="cuda").to(torch.bfloat16)
    dres = torch.randn(rows, hidden, generator=g, device="cuda").to(rdt) if with_dres else None
    f = K.residual_norm(x, r, w)
    got, dw = K.residual_norm_backward(dy, f.residual, w, f.rstd, dres)
    again = K.residual_norm_backward(dy, f.residual, w, f.rstd, dres)
    assert torch.equal(got, again[0]) and torch.equal(dw, again[1])
    rr = f.residual.double().requires_grad_()
    ww = w.double().requires_grad_()
    y = rr / torch.sqrt((rr * rr).mean(1, keepdim=True) + 1e-6) * ww
    a, c = torch.autograd.grad((y * dy.double()).sum(), (rr, ww))
    if dres is not None:
        a = a + dres.double()
    if rows:
        size = a.abs().amax(1, keepdim=True)
        assert ((got.double() - a).abs() <= 2.0 ** -16 * size + HALF[rdt] * a.abs()).all()
    # dweight: `rows` terms, summed in a fixed tree
    lim = 2.0 ** -18 * max(1.0, math.sqrt(rows)) * max(1.0, float(c.abs().max()))
    assert ((dw.double() - c).abs() <= lim).all()


def test_residual_norm_gradient_against_differences(K):
    x, r, w = norm_inputs(4, 256, torch.float32, torch.float32)
    f = K.residual_norm(x, r, w)
    g = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.randn(4, 256, generator=g, device="cuda").to(torch.bfloat16)
    d = torch.randn(4, 256, generator=g, device="cuda", dtype=torch.float64)
    got, dw = K.residual_norm_backward(dy, f.residual, w, f.rstd)

    def value(h):
        rr = f.residual.double() + h * d
        return float((rr / torch.sqrt((rr * rr).mean(1, keepdim=True) + 1e-6) * w.double() * dy.double()).sum())
    h = 1e-5
    want = (value(h) - value(-h)) / (2 * h)
    assert abs(float((got.double() * d).sum()) - want) <= 2.0 ** -16 * float(got.abs().max()) * math.sqrt(d.numel()) + 1e-6


def test_residual_norm_refusals(K):
    x, r, w = norm_inputs(4, 256, torch.float32, torch.float32)
    from linear_attention_layer_kda_b200.binding import KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED_SHAPE, KdaError
    for args, text in (((x.cpu(), r, w), "x must be a CUDA"), ((x.half(), r, w), "x must be float32"),
                       ((x, r.half(), w), "residual must be"), ((x, r[:3], w), "residual must have"),
                       ((x, r, w.float()), "weight must be"), ((x, r, w[:128]), "weight must have"),
                       ((x.t().contiguous().t(), r, w), "contiguous")):
        with pytest.raises(ValueError, match=text):
            K.residual_norm(*args)
    with pytest.raises(KdaError) as ei:
        K.residual_norm(x[:, :64].contiguous(), r[:, :64].contiguous(), w[:64].contiguous())
    assert ei.value.status == KDA_ERR_UNSUPPORTED_SHAPE
    for eps in (-1.0, float("nan")):
        with pytest.raises(KdaError) as ei:
            K.residual_norm(x, r, w, eps=eps)
        assert ei.value.status == KDA_ERR_INVALID_ARG
    both = torch.zeros(5, 256, device="cuda")
    with pytest.raises(KdaError) as ei:
        K.residual_norm(both[:4], None, w, residual_out=both[1:])   # shifted by a row
    assert ei.value.status == KDA_ERR_INVALID_ARG
    f = K.residual_norm(x, r, w)
    with pytest.raises(ValueError, match="rstd must have"):
        K.residual_norm_backward(x.bfloat16(), f.residual, w, f.rstd[:3])
    with pytest.raises(ValueError, match="dresidual must be"):
        K.residual_norm_backward(x.bfloat16(), f.residual, w, f.rstd, x.bfloat16())


# ------------------------------------------------------------------ rows of a pool

def check_rows(K, pool, src, dst, source=None):
    old, want = (pool if source is None else source).clone(), pool.clone()
    for a, d in zip(src, dst):
        want[d] = old[a] if a >= 0 else 0
    K.state_rows(pool, src, dst, source_pool=source)
    assert torch.equal(pool, want)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.uint8])
@pytest.mark.parametrize("row", [16, 1040, 16384, 4 * 128 * 128 + 16])
def test_rows_moves(K, row, dt):
    rng = random.Random(row)
    pool = torch.randint(0, 100, (40, row), device="cuda").to(dt)
    check_rows(K, pool, [], [])
    check_rows(K, pool, [3], [3])
    check_rows(K, pool, [1, 0], [0, 1])                        # a swap
    check_rows(K, pool, [1, 2, 3, 0, 0, -1], [0, 1, 2, 3, 4, 5])  # a cycle with a fork out of it
    check_rows(K, pool, [0, 1, 2, 3], [1, 2, 3, 4])            # a shift, read before written
    check_rows(K, pool, [7] * 39, [i for i in range(40) if i != 7])
    for _ in range(20):
        n = rng.randint(1, 40)
        dst = rng.sample(range(40), n)
        check_rows(K, pool, [rng.randint(-1, 39) for _ in range(n)], dst)
    p = list(range(40))
    rng.shuffle(p)
    check_rows(K, pool, p, list(range(40)))                    # a permutation of all
    other = torch.randint(0, 100, (11, row), device="cuda").to(dt)
    check_rows(K, pool, [10, 3, 3, -1], [0, 39, 10, 4], other)


def test_rows_moves_many(K):
    rng = random.Random(1)
    pool = torch.randn(1500, 64, device="cuda")
    for n in (64, 65, 1024):
        dst = rng.sample(range(1500), n)
        check_rows(K, pool, [rng.randint(-1, 1499) for _ in range(n)], dst)
    p = list(range(1024))
    rng.shuffle(p)
    check_rows(K, pool, p, list(range(1024)))


def test_rows_moves_past_32_bits(K):
    """A pool of more than 2^32 bytes: its last rows."""
    row = 1 << 24
    pool = torch.zeros(300, row, dtype=torch.uint8, device="cuda")
    pool[299], pool[1] = 5, 9
    K.state_rows(pool, [299, 1, -1], [280, 299, 1])
    assert (pool[280] == 5).all() and (pool[299] == 9).all() and (pool[1] == 0).all() and (pool[279] == 0).all()


def test_rows_refusals(K):
    from linear_attention_layer_kda_b200.binding import KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED_SHAPE, KdaError
    pool = torch.randn(8, 4, 64, device="cuda")
    keep = pool.clone()
    for src, dst in (([0], [8]), ([8], [0]), ([-2], [0]), ([0], [-1]), ([1, 2], [0, 0]), ([0] * 1025, list(range(1025)))):
        with pytest.raises(KdaError) as ei:
            K.state_rows(pool, src, dst)
        assert ei.value.status == KDA_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="same length"):
        K.state_rows(pool, [1, 2], [0])
    with pytest.raises(ValueError, match="32 bits"):
        K.state_rows(pool, [1 << 32], [0])
    with pytest.raises(TypeError):
        K.state_rows(pool, [1.5], [0])
    with pytest.raises(KdaError) as ei:
        K.state_rows(pool, [0], [1], source_pool=pool[1:])   # overlaps, another start
    assert ei.value.status == KDA_ERR_INVALID_ARG
    with pytest.raises(KdaError) as ei:
        K.state_rows(torch.zeros(4, 3, device="cuda"), [0], [1])
    assert ei.value.status == KDA_ERR_UNSUPPORTED_SHAPE
    with pytest.raises(ValueError, match="same shape"):
        K.state_rows(pool, [0], [1], source_pool=torch.zeros(4, 64, device="cuda"))
    with pytest.raises(ValueError, match="source_pool must be"):
        K.state_rows(pool, [0], [1], source_pool=torch.zeros(8, 4, 64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        K.state_rows(pool[:, :2], [0], [1])
    assert torch.equal(pool, keep)


# ------------------------------------------------------------------ together

def test_a_serving_loop_of_layer_steps_norms_and_row_moves(K):
    """Two layer halves with the norm between them, sequences that fork and finish: every sequence's
    state is that of a run of its own."""
    from linear_attention_layer_kda_b200 import binding, inputs as I, tensors
    shape = I.CONFIGS[0].replace(batch=4, steps=6)
    inp = I.generate(shape)
    H = shape.hidden
    w = tensors.weights_struct(tensors.to_device_weights(inp))
    weight = torch.linspace(0.5, 1.5, H, device="cuda").to(torch.bfloat16)
    dec = binding.KdaDecoder(H, shape.num_heads, shape.head_dk, shape.head_dv, shape.alpha_rank, 4)
    x = [tensors.bf16_tensor(inp.x[t]) for t in range(6)]
    shp = (shape.num_heads, shape.head_dk, shape.head_dv)

    def step(xs, states):
        """Layer half, residual and norm, layer half (the same weights): the second one's out."""
        n = xs.shape[0]
        out = torch.empty(n, H, device="cuda")
        dec.step(xs, w, states[0], out, n)
        f = K.residual_norm(out, xs, weight)
        dec.step(f.y, w, states[1], out, n)
        return K.residual_norm(out, f.residual, weight).y

    try:
        pool = [torch.zeros(4, *shp, device="cuda") for _ in range(2)]
        step(x[0][:2], pool)                       # sequences a, b
        for p in pool:
            K.state_rows(p, [0, 0], [2, 3])        # a continues three ways: rows a, b, a', a''
        step(x[1], pool)
        for p in pool:
            K.state_rows(p, [3, -1], [1, 3])       # b has finished: a'' takes its row
        y = step(x[2][:3], pool)                   # a, a'', a'
        for row, tokens in ((0, (x[0][0], x[1][0], x[2][0])), (1, (x[0][0], x[1][3], x[2][1])),
                            (2, (x[0][0], x[1][2], x[2][2]))):
            own = [torch.zeros(1, *shp, device="cuda") for _ in range(2)]
            for t in tokens:
                z = step(t[None].contiguous(), own)
            for a, c in zip(own, pool):
                assert ((a[0] - c[row]).abs().max() <= 1e-3 * a.abs().max())   # the step's own tolerance
            assert ((z[0].float() - y[row].float()).abs().max() <= (2e-3 + 2.0 ** -8) * 4 * z.float().abs().max())
        dec.sync()
    finally:
        dec.close()


def test_scan_continues_a_prefilled_state(K):
    """kda_prefill's state, continued by the recurrence on projections of the caller's own, equals
    the fp64 recurrence from that state."""
    from linear_attention_layer_kda_b200 import binding, inputs as I, tensors
    shape = I.CONFIGS[0].replace(steps=40)
    inp = I.generate(shape)
    w = tensors.weights_struct(tensors.to_device_weights(inp))
    import numpy as np
    xs = tensors.bf16_tensor(np.concatenate([inp.x[t] for t in range(40)]))
    dec = binding.KdaDecoder(shape.hidden, shape.num_heads, shape.head_dk, shape.head_dv, shape.alpha_rank, 1)
    try:
        S = tensors.state_tensor(inp.state0)
        out = torch.empty(40, shape.hidden, device="cuda")
        dec.prefill(xs, w, S, out, 1, 40)
        x, e = inputs([90], shape.num_heads, shape.head_dk, shape.head_dv, torch.float32, state=False)
        e["state0"] = S
        check_forward(K, x, e, [90])
        check_backward(K, x, e, [90])
        dec.sync()
    finally:
        dec.close()


def test_a_training_step_through_norm_and_recurrence(K):
    """residual norm -> projections -> recurrence and back: the gradient of the residual equals
    that of the same graph in fp64 (bf16 values passed between the parts as they are)."""
    nh, d, hidden, lens = 2, 64, 256, [40, 70]
    n = sum(lens)
    x, r, w = norm_inputs(n, hidden, torch.float32, torch.float32)
    g = torch.Generator(device="cuda").manual_seed(4)
    W = {m: torch.randn(hidden, nh * (1 if m == "b" else d), generator=g, device="cuda") / 16 for m in "qkvzb"}
    do = torch.randn(n, nh, d, generator=g, device="cuda")
    cu = torch.tensor([0, 40, 110], dtype=torch.int32, device="cuda")
    f = K.residual_norm(x, r, w)
    p = {m: (f.y.float() @ W[m]).view(n, nh, -1).contiguous() for m in "qkvz"}
    p["b"] = f.y.float() @ W["b"]
    gr = K.scan_backward(*(p[m] for m in "qkvzb"), do, cu_seqlens=cu)
    dy = sum(gr["d" + m].reshape(n, -1) @ W[m].t() for m in "qkvzb")
    dres, dw = K.residual_norm_backward(dy.bfloat16(), f.residual, w, f.rstd)

    rr, ww = f.residual.double().requires_grad_(), w.double().requires_grad_()
    y = rr / torch.sqrt((rr * rr).mean(1, keepdim=True) + 1e-6) * ww
    q = {m: (y @ W[m].double()).view(n, nh, -1) for m in "qkvz"}
    o, _ = R.scan(q["q"], q["k"], q["v"], q["z"], y @ W["b"].double(), lens)
    a, c = torch.autograd.grad((o * do.double()).sum(), (rr, ww))
    # y and dy pass in bf16 (half a step, 2^-8, each); torch's matrix products in fp32
    assert float((dres.double() - a).norm() / a.norm()) <= 2 * 2.0 ** -8
    assert float((dw.double() - c).norm() / c.norm()) <= 2 * 2.0 ** -8
