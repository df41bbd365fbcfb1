"""The operators around the decode step, as they are measured: the recurrence over whole (ragged)
sequences with its backward pass, the residual's root-mean-square norm with an 8-bit output and its
backward pass, and the moves of state rows inside a pool.

``run`` computes each of them in a plain form (elementary torch operations, fp32) where ``own`` is
false, and through the package's entry points where it is true.  ``exact`` computes the same from
the definitions in fp64, token by token, written apart from the plain form.

The recurrence, per head, with k^ = k / |k| (0 for a zero key), alpha = exp(-softplus(z)) per key
channel and beta = sigmoid(b):
    S_t = (I - beta k^ k^T) diag(alpha) S_{t-1} + beta k^ v^T,      o_t = S_t^T q_t.
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 128        # columns that share one 8-bit scale
E4M3_MAX = 448.0
CHUNK = 32         # tokens per chunk of the plain form


def listed():
    bf, fp = "bf16", "fp32"
    return [
        # one token of one sequence at the smallest layer: nothing but latency
        dict(name="scan_step_1seq_2x64", op="scan", lens="1", nh=2, dk=64, dv=64, dtype=bf, state=True, zmean=0.0),
        # one token of 64 sequences at 48 heads: the serving step, the state's bytes
        dict(name="scan_step_64seq_48x128", op="scan", lens="64x1", nh=48, dk=128, dv=128, dtype=bf,
             state=True, zmean=0.0),
        # prompts of many lengths in one batch (one token, an empty one, long ones)
        dict(name="scan_ragged_32x128", op="scan", lens="1,517,2048,33,0,1201,255,41", nh=32, dk=128, dv=128, dtype=bf,
             state=True, zmean=-2.0),
        # one long prompt, few heads, fp32 activations, dk < dv
        dict(name="scan_long_fp32_8x64x128", op="scan", lens="4096", nh=8, dk=64, dv=128, dtype=fp, state=False,
             zmean=-4.0),
        # a training batch: four sequences of 2048 tokens through the layer's 32 heads
        dict(name="scan_grad_4x2048_32x128", op="scan_grad", lens="4x2048", nh=32, dk=128, dv=128, dtype=bf, state=False,
             zmean=-2.0),
        # packed short documents, fp32, dk > dv, a gradient that reaches the initial states
        dict(name="scan_grad_ragged_fp32", op="scan_grad", lens="700,3,129,64,1", nh=4, dk=128, dv=64, dtype=fp,
             state=True, zmean=-1.0),
        # one long sequence, the heads of one tensor-parallel rank
        dict(name="scan_grad_long_8x128", op="scan_grad", lens="4096", nh=8, dk=128, dv=128, dtype=bf, state=True,
             zmean=-4.0),
        # between two layer halves of the batch-8 decode step
        dict(name="norm_8x4096", op="norm", rows=8, hidden=4096, xdt=fp, rdt=bf),
        # the same for a prompt at the widest layer
        dict(name="norm_8192x6144", op="norm", rows=8192, hidden=6144, xdt=bf, rdt=bf),
        # its gradient for a training batch
        dict(name="norm_grad_8192x4096", op="norm_grad", rows=8192, hidden=4096, xdt=bf, rdt=bf),
        # finished sequences leave holes: the last rows move into them, what they leave is cleared
        dict(name="rows_compact_64x48x128", op="rows", pool=64, row=48 * 128 * 128, fork=1, sources=20, free=20, dt=fp),
        # a shared prefix's state is forked for its continuations
        dict(name="rows_fork_128x32x128", op="rows", pool=128, row=32 * 128 * 128, fork=15, sources=4, free=8, dt=fp),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "scan", "scan", "scan_grad", "scan_grad", "norm", "norm_grad", "rows"])
    if kind in ("scan", "scan_grad", "step"):
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        case = dict(op="scan" if kind == "step" else kind, dk=dk, dv=dv, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    state=rng.random() < 0.7, zmean=round(rng.uniform(-5.0, 0.5), 2))
        if kind == "step":
            return dict(case, nh=rng.choice([1, 2, 5, 16, 32, 48]), lens="%dx1" % _log(rng, 1, 64))
        nh = _log(rng, 1, 32)
        lens = [_log(rng, 1, 2500) if rng.random() < 0.9 else 0 for _ in range(_log(rng, 1, 12))]
        while sum(lens) * nh > (131072 if kind == "scan" else 65536):  # within the largest listed case
            lens[lens.index(max(lens))] //= 2
        return dict(case, nh=nh, lens=",".join(map(str, lens + [rng.randint(1, 70)])))
    if kind in ("norm", "norm_grad"):
        hidden = 128 * _log(rng, 1, 64)
        rows = min(_log(rng, 1, 16384), (48 << 20) // hidden)
        return dict(op=kind, rows=rows, hidden=hidden, xdt=rng.choice(["bf16", "fp32"]), rdt=rng.choice(["bf16", "fp32"]))
    pool = _log(rng, 6, 96)
    sources = rng.randint(1, max(1, pool // 4))
    fork = rng.randint(1, max(1, (pool // 2) // sources))
    return dict(op="rows", pool=pool, row=8 * _log(rng, 8, 98304), fork=fork, sources=sources,
                free=rng.randint(0, pool - sources * (fork + 1)), dt=rng.choice(["fp32", "bf16"]))


def _lens(case):
    s = case["lens"]
    if "x" in s:
        n, t = s.split("x")
        return [int(t)] * int(n)
    return [int(t) for t in s.split(",")]


_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _normal(gen, *shape, scale=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("scan", "scan_grad"):
        lens = _lens(case)
        n, nh, dk, dv, dt = sum(lens), case["nh"], case["dk"], case["dv"], _DT[case["dtype"]]
        cu = [0]
        for t in lens:
            cu.append(cu[-1] + t)
        s = dict(case=case, lens=lens,
                 cu=None if len(set(lens)) == 1 else torch.tensor(cu, dtype=torch.int32, device="cuda"),
                 q=_normal(gen, n, nh, dk, dtype=dt), k=_normal(gen, n, nh, dk, dtype=dt),
                 v=_normal(gen, n, nh, dv, dtype=dt), z=_normal(gen, n, nh, dk, mean=case["zmean"], dtype=dt),
                 b=_normal(gen, n, nh, dtype=dt), state0=None)
        if case["state"]:
            s["state0"] = _normal(gen, len(lens), nh, dk, dv, scale=0.1)
        if op == "scan_grad":
            s["do"] = _normal(gen, n, nh, dv, dtype=dt)
            s["dstate"] = _normal(gen, len(lens), nh, dk, dv, scale=0.1) if case["state"] else None
        return s
    if op in ("norm", "norm_grad"):
        n, h = case["rows"], case["hidden"]
        s = dict(case=case, x=_normal(gen, n, h, dtype=_DT[case["xdt"]]),
                 residual=_normal(gen, n, h, scale=3.0, dtype=_DT[case["rdt"]]),
                 weight=_normal(gen, h, scale=0.2, mean=1.0, dtype=torch.bfloat16))
        if op == "norm_grad":  # what the forward call left, and the gradients of its outputs
            s["residual"] = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
            s["rstd"] = (s["residual"].float().square().mean(1) + EPS).rsqrt()
            s["dy"] = _normal(gen, n, h, dtype=torch.bfloat16)
            s["dresidual"] = _normal(gen, n, h, dtype=_DT[case["rdt"]])
        return s
    pool = _normal(gen, case["pool"], case["row"], dtype=_DT[case["dt"]])
    order = torch.randperm(case["pool"], generator=gen, device="cuda").tolist()
    ns, nf = case["sources"], case["fork"]
    src = [order[i] for i in range(ns) for _ in range(nf)]
    dst = order[ns:ns + ns * nf]
    free = order[ns + ns * nf:ns + ns * nf + case["free"]]
    return dict(case=case, pool=pool, src=src + [-1] * len(free), dst=dst + free)


# ---------------------------------------------------------------- plain forms

def _chunk(S, q, k, v, la, beta):
    """CHUNK tokens of every sequence and head from the state S: (o, S')."""
    L = la.cumsum(1)                                                  # [B, C, dk]
    C = q.shape[1]
    lower = torch.ones(C, C, device=q.device, dtype=torch.bool).tril()
    gamma = (L[:, :, None] - L[:, None]).masked_fill(~lower[..., None], -math.inf).exp()
    kg = gamma * k[:, None]
    P = (kg * k[:, :, None]).sum(-1).tril(-1)
    M = (kg * q[:, :, None]).sum(-1)
    eye = torch.eye(C, device=q.device)
    N = -beta[..., None] * P
    inv = eye + N
    for _ in range(int(math.log2(CHUNK)) - 1):                        # (I - N)^-1 = (I + N)(I + N^2)(I + N^4)...
        N = N @ N
        inv = inv + inv @ N
    g = L.exp()
    U = inv @ (beta[..., None] * (v - (g * k) @ S))
    o = (g * q) @ S + M @ U
    W = (L[:, -1:] - L).exp() * k
    return o, g[:, -1, :, None] * S + W.transpose(1, 2) @ U


def _plain_scan(q, k, v, z, b, state0, lens):
    n, nh, dk = q.shape
    dv, B = v.shape[-1], len(lens)
    T = max(CHUNK, -(-max(lens) // CHUNK) * CHUNK) if max(lens) > 1 else 1
    at = torch.arange(T, device=q.device)[None] < torch.tensor(lens, device=q.device)[:, None]      # [B, T]

    def pad(x):  # rows [n, nh, d] -> [B * nh, T, d], zero where a sequence has ended
        y = torch.zeros(B, T, nh, x.shape[-1], device=x.device).masked_scatter(at[:, :, None, None], x)
        return y.transpose(1, 2).reshape(B * nh, T, x.shape[-1])

    norm = k.square().sum(-1, keepdim=True)
    k = torch.where(norm > 0, k * torch.where(norm > 0, norm, 1.0).rsqrt(), 0.0)
    q, k, v, la, beta = pad(q), pad(k), pad(v), pad(-torch.nn.functional.softplus(z, threshold=100.0)), pad(b.sigmoid()[..., None])
    S = torch.zeros(B * nh, dk, dv, device=q.device) if state0 is None else state0.reshape(B * nh, dk, dv)
    o, step = [], min(CHUNK, T)
    for c in range(0, T, step):
        e = slice(c, c + step)
        oc, S = _chunk(S, q[:, e], k[:, e], v[:, e], la[:, e], beta[:, e, 0])
        o.append(oc)
    o = torch.cat(o, 1).reshape(B, nh, T, dv).transpose(1, 2)
    return o[at], S.reshape(B, nh, dk, dv)


def _plain_norm(s):
    r = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    rf = r.float()
    rstd = (rf.square().mean(1) + EPS).rsqrt()
    y = rf * rstd[:, None] * s["weight"].float()
    g = y.reshape(y.shape[0], -1, GROUP)
    amax = g.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    codes = (g / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).reshape(y.shape).to(torch.float8_e4m3fn)
    return dict(residual=r, y=y.to(torch.bfloat16), y8=codes, scale=scale, rstd=rstd)


def _plain_norm_grad(s):
    rf, rstd = s["residual"].float(), s["rstd"][:, None]
    n = rf * rstd
    dy = s["dy"].float()
    dn = dy * s["weight"].float()
    d = rstd * (dn - n * (dn * n).mean(1, keepdim=True)) + s["dresidual"].float()
    return dict(dresidual=d.to(s["residual"].dtype), dweight=(dy * n).sum(0))


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from linear_attention_layer_kda_b200 import operators as K
        if op == "scan":
            o, S = K.scan_forward(s["q"], s["k"], s["v"], s["z"], s["b"], state0=s["state0"], cu_seqlens=s["cu"],
                                  nseq=len(s["lens"]))
            return dict(o=o, state=S)
        if op == "scan_grad":
            return K.scan_backward(s["q"], s["k"], s["v"], s["z"], s["b"], s["do"], dstate=s["dstate"],
                                   state0=s["state0"], cu_seqlens=s["cu"], nseq=len(s["lens"]))
        if op == "norm":
            r, y, y8, scale, rstd = K.residual_norm(s["x"], s["residual"], s["weight"], eps=EPS, fp8=True)
            return dict(residual=r, y=y, y8=y8, scale=scale, rstd=rstd)
        if op == "norm_grad":
            d, dw = K.residual_norm_backward(s["dy"], s["residual"], s["weight"], s["rstd"], dresidual=s["dresidual"])
            return dict(dresidual=d, dweight=dw)
        K.state_rows(s["pool"], s["src"], s["dst"])
        return s["pool"]
    if op == "scan":
        dt = s["v"].dtype
        q, k, v, z, b = (s[n].float() for n in "qkvzb")
        o, S = _plain_scan(q, k, v, z, b, s["state0"], s["lens"])
        return dict(o=o.to(dt), state=S)
    if op == "scan_grad":
        dt = s["v"].dtype
        leaves = [s[n].float().requires_grad_() for n in "qkvzb"]
        state0 = None if s["state0"] is None else s["state0"].detach().requires_grad_()
        o, S = _plain_scan(*leaves, state0, s["lens"])
        outs, grads = [o], [s["do"].float()]
        if s["dstate"] is not None:
            outs, grads = [o, S], grads + [s["dstate"]]
        got = torch.autograd.grad(outs, leaves + ([] if state0 is None else [state0]), grads)
        r = {"d" + n: g.to(dt) for n, g in zip("qkvzb", got)}
        if state0 is not None:
            r["dstate0"] = got[5]
        return r
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    pool, moved = s["pool"], [(a, d) for a, d in zip(s["src"], s["dst"]) if a >= 0]
    pool[[d for _, d in moved]] = pool[[a for a, _ in moved]]
    pool[[d for a, d in zip(s["src"], s["dst"]) if a < 0]] = 0
    return pool


# ---------------------------------------------------------------- definitions in 64 bits

def _exact_scan(s, grad):
    """Token by token in fp64; the gradient by the adjoint recurrence, states recomputed by segments."""
    lens, (n, nh, dk), dv = s["lens"], s["q"].shape, s["v"].shape[-1]
    B, T = len(lens), max(lens)
    q, k, v, z, b = (s[x].double() for x in "qkvzb")
    size = (k * k).sum(-1, keepdim=True).sqrt()
    safe = torch.where(size > 0, size, torch.ones_like(size))
    kh = torch.where(size > 0, k / safe, torch.zeros_like(k))
    alpha, beta = 1.0 / (1.0 + torch.exp(z)), 1.0 / (1.0 + torch.exp(-b))
    starts = [sum(lens[:i]) for i in range(B)]
    live = [[i for i in range(B) if lens[i] > t] for t in range(T)]
    idx = [torch.tensor(x, device=q.device) for x in live]
    row = [torch.tensor([starts[i] + t for i in x], device=q.device) for t, x in enumerate(live)]
    S = torch.zeros(B, nh, dk, dv, dtype=torch.float64, device=q.device) if s["state0"] is None else s["state0"].double()
    o = torch.zeros(n, nh, dv, dtype=torch.float64, device=q.device)

    def step(S, t, out=None):
        r = row[t]
        D = alpha[r][..., None] * S[idx[t]]
        e = v[r] - torch.einsum("bhd,bhdv->bhv", kh[r], D)
        new = D + torch.einsum("bhd,bhv->bhdv", beta[r][..., None] * kh[r], e)
        S = S.clone()
        S[idx[t]] = new
        if out is not None:
            out[r] = torch.einsum("bhd,bhdv->bhv", q[r], new)
        return S

    SEG = 64
    at = []
    for t in range(T):
        if grad and t % SEG == 0:
            at.append(S)
        S = step(S, t, o)
    if not grad:
        return dict(o=o, state=S)
    dS = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    dq, dk_, dv_, dz, db = (torch.zeros_like(x) for x in (q, k, v, z, b))
    do = s["do"].double()
    for c in reversed(range(len(at))):
        seg = [at[c]]
        for t in range(c * SEG, min(T, (c + 1) * SEG)):
            seg.append(step(seg[-1], t))
        for t in reversed(range(c * SEG, min(T, (c + 1) * SEG))):
            i, r = idx[t], row[t]
            old, new = seg[t - c * SEG][i], seg[t - c * SEG + 1][i]
            dq[r] = torch.einsum("bhdv,bhv->bhd", new, do[r])
            G = dS[i] + torch.einsum("bhd,bhv->bhdv", q[r], do[r])           # gradient of the new state
            D = alpha[r][..., None] * old
            e = v[r] - torch.einsum("bhd,bhdv->bhv", kh[r], D)
            kG = torch.einsum("bhd,bhdv->bhv", kh[r], G)
            dbeta = (kG * e).sum(-1)
            de = beta[r][..., None] * kG
            dkh = torch.einsum("bhdv,bhv->bhd", G, e) * beta[r][..., None] - torch.einsum("bhdv,bhv->bhd", D, de)
            dD = G - torch.einsum("bhd,bhv->bhdv", kh[r], de)
            dv_[r] = de
            db[r] = dbeta * beta[r] * (1 - beta[r])
            dz[r] = (dD * old).sum(-1) * -alpha[r] * (1 - alpha[r])
            dk_[r] = torch.where(size[r] > 0, (dkh - kh[r] * (kh[r] * dkh).sum(-1, keepdim=True)) / safe[r], 0.0)
            dS = dS.clone()
            dS[i] = alpha[r][..., None] * dD
    r = dict(dq=dq, dk=dk_, dv=dv_, dz=dz, db=db)
    if s["state0"] is not None:
        r["dstate0"] = dS
    return r


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "scan_grad"):
        return _exact_scan(s, op == "scan_grad")
    if op == "norm":
        r = (s["x"].double() + s["residual"].double()).to(s["residual"].dtype).double()
        rstd = 1.0 / torch.sqrt((r * r).mean(1) + EPS)
        y = r * rstd[:, None] * s["weight"].double()
        g = y.reshape(y.shape[0], -1, GROUP)
        amax = g.abs().amax(-1)
        scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        a = (g / scale[..., None]).reshape(y.shape)
        _, ex = torch.frexp(a)
        quantum = torch.ldexp(torch.ones_like(a), torch.clamp(ex - 1, min=-6) - 3)
        return dict(residual=r, y=y, y8=torch.round(a / quantum) * quantum, scale=scale, rstd=rstd)
    if op == "norm_grad":
        r, rstd, dy = s["residual"].double(), s["rstd"].double()[:, None], s["dy"].double()
        dn = dy * s["weight"].double()
        n = r * rstd
        d = rstd * dn - rstd * n * (dn * n).sum(1, keepdim=True) / r.shape[1] + s["dresidual"].double()
        return dict(dresidual=d, dweight=torch.einsum("nh,nh->h", dy, n))
    old = s["pool"].double()
    new = old.clone()
    for a, d in zip(s["src"], s["dst"]):
        new[d] = old[a] if a >= 0 else torch.zeros_like(old[d])
    return new


def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op in ("scan", "scan_grad"):
        lens = _lens(case)
        n, nh, dk, dv, e = sum(lens), case["nh"], case["dk"], case["dv"], size[case["dtype"]]
        rows = n * nh * (3 * dk + dv + 1) * e
        states = len(lens) * nh * dk * dv * 4
        token = n * nh * dk * dv
        if op == "scan":  # inputs, o, the state in and out; k^T S, the update and S^T q for each token
            return dict(bytes=rows + n * nh * dv * e + states * (2 if case["state"] else 1), flops=7 * token)
        # inputs, do and the gradients; the forward's products and those of the adjoint state
        return dict(bytes=2 * rows + n * nh * dv * e + states * (3 if case["state"] else 0), flops=20 * token)
    if op in ("norm", "norm_grad"):
        n, h = case["rows"], case["hidden"]
        x, r = size[case["xdt"]], size[case["rdt"]]
        if op == "norm":
            return dict(bytes=n * h * (x + 2 * r + 2 + 1) + n * h // GROUP * 4 + n * 4 + 2 * h, flops=8 * n * h)
        return dict(bytes=n * h * (2 + 3 * r) + n * 4 + 6 * h, flops=10 * n * h)
    row = case["row"] * size[case["dt"]]
    # each source row read once, each destination and each freed row written once
    return dict(bytes=row * (case["sources"] * (1 + case["fork"]) + case["free"]), flops=0)
