"""The recurrence over sequences, the residual norm and the moves of rows as defined, in 64 bits (torch)."""
import torch


def scan(q, k, v, z, b, lens, state0=None, first=0):
    """Token by token; lens are the sequences' lengths from row `first` on. Differentiable in fp64."""
    nh, dk = q.shape[1:]
    dv = v.shape[2]
    q, k, v, z, b = (t.double() for t in (q, k, v, z, b))
    size = (k * k).sum(-1, keepdim=True)
    kh = torch.where(size > 0, k / torch.where(size > 0, size, torch.ones_like(size)).sqrt(), torch.zeros_like(k))
    alpha, beta = torch.sigmoid(-z), torch.sigmoid(b)
    outs, states, r = [], [], first
    for i, n in enumerate(lens):
        S = torch.zeros(nh, dk, dv, dtype=torch.float64, device=q.device) if state0 is None else state0[i].double()
        for t in range(r, r + n):
            D = alpha[t][:, :, None] * S
            e = beta[t][:, None] * (v[t] - torch.einsum("hd,hdv->hv", kh[t], D))
            S = D + kh[t][:, :, None] * e[:, None, :]
            outs.append(torch.einsum("hd,hdv->hv", q[t], S))
        r += n
        states.append(S)
    o = torch.stack(outs) if outs else v[:0]
    return o, torch.stack(states)


def scan_grads(q, k, v, z, b, lens, do, dstate=None, state0=None, first=0):
    """Gradients by torch's differentiation of the fp64 recurrence."""
    leaves = [t.double().detach().requires_grad_() for t in (q, k, v, z, b)]
    s0 = None if state0 is None else state0.double().detach().requires_grad_()
    n = sum(lens)
    o, S = scan(*leaves, lens, s0, first)
    f = (o * do[first:first + n].double()).sum()
    if dstate is not None:
        f = f + (S * dstate.double()).sum()
    g = torch.autograd.grad(f, leaves + ([] if s0 is None else [s0]), allow_unused=True)
    r = {"d" + x: (torch.zeros_like(l) if y is None else y) for x, y, l in zip("qkvzb", g, leaves)}
    if s0 is not None:
        r["dstate0"] = g[5]
    return r


def residual_norm(x, residual, weight, eps):
    """(r as its type holds it, y, scale, y / scale) in fp64."""
    r = x.double() if residual is None else (x.float() + residual.float()).to(residual.dtype).double()
    rstd = 1.0 / torch.sqrt((r * r).mean(1) + eps)
    y = r * rstd[:, None] * weight.double()
    amax = y.view(y.shape[0], -1, 128).abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return r, y, scale, rstd
