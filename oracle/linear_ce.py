"""Reference of the output layer's cross-entropy in fp64 (torch, on the device of its arguments), a block
of rows at a time: plain matrix products, logsumexp and softmax of whole rows of logits."""
import torch


def _logits(hidden, weight, scale, rows=2048):
    w = weight.double()
    for r in range(0, hidden.shape[0], rows):
        at = slice(r, min(r + rows, hidden.shape[0]))
        yield at, scale * (hidden[at].double() @ w.t())


def forward(hidden, weight, target, z_loss=0.0, scale=1.0):
    """(loss, lse); targets outside the vocabulary are ignored."""
    n, v = hidden.shape[0], weight.shape[0]
    loss = torch.zeros(n, dtype=torch.float64, device=hidden.device)
    lse = torch.zeros_like(loss)
    for at, z in _logits(hidden, weight, scale):
        t = target[at].long()
        counts = (t >= 0) & (t < v)
        lse[at] = torch.logsumexp(z, 1)
        zt = z.gather(1, t.clamp(0, v - 1)[:, None])[:, 0]
        loss[at] = torch.where(counts, lse[at] - zt + z_loss * lse[at] ** 2, 0.0)
    return loss, lse


def backward(hidden, weight, target, dloss=None, z_loss=0.0, scale=1.0, grad_scale=1.0, lse=None,
             rel=0.0, rounding=0.0):
    """(dhidden, dweight), and bounds of what they may be off by, before their own rounding, when each
    softmax value is off by `rel` of it and each logit gradient by `rounding` of it. Ignored rows count as
    zeros, whatever they hold."""
    n, v = hidden.shape[0], weight.shape[0]
    valid = (target >= 0) & (target < v)
    h = torch.where(valid[:, None], hidden.double(), 0.0)
    w = weight.double()
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    eh, ew = torch.zeros_like(h), torch.zeros_like(w)
    for at, z in _logits(h, weight, scale):
        t, ok = target[at].long(), valid[at]
        e = torch.logsumexp(z, 1) if lse is None else lse[at].double()
        g = grad_scale * (torch.ones_like(e) if dloss is None else dloss[at].double())
        g = torch.where(ok, g, 0.0)
        c = torch.where(ok, g * (1.0 + 2.0 * z_loss * e), 0.0)
        p = torch.exp(z - torch.where(ok, e, 0.0)[:, None]) * c[:, None]
        dz = p.clone()
        dz.scatter_add_(1, t.clamp(0, v - 1)[:, None], -g[:, None])
        dh[at] = scale * (dz @ w)
        dw += scale * (dz.t() @ h[at])
        off = rel * p.abs() + rounding * dz.abs()
        eh[at] = scale * (off @ w.abs())
        ew += scale * (off.t() @ h[at].abs())
    return dh, dw, eh, ew
