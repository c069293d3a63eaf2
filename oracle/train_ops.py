"""The training-step operators' definitions in float64 torch (any device), written from the
formulas; shares no code with the library.

Each function takes tensors of any floating type, converts them to float64 and returns
float64 results that are not rounded.
"""
import torch


def embed(table, ids, scale):
    return scale * table.double()[ids]


def embed_grad(dout, ids, vocab, scale, padding_idx=None):
    """dE[v] = scale * sum of dout[t] over the tokens with id v, by a dense one-hot product
    a few thousand tokens at a time."""
    out = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device=dout.device)
    v = torch.arange(vocab, device=dout.device)
    for t in range(0, ids.numel(), 2048):
        hot = (ids[t:t + 2048, None] == v).double()
        if padding_idx is not None:
            hot[:, padding_idx] = 0
        out += hot.t() @ dout[t:t + 2048].double()
    return scale * out


def _rotation(cos, sin, pos, D, interleaved):
    """Dense [.., D, D] rotation matrices of the tokens' positions."""
    c, s = cos.double()[pos], sin.double()[pos]
    half = c.shape[-1]
    R = torch.eye(D, dtype=torch.float64, device=c.device).expand(*pos.shape, D, D).clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        R[..., a, a], R[..., a, b] = c[..., i], -s[..., i]
        R[..., b, a], R[..., b, b] = s[..., i], c[..., i]
    return R


def norm_rope(x, w, cos, sin, pos, eps, interleaved):
    """x [B, S, H, D], pos [B, S]: rotation of x / rms(x) * w."""
    x = x.double()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        n = n * w.double()
    return torch.einsum("bsij,bshj->bshi", _rotation(cos, sin, pos, x.shape[-1], interleaved), n)


def norm_rope_grad(dout, x, w, cos, sin, pos, eps, interleaved):
    x, d = x.double(), dout.double()
    D = x.shape[-1]
    w = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    dy = torch.einsum("bsij,bshi->bshj", _rotation(cos, sin, pos, D, interleaved), d)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dw = (dy * x * r).sum((0, 1, 2))
    u = dy * w
    return r * u - r ** 3 * x * (u * x).sum(-1, keepdim=True) / D, dw


def xent(x, w, targets, ignore_index, scale=1.0):
    """(loss, lse) of the logits scale * x w^T."""
    z = scale * x.double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    loss = torch.zeros_like(lse)
    for t, y in enumerate(targets.tolist()):
        if y != ignore_index:
            loss[t] = lse[t] - z[t, y]
    return loss, lse


def xent_grad(x, w, targets, dloss, ignore_index, scale=1.0):
    """(dX, dW, G, |P| g): the gradients, the logits' gradient and its softmax part."""
    z = scale * x.double() @ w.double().t()
    p = torch.softmax(z, 1)
    used = (targets != ignore_index).double()[:, None]
    g = scale * dloss.double()[:, None] * used
    hot = (targets[:, None] == torch.arange(w.shape[0], device=x.device)).double()
    G = g * (p - hot)
    return G @ w.double(), G.t() @ x.double(), G, (g * p).abs()


def clip(grads, max_norm):
    norm = torch.sqrt(sum((g.double() ** 2).sum() for g in grads))
    f = max_norm / norm if norm > max_norm else 1.0
    return norm, [g.double() * f for g in grads]
