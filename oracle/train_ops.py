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


def _group(x, g):
    """Key heads [B, S, Hk, D] for each query head, [B, Hk * g, S, D]."""
    return x.double().transpose(1, 2).repeat_interleave(g, 1)


def cross_attn(q, k, v, lens, scale):
    """(O [B, Sq, Hq, D], LSE [B, Hq, Sq], P) of queries over the first lens[b] keys; keys and
    values behind a length are not looked at."""
    B, Sq, Hq, D = q.shape
    Sk, g = k.shape[1], Hq // k.shape[2]
    out = torch.zeros(B, Hq, Sq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq, Sq), float("-inf"), dtype=torch.float64, device=q.device)
    p = torch.zeros(B, Hq, Sq, Sk, dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        z = scale * q[b].double().transpose(0, 1) @ _group(k[b:b + 1, :n], g)[0].transpose(1, 2)
        lse[b] = torch.logsumexp(z, -1)
        p[b, :, :, :n] = torch.softmax(z, -1)
        out[b] = p[b, :, :, :n] @ _group(v[b:b + 1, :n], g)[0]
    return out.transpose(1, 2), lse, p


def cross_attn_grad(q, k, v, o, do, lse, lens, scale):
    """(dQ, dK, dV, P, dS) with P = exp(scale q k - lse) and the given o, as the operator is defined;
    P and dS are [B, Hq, Sq, Sk]."""
    B, Sq, Hq, D = q.shape
    Sk, Hk = k.shape[1], k.shape[2]
    g = Hq // Hk
    qd, dd = q.double().transpose(1, 2), do.double().transpose(1, 2)
    delta = (dd * o.double().transpose(1, 2)).sum(-1, keepdim=True)
    p = torch.zeros(B, Hq, Sq, Sk, dtype=torch.float64, device=q.device)
    ds = torch.zeros_like(p)
    dq = torch.zeros_like(qd)
    dk = torch.zeros(B, Sk, Hk, D, dtype=torch.float64, device=q.device)
    dv = torch.zeros_like(dk)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        kb, vb = _group(k[b:b + 1, :n], g)[0], _group(v[b:b + 1, :n], g)[0]
        p[b, :, :, :n] = torch.exp(scale * qd[b] @ kb.transpose(1, 2) - lse[b].double()[..., None])
        ds[b, :, :, :n] = p[b, :, :, :n] * (dd[b] @ vb.transpose(1, 2) - delta[b])
        dq[b] = scale * ds[b, :, :, :n] @ kb
        dk[b] = scale * (ds[b].transpose(1, 2) @ qd[b]).view(Hk, g, Sk, D).sum(1).transpose(0, 1)
        dv[b] = (p[b].transpose(1, 2) @ dd[b]).view(Hk, g, Sk, D).sum(1).transpose(0, 1)
    return dq.transpose(1, 2), dk, dv, p, ds


def norm_rope_axes(x, w, cos, sin, pos, sections, eps, interleaved):
    """norm_rope with a position of each axis: pos [axes, B, S], sections the numbers of pairs."""
    c, s, i = _axes_tables(cos, sin, pos, sections)
    return norm_rope(x, w, c, s, i, eps, interleaved)


def norm_rope_axes_grad(dout, x, w, cos, sin, pos, sections, eps, interleaved):
    c, s, i = _axes_tables(cos, sin, pos, sections)
    return norm_rope_grad(dout, x, w, c, s, i, eps, interleaved)


def _axes_tables(cos, sin, pos, sections):
    """Tables with a row for every token, and the tokens' numbers."""
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    rows = [torch.stack([t[pos[a].flatten().long(), i] for i, a in enumerate(axis)], -1) if axis
            else t.new_zeros(pos[0].numel(), 0) for t in (cos, sin)]
    return rows[0], rows[1], torch.arange(pos[0].numel(), device=cos.device).view(pos[0].shape)


def group_norm(x, w, b, groups, eps, act):
    """(y, mean, rstd) for x [N, S, C]."""
    N, S, C = x.shape
    xg = x.double().view(N, S, groups, C // groups)
    mean = xg.mean((1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = 1 / torch.sqrt(var + eps)
    z = _affine(x, w, b, mean, rstd, groups)[1]
    return (z * torch.sigmoid(z) if act == "silu" else z), mean, rstd


def _affine(x, w, b, mean, rstd, groups):
    per = x.shape[2] // groups
    m, r = (t.double().repeat_interleave(per, 1)[:, None] for t in (mean, rstd))
    xh = (x.double() - m) * r
    z = xh * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    return xh, z, r


def group_norm_grad(dy, x, w, b, mean, rstd, groups, act):
    """(dx, dw, db, dz, xh) with the given mean and rstd."""
    N, S, C = x.shape
    xh, z, r = _affine(x, w, b, mean, rstd, groups)
    dz = dy.double()
    if act == "silu":
        sg = torch.sigmoid(z)
        dz = dz * (sg + z * sg * (1 - sg))
    u = dz * (1.0 if w is None else w.double())
    over = lambda t: t.view(N, S, groups, -1).mean((1, 3)).repeat_interleave(C // groups, 1)[:, None]  # noqa: E731
    return r * (u - over(u) - xh * over(u * xh)), (dz * xh).sum((0, 1)), dz.sum((0, 1)), dz, xh
