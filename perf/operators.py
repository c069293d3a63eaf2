"""The operators around the attention in a reproducible training step, as cases that can be
timed and checked: token embedding and its gradient, the norm and rotation of queries and
keys, the cross entropy of a large vocabulary with its gradient, and gradient clipping.

`run` computes a case either in plain torch operations in 32 bits (`own` false) or with this
package's operators (`own` true); `exact` gives the same outputs from the definitions in 64
bits. Sizes: sequence lengths, heads and head dimensions are those of the attention
benchmark (16384 tokens, 16 or 32 heads of 64 or 128, so widths of 1024 to 4096); vocabularies
are generic.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_IGNORE = -100

_da = None


def _lib():
    global _da
    if _da is None:
        import reproducible_deterministic_attn_gb300 as da
        _da = da
    return _da


# ---- cases --------------------------------------------------------------------------------

def listed():
    return [
        # a short batch's lookup: what counts is the launch
        {"name": "embed_fwd_short", "op": "embed", "dir": "fwd", "T": 509, "V": 32768, "D": 1024,
         "dtype": "bf16", "skew": 1.0},
        # one step's 16384 tokens, lookup and the dense gradient of the table
        {"name": "embed_step", "op": "embed", "dir": "both", "T": 16384, "V": 65536, "D": 2048,
         "dtype": "bf16", "skew": 1.0},
        # fp32 gradients of an odd table whose rows are not 16-byte multiples, few tokens repeated often
        {"name": "embed_bwd_odd", "op": "embed", "dir": "bwd", "T": 8191, "V": 5003, "D": 1023,
         "dtype": "fp32", "skew": 1.2},
        # one new token for each of a few sequences, far positions, grouped heads
        {"name": "qk_fwd_token", "op": "qk", "dir": "fwd", "B": 7, "S": 1, "Hq": 32, "Hk": 8, "D": 128,
         "R": 128, "P": 32768, "dtype": "bf16", "interleaved": False},
        # fp16, adjacent pairs, half of the head rotated
        {"name": "qk_bwd_partial", "op": "qk", "dir": "bwd", "B": 3, "S": 1023, "Hq": 16, "Hk": 16, "D": 64,
         "R": 32, "P": 2048, "dtype": "fp16", "interleaved": True},
        # the long causal attention's queries and keys, forward and backward
        {"name": "qk_step", "op": "qk", "dir": "both", "B": 1, "S": 16384, "Hq": 32, "Hk": 32, "D": 128,
         "R": 128, "P": 16384, "dtype": "bf16", "interleaved": False},
        # a small odd vocabulary and a short batch
        {"name": "xent_step_small", "op": "xent", "dir": "both", "T": 333, "V": 5003, "D": 1024},
        # the loss alone (validation)
        {"name": "xent_fwd", "op": "xent", "dir": "fwd", "T": 4096, "V": 32768, "D": 2048},
        # a training step's loss and gradients
        {"name": "xent_step", "op": "xent", "dir": "both", "T": 8192, "V": 65536, "D": 4096},
        # a few small tensors, as of one block's norms and biases
        {"name": "clip_small", "op": "clip", "n": 9, "largest": 70000, "dtype": "fp32", "clips": True},
        # the usual step: the norm is below the limit, the gradients stay as they are
        {"name": "clip_below", "op": "clip", "n": 40, "largest": 16777216, "dtype": "bf16", "clips": False},
        # a model's gradients, clipped into the optimizer's buffers
        {"name": "clip_large", "op": "clip", "n": 48, "largest": 67108864, "dtype": "bf16", "clips": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "qk", "xent", "clip"])
    if op == "embed":
        return {"op": "embed", "dir": rng.choice(["fwd", "bwd", "both"]), "T": _log_int(rng, 1, 16384),
                "V": _log_int(rng, 100, 65536), "D": _log_int(rng, 16, 2048),
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "skew": rng.choice([0.0, 1.0, 1.2])}
    if op == "qk":
        D = rng.choice([64, 96, 128, 256])
        R = rng.choice([D, D // 2, D // 4])
        Hk = rng.choice([1, 2, 4, 8])
        S = _log_int(rng, 1, 4096)
        return {"op": "qk", "dir": rng.choice(["fwd", "bwd", "both"]), "B": rng.randint(1, 4), "S": S,
                "Hq": Hk * rng.choice([1, 2, 4]), "Hk": Hk, "D": D, "R": R, "P": S + rng.randint(0, 4096),
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "interleaved": rng.random() < 0.5}
    if op == "xent":
        return {"op": "xent", "dir": rng.choice(["fwd", "both"]), "T": _log_int(rng, 1, 4096),
                "V": _log_int(rng, 100, 65536), "D": 8 * _log_int(rng, 8, 256)}
    return {"op": "clip", "n": rng.randint(1, 48), "largest": _log_int(rng, 100, 16777216),
            "dtype": rng.choice(["bf16", "fp16", "fp32"]), "clips": rng.random() < 0.6}


# ---- inputs -------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _zipf(T, V, skew, g):
    """Token ids whose frequency falls as rank^-skew (0: uniform), ranks dealt over the table."""
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    if skew <= 0:
        rank = (u * V).long()
    else:
        p = torch.arange(1, V + 1, device="cuda", dtype=torch.float64).pow(-skew).cumsum(0)
        rank = torch.searchsorted(p / p[-1], u)
    order = torch.randperm(V, generator=g, device="cuda")
    return order[rank.clamp_(0, V - 1)]


def _clip_sizes(case):
    """Tensor sizes as of a model's parameter list: a few large ones, the others smaller, some tiny."""
    sizes = []
    for i in range(case["n"]):
        sizes.append(max(1, case["largest"] // (1, 4, 16, 3, 1023)[i % 5] - (0, 1, 7, 0, 5)[i % 5]))
    return sizes


def prepare(case, seed):
    g = _gen(seed)

    def randn(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op == "embed":
        T, V, D, t = case["T"], case["V"], case["D"], _TYPES[case["dtype"]]
        s["scale"] = math.sqrt(D)
        s["ids"] = _zipf(T, V, case["skew"], g)
        if case["dir"] != "bwd":
            s["table"] = randn(V, D, dtype=t, std=0.02)
        if case["dir"] != "fwd":
            s["dout"] = randn(T, D, dtype=t, std=1e-2)
            if own:
                s["ws"] = _lib().new_embed_workspace(T, V, D, "cuda")
    elif op == "qk":
        B, S, Hq, Hk, D, R, t = (case["B"], case["S"], case["Hq"], case["Hk"], case["D"], case["R"],
                                 _TYPES[case["dtype"]])
        # q and k are the first heads of one fused projection's output
        qkv = randn(B, S, Hq + 2 * Hk, D, dtype=t)
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        s["wq"] = 1 + randn(D, std=0.1)
        s["wk"] = 1 + randn(D, std=0.1)
        inv = torch.pow(10000.0, -torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        ang = torch.arange(case["P"], device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        start = torch.randint(0, case["P"] - S + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = (start + torch.arange(S, device="cuda")).to(torch.int32)
        s["eps"] = 1e-6
        if case["dir"] != "fwd":
            s["dq_out"] = randn(B, S, Hq, D, dtype=t, std=0.1)
            s["dk_out"] = randn(B, S, Hk, D, dtype=t, std=0.1)
            if own:
                s["ws"] = _lib().new_qk_norm_rope_workspace(B, S, Hq, Hk, D, "cuda")
    elif op == "xent":
        T, V, D = case["T"], case["V"], case["D"]
        s["w"] = randn(V, D, dtype=torch.bfloat16, std=1.28 / math.sqrt(D))
        y = _zipf(T, V, 1.0, g)
        # hidden states that point to their target more or less, as of a model in training
        toward = torch.rand(T, 1, generator=g, device="cuda") * 8
        s["x"] = (randn(T, D) + toward * s["w"][y].float()).to(torch.bfloat16)
        skip = torch.rand(T, generator=g, device="cuda") < 0.1
        s["y"] = torch.where(skip, torch.full_like(y, _IGNORE), y)
        s["dloss"] = torch.full((T,), 1.0 / T, device="cuda")
        if own:
            s["ws"] = _lib().new_linear_xent_workspace(T, V, D, "cuda")
    else:
        t = _TYPES[case["dtype"]]
        # one tensor in seven keeps 32 bits whatever the others have (norm weights, biases)
        s["grads"] = [randn(n, dtype=torch.float32 if i % 7 == 6 else t, std=1e-3 * (1 + i % 3))
                      for i, n in enumerate(_clip_sizes(case))]
        rough = 1e-3 * math.sqrt(sum(n * (1 + i % 3) ** 2 for i, n in enumerate(_clip_sizes(case))))
        s["max_norm"] = rough * (0.3 if case["clips"] else 4.0)
        if own:
            out = [torch.empty_like(x) for x in s["grads"]] if case["clips"] else None
            s["plan"] = _lib().grad_clip_plan(s["grads"], out)
    return s


# ---- the operators ------------------------------------------------------------------------

def _plain_embed(s):
    c, out = s["case"], []
    if c["dir"] != "bwd":
        out.append((s["table"][s["ids"]].float() * s["scale"]).to(s["table"].dtype))
    if c["dir"] != "fwd":
        d = torch.zeros(c["V"], c["D"], device="cuda")
        d.index_add_(0, s["ids"], s["dout"].float())
        out.append((d * s["scale"]).to(s["dout"].dtype))
    return out


def _own_embed(s):
    c, out, da = s["case"], [], _lib()
    if c["dir"] != "bwd":
        out.append(da.embed_forward(s["table"], s["ids"], s["scale"]))
    if c["dir"] != "fwd":
        out.append(da.embed_backward(s["dout"], s["ids"], c["V"], s["scale"], workspace=s["ws"], check=False))
    return out


def _pairs(x, R, interleaved):
    return (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])


def _joined(a, b, rest, interleaved):
    ab = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _plain_qk(s):
    c, out = s["case"], []
    R, il = c["R"], c["interleaved"]
    cos, sin = s["cos"][s["pos"].long()][:, :, None], s["sin"][s["pos"].long()][:, :, None]
    if c["dir"] != "bwd":
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            xf = x.float()
            y = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + s["eps"]) * w
            a, b = _pairs(y, R, il)
            out.append(_joined(a * cos - b * sin, b * cos + a * sin, y[..., R:], il).to(x.dtype))
    if c["dir"] != "fwd":
        dxs, dws = [], []
        for x, w, d in ((s["q"], s["wq"], s["dq_out"]), (s["k"], s["wk"], s["dk_out"])):
            xf, df = x.float(), d.float()
            r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + s["eps"])
            a, b = _pairs(df, R, il)
            dy = _joined(a * cos + b * sin, b * cos - a * sin, df[..., R:], il)
            n = xf * r
            dws.append((dy * n).sum((0, 1, 2)))
            dn = dy * w
            dxs.append((r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(x.dtype))
        out += dxs + dws
    return out


def _own_qk(s):
    c, out, da = s["case"], [], _lib()
    if c["dir"] != "bwd":
        out += da.qk_norm_rope_forward(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"],
                                       eps=s["eps"], interleaved=c["interleaved"])
    if c["dir"] != "fwd":
        out += da.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["wq"], s["wk"], s["cos"],
                                        s["sin"], s["pos"], eps=s["eps"], interleaved=c["interleaved"],
                                        workspace=s["ws"], check=False)
    return out


_PIECE = 8192


def _plain_xent(s):
    c, x, w, y = s["case"], s["x"].float(), s["w"], s["y"]
    T, V = c["T"], c["V"]
    keep = y != _IGNORE
    m = torch.full((T,), float("-inf"), device="cuda")
    total = torch.zeros(T, device="cuda")
    at = torch.zeros(T, device="cuda")
    for v in range(0, V, _PIECE):
        z = x @ w[v:v + _PIECE].float().t()
        new = torch.maximum(m, z.max(1).values)
        total = total * (m - new).exp() + (z - new[:, None]).exp().sum(1)
        m = new
        here = (y >= v) & (y < v + z.shape[1])
        at = torch.where(here, z.gather(1, torch.where(here, y - v, 0)[:, None])[:, 0], at)
    lse = m + total.log()
    out = [torch.where(keep, lse - at, 0.0), lse]
    if c["dir"] == "both":
        g = torch.where(keep, s["dloss"], 0.0)[:, None]
        dx = torch.zeros_like(x)
        dw = torch.empty_like(w)
        for v in range(0, V, _PIECE):
            wp = w[v:v + _PIECE].float()
            p = (x @ wp.t() - lse[:, None]).exp()
            here = (y >= v) & (y < v + p.shape[1])
            p -= (torch.where(here, y - v, -1)[:, None] == torch.arange(p.shape[1], device="cuda")).float()
            p *= g
            dx += p @ wp
            dw[v:v + _PIECE] = (p.t() @ x).to(w.dtype)
        out += [dx.to(s["x"].dtype), dw]
    return out


def _own_xent(s):
    c, da = s["case"], _lib()
    loss, lse = da.linear_xent_forward(s["x"], s["w"], s["y"], ignore_index=_IGNORE, workspace=s["ws"], check=False)
    out = [loss, lse]
    if c["dir"] == "both":
        out += da.linear_xent_backward(s["x"], s["w"], s["y"], lse, s["dloss"], ignore_index=_IGNORE,
                                       workspace=s["ws"], check=False)
    return out


def _plain_clip(s):
    total = torch.zeros((), device="cuda")
    for x in s["grads"]:
        f = x.float()
        total += (f * f).sum()
    norm = total.sqrt()
    if not s["case"]["clips"]:
        # multiplied in place by a factor that is one below the limit
        f = torch.clamp(s["max_norm"] / norm, max=1.0)
        for x in s["grads"]:
            x.mul_(f)
        return [norm] + s["grads"]
    f = torch.clamp(s["max_norm"] / norm, max=1.0)
    return [norm] + [(x.float() * f).to(x.dtype) for x in s["grads"]]


def _own_clip(s):
    norm, grads = _lib().grad_clip(s["plan"], s["max_norm"])
    return [norm] + list(grads)


def run(state):
    op = state["case"]["op"]
    f = {"embed": (_plain_embed, _own_embed), "qk": (_plain_qk, _own_qk), "xent": (_plain_xent, _own_xent),
         "clip": (_plain_clip, _own_clip)}[op]
    return f[1 if own else 0](state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "embed":
        T, V, D, e = case["T"], case["V"], case["D"], _BYTES[case["dtype"]]
        b = f = 0
        if case["dir"] != "bwd":
            b += T * 8 + min(T, V) * D * e + T * D * e
            f += T * D
        if case["dir"] != "fwd":
            b += T * 8 + T * D * e + V * D * e
            f += 2 * T * D
        return {"bytes": b, "flops": f}
    if op == "qk":
        rows, e = case["B"] * case["S"] * (case["Hq"] + case["Hk"]), _BYTES[case["dtype"]]
        D, R = case["D"], case["R"]
        tab = case["B"] * case["S"] * (4 + R * 4) + 8 * D
        b = f = 0
        if case["dir"] != "bwd":
            b += 2 * rows * D * e + tab
            f += rows * (4 * D + 3 * R)
        if case["dir"] != "fwd":
            b += 3 * rows * D * e + tab + 8 * D
            f += rows * (11 * D + 3 * R)
        return {"bytes": b, "flops": f}
    if op == "xent":
        T, V, D = case["T"], case["V"], case["D"]
        b, f = (T + V) * D * 2 + T * 16, 2 * T * V * D
        if case["dir"] == "both":
            # the logits are not kept, so the gradient takes their product once more
            b += 2 * (T + V) * D * 2 + T * 16
            f += 6 * T * V * D
        return {"bytes": b, "flops": f}
    e = _BYTES[case["dtype"]]
    total = sum(n * (4 if i % 7 == 6 else e) for i, n in enumerate(_clip_sizes(case)))
    # clipped: the factor is known only when all has been read, but one read and one write would do
    # on a card that could hold the gradients
    return {"bytes": total * (2 if case["clips"] else 1), "flops": 2 * sum(_clip_sizes(case))}


# ---- the definitions in 64 bits -------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "xent" and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    if op == "embed":
        out = []
        if case["dir"] != "bwd":
            out.append(s["table"].index_select(0, s["ids"]).double().mul_(s["scale"]))
        if case["dir"] != "fwd":
            # tokens in the order of their ids, then a running sum's differences would lose bits:
            # each id's rows are added one repetition after the other
            order = torch.argsort(s["ids"], stable=True)
            ids = s["ids"][order]
            first = torch.searchsorted(ids, ids)
            rep = torch.arange(ids.numel(), device="cuda") - first
            d = torch.zeros(case["V"], case["D"], dtype=torch.float64, device="cuda")
            by = torch.argsort(rep, stable=True)
            counts = torch.bincount(rep).tolist()
            at = 0
            for n in counts:
                sel = by[at:at + n]
                at += n
                d[ids[sel]] += s["dout"][order[sel]].double()
            out.append(d.mul_(s["scale"]))
        return out
    if op == "qk":
        outs, dxs, dws = [], [], []
        R, D = case["R"], case["D"]
        i = torch.arange(R // 2, device="cuda")
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
        c, sn = s["cos"].double()[s["pos"].long()], s["sin"].double()[s["pos"].long()]
        for name in ("q", "k"):
            w = s["w" + name].double()
            x = s[name].double()
            dst = torch.empty_like(x) if case["dir"] != "bwd" else None
            if case["dir"] != "fwd":
                dx, dw = torch.empty_like(x), torch.zeros(D, dtype=torch.float64, device="cuda")
            for h in range(x.shape[2]):
                xh = x[:, :, h]
                r = 1.0 / torch.sqrt(xh.square().sum(-1, keepdim=True) / D + s["eps"])
                if dst is not None:
                    y = xh * r * w
                    z = y.clone()
                    z[..., lo] = y[..., lo] * c - y[..., hi] * sn
                    z[..., hi] = y[..., lo] * sn + y[..., hi] * c
                    dst[:, :, h] = z
                if case["dir"] != "fwd":
                    d = s["d%s_out" % name][:, :, h].double()
                    dy = d.clone()
                    dy[..., lo] = d[..., lo] * c + d[..., hi] * sn
                    dy[..., hi] = d[..., hi] * c - d[..., lo] * sn
                    dw += (dy * xh * r).sum((0, 1))
                    u = w * dy
                    dx[:, :, h] = r * u - xh * r.pow(3) * (u * xh).sum(-1, keepdim=True) / D
            if dst is not None:
                outs.append(dst)
            if case["dir"] != "fwd":
                dxs.append(dx)
                dws.append(dw)
        return outs + dxs + dws
    if op == "xent":
        T, V = case["T"], case["V"]
        x, w, y = s["x"].double(), s["w"].double(), s["y"]
        used = y != _IGNORE
        loss = torch.zeros(T, dtype=torch.float64, device="cuda")
        lse = torch.empty(T, dtype=torch.float64, device="cuda")
        dx, dw = torch.empty_like(x), torch.zeros_like(w)
        for t in range(0, T, 1024):  # rows at a time, each with its whole vocabulary
            z = x[t:t + 1024] @ w.t()
            lse[t:t + 1024] = torch.logsumexp(z, 1)
            u = used[t:t + 1024].nonzero()[:, 0]
            yt = y[t:t + 1024][u]
            loss[t + u] = lse[t + u] - z[u, yt]
            if case["dir"] == "both":
                p = torch.softmax(z, 1)
                p[u, yt] -= 1.0
                p *= (s["dloss"][t:t + 1024].double() * used[t:t + 1024])[:, None]
                dx[t:t + 1024] = p @ w
                dw += p.t() @ x[t:t + 1024]
        return [loss, lse] + ([dx, dw] if case["dir"] == "both" else [])
    n = math.sqrt(math.fsum(float(x.double().square().sum()) for x in s["grads"]))
    f = min(1.0, s["max_norm"] / n)
    return [torch.tensor(n, dtype=torch.float64, device="cuda")] + [x.double() * f for x in s["grads"]]
