"""The operators that a reproducible training step of image, video and encoder-decoder models has
beside those of a language model, as cases that can be timed and checked: cross attention to an
encoder's states of another length, the norm and rotation of queries and keys by positions with
several axes, and group norm with an activation over channels-last tensors.

`run` computes a case either in plain torch operations in 32 bits (`own` false) or with this
package's operators (`own` true); `exact` gives the same outputs from the definitions in 64
bits. Sequence lengths, heads and head dimensions are those of the attention benchmark (up to
16384 tokens, 16 or 32 heads of 64 or 128); encoder lengths and channels are generic.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}

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
        # one new token of each of a few sequences against encoder states of unlike lengths
        {"name": "cross_token", "op": "cross", "dir": "fwd", "B": 7, "Sq": 1, "Sk": 1500, "Hq": 32, "Hk": 8,
         "D": 128, "ragged": True, "empty": False},
        # image tokens that look at short captions of unlike lengths, evaluation
        {"name": "cross_text_fwd", "op": "cross", "dir": "fwd", "B": 4, "Sq": 4096, "Sk": 77, "Hq": 16, "Hk": 16,
         "D": 64, "ragged": True, "empty": False},
        # few queries over a long odd encoder, shared key heads, one sequence without a condition: gradients
        {"name": "cross_bwd_odd", "op": "cross", "dir": "bwd", "B": 3, "Sq": 333, "Sk": 2049, "Hq": 16, "Hk": 4,
         "D": 80, "ragged": True, "empty": True},
        # a training step of long image sequences over text: forward and gradients
        {"name": "cross_step", "op": "cross", "dir": "both", "B": 2, "Sq": 8192, "Sk": 512, "Hq": 16, "Hk": 16,
         "D": 128, "ragged": True, "empty": False},
        # long queries over long states, shared key heads
        {"name": "cross_long_fwd", "op": "cross", "dir": "fwd", "B": 1, "Sq": 16384, "Sk": 4096, "Hq": 32, "Hk": 8,
         "D": 128, "ragged": False, "empty": False},
        # one new token for each of a few sequences after an image, three axes
        {"name": "axes_fwd_token", "op": "axes", "dir": "fwd", "B": 7, "S": 1, "Hq": 32, "Hk": 8, "D": 128,
         "sections": "16,24,24", "P": 32768, "dtype": "bf16", "interleaved": False},
        # video frames, sections of the pairs that are no multiples of four, gradients in fp16
        {"name": "axes_bwd_video", "op": "axes", "dir": "bwd", "B": 3, "S": 1023, "Hq": 16, "Hk": 16, "D": 128,
         "sections": "22,21,21", "P": 1024, "dtype": "fp16", "interleaved": True},
        # the long attention's queries and keys as image patches among text, forward and backward
        {"name": "axes_step", "op": "axes", "dir": "both", "B": 1, "S": 16384, "Hq": 32, "Hk": 32, "D": 128,
         "sections": "16,24,24", "P": 16384, "dtype": "bf16", "interleaved": False},
        # a small map deep in a network: what counts is the launch
        {"name": "gn_fwd_small", "op": "gn", "dir": "fwd", "N": 2, "S": 64, "C": 320, "G": 32, "dtype": "bf16",
         "act": "silu"},
        # odd channels that fill no vector, fp32, no activation: gradients
        {"name": "gn_bwd_odd", "op": "gn", "dir": "bwd", "N": 3, "S": 1021, "C": 250, "G": 25, "dtype": "fp32",
         "act": "none"},
        # a training step's 64 x 64 maps
        {"name": "gn_step", "op": "gn", "dir": "both", "N": 4, "S": 4096, "C": 512, "G": 32, "dtype": "bf16",
         "act": "silu"},
        # the large maps of an image decoder, 256 x 256
        {"name": "gn_step_large", "op": "gn", "dir": "both", "N": 2, "S": 65536, "C": 512, "G": 32, "dtype": "bf16",
         "act": "silu"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "axes", "gn"])
    if op == "cross":
        Hk = rng.choice([1, 2, 4, 8])
        return {"op": "cross", "dir": rng.choice(["fwd", "bwd", "both"]), "B": rng.randint(1, 4),
                "Sq": _log_int(rng, 1, 4096), "Sk": _log_int(rng, 1, 4096), "Hq": Hk * rng.choice([1, 2, 3, 4]),
                "Hk": Hk, "D": rng.choice([40, 64, 80, 96, 128]), "ragged": rng.random() < 0.7,
                "empty": rng.random() < 0.2}
    if op == "axes":
        D = rng.choice([64, 96, 128])
        half = rng.choice([D, D // 2]) // 2
        cuts = sorted(rng.randint(0, half) for _ in range(rng.choice([1, 2, 2, 3])))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [half])]
        Hk = rng.choice([1, 2, 4, 8])
        S = _log_int(rng, 1, 4096)
        return {"op": "axes", "dir": rng.choice(["fwd", "bwd", "both"]), "B": rng.randint(1, 4), "S": S,
                "Hq": Hk * rng.choice([1, 2, 4]), "Hk": Hk, "D": D, "sections": ",".join(map(str, sections)),
                "P": S + rng.randint(0, 4096), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "interleaved": rng.random() < 0.5}
    G = rng.choice([1, 4, 8, 25, 32])
    return {"op": "gn", "dir": rng.choice(["fwd", "bwd", "both"]), "N": rng.randint(1, 8), "S": _log_int(rng, 1, 16384),
            "C": G * rng.choice([1, 2, 3, 7, 8, 10, 16]), "G": G, "dtype": rng.choice(["bf16", "fp16", "fp32"]),
            "act": rng.choice(["none", "silu"])}


# ---- inputs -------------------------------------------------------------------------------

def _lens(case):
    """The batch's lengths, in some order: the full one, shorter ones, perhaps none at all."""
    B, Sk = case["B"], case["Sk"]
    lens = [Sk - (3 * Sk * b) // (4 * B) if case["ragged"] else Sk for b in range(B)]
    if case["empty"]:
        lens[-1] = 0
    return lens


def _sections(case):
    return [int(x) for x in case["sections"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": case}
    if case["op"] == "cross":
        B, Sq, Sk, Hq, Hk, D = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hk", "D"))
        t = torch.bfloat16
        s["scale"] = 1.0 / math.sqrt(D)
        s["q"] = randn(B, Sq, Hq, D, dtype=t)
        # keys and values are the halves of one projection of the encoder's states
        kv = randn(B, Sk, 2 * Hk, D, dtype=t)
        s["k"], s["v"] = kv[:, :, :Hk], kv[:, :, Hk:]
        s["lens"] = None
        if case["ragged"] or case["empty"]:
            lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
            s["lens"] = lens[torch.randperm(B, generator=g, device="cuda")]
        if case["dir"] != "fwd":
            s["do"] = randn(B, Sq, Hq, D, dtype=t, std=0.1)
        if case["dir"] == "bwd":                     # what the forward left
            o, lse = _cross_plain_forward(s)
            s["o"], s["lse"] = o.to(t), lse
        if own:
            s["ws"] = _lib().new_cross_attn_workspace(B, Sq, Sk, Hq, Hk, D, "cuda")
    elif case["op"] == "axes":
        B, S, Hq, Hk, D, t = case["B"], case["S"], case["Hq"], case["Hk"], case["D"], _TYPES[case["dtype"]]
        sec = _sections(case)
        R = 2 * sum(sec)
        # q and k are the first heads of one fused projection's output
        qkv = randn(B, S, Hq + 2 * Hk, D, dtype=t)
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        s["wq"] = 1 + randn(D, std=0.1)
        s["wk"] = 1 + randn(D, std=0.1)
        # one ladder of frequencies over all pairs, as of sections cut out of a text model's rotation
        inv = torch.pow(10000.0, -torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        ang = torch.arange(case["P"], device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        # patches in rows of a grid, one frame after the other, from some place on
        side = max(1, math.isqrt(max(1, S // 4)))
        i = torch.arange(S, device="cuda")
        grid = torch.stack([i // (side * side), (i // side) % side, i % side] + [i] * max(0, len(sec) - 3))[:len(sec)]
        start = torch.randint(0, case["P"] - S + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = (grid[:, None, :] + start[None]).to(torch.int32).contiguous()          # [axes, B, S]
        s["sections"] = sec
        s["eps"] = 1e-6
        if case["dir"] != "fwd":
            s["dq_out"] = randn(B, S, Hq, D, dtype=t, std=0.1)
            s["dk_out"] = randn(B, S, Hk, D, dtype=t, std=0.1)
            if own:
                s["ws"] = _lib().new_qk_norm_rope_workspace(B, S, Hq, Hk, D, "cuda")
    else:
        N, S, C, G, t = case["N"], case["S"], case["C"], case["G"], _TYPES[case["dtype"]]
        # maps whose channels have means and spreads of their own
        x = torch.randn(N, S, C, generator=g, device="cuda")
        s["x"] = x.mul_(1 + 0.5 * torch.rand(C, generator=g, device="cuda")).add_(randn(C, std=0.7)).to(t)
        del x
        s["w"] = 1 + randn(C, std=0.1)
        s["b"] = randn(C, std=0.1)
        s["eps"] = 1e-5
        if case["dir"] != "fwd":
            s["dy"] = randn(N, S, C, dtype=t, std=0.1)
        if case["dir"] == "bwd":                     # what the forward left
            s["mean"], s["rstd"] = _gn_plain_stats(s)
        if own:
            s["ws"] = _lib().new_group_norm_workspace(N, S, C, G, "cuda")
    return s


# ---- cross attention ------------------------------------------------------------------------

def _cross_hidden(s):
    """[B, 1, 1, Sk]: keys beyond a sequence's length."""
    c = s["case"]
    lens = s["lens"]
    if lens is None:
        lens = torch.full((c["B"],), c["Sk"], device="cuda")
    return (torch.arange(c["Sk"], device="cuda")[None] >= lens[:, None])[:, None, None]


def _cross_heads(s, x):
    """Key or value heads [B, Sk, Hk, D] as [B, Hq, Sk, D] in 32 bits."""
    return x.float().transpose(1, 2).repeat_interleave(s["case"]["Hq"] // s["case"]["Hk"], 1)


def _cross_plain_forward(s):
    q = s["q"].float().transpose(1, 2)
    z = (q @ _cross_heads(s, s["k"]).transpose(2, 3)).mul_(s["scale"])
    z.masked_fill_(_cross_hidden(s), float("-inf"))
    m = z.max(3, keepdim=True).values
    m = torch.where(m == float("-inf"), 0.0, m)
    p = z.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    o = (p @ _cross_heads(s, s["v"])) / torch.where(total == 0, 1.0, total)
    return o.transpose(1, 2).contiguous(), (m + total.log())[..., 0]


def _plain_cross(s):
    c, out, t = s["case"], [], s["q"].dtype
    if c["dir"] != "bwd":
        o, lse = _cross_plain_forward(s)
        out = [o.to(t), lse]
    else:
        o, lse = s["o"].float(), s["lse"]
    if c["dir"] != "fwd":
        B, Sk, Hk, D = c["B"], c["Sk"], c["Hk"], c["D"]
        q, do = s["q"].float().transpose(1, 2), s["do"].float().transpose(1, 2)
        k, v = _cross_heads(s, s["k"]), _cross_heads(s, s["v"])
        p = (q @ k.transpose(2, 3)).mul_(s["scale"])
        p = p.sub_(lse[..., None]).exp_().masked_fill_(_cross_hidden(s), 0.0)
        dv = p.transpose(2, 3) @ do
        ds = (do @ v.transpose(2, 3)).sub_((do * o.transpose(1, 2)).sum(3, keepdim=True)).mul_(p)
        dq = (ds @ k) * s["scale"]
        dk = (ds.transpose(2, 3) @ q) * s["scale"]
        shared = lambda x: x.view(B, Hk, -1, Sk, D).sum(2).transpose(1, 2).to(t)  # noqa: E731
        out += [dq.transpose(1, 2).to(t), shared(dk), shared(dv)]
    return out


def _own_cross(s):
    c, da, out = s["case"], _lib(), []
    if c["dir"] != "bwd":
        o, lse = da.cross_attn_forward(s["q"], s["k"], s["v"], s["scale"], s["lens"], workspace=s["ws"])
        out = [o, lse]
    else:
        o, lse = s["o"], s["lse"]
    if c["dir"] != "fwd":
        out += da.cross_attn_backward(s["q"], s["k"], s["v"], o, s["do"], lse, s["scale"], s["lens"],
                                      workspace=s["ws"], check=False)
    return out


# ---- norm and rotation over several axes ------------------------------------------------------

def _pairs(x, R, interleaved):
    return (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])


def _joined(a, b, rest, interleaved):
    ab = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _plain_axes(s):
    c, out, il = s["case"], [], s["case"]["interleaved"]
    R = 2 * sum(s["sections"])
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"))
    pos = s["pos"].long()[axis].permute(1, 2, 0)                    # [B, S, pairs]
    cos, sin = s["cos"].expand(1, 1, -1, -1), s["sin"].expand(1, 1, -1, -1)
    pair = torch.arange(R // 2, device="cuda")
    cos, sin = cos[0, 0][pos, pair][:, :, None], sin[0, 0][pos, pair][:, :, None]
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


def _own_axes(s):
    c, out, da = s["case"], [], _lib()
    if c["dir"] != "bwd":
        out += da.qk_norm_rope_axes_forward(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"],
                                            s["sections"], eps=s["eps"], interleaved=c["interleaved"])
    if c["dir"] != "fwd":
        out += da.qk_norm_rope_axes_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["wq"], s["wk"], s["cos"],
                                             s["sin"], s["pos"], s["sections"], eps=s["eps"],
                                             interleaved=c["interleaved"], workspace=s["ws"], check=False)
    return out


# ---- group norm with an activation ------------------------------------------------------------

def _gn_plain_stats(s):
    c, x = s["case"], s["x"].float()
    x = x.view(c["N"], c["S"], c["G"], -1)
    mean = x.mean((1, 3), keepdim=True)
    var = (x - mean).square().mean((1, 3))
    return mean[:, 0, :, 0].contiguous(), torch.rsqrt(var + s["eps"])


def _plain_gn(s):
    c, out = s["case"], []
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    if c["dir"] != "bwd":
        mean, rstd = _gn_plain_stats(s)
    else:
        mean, rstd = s["mean"], s["rstd"]
    m, r = (t.repeat_interleave(C // G, 1)[:, None] for t in (mean, rstd))
    xh = (s["x"].float() - m) * r
    z = xh * s["w"] + s["b"]
    if c["dir"] != "bwd":
        y = z / (1 + (-z).exp()) if c["act"] == "silu" else z
        out += [y.to(s["x"].dtype), mean, rstd]
    if c["dir"] != "fwd":
        dz = s["dy"].float()
        if c["act"] == "silu":
            sg = 1 / (1 + (-z).exp())
            dz = dz * sg * (1 + z * (1 - sg))
        db, dw = dz.sum((0, 1)), (dz * xh).sum((0, 1))
        dn = dz * s["w"]
        over = lambda t: t.view(N, S, G, -1).mean((1, 3)).repeat_interleave(C // G, 1)[:, None]  # noqa: E731
        dx = (dn - over(dn) - xh * over(dn * xh)) * r
        out += [dx.to(s["x"].dtype), dw, db]
    return out


def _own_gn(s):
    c, out, da = s["case"], [], _lib()
    if c["dir"] != "bwd":
        y, mean, rstd = da.group_norm_act_forward(s["x"], s["w"], s["b"], c["G"], eps=s["eps"], activation=c["act"],
                                                  workspace=s["ws"])
        out += [y, mean, rstd]
    else:
        mean, rstd = s["mean"], s["rstd"]
    if c["dir"] != "fwd":
        out += da.group_norm_act_backward(s["dy"], s["x"], s["w"], s["b"], mean, rstd, c["G"], activation=c["act"],
                                          workspace=s["ws"])
    return out


def run(state):
    f = {"cross": (_plain_cross, _own_cross), "axes": (_plain_axes, _own_axes), "gn": (_plain_gn, _own_gn)}
    return f[state["case"]["op"]][1 if own else 0](state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "cross":
        B, Sq, Hq, Hk, D = case["B"], case["Sq"], case["Hq"], case["Hk"], case["D"]
        keys = sum(_lens(case))
        rows, kv = B * Sq * Hq * D * 2, keys * Hk * D * 2
        pairs = Sq * keys * Hq
        b = f = 0
        if case["dir"] != "bwd":
            b += 2 * rows + 2 * kv + 4 * B * Sq * Hq
            f += 4 * pairs * D
        if case["dir"] != "fwd":
            # q, o, do and dq; k, v, dk and dv (zeros behind the lengths too); the scores are not kept
            b += 4 * rows + 2 * kv + 2 * B * case["Sk"] * Hk * D * 2 + 4 * B * Sq * Hq
            f += 10 * pairs * D
        return {"bytes": b, "flops": f}
    if op == "axes":
        rows, e = case["B"] * case["S"] * (case["Hq"] + case["Hk"]), _BYTES[case["dtype"]]
        sec = _sections(case)
        D, R = case["D"], 2 * sum(sec)
        tab = case["B"] * case["S"] * (4 * len(sec) + R * 4) + 8 * D
        b = f = 0
        if case["dir"] != "bwd":
            b += 2 * rows * D * e + tab
            f += rows * (4 * D + 3 * R)
        if case["dir"] != "fwd":
            b += 3 * rows * D * e + tab + 8 * D
            f += rows * (11 * D + 3 * R)
        return {"bytes": b, "flops": f}
    n, e = case["N"] * case["S"] * case["C"], _BYTES[case["dtype"]]
    b = f = 0
    if case["dir"] != "bwd":
        # the statistics are known only when all of a group has been read: one read would do where a
        # sample stays on the chip
        b += 2 * n * e + 8 * case["C"] + 8 * case["N"] * case["G"]
        f += 8 * n
    if case["dir"] != "fwd":
        b += 3 * n * e + 16 * case["C"] + 8 * case["N"] * case["G"]
        f += 20 * n
    return {"bytes": b, "flops": f}


# ---- the definitions in 64 bits -------------------------------------------------------------

def _exact_cross(case, s):
    B, Sq, Sk, Hq, Hk, D = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hk", "D"))
    fwd, bwd = case["dir"] != "bwd", case["dir"] != "fwd"
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(B, Sq, Hq, D, **f64), torch.full((B, Hq, Sq), -math.inf, **f64)
    dq, dk, dv = torch.zeros(B, Sq, Hq, D, **f64), torch.zeros(B, Sk, Hk, D, **f64), torch.zeros(B, Sk, Hk, D, **f64)
    lens = [Sk] * B if s["lens"] is None else s["lens"].tolist()
    for b in range(B):
        n = lens[b]                                  # only the keys that count are looked at
        if n == 0:
            continue
        for h in range(Hq):
            kh = h * Hk // Hq
            k, v = s["k"][b, :n, kh].double(), s["v"][b, :n, kh].double()
            for t in range(0, Sq, 4096):
                at = slice(t, t + 4096)
                q = s["q"][b, at, h].double()
                z = torch.einsum("id,jd->ij", q, k) * s["scale"]
                if fwd:
                    lse[b, h, at] = torch.logsumexp(z, 1)
                    o[b, at, h] = torch.softmax(z, 1) @ v
                if bwd:
                    if fwd:
                        p, oh = torch.softmax(z, 1), o[b, at, h]
                    else:
                        p, oh = torch.exp(z - s["lse"][b, h, at].double()[:, None]), s["o"][b, at, h].double()
                    d = s["do"][b, at, h].double()
                    dv[b, :n, kh] += p.t() @ d
                    ds = p * (d @ v.t() - (d * oh).sum(1, keepdim=True)) * s["scale"]
                    dq[b, at, h] = ds @ k
                    dk[b, :n, kh] += ds.t() @ q
    return ([o, lse] if fwd else []) + ([dq, dk, dv] if bwd else [])


def _exact_axes(case, s):
    outs, dxs, dws = [], [], []
    D, half = case["D"], sum(s["sections"])
    c = torch.empty(case["B"], case["S"], half, dtype=torch.float64, device="cuda")
    sn = torch.empty_like(c)
    at = 0
    for a, n in enumerate(s["sections"]):
        c[..., at:at + n] = s["cos"].double()[s["pos"][a].long(), at:at + n]
        sn[..., at:at + n] = s["sin"].double()[s["pos"][a].long(), at:at + n]
        at += n
    i = torch.arange(half, device="cuda")
    lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    for name in ("q", "k"):
        w, x = s["w" + name].double(), s[name]
        y_all = torch.empty(x.shape, dtype=torch.float64, device="cuda") if case["dir"] != "bwd" else None
        dx = torch.empty(x.shape, dtype=torch.float64, device="cuda") if case["dir"] != "fwd" else None
        dw = torch.zeros(D, dtype=torch.float64, device="cuda")
        for h in range(x.shape[2]):
            xh = x[:, :, h].double()
            r = 1.0 / torch.sqrt(xh.square().sum(-1, keepdim=True) / D + s["eps"])
            if y_all is not None:
                y = xh * r * w
                z = y.clone()
                z[..., lo] = y[..., lo] * c - y[..., hi] * sn
                z[..., hi] = y[..., lo] * sn + y[..., hi] * c
                y_all[:, :, h] = z
            if dx is not None:
                d = s["d%s_out" % name][:, :, h].double()
                dy = d.clone()
                dy[..., lo] = d[..., lo] * c + d[..., hi] * sn
                dy[..., hi] = d[..., hi] * c - d[..., lo] * sn
                dw += (dy * xh * r).sum((0, 1))
                u = w * dy
                dx[:, :, h] = r * u - xh * r.pow(3) * (u * xh).sum(-1, keepdim=True) / D
        if y_all is not None:
            outs.append(y_all)
        if dx is not None:
            dxs.append(dx)
            dws.append(dw)
    return outs + dxs + dws


def _exact_gn(case, s):
    N, S, C, G = case["N"], case["S"], case["C"], case["G"]
    per, f64 = C // G, dict(dtype=torch.float64, device="cuda")
    fwd, bwd = case["dir"] != "bwd", case["dir"] != "fwd"
    y, dx = (torch.empty(N, S, C, **f64) if on else None for on in (fwd, bwd))
    mean, rstd = torch.empty(N, G, **f64), torch.empty(N, G, **f64)
    dw, db = torch.zeros(C, **f64), torch.zeros(C, **f64)
    for n in range(N):
        for g in range(G):
            at = slice(g * per, g * per + per)
            x = s["x"][n, :, at].double()
            if fwd:
                m = x.sum() / x.numel()
                r = 1.0 / torch.sqrt((x - m).pow(2).sum() / x.numel() + s["eps"])
                mean[n, g], rstd[n, g] = m, r
            else:
                m, r = s["mean"][n, g].double(), s["rstd"][n, g].double()
            w, b = s["w"][at].double(), s["b"][at].double()
            xh = (x - m) * r
            z = xh * w + b
            if fwd:
                y[n, :, at] = z * torch.sigmoid(z) if case["act"] == "silu" else z
            if bwd:
                d = s["dy"][n, :, at].double()
                if case["act"] == "silu":
                    e = torch.exp(-z)
                    d = d * (1 + e + z * e) / (1 + e).pow(2)
                db[at] += d.sum(0)
                dw[at] += (d * xh).sum(0)
                u = d * w
                dx[n, :, at] = r * (u - (u.sum() + xh * (u * xh).sum()) / x.numel())
    return ([y, mean, rstd] if fwd else []) + ([dx, dw, db] if bwd else [])


def exact(case, seed):
    s = prepare(case, seed)
    return {"cross": _exact_cross, "axes": _exact_axes, "gn": _exact_gn}[case["op"]](case, s)
