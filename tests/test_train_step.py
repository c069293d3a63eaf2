"""GPU: the training-step operators run together with the attention, as the example has them:
its gradients against float64 autograd, its loss goes down and a second run has equal bits."""
import importlib.util
import math
import os

import pytest
import torch

import reproducible_deterministic_attn_gb300 as da
from tests._lib import ensure_built, has_gpu

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not has_gpu(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    ensure_built()
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_loss_falls_and_runs_are_equal(example):
    a, pa = example.train(12)
    b, pb = example.train(12)
    assert a == b and all(torch.equal(pa[n], pb[n]) for n in pa)
    assert a[-1] < a[0] - 0.5


def test_step_gradients_match_float64_autograd(example):
    model = example.Model(500, 128, 2, seed=3)
    tr = example.Trainer(model, 1, 128, lr=0.0, max_norm=math.inf)
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(0, 500, (1, 128), generator=g, device="cuda")
    y = torch.randint(0, 500, (1, 128), generator=g, device="cuda")
    y[0, :9] = -100
    loss, _ = tr.step(ids, y)
    tr.check()

    p = {n: t.double().requires_grad_() for n, t in model.p.items()}
    H, D, T = 2, 64, 128
    x = p["embed"][ids[0]] * model.scale
    qkv = (x @ p["qkv"].t()).view(T, 3 * H, D)

    def norm_rope(z, w):
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-6) * w
        a, b = z[..., :D // 2], z[..., D // 2:]
        c, s = tr.cos.double()[:, None], tr.sin.double()[:, None]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    q, k, v = norm_rope(qkv[:, :H], p["wq"]), norm_rope(qkv[:, H:2 * H], p["wk"]), qkv[:, 2 * H:]
    z = torch.einsum("thd,shd->hts", q, k) / math.sqrt(D)
    z = z.masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    o = torch.einsum("hts,shd->thd", torch.softmax(z, -1), v).reshape(T, H * D)
    logits = (x + o @ p["out"].t()) @ p["embed"].t()
    want = torch.nn.functional.cross_entropy(logits, y[0], ignore_index=-100)
    want.backward()
    # activations and their gradients are rounded to bf16 at some ten places on the way; each
    # is 2^-8 of a value at most, and they add up against the largest value of a gradient
    want = float(want.detach())
    assert abs(float(loss) - want) <= 10 * 2.0 ** -8 * want
    for n, t in tr.grads.items():
        err = (t.double() - p[n].grad).abs().max() / p[n].grad.abs().max()
        assert float(err) <= 10 * 2.0 ** -8, (n, float(err))


def test_calls_on_a_given_stream_allocate_there(example):
    """Each call with stream= (a torch stream or its handle), without a workspace and without
    waiting, while other work fills and frees memory on the current stream."""
    g = torch.Generator(device="cuda").manual_seed(9)
    T, V, W = 256, 600, 128
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    table = torch.randn(V, W, generator=g, device="cuda").bfloat16()
    dout = torch.randn(T, W, generator=g, device="cuda").bfloat16()
    qkv = torch.randn(1, T, 6, 64, generator=g, device="cuda").bfloat16()
    q, k = qkv[:, :, :2], qkv[:, :, 2:4]
    dq = torch.randn(1, T, 2, 64, generator=g, device="cuda").bfloat16()
    cos, sin = da.rope_table(T, 64)
    w = torch.ones(64, device="cuda")
    dl = torch.full((T,), 1.0 / T, device="cuda")
    grad = torch.randn(100000, generator=g, device="cuda")

    def run(stream):
        x = da.embed_forward(table, ids, 2.0, stream=stream)
        qk = da.qk_norm_rope_forward(q, k, w, w, cos, sin, stream=stream)
        loss, lse = da.linear_xent_forward(x, table, ids, stream=stream, check=False)
        out = [x, *qk, loss, lse]
        out += da.linear_xent_backward(x, table, ids, lse, dl, stream=stream, check=False)
        out += da.qk_norm_rope_backward(dq, dq, q, k, w, w, cos, sin, stream=stream, check=False)
        out.append(da.embed_backward(dout, ids, V, 2.0, stream=stream, check=False))
        clipped = torch.empty_like(grad)
        plan = da.grad_clip_plan([grad], [clipped], stream=stream)
        out.append(da.grad_clip(plan, 1.0, stream=stream)[0].clone() if stream is None
                   else da.grad_clip(plan, 1.0, stream=stream)[0])
        return out + [clipped]

    want = run(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        got = run(given)
        for _ in range(20):                       # memory that a wrong owner would hand out again
            torch.full((1 << 20,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
