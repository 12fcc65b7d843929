"""The operators together around the MoE layer (examples/moe_block.py), against
plain 64-bit formulas fed the GPU's own routing ids (a near-tie may go either
way).  The layer's tolerances are those of its own tests; h' and y' take one
more bf16 rounding."""
import importlib.util
import os

import pytest
import torch

from router_experts_gb300 import moe
from router_experts_gb300 import workloads as W

from _gpu import LAYER_RTOL_BF16, LAYER_RTOL_LOWBIT

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LOWBIT = W.Workload("lowbit_small", H=256, E=16, k=2, F=128, scoring="sigmoid", bias=True,
                    lowbit=True)


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location(
        "moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def norm(s, w):
    return s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6) * w.double()


def swiglu(v, n):
    return v[:, :n] * torch.sigmoid(v[:, :n]) * v[:, n:]


def dequantise(codes, scales):
    """e2m1 pairs (low nibble first) with a UE8M0 scale per 32 values."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=torch.float64, device="cuda")
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def close(got, want, rtol):
    err = (got.double() - want).abs().max() / want.abs().max()
    assert float(err) <= rtol, float(err)


@pytest.mark.parametrize("w,T,shared", [(W.WORKLOADS["toy"], 16, 40), (W.WORKLOADS["toy"], 1, 32),
                                        (W.WORKLOADS["qwen3"], 33, 768), (LOWBIT, 50, 128)])
def test_block(block, w, T, shared):
    p = block.make_params(w, shared, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    attn, h = (torch.randn((T, w.H), generator=g, device="cuda").to(torch.bfloat16)
               for _ in range(2))
    ws = moe.Workspace("cuda")
    r = block.moe_block(w, p, attn, h, coef=0.1, ws=ws)
    torch.cuda.synchronize()
    assert moe.read_device_error(ws.buf) == 0
    rtol = LAYER_RTOL_LOWBIT if w.lowbit else LAYER_RTOL_BF16

    s = attn.double() + h.double()
    y = norm(s, p["norm_in"])
    close(r["h_in"], s, 2 ** -8)
    assert ((r["layer_in"].double() - y).abs() <= y.abs() * 2.0 ** -7.9).all()
    # from here on the rows that the next operators read
    y, s = r["layer_in"].double(), r["h_in"].double()
    logits = y @ p["gate"].to(torch.bfloat16).double().t()
    close(r["logits"], logits, 1e-5)
    # routed experts, for the ids that the router gave
    x = y
    if w.lowbit:
        _, _, codes, scales = moe.add_rms_norm(attn, p["norm_in"], h, 1e-6, e4m3=True)
        x = (codes.view(torch.float8_e4m3fn).double()
             * torch.exp2(scales.double() - 127).repeat_interleave(32, 1))
        w13, w2 = (dequantise(p[n], p[n + "_scale"]) for n in ("w13", "w2"))
    else:
        w13, w2 = p["w13"].double(), p["w2"].double()
    gate_logits = x @ p["gate"].double().t()
    score = (torch.softmax(gate_logits, 1) if w.scoring == "softmax"
             else torch.sigmoid(gate_logits))
    ids = r["ids"].long()
    wt = score.gather(1, ids)
    wt = wt / wt.sum(1, keepdim=True) * w.scaling
    m = torch.zeros_like(x)
    for j in range(w.k):
        for t in range(T):
            e = ids[t, j]
            m[t] += wt[t, j] * (w2[e] @ swiglu((w13[e] @ x[t])[None], w.F)[0])
    close(r["routed"], m, rtol)
    # the shared expert on top of the routed output as it is
    a = swiglu(y @ p["shared_w13"].double().t(), shared)
    o = a @ p["shared_w2"].double().t() + r["routed"].double()
    close(r["block"], o, LAYER_RTOL_BF16)
    s2 = r["block"].double() + s
    close(r["h"], s2, 2 ** -8)
    y2 = norm(s2, p["norm_out"])
    assert ((r["y"].double() - y2).abs() <= y2.abs() * 2.0 ** -7.9).all()
    # loss, counts and the logits' gradient by automatic differentiation in 64 bits
    counts = torch.bincount(ids.reshape(-1), minlength=w.E)
    assert torch.equal(r["counts"][0].long(), counts)
    l = r["logits"].double().requires_grad_()
    prob = torch.softmax(l, 1) if w.scoring == "softmax" else torch.sigmoid(l)
    prob = prob / prob.sum(1, keepdim=True)
    f = counts.double() * w.E / (T * w.k)
    loss = 0.1 * (f * prob.mean(0)).sum()
    loss.backward()
    want = loss.item()
    assert abs(float(r["loss"]) - want) <= 1e-5 * want
    close(r["dlogits"], l.grad, 1e-5)
    # the gradient goes into the gate like any other
    leaf = r["logits"].clone().requires_grad_()
    leaf.backward(r["dlogits"])
    assert torch.equal(leaf.grad, r["dlogits"])


def test_block_in_a_graph(block):
    w = W.WORKLOADS["qwen3"]
    p = block.make_params(w, 768, seed=2)
    ws = moe.Workspace("cuda")
    ws.get(moe.layer_workspace_bytes(40, w.H, w.F, w.E, w.k))
    attn, h = (torch.randn((40, w.H), device="cuda").to(torch.bfloat16) for _ in range(2))
    eager = block.moe_block(w, p, attn, h, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = block.moe_block(w, p, attn, h, ws=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for k in eager:
        assert torch.equal(eager[k], captured[k]), k
    assert moe.read_device_error(ws.buf) == 0
