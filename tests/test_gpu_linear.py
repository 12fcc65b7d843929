"""moe.linear against the formula in 64 bits.

Tolerances.  Products of bf16 are exact in 32 bits; the sum takes K / 16
steps of the tensor core, each of which may cut the running sum and its 16
addends at 2^-23, and the splits and the bias a few more: v is off by at most
dv = (K/16 + 24) 2^-23 sum|x w| (+ |bias|).  The activations have slopes
below 1.13; swiglu carries the error of each factor times the other.  Their
own evaluation is good to 2^-20, the residual's addition to 2^-24, and the
result is rounded once to its type.  Beside that worst case, 32-bit outputs
are held to 1e-5 in the 2-norm."""
import pytest
import torch

from router_experts_gb300 import moe

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(T, K, N, act=None, bias=False, res=None, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows = 2 * N if act == "swiglu" else N
    x = torch.randn((T, K), generator=g, device="cuda").to(BF16)
    w = (torch.randn((rows, K), generator=g, device="cuda") * 1.5 / K ** 0.5).to(BF16)
    b = torch.randn(rows, generator=g, device="cuda") if bias else None
    r = torch.randn((T, N), generator=g, device="cuda").to(res) if res is not None else None
    return x, w, b, r


def reference(x, w, b, act, r):
    """-> (output, tolerance before its rounding), both in 64 bits."""
    xd, wd = x.double(), w.double()
    v = xd @ wd.t()
    dv = (xd.abs() @ wd.abs().t()) * (x.shape[1] / 16 + 24) * 2.0 ** -23
    if b is not None:
        v = v + b.double()
        dv = dv + b.double().abs() * 2.0 ** -23
    if act == "swiglu":
        n = w.shape[0] // 2
        g, u, dg, du = v[:, :n], v[:, n:], dv[:, :n], dv[:, n:]
        o = g * torch.sigmoid(g) * u
        tol = 1.13 * dg * u.abs() + (g * torch.sigmoid(g)).abs() * du + 1.13 * dg * du
    else:
        o, tol = v, 1.13 * dv
        if act == "silu":
            o = v * torch.sigmoid(v)
        elif act == "gelu":
            o = v * torch.special.ndtr(v)
    tol = tol + o.abs() * 2.0 ** -20 + 1e-30
    if r is not None:
        o = o + r.double()
        tol = tol + o.abs() * 2.0 ** -23
    return o, tol


def check(got, x, w, b, act, r):
    o, tol = reference(x, w, b, act, r)
    err = (got.double() - o).abs()
    half = torch.finfo(got.dtype).eps / 2
    bad = err > tol + (o.abs() + tol) * half
    assert not bad.any(), (int(bad.sum()), float(err.max()), bad.nonzero()[:4].tolist())
    if got.dtype == F32 and o.numel():
        assert float(err.norm() / o.norm()) <= 1e-5


ACTS = [None, "silu", "gelu", "swiglu"]


@pytest.mark.parametrize("T,K,N", [
    (1, 8, 1), (1, 64, 128), (2, 72, 3), (3, 8, 257), (16, 128, 130), (17, 200, 64),
    (33, 2048, 96), (64, 1000, 500), (65, 512, 128), (100, 64, 1000), (127, 4088, 31),
    (128, 256, 256), (129, 136, 129), (255, 512, 384), (256, 448, 512), (257, 520, 300),
    (300, 7168, 65), (513, 320, 640), (1023, 1000, 777)])
@pytest.mark.parametrize("act", ACTS)
def test_shapes(T, K, N, act):
    x, w, b, _ = make(T, K, N, act, bias=True, seed=T + N)
    check(moe.linear(x, w, b, act), x, w, b, act, None)


@pytest.mark.parametrize("T", [1, 16, 40, 100, 300, 2000])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_long_sums_in_32_bits(T, act):
    # a chain of 8192 terms on the tensor core is 9e-6 low; in pieces of 512 it
    # is half a part in a million (twice that for the product of two such sums)
    x, w, _, _ = make(T, 8192, 640, act, seed=T)
    got = moe.linear(x, w, None, act, out_dtype=F32).double()
    o, _ = reference(x, w, None, act, None)
    assert float((got - o).norm() / o.norm()) <= (2e-6 if act else 1e-6)


@pytest.mark.parametrize("T", [1, 2, 4, 5, 8, 15, 24, 48, 96, 200, 400, 640, 1100])
@pytest.mark.parametrize("K,N", [(7168, 256), (2048, 768)])
def test_tokens(T, K, N):
    for act in (None, "swiglu"):
        x, w, b, r = make(T, K, N, act, res=BF16, seed=T)
        check(moe.linear(x, w, None, act, r), x, w, None, act, r)


@pytest.mark.parametrize("res", [None, BF16, F32])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,K,N", [(1, 512, 200), (70, 768, 333), (260, 256, 520)])
def test_types(res, out, bias, T, K, N):
    for act in ACTS:
        x, w, b, r = make(T, K, N, act, bias, res, seed=7)
        check(moe.linear(x, w, b, act, r, out_dtype=out), x, w, b, act, r)


@pytest.mark.parametrize("T,K,N,act", [(64, 2048, 7168, None), (1, 7168, 2048, "swiglu"),
                                       (512, 7168, 256, None), (2048, 4096, 2048, "swiglu"),
                                       (3000, 2048, 3001, "silu"), (4096, 7168, 512, None)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_larger(T, K, N, act, out):
    x, w, b, r = make(T, K, N, act, True, out, seed=11)
    check(moe.linear(x, w, b, act, r, out_dtype=out), x, w, b, act, r)


def test_residual_in_place():
    for T in (3, 70, 700):
        x, w, b, r = make(T, 512, 384, None, True, BF16, seed=T)
        want = moe.linear(x, w, b, None, r)
        mine = r.clone()
        moe.linear(x, w, b, None, mine, out=mine)
        assert torch.equal(mine, want)


def test_unaligned_output_and_residual():
    # only x and w need 16-byte bases
    for T, N in ((5, 128), (300, 256), (600, 1024)):
        x, w, b, r = make(T, 256, N, None, True, BF16, seed=T)
        out = torch.empty(T * N + 1, dtype=BF16, device="cuda")[1:].view(T, N)
        ru = torch.empty(T * N + 1, dtype=BF16, device="cuda")[1:].view(T, N)
        ru.copy_(r)
        check(moe.linear(x, w, b, None, ru, out=out), x, w, b, None, r)


def test_extreme_values():
    # large and tiny pre-activations, infinities and NaN in the residual
    T, K, N = 20, 64, 96
    x = torch.zeros((T, K), dtype=BF16, device="cuda")
    w = torch.zeros((N, K), dtype=BF16, device="cuda")
    x[:, 0] = 1
    w[:, 0] = torch.linspace(-120, 120, N, device="cuda").to(BF16)
    for act in ("silu", "gelu"):
        check(moe.linear(x, w, None, act, out_dtype=F32), x, w, None, act, None)
    r = torch.zeros((T, N), dtype=BF16, device="cuda")
    r[1, 2], r[3, 4] = float("inf"), float("nan")
    y = moe.linear(x, w, None, None, r)
    assert y[1, 2] == float("inf") and y[3, 4].isnan() and int((~y.isfinite()).sum()) == 2


def test_same_bits_every_time():
    for T in (1, 40, 512):
        x, w, b, _ = make(T, 7168, 256, None, True, seed=2)
        first = moe.linear(x, w, b, out_dtype=F32)
        for _ in range(3):
            assert torch.equal(first, moe.linear(x, w, b, out_dtype=F32))
    assert moe.read_device_error(moe.default_workspace("cuda").buf) == 0


def test_no_tokens():
    x, w, _, _ = make(1, 64, 32)
    assert moe.linear(x[:0], w).shape == (0, 32)


def test_64bit_offsets():
    T, K, N = 300_000, 64, 7168
    assert T * N > 2 ** 31
    x, w, _, _ = make(1, K, N, seed=1)
    x = x.expand(T, K).contiguous()
    x[-3:] = torch.randn((3, K), device="cuda").to(BF16)
    y = moe.linear(x, w)
    check(y[-8:], x[-8:], w, None, None, None)
    check(y[:3], x[:3], w, None, None, None)


def test_other_stream_and_graph():
    for T in (2, 300):
        x, w, b, r = make(T, 2048, 512, "swiglu", True, BF16, seed=5)
        want = moe.linear(x, w, b, "swiglu", r)
        torch.cuda.synchronize()
        out, ws = torch.empty_like(want), moe.Workspace("cuda")
        ws.get(moe.linear_workspace_bytes(T, 2048, 512, "swiglu"))
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            moe.linear(x, w, b, "swiglu", r, ws=ws, out=out)
        st.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.linear(x, w, b, "swiglu", r, ws=ws, out=out)
        x.copy_(x * 2)
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, w, b, "swiglu", r)
