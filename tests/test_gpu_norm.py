"""moe.add_rms_norm against the formula in 64 bits.

Tolerances.  The 32-bit sum s = x + r has one rounding, residual_out one more
to its type.  y: a thread adds at most H/32 squares one after the other and
the rest in a tree, all positive, so the mean is off by at most
(H/32 + 16) 2^-24 relative, its root by half of that, and the remaining
operations add a few 2^-24; then one rounding to bf16 (2^-8) or e4m3 (2^-4,
or half a subnormal step, 2^-10)."""
import pytest
import torch

from router_experts_gb300 import moe

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(T, H, x_dt=BF16, res_dt=BF16, w_dt=BF16, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn((T, H), generator=g, device="cuda") * 0.7).to(x_dt)
    r = None
    if res_dt is not None:
        r = (torch.randn((T, H), generator=g, device="cuda") * 3).to(res_dt)
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(w_dt)
    return x, r, w


def y_err(H):
    return (H / 64 + 16) * 2.0 ** -24


def reference(x, r, w, eps):
    s = x.double() if r is None else x.double() + r.double()
    return s, s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * w.double()


def decode(codes, scales):
    c = codes.view(torch.float8_e4m3fn).double()
    p = torch.exp2(scales.double() - 127)
    return c * p.repeat_interleave(32, dim=1), p


def check(x, r, w, eps, got):
    T, H = x.shape
    s, y = reference(x, r, w, eps)
    ro, yo, codes, scales = got
    if r is not None:
        half = torch.finfo(r.dtype).eps / 2
        assert ((ro.double() - s).abs() <= s.abs() * (half + 2.0 ** -23)).all()
    if yo is not None:
        assert ((yo.double() - y).abs() <= y.abs() * (2.0 ** -8 + y_err(H)) + 1e-38).all()
    if codes is not None:
        v, p = decode(codes, scales)
        p32 = p.repeat_interleave(32, dim=1)
        off = torch.maximum(y.abs() * 2.0 ** -4, p32 * 2.0 ** -10) + y.abs() * y_err(H)
        assert ((v - y).abs() <= off).all()
        # the scale is the smallest power of two with amax / 2^p <= 448
        amax = y.view(T, H // 32, 32).abs().amax(2)
        live = amax > 0
        assert (amax <= 448 * p * (1 + y_err(H)))[live].all()
        low = live & (scales > 0)
        assert (amax > 224 * p * (1 - y_err(H)))[low].all()
        assert (scales[~live] == 127).all() and (codes.view(T, H // 32, 32)[~live] == 0).all()


@pytest.mark.parametrize("T,H", [
    (1, 1), (3, 2), (5, 7), (2, 8), (9, 31), (4, 40), (7, 64), (3, 257), (33, 1000), (5, 1001),
    (130, 2045), (1, 2048), (64, 4096), (2, 4100), (700, 4096), (1, 7168), (5, 7168), (300, 7168),
    (3, 8200), (2, 9001), (2, 16384), (2, 20008), (3, 40000), (1, 70001), (700, 2048),
    (1300, 7168), (620, 16384), (640, 32768), (2000, 2001), (1500, 1031), (500, 8193)])
def test_rows(T, H):
    x, r, w = make(T, H, seed=T + H)
    check(x, r, w, 1e-6, moe.add_rms_norm(x, w, r, 1e-6))


@pytest.mark.parametrize("x_dt", [BF16, F32])
@pytest.mark.parametrize("res_dt", [None, BF16, F32])
@pytest.mark.parametrize("w_dt", [BF16, F32])
@pytest.mark.parametrize("T,H", [(6, 96), (37, 1003), (3, 5120)])
def test_types(x_dt, res_dt, w_dt, T, H):
    x, r, w = make(T, H, x_dt, res_dt, w_dt, seed=H)
    check(x, r, w, 1e-5, moe.add_rms_norm(x, w, r, 1e-5, e4m3=H % 32 == 0))


@pytest.mark.parametrize("T,H", [(1, 32), (3, 64), (2, 96), (17, 1056), (1, 4096), (64, 4096),
                                 (1, 7168), (600, 7168), (1300, 7168), (1250, 4096), (2500, 1056), (2, 8224),
                                 (3, 33024), (3, 40992)])
@pytest.mark.parametrize("y", [False, True])
def test_e4m3(T, H, y):
    x, r, w = make(T, H, seed=T * 7 + H)
    got = moe.add_rms_norm(x, w, r, 1e-6, y=y, e4m3=True)
    assert (got[1] is not None) == y
    check(x, r, w, 1e-6, got)


def test_e4m3_feeds_the_cast_format():
    # where y is exact in bf16 the codes and scales are moe_cast_e4m3's bytes
    T, H = 4, 256
    x = torch.ones((T, H), dtype=BF16, device="cuda")
    w = torch.exp2(torch.randint(-6, 7, (H,), device="cuda").float())
    _, y, codes, scales = moe.add_rms_norm(x, w, None, 0.0, e4m3=True)
    assert torch.equal(y, w.to(BF16).expand(T, H))
    c2, s2 = moe.cast_e4m3(y)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)


def test_unaligned_rows():
    # bases that are no multiple of 16 bytes: the element-wise path
    T, H = 5, 512
    x, r, w = make(T, H + 8, seed=3)
    flat = [torch.empty(T * H + 1, dtype=BF16, device="cuda")[1:].view(T, H) for _ in range(2)]
    flat[0].copy_(x[:, :H])
    flat[1].copy_(r[:, :H])
    w1 = w[1:H + 1]
    got = moe.add_rms_norm(flat[0], w1, flat[1], 1e-6)
    check(flat[0], flat[1], w1, 1e-6, got)
    with pytest.raises(moe.MoeError):
        moe.add_rms_norm(flat[0], w1, flat[1], 1e-6, e4m3=True)


@pytest.mark.parametrize("T,H", [(40, 2048), (40, 2045), (1300, 1003), (2000, 2048), (1400, 7168)])
def test_in_place_residual(T, H):
    x, r, w = make(T, H, seed=9)
    want = moe.add_rms_norm(x, w, r, 1e-6)
    y = torch.empty_like(x)
    mine = r.clone()
    moe.add_rms_norm(x, w, mine, 1e-6, out=(mine, y, None, None))
    assert torch.equal(mine, want[0]) and torch.equal(y, want[1])


@pytest.mark.parametrize("H", [2045, 2048])
def test_zero_nan_and_infinite_rows(H):
    x, r, w = make(6, H, seed=4)
    x[1], r[1] = 0, 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    ro, y, codes, scales = moe.add_rms_norm(x, w, r, 1e-6, e4m3=H % 32 == 0)
    assert (y[1] == 0).all()
    assert y[2].isnan().all()
    assert y[3, 7].isnan() and (torch.cat([y[3, :7], y[3, 8:]]) == 0).all()
    keep = [0, 4, 5]
    check(x[keep], r[keep], w, 1e-6, (ro[keep], y[keep], None, None))
    if codes is not None:
        assert (codes[1] == 0).all() and (scales[1] == 127).all()
        assert codes[2].view(torch.float8_e4m3fn).float().isnan().all()
    # no eps: a zero row is 0 * inf
    assert moe.add_rms_norm(x, w, r, 0.0)[1][1].isnan().all()


def test_no_tokens():
    x, r, w = make(1, 64)
    ro, y, codes, scales = moe.add_rms_norm(x[:0], w, r[:0], 1e-6, e4m3=True)
    assert y.shape == (0, 64) and scales.shape == (0, 2)


def test_64bit_offsets():
    T, H = 300_000, 7168
    assert T * H > 2 ** 31
    x = torch.empty((T, H), dtype=BF16, device="cuda")
    x.copy_(torch.randn((1, H), device="cuda").to(BF16).expand(T, H))
    x[-3:] = torch.randn((3, H), device="cuda").to(BF16)
    _, _, w = make(1, H)
    _, y, codes, scales = moe.add_rms_norm(x, w, None, 1e-6, e4m3=True)
    check(x[-8:], None, w, 1e-6, (None, y[-8:], codes[-8:], scales[-8:]))
    check(x[:2], None, w, 1e-6, (None, y[:2], codes[:2], scales[:2]))


def test_other_stream_and_graph():
    x, r, w = make(64, 4096, seed=5)
    want = moe.add_rms_norm(x, w, r, 1e-6, e4m3=True)
    torch.cuda.synchronize()
    out = tuple(torch.empty_like(t) for t in want)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        moe.add_rms_norm(x, w, r, 1e-6, e4m3=True, out=out)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.add_rms_norm(x, w, r, 1e-6, e4m3=True, out=out)
    x.copy_(x * 2)
    graph.replay()
    torch.cuda.synchronize()
    check(x, r, w, 1e-6, out)
