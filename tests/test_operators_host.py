"""Refusals of the operators around the layer, without a GPU: the C entries'
argument checks on placeholder addresses that must be rejected before anything
is launched, and the binding's checks of tensors."""
import ctypes

import pytest
import torch

no_device = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="placeholder pointers: host-only test")
P = ctypes.c_void_p
A = 1 << 12  # an aligned placeholder


@pytest.fixture(scope="module")
def lib():
    from router_experts_gb300 import build, moe
    build.build()
    return moe.load()


def norm(lib, x=A, x_dt=0, res=A, res_dt=0, w=A, w_dt=0, eps=1e-6, T=4, H=64, ro=A, y=A, c=None,
         s=None):
    return lib.moe_add_rms_norm(P(x), x_dt, P(res), res_dt, P(w), w_dt, eps, T, H, P(ro), P(y),
                                P(c), P(s), None)


@no_device
def test_norm_refusals(lib):
    assert norm(lib, x_dt=2) == 2 and norm(lib, w_dt=3) == 2 and norm(lib, res_dt=2) == 2
    assert norm(lib, T=-1) == 1 and norm(lib, H=0) == 1
    assert norm(lib, eps=-1.0) == 1 and norm(lib, eps=float("nan")) == 1
    assert norm(lib, x=None) == 1 and norm(lib, w=None) == 1
    assert norm(lib, y=None) == 1                       # nothing to write
    assert norm(lib, ro=None) == 1 and norm(lib, res=None) == 1
    assert norm(lib, c=A) == 1 and norm(lib, s=A) == 1  # codes and scales come together
    assert norm(lib, H=40, c=A, s=A) == 1               # part of a scale group
    assert norm(lib, x=A + 1) == 1                      # not aligned to its element
    assert norm(lib, x_dt=1, x=A + 2) == 1
    assert norm(lib, x=A + 2, c=A, s=A) == 1            # codes want 16-byte bases
    assert norm(lib, c=A + 8, s=A) == 1
    assert norm(lib, T=0) == 0


def linear(lib, x=A, w=A, b=None, act=0, res=None, res_dt=0, T=4, K=64, N=32, out=A, out_dt=0,
           ws=A, nbytes=1 << 40):
    return lib.moe_linear(P(x), P(w), P(b), act, P(res), res_dt, T, K, N, P(out), out_dt, P(ws),
                          nbytes, None)


@no_device
def test_linear_refusals(lib):
    assert linear(lib, K=60) == 1 and linear(lib, K=0) == 1 and linear(lib, N=0) == 1
    assert linear(lib, T=-1) == 1
    assert linear(lib, act=4) == 1 and linear(lib, act=-1) == 1
    assert linear(lib, act=3, N=1 << 30) == 1           # 2N past 32 bits
    assert linear(lib, out_dt=2) == 2 and linear(lib, res=A, res_dt=3) == 2
    for name in ("x", "w", "out", "ws"):
        assert linear(lib, **{name: None}) == 1
    assert linear(lib, x=A + 8) == 1 and linear(lib, w=A + 8) == 1
    assert linear(lib, out=A + 1) == 1 and linear(lib, res=A + 1) == 1 and linear(lib, b=A + 2) == 1
    assert linear(lib, out=A + 2, out_dt=1) == 1
    assert linear(lib, ws=A + 128) == 1
    assert linear(lib, T=0) == 0
    assert lib.moe_linear_workspace_bytes(4, 60, 32, 0) == 0
    assert lib.moe_linear_workspace_bytes(4, 64, 32, 0) > 0
    assert linear(lib, nbytes=1024) == 1


def balance(lib, logits=A, dt=1, ids=A, mask=None, starts=None, B=1, T=4, E=16, k=2, sc=0,
            coef=1.0, loss=A, counts=A, tokens=A, dl=A, ws=A, nbytes=1 << 40):
    return lib.moe_balance_loss(P(logits), dt, P(ids), P(mask), P(starts), B, T, E, k, sc, coef,
                                P(loss), P(counts), P(tokens), P(dl), P(ws), nbytes, None)


@no_device
def test_balance_refusals(lib):
    assert balance(lib, dt=2) == 2
    assert balance(lib, E=513) == 1 and balance(lib, E=0) == 1 and balance(lib, T=-1) == 1
    assert balance(lib, k=0) == 1 and balance(lib, k=17, E=32) == 1 and balance(lib, k=3, E=2) == 1
    assert balance(lib, sc=3) == 1 and balance(lib, coef=float("nan")) == 1
    assert balance(lib, B=0, starts=A) == 1 and balance(lib, B=2) == 1  # sequences without starts
    assert balance(lib, B=65537, starts=A) == 1
    assert balance(lib, T=1 << 28, k=16, E=16) == 1     # T * k past 32 bits
    for name in ("logits", "ids", "loss", "counts", "tokens", "ws"):
        assert balance(lib, **{name: None}) == 1
    assert balance(lib, logits=A + 2) == 1 and balance(lib, dl=A + 2) == 1
    assert balance(lib, ids=A + 2) == 1 and balance(lib, starts=A + 2, B=2) == 1
    assert balance(lib, ws=A + 64) == 1 and balance(lib, nbytes=1024) == 1

    def back(dloss=A, logits=A, dt=1, counts=A, tokens=A, B=1, T=4, E=16, sc=0, dl=A):
        return lib.moe_balance_loss_backward(P(dloss), P(logits), dt, P(counts), P(tokens), None,
                                             None, B, T, E, sc, 1.0, P(dl), None)
    for name in ("dloss", "logits", "counts", "tokens", "dl"):
        assert back(**{name: None}) == 1
    assert back(dt=3) == 2 and back(E=600) == 1 and back(B=3) == 1
    assert back(T=0) == 0
    assert lib.moe_balance_loss_workspace_bytes(4, 600, 1) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    from router_experts_gb300 import moe
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.add_rms_norm(x, torch.ones(64), None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.linear(x, torch.zeros((8, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.balance_loss(torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32), 1.0)
    with pytest.raises(ValueError, match="nothing to write"):
        moe.add_rms_norm(x, torch.ones(64), None, y=False)
    with pytest.raises(ValueError, match="groups of 32"):
        moe.add_rms_norm(x[:, :40], torch.ones(40), None, e4m3=True)
    with pytest.raises(ValueError, match="gate rows"):
        moe.linear(x, torch.zeros((7, 64), dtype=torch.bfloat16), activation="swiglu")
    with pytest.raises(ValueError, match="matrix"):
        moe.linear(x[0], x)


def test_balance_header_word_matches_the_binding():
    import os
    import re
    from router_experts_gb300 import moe
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "moe.h")).read()
    defs = dict(re.findall(r"#define\s+(MOE_WS_\w+)\s+(\d+)", src))
    assert int(defs["MOE_WS_BALANCE_BARRIER_OFFSET"]) == moe.WS_BALANCE_BARRIER_OFFSET


@pytest.mark.gpu
def test_binding_refuses_what_the_kernels_cannot_hold():
    from router_experts_gb300 import moe
    d, bf = "cuda", torch.bfloat16
    x = torch.zeros((4, 64), dtype=bf, device=d)
    w = torch.ones(64, device=d)
    for bad in (torch.ones(63, device=d), torch.ones(128, device=d)[::2], w.half(), w.cpu()):
        with pytest.raises(ValueError):
            moe.add_rms_norm(x, bad, None)
    with pytest.raises(ValueError, match="shape"):
        moe.add_rms_norm(x, w, torch.zeros((3, 64), dtype=bf, device=d))
    with pytest.raises(ValueError, match="exactly"):
        moe.add_rms_norm(x, w, None, out=(x, x, None, None))
    m = torch.zeros((8, 64), dtype=bf, device=d)
    with pytest.raises(ValueError, match="shape"):
        moe.linear(x, torch.zeros((8, 72), dtype=bf, device=d))
    with pytest.raises(ValueError, match="contiguous"):
        moe.linear(torch.zeros((64, 4), dtype=bf, device=d).t(), m)
    with pytest.raises(ValueError, match="shape"):
        moe.linear(x, m, torch.zeros(7, device=d))
    with pytest.raises(ValueError, match="dtype"):
        moe.linear(x, m, torch.zeros(8, dtype=bf, device=d))
    with pytest.raises(ValueError, match="shape"):
        moe.linear(x, m, out=torch.zeros((4, 9), dtype=bf, device=d))
    with pytest.raises(moe.MoeError):
        moe.linear(x[:, :60].contiguous(), m[:, :60].contiguous())
    lg, ids = torch.zeros((4, 8), device=d), torch.zeros((4, 2), dtype=torch.int32, device=d)
    for kw in ({"token_mask": torch.ones(3, dtype=torch.bool, device=d)},
               {"seq_starts": torch.zeros(1, dtype=torch.int32, device=d)},
               {"seq_starts": torch.zeros(3, dtype=torch.int64, device=d)}):
        with pytest.raises(ValueError):
            moe.balance_loss(lg, ids, 1.0, **kw)
    with pytest.raises(ValueError):
        moe.balance_loss(lg, ids.long(), 1.0)
    with pytest.raises(ValueError):
        moe.balance_loss(lg, ids[:3], 1.0)
