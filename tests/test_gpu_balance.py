"""moe.balance_loss and its gradient against the definition in 64 bits.

Tolerances.  Counts are whole numbers: equal.  A probability takes an
exponential, a root or a reciprocal (each good to a few 2^-24) and a sum of at
most 512 scores in 32 bits (16 of a lane one after the other, then a tree): 2^-19
relative is more than twice their sum.  The loss adds tokens in pairs of
floats: 2^-18.  In the gradient c d (g_e - sum g p) each part has that error:
2^-18 c d (|g_e| + sum |g| p), and one rounding to the logits' type."""
import pytest
import torch

from router_experts_gb300 import moe

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SCORINGS = ["softmax", "sigmoid", "sqrt_softplus"]
COEF = 0.01


def make(T, E, k, dt=F32, seed=0, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    logits = (torch.randn((T, E), generator=g, device="cuda") * spread
              + torch.randn(E, generator=g, device="cuda")).to(dt)
    ids = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    mask = torch.rand(T, generator=g, device="cuda") < 0.8
    return logits, ids, mask


def starts_of(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def probabilities(l, scoring):
    """p, its derivative's factor d, and 1 - sum p, which 64 bits do not hold
    next to a sum of one."""
    if scoring == "softmax":
        p = torch.softmax(l, 1)
        empty = torch.isneginf(l).all(1, keepdim=True)
        p = torch.where(empty, torch.zeros_like(p), p)
        return p, p, empty.double()
    q = torch.sigmoid(l)
    if scoring == "sigmoid":
        s, ds = q, q * torch.sigmoid(-l)
    else:
        s = torch.sqrt(torch.nn.functional.softplus(l, threshold=1e9))
        ds = torch.where(l < -30, s / 2, q / (2 * s))
    total = s.sum(1, keepdim=True) + 1e-20
    return s / total, ds / total, 1e-20 / total


def reference(logits, ids, scoring, mask=None, starts=None, dloss=1.0):
    l = logits.double()
    T, E = l.shape
    bounds = [0, T] if starts is None else starts.tolist()
    B = len(bounds) - 1
    p, d, rest = probabilities(l, scoring)
    counts = torch.zeros((B, E), dtype=torch.int32, device="cuda")
    tokens = torch.zeros(B, dtype=torch.int32, device="cuda")
    at = []
    for b in range(B):
        i = torch.arange(bounds[b], max(bounds[b], bounds[b + 1]), device="cuda")
        i = i[(i >= 0) & (i < T)]
        if mask is not None:
            i = i[mask[i] != 0]
        at.append(i)
        tokens[b] = i.numel()
        e = ids[i].reshape(-1)
        e = e[(e >= 0) & (e < E)]
        counts[b] = torch.bincount(e.long(), minlength=E)
    Bp = max(1, sum(len(i) > 0 for i in at))
    loss = torch.zeros((), dtype=torch.float64, device="cuda")
    dl, tol = torch.zeros_like(l), torch.zeros_like(l)
    for b, i in enumerate(at):
        if len(i):
            c = counts[b].double()
            f = c * E / c.sum() if c.sum() else torch.zeros_like(c)
            loss += COEF / Bp * (f * p[i]).sum(1).mean()
            coef = COEF / (Bp * len(i)) * abs(dloss) * d[i]
            g = f - 1
            dl[i] = coef * (g - (g * p[i]).sum(1, keepdim=True) + rest[i]) * (1 if dloss >= 0 else -1)
            tol[i] = 2.0 ** -18 * coef * (g.abs() + (g.abs() * p[i]).sum(1, keepdim=True)
                                          + 1e-20)
    return loss, counts, tokens, dl, tol


def check(logits, ids, scoring, mask=None, starts=None):
    got = moe.balance_loss(logits, ids, COEF, scoring, token_mask=mask, seq_starts=starts,
                           grad=True)
    loss, counts, tokens, dl, tol = reference(logits, ids, scoring, mask, starts)
    assert torch.equal(got[1], counts) and torch.equal(got[2], tokens)
    assert abs(float(got[0]) - float(loss)) <= 2.0 ** -18 * abs(float(loss))
    half = torch.finfo(logits.dtype).eps / 2
    err = (got[3].double() - dl).abs()
    assert (err <= tol + dl.abs() * half + 1e-38).all(), float((err - tol).max())
    # without the gradient: the same loss; the backward call: the same gradient
    alone = moe.balance_loss(logits, ids, COEF, scoring, token_mask=mask, seq_starts=starts)
    assert torch.equal(alone[0], got[0]) and torch.equal(alone[1], counts) and alone[3] is None
    dloss = torch.tensor([-2.5], device="cuda")
    back = moe.balance_loss_backward(dloss, logits, counts, tokens, COEF, scoring,
                                     token_mask=mask, seq_starts=starts)
    *_, dl, tol = reference(logits, ids, scoring, mask, starts, dloss=-2.5)
    assert ((back.double() - dl).abs() <= tol + dl.abs() * half + 1e-38).all()
    return got


@pytest.mark.parametrize("scoring", SCORINGS)
@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 2, 1), (1, 8, 2), (5, 3, 3), (7, 31, 4), (16, 32, 16), (33, 33, 2),
    (40, 63, 8), (64, 128, 8), (100, 130, 1), (129, 256, 8), (65, 257, 5), (50, 288, 8),
    (31, 384, 6), (20, 510, 3), (600, 512, 16), (5000, 64, 6)])
def test_shapes(T, E, k, scoring):
    logits, ids, _ = make(T, E, k, seed=T + E)
    check(logits, ids, scoring)


@pytest.mark.parametrize("scoring", SCORINGS)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,E,k", [(77, 96, 4), (300, 61, 3), (1000, 256, 8)])
def test_types_masks_and_sequences(T, E, k, dt, scoring):
    logits, ids, mask = make(T, E, k, dt, seed=T)
    check(logits, ids, scoring, mask)
    for starts in (starts_of(0, T), starts_of(0, 1, 1, T // 2, T),
                   starts_of(3, 10, T - 5), starts_of(0, 0, 0, T // 3, T // 3, T, T)):
        check(logits, ids, scoring, None, starts)
        check(logits, ids, scoring, mask, starts)


def test_many_short_sequences():
    logits, ids, mask = make(3000, 64, 4, seed=8)
    check(logits, ids, "softmax", mask, torch.arange(0, 3001, 3, dtype=torch.int32, device="cuda"))


def test_more_sequences_than_counters():
    # B (E + 1) past the workspace's table, B past the starts in shared memory
    T, E = 9000, 512
    logits, ids, mask = make(T, E, 2, seed=9)
    check(logits, ids, "sigmoid", mask, torch.arange(0, T + 1, 60, dtype=torch.int32, device="cuda"))
    logits, ids, mask = make(T, 16, 2, seed=10)
    check(logits, ids, "softmax", mask, torch.arange(0, T + 1, 5, dtype=torch.int32, device="cuda"))
    check(logits[:40], ids[:40], "softmax", mask[:40],
          torch.arange(0, 41, 1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("T", [97, 500, 513, 1500])
def test_one_cta_cluster_and_grid(T):
    # one CTA up to 96 tokens of this width, one cluster up to 512, then the grid
    logits, ids, mask = make(T, 256, 8, seed=T)
    check(logits, ids, "sigmoid")
    check(logits, ids, "softmax", mask, starts_of(0, T // 3, T // 3 + 2, T))


@pytest.mark.parametrize("scoring", SCORINGS)
def test_nothing_counted(scoring):
    logits, ids, mask = make(50, 16, 2, seed=1)
    mask[:] = False
    got = check(logits, ids, scoring, mask)
    assert float(got[0]) == 0 and not got[3].any() and not got[1].any()
    mask[20:25] = True  # one sequence of three holds tokens
    got = check(logits, ids, scoring, mask, starts_of(0, 10, 30, 50))
    assert got[2].tolist() == [0, 5, 0]


@pytest.mark.parametrize("scoring", SCORINGS)
def test_masked_and_extreme_logits(scoring):
    logits, ids, _ = make(12, 48, 3, seed=6)
    logits[0, :40] = float("-inf")
    logits[1, :40] = torch.finfo(F32).min
    logits[2] = torch.finfo(F32).min
    logits[3] = -60.0
    logits[4, 5] = 80.0
    logits[5] = 30.0
    check(logits, ids, scoring)
    logits[6] = float("-inf")
    got = moe.balance_loss(logits, ids, COEF, scoring, grad=True)
    assert got[0].isfinite() and (got[3][6] == 0).all() and got[3].isfinite().all()


def test_nan_stays_in_its_row():
    logits, ids, _ = make(9, 32, 2, seed=6)
    logits[4, 3] = float("nan")
    for scoring in SCORINGS:
        loss, _, _, dl = moe.balance_loss(logits, ids, COEF, scoring, grad=True)
        assert loss.isnan().all() and dl[4].isnan().all()
        assert dl[:4].isfinite().all() and dl[5:].isfinite().all()
    # a token that is not counted is not read
    mask = torch.ones(9, dtype=torch.uint8, device="cuda")
    mask[4] = 0
    loss, _, _, dl = moe.balance_loss(logits, ids, COEF, token_mask=mask, grad=True)
    assert loss.isfinite().all() and (dl[4] == 0).all()


def test_bad_ids_are_skipped_and_flagged():
    logits, ids, _ = make(30, 16, 2, seed=2)
    ids[3, 1], ids[7, 0] = -1, 16
    ws = moe.Workspace("cuda")
    loss, counts, tokens, _ = moe.balance_loss(logits, ids, COEF, ws=ws)
    want = reference(logits, ids, "softmax")
    assert torch.equal(counts, want[1]) and torch.equal(tokens, want[2])
    assert abs(float(loss) - float(want[0])) <= 2.0 ** -18 * float(want[0])
    assert moe.read_device_error(ws.buf) == moe.DEVERR_BAD_EXPERT_ID


@pytest.mark.parametrize("scoring", SCORINGS)
def test_gradient_against_differences(scoring):
    # the loss in 64 bits at l +- h, the counts held
    logits, ids, mask = make(6, 8, 2, seed=3)
    starts = starts_of(0, 4, 6)
    _, counts, _, dl = moe.balance_loss(logits, ids, COEF, scoring, token_mask=mask,
                                        seq_starts=starts, grad=True)
    *_, tol = reference(logits, ids, scoring, mask, starts)
    h = 1e-4
    for t in range(6):
        for e in range(8):
            pair = []
            for step in (h, -h):
                l = logits.double()
                l[t, e] += step
                pair.append(float(reference(l, ids, scoring, mask, starts)[0]))
            diff = (pair[0] - pair[1]) / (2 * h)
            # the gradient's own tolerance and rounding, and h^2 / 6 times a
            # third derivative below COEF * E
            off = float(tol[t, e]) + abs(diff) * 2.0 ** -23 + COEF * 8 * h * h
            assert abs(diff - float(dl[t, e])) <= off


def test_ids_of_the_router():
    # ids as moe.router gives them, counted as align sees them
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((200, 256), generator=g, device="cuda").to(BF16)
    gate = (torch.randn((32, 256), generator=g, device="cuda") / 16).to(BF16)
    ids, _ = moe.router(x, gate, None, 4)
    logits = moe.linear(x, gate, out_dtype=F32)
    got = check(logits, ids, "softmax")
    assert torch.equal(got[1][0].long(), torch.bincount(ids.reshape(-1).long(), minlength=32))


def test_same_bits_every_time():
    logits, ids, mask = make(20000, 256, 8, seed=2)
    first = moe.balance_loss(logits, ids, COEF, "sigmoid", token_mask=mask, grad=True)
    for _ in range(3):
        again = moe.balance_loss(logits, ids, COEF, "sigmoid", token_mask=mask, grad=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_barrier_wait_expires_and_reports():
    # arrivals preset far below zero never reach the grid's size: the wait runs
    # out (a millisecond by the test hook) and is reported; the tokens' outputs
    # stay as they were, and a zeroed workspace works again
    logits, ids, _ = make(2000, 64, 4, seed=7)
    ws = moe.Workspace("cuda")
    moe.balance_loss(logits, ids, COEF, ws=ws)
    head = ws.buf[:8192]
    head[moe.WS_BALANCE_BARRIER_OFFSET:][:4].view(torch.int32).fill_(-2 ** 30)
    head[moe.WS_WAIT_LIMIT_OFFSET:][:8].view(torch.int64).fill_(2 ** 21)
    out = (torch.full((1,), 7.0, device="cuda"),
           torch.empty((1, 64), dtype=torch.int32, device="cuda"),
           torch.empty(1, dtype=torch.int32, device="cuda"), torch.full_like(logits, 7.0))
    moe.balance_loss(logits, ids, COEF, grad=True, ws=ws, out=out)
    assert moe.read_device_error(ws.buf) == moe.DEVERR_WAIT_TIMEOUT
    assert float(out[0]) == 7 and (out[3] == 7).all()
    ws.buf.zero_()
    loss, counts, tokens, dl, tol = reference(logits, ids, "softmax")
    got = moe.balance_loss(logits, ids, COEF, grad=True, ws=ws)
    assert torch.equal(got[1], counts)
    assert ((got[3].double() - dl).abs() <= tol + dl.abs() * 2.0 ** -24 + 1e-38).all()
    assert moe.read_device_error(ws.buf) == 0


def test_no_tokens():
    logits, ids, _ = make(4, 16, 2)
    loss, counts, tokens, dl = moe.balance_loss(logits[:0], ids[:0], COEF, grad=True)
    assert float(loss) == 0 and not counts.any() and not tokens.any() and dl.shape == (0, 16)


def test_64bit_offsets():
    T, E, k = 4_250_000, 512, 2
    assert T * E > 2 ** 31
    row = torch.randn((1, E), device="cuda").to(BF16)
    logits = row.expand(T, E).contiguous()
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    loss, counts, tokens, dl = moe.balance_loss(logits, ids, COEF, grad=True)
    assert torch.equal(counts[0].long(), torch.bincount(ids.reshape(-1).long(), minlength=E))
    assert int(tokens) == T
    p = torch.softmax(row.double(), 1)
    f = counts.double() * E / (T * k)
    assert abs(float(loss) - COEF * float((f * p).sum())) <= 2.0 ** -18 * float(loss)
    want = COEF / T * p * (f - (f * p).sum())
    for t in (0, T // 2, T - 1):
        tol = 2.0 ** -18 * COEF / T * p * ((f - 1).abs() + ((f - 1).abs() * p).sum())
        assert ((dl[t].double() - want).abs() <= tol + want.abs() * 2.0 ** -8).all()


def test_other_stream_and_graph():
    logits, ids, mask = make(2000, 128, 8, seed=5)
    want = moe.balance_loss(logits, ids, COEF, token_mask=mask, grad=True)
    torch.cuda.synchronize()
    ws = moe.Workspace("cuda")
    ws.get(moe.load().moe_balance_loss_workspace_bytes(2000, 128, 1))
    out = tuple(torch.empty_like(t) for t in want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        moe.balance_loss(logits, ids, COEF, token_mask=mask, grad=True, ws=ws, out=out)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.balance_loss(logits, ids, COEF, token_mask=mask, grad=True, ws=ws, out=out)
    l2, i2, m2 = make(2000, 128, 8, seed=6)
    logits.copy_(l2), ids.copy_(i2), mask.copy_(m2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    want = moe.balance_loss(l2, i2, COEF, token_mask=m2, grad=True)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
