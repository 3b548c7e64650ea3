"""The gated feed-forward block, the cross entropy of a quantized head and the backward
passes through quantized weights (libhqq_layers.so) against their definitions in 64 bits.

Bounds.  W_hat is the dtype's rounding of an fp32 quotient, the same on both sides.
Products of 16-bit values are exact in fp32, so a kernel's fp32 sum of R products is within
R 2^-24 times the sum of their magnitudes (any order; 1.01 covers the higher orders).  An
output's rounding adds half a step, eps / 2 of its size (fp16 2^-11, bf16 2^-8), and below
fp16's normal range 2^-25.  The elementary functions (exp2, reciprocal and erfc of an
fp32 argument z) are within (8 + 2 |z|) 2^-24, at most 2^-16 for |z| <= 120 where their
values still count.  What a call rounds in between is said at its bound.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
FN = 2.0 ** -16
DTYPES = [torch.float16, torch.bfloat16]
PER_WORD = {8: 4, 4: 8, 2: 16, 1: 32}


@pytest.fixture(scope="module")
def hq():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import weight_quantization_group_amd as w

    w.load_layers_library()
    return w


@pytest.fixture(params=["codes", "tiled"])
def path(request, monkeypatch):
    """Each route in turn, whatever the sizes: straight from the codes, and the tiled product."""
    monkeypatch.setenv("HQQ_LAYERS_PATH", request.param)
    return request.param


def make_weight(seed, N, K, nbits, gs, dtype, std=None):
    """((packed, scale, zero) on the GPU, W_hat in 64 bits on the GPU) of random codes."""
    rng = np.random.RandomState(seed)
    qmax = (1 << nbits) - 1
    q = rng.randint(0, qmax + 1, size=(N, K)).astype(np.uint32)
    std = std or 1.0 / math.sqrt(K)
    lo = -np.abs(rng.normal(2, 0.5, (N, K // gs))) * std
    hi = np.abs(rng.normal(2, 0.5, (N, K // gs))) * std + 1e-3 * std
    scale = (qmax / (hi - lo)).astype(np.float32)
    zero = (-lo * scale).astype(np.float32)
    C = PER_WORD[nbits]
    shifts = (np.arange(C) * nbits).astype(np.uint32)
    words = np.bitwise_or.reduce(q.reshape(N, K // C, C) << shifts, axis=2).astype(np.uint32)
    w32 = (q.astype(np.float32) - np.repeat(zero, gs, 1)) / np.repeat(scale, gs, 1)
    what = torch.from_numpy(w32).to(dtype).double().cuda()
    return (torch.from_numpy(words.view(np.int32)).cuda(), torch.from_numpy(scale).cuda(),
            torch.from_numpy(zero).cuda()), what


def normal(seed, shape, dtype, std=1.0):
    return (torch.from_numpy(np.random.RandomState(seed).randn(*shape)) * std).to(dtype).cuda()


def within(got, ref, bound, tag=""):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, tag
    assert torch.isfinite(got).all(), f"{tag}: not finite"
    worst = ((got - ref).abs() / bound).max().item()
    assert worst <= 1.0, f"{tag}: worst error / bound {worst:.3g}"


def act64(act, g):
    g = g.detach().requires_grad_(True)
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}[act](g)
    d, = torch.autograd.grad(f.sum(), g)
    return f.detach(), d


def gated_terms(X, Wg, Wu, act):
    """G, U, act(G), act'(G) and the bounds of the fp32 sums G and U."""
    x = X.double()
    e = 1.01 * X.shape[1] * 2.0 ** -24
    G, Up = x @ Wg.T, x @ Wu.T
    f, d = act64(act, G)
    return G, Up, f, d, e * (x.abs() @ Wg.abs().T), e * (x.abs() @ Wu.abs().T)


def check_gated(Y, X, Wg, Wu, act, tag=""):
    G, Up, f, d, eG, eU = gated_terms(X, Wg, Wu, act)
    ref = f * Up
    # |act'| <= 1.2
    bound = (U[X.dtype] + FN) * ref.abs() + 1.01 * (1.2 * eG * (Up.abs() + eU) + f.abs() * eU) + TINY[X.dtype]
    within(Y, ref, bound, tag)


def grad_bound(terms, errors, weights, dtype):
    """(sum_i T_i W_i, bound) where the kernel multiplies T_i' with |T_i' - T_i| <= errors_i."""
    ref = sum(t @ w for t, w in zip(terms, weights))
    R = sum(t.shape[1] for t in terms)
    off = sum(e @ w.abs() for e, w in zip(errors, weights))
    size = sum((t.abs() + e) @ w.abs() for t, e, w in zip(terms, errors, weights))
    return ref, U[dtype] * ref.abs() + 1.01 * off + 1.01 * (R + 64) * 2.0 ** -24 * size + TINY[dtype]


def check_gated_backward(dX, dY, X, Wg, Wu, act, tag=""):
    G, Up, f, d, eG, eU = gated_terms(X, Wg, Wu, act)
    y = dY.double()
    dG, dU = y * Up * d, y * f
    # |act''| <= 1.2; dG and dU are rounded once, in fp16 relative to a row scaled to [2^-7, 2^-6)
    u = U[X.dtype]
    floor = 2.0 ** -25 * 2.0 ** 7 * y.abs().amax(1, keepdim=True) if X.dtype == torch.float16 else 1e-38
    act_off = FN * (d.abs() + G.abs())      # act' is a sum of two terms of at most these sizes
    errG = 1.01 * y.abs() * ((Up.abs() + eU) * (1.2 * eG + act_off) + d.abs() * eU) + u * dG.abs() + floor
    errU = 1.01 * y.abs() * (1.2 * eG + FN * f.abs()) + u * dU.abs() + floor
    ref, bound = grad_bound([dG, dU], [errG * 1.01, errU * 1.01], [Wg, Wu], X.dtype)
    within(dX, ref, bound, tag)


def loss_terms(X, W):
    x = X.double()
    return x @ W.T, 1.01 * X.shape[1] * 2.0 ** -24 * (x.abs() @ W.abs().T)


def check_loss(loss, lse, X, W, targets, tag=""):
    L, eL = loss_terms(X, W)
    N = W.shape[0]
    keep = (targets >= 0) & (targets < N)
    ref = torch.logsumexp(L, 1)
    # each exponential is within FN (and its logit's error); up to 2^10 joins of fp32 sums in the
    # longest chain; the logarithm and the final sums round at the size of lse
    e = eL.amax(1) + 2 * FN + 2.0 ** -14 + 2.0 ** -22 * (1 + ref.abs() + L.abs().amax(1))
    within(lse, ref, e, tag + " lse")
    assert (loss[~keep] == 0).all(), tag
    if keep.any():
        at = targets.clamp(0, N - 1)[:, None]
        lr = (ref - L.gather(1, at)[:, 0])[keep]
        if N > 1:
            rest = torch.logsumexp(L.scatter(1, at, -math.inf), 1)[keep]
            lr = torch.nn.functional.softplus(rest - L.gather(1, at)[keep, 0])
        # loss = log(1 + exp(d)) with |d - d_ref| <= 2 e: relative to a small loss
        within(loss[keep], lr, torch.clamp(lr, max=1.0) * 2 * e[keep] * 1.01 + 2.0 ** -21 * lr + 1e-37, tag + " loss")


def check_loss_backward(dX, dloss, X, W, targets, lse, tag=""):
    L, eL = loss_terms(X, W)
    N = W.shape[0]
    keep = (targets >= 0) & (targets < N)
    P = torch.exp(torch.where(keep[:, None], L - lse.double()[:, None], torch.zeros_like(L)))
    P = torch.where(keep[:, None], P, torch.zeros_like(P))
    S = P.clone()
    rows = torch.arange(len(targets), device=S.device)[keep]
    S[rows, targets[keep]] -= 1.0
    dl = torch.where(keep, dloss.double(), torch.zeros_like(lse.double()))[:, None]
    floor = 2.0 ** -40 if X.dtype == torch.float16 else 1e-38
    # p from a logit off by eL and rounded sums of it and lse, the difference rounded once
    off = P * 1.01 * (eL + FN + 2.0 ** -23 * (L.abs() + lse.double().abs()[:, None])) + U[X.dtype] * S.abs() + floor
    off = torch.where(keep[:, None], off, torch.zeros_like(off))
    ref, bound = grad_bound([S], [off * 1.01], [W], X.dtype)
    u = U[X.dtype]
    bound = dl.abs() * bound + u * (dl * ref).abs() + 2.0 ** -23 * (dl * ref).abs() + TINY[X.dtype]
    within(dX, dl * ref, bound, tag)
    assert (dX[~keep] == 0).all(), tag


# (M, K, N, nbits, gs): one row, few rows, many; depths that end inside a step; widths of one,
# odd, and across tiles; every code width and group size
SIZES = [
    (1, 32, 1, 4, 8),
    (1, 64, 5, 4, 32),
    (1, 4096, 200, 4, 64),
    (2, 96, 33, 4, 32),
    (3, 256, 64, 8, 256),
    (5, 160, 100, 2, 16),
    (8, 128, 257, 1, 32),
    (16, 512, 130, 4, 128),
    (17, 320, 66, 4, 64),
    (31, 1056, 129, 2, 32),
    (32, 256, 48, 1, 64),
    (33, 192, 71, 8, 8),
    (64, 64, 64, 4, 16),
    (100, 544, 301, 4, 32),
    (129, 128, 127, 2, 8),
    (200, 768, 520, 4, 64),
    (257, 96, 255, 8, 32),
    (300, 1024, 1000, 4, 256),
    (513, 256, 640, 1, 128),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,nbits,gs", SIZES)
def test_gated(hq, path, M, K, N, nbits, gs, dtype):
    act = ("silu", "gelu", "gelu_tanh")[(M + N) % 3]
    gate, Wg = make_weight(M + N, N, K, nbits, gs, dtype)
    up, Wu = make_weight(M + N + 1, N, K, nbits, gs, dtype)
    X, dY = normal(K, (M, K), dtype, 1.5), normal(K + 1, (M, N), dtype)
    Y = hq.hqq_linear_gated(X, gate, up, N, nbits, gs, activation=act)
    check_gated(Y, X, Wg, Wu, act, f"{act}")
    dX = hq.hqq_linear_gated_backward(dY, X, gate, up, N, nbits, gs, activation=act)
    check_gated_backward(dX, dY, X, Wg, Wu, act, f"{act}")


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,nbits,gs", SIZES)
def test_linear_backward(hq, path, M, K, N, nbits, gs, dtype):
    w, W = make_weight(3 * M + N, N, K, nbits, gs, dtype)
    dY = normal(N, (M, N), dtype)
    dX = hq.hqq_linear_backward(dY, *w, K, nbits, gs)
    y = dY.double()
    within(dX, *grad_bound([y], [torch.zeros_like(y)], [W], dtype))


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M,K,nbits,gs,Ns", [
    (1, 256, 4, 64, [64, 17, 300]),
    (7, 128, 2, 32, [8, 16, 24, 7]),
    (40, 512, 8, 64, [512, 128, 128]),
    (150, 96, 4, 32, [1, 63, 65, 64]),
    (260, 320, 1, 64, list(range(1, 17))),
])
def test_linear_batch_backward(hq, path, M, K, nbits, gs, Ns, dtype):
    """One sum over all weights; each alone in the other rows' place."""
    ws = [make_weight(50 + i, N, K, nbits, gs, dtype) for i, N in enumerate(Ns)]
    dYs = [normal(90 + i, (M, N), dtype) for i, N in enumerate(Ns)]
    dX = hq.hqq_linear_batch_backward(dYs, [w[0] + (N,) for w, N in zip(ws, Ns)], K, nbits, gs)
    y = [d.double() for d in dYs]
    within(dX, *grad_bound(y, [torch.zeros_like(d) for d in y], [w[1] for w in ws], dtype))


def some_targets(seed, M, N):
    """Random classes, the first and the last among them, some ignored."""
    rng = np.random.RandomState(seed)
    t = rng.randint(0, N, M)
    t[rng.rand(M) < 0.2] = -100
    t[0] = N - 1
    if M > 2:
        t[1], t[2] = 0, N                   # N itself is no class
    return torch.from_numpy(t.astype(np.int64)).cuda()


def loss_case(hq, M, K, N, nbits, gs, dtype, spread=1.0, targets=None):
    head, W = make_weight(7 * M + N, N, K, nbits, gs, dtype)
    X = normal(M + K, (M, K), dtype, spread)
    t = some_targets(M, M, N) if targets is None else targets
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, nbits, gs)
    check_loss(loss, lse, X, W, t)
    dloss = normal(M + 3, (M,), torch.float32, 0.1)
    dX = hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *head, N, nbits, gs)
    check_loss_backward(dX, dloss, X, W, t, lse)
    return loss, lse, dX


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,nbits,gs", SIZES)
def test_cross_entropy(hq, path, M, K, N, nbits, gs, dtype):
    loss_case(hq, M, K, N, nbits, gs, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 20001), (9, 8192, 9001), (70, 4096, 17000), (300, 8192, 8300)])
def test_cross_entropy_in_pieces(hq, path, M, K, N, dtype):
    """More classes than a piece of the tiled route: targets in every piece, and at its first and last class."""
    t = torch.randint(0, N, (M,), generator=torch.Generator().manual_seed(M))
    for i, edge in enumerate((8191, 8192, 16383, 16384, N - 1, 4095, 4096)):
        if i < M and edge < N:
            t[i] = edge
    loss_case(hq, M, K, N, 4, 64, dtype, targets=t.cuda())


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
def test_cross_entropy_peaked_rows(hq, path, dtype):
    """Logits far apart: one class holds nearly everything, as the target and as another."""
    M, K, N = 24, 256, 500
    head, W = make_weight(5, N, K, 4, 64, dtype)
    t = torch.arange(M).cuda() * 7
    lead = t.clone()
    lead[::2] += 1
    X = (W[lead] * torch.linspace(2, 30, M, device="cuda", dtype=torch.float64)[:, None]).to(dtype)
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, 4, 64)
    check_loss(loss, lse, X, W, t)
    assert loss.max() > 20 and 0 < loss.min() < 1e-4
    dloss = torch.ones(M, device="cuda")
    dX = hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *head, N, 4, 64)
    check_loss_backward(dX, dloss, X, W, t, lse)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M", [3, 70])
def test_cross_entropy_ignored_rows(hq, path, dtype, M):
    """Rows without a target give 0, whatever their inputs hold; all rows may be such."""
    K, N = 128, 300
    head, W = make_weight(5, N, K, 4, 64, dtype)
    X = normal(1, (M, K), dtype)
    t = torch.full((M,), -100, dtype=torch.int64, device="cuda")
    X[1], t[1] = math.nan, N
    X[2], t[2] = math.inf, 1 << 40
    t[0] = 5
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, 4, 64)
    dloss = torch.full((M,), 2.0, device="cuda")
    dloss[1] = math.nan
    dX = hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *head, N, 4, 64)
    assert (loss[1:] == 0).all() and (dX[1:] == 0).all()
    check_loss(loss[:1], lse[:1], X[:1], W, t[:1])
    check_loss_backward(dX[:1], dloss[:1], X[:1], W, t[:1], lse[:1])
    t[0] = -1
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, 4, 64)
    dX = hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *head, N, 4, 64)
    assert (loss == 0).all() and (dX == 0).all()


def test_fp16_small_gradients_keep_their_precision(hq, path):
    """Gradients near fp16's smallest normal number (a loss scale too low): dG and dU are formed
    relative to the row."""
    dtype = torch.float16
    M, K, N = 40, 256, 200
    gate, Wg = make_weight(1, N, K, 4, 64, dtype, std=1.0)
    up, Wu = make_weight(2, N, K, 4, 64, dtype, std=1.0)
    X = normal(3, (M, K), dtype, 2.0 ** -5)
    dY = normal(4, (M, N), dtype, 2.0 ** -13)
    dY[7] = 0
    dY[8] = 2.0 ** -24
    check_gated_backward(hq.hqq_linear_gated_backward(dY, X, gate, up, N, 4, 64), dY, X, Wg, Wu, "silu")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [4, 96])
def test_gated_saturated_activations(hq, path, act, M):
    """Projections up to several hundred: the activation's flat and linear ends."""
    dtype, K, N = torch.bfloat16, 64, 96
    gate, Wg = make_weight(1, N, K, 8, 64, dtype, std=4.0)
    up, Wu = make_weight(2, N, K, 8, 64, dtype, std=0.2)
    X, dY = normal(3, (M, K), dtype, 4.0), normal(4, (M, N), dtype)
    Y = hq.hqq_linear_gated(X, gate, up, N, 8, 64, activation=act)
    dX = hq.hqq_linear_gated_backward(dY, X, gate, up, N, 8, 64, activation=act)
    assert torch.isfinite(Y).all() and torch.isfinite(dX).all()
    G, Up, f, d, eG, eU = gated_terms(X, Wg, Wu, act)
    assert G.abs().max() > 100
    # the exponent's own rounding grows with it: at most 2^-24 |z| for the exponents |z| < 10^7
    # that occur, times |act| <= |G| where the activation has not reached its end
    live = (G.abs() < 30).double()
    ref = f * Up
    bound = (U[dtype] + FN) * ref.abs() + 1.01 * (1.2 * eG * (Up.abs() + eU) + f.abs() * eU) + 2.0 ** -12 * live * ref.abs() + 1e-9
    within(Y, ref, bound)
    check_gated_backward(dX, dY, X, Wg, Wu, act)


def chain(hq, dtype, M=37, K=128, F=192, V=400, nbits=4, gs=64):
    """A small block and head: h = down(gated(x)), loss(h)."""
    gate, Wg = make_weight(1, F, K, nbits, gs, dtype)
    up, Wu = make_weight(2, F, K, nbits, gs, dtype)
    down, Wd = make_weight(3, K, F, nbits, gs, dtype)
    head, Wh = make_weight(4, V, K, nbits, gs, dtype, std=1.0)
    t = some_targets(9, M, V)

    def forward(x):
        y = hq.hqq_linear_gated(x, gate, up, F, nbits, gs)
        h = hq.hqq_linear(y, *down, K, nbits, gs)
        loss, lse = hq.hqq_linear_cross_entropy(h, t, *head, V, nbits, gs)
        return y, h, loss, lse

    def backward(x, h, lse, dloss):
        dh = hq.hqq_linear_cross_entropy_backward(dloss, h, t, lse, *head, V, nbits, gs)
        dy = hq.hqq_linear_backward(dh, *down, F, nbits, gs)
        return hq.hqq_linear_gated_backward(dy, x, gate, up, F, nbits, gs)

    def total64(x):
        y = torch.nn.functional.silu(x @ Wg.T) * (x @ Wu.T)
        L = (y @ Wd.T) @ Wh.T
        keep = (t >= 0) & (t < V)
        return torch.nn.functional.cross_entropy(L[keep], t[keep], reduction="sum")

    return forward, backward, total64, normal(7, (M, K), dtype, 2.0), t


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
def test_operators_together(hq, path, dtype):
    """A block and a head as a fine-tuning step runs them: loss and gradient against autograd and
    against differences in 64 bits.  Three 16-bit intermediates on the way forward and three on the
    way back, each off by u of its size: as independent errors well within 16 u of the norm."""
    forward, backward, total64, X, t = chain(hq, dtype)
    _, h, loss, lse = forward(X)
    dX = backward(X, h, lse, torch.ones(len(t), device="cuda")).double()
    x = X.double().requires_grad_(True)
    ref = total64(x)
    g, = torch.autograd.grad(ref, x)
    u = U[dtype]
    assert abs(loss.double().sum() - ref).item() <= 16 * u * abs(ref.item())
    assert (dX - g).norm() <= 16 * u * g.norm()
    v = normal(21, tuple(X.shape), torch.float64)
    step = 1e-5
    diff = (total64(x.detach() + step * v) - total64(x.detach() - step * v)) / (2 * step)
    # the step's own error is of order step^2; the gradient's along v is that of its norm
    assert abs((dX * v).sum() - diff).item() <= 16 * u * (g.norm() * v.norm()).item() + 1e-6


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 20, 150])
def test_captured_and_replayed(hq, path, dtype, M):
    """The whole step in a HIP graph, replayed with new inputs between eager calls: the same bits."""
    forward, backward, _, X, t = chain(hq, dtype, M=M)
    dloss = torch.ones(M, device="cuda")

    def step(x):
        y, h, loss, lse = forward(x)
        return y, loss, lse, backward(x, h, lse, dloss)

    buf = X.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(buf)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(buf)
    for i in range(4):
        new = normal(100 + i, tuple(X.shape), dtype)
        buf.copy_(new)
        graph.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        for a, b in zip(got, step(new)):
            assert torch.equal(a, b), i


def everything(hq, dtype, M, K, N, nbits, gs, ws=None):
    """Every operator once, with workspaces from ws(bytes)."""
    a, _ = make_weight(1, N, K, nbits, gs, dtype)
    b, _ = make_weight(2, N, K, nbits, gs, dtype)
    X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)
    t = some_targets(5, M, N)
    dl = torch.ones(M, device="cuda")
    ws = ws or (lambda n: None)
    s = (M, K, N, nbits, gs)
    f = (N, nbits, gs)
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *a, *f, workspace=ws(hq.hqq_linear_cross_entropy_workspace(*s)))
    return [hq.hqq_linear_gated(X, a, b, *f, workspace=ws(hq.hqq_linear_gated_workspace(*s))),
            hq.hqq_linear_gated_backward(dY, X, a, b, *f, workspace=ws(hq.hqq_linear_gated_backward_workspace(*s))),
            hq.hqq_linear_batch_backward([dY, dY], [a + (N,), b + (N,)], K, nbits, gs,
                                         workspace=ws(hq.hqq_linear_batch_backward_workspace(M, K, [N, N], nbits, gs))),
            loss, lse,
            hq.hqq_linear_cross_entropy_backward(dl, X, t, lse, *a, *f,
                                                 workspace=ws(hq.hqq_linear_cross_entropy_backward_workspace(*s)))]


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(1, 160, 77), (13, 256, 300), (200, 352, 515)])
def test_workspace_contents_and_repeats(hq, path, dtype, M, K, N):
    """A caller's workspace of the stated size, full of NaN (bytes 0xff) with a guard behind it:
    the same bits as without, twice, and the guard untouched."""
    plain = everything(hq, dtype, M, K, N, 4, 32)
    guards = []

    def ws(n):
        t = torch.full((n + 4096,), 0xff, dtype=torch.uint8, device="cuda")
        guards.append(t[n:])
        return t[:n]

    for _ in range(2):
        for a, b in zip(everything(hq, dtype, M, K, N, 4, 32, ws), plain):
            assert torch.equal(a, b)
    for g in guards:
        assert (g == 0xff).all()


def test_outputs_in_larger_buffers(hq, path):
    """Nothing is written outside the outputs (odd widths end inside vector stores)."""
    dtype, M, K, N = torch.float16, 45, 96, 67
    a, _ = make_weight(1, N, K, 4, 32, dtype)
    X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)

    def guarded(n, dt):
        whole = torch.full((n + 512,), 7.0, dtype=dt, device="cuda")
        return whole, whole[256:256 + n]

    for shape, call in [((M, N), lambda o: hq.hqq_linear_gated(X, a, a, N, 4, 32, out=o)),
                        ((M, K), lambda o: hq.hqq_linear_gated_backward(dY, X, a, a, N, 4, 32, out=o)),
                        ((M, K), lambda o: hq.hqq_linear_backward(dY, *a, K, 4, 32, out=o))]:
        whole, part = guarded(shape[0] * shape[1], dtype)
        call(part.view(shape))
        assert (whole[:256] == 7).all() and (whole[256 + part.numel():] == 7).all()
        assert (part != 7).any()


@pytest.mark.parametrize("M", [1, 8, 9, 32, 33, 64, 65, 96, 256, 257])
def test_route_boundaries(hq, M):
    """The sizes at which the library changes its route by itself, each operator."""
    dtype, K, N = torch.bfloat16, 512, 1100
    for nbits, gs in ((4, 64), (2, 16)):
        a, Wa = make_weight(1, N, K, nbits, gs, dtype)
        b, Wb = make_weight(2, N, K, nbits, gs, dtype)
        X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)
        check_gated(hq.hqq_linear_gated(X, a, b, N, nbits, gs), X, Wa, Wb, "silu")
        check_gated_backward(hq.hqq_linear_gated_backward(dY, X, a, b, N, nbits, gs), dY, X, Wa, Wb, "silu")
        y = dY.double()
        within(hq.hqq_linear_backward(dY, *a, K, nbits, gs), *grad_bound([y], [torch.zeros_like(y)], [Wa], dtype))
        loss_case(hq, M, K, N, nbits, gs, dtype)


def test_two_streams_with_their_own_workspaces(hq):
    """The same calls on two streams at once give what they give alone."""
    want = everything(hq, torch.bfloat16, 150, 256, 333, 4, 64)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(everything(hq, torch.bfloat16, 150, 256, 333, 4, 64))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_same_weight_and_gradient_twice(hq):
    """One weight given as both projections, and one gradient for two weights."""
    dtype, M, K, N = torch.bfloat16, 19, 128, 80
    w, W = make_weight(1, N, K, 4, 64, dtype)
    X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)
    check_gated(hq.hqq_linear_gated(X, w, w, N, 4, 64), X, W, W, "silu")
    y = dY.double()
    dX = hq.hqq_linear_batch_backward([dY, dY], [w + (N,), w + (N,)], K, 4, 64)
    z = torch.zeros_like(y)
    within(dX, *grad_bound([y, y], [z, z], [W, W], dtype))


def test_shapes_are_checked(hq):
    """The binding refuses what does not fit, before anything runs."""
    dtype, M, K, N = torch.float16, 4, 128, 80
    w, _ = make_weight(1, N, K, 4, 64, dtype)
    X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)
    t = torch.zeros(M, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        hq.hqq_linear_gated(X, w, w, N + 1, 4, 64)
    with pytest.raises(ValueError):
        hq.hqq_linear_gated(X, w, w, N, 8, 64)
    with pytest.raises(ValueError):
        hq.hqq_linear_gated(X, w, w, N, 4, 64, activation="relu")
    with pytest.raises(ValueError):
        hq.hqq_linear_gated(X.t().contiguous().t(), w, w, N, 4, 64)
    with pytest.raises(TypeError):
        hq.hqq_linear_gated_backward(dY.bfloat16(), X, w, w, N, 4, 64)
    with pytest.raises(ValueError):
        hq.hqq_linear_backward(dY[:, :-1].contiguous(), *w, K, 4, 64)
    with pytest.raises(TypeError):
        hq.hqq_linear_cross_entropy(X, t.int(), *w, N, 4, 64)
    with pytest.raises(ValueError):
        hq.hqq_linear_cross_entropy(X, t[:3], *w, N, 4, 64)
    with pytest.raises(hq.LayersError):
        hq.hqq_linear_gated(X[:0], w, w, N, 4, 64)
    need = hq.hqq_linear_gated_backward_workspace(M, K, N, 4, 64)
    with pytest.raises(hq.LayersError) as e:
        hq.hqq_linear_gated_backward(dY, X, w, w, N, 4, 64, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -11


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("K,N", [(96, 200), (512, 4500)])
def test_more_rows_than_a_chunk(hq, dtype, K, N):
    """The backward passes go over 8192 rows at a time: the last chunk is a short one."""
    M = 8192 + 70
    gate, Wg = make_weight(1, N, K, 4, 32, dtype)
    up, Wu = make_weight(2, N, K, 4, 32, dtype)
    X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)
    t = torch.from_numpy(np.random.RandomState(5).randint(-1, N + 1, M)).cuda()
    dX = hq.hqq_linear_gated_backward(dY, X, gate, up, N, 4, 32)
    dXb = hq.hqq_linear_batch_backward([dY, dY], [gate + (N,), up + (N,)], K, 4, 32)
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *gate, N, 4, 32)
    dloss = normal(6, (M,), torch.float32)
    dXl = hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *gate, N, 4, 32)
    for part in (slice(0, 40), slice(8150, 8230), slice(M - 30, M)):
        x, y = X[part], dY[part]
        check_gated_backward(dX[part], y, x, Wg, Wu, "silu", f"rows {part.start}")
        z = torch.zeros_like(y.double())
        within(dXb[part], *grad_bound([y.double()] * 2, [z, z], [Wg, Wu], dtype), f"rows {part.start}")
        check_loss(loss[part], lse[part], x, Wg, t[part], f"rows {part.start}")
        check_loss_backward(dXl[part], dloss[part], x, Wg, t[part], lse[part], f"rows {part.start}")


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M", [4, 20, 90])
def test_bad_rows_keep_to_themselves(hq, path, dtype, M):
    """NaN and infinities in one row of an input change that row of the results only."""
    K, N = 160, 333
    gate, _ = make_weight(1, N, K, 4, 32, dtype)
    up, _ = make_weight(2, N, K, 4, 32, dtype)
    X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)
    t = torch.from_numpy(np.random.RandomState(5).randint(0, N, M)).cuda()
    dloss = normal(6, (M,), torch.float32)

    def step(X, dY, dloss):
        loss, lse = hq.hqq_linear_cross_entropy(X, t, *gate, N, 4, 32)
        return (hq.hqq_linear_gated(X, gate, up, N, 4, 32), hq.hqq_linear_gated_backward(dY, X, gate, up, N, 4, 32),
                hq.hqq_linear_backward(dY, *gate, K, 4, 32), loss, lse,
                hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *gate, N, 4, 32))

    clean = step(X, dY, dloss)
    X2, dY2, dloss2 = X.clone(), dY.clone(), dloss.clone()
    X2[M - 1], dY2[M - 1, 7], dloss2[M - 1] = math.nan, math.nan, math.nan
    X2[1, 5], dY2[1, 9], dloss2[1] = math.inf, -math.inf, math.inf
    good = [m for m in range(M) if m not in (1, M - 1)]
    for a, b in zip(step(X2, dY2, dloss2), clean):
        assert torch.equal(a[good], b[good])
        assert not torch.isfinite(a[M - 1]).any() and not torch.isfinite(a[1]).all()


def test_the_most_rows(hq):
    """2^20 rows: outputs past 4 GB, and a loss over half a million classes whose tiles fill a grid."""
    dtype, M, K, N = torch.bfloat16, 1 << 20, 64, 2500
    X = torch.randn(M, K, device="cuda", dtype=dtype)
    rows = torch.tensor([0, 1, 12345, M // 2, M - 2, M - 1], device="cuda")
    gate, Wg = make_weight(1, N, K, 4, 64, dtype)
    up, Wu = make_weight(2, N, K, 4, 64, dtype)
    Y = hq.hqq_linear_gated(X, gate, up, N, 4, 64)
    assert Y.numel() * 2 > 1 << 32
    check_gated(Y[rows], X[rows], Wg, Wu, "silu")
    dX = hq.hqq_linear_gated_backward(Y, X, gate, up, N, 4, 64)
    check_gated_backward(dX[rows], Y[rows], X[rows], Wg, Wu, "silu")
    del Y, dX
    torch.cuda.empty_cache()
    N = 1 << 19
    head, W = make_weight(3, N, K, 1, 64, dtype)
    t = torch.randint(0, N, (M,), device="cuda")
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, 1, 64)
    check_loss(loss[rows], lse[rows], X[rows], W, t[rows])
    torch.cuda.empty_cache()


@pytest.mark.parametrize("gs", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("nbits", [1, 2, 4, 8])
def test_every_format(hq, path, nbits, gs):
    """Each code width and group size, with depths that end on a 256-wide step and inside one."""
    for K in (512, 544 if gs <= 32 else 9 * gs if gs == 64 else 5 * gs):
        for M, N in ((2, 50), (9, 33), (20, 70), (70, 40)):
            for dtype in DTYPES:
                tag = f"{M} x {K} x {N} {dtype}"
                gate, Wg = make_weight(nbits, N, K, nbits, gs, dtype)
                up, Wu = make_weight(gs, N, K, nbits, gs, dtype)
                X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)
                check_gated(hq.hqq_linear_gated(X, gate, up, N, nbits, gs), X, Wg, Wu, "silu", tag)
                check_gated_backward(hq.hqq_linear_gated_backward(dY, X, gate, up, N, nbits, gs), dY, X, Wg, Wu, "silu", tag)
                y = dY.double()
                dX = hq.hqq_linear_batch_backward([dY, dY], [gate + (N,), up + (N,)], K, nbits, gs)
                within(dX, *grad_bound([y, y], [torch.zeros_like(y)] * 2, [Wg, Wu], dtype), tag)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("nbits,gs", [(1, 32), (2, 16), (2, 64), (4, 8), (4, 16), (4, 32), (4, 64), (8, 8), (8, 32), (8, 128)])
def test_weights_are_the_dequantized_ones(hq, path, nbits, gs, dtype):
    """One-hot inputs give back W_hat, bit for bit what hqq_dequantize writes: rows through the
    backward pass, and a single class's weights through the log-sum-exp of one logit."""
    N, K = 200, 256
    w, _ = make_weight(nbits + gs, N, K, nbits, gs, dtype, std=3.0)
    want = hq.hqq_dequantize(*w, N, K, nbits, gs, 1, dtype=dtype)
    eye = torch.eye(N, device="cuda", dtype=dtype)
    assert torch.equal(hq.hqq_linear_backward(eye, *w, K, nbits, gs), want)
    X, t = torch.eye(K, device="cuda", dtype=dtype), torch.zeros(K, dtype=torch.int64, device="cuda")
    for n in (0, 7, N - 1):
        row = tuple(a[n:n + 1].clone() for a in w)
        _, lse = hq.hqq_linear_cross_entropy(X, t, *row, 1, nbits, gs)
        assert torch.equal(lse, want[n].float()), n


def test_a_tensor_given_twice_has_to_fit(hq):
    """The first gradient of a batch, and X given again as a gradient or as the output, are refused
    where their width is not the weight's."""
    dtype, M, K, N = torch.float16, 4, 128, 80
    w, _ = make_weight(1, N, K, 4, 64, dtype)
    X, narrow = normal(3, (M, K), dtype), normal(4, (M, 16), dtype)
    with pytest.raises(ValueError):
        hq.hqq_linear_batch_backward([narrow], [w + (N,)], K, 4, 64)
    with pytest.raises(ValueError):
        hq.hqq_linear_batch_backward([X, X], [w + (N,), w + (N,)], K, 4, 64)
    with pytest.raises(ValueError):
        hq.hqq_linear_gated_backward(X, X, w, w, N, 4, 64)
    with pytest.raises(ValueError):
        hq.hqq_linear_gated(X, w, w, N, 4, 64, out=X)


@pytest.mark.parametrize("M", [5, 40])
@pytest.mark.parametrize("gate_std,up_std", [(1.0, 1.0), (2.0 ** -6, 2.0 ** 6)])
@pytest.mark.parametrize("xs", [2.0 ** -14, 2.0 ** -11, 2.0 ** -8, 2.0 ** -5, 1.0, 2.0 ** 10])
def test_fp16_small_projections_keep_their_precision(hq, path, xs, gate_std, up_std, M):
    """dG and dU shrink with the projections (activations of size xs) and with one weight beside
    another, while dX stays of one size: they are formed relative to a bound b = max |dY| sum |X|
    max |W_hat| of the row, brought to 2^13 at least.  Below fp16's normal range, 2^-14 there, a
    rounding is off by 2^-25: by at most 2^-38 b in all."""
    dtype, K, N = torch.float16, 512, 200
    size = 1.0 / math.sqrt(K)
    gate, Wg = make_weight(1, N, K, 4, 64, dtype, std=size * gate_std)
    up, Wu = make_weight(2, N, K, 4, 64, dtype, std=size * up_std)
    X, dY = normal(3, (M, K), dtype, xs), normal(4, (M, N), dtype, 2.0 ** -6 / xs)
    dX = hq.hqq_linear_gated_backward(dY, X, gate, up, N, 4, 64)
    G, Up, f, d, eG, eU = gated_terms(X, Wg, Wu, "silu")
    y, u = dY.double(), U[dtype]
    dG, dU = y * Up * d, y * f
    b = y.abs().amax(1, keepdim=True) * X.double().abs().sum(1, keepdim=True) * max(Wg.abs().max(), Wu.abs().max())
    act_off = FN * (d.abs() + G.abs())
    errG = 1.01 * y.abs() * ((Up.abs() + eU) * (1.2 * eG + act_off) + d.abs() * eU) + u * dG.abs() + 2.0 ** -38 * b
    errU = 1.01 * y.abs() * (1.2 * eG + FN * f.abs()) + u * dU.abs() + 2.0 ** -38 * b
    ref, bound = grad_bound([dG, dU], [errG * 1.01, errU * 1.01], [Wg, Wu], dtype)
    within(dX, ref, bound)
    # as independent errors, at most u of dG, dU and dX each: well within 4 u of the norm
    assert (dX.double() - ref).norm() <= 4 * u * ref.norm()


@pytest.mark.parametrize("M", [3, 70])
def test_fp16_rows_without_a_gradient(hq, path, M):
    """Rows of zeros in dY or X give zeros, the least and the largest values that fp16 has stay finite."""
    dtype, K, N = torch.float16, 96, 33
    gate, _ = make_weight(1, N, K, 4, 32, dtype)
    up, _ = make_weight(2, N, K, 4, 32, dtype)
    X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)
    dY[0] = 0
    X[1] = 0
    dY[2], X[2] = 2.0 ** -24, 2.0 ** -24
    dX = hq.hqq_linear_gated_backward(dY, X, gate, up, N, 4, 32)
    assert (dX[:3] == 0).all() and torch.isfinite(dX).all()
    X[1], dY[1] = 65504.0, 2.0 ** -24
    dX = hq.hqq_linear_gated_backward(dY, X, gate, up, N, 4, 32)
    assert torch.isfinite(dX[1]).all()


def test_workspace_of_another_stream_is_kept(hq):
    """A workspace allocated on one stream, used on another and dropped: while the call may still
    write it, the allocator does not give its memory to the first stream again."""
    dtype, M, K, N = torch.bfloat16, 300, 128, 200
    w, _ = make_weight(1, N, K, 4, 64, dtype)
    X = normal(3, (M, K), dtype)
    need = hq.hqq_linear_gated_workspace(M, K, N, 4, 64)
    busy = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(50):
        busy = busy @ busy * 1e-2                       # tens of milliseconds before the call's turn
    Y = hq.hqq_linear_gated(X, w, w, N, 4, 64, workspace=ws)
    where = ws.data_ptr()
    del ws
    with torch.cuda.stream(side):
        again = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert not torch.cuda.current_stream().query()      # the call was still ahead
    assert again.data_ptr() != where
    torch.cuda.synchronize()
    assert torch.equal(Y, hq.hqq_linear_gated(X, w, w, N, 4, 64))


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M", [9, 70])
def test_cross_entropy_infinite_logits(hq, path, dtype, M):
    """Infinities among a row's logits give what the definition gives in IEEE arithmetic: lse is +inf
    with a +inf logit and -inf where all are -inf, loss = lse - l_t."""
    K, N = 160, 333
    (packed, scale, zero), _ = make_weight(5, N, K, 4, 32, dtype)
    zero[:, 0] = -1.0                                   # W_hat > 0 in the first 32 columns
    W = hq.hqq_dequantize(packed, scale, zero, N, K, 4, 32, 1, dtype=dtype).double()
    assert (W != 0).all() and (W[:, 40] > 0).any() and (W[:, 40] < 0).any()
    X = normal(1, (M, K), dtype)
    t = torch.randint(0, N, (M,), generator=torch.Generator().manual_seed(1)).cuda()
    X[0, 3], X[1, 3] = math.inf, -math.inf              # all logits +inf, all -inf
    X[2:5, 40] = math.inf                               # both
    t[2], t[3], t[4] = int(W[:, 40].argmax()), int(W[:, 40].argmin()), -100
    X[5, 7] = math.nan
    loss, lse = hq.hqq_linear_cross_entropy(X, t, packed, scale, zero, N, 4, 32)
    L = X.double() @ W.T
    ref = torch.logsumexp(L, 1)
    want = torch.where((t >= 0) & (t < N), ref - L.gather(1, t.clamp(min=0)[:, None])[:, 0], torch.zeros_like(ref))
    assert ref[:6].tolist()[:5] == [math.inf, -math.inf, math.inf, math.inf, math.inf] and want[3] == math.inf
    for got, r in ((lse, ref), (loss, want)):
        torch.testing.assert_close(got[:6].double(), r[:6], rtol=0, atol=0, equal_nan=True)
    check_loss(loss[6:], lse[6:], X[6:], W, t[6:])


@pytest.mark.parametrize("M", [3, 70])
def test_cross_entropy_near_the_largest_logits(hq, path, M):
    """Logits up to fp32's last binade: lse is their maximum."""
    K, N, dtype = 64, 200, torch.bfloat16
    head, W = make_weight(5, N, K, 8, 64, dtype, std=0.5)
    X = torch.zeros(M, K, dtype=dtype, device="cuda")
    X[:, 9] = 1.1875 * 2.0 ** 127
    L = X.double() @ W.T
    assert 2.4e38 < L.max() < 3.4e38 and L.max() - L.min() > 3.5e38
    t = torch.full((M,), int(L[0].argmin()), device="cuda")
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, 8, 64)
    # one exact product per logit; the least is about as far below 0: the difference overflows
    assert torch.equal(lse.double(), L.amax(1)) and (loss == math.inf).all()
    t = L.argmax(1)
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, 8, 64)
    assert torch.equal(lse.double(), L.amax(1)) and (loss == 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [4, 96])
def test_gated_huge_projections(hq, path, act, M):
    """Projections up to 2^60, whose squares and cubes overflow: act is 0 or the identity there and
    act' 0 or 1.  (Exact inputs of one term per sum, so that G and U carry no error; dG and dU are
    then off by a rounding each, and dX = dG Wg + dU Wu by two, its sum and its own.)"""
    dtype, K, N = torch.bfloat16, 64, 96
    gate, Wg = make_weight(1, N, K, 8, 64, dtype)
    up, Wu = make_weight(2, N, K, 8, 64, dtype)
    X = torch.zeros(M, K, dtype=dtype, device="cuda")
    for m in range(M):
        X[m, m % K] = (-1.0) ** m * 2.0 ** (45 + 15 * m / M // 1)
    dY = normal(4, (M, N), dtype)
    Y = hq.hqq_linear_gated(X, gate, up, N, 8, 64, activation=act)
    dX = hq.hqq_linear_gated_backward(dY, X, gate, up, N, 8, 64, activation=act)
    x, y = X.double(), dY.double()
    G, Up = x @ Wg.T, x @ Wu.T
    assert G.abs().min() > 2.0 ** 20 and G.abs().max() > 2.0 ** 50
    on = (G > 0).double()
    u = U[dtype]
    within(Y, on * G * Up, (u + FN) * (on * G * Up).abs() + 1e-30)
    dG, dU = y * Up * on, y * G * on
    within(dX, *grad_bound([dG, dU], [(u + FN) * 1.01 * dG.abs() + 1e-30, (u + FN) * 1.01 * dU.abs() + 1e-30], [Wg, Wu], dtype))


def device_weight(seed, N, K, nbits, gs, dtype):
    """make_weight for large weights: made on the GPU."""
    g = torch.Generator("cuda").manual_seed(seed)
    words = torch.randint(-2 ** 31, 2 ** 31, (N, K * nbits // 32), dtype=torch.int32, device="cuda", generator=g)
    qmax, std = (1 << nbits) - 1, 1.0 / math.sqrt(K)
    lo, hi = ((2 + 0.5 * torch.randn(N, K // gs, device="cuda", generator=g)).abs() * std for _ in range(2))
    scale = qmax / (hi + lo + 1e-3 * std)
    zero = lo * scale
    shifts = torch.arange(PER_WORD[nbits], dtype=torch.int32, device="cuda") * nbits
    q = ((words[..., None] >> shifts) & qmax).float().view(N, K // gs, gs)
    return (words, scale, zero), ((q - zero[..., None]) / scale[..., None]).to(dtype).view(N, K).double()


def piece_edges(K, N, limit):
    """Every class at which a piece of the vocabulary may begin: pieces are of p - 3 s to p + 2 s classes in
    steps of s, p of those that 128 MiB of W_hat hold (at most `limit`, at least 4096) and s an eighth."""
    p = max(4096, min((64 << 20) // (-(-K // 64) * 64 + 64) // 256 * 256, limit))
    s = p // 8 // 256 * 256
    assert N > p + 2 * s                                # more than one piece, whatever its width
    return sorted({e for w in range(p - 3 * s, p + 2 * s + 1, s) for e in range(w, N, w)})


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M", [1, 9, 70, 300])
def test_cross_entropy_at_piece_edges(hq, monkeypatch, M, dtype):
    """More classes than a piece of the tiled route holds: targets at the last class of each piece and
    the first of the next.  (A workspace smaller than W_hat shows that there are pieces.)"""
    monkeypatch.setenv("HQQ_LAYERS_PATH", "tiled")
    K, N = 16384, 9000
    assert hq.hqq_linear_cross_entropy_workspace(M, K, N, 4, 64) < 2 * N * (K + 64)
    assert hq.hqq_linear_cross_entropy_backward_workspace(M, K, N, 4, 64) < 2 * N * (K + 64)
    head, W = device_weight(M, N, K, 4, 64, dtype)
    classes = [c for e in piece_edges(K, N, 1 << 25) for c in (e - 1, e)] + [0, N - 1]
    X, dloss = normal(1, (M, K), dtype), normal(2, (M,), torch.float32)
    for i in range(0, len(classes), M):
        t = torch.full((M,), 77)
        part = classes[i:i + M]
        t[:len(part)] = torch.tensor(part)
        t = t.cuda()
        loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, 4, 64)
        check_loss(loss, lse, X, W, t, str(part))
        dX = hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *head, N, 4, 64)
        check_loss_backward(dX, dloss, X, W, t, lse, str(part))


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
def test_pieces_of_a_chunk_of_rows(hq, dtype):
    """Pieces within chunks of 8192 rows, of which the last is a short one: the gradients of 8192
    rows times all classes would not fit the workspace."""
    M, K, N = 8192 + 70, 64, 5300
    assert hq.hqq_linear_cross_entropy_backward_workspace(M, K, N, 4, 32) < 8192 * N * 2
    head, W = device_weight(1, N, K, 4, 32, dtype)
    X, dloss = normal(1, (M, K), dtype), normal(2, (M,), torch.float32)
    classes = torch.tensor([c for e in piece_edges(K, N, 4096) for c in (e - 1, e)] + [0, N - 1, -1, N])
    t = classes[torch.arange(M) % len(classes)].cuda()
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, 4, 32)
    dX = hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *head, N, 4, 32)
    for part in (slice(0, 40), slice(8150, 8230), slice(M - 30, M)):
        check_loss(loss[part], lse[part], X[part], W, t[part], f"rows {part.start}")
        check_loss_backward(dX[part], dloss[part], X[part], W, t[part], lse[part], f"rows {part.start}")


@pytest.mark.parametrize("K,N,rows", [(512, 4000, [32, 33, 64, 65, 128, 129, 160, 161]), (2048, 10240, [32, 33, 64, 65])])
def test_on_both_sides_of_the_route_limits(hq, K, N, rows):
    """The operators on the rows at which each changes its route by itself: 64 and 160, 64, 64, 160 and 128 for
    the smaller weight (gated, its gradient, the linear gradient, loss, its gradient), and 64 and 32 for the larger."""
    dtype, nbits, gs = torch.bfloat16, 4, 64
    a, Wa = device_weight(1, N, K, nbits, gs, dtype)
    b, Wb = device_weight(2, N, K, nbits, gs, dtype)
    for M in rows:
        tag = f"{M} rows"
        X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype)
        check_gated(hq.hqq_linear_gated(X, a, b, N, nbits, gs), X, Wa, Wb, "silu", tag)
        check_gated_backward(hq.hqq_linear_gated_backward(dY, X, a, b, N, nbits, gs), dY, X, Wa, Wb, "silu", tag)
        y = dY.double()
        within(hq.hqq_linear_backward(dY, *a, K, nbits, gs), *grad_bound([y], [torch.zeros_like(y)], [Wa], dtype), tag)
        t, dloss = some_targets(M, M, N), normal(6, (M,), torch.float32)
        loss, lse = hq.hqq_linear_cross_entropy(X, t, *a, N, nbits, gs)
        check_loss(loss, lse, X, Wa, t, tag)
        check_loss_backward(hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *a, N, nbits, gs), dloss, X, Wa, t, lse, tag)


# The largest tiles run where they fill the 256 CUs in one round (a few rows and columns less, so that
# tiles end inside): rows, and columns per 2 N of the gated block or per N of the head
LARGE = {"256x256": (2043, 8186), "256x128": (2043, 4090), "128x128": (1019, 4090)}


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tile", LARGE)
def test_large_tiles_gated(hq, tile, act, dtype):
    M, N, K = LARGE[tile][0], LARGE[tile][1] // 2, 160
    gate, Wg = device_weight(1, N, K, 4, 32, dtype)
    up, Wu = device_weight(2, N, K, 4, 32, dtype)
    X, dY = normal(3, (M, K), dtype, 1.5), normal(4, (M, N), dtype)
    check_gated(hq.hqq_linear_gated(X, gate, up, N, 4, 32, activation=act), X, Wg, Wu, act)
    check_gated_backward(hq.hqq_linear_gated_backward(dY, X, gate, up, N, 4, 32, activation=act), dY, X, Wg, Wu, act)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("tile", LARGE)
def test_large_tiles_loss(hq, tile, dtype):
    M, N = LARGE[tile]
    K = 160
    head, W = device_weight(5, N, K, 4, 32, dtype)
    X, dloss, t = normal(1, (M, K), dtype), normal(2, (M,), torch.float32), some_targets(3, M, N)
    loss, lse = hq.hqq_linear_cross_entropy(X, t, *head, N, 4, 32)
    check_loss(loss, lse, X, W, t)
    check_loss_backward(hq.hqq_linear_cross_entropy_backward(dloss, X, t, lse, *head, N, 4, 32), dloss, X, W, t, lse)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", [
    (2043, 8192, 200),        # one round of 256 x 256 tiles of dX, a few steps along N: not split
    (2043, 4096, 200),        # of 256 x 128
    (1019, 4096, 200),        # of 128 x 128
    (2043, 8192, 20001),      # hundreds of steps, not split
    (2043, 4096, 20001),      # half a round of 256 x 256: split
])
def test_large_tiles_gradient(hq, M, K, N, dtype):
    w, W = device_weight(7, N, K, 4, 64, dtype)
    dY = normal(4, (M, N), dtype)
    dX = hq.hqq_linear_backward(dY, *w, K, 4, 64)
    for part in (slice(0, 300), slice(900, 1019), slice(M - 200, M)):
        y = dY[part].double()
        within(dX[part], *grad_bound([y], [torch.zeros_like(y)], [W], dtype), f"rows {part.start}")


@pytest.mark.parametrize("nbits,gs", [(1, 8), (4, 8), (8, 64)])
def test_fp16_groups_of_equal_weights(hq, path, nbits, gs):
    """Groups of equal weights hold one code at scale 1, and the bound of the weights counts the whole
    range of codes there (255 beside weights of 2^-14): small weights keep their precision among them."""
    dtype, M, K, N = torch.float16, 12, 544 if gs == 8 else 576, 200
    weights = []
    for seed, value in ((1, 0.0), (2, 2.0 ** -13)):
        (packed, scale, zero), _ = make_weight(seed, N, K, nbits, gs, dtype, std=2.0 ** -14)
        scale[::3, 1::2], zero[::3, 1::2] = 1.0, -value
        codes = hq.hqq_unpack(packed, N, K, nbits, gs, 1)
        codes.view(N, K // gs, gs)[::3, 1::2] = 0
        packed = hq.hqq_pack(codes, nbits, gs, 1)
        weights.append(((packed, scale, zero), hq.hqq_dequantize(packed, scale, zero, N, K, nbits, gs, 1, dtype=dtype).double()))
    (gate, Wg), (up, Wu) = weights
    assert max(Wg.abs().max(), Wu.abs().max()) < 2.0 ** -11
    X, dY = normal(3, (M, K), dtype), normal(4, (M, N), dtype, 2.0 ** 13)
    dX = hq.hqq_linear_gated_backward(dY, X, gate, up, N, nbits, gs)
    G, Up, f, d, eG, eU = gated_terms(X, Wg, Wu, "silu")
    ref = (dY.double() * Up * d) @ Wg + (dY.double() * f) @ Wu
    # dX is about 2^-7, within the normal range:
    # as independent errors, at most u of dG, dU and dX each
    assert ref.abs().mean() > 2.0 ** -14
    assert (dX.double() - ref).norm() <= 4 * U[dtype] * ref.norm()
