"""GPU parity of streaming attention (sla2_window_forward / _backward, sla2_cache_append / _attention)
against the fp64 oracle, element by element.

The tolerances are bounds, from the roundings that the operators' definition names:
- u = eps / 2 of the 16-bit type for each rounding to it (weights, gradients of the logits, outputs);
- the logits' fp32 accumulation, taken at 2^-22 for each of d additions relative to sum |q||k| scale
  (tensor cores may truncate), which is a relative error of the weights; 2^-20 for the exponential;
- 2^-22 for each addition of a sum over keys or queries.
"""
import numpy as np
import pytest
import torch

from oracle import streaming_oracle as S

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def sla2():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from block_sparse_linear_router_b200 import build
    build.build()
    from block_sparse_linear_router_b200 import sla2 as L
    L.load_library()
    return L


def _np(t):
    return t.double().cpu().numpy()


def _u(dt):
    return torch.finfo(dt).eps / 2


def _tiny(dt):
    return torch.finfo(dt).smallest_normal


def _near(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst by {np.nanmax(np.abs(got - want) / tol):.2f} tolerances"


def _weight_error(Q, K, mask, scale):
    """Relative error of a row's weights from its logits."""
    d = Q.shape[1]
    M = np.where(mask, np.abs(Q) @ np.abs(K).T, 0).max(axis=1, initial=0) * scale
    return 2 * (d * 2.0 ** -22 * M + 2.0 ** -20)


def _check_head(dt, Q, K, V, O, lse, window, sinks, causal, scale, grads=None):
    n, u, tiny = Q.shape[0], _u(dt), _tiny(dt)
    if n == 0:
        return
    want, wl, P = S.window_head(Q, K, V, window, sinks, causal, scale)
    mask = S.visible(np.arange(n), n, window, sinks, causal)
    el = _weight_error(Q, K, mask, scale)[:, None]
    add = 2.0 ** -22 * mask.sum(1, keepdims=True)
    A = P @ np.abs(V)
    # a weight is at most 1 against the row's largest: below the type's normal range it is off by an absolute u * tiny
    low = u * tiny * mask.sum(1, keepdims=True) * np.abs(V).max()
    tol_o = (u + el + add) * A + u * np.abs(want) + low + tiny * u
    _near(O, want, tol_o, "out")
    _near(lse, wl, el[:, 0] + add[:, 0] + 2.0 ** -22 * np.abs(wl), "lse")
    if grads is None:
        return
    dO, dQ, dK, dV, O_in = grads
    wq, wk, wv = S.window_head_backward(Q, K, V, dO, window, sinks, causal, scale)
    d = Q.shape[1]
    dP = dO @ V.T
    delta = (dO * want).sum(1, keepdims=True)
    dS = P * (dP - delta) * scale
    adO = np.abs(dO)
    e_delta = (adO * np.abs(O_in - want)).sum(1, keepdims=True) + d * 2.0 ** -22 * (adO * np.abs(want)).sum(1, keepdims=True)
    e_dp = d * 2.0 ** -22 * (adO @ np.abs(V).T)
    e_ds = (u + el + 2.0 ** -20) * np.abs(dS) + P * scale * (e_delta + e_dp) * (1 + u) + np.where(mask, u * tiny, 0)
    e_p = (u + el) * P + np.where(mask, u * tiny, 0)
    addq, addk = add, 2.0 ** -22 * mask.sum(0)[:, None]
    tol_q = e_ds @ np.abs(K) + addq * (np.abs(dS) @ np.abs(K)) + u * np.abs(wq) + tiny * u
    tol_k = e_ds.T @ np.abs(Q) + addk * (np.abs(dS).T @ np.abs(Q)) + u * np.abs(wk) + tiny * u
    tol_v = e_p.T @ adO + addk * (P.T @ adO) + u * np.abs(wv) + tiny * u
    _near(dQ, wq, tol_q, "dq")
    return (wk, tol_k), (wv, tol_v)


def _window_case(sla2, B, Hq, Hkv, N, d, dt, window, sinks, causal, lens=None, scale=None, seed=0, layout="bhnd", train=True,
                 pad=float("nan")):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda H: torch.randn(B, H, N, d, generator=g).to(dt)
    q, k, v, do = rnd(Hq), rnd(Hkv), rnd(Hkv), rnd(Hq)
    ln = [N] * B if lens is None else lens
    for b in range(B):
        for t in (q, k, v, do):
            t[b, :, ln[b]:] = pad
    if layout == "bhnd":
        Q, K, V, DO = (t.cuda() for t in (q, k, v, do))
    else:               # one packed projection: token-major rows q | k | v | dout, more columns behind them
        H = 2 * Hq + 2 * Hkv
        buf = torch.full((B, N, H + 1, d), pad, dtype=dt).cuda()
        at = 0
        outs = []
        for t in (q, k, v, do):
            buf[:, :, at:at + t.shape[1]] = t.transpose(1, 2).cuda()
            outs.append(buf[:, :, at:at + t.shape[1]].transpose(1, 2))
            at += t.shape[1]
        Q, K, V, DO = outs
    kw = dict(window=window, sinks=sinks, causal=causal, scale=scale,
              lens=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda())
    out, lse = sla2.window_forward(Q, K, V, return_lse=True, **kw)
    grads = sla2.window_backward(Q, K, V, out, lse, DO, **kw) if train else None
    torch.cuda.synchronize()
    sc = d ** -0.5 if scale is None else scale
    O, L = _np(out), _np(lse)
    q, k, v, do = (_np(t) for t in (q, k, v, do))
    if train:
        dQ, dK, dV = (_np(t) for t in grads)
    for b in range(B):
        n = max(0, min(N, ln[b]))
        assert not O[b, :, n:].any() and (L[b, :, n:] == -np.inf).all(), "padding comes out as zero"
        if train:
            assert not dQ[b, :, n:].any() and not dK[b, :, n:].any() and not dV[b, :, n:].any()
        for hk in range(Hkv):
            sums = []
            for h in range(hk * (Hq // Hkv), (hk + 1) * (Hq // Hkv)):
                r = _check_head(dt, q[b, h, :n], k[b, hk, :n], v[b, hk, :n], O[b, h, :n], L[b, h, :n], window, sinks, causal,
                                sc, (do[b, h, :n], dQ[b, h, :n], None, None, O[b, h, :n]) if train else None)
                if r:
                    sums.append(r)
            if sums:
                for i, got in enumerate((dK, dV)):
                    want = sum(x[i][0] for x in sums)
                    # the heads' sums are rounded once; each head's own tolerance counted that rounding on its part
                    _near(got[b, hk, :n], want, sum(x[i][1] for x in sums) + _u(dt) * np.abs(want), ("dk", "dv")[i])


WINDOW_CASES = [
    # B, Hq, Hkv, N, d, dtype, window, sinks, causal, lens
    (1, 1, 1, 1, 64, BF, 1, 0, True, None),
    (1, 1, 1, 1, 128, FP, 5, 3, False, None),
    (2, 2, 1, 17, 64, FP, 4, 2, True, None),
    (1, 2, 2, 128, 128, BF, 128, 0, True, None),
    (1, 1, 1, 129, 128, BF, 1, 1, True, None),
    (1, 3, 1, 255, 64, BF, 64, 5, False, None),
    (1, 2, 1, 300, 128, FP, 1000, 0, True, None),
    (1, 2, 1, 300, 128, BF, 1000, 7, False, None),
    (2, 4, 2, 511, 128, BF, 100, 130, True, None),
    (2, 4, 4, 640, 64, BF, 129, 4, True, None),
    (1, 4, 1, 900, 64, FP, 127, 300, False, None),
    (1, 2, 1, 1153, 128, FP, 300, 16, False, None),
    (1, 1, 1, 2000, 128, BF, 700, 64, True, None),
    (5, 2, 1, 400, 128, BF, 96, 9, True, [400, 0, 1, 129, 256]),
    (4, 2, 2, 513, 64, FP, 200, 140, False, [512, 130, 0, 513]),
    (3, 3, 3, 260, 128, FP, 30, 0, False, [-4, 300, 257]),
]


@pytest.mark.parametrize("case", WINDOW_CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c[:9]))
def test_window_attention_and_its_gradients(sla2, case):
    B, Hq, Hkv, N, d, dt, window, sinks, causal, lens = case
    _window_case(sla2, B, Hq, Hkv, N, d, dt, window, sinks, causal, lens, seed=N)


@pytest.mark.parametrize("pad", [float("inf"), torch.finfo(BF).min])
def test_window_padding_may_hold_anything(sla2, pad):
    _window_case(sla2, 3, 2, 1, 200, 64, BF, 50, 130, False, [140, 60, 199], seed=3, pad=pad)


def test_window_strided_views_of_one_projection(sla2):
    _window_case(sla2, 2, 4, 2, 300, 128, BF, 70, 3, True, [300, 211], seed=4, layout="packed")
    _window_case(sla2, 1, 3, 1, 129, 64, FP, 70, 3, False, None, seed=5, layout="packed")


def test_window_scale_and_large_logits(sla2):
    _window_case(sla2, 1, 2, 1, 300, 64, BF, 90, 2, True, scale=1.5, seed=6)      # weights close to one-hot
    _window_case(sla2, 1, 2, 1, 300, 64, FP, 90, 2, False, scale=1e-3, seed=7)    # close to uniform


def test_window_fp16_of_many_keys_far_below_one(sla2):
    """The same in the window's forward pass: one sink, 32767 keys whose weights are 2^-22 to 2^-26 of its."""
    N, d = 32768, 64
    g = torch.Generator().manual_seed(25)
    q, k = torch.zeros(1, 4, N, d), torch.zeros(1, 1, N, d)
    q[0, :, :, 0] = torch.tensor([15.5, 16.5, 17, 18])[:, None]
    k[0, 0, :, 0] = torch.randn(N, generator=g) / 64
    k[0, 0, 0, 0] = 1
    v = 1 + torch.randn(1, 1, N, d, generator=g) / 8
    v[0, 0, 0] = 0
    q, k, v = (t.to(FP).cuda() for t in (q, k, v))
    out, lse = sla2.window_forward(q, k, v, N, scale=1.0, return_lse=True)
    x = (q[0, :, -1:].double() @ k[0].double().transpose(-1, -2))
    want = (torch.softmax(x, -1) @ v[0].double())[:, 0]
    # the weights' and the output's roundings, fp32 sums, and 2^-32 of the largest weight for one that is below fp16's range
    tol = (2 * _u(FP) + 2.0 ** -19 + N * 2.0 ** -24) * want.abs() + 2.0 ** -32 * N * 2
    assert ((out[0, :, -1].double() - want).abs() <= tol).all(), ((out[0, :, -1].double() - want).abs() / tol).amax(1)
    assert (lse[0, :, -1].double() - torch.logsumexp(x, -1)[:, 0]).abs().max() < 1e-5


def test_window_more_blocks_than_sms(sla2):
    """Every CTA of a persistent grid takes several items."""
    _window_case(sla2, 1, 8, 2, 5000, 64, BF, 140, 4, True, seed=8, train=False)
    _window_case(sla2, 2, 6, 2, 3333, 128, FP, 150, 20, False, [3333, 2100], seed=9)


def test_window_more_heads_than_a_grid_is_high(sla2):
    """1100 sequences of 64 heads: more than 65535 in all."""
    g = torch.Generator().manual_seed(27)
    q, do = (torch.randn(1100, 64, 3, 64, generator=g).to(BF).cuda() for _ in range(2))
    k, v = (torch.randn(1100, 1, 3, 64, generator=g).to(BF).cuda() for _ in range(2))

    def step(p):
        out, lse = sla2.window_forward(q[p], k[p], v[p], 2, return_lse=True)
        return (out, lse) + sla2.window_backward(q[p], k[p], v[p], out, lse, do[p], 2)

    whole = step(slice(0, 1100))
    for p in (slice(0, 500), slice(500, 1100)):
        for a, b in zip(whole, step(p)):
            assert torch.allclose(a[p].float(), b.float(), rtol=2.0 ** -7, atol=1e-5)      # dk, dv may be summed in other parts


def test_window_gradients_against_differences(sla2):
    """The gradient of sum(out * dout) along a direction, against the operator's own outputs."""
    B, H, N, d, dt = 1, 2, 200, 64, FP
    g = torch.Generator().manual_seed(10)
    q, k, v, do = (torch.randn(B, H, N, d, generator=g).to(dt).cuda() for _ in range(4))
    kw = dict(window=60, sinks=3, causal=True)
    out, lse = sla2.window_forward(q, k, v, return_lse=True, **kw)
    grads = sla2.window_backward(q, k, v, out, lse, do, **kw)
    f = lambda *x: float((sla2.window_forward(*x, **kw).double() * do.double()).sum())
    for i, grad in enumerate(grads):
        x = [q, k, v]
        step = grad.double() / grad.double().norm() * 2.0       # a step along the gradient
        hi, lo = (x[i].double() + step).to(dt), (x[i].double() - step).to(dt)
        moved = (grad.double() * (hi.double() - lo.double())).sum().item()
        x[i] = hi
        up = f(*x)
        x[i] = lo
        # outputs carry roundings of 2^-11 * |out| that add at random over N*H*d terms, and the step's third order stays below 2%
        noise = 4 * 2.0 ** -11 * float((out.double() * do.double()).norm())
        assert abs((up - f(*x)) - moved) <= 0.02 * abs(moved) + noise, i


def test_window_same_bits_and_other_streams_and_graphs(sla2):
    g = torch.Generator().manual_seed(11)
    q, do = (torch.randn(2, 4, 700, 128, generator=g).to(BF).cuda() for _ in range(2))
    k, v = (torch.randn(2, 2, 700, 128, generator=g).to(BF).cuda() for _ in range(2))
    kw = dict(window=150, sinks=8, causal=True)

    def step(stream=None):
        out, lse = sla2.window_forward(q, k, v, return_lse=True, stream=stream, **kw)
        return (out, lse) + tuple(sla2.window_backward(q, k, v, out, lse, do, stream=stream, **kw))

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for got in (step(), step(side)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.fill_(7)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    # two calls in flight at once, on two streams
    a, b = step(side), step()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, a)) and all(torch.equal(x, y) for x, y in zip(ref, b))


def test_window_gradients_back_to_back_in_one_workspace(sla2):
    """Calls that follow each other at once in one workspace, eagerly and as two graphs replayed in turn."""
    from block_sparse_linear_router_b200.sla2 import WindowDesc
    g = torch.Generator().manual_seed(13)
    jobs = []
    for B, Hq, Hkv, N, d, W, causal in ((1, 4, 2, 515, 64, 100, False), (2, 3, 3, 1300, 64, 300, True), (1, 2, 1, 129, 64, 5, True)):
        q, do = (torch.randn(B, Hq, N, d, generator=g).to(BF).cuda() for _ in range(2))
        k, v = (torch.randn(B, Hkv, N, d, generator=g).to(BF).cuda() for _ in range(2))
        kw = dict(window=W, sinks=3, causal=causal)
        out, lse = sla2.window_forward(q, k, v, return_lse=True, **kw)
        ref = sla2.window_backward(q, k, v, out, lse, do, **kw)
        desc = WindowDesc(B=B, Hq=Hq, Hkv=Hkv, N=N, d=d, window=W, sinks=3, causal=int(causal), dtype=0, scale=0.125)
        need = sla2.load_library().sla2_window_backward_workspace_size(desc)
        jobs.append(((q, k, v, out, lse, do), kw, ref, need))
    ws = torch.empty(max(j[3] for j in jobs), dtype=torch.uint8, device="cuda")
    run = lambda j: sla2.window_backward(*j[0], workspace=ws, **j[1])
    got = [(j, run(j)) for _ in range(8) for j in jobs]
    torch.cuda.synchronize()
    for j, y in got:
        assert all(torch.equal(a, b) for a, b in zip(j[2], y))
    graphs = []
    for j in jobs[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = [run(j) for _ in range(2)]
        graphs.append((graph, j, y))
    for _ in range(4):
        for graph, j, y in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, j, y in graphs:
        assert all(torch.equal(a, b) for z in y for a, b in zip(j[2], z))


def test_window_gradients_of_many_short_sequences(sla2):
    """More sequences than the padded batches' own order of work counts through, and fewer, with the same rows."""
    g = torch.Generator().manual_seed(17)
    B, N = 70, 300
    q, do = (torch.randn(B, 2, N, 64, generator=g).to(FP).cuda() for _ in range(2))
    k, v = (torch.randn(B, 1, N, 64, generator=g).to(FP).cuda() for _ in range(2))
    lens = torch.tensor([(37 * b) % (N + 1) for b in range(B)], dtype=torch.int32).cuda()
    kw = dict(window=40, sinks=2, causal=True)

    def step(part):
        x = [t[part] for t in (q, k, v)]
        out, lse = sla2.window_forward(*x, return_lse=True, lens=lens[part], **kw)
        return (out, lse) + sla2.window_backward(*x, out, lse, do[part], lens=lens[part], **kw)

    whole = step(slice(0, B))
    for part in (slice(0, 9), slice(9, 64), slice(64, B)):
        for a, b in zip(whole, step(part)):
            # the same arithmetic; a key tile that two blocks share may be summed in two parts instead of one
            assert torch.allclose(a[part].float(), b.float(), rtol=2.0 ** -10, atol=1e-4, equal_nan=True)
    behind = torch.arange(N, device="cuda")[None] >= lens[:, None]
    for t in (whole[0], *whole[2:]):
        assert (t.transpose(1, 2)[behind] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_window_dq_does_not_depend_on_the_order_of_work(sla2, d):
    """dq of a padded batch, and of its parts that are small enough for an order of their own, bit by bit."""
    g = torch.Generator().manual_seed(28)
    B, N = 7, 600
    q, do = (torch.randn(B, 4, N, d, generator=g).to(BF).cuda() for _ in range(2))
    k, v = (torch.randn(B, 2, N, d, generator=g).to(BF).cuda() for _ in range(2))
    lens = torch.tensor([600, 0, 129, 128, 511, 1, 300], dtype=torch.int32).cuda()
    kw = dict(window=150, sinks=3, causal=False)

    def dq(p):
        out, lse = sla2.window_forward(q[p], k[p], v[p], return_lse=True, lens=lens[p], **kw)
        return sla2.window_backward(q[p], k[p], v[p], out, lse, do[p], lens=lens[p], **kw)[0]

    whole = dq(slice(0, B))
    for a, b in ((0, 4), (1, 2), (2, 5), (4, 7), (0, 5), (1, 7)):
        assert torch.equal(whole[a:b], dq(slice(a, b))), (a, b)


@pytest.mark.parametrize("W,sinks,causal,dt", [(2, 0, True, BF), (3, 1, True, FP), (2, 3, False, BF), (4, 4, True, BF),
                                               (8, 0, True, FP), (9, 0, True, BF), (40, 2, True, BF)])
def test_window_dq_is_as_exact_as_its_type(sla2, W, sinks, causal, dt):
    """dQ's own rounding is the error of its size also where few keys are seen, and dP - delta cancels."""
    g = torch.Generator().manual_seed(19)
    q, k, v, do = (torch.randn(1, 2, 400, 64, generator=g).to(dt).cuda() for _ in range(4))
    lens = torch.tensor([390], dtype=torch.int32).cuda()
    kw = dict(window=W, sinks=sinks, causal=causal, lens=lens)
    out, lse = sla2.window_forward(q, k, v, return_lse=True, **kw)
    dq = sla2.window_backward(q, k, v, out, lse, do, **kw)[0]
    Q, K, V, G = (t.double()[:, :, :390] for t in (q, k, v, do))
    i, j = torch.arange(390, device="cuda")[:, None], torch.arange(390, device="cuda")[None]
    sees = ((j > i - W) & (j <= i)) | ((j < sinks) & (j <= i)) if causal else ((i - j).abs() < W) | (j < sinks)
    p = torch.softmax((Q @ K.transpose(-1, -2) / 8).masked_fill(~sees, -torch.inf), -1)
    dp = G @ V.transpose(-1, -2)
    want = (p * (dp - (p * dp).sum(-1, keepdim=True)) / 8) @ K
    off = float((dq[:, :, :390].double() - want).norm() / want.norm())
    # each element's rounding is off by half a step, eps / 2, at most (0.58 of it on average). Beside it, delta's:
    # from 9 keys on O's roundings of eps / 2 an element, which add at random in a sum over d and lose against
    # dP by the square root of the keys seen: not more than a third of the rounding, in squares a ninth
    assert off <= torch.finfo(dt).eps / 2 * (1 if W + sinks <= 8 else (1 + 1 / 9) ** 0.5)


def _normal_rounding(x, dt):
    """What rounding x to dt costs, in norm, were all of it in the type's normal range."""
    y = x * 2.0 ** -float(torch.log2(x.abs().max()).floor())
    return float((y.to(dt).double() - y).norm() / y.norm())


@pytest.mark.parametrize("size,vsize,qsize", [(1.0, 1.0, 1.0), (1e-2, 1.0, 1.0), (1e-3, 1.0, 1.0), (1e-4, 1.0, 1.0), (1e-5, 8.0, 1.0),
                                              (1e-3, 1e-2, 1.0), (2e3, 100.0, 0.01)])
def test_window_fp16_gradients_of_any_size(sla2, size, vsize, qsize):
    """Gradients as exact as their type for dout far below and above 1: nothing on the way to them vanishes or overflows."""
    g = torch.Generator().manual_seed(23)
    N, d, dt = 1100, 64, FP
    q, do = (torch.randn(2, 4, N, d, generator=g) for _ in range(2))
    k, v = (torch.randn(2, 2, N, d, generator=g) for _ in range(2))
    do[1] *= 0.25                            # sequences and heads of unlike size
    do[:, 2:] *= 0.125
    q, k, v, do = ((t * f).to(dt).cuda() for t, f in ((q, qsize), (k, qsize), (v, vsize), (do, size)))
    kw = dict(window=300, sinks=2, causal=True)
    out, lse = sla2.window_forward(q, k, v, return_lse=True, **kw)
    grads = sla2.window_backward(q, k, v, out, lse, do, **kw)
    Q, G = q.double(), do.double()
    K, V = (t.double().repeat_interleave(2, 1) for t in (k, v))
    i, j = torch.arange(N, device="cuda")[:, None], torch.arange(N, device="cuda")[None]
    sees = ((j > i - 300) | (j < 2)) & (j <= i)
    p = torch.softmax((Q @ K.transpose(-1, -2) / 8).masked_fill(~sees, -torch.inf), -1)
    dp = G @ V.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / 8
    pair = lambda x: x.view(2, 2, 2, N, d).sum(2)
    for name, got, want in zip(("dq", "dk", "dv"), grads, (ds @ K, pair(ds.transpose(-1, -2) @ Q), pair(p.transpose(-1, -2) @ G))):
        assert torch.isfinite(got).all()
        for b in range(2):
            for h in range(got.shape[1]):
                w = want[b, h]
                off = float((got[b, h].double() - w).norm() / w.norm())
                own = float((w.to(dt).double() - w).norm() / w.norm())
                full = _normal_rounding(w, dt)
                # the output's own rounding, and one of the operands (P; dS for dk; what O's leaves in delta for dq, less
                # than that), each pair's on its own and so as large in norm; a tenth for what a sample is off
                assert off <= 1.1 * (own ** 2 + full ** 2) ** 0.5, (name, b, h, off / own)


def test_window_fp16_dv_of_many_keys(sla2):
    """Weights of 1 / 83679, between 200 and 201 of fp16's smallest steps, reach dv as they are."""
    N, d = int(2 ** 24 / 200.5), 64
    g = torch.Generator().manual_seed(26)
    q = torch.zeros(1, 1, N, d, dtype=FP).cuda()
    k, v = (torch.randn(1, 1, N, d, generator=g).to(FP).cuda() for _ in range(2))
    do = torch.zeros(1, 1, N, d, dtype=FP).cuda()
    rows = torch.randperm(N, generator=g)[:64].cuda()
    do[0, 0, rows] = (1 + torch.randn(64, d, generator=g) / 8).to(FP).cuda()
    out, lse = sla2.window_forward(q, k, v, N, causal=False, return_lse=True)
    dv = sla2.window_backward(q, k, v, out, lse, do, N, causal=False)[2]
    want = (do.double().sum(2) / N)[0, 0]
    # P's rounding, the output's, and fp32 sums of 64 numbers
    assert ((dv[0, 0].double() - want).abs() <= (2 * _u(FP) + 2.0 ** -15) * want).all()


def test_window_rows_that_see_few_keys_have_exact_gradients(sla2):
    """Under a wide window too, dq of rows with 2 to 8 keys is off by its own rounding alone: the first rows of a causal
    sequence, and short sequences of a padded batch."""
    g = torch.Generator().manual_seed(24)
    for dt in (BF, FP):
        for causal, lens, rows in ((True, [200] * 4, (1, 2)), (True, [200] * 4, (2, 4)), (True, [5, 200, 8, 3], (1, 3)), (False, [2] * 4, (0, 2)),
                                   (False, [3, 4, 200, 5], (0, 3))):
            q, do = (torch.randn(4, 16, 200, 64, generator=g).to(dt).cuda() for _ in range(2))
            k, v = (torch.randn(4, 8, 200, 64, generator=g).to(dt).cuda() for _ in range(2))
            kw = dict(window=150, sinks=2, causal=causal, lens=torch.tensor(lens, dtype=torch.int32).cuda())
            out, lse = sla2.window_forward(q, k, v, return_lse=True, **kw)
            dq = sla2.window_backward(q, k, v, out, lse, do, **kw)[0]
            off = want = own = 0.0
            for b, n in enumerate(lens):
                if not causal and n > 8:
                    continue
                n = min(n, 8)
                Q, G = (t[b, :, :n].double() for t in (q, do))
                K, V = (t[b, :, :n].double().repeat_interleave(2, 0) for t in (k, v))
                x = Q @ K.transpose(-1, -2) / 8
                if causal:
                    x = x.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -torch.inf)
                p = torch.softmax(x, -1)
                dp = G @ V.transpose(-1, -2)
                w = (p * (dp - (p * dp).sum(-1, keepdim=True)) / 8 @ K)[:, rows[0]:rows[1]]
                off += float((dq[b, :, :n].double()[:, rows[0]:rows[1]] - w).square().sum())
                own += float((w.to(dt).double() - w).square().sum())
            assert off ** 0.5 <= 1.05 * own ** 0.5, (dt, causal, lens, rows, (off / own) ** 0.5)


def test_window_given_output_and_status(sla2):
    q, k, v = (torch.randn(1, 2, 150, 64, dtype=torch.float32).to(BF).cuda() for _ in range(3))
    ref = sla2.window_forward(q, k, v, 40)
    big = torch.full((1, 150, 3, 64), 5.0, dtype=BF).cuda()
    status = torch.full((1,), 99, dtype=torch.int32).cuda()
    out = big[:, :, :2].transpose(1, 2)
    assert sla2.window_forward(q, k, v, 40, out=out, status=status) is out
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and (big[:, :, 2] == 5).all() and status.item() == 0


def test_window_far_rows(sla2):
    """Token strides that put rows more than 2^31 elements from the base."""
    N, d, stride = 2200, 64, 1 << 20
    buf = torch.empty(N * stride, dtype=BF, device="cuda")
    x = torch.randn(1, 3, N, d, generator=torch.Generator().manual_seed(12)).to(BF).cuda()
    far = buf.as_strided((1, 3, N, d), (3 * d, d, stride, 1))
    far.copy_(x)
    q, k, v = (far[:, i:i + 1] for i in range(3))
    out, lse = sla2.window_forward(q, k, v, 50, 2, return_lse=True)
    o2, l2 = sla2.window_forward(*(x[:, i:i + 1].contiguous() for i in range(3)), 50, 2, return_lse=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    g1 = sla2.window_backward(q, k, v, out, lse, q, 50, 2)
    g2 = sla2.window_backward(*(x[:, i:i + 1].contiguous() for i in range(3)), o2, l2, x[:, :1].contiguous(), 50, 2)
    assert all(torch.equal(a, b) for a, b in zip(g1, g2))


def test_window_refuses_broadcast_strides(sla2):
    q = torch.zeros(1, 2, 16, 64, dtype=BF).cuda()
    with pytest.raises(sla2.Sla2Error):
        sla2.window_forward(q, q[:, :1].expand(1, 2, 16, 64), q, 4)


# ------------------------------------------------------------------ the cache

class Book:
    """A cache kept by the oracle beside the GPU's."""

    def __init__(self, pages, Hkv, page, d, seed):
        rng = np.random.default_rng(seed)
        self.page = page
        self.codes = [rng.integers(-127, 128, (pages, Hkv, page, d)).astype(np.int8) for _ in range(2)]
        self.scale = [rng.uniform(0.001, 0.02, (pages, Hkv)).astype(np.float32) for _ in range(2)]
        self.left_out = False

    def cuda(self, sla2):
        c = [torch.from_numpy(x.copy()).cuda() for x in self.codes + self.scale]
        return sla2.KVCache(*c)

    def append(self, k, v, table, lens, cu, rope, interleaved, dt, q=None):
        """Returns rotated q, k; rows that are left out keep NaN."""
        out = [None if x is None else np.full(x.shape, np.nan) for x in (q, k)]
        for b, n0 in enumerate(lens):
            for t in range(cu[b], cu[b + 1]):
                pos = n0 + t - cu[b]
                if pos // self.page >= table.shape[1] or not 0 <= table[b, pos // self.page] < len(self.codes[0]) or (
                        rope is not None and pos >= len(rope[0])):
                    self.left_out = True
                    continue
                turn = (lambda x: x) if rope is None else (lambda x: S.rotate(x, rope[0][pos], rope[1][pos], interleaved, dt))
                for x, o in ((q, out[0]), (k, out[1])):
                    if x is not None:
                        o[t] = np.stack([turn(row) for row in x[t]])
            at, end = n0, n0 + cu[b + 1] - cu[b]
            while at < end:                       # the rows that one page takes
                stop = min(end, (at // self.page + 1) * self.page)
                rows = slice(cu[b] + at - n0, cu[b] + stop - n0)
                ok = ~np.isnan(out[1][rows]).all(axis=(1, 2)) | np.isnan(k[rows]).any(axis=(1, 2))
                pi = at // self.page
                ok &= pi < table.shape[1] and 0 <= table[b, min(pi, table.shape[1] - 1)] < len(self.codes[0])
                if rope is not None:
                    ok &= np.arange(at, stop) < len(rope[0])
                n = int(ok.sum())
                if n:
                    p = table[b, pi]
                    for which, x in enumerate((out[1], v)):
                        for h in range(k.shape[1]):
                            self.codes[which][p, h], self.scale[which][p, h] = S.append_rows(
                                self.codes[which][p, h], self.scale[which][p, h], at % self.page, x[rows][:n, h])
                at = stop
        return out

    def values(self, which, pages, h, n):
        x = self.codes[which][pages, h].astype(np.float64) * self.scale[which][pages, h].astype(np.float64)[:, None, None]
        return x.reshape(-1, x.shape[-1])[:n]


def _cu(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int32)


def _table(lens, page, pages, seed, width=None):
    held = [-(-int(n) // page) for n in lens]
    order = np.random.default_rng(seed).permutation(pages)
    assert sum(held) <= pages
    t = np.full((len(lens), width or max(max(held), 1)), -7, np.int32)      # entries that nobody needs
    at = 0
    for b, n in enumerate(held):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def _dev(x, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dt is None else t.to(dt)


def _rope(rows, half, seed=0):
    a = np.arange(rows)[:, None] * np.geomspace(1, 0.01, half)[None] + seed
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _same_cache(cache, book, what=""):
    for got, want in ((cache.k_codes, book.codes[0]), (cache.v_codes, book.codes[1])):
        assert np.array_equal(got.cpu().numpy(), want), what + "codes"
    for got, want in ((cache.k_scale, book.scale[0]), (cache.v_scale, book.scale[1])):
        assert np.array_equal(got.cpu().numpy(), want, equal_nan=True), what + "scales"


APPEND_CASES = [
    # Hq, Hkv, page, d, dtype, lens, news, rope_dim, interleaved
    (1, 1, 16, 64, BF, [0], [1], 64, False),
    (4, 2, 64, 128, BF, [5, 63, 64, 130], [1, 1, 1, 1], 128, False),
    (6, 3, 32, 64, FP, [0, 31, 7, 100, 32], [3, 2, 0, 70, 33], 32, True),
    (2, 2, 128, 128, FP, [127, 0, 40], [300, 129, 0], 64, True),
    (3, 1, 16, 128, BF, [15, 16, 17, 0], [1, 200, 15, 16], 112, False),
    (8, 1, 64, 64, BF, [10], [500], 0, False),
    (4, 4, 128, 128, BF, [50, 3], [60, 0], 48, True),
    (2, 1, 16, 64, FP, list(range(300)), [1] * 300, 16, False),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c[:5] + c[7:]))
def test_append_to_the_bit(sla2, case):
    Hq, Hkv, page, d, dt, lens, news, rot, inter = case
    rng = np.random.default_rng(len(lens) + d)
    cu, T = _cu(news), sum(news)
    total = [a + b for a, b in zip(lens, news)]
    pages = sum(-(-n // page) for n in total) + 3
    table = _table(total, page, pages, 1)
    # values over several powers of two, so that some pages' scales grow and others' do not
    q, k, v = (S.round_to(rng.standard_normal((T, H, d)) * np.exp2(rng.integers(-6, 3, (T, H, 1))), dt) for H in (Hq, Hkv, Hkv))
    rope = _rope(max(total) + 1, rot // 2) if rot else None
    book = Book(pages, Hkv, page, d, 2)
    cache = book.cuda(sla2)
    k_out = torch.empty(T, Hkv, d, dtype=dt).cuda()
    status = torch.full((1,), 9, dtype=torch.int32).cuda()
    args = (_dev(k, dt), _dev(v, dt), _dev(table), _dev(np.array(lens, np.int32)), _dev(cu))
    dr = None if rope is None else tuple(_dev(x) for x in rope)
    q_out = sla2.cache_append(cache, *args, rope=dr, interleaved=inter, q=_dev(q, dt), k_out=k_out, status=status)
    torch.cuda.synchronize()
    wq, wk = book.append(k, v, table, lens, cu, rope, inter, dt, q)
    assert status.item() == 0
    assert np.array_equal(_np(q_out), wq) and np.array_equal(_np(k_out), wk)
    _same_cache(cache, book)
    # without queries, on strided rows, the same cache again
    c2 = Book(pages, Hkv, page, d, 2).cuda(sla2)
    packed = torch.zeros(T, 2 * Hkv + 1, d, dtype=dt).cuda()
    packed[:, :Hkv], packed[:, Hkv:2 * Hkv] = args[0], args[1]
    assert sla2.cache_append(c2, packed[:, :Hkv], packed[:, Hkv:2 * Hkv], *args[2:], rope=dr, interleaved=inter) is None
    _same_cache(c2, book)


def test_append_borders_between_codes(sla2):
    """Quotients that fall on, and next to, the middle between two codes."""
    d, page = 64, 16
    for dt in (BF, FP):
        for top in (127.0, 254.0, 381.0 if dt == FP else 63.5, 1.0, 100.0):
            s = float(np.float32(np.float32(top) / np.float32(127)))
            mid = (np.arange(d * 6) % 127 + 0.5) * s * np.where(np.arange(d * 6) % 2, 1, -1)
            rows = S.round_to(np.concatenate([[top], mid[:-1]]).reshape(6, 1, d), dt)
            book = Book(2, 1, page, d, 3)
            cache = book.cuda(sla2)
            table, cu = np.array([[1]], np.int32), _cu([6])
            sla2.cache_append(cache, _dev(rows, dt), _dev(rows, dt), _dev(table), _dev(np.zeros(1, np.int32)), _dev(cu))
            book.append(rows, rows, table, [0], cu, None, False, dt)
            _same_cache(cache, book, f"{dt} {top}: ")


def test_append_extremes(sla2):
    """Zeros, the smallest and the largest values, and what is not finite."""
    d, page, dt = 64, 16, BF
    big, small = torch.finfo(dt).max, 2.0 ** -133
    for first, then in ((0.0, 0.0), (0.0, small), (small, small * 3), (small, big), (big, small), (1.0, float("inf")),
                        (float("nan"), 1.0), (2.0, float("nan"))):
        book = Book(1, 1, page, d, 4)
        cache = book.cuda(sla2)
        for n, x in enumerate((first, then)):
            row = np.zeros((1, 1, d))
            row[0, 0, :3] = [x, -x / 2 if np.isfinite(x) else 1, 0]
            row = S.round_to(row, dt)
            table, cu = np.zeros((1, 1), np.int32), _cu([1])
            sla2.cache_append(cache, _dev(row, dt), _dev(row, dt), _dev(table), _dev(np.array([n], np.int32)), _dev(cu))
            for w in range(2):
                book.codes[w][0, 0], book.scale[w][0, 0] = S.append_rows(book.codes[w][0, 0], book.scale[w][0, 0], n, row[:, 0])
        got = cache.k_scale.cpu().numpy()
        assert np.array_equal(got, book.scale[0], equal_nan=True), (first, then)
        if np.isfinite(got).all():
            assert np.array_equal(cache.k_codes.cpu().numpy()[:, :, :2], book.codes[0][:, :, :2]), (first, then)


def test_append_leaves_out_what_is_out_of_range(sla2):
    d, page, dt, Hkv = 64, 16, FP, 2
    lens, news = [10, 0, 30, 5], [10, 4, 5, 2]
    cu, T = _cu(news), sum(news)
    table = np.array([[0, 99], [-1, 2], [3, 4], [5, 5]], np.int32)      # 99 and -1 are no pages; 34 tokens need 3 entries
    rng = np.random.default_rng(7)
    q, k, v = (S.round_to(rng.standard_normal((T, Hkv, d)), dt) for _ in range(3))
    for rows, lost in ((64, True), (33, True)):
        rope = _rope(rows, 16)
        book = Book(6, Hkv, page, d, 5)
        cache = book.cuda(sla2)
        status = torch.zeros(1, dtype=torch.int32).cuda()
        q_out, k_out = (torch.full((T, Hkv, d), float("nan"), dtype=dt).cuda() for _ in range(2))
        sla2.cache_append(cache, _dev(k, dt), _dev(v, dt), _dev(table), _dev(np.array(lens, np.int32)), _dev(cu),
                          rope=tuple(_dev(x) for x in rope), q=_dev(q, dt), q_out=q_out, k_out=k_out, status=status)
        torch.cuda.synchronize()
        wq, wk = book.append(k, v, table, lens, cu, rope, False, dt, q)
        assert status.item() == 6 and book.left_out == lost
        assert np.array_equal(_np(q_out), wq, equal_nan=True) and np.array_equal(_np(k_out), wk, equal_nan=True)
        _same_cache(cache, book)
    # offsets that go down, reach behind the rows, or lengths below zero: nothing happens for those sequences
    for bad_cu, bad_len in (([0, 10, 5, 14, 16], lens), ([0, 10, 14, 400, 400], lens), (list(cu), [10, 0, -3, 5])):
        book = Book(6, Hkv, page, d, 6)
        cache = book.cuda(sla2)
        status.zero_()
        sla2.cache_append(cache, _dev(k, dt), _dev(v, dt), _dev(table), _dev(np.array(bad_len, np.int32)),
                          _dev(np.array(bad_cu, np.int32)), status=status)
        assert status.item() == 6


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("inter", [False, True])
def test_append_turns_to_the_bit(sla2, dt, inter):
    """Sums that cancel, that fall on the middle between two values of the type, overflow or vanish."""
    rng = np.random.default_rng(21)
    T, d, page = 400, 64, 64
    big, small = torch.finfo(dt).max, torch.finfo(dt).smallest_normal
    x = S.round_to(rng.standard_normal((T, 2, d)) * np.exp2(rng.integers(-12, 12, (T, 2, d))), dt)
    pick = rng.integers(0, 12, x.shape)
    for n, value in enumerate((0.0, -0.0, big, -big, small, small * torch.finfo(dt).eps, 1.0, float("inf"), float("nan"))):
        x[pick == n] = S.round_to(np.full((pick == n).sum(), value), dt)
    x[:200] = np.where(np.isfinite(x[:200]), x[:200], 1.0)
    cos, sin = _rope(T, d // 2)
    # equal members and angles: differences that cancel to the last bits, or altogether
    if inter:
        x[:100, :, 1::2] = x[:100, :, 0::2]
    else:
        x[:100, :, d // 2:] = x[:100, :, :d // 2]
    sin[:50] = np.nextafter(cos[:50], np.float32(9))
    sin[50:60] = cos[50:60]
    # halves of a step of the type: p c is an odd multiple of half a step
    cos[100:150], sin[100:150] = np.float32(1 + torch.finfo(dt).eps / 2), 0
    cos[150:170], sin[150:170] = np.float32(1.5), np.float32(2.0 ** -30)
    cos[170:200], sin[170:200] = np.float32(2.0 ** -130), np.float32(-2.0 ** -140)
    cos[300:310], sin[310:320] = np.float32("inf"), np.float32("nan")
    cos[320:340], sin[320:340] = np.float32(3e38), np.float32(3e38)
    cache = sla2.KVCache.empty(T // page + 1, 2, page, d)
    table = torch.arange(T // page + 1, dtype=torch.int32).cuda()[None]
    k = _dev(x, dt)
    k_out = torch.empty_like(k)
    q_out = sla2.cache_append(cache, k, k, table, _dev(np.zeros(1, np.int32)), _dev(_cu([T])), rope=(_dev(cos), _dev(sin)),
                              interleaved=inter, q=k, k_out=k_out)
    with np.errstate(all="ignore"):
        want = np.stack([[S.rotate(x[t, h], cos[t], sin[t], inter, dt) for h in range(2)] for t in range(T)])
    for got in (_np(k_out), _np(q_out)):
        assert np.array_equal(got, want, equal_nan=True)
        live = ~np.isnan(want)
        assert np.array_equal(np.signbit(got[live]), np.signbit(want[live]))


def test_append_rows_that_start_late(sla2):
    """The first offset need not be 0, and rows between nobody's offsets stay: one token each behind 5 rows."""
    d, page, dt = 64, 16, BF
    rng = np.random.default_rng(22)
    lens, cu, T = [3, 15, 16, 0], np.array([5, 6, 6, 7, 9], np.int32), 12
    k = S.round_to(rng.standard_normal((T, 2, d)), dt)
    table = _table([n + c for n, c in zip(lens, np.diff(cu))], page, 8, 3)
    book = Book(8, 2, page, d, 9)
    cache = book.cuda(sla2)
    q_out = torch.full((T, 2, d), 4.0, dtype=dt).cuda()
    rope = _rope(64, 32)
    sla2.cache_append(cache, _dev(k, dt), _dev(k, dt), _dev(table), _dev(np.array(lens, np.int32)), _dev(cu),
                      rope=tuple(_dev(x) for x in rope), q=_dev(k, dt), q_out=q_out)
    wq, _ = book.append(k, k, table, lens, cu, rope, False, dt, k)
    _same_cache(cache, book)
    got = _np(q_out)
    assert np.array_equal(got[5:9], wq[5:9]) and (got[:5] == 4).all() and (got[9:] == 4).all()


def _in_order(cu, lens, T):
    """The sequences that a step takes: those before the first whose offsets go down or leave the rows, but for lengths below zero."""
    ok = [0 <= a <= b <= T for a, b in zip(cu, cu[1:])] + [False]
    return [b for b in range(ok.index(False)) if lens[b] >= 0]


@pytest.mark.parametrize("cu,lens,good", [([0, 100, 5, 6, 8], [20, 0, 3, 9], 1), ([0, 10, 5, 40, 41], [10, 0, 30, 5], 1),
                                          ([0, 10, 14, 400, 400], [10, 0, 30, 5], 2), ([0, 10, 14, 33, 50], [10, -3, 0, 40], 3),
                                          ([-4, 10, 12, 30, 31], [0, 15, 16, 1], 0), ([7, 3, 90, 90, 100], [1, 60, 5, 0], 0),
                                          ([3, 40, 40, 77, 76], [100, 3, 0, 5], 3)])
def test_append_of_bad_offsets_leaves_out_what_is_behind(sla2, cu, lens, good):
    """Sequences before the first bad pair of offsets are appended whole; that one's and those behind it stay as they were."""
    d, page, dt, Hkv, T = 64, 16, BF, 2, 100
    rng = np.random.default_rng(37)
    table = np.arange(4 * 12, dtype=np.int32).reshape(4, 12)
    k, v = (S.round_to(rng.standard_normal((T, Hkv, d)), dt) for _ in range(2))
    book = Book(4 * 12, Hkv, page, d, 38)
    cache = book.cuda(sla2)
    status = torch.zeros(1, dtype=torch.int32).cuda()
    q_out, k_out = (torch.full((T, Hkv, d), 3.0, dtype=dt).cuda() for _ in range(2))
    sla2.cache_append(cache, _dev(k, dt), _dev(v, dt), _dev(table), _dev(np.array(lens, np.int32)), _dev(np.array(cu, np.int32)),
                      q=_dev(k, dt), q_out=q_out, k_out=k_out, status=status)
    assert status.item() == 6
    taken = _in_order(cu, lens, T)
    assert len(taken) == good
    want = np.full((T, Hkv, d), 3.0)
    for b in taken:
        book.append(k, v, table[b:b + 1], lens[b:b + 1], cu[b:b + 2], None, False, dt)
        want[cu[b]:cu[b + 1]] = k[cu[b]:cu[b + 1]]
    _same_cache(cache, book)
    assert np.array_equal(_np(k_out), want) and np.array_equal(_np(q_out), want)


@pytest.mark.parametrize("at", [1, 300, 699])
def test_append_and_attention_of_many_sequences_up_to_a_bad_offset(sla2, at):
    """More sequences than a block has threads, the offsets of sequence `at` going down."""
    d, page, dt, B = 64, 16, BF, 700
    rng = np.random.default_rng(40)
    cu = np.arange(B + 1, dtype=np.int32)
    cu[at + 1] = 0
    lens = (np.arange(B) % 13).astype(np.int32)
    table = np.arange(B, dtype=np.int32)[:, None]
    k, v = (S.round_to(rng.standard_normal((B, 1, d)), dt) for _ in range(2))
    for width in (1, 20):                    # items of a warp, and of a thread block
        book = Book(B, 1, page, d, 41)
        cache = book.cuda(sla2)
        wide = np.full((B, width), -1, np.int32)
        wide[:, :1] = table
        status = torch.zeros(1, dtype=torch.int32).cuda()
        args = (_dev(wide), _dev(lens), _dev(cu))
        sla2.cache_append(cache, _dev(k, dt), _dev(v, dt), *args, status=status)
        assert status.item() == 6
        for b in range(at):
            book.append(k, v, table[b:b + 1], lens[b:b + 1], [b, b + 1], None, False, dt)
        _same_cache(cache, book)
        status.zero_()
        o = torch.full((B, 2, d), 6.0, dtype=dt).cuda()
        q = S.round_to(rng.standard_normal((B, 2, d)), dt)
        sla2.cache_attention(cache, _dev(q, dt), *args, out=o, status=status)
        assert status.item() == 6
        o = _np(o)
        assert (o[at:] == 6).all()
        for b in range(at):
            n = int(lens[b]) + 1
            K, V = (book.values(w, table[b], 0, n) for w in (0, 1))
            for h in range(2):
                _near_decode(dt, o[b:b + 1, h], q[b:b + 1, h], K, V, np.ones((1, n), bool), d ** -0.5, f"{b} {h}")


def test_append_rows_behind_the_last_sequence_stay(sla2):
    d, page, dt = 64, 32, BF
    cu = _cu([2, 1])
    k = torch.randn(8, 1, d).to(dt).cuda()
    k[3:] = float("nan")
    table = np.array([[1], [0]], np.int32)
    cache = Book(3, 1, page, d, 8).cuda(sla2)
    before = cache.k_codes.clone()
    out = torch.full((8, 1, d), 3.0, dtype=dt).cuda()
    sla2.cache_append(cache, k, k, _dev(table), _dev(np.zeros(2, np.int32)), _dev(cu), q=k.clone(), q_out=out)
    assert (out[3:] == 3).all() and torch.equal(cache.k_codes[2], before[2])
    assert torch.equal(cache.k_codes[1, :, 2:], before[1, :, 2:]) and torch.isfinite(cache.k_scale).all()
    assert sla2.cache_append(cache, k[:0], k[:0], _dev(table), _dev(np.zeros(2, np.int32)), _dev(np.zeros(3, np.int32)),
                             q=k[:0]).shape == (0, 1, d)


def _check_decode(sla2, Hq, Hkv, page, d, dt, lens, news, window, sinks, seed=0, scale=None, spread=1.0, extra_rows=0):
    """cache_attention over random codes against the oracle."""
    rng = np.random.default_rng(seed)
    cu, T = _cu(news), sum(news) + extra_rows
    total = [a + b for a, b in zip(lens, news)]
    pages = sum(-(-n // page) for n in total) + 2
    table = _table(total, page, pages, seed + 1)
    book = Book(pages, Hkv, page, d, seed + 2)
    q = S.round_to(rng.standard_normal((T, Hq, d)) * spread, dt)
    if window is not None:      # pages that no query sees may be gone
        for b, n in enumerate(lens):
            for p in range(sinks // page + 1, (n - window) // page):
                if p * page >= sinks and news[b]:
                    table[b, p] = -5
    cache = book.cuda(sla2)
    status = torch.zeros(1, dtype=torch.int32).cuda()
    out = torch.full((T, Hq, d), 11.0, dtype=dt).cuda()
    sla2.cache_attention(cache, _dev(q, dt), _dev(table), _dev(np.array(lens, np.int32)), _dev(cu), window=window, sinks=sinks,
                         scale=scale, out=out, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    got, g, u = _np(out), Hq // Hkv, _u(dt)
    sc = d ** -0.5 if scale is None else scale
    assert (got[cu[-1]:] == 11).all(), "rows behind the last sequence stay"
    for b, n0 in enumerate(lens):
        if not news[b]:
            continue
        n = total[b]
        rows = slice(cu[b], cu[b + 1])
        mask = S.visible(np.arange(n0, n), n, n if window is None else window, sinks, True)
        held = table[b, :-(-n // page)]
        for h in range(Hq):
            K, V = (book.values(w, held, h // g, n) for w in (0, 1))
            Q = q[rows, h]
            P, _ = S.weights(Q, K, mask, sc)
            want = P @ V
            el = _weight_error(Q, K, mask, sc)[:, None]
            # a query row is rounded to steps of its largest magnitude / 32639: each element is off by half a step,
            # 2^-15.99 of that magnitude, so a logit by at most that times sum |k| scale, and a weight, relative to
            # the others, by twice that (the row's largest logit moves too)
            el = el + 2 * 2.0 ** -15.9 * np.abs(Q).max(1, keepdims=True) * np.abs(K).sum(1).max() * sc
            seen = mask.sum(1, keepdims=True)
            A = P @ np.abs(V)
            tol = (2.0 ** -11 + el + 2.0 ** -22 * seen) * A + u * np.abs(want) + 2.0 ** -25 * seen * np.abs(V).max() + _tiny(dt) * u
            _near(got[rows, h], want, tol, f"sequence {b} head {h}")


DECODE_CASES = [
    # Hq, Hkv, page, d, dtype, lens, news, window, sinks
    (1, 1, 16, 64, BF, [0], [1], None, 0),
    (1, 1, 16, 64, FP, [1], [1], 1, 0),
    (4, 2, 16, 64, BF, [40, 15, 16, 17], [1, 1, 1, 1], None, 0),
    (8, 1, 64, 128, BF, [1000, 63, 64, 0], [1, 1, 1, 1], None, 0),
    (12, 12, 32, 128, FP, [500], [1], None, 0),
    (6, 2, 128, 128, BF, [300, 700], [1, 2], 100, 5),
    (32, 2, 64, 64, FP, [257, 90, 128], [1, 1, 1], 64, 4),
    (7, 1, 16, 128, FP, [333, 0, 45], [3, 5, 0], 50, 33),
    (16, 2, 32, 128, BF, [150, 64, 9], [4, 7, 20], 40, 3),
    (24, 1, 64, 64, BF, [100, 200], [1, 9], None, 0),
    (3, 3, 128, 64, FP, [5000], [1], 4096, 64),
    (2, 1, 16, 128, BF, list(range(0, 600, 3)), [1] * 200, None, 0),
]


@pytest.mark.parametrize("case", DECODE_CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c[:5] + c[7:]))
def test_cache_attention(sla2, case):
    Hq, Hkv, page, d, dt, lens, news, window, sinks = case
    _check_decode(sla2, Hq, Hkv, page, d, dt, lens, news, window, sinks, seed=d + len(lens))


SHORT_CASES = [
    # Hq, Hkv, page, d, dtype, lens, news, window, sinks: tables of 256 keys at most
    (8, 8, 16, 64, BF, [i % 60 for i in range(300)], [1] * 300, None, 0),       # more items than warps
    (3, 3, 32, 128, FP, [14, 0, 90], [7, 1, 3], None, 0),
    (14, 2, 64, 128, BF, [100, 185, 0, 63], [5, 7, 0, 1], 33, 2),
    (32, 2, 128, 64, FP, [200, 128, 255], [1, 1, 1], 20, 100),
    (7, 1, 16, 64, BF, [230, 17], [26, 2], 200, 17),
    (4, 1, 128, 128, BF, [255], [1], None, 0),
]


@pytest.mark.parametrize("case", SHORT_CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c[:5] + c[7:]))
def test_cache_attention_short_tables(sla2, case):
    _check_decode(sla2, *case, seed=sum(case[5]), extra_rows=3)


def test_cache_attention_lengths_behind_a_short_table(sla2):
    """What a length says beyond the table's pages is left out and reported; the other sequences do not mind."""
    d, page, Hkv, g, dt = 64, 32, 2, 4, BF
    rng = np.random.default_rng(31)
    cache = Book(12, Hkv, page, d, 32).cuda(sla2)
    table = _dev(np.arange(12, dtype=np.int32).reshape(3, 4))
    q = _dev(rng.standard_normal((3, Hkv * g, d)), dt)
    cu = _dev(_cu([1, 1, 1]))
    for window in (None, 50):
        ref = sla2.cache_attention(cache, q, table, _dev(np.array([100, 90, 127], np.int32)), cu, window=window)
        for bad in (128, 5000, 2_000_000_000, -1):
            status = torch.zeros(1, dtype=torch.int32).cuda()
            out = sla2.cache_attention(cache, q, table, _dev(np.array([100, bad, 127], np.int32)), cu, window=window, status=status)
            torch.cuda.synchronize()
            assert status.item() == 6
            assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])


def _near_decode(dt, got, Q, K, V, mask, sc, what, low=2.0 ** -25):
    """Rows of cache_attention against the oracle, with the tolerance of _check_decode (its reasons stand there)."""
    P, _ = S.weights(Q, K, mask, sc)
    want = P @ V
    el = _weight_error(Q, K, mask, sc)[:, None] + 2 * 2.0 ** -15.9 * np.abs(Q).max(1, keepdims=True) * np.abs(K).sum(1).max(initial=0) * sc
    seen = mask.sum(1, keepdims=True)
    tol = (2.0 ** -11 + el + 2.0 ** -22 * seen) * (P @ np.abs(V)) + _u(dt) * np.abs(want) + low * seen * np.abs(V).max(initial=0)
    _near(got, want, tol + _tiny(dt) * _u(dt), what)


@pytest.mark.parametrize("news", [[1, 1, 1], [3, 2, 5]])
def test_cache_attention_lengths_behind_a_wide_table(sla2, news):
    """A length far behind a table costs what the table holds; what it says beyond is left out and reported."""
    d, page, Hkv, g, dt, width = 64, 32, 2, 4, BF, 40
    rng = np.random.default_rng(33)
    book = Book(3 * width, Hkv, page, d, 34)
    cache = book.cuda(sla2)
    table = _dev(np.arange(3 * width, dtype=np.int32).reshape(3, width))
    cu, n = _cu(news), width * page
    q = S.round_to(rng.standard_normal((cu[-1], Hkv * g, d)), dt)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    sla2.cache_attention(cache, _dev(q, dt), table, _dev(np.array([1000, 900, 1270], np.int32)), _dev(cu))
    for window, sinks in ((None, 0), (50, 0), (50, 40)):
        for bad in (n, n + 700, 2_000_000_000, 0x7fffffff - news[1]):
            lens = [1000, bad, 1270]
            status = torch.zeros(1, dtype=torch.int32).cuda()
            args = (_dev(q, dt), table, _dev(np.array(lens, np.int32)), _dev(cu))
            start.record()
            out = sla2.cache_attention(cache, *args, window=window, sinks=sinks, status=status)
            end.record()
            torch.cuda.synchronize()
            assert status.item() == 6
            assert start.elapsed_time(end) < 200      # ms; the valid lengths alone take well below one
            out = _np(out)
            for b, n0 in enumerate(lens):
                i, j = n0 + np.arange(news[b])[:, None], np.arange(n)[None]
                mask = (j <= i) & ((j > i - (window or 1 << 40)) | (j < sinks))
                for h in range(Hkv * g):
                    K, V = (book.values(w, np.arange(b * width, (b + 1) * width), h // g, n) for w in (0, 1))
                    _near_decode(dt, out[cu[b]:cu[b + 1], h], q[cu[b]:cu[b + 1], h], K, V, mask, d ** -0.5, f"{bad}: {b} {h}")


def test_cache_attention_long_and_lone(sla2):
    """One sequence over every SM, and sinks far from the window."""
    _check_decode(sla2, 4, 1, 64, 128, BF, [40000], [1], None, 0, seed=20)
    _check_decode(sla2, 2, 2, 16, 64, FP, [30011], [2], 1000, 200, seed=21)


def test_cache_attention_of_many_keys_far_below_one(sla2):
    """Weights far below the largest, in fp16 too small for its normal range next to it, are not lost where there are many."""
    d, page, B, g, n = 64, 64, 160, 6, 200000
    rng = np.random.default_rng(35)
    pages = n // page
    book = Book(pages, 1, page, d, 36)
    book.codes[0][...] = 0
    book.codes[0][:, 0, :, 0] = rng.integers(-3, 4, (pages, page))
    book.codes[1][...] = rng.integers(80, 121, (pages, 1, page, d))
    book.scale[0][...], book.scale[1][...] = 1 / 127, 0.01
    for u in range(16):                       # a key for each warp of the block that has the first of them
        book.codes[0][u * 32 // page, 0, u * 32 % page, 0] = 127
        book.codes[1][u * 32 // page, 0, u * 32 % page] = 0
    q = np.zeros((B, g, d))
    q[:, :, 0] = [10, 14, 16, 16.5, 17, 18.5]
    table = torch.arange(pages, dtype=torch.int32).cuda().expand(B, pages).contiguous()
    out = _np(sla2.cache_attention(book.cuda(sla2), _dev(q, FP), table, _dev(np.full(B, n - 1, np.int32)), _dev(_cu([1] * B)), scale=1.0))
    K, V = (book.values(w, np.arange(pages), 0, n) for w in (0, 1))
    P, _ = S.weights(q[0], K, np.ones((g, n), bool), 1.0)
    want = P @ V
    # q's one channel and its codes are exact, so are the logits but for fp32 roundings; a weight is rounded to fp16, next
    # to 2^7 for the largest: a lost one is 2^-32 of that at most
    for h in range(g):
        tol = (2.0 ** -11 + 2.0 ** -19 + 2.0 ** -22 * n / 148) * want[h] + _u(FP) * want[h] + 2.0 ** -32 * n
        _near(out[:, h], np.broadcast_to(want[h], out[:, h].shape), np.broadcast_to(tol, out[:, h].shape), f"head {h}")


def test_cache_attention_values_and_scales(sla2):
    _check_decode(sla2, 4, 2, 16, 64, BF, [100, 50], [1, 2], None, 0, seed=22, spread=300.0)      # close to one-hot
    _check_decode(sla2, 4, 2, 16, 64, BF, [100, 50], [1, 2], None, 0, seed=23, spread=1e-30)      # close to uniform
    _check_decode(sla2, 4, 2, 16, 64, FP, [100, 50], [1, 2], 30, 2, seed=24, scale=2.0)
    _check_decode(sla2, 4, 2, 32, 128, BF, [100, 50, 3], [1, 2, 1], 30, 2, seed=25, extra_rows=5)


def test_cache_attention_queries_with_one_large_channel(sla2):
    """A channel a thousand times the others: they are rounded to steps of its size, as documented, and no worse."""
    d, page, dt, Hkv, g = 128, 64, BF, 2, 4
    rng = np.random.default_rng(43)
    lens, n = [700, 130], [701, 131]
    table = _table(n, page, 16, 44)
    book = Book(16, Hkv, page, d, 45)
    q = rng.standard_normal((2, Hkv * g, d))
    q[:, :, 5] *= 1000
    book.codes[0][:, :, :, 5] = rng.integers(-2, 3, book.codes[0].shape[:3])
    q = S.round_to(q, dt)
    out = _np(sla2.cache_attention(book.cuda(sla2), _dev(q, dt), _dev(table), _dev(np.array(lens, np.int32)), _dev(_cu([1, 1]))))
    for b in range(2):
        for h in range(Hkv * g):
            K, V = (book.values(w, table[b, :-(-n[b] // page)], h // g, n[b]) for w in (0, 1))
            _near_decode(dt, out[b:b + 1, h], q[b:b + 1, h], K, V, np.ones((1, n[b]), bool), d ** -0.5, f"{b} {h}")


def test_cache_attention_scales_far_apart(sla2):
    """Pages whose scales differ by many powers of two, and pages of zeros."""
    d, page, dt, n = 64, 16, BF, 200
    book = Book(14, 1, page, d, 30)
    for w in range(2):
        book.scale[w][:, 0] = np.exp2(np.linspace(-40, 3, 14)).astype(np.float32)
        book.scale[w][[3, 7], 0] = 0
    cache = book.cuda(sla2)
    table = np.arange(13, dtype=np.int32)[None]
    q = S.round_to(np.random.default_rng(31).standard_normal((1, 2, d)), dt)
    out = sla2.cache_attention(cache, _dev(q, dt), _dev(table), _dev(np.array([n - 1], np.int32)), _dev(_cu([1])), scale=1e-3)
    K, V = (book.values(w, table[0], 0, n) for w in (0, 1))
    for h in range(2):
        P, _ = S.weights(q[:, h], K, np.ones((1, n), bool), 1e-3)
        el = _weight_error(q[:, h], K, np.ones((1, n), bool), 1e-3)
        el = el + 2 * 2.0 ** -15.9 * np.abs(q[:, h]).max() * np.abs(K).sum(1).max() * 1e-3      # the row's rounding, as above
        A = P @ np.abs(V)
        want = P @ V
        _near(_np(out)[:, h], want, (2.0 ** -11 + el + 2.0 ** -22 * n) * A + _u(dt) * np.abs(want) + 2.0 ** -25 * n * np.abs(V).max(),
              "far scales")


def test_cache_attention_rows_that_see_nothing_and_bad_pages(sla2):
    d, page, dt = 64, 16, BF
    book = Book(8, 1, page, d, 40)
    cache = book.cuda(sla2)
    q = torch.randn(4, 2, d, generator=torch.Generator().manual_seed(41)).to(dt).cuda()
    cu, lens = _cu([1, 1, 1, 1]), np.array([20, 10, 40, 70], np.int32)
    table = np.array([[0, 1, -1], [-3, 2, 2], [3, 800, 4], [5, 6, 7]], np.int32)      # the last needs five entries
    status = torch.zeros(1, dtype=torch.int32).cuda()
    out = _np(sla2.cache_attention(cache, q, _dev(table), _dev(lens), _dev(cu), status=status))
    assert status.item() == 6
    assert not out[1].any(), "nothing is left to see"
    for b, pages, keys in ((0, [0, 1], range(21)), (2, [3, 4], list(range(16)) + list(range(16, 25))), (3, [5, 6, 7], range(48))):
        K, V = (book.values(w, np.array(pages), 0, 48) for w in (0, 1))
        keys = list(keys)
        for h in range(2):
            P, _ = S.weights(_np(q)[b:b + 1, h], K[keys], np.ones((1, len(keys)), bool), d ** -0.5)
            assert np.abs(out[b, h] - P @ V[keys]).max() < 0.02, b
    # a NaN scale reaches the rows that see the page, and no others
    cache.v_scale[6] = float("nan")
    cache.k_scale[0] = float("nan")
    out = sla2.cache_attention(cache, q, _dev(table), _dev(lens), _dev(cu)).float()
    assert out[[0, 3]].isnan().all() and not out[[1, 2]].isnan().any()
    # offsets that go down or reach behind the rows: those sequences' rows stay
    for bad in ([0, 3, 2, 3, 4], [0, 1, 2, 3, 9]):
        o = torch.full_like(q, 6)
        status.zero_()
        sla2.cache_attention(cache, q, _dev(table), _dev(lens), _dev(np.array(bad, np.int32)), out=o, status=status)
        assert status.item() == 6


@pytest.mark.parametrize("width", [2, 40])   # items of a warp, and of a thread block
@pytest.mark.parametrize("cu,lens,good", [([0, 1, 9, 2, 3], [20, 9, 14, 30], 1), ([0, 1, 2, 3, 4], [20, -1, 14, 30], 3),
                                          ([0, 1, 2, 1, 4], [20, 9, 14, 30], 2), ([-1, 1, 2, 3, 4], [20, 9, 14, 30], 0)])
def test_cache_attention_of_bad_offsets_leaves_rows_behind(sla2, cu, lens, good, width):
    d, page, dt = 64, 16, BF
    book = Book(8, 1, page, d, 39)
    rng = np.random.default_rng(42)
    q = S.round_to(rng.standard_normal((4, 2, d)), dt)
    table = np.full((4, width), -1, np.int32)
    table[:, :2] = np.arange(8).reshape(4, 2)
    o = torch.full((4, 2, d), 6.0, dtype=dt).cuda()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    sla2.cache_attention(book.cuda(sla2), _dev(q, dt), _dev(table), _dev(np.array(lens, np.int32)), _dev(np.array(cu, np.int32)),
                         out=o, status=status)
    assert status.item() == 6
    o, taken = _np(o), _in_order(cu, lens, 4)
    assert len(taken) == good
    for b in range(4):
        if b not in taken:
            assert (o[b] == 6).all()
            continue
        n = lens[b] + 1
        K, V = (book.values(w, table[b, :2], 0, n) for w in (0, 1))
        for h in range(2):
            _near_decode(dt, o[b:b + 1, h], q[b:b + 1, h], K, V, np.ones((1, n), bool), d ** -0.5, f"{b} {h}")


def test_append_and_attention_without_tokens_clear_the_status(sla2):
    cache = sla2.KVCache.empty(2, 1, 16, 64)
    k = torch.zeros(0, 1, 64, dtype=BF).cuda()
    args = (_dev(np.zeros((1, 1), np.int32)), _dev(np.zeros(1, np.int32)), _dev(np.zeros(2, np.int32)))
    for stream in (None, torch.cuda.Stream()):
        status = torch.full((1,), 6, dtype=torch.int32).cuda()
        torch.cuda.synchronize()
        sla2.cache_append(cache, k, k, *args, status=status, stream=stream)
        torch.cuda.synchronize()
        assert status.item() == 0
        status.fill_(6)
        torch.cuda.synchronize()
        sla2.cache_attention(cache, k, *args, status=status, stream=stream)
        torch.cuda.synchronize()
        assert status.item() == 0


def test_cache_attention_page_that_ends_in_garbage(sla2):
    """Codes and pages behind a sequence's last token, whatever they hold, change nothing."""
    d, page, dt = 128, 64, FP
    book = Book(6, 2, page, d, 50)
    cache = book.cuda(sla2)
    q = torch.randn(2, 4, d, generator=torch.Generator().manual_seed(51)).to(dt).cuda()
    args = (_dev(np.array([[0, 1, -1], [2, 3, 4]], np.int32)), _dev(np.array([69, 128], np.int32)), _dev(_cu([1, 1])))
    ref = sla2.cache_attention(cache, q, *args)
    cache.k_codes[1, :, 6:], cache.v_codes[1, :, 6:] = -128, 127
    cache.k_codes[4, :, 1:], cache.v_codes[4, :, 1:] = 127, -128
    cache.k_scale[5], cache.v_scale[5] = float("nan"), float("inf")
    assert torch.equal(ref, sla2.cache_attention(cache, q, *args))


def test_cache_beyond_32_bit_offsets(sla2):
    """Pages whose codes lie more than 2^31 bytes from the cache's base."""
    Hkv, page, d, dt = 8, 128, 128, BF
    pages = (1 << 31) // (Hkv * page * d) + 40
    codes = [torch.empty(pages, Hkv, page, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages, Hkv, device="cuda") for _ in range(2)]
    for c in codes:
        c[-40:].zero_()
    far = sla2.KVCache(*codes, *scales)
    near = sla2.KVCache.empty(40, Hkv, page, d)
    lens, news = np.array([0, 0], np.int32), [1500, 900]
    cu, T = _cu(news), sum(news)
    g = torch.Generator().manual_seed(60)
    k, v, q = (torch.randn(T, H, d, generator=g).to(dt).cuda() for H in (Hkv, Hkv, 16))
    table = _table(news, page, 40, 61)
    outs = []
    for cache, t in ((near, table), (far, np.where(table >= 0, table + pages - 40, table).astype(np.int32))):
        sla2.cache_append(cache, k, v, _dev(t), _dev(lens), _dev(cu))
        last = torch.stack([q[1499], q[2399]])
        outs.append(sla2.cache_attention(cache, last, _dev(t), _dev(np.array(news, np.int32) - 1), _dev(_cu([1, 1]))))
    same = torch.equal(outs[0], outs[1]), torch.equal(near.k_codes, far.k_codes[-40:])
    assert same == (True, True)


def test_generation_as_it_is_used(sla2):
    """A prompt through append and window_forward, then steps of append and cache_attention, one of them
    replayed from a graph: queries, cache and outputs at every step against the oracle."""
    Hq, Hkv, page, d, dt, window, sinks = 4, 2, 16, 64, BF, 40, 3
    rng = np.random.default_rng(70)
    prompt = [37, 90]
    steps = 6
    total = [n + steps + 1 for n in prompt]
    pages = sum(-(-n // page) for n in total)
    table = _table(total, page, pages, 71)
    rope = _rope(max(total), 32)
    dr = tuple(_dev(x) for x in rope)
    book = Book(pages, Hkv, page, d, 72)
    cache = book.cuda(sla2)
    lens = np.zeros(2, np.int32)

    def draw(T):
        return [S.round_to(rng.standard_normal((T, H, d)), dt) for H in (Hq, Hkv, Hkv)]

    q, k, v = draw(sum(prompt))
    cu = _cu(prompt)
    k_out = torch.empty(sum(prompt), Hkv, d, dtype=dt).cuda()
    q_rot = sla2.cache_append(cache, _dev(k, dt), _dev(v, dt), _dev(table), _dev(lens), _dev(cu), rope=dr, q=_dev(q, dt), k_out=k_out)
    wq, wk = book.append(k, v, table, lens, cu, rope, False, dt, q)
    assert np.array_equal(_np(q_rot), wq) and np.array_equal(_np(k_out), wk)
    for b in range(2):
        rows = slice(cu[b], cu[b + 1])
        x = [t[rows].transpose(0, 1)[None] for t in (q_rot, k_out, _dev(v, dt))]
        out = _np(sla2.window_forward(*x, window, sinks))
        for h in range(Hq):
            want, _, P = S.window_head(wq[rows, h], wk[rows, h // 2], v[rows, h // 2], window, sinks, True, d ** -0.5)
            assert np.abs(out[0, h] - want).max() <= 3 * _u(dt) * np.abs(v).max()
    lens = np.array(prompt, np.int32)
    cu = _cu([1, 1])
    held = [torch.zeros(2, H, d, dtype=dt).cuda() for H in (Hq, Hkv, Hkv)]
    dl, dt_, dc = _dev(lens), _dev(table), _dev(cu)

    def one():
        q_rot = sla2.cache_append(cache, held[1], held[2], dt_, dl, dc, rope=dr, q=held[0])
        return sla2.cache_attention(cache, q_rot, dt_, dl, dc, window=window, sinks=sinks)

    graph = None
    for step in range(steps):
        q, k, v = draw(2)
        for h, x in zip(held, (q, k, v)):
            h.copy_(_dev(x, dt))
        dl.copy_(_dev(lens))
        if step < 2:
            out = one()
        else:
            if graph is None:
                keep = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)]
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    out = one()
                assert all(torch.equal(a, b) for a, b in zip(keep, (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)))
            graph.replay()
        torch.cuda.synchronize()
        wq, _ = book.append(k, v, table, lens, cu, rope, False, dt, q)
        _same_cache(cache, book, f"step {step}: ")
        for b in range(2):
            n = int(lens[b]) + 1
            mask = S.visible([n - 1], n, window, sinks, True)
            for h in range(Hq):
                K, V = (book.values(w, table[b, :-(-n // page)], h // 2, n) for w in (0, 1))
                P, _ = S.weights(wq[b:b + 1, h], K, mask, d ** -0.5)
                assert np.abs(_np(out)[b, h] - P @ V).max() <= 3 * _u(dt) * np.abs(V).max()
        lens = lens + 1


def test_cache_attention_same_bits_on_streams_and_shared_workspace(sla2):
    book = Book(60, 2, 64, 128, 80)
    cache = book.cuda(sla2)
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(81)).to(BF).cuda()
    table = _table([1500, 700, 1400], 64, 60, 82)
    args = (_dev(table), _dev(np.array([1499, 699, 1399], np.int32)), _dev(_cu([1, 1, 1])))
    ref = sla2.cache_attention(cache, q, *args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [sla2.cache_attention(cache, q, *args, stream=side), sla2.cache_attention(cache, q, *args)]
    n = sla2.cache_attention_workspace_size(cache, 3, 8, 3, table.shape[1])
    ws = torch.full((n,), 255, dtype=torch.uint8).cuda()
    outs = []
    graphs = []
    for _ in range(2):          # two graphs that share a workspace, replayed one after the other
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(sla2.cache_attention(cache, q, *args, workspace=ws))
        graphs.append(gr)
    for gr in graphs + graphs:
        gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(ref, x) for x in got + outs)
