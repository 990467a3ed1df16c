"""The linear and gated layers and their backward passes on the GPU, every
element against the 64-bit reference of ffn_ref within its derived bound:
types, layouts, activations, ragged and tiny sizes, padded strides, every
tile form and K split the planner takes, in-place residuals, streams, graphs
and offsets past 2^31 elements."""
import numpy as np
import pytest
import torch

import ffn_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ff():
    from hierarchical_gemm_gb300 import tsffn
    return tsffn


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(r, c, dtype, g, pad=0, std=1.0):
    ld = (c + 7) // 8 * 8 + pad
    x = torch.randn((r, ld), generator=g, device="cuda").mul_(std).to(dtype)
    return x[:, :c]


def unset(r, c, dtype, pad=0):
    ld = (c + 7) // 8 * 8 + pad
    return torch.full((r, ld), float("nan"), dtype=dtype, device="cuda")[:, :c]


def weights(K, N, rcr, dtype, g, pad=0):
    w = rows(N, K, dtype, g, pad, K ** -0.5) if rcr else rows(K, N, dtype, g, pad, K ** -0.5)
    return w.t() if rcr else w


def check_linear(ff, M, N, K, rcr=False, dtype=BF, act="none", bias=None, residual=False, out=None, pad=0, train=False,
                 seed=1, in_place=False, dw_dtype=None):
    g = _gen(seed)
    out = out or dtype
    x, w = rows(M, K, dtype, g, pad), weights(K, N, rcr, dtype, g, pad)
    b = None if bias is None else torch.randn(N, generator=g, device="cuda").to(bias)
    r = rows(M, N, out, g, pad) if residual else None
    want = ref.linear(ref.f64(x), ref.f64(w), None if b is None else ref.f64(b), act,
                      None if r is None else ref.f64(r), out)
    C = r if in_place else unset(M, N, out, pad)
    got, saved = ff.linear(x, w, bias=b, act=act, residual=r, C=C, save=True)
    torch.cuda.synchronize()
    assert ff.status() == 0 and got.data_ptr() == C.data_ptr()
    ref.check(C, want["c"], "C")
    if act == "none":
        assert saved is None
    else:
        ref.check(saved[:, :N], want["z"], "saved")
    if not train:
        return
    dc = rows(M, N, dtype, g, pad)
    dx = unset(M, K, dtype, pad)
    db = None if b is None else torch.full((N,), float("nan"), dtype=b.dtype, device="cuda")
    dx2, dw, db2 = ff.linear_backward(dc, x, w, saved, act=act, dX=dx, dbias=db, dw_dtype=dw_dtype)
    torch.cuda.synchronize()
    assert ff.status() == 0
    want = ref.linear_backward(ref.f64(dc), ref.f64(x), ref.f64(w), None if b is None else ref.f64(b), act, dtype,
                               dw_dtype or dtype, FL if db is None else db.dtype)
    ref.check(dx, want["dx"], "dX")
    ref.check(dw, want["dw"], "dW")
    if db is not None:
        ref.check(db, want["db"], "dbias")


def check_gated(ff, M, F, K, rcr=False, dtype=BF, act="silu", pad=0, train=False, seed=1, dw_dtype=None):
    g = _gen(seed)
    x, w = rows(M, K, dtype, g, pad), weights(K, 2 * F, rcr, dtype, g, pad)
    H = unset(M, F, dtype, pad)
    want = ref.gated(ref.f64(x), ref.f64(w), act, dtype)
    got = ff.gated(x, w, act=act, H=H, save=train)
    torch.cuda.synchronize()
    assert ff.status() == 0
    ref.check(H, want["h"], "H")
    if not train:
        return
    saved = got[1]
    ref.check(saved, want["z"], "saved")
    dh = rows(M, F, dtype, g, pad)
    dx = unset(M, K, dtype, pad)
    _, dw = ff.gated_backward(dh, x, w, saved, act=act, dX=dx, dw_dtype=dw_dtype)
    torch.cuda.synchronize()
    assert ff.status() == 0
    want = ref.gated_backward(ref.f64(dh), ref.f64(x), ref.f64(w), act, dtype, dw_dtype or dtype)
    ref.check(dx, want["dx"], "dX")
    ref.check(dw, want["dw"], "dW")


SHAPES = [(1, 64, 64), (1, 1000, 517), (2, 72, 2048), (3, 8, 8), (5, 1, 40), (7, 31, 1), (8, 264, 1024), (9, 520, 136),
          (64, 640, 300), (127, 130, 65), (128, 128, 64), (200, 385, 72), (257, 512, 256), (300, 1041, 96)]


@pytest.mark.parametrize("rcr", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_shapes(ff, M, N, K, rcr):
    check_linear(ff, M, N, K, rcr, act="gelu", bias=BF, residual=True, train=True, seed=M + N + K)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M", [3, 70])
def test_linear_activations(ff, act, dtype, M):
    check_linear(ff, M, 200, 144, act=act, dtype=dtype, bias=FL, residual=True, train=True, seed=3, pad=8)


@pytest.mark.parametrize("dtype,out,bias", [(BF, FL, BF), (HF, FL, FL), (HF, HF, HF), (BF, BF, FL), (BF, FL, None)])
@pytest.mark.parametrize("M,N", [(1, 77), (6, 640), (150, 333)])
def test_linear_types(ff, dtype, out, bias, M, N):
    check_linear(ff, M, N, 192, True, dtype, "silu", bias, True, out, pad=16, seed=4)
    check_linear(ff, M, N, 192, False, dtype, "none", bias, False, out, seed=5)


@pytest.mark.parametrize("M", [1, 4, 16, 40, 130, 300])
@pytest.mark.parametrize("rcr", [False, True])
def test_long_k(ff, M, rcr):
    # few tiles and many K slices: the K split with its reduction
    check_linear(ff, M, 136, 8200, rcr, act="silu", bias=BF, residual=True, seed=6)
    check_gated(ff, M, 136, 8200, rcr, seed=7)


@pytest.mark.parametrize("rcr", [False, True])
@pytest.mark.parametrize("out", [BF, FL])
def test_residual_in_place(ff, rcr, out):
    for M, N, K in [(1, 256, 512), (5, 256, 4096), (200, 264, 128), (256, 256, 8192)]:
        check_linear(ff, M, N, K, rcr, act="none", bias=BF, residual=True, out=out, in_place=True, seed=8)


@pytest.mark.parametrize("rcr", [False, True])
def test_dw_f32(ff, rcr):
    check_linear(ff, 70, 96, 136, rcr, act="gelu", bias=FL, train=True, dw_dtype=FL)
    check_gated(ff, 70, 96, 136, rcr, train=True, dw_dtype=FL)


@pytest.mark.parametrize("rcr", [False, True])
@pytest.mark.parametrize("M,F,K", [(1, 32, 64), (1, 1000, 517), (2, 8, 2048), (3, 8, 8), (8, 264, 1024), (9, 520, 136),
                                   (64, 640, 300), (127, 136, 65), (128, 128, 64), (200, 384, 72), (257, 512, 256),
                                   (300, 1040, 96), (6, 40, 1)])
def test_gated_shapes(ff, M, F, K, rcr):
    check_gated(ff, M, F, K, rcr, train=True, seed=M + F + K)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M", [2, 70])
def test_gated_activations(ff, act, dtype, M):
    check_gated(ff, M, 200, 144, act=act, dtype=dtype, train=True, seed=3, pad=8)


@pytest.mark.parametrize("rcr", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 40, 33), (8, 129, 250), (12, 300, 1000), (16, 16, 4111), (17, 136, 520),
                                   (24, 1031, 77), (31, 260, 2056), (32, 512, 512), (33, 512, 512), (2, 5200, 96),
                                   (10, 9000, 72), (1, 2048, 2048), (20, 1544, 1544)])
def test_few_rows(ff, M, N, K, rcr):
    # 1, 2 and 4 groups of 8 rows, K split over 1 to 8 blocks of a cluster,
    # more strips of columns than SMs, ragged ends of every kind
    check_linear(ff, M, N, K, rcr, act="silu", bias=BF, residual=True, pad=8, seed=M * 31 + N)
    check_gated(ff, M, max(8, N // 8 * 8), K, rcr, pad=8, train=M % 2 == 1, seed=M * 31 + N)


def test_few_rows_ignore_what_lies_outside(ff):
    # NaN in the padding of every row, in W's rows past N and in X's past M:
    # products of them with zeros would be NaN
    g = _gen(22)
    for M, N, K in [(1, 33, 37), (5, 129, 250), (12, 70, 1003), (30, 136, 72)]:
        for rcr in (False, True):
            def guarded(r, c):
                t = torch.full((r + 9, (c + 7) // 8 * 8 + 16), float("nan"), dtype=BF, device="cuda")
                t[:r, :c] = torch.randn((r, c), generator=g, device="cuda").to(BF)
                return t[:r, :c]
            x = guarded(M, K)
            w = guarded(N, K).t() if rcr else guarded(K, N)
            want = ref.linear(ref.f64(x), ref.f64(w), None, "none", None, BF)
            C, _ = ff.linear(x, w, save=True)
            ref.check(C, want["c"], "C")
            F = N // 16 * 8
            wg = guarded(2 * F, K).t() if rcr else guarded(K, 2 * F)
            want = ref.gated(ref.f64(x), ref.f64(wg), "silu", BF)
            ref.check(ff.gated(x, wg), want["h"], "H")


def _sampled(M, n, seed):
    return np.sort(np.random.default_rng(seed).choice(M, n, replace=False))


@pytest.mark.parametrize("rcr", [False, True])
@pytest.mark.parametrize("M,N,K", [(1000, 8176, 8200),  # 256 x 512 pair tiles, part of a round, long K
                                   (2000, 2608, 72),    # 256-wide pair tiles, a round and a bit
                                   (5100, 9712, 200),   # 256 x 512 pair tiles, five rounds
                                   (2300, 2192, 520)])  # 256-wide pair tiles with a ragged edge
def test_large_tiles(ff, M, N, K, rcr):
    # sampled rows against the reference (a row of C depends on its row of X)
    g = _gen(11)
    x, w = rows(M, K, BF, g), weights(K, N, rcr, BF, g)
    b = torch.randn(N, generator=g, device="cuda").to(BF)
    r = rows(M, N, BF, g)
    at = _sampled(M, 40, 1)
    xs, w64 = ref.f64(x)[at], ref.f64(w)
    C, Z = ff.linear(x, w, bias=b, act="gelu_tanh", residual=r, C=unset(M, N, BF), save=True)
    H, GU = ff.gated(x, w, act="silu", H=unset(M, N // 2, BF), save=True)
    torch.cuda.synchronize()
    assert ff.status() == 0
    want = ref.linear(xs, w64, ref.f64(b), "gelu_tanh", ref.f64(r)[at], BF)
    ref.check(C[at], want["c"], "C")
    ref.check(Z[at][:, :N], want["z"], "saved")
    want = ref.gated(xs, w64, "silu", BF)
    ref.check(H[at], want["h"], "H")
    ref.check(GU[at], want["z"], "saved")
    assert bool(torch.isfinite(C.float()).all()) and bool(torch.isfinite(H.float()).all())


@pytest.mark.parametrize("rcr", [False, True])
def test_large_products_of_the_backward_pass(ff, rcr):
    # 256 x 512 tiles for a long contraction (dX) and for the weight
    # gradient's layout (dW), sampled rows against the reference
    g = _gen(12)
    M, N, K = 4100, 8200, 4088
    x, w = rows(M, K, BF, g), weights(K, N, rcr, BF, g)
    dc = rows(M, N, BF, g)
    dx, dw, _ = ff.linear_backward(dc, x, w)
    torch.cuda.synchronize()
    assert ff.status() == 0
    at = _sampled(M, 12, 2)
    d64, w64 = ref.f64(dc[at]), ref.f64(w)
    v, e = ref.product(d64, w64.T)
    ref.check(dx[at], (v, ref.rounded(v, e, BF)), "dX")
    M, N, K = 1030, 9720, 9736
    x, w = rows(M, K, BF, g), weights(K, N, rcr, BF, g)
    dc = rows(M, N, BF, g)
    _, dw, _ = ff.linear_backward(dc, x, w, need=("dW",))
    at = _sampled(K, 12, 3)
    v, e = ref.product(ref.f64(x).T[at], ref.f64(dc))
    ref.check(dw[at], (v, ref.rounded(v, e, BF)), "dW")
    assert bool(torch.isfinite(dw.float()).all()) and ff.status() == 0


@pytest.mark.parametrize("rcr", [False, True])
def test_integers_are_exact(ff, rcr):
    # integer operands whose sums fp32 holds: one rounding, so equal bits
    g = _gen(12)
    for M, N, K in [(1, 128, 256), (7, 144, 1000), (150, 272, 320), (600, 528, 640)]:
        x = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(BF)
        w = torch.randint(-2, 3, (N, K) if rcr else (K, N), generator=g, device="cuda").to(BF)
        w = w.t() if rcr else w
        b = torch.randint(-3, 4, (N,), generator=g, device="cuda").to(BF)
        r = torch.randint(-3, 4, (M, N), generator=g, device="cuda").to(BF)
        dc = torch.randint(-2, 3, (M, N), generator=g, device="cuda").to(BF)
        z = x.double() @ w.double() + b.double()
        C, saved = ff.linear(x, w, bias=b, act="relu", residual=r, save=True)
        assert torch.equal(saved[:, :N].double(), z)
        assert torch.equal(C, (z.clamp(min=0) + r.double()).to(BF))
        dz = dc.double() * (z > 0)
        dx, dw, db = ff.linear_backward(dc, x, w, saved, act="relu", need=("dX", "dW", "dbias"))
        assert torch.equal(dx, (dz @ w.double().t()).to(BF)) and torch.equal(db, dz.sum(0).to(BF))
        assert torch.equal(dw, (x.double().t() @ dz).to(BF))
        F = N // 2
        H, saved = ff.gated(x, w, act="none", save=True)
        z = x.double() @ w.double()
        assert torch.equal(saved.double(), z) and torch.equal(H, (z[:, :F] * z[:, F:]).to(BF))
        assert ff.status() == 0


def test_reproducible(ff):
    g = _gen(13)
    for M, N, K in [(4, 512, 8192), (200, 304, 4096), (1000, 1024, 512)]:
        x, w, dc = rows(M, K, BF, g), weights(K, N, True, BF, g), rows(M, N, BF, g)
        one = None
        for _ in range(4):
            C, saved = ff.linear(x, w, act="gelu", save=True)
            out = (C, saved[:, :N]) + ff.linear_backward(dc, x, w, saved, act="gelu", need=("dX", "dW", "dbias"))
            out += (ff.gated(x, w),)
            out = [t.clone() for t in out]
            assert one is None or all(torch.equal(a, b) for a, b in zip(one, out))
            one = out


def test_extreme_preactivations(ff):
    # values far out: activations saturate without NaN, as their limits do
    for act in ref.ACTS:
        x = torch.full((3, 8), 1.0, dtype=BF, device="cuda")
        w = torch.zeros((8, 64), dtype=BF, device="cuda")
        w[0] = torch.tensor([s * 10.0 ** e for e in range(-16, 16) for s in (1, -1)], device="cuda").to(BF)
        want = ref.linear(ref.f64(x), ref.f64(w), None, act, None, FL)
        C, saved = ff.linear(x, w, act=act, out_dtype=FL, save=True)
        ref.check(C, want["c"], act)
        dc = torch.ones((3, 64), dtype=BF, device="cuda")
        dx, dw, db = ff.linear_backward(dc, x, w, saved, act=act, need=("dX", "dW", "dbias"))
        d = ref.act(ref.f64(x) @ ref.f64(w), act)[1]
        assert bool(torch.isfinite(db.float()).all())
        assert np.allclose(ref.f64(db), 3 * d[0], rtol=2.0 ** -7, atol=1e-5), act


@pytest.mark.parametrize("act", ["gelu", "silu", "gelu_tanh", "sigmoid"])
def test_gradient_against_differences(ff, act):
    # d/dh sum(dC * linear(X, W + h V)) against sum(dW * V): fp32 outputs, W in
    # steps of 1/64 so that W +- V / 64 is exact; central differences leave
    # h^2 / 6 of the third derivative along V, under 2e-3 of the sum's scale here
    g = _gen(14)
    M, N, K = 40, 64, 48
    x = (torch.randint(-16, 17, (M, K), generator=g, device="cuda") / 32).to(BF)
    w = (torch.randint(-16, 17, (K, N), generator=g, device="cuda") / 64).to(BF)
    v = torch.randint(-1, 2, (K, N), generator=g, device="cuda").to(BF)
    dc = torch.randint(-2, 3, (M, N), generator=g, device="cuda").to(BF)
    h = 1 / 64
    up, down = ((ff.linear(x, w + s * h * v, act=act, out_dtype=FL).double() * dc).sum() for s in (1, -1))
    _, saved = ff.linear(x, w, act=act, save=True)
    _, dw, _ = ff.linear_backward(dc, x, w, saved, act=act)
    scale = float((dw.double() * v).abs().sum())
    assert abs(float((up - down) / (2 * h) - (dw.double() * v).sum())) <= 4e-3 * scale
    up, down = ((ff.gated(x, w + s * h * v, act=act).double() * dc[:, :32]).sum() for s in (1, -1))
    _, saved = ff.gated(x, w, act=act, save=True)
    _, dw = ff.gated_backward(dc[:, :32].contiguous(), x, w, saved, act=act)
    scale = float((dw.double() * v).abs().sum())
    # (H comes in bf16: each of M F values is off by 2^-8 of itself at most,
    # and they add up at random: six deviations of that)
    noise = 6 * 2.0 ** -8 * float((ff.gated(x, w, act=act).double() * dc[:, :32]).norm()) / h
    assert abs(float((up - down) / (2 * h) - (dw.double() * v).sum())) <= 4e-3 * scale + noise


def test_streams_and_handles(ff):
    g = _gen(15)
    x, w = rows(300, 2048, BF, g), weights(2048, 256, False, BF, g)
    want = ff.linear(x, w, act="silu")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[] for _ in streams]
    for _ in range(8):
        for s, o in zip(streams, outs):
            o.append(ff.linear(x, w, act="silu", stream=s, C=torch.empty_like(want)))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for o in outs for t in o)
    assert len({ff.handle(s).raw for s in streams}) == 3 and all(ff.status(s) == 0 for s in streams)
    h = ff.Handle()
    assert torch.equal(ff.linear(x, w, act="silu", handle=h), want) and h.status() == 0
    torch.cuda.synchronize()
    h.close()


@pytest.mark.parametrize("M", [1, 20, 200])
def test_chain_without_waiting(ff, M):
    # kernels of a chain start before the one before has ended: every buffer
    # is written, read and written again along it, by them and by torch, and
    # the result has the bits of a chain that waits after every call
    g = _gen(23)
    K, F = 512, 768
    w1, w2 = weights(K, 2 * F, True, BF, g), weights(F, K, M == 20, BF, g)
    x0 = rows(M, K, BF, g)
    results = []
    for wait in (True, False):
        def step_over():
            if wait:
                torch.cuda.synchronize()
        x, h, y = x0.clone(), unset(M, F, BF), unset(M, K, BF)
        wa, out = w1.t().clone().t(), []
        dw = torch.empty_like(wa)
        for i in range(30):
            _, saved = ff.gated(x, wa, H=h, save=True)
            step_over()
            ff.linear(h, w2, residual=x, C=y)
            step_over()
            dx, _ = ff.gated_backward(h, x, wa, saved, dW=dw)
            step_over()
            norm = ff.clip_grad_norm([dw.t()], 0.01)
            step_over()
            ff.linear(y, w2.t(), C=h, residual=h)
            step_over()
            wa.sub_(dw)
            torch.mul(y, 0.5, out=x)
            out.append((norm, dx, y.clone(), h.clone()))
        torch.cuda.synchronize()
        results.append(out)
    for a, b in zip(*results):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert ff.status() == 0


def test_graph_capture(ff):
    # a training step captured with a handle of its own (made while capturing)
    # and replayed on new inputs, beside eager calls
    g = _gen(16)
    M, F, K = 200, 256, 512
    x, w, dh = rows(M, K, BF, g), weights(K, 2 * F, True, BF, g), rows(M, F, BF, g)
    H, dx, dw = unset(M, F, BF), unset(M, K, BF), unset(2 * F, K, BF).t()
    clipped = torch.empty((2 * F, K), dtype=BF, device="cuda")
    norm = torch.empty((), device="cuda")
    graph = torch.cuda.CUDAGraph()
    handles = []

    def step(h):
        _, saved = ff.gated(x, w, H=H, save=True, handle=h)
        ff.gated_backward(dh, x, w, saved, dX=dx, dW=dw, handle=h)
        ff.clip_grad_norm([dw.t()], 0.5, out=[clipped], norm=norm, handle=h)

    step(None)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        handles.append(ff.Handle())
        step(handles[0])
    for seed in (17, 18):
        x.copy_(rows(M, K, BF, _gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (H, dx, dw, clipped, norm)]
        for t in (H, dx, dw, clipped):
            t.fill_(float("nan"))
        step(None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (H, dx, dw, clipped, norm)))
    assert handles[0].status() == 0


def test_refusals_on_the_device(ff):
    from hierarchical_gemm_gb300.tsgemm import TsgemmError
    x, w = torch.zeros((4, 64), dtype=BF, device="cuda"), torch.zeros((64, 32), dtype=BF, device="cuda")
    for args, code in [(dict(X=x.cpu(), W=w, C=torch.empty_like(w[:4])), 1), (dict(X=x[:, 1:], W=w[:63]), 3),
                       (dict(X=x, W=w, C=x[:, 32:]), 1), (dict(X=torch.zeros((4, 63), dtype=BF, device="cuda"), W=w[:63]), 3)]:
        with pytest.raises(TsgemmError) as e:
            ff.linear(**args)
        assert e.value.status == code
    with pytest.raises(TsgemmError) as e:
        ff.gated(x, torch.zeros((64, 24), dtype=BF, device="cuda"))  # F = 12
    assert e.value.status == 3
    assert ff.status() == 0


def test_column_slices_of_one_buffer(ff):
    g = _gen(19)
    buf = rows(50, 192, BF, g)
    x, C, w = buf[:, :64], buf[:, 64:128], weights(64, 64, False, BF, g)
    keep = buf[:, 128:].clone()
    want = ref.linear(ref.f64(x), ref.f64(w), None, "relu", None, BF)
    ff.linear(x, w, act="relu", C=C)
    ref.check(C, want["c"], "C")
    assert torch.equal(buf[:, 128:], keep)


def test_writes_stay_inside(ff):
    # the padding of strided outputs, and the rows past M, keep their bytes
    g = _gen(20)
    for M, N, K in [(1, 33, 64), (5, 70, 261), (130, 77, 96)]:
        for out in (BF, FL):
            x, w, dc = rows(M, K, BF, g), weights(K, N, False, BF, g), rows(M, N, BF, g)
            big = torch.full((M + 3, 128), 7.0, dtype=out, device="cuda")
            C = big[:M, :N]
            _, saved = ff.linear(x, w, act="silu", C=C, save=True)
            bigx = torch.full((M + 3, 320), 7.0, dtype=BF, device="cuda")
            bigw = torch.full((K + 3, 96), 7.0, dtype=out, device="cuda")
            ff.linear_backward(dc, x, w, saved, act="silu", dX=bigx[:M, :K], dW=bigw[:K, :N])
            H = torch.full((M + 3, 128), 7.0, dtype=BF, device="cuda")
            if N >= 64:
                ff.gated(x, w[:, :48], H=H[:M, :24])
            torch.cuda.synchronize()
            assert bool((big[M:] == 7).all()) and bool((big[:, N:] == 7).all())
            assert bool((bigx[M:] == 7).all()) and bool((bigx[:, K:] == 7).all())
            assert bool((bigw[K:] == 7).all()) and bool((bigw[:, N:] == 7).all())
            assert bool((H[M:] == 7).all()) and bool((H[:, 24:] == 7).all())


def test_offsets_past_32_bits(ff):
    # rows 2^20 elements apart, and saved pre-activations of more than 2^31
    # values: the last rows are where a 32-bit offset would have wrapped
    g = _gen(21)
    M, K, N = 2200, 64, 72
    x = torch.zeros((M, 1 << 20), dtype=BF, device="cuda")[:, :K]
    x.copy_(rows(M, K, BF, g))
    C = torch.zeros((M, 1 << 20), dtype=BF, device="cuda")[:, :N]
    w = weights(K, N, False, BF, g)
    for act in ("silu",):
        want = ref.linear(ref.f64(x), ref.f64(w), None, act, None, BF)
        ff.linear(x, w, act=act, C=C)
        ref.check(C, want["c"], "C")
        ff.linear(x[-3:], w, act=act, C=C[-3:])
        ref.check(C, want["c"], "C")
    del x, C
    torch.cuda.empty_cache()
    M, F, K = 70000, 16384, 64
    x, w, dh = rows(M, K, BF, g), weights(K, 2 * F, True, BF, g), rows(M, F, BF, g)
    H, saved = ff.gated(x, w, save=True)
    dx, _ = ff.gated_backward(dh, x, w, saved, need=("dX",))
    at = [0, 1, M // 2, M - 2, M - 1]
    xs, w64 = ref.f64(x[at]), ref.f64(w)
    want = ref.gated(xs, w64, "silu", BF)
    ref.check(H[at], want["h"], "H")
    ref.check(saved[at], want["z"], "saved")
    ref.check(dx[at], ref.gated_backward(ref.f64(dh[at]), xs, w64, "silu", BF, BF)["dx"], "dX")
    assert ff.status() == 0
