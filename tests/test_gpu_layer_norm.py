"""Layer norm, its gradients and its fusion with the row-wise quantizer against
their definitions in 64 bits.

Tolerances, element by element, from f32 arithmetic (e = 2^-23, sums of n
terms off by at most (n + 8) e times the sum of magnitudes):
  mean   (K + 8) e <|x|>
  rstd   relative: half the relative error of var + eps
  y      the errors of x - mean and of rstd carried through, 4 e of the
         terms, and one rounding to the output type
  dx     the two row means' errors carried through
  dw, db (M + 8) e of the sums of magnitudes
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

E, TINY = 2.0 ** -23, 1e-30
f64 = torch.float64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: E}


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_quantized_linear_quant_amd as m
    return m


def _inputs(M, K, xt, wt, seed=0, mean=0.2, weight=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((M, K), generator=g) + mean).to(DTYPES[xt])
    dy = (torch.randn((M, K), generator=g) * 1e-2).to(DTYPES[xt])
    w = (torch.randn(K, generator=g) * 0.3 + 1).to(DTYPES[wt]) if weight else None
    b = (torch.randn(K, generator=g) * 0.3).to(DTYPES[wt]) if bias else None
    return x, dy, w, b


def _cuda(t):
    return None if t is None else t.cuda()


def _reference(x, w, b, eps):
    """y, mean, rstd in f64 and the bounds of their errors (y's without the
    rounding to its type)."""
    x = x.to(f64)
    K = x.shape[1]
    w = torch.ones(K, dtype=f64) if w is None else w.to(f64)
    b = torch.zeros(K, dtype=f64) if b is None else b.to(f64)
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    em = (K + 8) * E * x.abs().mean(1, keepdim=True)
    ed = em + E * (x.abs() + mean.abs())                              # error of x - mean
    ev = (K + 8) * E * var + (2 * d.abs() * ed + ed * ed).mean(1, keepdim=True)
    er = ev / (2 * (var + eps)) + 8 * E                               # relative error of rstd
    h = d * rstd
    eh = rstd * ed * (1 + er) + h.abs() * er + 2 * E * h.abs()
    y = h * w + b
    ey = eh * w.abs() + 4 * E * (h.abs() * w.abs() + b.abs())
    return y, mean[:, 0], rstd[:, 0], ey, em[:, 0], (er * rstd)[:, 0], h, eh


def _near(got, ref, bound, what):
    got = got.cpu().to(f64)
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= bound + TINY)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {i}: got {got[i]}, ref {ref[i]}, "
                             f"bound {bound[i]}")


def _grad_reference(dy, x, mean, rstd, w):
    x, dy, mean, rstd = x.to(f64), dy.to(f64), mean.to(f64)[:, None], rstd.to(f64)[:, None]
    M, K = x.shape
    w = torch.ones(K, dtype=f64) if w is None else w.to(f64)
    h, t = (x - mean) * rstd, dy * w
    eh = 4 * E * (rstd * (x.abs() + mean.abs()))
    c1, c2 = t.mean(1, keepdim=True), (t * h).mean(1, keepdim=True)
    e1 = (K + 8) * E * t.abs().mean(1, keepdim=True)
    e2 = (K + 8) * E * (t * h).abs().mean(1, keepdim=True) + (t.abs() * eh).mean(1, keepdim=True)
    dx = rstd * (t - c1 - h * c2)
    ex = rstd * (e1 + h.abs() * e2 + eh * c2.abs() + eh * e2 + 4 * E * (t.abs() + c1.abs() + (h * c2).abs()))
    dw, db = (dy * h).sum(0), dy.sum(0)
    ew = (M + 8) * E * (dy * h).abs().sum(0) + (dy.abs() * eh).sum(0)
    return dx, dw, db, ex + 2 * E * dx.abs(), ew, (M + 8) * E * dy.abs().sum(0)


def _check(w8, M, K, xt, wt, weight=True, bias=True, mean=0.2, eps=1e-5, seed=0, backward=True):
    what = f"M{M} K{K} {xt}/{wt}"
    print(f"[norm] {what} weight={weight} bias={bias} mean={mean}", flush=True)
    x, dy, w, b = _inputs(M, K, xt, wt, seed, mean, weight, bias)
    y, mu, rs = w8.layer_norm_forward(_cuda(x), _cuda(w), _cuda(b), eps=eps)
    ry, rmu, rrs, ey, em, er, _, _ = _reference(x, w, b, eps)
    _near(mu, rmu, em, what + " mean")
    _near(rs, rrs, er, what + " rstd")
    _near(y, ry, ey + ROUND[x.dtype] * (ry.abs() + ey), what + " y")
    if not backward:
        return
    dx, dw, db = w8.layer_norm_backward(_cuda(dy), _cuda(x), mu, rs, _cuda(w), need_params=True)
    rx, rw, rb, ex, ew, eb = _grad_reference(dy, x, mu.cpu(), rs.cpu(), w)
    _near(dx, rx, ex + ROUND[x.dtype] * (rx.abs() + ex), what + " dx")
    _near(dw, rw, ew, what + " dweight")
    _near(db, rb, eb, what + " dbias")


@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 8), (3, 7), (5, 64), (2, 513), (17, 1001), (9, 1024), (70, 1280), (4, 4096),
                                 (3, 5120), (2, 8200), (2, 12288), (1, 20000)])
def test_sizes_and_types(w8, M, K, xt, wt):
    _check(w8, M, K, xt, wt, seed=M + K)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_without_weight_or_bias(w8, xt, weight, bias):
    _check(w8, 21, 776, xt, xt, weight, bias)
    _check(w8, 21, 777, xt, xt, weight, bias)


@pytest.mark.parametrize("M,K", [(1500, 256), (9001, 72), (2600, 1032), (1030, 4104), (700, 8192),
                                 (5000, 2200), (2500, 4201)])
def test_many_rows(w8, M, K):
    """Several rows a workgroup, forward and backward."""
    _check(w8, M, K, "bf16", "f32", seed=K)


@pytest.mark.parametrize("K", [2500, 4096])
def test_a_mean_far_from_zero(w8, K):
    """mean 300 deviations from zero: <x^2> - mean^2 would keep no digits in
    f32; the variance about the mean stays inside the bound."""
    _check(w8, 6, K, "f32", "f32", mean=300.0)


def test_constant_rows_and_no_eps(w8):
    print("[norm] constant rows", flush=True)
    x = torch.full((4, 264), 3.0)
    x[1] = 0.0
    x[2] = -1e4
    x[3, ::2] = 5.0
    b = torch.linspace(-1, 1, 264)
    y, mu, rs = w8.layer_norm_forward(x.cuda(), None, b.cuda())
    assert torch.equal(y[:3].cpu(), b.expand(3, 264))                # h = 0: the bias alone
    assert torch.equal(mu.cpu(), torch.tensor([3.0, 0.0, -1e4, 4.0]))
    y, mu, rs = w8.layer_norm_forward(x.cuda(), eps=0.0)
    assert torch.isinf(rs[:3]).all() and y[:3].isnan().all()         # 0 * inf, as the formula says
    assert torch.equal(y[3].cpu(), torch.where(torch.arange(264) % 2 == 0, 1.0, -1.0))


def test_nan_and_infinity_stay_in_their_row(w8):
    print("[norm] non-finite", flush=True)
    x, dy, w, b = _inputs(9, 520, "bf16", "bf16", seed=3)
    clean = w8.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
    cx, cw, cb = w8.layer_norm_backward(dy.cuda(), x.cuda(), clean[1], clean[2], w.cuda())
    x2 = x.clone()
    x2[4, 100], x2[7, 3] = float("nan"), float("inf")
    y, mu, rs = w8.layer_norm_forward(x2.cuda(), w.cuda(), b.cuda())
    keep = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(y[keep], clean[0][keep]) and y[[4, 7]].isnan().all()
    dx, dw, db = w8.layer_norm_backward(dy.cuda(), x2.cuda(), mu, rs, w.cuda())
    assert torch.equal(dx[keep], cx[keep]) and dx[[4, 7]].isnan().all()
    assert dw.isnan().all() and torch.equal(db, cb)                  # dy itself is finite
    dy2 = dy.clone()
    dy2[2, 11] = float("inf")
    dx, dw, db = w8.layer_norm_backward(dy2.cuda(), x.cuda(), clean[1], clean[2], w.cuda())
    col = torch.arange(520) != 11
    assert torch.equal(dw.cpu()[col], cw.cpu()[col]) and torch.isinf(db[11]) and torch.equal(db.cpu()[col], cb.cpu()[col])


@pytest.mark.parametrize("M,K", [(0, 64), (0, 1001)])
def test_no_rows(w8, M, K):
    x = torch.empty(0, K, device="cuda")
    y, mu, rs = w8.layer_norm_forward(x)
    assert y.shape == (0, K) and mu.shape == (0,)
    dw, db = torch.full((K,), 5.0, device="cuda"), torch.full((K,), 5.0, device="cuda")
    dx, _, _ = w8.layer_norm_backward(x, x, mu, rs, dweight=dw, dbias=db, need_params=True)
    torch.cuda.synchronize()
    assert dx.shape == (0, K) and not dw.any() and not db.any()
    xq, sx = w8.w8a8_quant_act_rowwise_layer_norm(x)
    assert xq.shape == (0, K + (-K) % 16) and sx.shape == (0,)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("ld", [264, 257, 300])
def test_views_and_in_place(w8, xt, ld):
    """Rows further apart than their width, on and off 16-byte boundaries; y
    over x and dx over dy."""
    print(f"[norm] views {xt} {ld}", flush=True)
    M, K = 37, 256
    x, dy, w, b = _inputs(M, K, xt, "f32", seed=ld)
    want = w8.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
    grads = w8.layer_norm_backward(dy.cuda(), x.cuda(), want[1], want[2], w.cuda())
    bufs = [torch.full((M, ld), 2.0, dtype=DTYPES[xt], device="cuda") for _ in range(2)]
    vx, vdy = (v[:, :K] for v in bufs)
    vx.copy_(x)
    vdy.copy_(dy)
    g = w8.layer_norm_backward(vdy, vx, want[1], want[2], w.cuda(), out=vdy)
    y = w8.layer_norm_forward(vx, w.cuda(), b.cuda(), out=vx)
    for got, ref in zip((y[0], y[1], y[2], g[0]), (*want, grads[0])):
        d = (got.double() - ref.double()).abs()
        assert bool((d <= 2 * ROUND[DTYPES[xt]] * ref.double().abs() + 1e-5).all())
    for got, ref in zip(g[1:], grads[1:]):
        assert torch.allclose(got, ref, rtol=1e-4, atol=1e-4)
    assert all((v[:, K:] == 2).all() for v in bufs)


def test_rows_past_32_bit_offsets(w8):
    print("[norm] long strides", flush=True)
    M, K = 1090, 72
    x, dy, w, b = _inputs(M, K, "bf16", "bf16", seed=4)
    big = torch.empty((M, 1 << 21), dtype=torch.bfloat16, device="cuda")
    vx, vdy, vy, vdx = (big[:, 1024 * i:1024 * i + K] for i in range(4))
    vx.copy_(x)
    vdy.copy_(dy)
    want = w8.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
    got = w8.layer_norm_forward(vx, w.cuda(), b.cuda(), out=vy)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    want = w8.layer_norm_backward(dy.cuda(), x.cuda(), got[1], got[2], w.cuda())
    g = w8.layer_norm_backward(vdy, vx, got[1], got[2], w.cuda(), out=vdx)
    assert all(torch.equal(p, q) for p, q in zip(g, want))
    xq, sx = w8.w8a8_quant_act_rowwise_layer_norm(x.cuda(), w.cuda(), b.cuda())
    vq, vs = w8.w8a8_quant_act_rowwise_layer_norm(vx, w.cuda(), b.cuda())
    assert torch.equal(xq, vq) and torch.equal(sx, vs)


# ----------------------------------------------------------------- to codes
@pytest.mark.parametrize("qt", [0, 1])
@pytest.mark.parametrize("xt,M,K", [("bf16", 1, 16), ("bf16", 5, 1280), ("f32", 7, 1001), ("bf16", 130, 4096), ("f32", 3, 8208),
                                    ("bf16", 3, 17000), ("bf16", 2, 33), ("bf16", 5000, 2208), ("f32", 8300, 50)])
def test_codes(w8, qt, xt, M, K):
    """Scales are absmax / QMAX of the exact norm within its error; each code
    stands for a value within half a step (and y's error) of the exact one;
    columns past K are zero."""
    print(f"[norm] codes qt={qt} {xt} M{M} K{K}", flush=True)
    x, _, w, b = _inputs(M, K, xt, "f32", seed=K)
    mu, rs = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    xq, sx = w8.w8a8_quant_act_rowwise_layer_norm(x.cuda(), w.cuda(), b.cuda(), qtype=qt, mean=mu, rstd=rs)
    y, rmu, rrs, ey, em, er, _, _ = _reference(x, w, b, 1e-5)
    qmax = 127.0 if qt == 0 else 448.0
    _near(mu, rmu, em, "mean")
    _near(rs, rrs, er, "rstd")
    _near(sx, y.abs().amax(1) / qmax, ey.amax(1) / qmax + 4 * E * y.abs().amax(1) / qmax, "scale")
    assert xq.shape == (M, K + (-K) % 16)
    codes = xq.cpu()
    assert not codes[:, K:].to(torch.float32).any()
    s = sx.cpu().to(f64)[:, None]
    q = codes[:, :K].to(torch.float32).to(f64)
    v = y / s
    # half a code's step: 1/2 for int8; for e4m3 2^-4 of the value, at least half the subnormal step 2^-10
    half = 0.5 if qt == 0 else torch.maximum(v.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=f64))
    assert bool(((q - v).abs() <= half + ey / s * 1.1 + 8 * E * v.abs()).all())


@pytest.mark.parametrize("qt", [0, 1])
@pytest.mark.parametrize("xt,K", [("f32", 1024), ("f32", 1001), ("bf16", 4096)])
def test_codes_follow_the_norm(w8, qt, xt, K):
    """An f32 norm quantized by the shared rule on the host gives the same
    codes and scales bit for bit (the fused kernel's y is layer_norm_forward's
    before it is rounded)."""
    x, _, w, b = _inputs(33, K, xt, "f32", seed=5)
    y, _, _ = w8.layer_norm_forward(x.float().cuda(), w.cuda(), b.cuda())
    xq, sx = w8.w8a8_quant_act_rowwise_layer_norm(x.cuda(), w.cuda(), b.cuda(), qtype=qt)
    y = y.cpu().numpy()
    s = np.abs(y).max(1) / np.float32(127.0 if qt == 0 else 448.0)
    same = sx.cpu().numpy() == s
    # x of another type runs other registers' sums: where the statistics' last bits differ, so may the scale
    assert same.all() if xt == "f32" else same.mean() > 0.3
    v = torch.from_numpy(y[same] / s[same][:, None])
    q = torch.round(v) if qt == 0 else v.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    got = xq.cpu()[torch.from_numpy(same)][:, :K].float()
    assert (got == q).all() if xt == "f32" else (got == q).float().mean() > 0.999


def test_codes_of_zero_rows(w8):
    x = torch.full((3, 64), 2.0, dtype=torch.bfloat16).cuda()
    xq, sx = w8.w8a8_quant_act_rowwise_layer_norm(x)                  # h = 0 everywhere
    assert not xq.any() and (sx == 1e-10).all()


def test_codes_into_a_padded_buffer(w8):
    x, _, w, b = _inputs(6, 72, "bf16", "bf16")
    out = torch.full((6, 128), 9, dtype=torch.int8).cuda()
    xq, sx = w8.w8a8_quant_act_rowwise_layer_norm(x.cuda(), w.cuda(), b.cuda(), ldq=128, out=out)
    ref, rs = w8.w8a8_quant_act_rowwise_layer_norm(x.cuda(), w.cuda(), b.cuda())
    assert torch.equal(xq[:, :80], ref) and not xq[:, 72:].any() and torch.equal(sx, rs)


# ----------------------------------------------------------------- the rest
@pytest.mark.parametrize("M,K,xt", [(333, 1001, "f32"), (1030, 2048, "bf16"), (5, 4096, "bf16")])
def test_same_bits_every_time_and_under_graph_capture(w8, M, K, xt):
    print(f"[norm] graph M{M} K{K}", flush=True)
    x, dy, w, b = (_cuda(t) for t in _inputs(M, K, xt, xt))
    y, mu, rs = torch.empty_like(x), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    xq, sx = torch.empty(M, K + (-K) % 16, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    ws = torch.empty(w8.layer_norm_backward_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    outs = (y, mu, rs, dx, dw, db, xq, sx)

    def step():
        w8.layer_norm_forward(x, w, b, out=y, mean=mu, rstd=rs)
        w8.layer_norm_backward(dy, x, mu, rs, w, out=dx, dweight=dw, dbias=db, workspace=ws)
        w8.w8a8_quant_act_rowwise_layer_norm(x, w, b, out=xq, scale=sx)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    want = [v.clone() for v in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for v in outs:
            v.fill_(1)
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(v, q) for v, q in zip(outs, want))
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(v, q) for v, q in zip(outs, want))


@pytest.mark.parametrize("K", [40, 41])
def test_gradients_against_differences(w8, K):
    """dx, dweight and dbias against central differences of sum(y * dy) of the
    definition in f64, step h = 1e-4: its own error is h^2/6 times the third
    derivative, below 1e-6 here."""
    x, dy, w, b = _inputs(5, K, "f32", "f32", seed=2)
    y, mu, rs = w8.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
    got = dict(zip("xwb", w8.layer_norm_backward(dy.cuda(), x.cuda(), mu, rs, w.cuda())))

    def loss(**v):
        v = {**dict(x=x.to(f64), w=w.to(f64), b=b.to(f64)), **v}
        mean = v["x"].mean(1, keepdim=True)
        d = v["x"] - mean
        return float(((d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * v["w"] + v["b"]) * dy.to(f64)).sum())

    rng = np.random.default_rng(1)
    for name, t in (("x", x), ("w", w), ("b", b)):
        for _ in range(25):
            at = tuple(int(rng.integers(n)) for n in t.shape)
            side = []
            for h in (1e-4, -1e-4):
                v = t.to(f64)
                v[at] += h
                side.append(loss(**{name: v}))
            diff = (side[0] - side[1]) / 2e-4
            assert abs(float(got[name][at]) - diff) <= 2e-6, (name, at)


def test_binding_refusals(w8):
    x, dy, w, b = (_cuda(t) for t in _inputs(8, 64, "bf16", "bf16"))
    mu = rs = torch.zeros(8, device="cuda")
    bad = [((x.half(),), {}), ((x[0],), {}), ((x.t(),), {}), ((x, w[:60]), {}), ((x, w.half()), {}), ((x, w, b.float()), {}),
           ((x, w, b[::2]), {}), ((x,), dict(out=torch.empty(8, 63, dtype=torch.bfloat16).cuda())), ((x,), dict(out=x.float())),
           ((x,), dict(mean=mu[:4])), ((x,), dict(rstd=mu.double())), ((x[:1].expand(8, 64),), {})]
    for args, kw in bad:
        with pytest.raises((TypeError, ValueError)):
            w8.layer_norm_forward(*args, **kw)
    with pytest.raises(w8.W8A8Error):
        w8.layer_norm_forward(x, eps=-1.0)
    for args, kw in [((dy[:4], x, mu, rs), {}), ((dy.float(), x, mu, rs), {}), ((dy, x, mu[:4], rs), {}),
                     ((dy, x, mu, rs.double()), {}), ((dy, x, mu, rs, w), dict(dweight=torch.empty(63).cuda())),
                     ((dy, x, mu, rs, w), dict(workspace=torch.empty(1).cuda()))]:
        with pytest.raises((TypeError, ValueError)):
            w8.layer_norm_backward(*args, **kw)
    for kw in (dict(qtype=3), dict(ldq=80, out=torch.empty(8, 64, dtype=torch.int8).cuda()), dict(scale=mu[:3])):
        with pytest.raises((TypeError, ValueError)):
            w8.w8a8_quant_act_rowwise_layer_norm(x, w, b, **kw)


# ------------------------------------------------- non-finite rows to codes
CODE_K = [40, 520, 1001, 4096, 4100, 16384, 17000]     # one wave, several, both sides of the streamed rows


@pytest.mark.parametrize("qt", [0, 1])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("K", CODE_K)
def test_codes_keep_nan_and_infinity(w8, qt, xt, K):
    """A NaN or an infinity in x makes the whole norm of its row NaN: the
    absmax and so the scale are NaN, and so are e4m3's codes (int8 has none:
    0).  The other rows' bits do not change, columns past K stay zero, and a
    product with such a row is NaN, not the bias."""
    print(f"[norm] non-finite codes qt={qt} {xt} K{K}", flush=True)
    M = 9
    x, _, w, b = _inputs(M, K, xt, "f32", seed=K)
    cq, cs = w8.w8a8_quant_act_rowwise_layer_norm(x.cuda(), w.cuda(), b.cuda(), qtype=qt)
    x[4, K - 1], x[6, K // 2], x[7, 3] = float("nan"), float("-inf"), float("inf")
    xq, sx = w8.w8a8_quant_act_rowwise_layer_norm(x.cuda(), w.cuda(), b.cuda(), qtype=qt)
    keep, gone = [0, 1, 2, 3, 5, 8], [4, 6, 7]
    assert torch.equal(xq[keep].view(torch.uint8), cq[keep].view(torch.uint8)) and torch.equal(sx[keep], cs[keep])
    assert sx[gone].isnan().all()
    codes = xq.float()
    assert not codes[:, K:].any()
    if qt == 1:
        assert codes[gone, :K].isnan().all()
    else:
        assert not codes[gone].any()
    wq = (torch.arange(16 * xq.shape[1], device="cuda").reshape(16, -1) % 3).to(torch.int8)
    wq = wq if qt == 0 else wq.float().to(torch.float8_e4m3fn)
    one = torch.ones(1, device="cuda")
    y = w8.w8a8_linear(xq, sx, wq, one, torch.zeros(16, dtype=torch.bfloat16, device="cuda"))
    assert y[gone].isnan().all() and y[keep].isfinite().all()


@pytest.mark.parametrize("qt", [0, 1])
@pytest.mark.parametrize("K", [1001, 4096, 17000])
def test_codes_of_an_infinite_or_nan_column(w8, qt, K):
    """An infinite bias makes one column of y infinite: the scale is infinite,
    a finite value over it is a zero of its sign, inf / inf is NaN (int8: 0).
    A NaN in the weight makes every row's scale NaN."""
    x, _, w, b = _inputs(5, K, "bf16", "f32", seed=K)
    b[7] = float("-inf")
    y, _, _ = w8.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
    xq, sx = w8.w8a8_quant_act_rowwise_layer_norm(x.cuda(), w.cuda(), b.cuda(), qtype=qt)
    assert torch.isposinf(sx).all()
    codes, col = xq.float()[:, :K], torch.arange(K) != 7
    assert not codes[:, col].any() and not xq.float()[:, K:].any()
    if qt == 1:
        assert codes[:, 7].isnan().all()
        assert torch.equal(torch.signbit(codes[:, col]), torch.signbit(y[:, col]))
    else:
        assert not codes[:, 7].any()
    b[7], w[9] = 0.0, float("nan")
    xq, sx = w8.w8a8_quant_act_rowwise_layer_norm(x.cuda(), w.cuda(), b.cuda(), qtype=qt)
    assert sx.isnan().all() and (qt == 0 or xq.float()[:, :K].isnan().all()) and not xq.float()[:, K:].any()


@pytest.mark.parametrize("K", [100, 101, 600])
def test_backward_of_constant_rows_of_huge_values(w8, K):
    """x - mean is 0 in every column that there is, so h is 0 and dx is
    rstd (t - <t>), however large the mean; columns past K count for nothing."""
    x, dy, w, _ = _inputs(4, K, "f32", "f32", seed=K)
    x[1] = 2.0 ** (127 - int(np.ceil(np.log2(K))))               # the row's sum is finite, mean / sqrt(eps) is not
    x[2] = -x[1]
    y, mu, rs = w8.layer_norm_forward(x.cuda(), w.cuda(), eps=1e-7)
    assert torch.equal(mu[1:3].cpu(), x[1:3, 0]) and not y[1:3].any()
    for params in (True, False):
        dx, dw, db = w8.layer_norm_backward(dy.cuda(), x.cuda(), mu, rs, w.cuda(), need_params=params)
        rx, rw, rb, ex, ew, eb = _grad_reference(dy, x, mu.cpu(), rs.cpu(), w)
        t = (dy * w).to(f64)
        rx[1:3] = (rs.cpu().to(f64)[:, None] * (t - t.mean(1, keepdim=True)))[1:3]
        ex[1:3] = (rs.cpu().to(f64)[:, None] * (K + 8) * E * (t.abs() + t.abs().mean(1, keepdim=True)))[1:3]
        _near(dx, rx, ex, "dx")


def test_dx_alone_of_very_many_rows(w8):
    """2^26 rows and a few: more than one launch may have threads for with a
    row each."""
    M, K = 2 ** 26 + 3, 8
    print(f"[norm] dx alone M{M}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)
    y, mu, rs = w8.layer_norm_forward(x)
    dx, _, _ = w8.layer_norm_backward(dy, x, mu, rs)
    for first in (0, 2 ** 22 - 50, 2 ** 24 - 50, 2 ** 25 + 7, M - 100):
        rows = slice(first, first + 100)
        rx, _, _, ex, _, _ = _grad_reference(dy[rows].cpu(), x[rows].cpu(), mu[rows].cpu(), rs[rows].cpu(), None)
        _near(dx[rows], rx, ex + ROUND[torch.bfloat16] * (rx.abs() + ex), f"rows from {first}")
        ry, rmu, rrs, ey, em, er, _, _ = _reference(x[rows].cpu(), None, None, 1e-5)
        _near(y[rows], ry, ey + ROUND[torch.bfloat16] * (ry.abs() + ey), f"y from {first}")
    again = torch.empty_like(dx)
    for i in range(0, M, 2 ** 24):                                 # the same rows in smaller calls: the same bits
        rows = slice(i, min(i + 2 ** 24, M))
        w8.layer_norm_backward(dy[rows], x[rows], mu[rows], rs[rows], out=again[rows])
    assert torch.equal(again, dx)


# ---------------------------------------------------------- the other variants
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2000, 2001, 14000, 16001, 16384])
def test_the_widest_resident_rows(w8, K, xt):
    _check(w8, 5, K, xt, "f32", seed=K)


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(3, 3), (70, 504), (9, 501), (70, 1000), (9, 1001), (70, 2040), (9, 2041), (70, 4088),
                                 (9, 4089), (30, 8184), (9, 8185), (9, 16377), (3, 17001)])
def test_dx_alone(w8, M, K, xt, weight):
    """The input gradient without the parameters' (the default without a
    weight), in each of its layouts, even widths and odd."""
    print(f"[norm] dx alone M{M} K{K} {xt} weight={weight}", flush=True)
    x, dy, w, _ = _inputs(M, K, xt, "f32", seed=M + K, weight=weight)
    _, mu, rs = w8.layer_norm_forward(x.cuda())
    dx, dw, db = w8.layer_norm_backward(dy.cuda(), x.cuda(), mu, rs, _cuda(w), need_params=False)
    assert dw is None and db is None
    rx, _, _, ex, _, _ = _grad_reference(dy, x, mu.cpu(), rs.cpu(), w)
    _near(dx, rx, ex + ROUND[x.dtype] * (rx.abs() + ex), "dx")
    if not weight:
        assert torch.equal(w8.layer_norm_backward(dy.cuda(), x.cuda(), mu, rs)[0], dx)
    over = dy.cuda()
    assert torch.equal(w8.layer_norm_backward(over, x.cuda(), mu, rs, _cuda(w), out=over, need_params=False)[0], dx)


@pytest.mark.parametrize("M,K,xt", [(70, 504, "bf16"), (1030, 2201, "f32"), (300, 8185, "bf16"), (70, 9001, "bf16")])
def test_parameters_alone_and_one_of_them(w8, M, K, xt):
    """dweight and dbias without dx, and through the C entry each by itself,
    are the bits of the whole call."""
    x, dy, w, b = (_cuda(t) for t in _inputs(M, K, xt, "f32", seed=K))
    _, mu, rs = w8.layer_norm_forward(x, w, b)
    _, dw, db = w8.layer_norm_backward(dy, x, mu, rs, w)
    none, aw, ab = w8.layer_norm_backward(dy, x, mu, rs, w, need_dx=False)
    assert none is None and torch.equal(aw, dw) and torch.equal(ab, db)
    ws = torch.empty(w8.layer_norm_backward_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for first in (True, False):
        got = torch.full((K,), 3.0, device="cuda")
        st = w8.library().layer_norm_backward(
            0 if xt == "bf16" else 1, dy.data_ptr(), K, x.data_ptr(), K, mu.data_ptr(), rs.data_ptr(), M, K, 1, w.data_ptr(),
            None, 0, got.data_ptr() if first else None, None if first else got.data_ptr(), ws.data_ptr(), stream)
        assert st == 0 and torch.equal(got, dw if first else db)


def test_binding_refuses_what_is_no_tensor(w8):
    x, dy, w, b = (_cuda(t) for t in _inputs(8, 64, "bf16", "bf16"))
    mu = torch.zeros(8, device="cuda")
    for args in ((x, [1.0]), (x, w, [1.0]), (x, None, 3.0), ([1.0],), (None,)):
        for f in (w8.layer_norm_forward, w8.w8a8_quant_act_rowwise_layer_norm):
            with pytest.raises(TypeError):
                f(*args)
    for args in ((dy, x, mu, mu, 3.0), (None, x, mu, mu), (dy, x, 1.0, mu)):
        with pytest.raises(TypeError):
            w8.layer_norm_backward(*args)
