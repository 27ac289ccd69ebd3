"""Low-rank adapters of many requests against their definition in 64 bits.

Tolerances come from the arithmetic, element by element:
  u, g   sums of K exact bf16 products in f32: (K + 8) 2^-23 sum |x||a| s
  out    the f32 sum over j, u taken as two bf16 halves (2^-16 of each term),
         and one rounding to bf16 (2^-8 of the result)
  da, db sums over rows in f32, their f32 factor kept to 24 bits:
         (rows + 16) 2^-23 sum |g||x|, and g's own error
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U23, TINY = 2.0 ** -23, 1e-30
f64 = torch.float64


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w8a8_quantized_linear_quant_amd as m
    return m


class Batch:
    """Requests, a pool and their tensors on the host (bf16 values)."""

    def __init__(self, lengths, adapters, K, N, R, L, ranks=None, scale=True, seed=0, garbage=False):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.adapters, self.L, self.K, self.N, self.R = lengths, adapters, L, K, N, R
        self.M = M = sum(lengths)
        rnd = lambda shape, std: (torch.randn(shape, generator=g) * std).bfloat16()  # noqa: E731
        self.x, self.dy = rnd((M, K), 1.0), rnd((M, N), 0.01)
        self.base, self.dbase = rnd((M, N), 1.0), rnd((M, K), 0.01)
        self.a, self.b = rnd((L, R, K), K ** -0.5), rnd((L, N, R), 0.1)
        self.scale = torch.rand(L, generator=g) + 0.5 if scale else None
        self.ranks = ranks
        if garbage:                       # beyond a rank the pool may hold anything
            for l in range(L):
                self.a[l, ranks[l]:] = float("nan")
                self.b[l, :, ranks[l]:] = float("inf")

    def spans(self):
        row = 0
        for n, l in zip(self.lengths, self.adapters):
            if n and l >= 0:
                r = self.R if self.ranks is None else min(max(self.ranks[l], 0), self.R)
                yield slice(row, row + n), l, r, 1.0 if self.scale is None else float(self.scale[l])
            row += n

    def forward(self):
        """(out, u) in f64 and the bounds of their errors."""
        x, a, b = self.x.to(f64), self.a.to(f64), self.b.to(f64)
        u, eu = torch.zeros(self.M, self.R, dtype=f64), torch.zeros(self.M, self.R, dtype=f64)
        out, eo = self.base.to(f64).clone(), torch.zeros(self.M, self.N, dtype=f64)
        for rows, l, r, s in self.spans():
            u[rows, :r] = s * (x[rows] @ a[l, :r].T)
            eu[rows, :r] = (self.K + 8) * U23 * s * (x[rows].abs() @ a[l, :r].abs().T)
            d = u[rows, :r].abs() * (2.0 ** -16 + (2 * r + 8) * U23) + eu[rows, :r]
            out[rows] += u[rows, :r] @ b[l, :, :r].T
            eo[rows] = d @ b[l, :, :r].abs().T
        return out, u, eo + 2.0 ** -8 * out.abs() + 4 * U23 * self.base.to(f64).abs(), eu

    def backward(self, u):
        x, dy, a, b, u = (t.to(f64) for t in (self.x, self.dy, self.a, self.b, u))
        dx, ex = self.dbase.to(f64).clone(), torch.zeros(self.M, self.K, dtype=f64)
        da, ea = torch.zeros(self.L, self.R, self.K, dtype=f64), torch.zeros(self.L, self.R, self.K, dtype=f64)
        db, eb = torch.zeros(self.L, self.N, self.R, dtype=f64), torch.zeros(self.L, self.N, self.R, dtype=f64)
        rows_of = {l: sum(n for n, q in zip(self.lengths, self.adapters) if q == l) for l in range(self.L)}
        for rows, l, r, s in self.spans():
            g = s * (dy[rows] @ b[l, :, :r])
            eg = (self.N + 8) * U23 * s * (dy[rows].abs() @ b[l, :, :r].abs())
            dx[rows] += g @ a[l, :r]
            ex[rows] = (g.abs() * (2.0 ** -16 + (2 * r + 8) * U23) + eg) @ a[l, :r].abs()
            da[l, :r] += g.T @ x[rows]
            db[l, :, :r] += dy[rows].T @ u[rows, :r]
            e = (rows_of[l] + 16) * U23
            ea[l, :r] += (e * g.abs() + eg).T @ x[rows].abs()
            eb[l, :, :r] += e * (dy[rows].abs().T @ u[rows, :r].abs())
        return dx, da, db, ex + 2.0 ** -8 * dx.abs() + 4 * U23 * self.dbase.to(f64).abs(), ea, eb

    def dev(self, w8):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        ranks = None if self.ranks is None else torch.tensor(self.ranks, dtype=torch.int32).cuda()
        plan = w8.lora_plan(self.lengths, self.adapters, self.L)
        return dict(a=c(self.a), b=c(self.b), plan=plan, scale=c(self.scale), ranks=ranks)


def _near(got, ref, bound, what):
    got = got.cpu().to(f64)
    bad = ~((got - ref).abs() <= bound + TINY)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {i}: got {got[i]}, ref {ref[i]}, "
                             f"bound {bound[i]}")


def _check(w8, t, what):
    print(f"[lora] {what}", flush=True)
    d = t.dev(w8)
    out, u = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **d)
    ref, refu, eo, eu = t.forward()
    _near(u, refu, eu, what + " u")
    _near(out, ref, eo, what + " out")
    dx, da, db = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, base=t.dbase.cuda(), **d)
    rx, ra, rb, ex, ea, eb = t.backward(u.cpu())
    _near(dx, rx, ex, what + " dx")
    _near(da, ra, ea, what + " da")
    _near(db, rb, eb, what + " db")


CASES = [
    # lengths, adapters, K, N, R, L
    ([1], [0], 8, 8, 8, 1),
    ([1], [0], 1024, 1024, 16, 2),
    ([1] * 17, list(range(7)) * 2 + [-1, 0, 0], 264, 136, 16, 7),
    ([63, 64, 65, 1, 0, 130], [0, 1, 0, -1, 2, 1], 136, 520, 24, 4),
    ([64], [0], 256, 128, 32, 1),
    ([129, 31], [1, 0], 1032, 72, 64, 2),
    ([15, 17, 16], [2, 1, 2], 512, 2056, 128, 3),
    ([700], [0], 1288, 1304, 8, 1),
    ([300, 333], [1, 1], 2048, 640, 40, 2),
    ([90], [0], 640, 256, 72, 1),
    ([33], [-1], 64, 64, 16, 2),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"M{sum(c[0])}-K{c[2]}-N{c[3]}-R{c[4]}-L{c[5]}")
def test_against_the_definition(w8, case):
    lengths, adapters, K, N, R, L = case
    _check(w8, Batch(lengths, adapters, K, N, R, L, seed=len(lengths) + K), str(case[2:]))


@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
def test_many_rows(w8, R):
    """Enough rows for 32 of them a workgroup, two launches at every rank and
    an adapter's rows split over workgroups."""
    _check(w8, Batch([5003, 1, 3400], [1, 0, 1], 136, 200, R, 2, seed=R), f"many rows R{R}")


@pytest.mark.parametrize("M,R", [(200, 64), (1000, 128), (3000, 32), (3000, 64), (3000, 128)])
def test_middling_rows(w8, M, R):
    """Ranks in parts, fewer and none, at 16 rows a workgroup."""
    _check(w8, Batch([M - 7, 7], [1, 0], 264, 520, R, 2, seed=M + R), f"{M} rows R{R}")


def test_one_adapter_of_many_holds_the_rows(w8):
    """A pool so large that no adapter's rows are split: one workgroup passes
    over more than 64 tiles, and the idle adapters' gradients are zero."""
    t = Batch([64 * 70 + 5, 3], [77, 2], 128, 72, 16, 128, seed=1)
    _check(w8, t, "128 adapters")


@pytest.mark.parametrize("R,ranks", [(16, [16, 1, 0, 9]), (64, [64, 33, 8, 0]), (128, [100, 65, 64, 7]), (24, [99, -3, 17, 24])])
def test_ranks_and_what_lies_beyond_them(w8, R, ranks):
    """Entries beyond an adapter's rank hold NaN and infinities; ranks outside
    [0, R] are clamped; a rank of 0 adds nothing."""
    t = Batch([40, 70, 3, 66], [0, 1, 2, 3], 200, 328, R, 4, ranks=ranks, seed=R)
    clamped = [min(max(r, 0), R) for r in ranks]
    for l in range(4):
        t.a[l, clamped[l]:] = float("nan")
        t.b[l, :, clamped[l]:] = float("inf")
    _check(w8, t, f"ranks {ranks}")


def test_no_scale_no_base_no_u(w8):
    print("[lora] defaults", flush=True)
    t = Batch([50, 20], [0, -1], 96, 160, 16, 1, scale=False)
    t.base.zero_()
    d = t.dev(w8)
    out, u = w8.lora_forward(t.x.cuda(), d["a"], d["b"], d["plan"], save_u=False)
    assert u is None
    ref, refu, eo, _ = t.forward()
    _near(out, ref, eo, "out")
    assert not out[50:].any()                                     # no adapter, no base: zero
    dx, da, db = w8.lora_backward(t.dy.cuda(), t.x.cuda(), None, d["a"], d["b"], d["plan"], need_weights=False)
    assert da is None and db is None
    t.dbase.zero_()
    rx, ra, rb, ex, ea, eb = t.backward(refu)
    _near(dx, rx, ex, "dx")
    _, u = w8.lora_forward(t.x.cuda(), d["a"], d["b"], d["plan"])
    dx, da, db = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, d["a"], d["b"], d["plan"], need_dx=False)
    assert dx is None
    rx, ra, rb, ex, ea, eb = t.backward(u.cpu())
    _near(da, ra, ea, "da")
    _near(db, rb, eb, "db")


def test_no_rows(w8):
    """Empty batches: outputs without rows, gradients of zero."""
    print("[lora] no rows", flush=True)
    for lengths, adapters in (([], []), ([0, 0], [0, 1])):
        t = Batch(lengths, adapters, 64, 72, 16, 2)
        d = t.dev(w8)
        out, u = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **d)
        assert out.shape == (0, 72) and u.shape == (0, 16)
        da, db = torch.full((2, 16, 64), 7.0).cuda(), torch.full((2, 72, 16), 7.0).cuda()
        dx, _, _ = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, da=da, db=db, **d)
        assert dx.shape == (0, 64) and not da.any() and not db.any()


def test_views_and_in_place(w8):
    """x, base, out, dy and dx as column slices of wider buffers (the query
    part of a fused projection); out and dx written in place over their base."""
    print("[lora] views", flush=True)
    t = Batch([70, 5, 64], [0, 1, 0], 264, 136, 32, 2, seed=9)
    d = t.dev(w8)

    def wide(v, before, after):
        buf = torch.full((v.shape[0], before + v.shape[1] + after), 3.0, dtype=torch.bfloat16).cuda()
        buf[:, before:before + v.shape[1]] = v.cuda()
        return buf, buf[:, before:before + v.shape[1]]

    (_, x), (ob, o), (_, dy), (xb, dx) = wide(t.x, 8, 16), wide(t.base, 24, 8), wide(t.dy, 8, 8), wide(t.dbase, 16, 0)
    want, wu = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **d)
    out, u = w8.lora_forward(x, base=o, out=o, **d)
    assert out.data_ptr() == o.data_ptr() and torch.equal(out, want) and torch.equal(u, wu)
    assert (ob[:, :24] == 3).all() and (ob[:, 160:] == 3).all()
    w = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, base=t.dbase.cuda(), **d)
    g = w8.lora_backward(dy, x, u, base=dx, out=dx, **d)
    assert all(torch.equal(p, q) for p, q in zip(w, g))
    assert (xb[:, :16] == 3).all()


def test_rows_past_32_bit_offsets(w8):
    """Row offsets beyond 2^32 bytes: a narrow slice of rows 4 MB apart."""
    print("[lora] long strides", flush=True)
    t = Batch([1030, 60], [0, 1], 72, 64, 16, 2, seed=4)
    big = torch.empty((1090, 1 << 21), dtype=torch.bfloat16, device="cuda")
    x, o, dy, dx = (big[:, 1024 * i:1024 * i + w] for i, w in enumerate((72, 64, 64, 72)))
    for v, s in ((x, t.x), (o, t.base), (dy, t.dy), (dx, t.dbase)):
        v.copy_(s)
    d = t.dev(w8)
    out, u = w8.lora_forward(x, base=o, out=o, **d)
    ref, refu, eo, eu = t.forward()
    _near(u, refu, eu, "u")
    _near(out, ref, eo, "out")
    got = w8.lora_backward(dy, x, u, base=dx, out=dx, **d)
    r = t.backward(u.cpu())
    for i, n in enumerate(("dx", "da", "db")):
        _near(got[i], r[i], r[3 + i], n)


def test_infinities_and_nan_stay_in_their_request(w8):
    print("[lora] non-finite", flush=True)
    t = Batch([10, 80, 30], [0, 1, 2], 128, 136, 16, 3, seed=5)
    clean = Batch([10, 80, 30], [0, 1, 2], 128, 136, 16, 3, seed=5)
    t.x[12, 5] = float("nan")               # a row of request 1
    t.x[20, 7] = float("inf")
    t.dy[15, 3] = float("nan")
    d = t.dev(w8)
    out, u = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **d)
    cout, cu = w8.lora_forward(clean.x.cuda(), base=clean.base.cuda(), **d)
    keep = torch.ones(120, dtype=torch.bool)
    keep[[12, 20]] = False
    assert torch.equal(out.cpu()[keep], cout.cpu()[keep]) and torch.equal(u.cpu()[keep], cu.cpu()[keep])
    assert out[12].isnan().all() and torch.isinf(u[20]).all()
    assert not out[20].isfinite().any()
    dx, da, db = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, base=t.dbase.cuda(), **d)
    cx, ca, cb = w8.lora_backward(clean.dy.cuda(), clean.x.cuda(), cu, base=clean.dbase.cuda(), **d)
    keep = torch.ones(120, dtype=torch.bool)
    keep[15] = False
    assert torch.equal(dx.cpu()[keep], cx.cpu()[keep]) and dx[15].isnan().all()
    for l in (0, 2):
        assert torch.equal(da[l], ca[l]) and torch.equal(db[l], cb[l])
    assert da[1].isnan().all() and db[1].isnan().all()


def test_an_infinite_u_gives_infinities(w8):
    """One row whose u is infinite: its output is the signed infinity of b,
    not NaN (the two halves of u must not make inf - inf)."""
    t = Batch([3], [0], 64, 64, 8, 1, seed=6)
    t.a[0, 1:] = 0
    t.a[0, 0] = 1.0
    t.x.zero_()
    t.x[1, 0] = float("inf")
    t.b[0, :, 0] = torch.where(torch.arange(64) % 2 == 0, 2.0, -2.0).bfloat16()
    t.b[0, :, 1:] = 0
    t.a[0, 1:, 0] = 0
    d = t.dev(w8)
    d["ranks"] = torch.tensor([1], dtype=torch.int32).cuda()
    out, u = w8.lora_forward(t.x.cuda(), **d)
    assert torch.isposinf(u[1, 0])
    assert torch.isposinf(out[1, ::2]).all() and torch.isneginf(out[1, 1::2]).all()
    assert not out[0].any() and not out[2].any()


def test_same_bits_every_time_and_under_graph_capture(w8):
    print("[lora] graph", flush=True)
    t = Batch([130, 1, 64, 200], [1, 0, 2, 1], 512, 768, 32, 3, seed=7)
    d = t.dev(w8)
    x, dy, base, dbase = t.x.cuda(), t.dy.cuda(), t.base.cuda(), t.dbase.cuda()
    out, u = torch.empty_like(base), torch.empty(t.M, 32, device="cuda")
    dx, da, db = torch.empty_like(dbase), torch.empty(3, 32, 512, device="cuda"), torch.empty(3, 768, 32, device="cuda")
    fw = torch.empty(w8.lora_forward_workspace_bytes(t.M, 32), dtype=torch.uint8, device="cuda")
    bw = torch.empty(w8.lora_backward_workspace_bytes(t.M, d["plan"].tiles, 512, 768, 32, 3), dtype=torch.uint8,
                     device="cuda")

    def step():
        w8.lora_forward(x, base=base, out=out, u=u, workspace=fw, **d)
        w8.lora_backward(dy, x, u, base=dbase, out=dx, da=da, db=db, workspace=bw, **d)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    want = [v.clone() for v in (out, u, dx, da, db)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for v in (out, u, dx, da, db):
            v.fill_(1.0)
        fw.fill_(255)
        bw.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(v, w) for v, w in zip((out, u, dx, da, db), want))
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(v, w) for v, w in zip((out, u, dx, da, db), want))


def test_gradients_against_differences(w8):
    """The gradients against central differences of sum(out * dy) in f64 on
    the definition (which is linear in each argument: exact differences)."""
    print("[lora] differences", flush=True)
    t = Batch([5, 9], [1, 0], 24, 16, 8, 2, seed=8)
    d = t.dev(w8)
    _, u = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **d)
    dx, da, db = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, base=torch.zeros_like(t.dbase).cuda(), **d)
    t.dbase.zero_()
    _, _, _, ex, ea, eb = t.backward(u.cpu())

    def loss(name, at, step):
        v = {n: getattr(t, n).to(f64) for n in ("x", "a", "b")}
        v[name][at] += step
        s = 0.0
        for rows, l, r, sc in t.spans():
            s += float((sc * (v["x"][rows] @ v["a"][l].T) @ v["b"][l].T * t.dy[rows].to(f64)).sum())
        return s

    rng = np.random.default_rng(0)
    for name, got, e in (("x", dx, ex), ("a", da, ea), ("b", db, eb)):
        got = got.cpu().to(f64)
        for _ in range(40):
            at = tuple(int(rng.integers(n)) for n in got.shape)
            diff = (loss(name, at, 0.5) - loss(name, at, -0.5))
            assert abs(float(got[at]) - diff) <= float(e[at]) + (t.K + 8) * U23 * abs(diff) + 1e-7, (name, at)


def test_binding_refusals(w8):
    print("[lora] refusals", flush=True)
    t = Batch([10, 6], [0, 1], 64, 72, 16, 2)
    d = t.dev(w8)
    x, base, u = t.x.cuda(), t.base.cuda(), torch.zeros(16, 16, device="cuda")
    bad = [dict(x=x[:-1]), dict(x=x.float()), dict(x=x[:, :56]), dict(a=d["a"][:1]), dict(a=d["a"].float()),
           dict(b=d["b"].transpose(0, 1)), dict(base=base[:, :-8]), dict(base=base.t().contiguous().t()),
           dict(scale=d["scale"][:1]), dict(scale=d["scale"].double()), dict(ranks=torch.zeros(2).cuda()),
           dict(out=torch.empty_like(base)[:, :64]), dict(u=u.half()), dict(u=u[:8]), dict(plan=None),
           dict(plan=w8.lora_plan([15], [0], 2)), dict(plan=w8.lora_plan([16], [0], 3)),
           dict(plan=w8.lora_plan([16], [0], 2, device="cpu")), dict(workspace=torch.empty(1, device="cuda"))]
    for b in bad:
        kw = dict(dict(x=x, base=base, **d), **b)
        with pytest.raises((TypeError, ValueError)):
            w8.lora_forward(**kw)
    buf = torch.zeros(16, 68, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        w8.lora_forward(buf[:, :64], base=base, **d)               # row stride not a multiple of 8
    with pytest.raises(ValueError):
        w8.lora_forward(torch.zeros(16, 72, dtype=torch.bfloat16, device="cuda")[:, 4:68], base=base, **d)
    with pytest.raises(ValueError):
        w8.lora_forward(x[:1].expand(16, 64), base=base, **d)
    dy = t.dy.cuda()
    for b in (dict(u=None), dict(dy=dy[:, :64]), dict(x=x[:8]), dict(da=torch.empty(2, 16, 72).cuda()),
              dict(db=torch.empty(2, 72, 16)), dict(base=base)):
        kw = dict(dict(dy=dy, x=x, u=u, **d), **b)
        with pytest.raises((TypeError, ValueError)):
            w8.lora_backward(**kw)


# ------------------------------------------------------ infinite operands
def _same(got, ref, bound, what):
    """The infinities (with their signs) and NaN of the definition in 64 bits,
    and its finite values within their bounds."""
    got = got.cpu().to(f64)
    for kind, f in (("NaN", torch.isnan), ("+inf", torch.isposinf), ("-inf", torch.isneginf)):
        wrong = f(got) != f(ref)
        assert not wrong.any(), f"{what}: {kind} differs at {int(wrong.sum())} of {wrong.numel()}: " \
            f"got {got[wrong][0]}, ref {ref[wrong][0]}"
    ok = ref.isfinite()
    _near(got[ok], ref[ok], bound[ok], what)


# few rows: one launch (R <= 16) or the ranks in parts; many columns or rows: 64 rows an up-projection workgroup
INFINITE = [(40, 264, 328, 8), (40, 264, 328, 16), (70, 264, 328, 32), (70, 264, 328, 72), (8300, 2056, 72, 16),
            (8300, 72, 2056, 64), (8300, 72, 2056, 128)]


@pytest.mark.parametrize("case", INFINITE, ids=lambda c: "M%d-K%d-N%d-R%d" % c)
def test_an_infinite_factor_gives_infinities(w8, case):
    """A finite u (or g) against an infinite entry of b (or a): the signed
    infinity of their product, NaN only where infinities of both signs (or
    0 * inf) meet.  u of row 0 is exactly two values of bf16, its other half 0."""
    M, K, N, R = case
    print(f"[lora] infinite factors {case}", flush=True)
    t = Batch([M - 9, 9], [1, 0], K, N, R, 2, seed=M + R)
    t.x[0] = 0
    t.x[0, 0] = 1.0                                              # u[0] = scale a[1, :, 0]
    t.scale[1] = 1.0
    d = t.dev(w8)
    _, u = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **d)  # of finite factors
    j, inf = R - 3, float("inf")
    t.b[1, 5, 2], t.b[1, 6, j], t.b[0, N - 1, 1] = inf, -inf, inf
    t.b[1, 9, 0], t.b[1, 9, j] = inf, inf                        # products of both signs in most rows
    out, _ = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **t.dev(w8))
    ref, _, eo, _ = t.forward()
    assert torch.isinf(ref).any() and ref.isnan().any()
    _same(out, ref, eo, "out")
    t = Batch([M - 9, 9], [1, 0], K, N, R, 2, seed=M + R)
    t.a[1, 2, 5], t.a[1, j, 6], t.a[0, 1, K - 1] = inf, -inf, inf
    t.a[1, 0, 9], t.a[1, j, 9] = -inf, inf
    dx, da, db = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, base=t.dbase.cuda(), **t.dev(w8))
    rx, ra, rb, ex, ea, eb = t.backward(u.cpu())
    assert torch.isinf(rx).any() and rx.isnan().any()
    _same(dx, rx, ex, "dx")
    _same(da, ra, ea, "da")
    _same(db, rb, eb, "db")


def test_a_u_near_the_largest_number(w8):
    """u is finite but nearest to no finite bf16: its products are finite."""
    t = Batch([3], [0], 64, 64, 8, 1, seed=6)
    t.x.zero_()
    t.a.zero_()
    t.x[1, 0], t.a[0, 0, 0] = torch.finfo(torch.bfloat16).max, 1.0
    t.scale = torch.tensor([1.003])
    t.b.zero_()
    t.b[0, :32, 0], t.b[0, 40, 0] = 2.0 ** -20, -2.0 ** -20
    t.base.zero_()
    out, u = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **t.dev(w8))
    ref, refu, eo, eu = t.forward()
    assert refu[1, 0] > 3.3962e38 and u.isfinite().all()
    _same(u, refu, eu, "u")
    _same(out, ref, eo, "out")


@pytest.mark.parametrize("R", [8, 32, 64, 128])
@pytest.mark.parametrize("lengths", [[70, 5], [700, 9]])
def test_infinite_rows_in_the_gradients(w8, lengths, R):
    """An infinity in dy or x against finite u and g: the signed infinity of
    their product in dB's and dA's entries, NaN only where the definition has
    it."""
    print(f"[lora] infinite rows {lengths} R{R}", flush=True)
    t = Batch(lengths, [1, 0], 136, 264, R, 2, seed=R)
    _, u = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **t.dev(w8))
    u = u.cpu()
    u[3] = u[3].bfloat16().float()                               # exactly bf16: its other parts are 0
    u[3, 1] = 1.0
    t.dy[3, 7], t.dy[30, 100], t.dy[31, 8] = float("inf"), float("-inf"), float("inf")
    t.dy[32, 8] = float("-inf")                                  # both signs in column 8: inf or NaN by u's signs
    t.x[5, 9], t.x[50, 135], t.x[lengths[0] + 1, 0] = float("inf"), float("-inf"), float("inf")
    dx, da, db = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u.cuda(), base=t.dbase.cuda(), **t.dev(w8))
    rx, ra, rb, ex, ea, eb = t.backward(u)
    assert torch.isinf(ra).any() and torch.isinf(rb).any() and rb.isnan().any()
    _same(db, rb, eb, "db")
    _same(da, ra, ea, "da")
    _same(dx, rx, ex, "dx")


@pytest.mark.parametrize("bits", [0x7FC00000, 0x7F800001, -0x7FFFFF])
@pytest.mark.parametrize("R", [8, 128])
def test_any_nan_of_u_is_a_nan_of_db(w8, bits, R):
    """Whatever the NaN's payload and sign (the cut to bf16 parts must not
    leave an infinity of one whose payload is in its low bits)."""
    t = Batch([70, 5], [1, 0], 136, 264, R, 2, seed=R)
    _, u = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **t.dev(w8))
    u = u.cpu()
    u[12, R - 1] = torch.tensor(bits, dtype=torch.int32).view(torch.float32)
    assert u[12, R - 1].isnan()
    _, da, db = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u.cuda(), base=t.dbase.cuda(), **t.dev(w8))
    _, ra, rb, _, ea, eb = t.backward(u)
    _same(db, rb, eb, "db")
    _same(da, ra, ea, "da")
    assert db[1, :, R - 1].isnan().all()


# ------------------------------------------------- more than one launch holds
def _rows_check(rows, l, s, x, u, out, base, a, b, what):
    """u and out of some rows of adapter l against the definition."""
    xf, af, bf, uf = x[rows].cpu().to(f64), a[l].cpu().to(f64), b[l].cpu().to(f64), u[rows].cpu().to(f64)
    ru = s * (xf @ af.T)
    eu = (xf.shape[1] + 8) * U23 * s * (xf.abs() @ af.abs().T)
    _near(u[rows], ru, eu, what + " u")
    basef = base[rows].cpu().to(f64)
    ro = basef + uf @ bf.T
    eo = (uf.abs() * (2.0 ** -16 + (2 * uf.shape[1] + 8) * U23)) @ bf.abs().T
    _near(out[rows], ro, eo + 2.0 ** -8 * ro.abs() + 4 * U23 * basef.abs(), what + " out")


@pytest.mark.parametrize("T,K,N", [(2 ** 22 + 3, 8, 8), (360001, 8, 1032), (360001, 1032, 8)])
def test_requests_beyond_one_launch(w8, T, K, N):
    """So many requests of one row that the workgroups' threads pass 2^32, or
    the columns' workgroups a launch's most; every third without an adapter,
    which comes first in the plan."""
    print(f"[lora] {T} requests K{K} N{N}", flush=True)
    R, L = 8, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x, dy, base, dbase, a, b = rnd(T, K), rnd(T, N), rnd(T, N), rnd(T, K), rnd(L, R, K), rnd(L, N, R)
    scale = torch.tensor([1.0, 0.5], device="cuda")
    adapters = ([0, 1, -1] * (T // 3 + 1))[:T]
    plan = w8.lora_plan([1] * T, adapters, L)
    assert plan.tiles == T
    out, u = w8.lora_forward(x, a, b, plan, scale=scale, base=base)
    dx, da, db = w8.lora_backward(dy, x, u, a, b, plan, scale=scale, base=dbase)
    v = torch.empty_like(u)                                      # g of the definition, rounded to f32
    for l in range(L):
        s = float(scale[l])
        v[l::3] = (s * torch.mm(dy[l::3].to(f64), b[l].to(f64))).float()
        picked = torch.tensor([l, l + 3 * (T // 9), l + 3 * (T // 6), l + 3 * ((T - 1 - l) // 3)])
        _rows_check(picked, l, s, x, u, out, base, a, b, f"adapter {l}")
        vr = v[picked].cpu().to(f64)
        rx = dbase[picked].cpu().to(f64) + vr @ a[l].cpu().to(f64)
        eg = (N + 8) * U23 * s * (dy[picked].cpu().to(f64).abs() @ b[l].cpu().to(f64).abs())
        ex = (vr.abs() * (2.0 ** -16 + (2 * R + 8) * U23) + eg) @ a[l].cpu().to(f64).abs()
        _near(dx[picked], rx, ex + 2.0 ** -8 * rx.abs() + 4 * U23 * dbase[picked].cpu().to(f64).abs(), "dx")
        vl, xl, ul, dl = (t[l::3].to(f64) for t in (v, x, u, dy))
        e = (vl.shape[0] + 16) * U23
        egl = (N + 8) * U23 * s * torch.mm(dl.abs(), b[l].to(f64).abs())
        _near(da[l], torch.mm(vl.t(), xl).cpu(), torch.mm((e * vl.abs() + egl).t(), xl.abs()).cpu(), "da")
        _near(db[l], torch.mm(dl.t(), ul).cpu(), (e * torch.mm(dl.abs().t(), ul.abs())).cpu(), "db")
    assert not u[2::3].any() and torch.equal(out[2::3], base[2::3]) and torch.equal(dx[2::3], dbase[2::3])
    # every row: the same rows a part of the batch at a time give what the whole gave, but for the sums' order
    for first in range(0, T, 3 * 2 ** 17):
        rows = slice(first, min(first + 3 * 2 ** 17, T))
        n = rows.stop - first
        po, pu = w8.lora_forward(x[rows], a, b, w8.lora_plan([1] * n, adapters[rows], L), scale=scale, base=base[rows])
        off = (po.float() - out[rows].float()).abs()
        assert bool((off <= 2.0 ** -7 * po.float().abs() + 1e-3).all()), first
        assert torch.allclose(pu, u[rows], rtol=1e-4, atol=1e-4), first


def test_a_pool_beyond_one_launch(w8):
    """The weights' gradients of 65535 adapters: more workgroups than a launch
    has; a few of the adapters are used."""
    print("[lora] 65535 adapters", flush=True)
    L, K, N, R = 65535, 8, 2056, 8
    used = [0, 777, 58254, 65534]
    small = Batch([70, 1, 9, 130, 3], [2, 0, 3, 1, -1], K, N, R, 4, scale=False, seed=11)
    a = torch.zeros((L, R, K), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((L, N, R), dtype=torch.bfloat16, device="cuda")
    a[used], b[used] = small.a.cuda(), small.b.cuda()
    plan = w8.lora_plan(small.lengths, [used[l] if l >= 0 else -1 for l in small.adapters], L)
    _, u = w8.lora_forward(small.x.cuda(), a, b, plan, base=small.base.cuda())
    da, db = torch.full((L, R, K), 7.0, device="cuda"), torch.full((L, N, R), 7.0, device="cuda")
    dx, _, _ = w8.lora_backward(small.dy.cuda(), small.x.cuda(), u, a, b, plan, base=small.dbase.cuda(), da=da, db=db)
    rx, ra, rb, ex, ea, eb = small.backward(u.cpu())
    _near(dx, rx, ex, "dx")
    _near(da[used], ra, ea, "da")
    _near(db[used], rb, eb, "db")
    da[used] = 0
    db[used] = 0
    assert not da.any() and not db.any()


# ---------------------------------------------------------- the other variants
@pytest.mark.parametrize("R", [8, 24, 64, 128])
def test_sixty_four_rows_an_up_workgroup(w8, R):
    """Enough tiles and columns, both ways, for an up-projection's workgroup to
    take all 64 rows of a tile, its last ones in part."""
    _check(w8, Batch([4100, 37, 4064], [1, -1, 0], 2056, 2104, R, 2, seed=R), f"64 rows R{R}")


@pytest.mark.parametrize("R", [8, 16])
@pytest.mark.parametrize("K,N", [(264, 4104), (4104, 264), (2056, 4104)])
@pytest.mark.parametrize("S", [1, 30])
def test_one_launch_of_several_column_groups(w8, S, K, N, R):
    """Down- and up-projection in one launch where an output is wider than one
    workgroup's columns: the further ones repeat the sums and leave u alone."""
    lengths = [1] * (S - 1) + [5]
    adapters = [i % 4 - 1 for i in range(S - 1)] + [2]
    t = Batch(lengths, adapters, K, N, R, 3, seed=S + K)
    _check(w8, t, f"{S} requests K{K} N{N} R{R}")
    d = t.dev(w8)
    want, wu = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **d)
    base = t.base.cuda()
    out, u = w8.lora_forward(t.x.cuda(), base=base, out=base, **d)
    assert torch.equal(out, want) and torch.equal(u, wu)
    alone, none = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), save_u=False, **d)
    assert none is None and torch.equal(alone, want)
    wdx = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, base=t.dbase.cuda(), **d)[0]
    dbase = t.dbase.cuda()
    assert torch.equal(w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, base=dbase, out=dbase, **d)[0], wdx)


def test_binding_refuses_what_is_no_tensor(w8):
    t = Batch([10, 6], [0, 1], 64, 72, 16, 2)
    d = t.dev(w8)
    x, dy, u = t.x.cuda(), t.dy.cuda(), torch.zeros(16, 16, device="cuda")
    for name in ("a", "b", "scale", "ranks"):
        for bad in ([1.0], 3, "a"):
            kw = dict(d, **{name: bad})
            with pytest.raises(TypeError):
                w8.lora_forward(x, **kw)
            with pytest.raises(TypeError):
                w8.lora_backward(dy, x, u, **kw)
    for name in ("a", "b"):
        with pytest.raises(TypeError):
            w8.lora_forward(x, **dict(d, **{name: None}))


@pytest.mark.parametrize("case", [(40, 264, 328, 8), (70, 264, 328, 32), (300, 264, 328, 128), (8300, 72, 2056, 16),
                                  (8300, 72, 2056, 64), (8300, 72, 2056, 128)], ids=lambda c: "M%d-K%d-N%d-R%d" % c)
def test_non_finite_values_of_base_stay_where_they_are(w8, case):
    """NaN and infinities in base: in out at the same places, every other
    element the bits of a base without them; rows with an adapter, without one
    and with a rank of 0, in place too."""
    M, K, N, R = case
    print(f"[lora] non-finite base {case}", flush=True)
    n = M // 3
    t = Batch([n, n, M - 2 * n], [0, -1, 1], K, N, R, 2, ranks=[R - 1, 0], seed=M + R)
    d = t.dev(w8)
    want, u = w8.lora_forward(t.x.cuda(), base=t.base.cuda(), **d)
    wdx, wa, wb = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, base=t.dbase.cuda(), **d)
    for cols, clean, grad in ((N, want, False), (K, wdx, True)):
        g = torch.Generator().manual_seed(R)
        at = torch.rand(M, cols, generator=g) < 3 / cols
        at[1], at[n + 1], at[2 * n + 1] = False, False, False
        bad = torch.where(torch.rand(M, cols, generator=g) < 0.5, float("nan"), float("-inf")).bfloat16()
        base = torch.where(at, bad, t.dbase if grad else t.base).cuda()
        for inplace in (False, True):
            b = base.clone()
            out = b if inplace else None
            if grad:
                got, ga, gb = w8.lora_backward(t.dy.cuda(), t.x.cuda(), u, base=b, out=out, **d)
                assert torch.equal(ga, wa) and torch.equal(gb, wb)
            else:
                got, gu = w8.lora_forward(t.x.cuda(), base=b, out=out, **d)
                assert torch.equal(gu, u)
            got = got.cpu()
            assert torch.equal(got[~at], clean.cpu()[~at])
            assert torch.equal(got[at].isnan(), bad[at].isnan()) and torch.equal(got[at].isneginf(), bad[at].isneginf())
