"""The input gradients of include/w8a8_experts.h through their own entry points."""
import inspect
import re

import pytest
import torch

import experts_helpers as ref
import w8a8_quantized_linear_quant_amd as w8

KINDS = ["int8", "e4m3", "mx"]


def test_the_binding_calls_every_entry_point():
    """Each entry point with a stream is launched by the function of its name."""
    with open(w8.EXPERTS_HEADER) as f:
        names = re.findall(r"(\w+)\([^()]*hipStream_t stream\)\s*;", f.read())
    assert len(names) == 9
    for name in names:
        assert f"_launch(_lib.{name}, " in inspect.getsource(getattr(w8, name)), name


class Recorder:
    """The library, with the names and sizes of the calls made through it."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        entry = getattr(self.lib, name)

        def call(*args):
            self.calls.append((name, [a for a in args if isinstance(a, int) and a < 1 << 16]))
            return entry(*args)
        return call


# lengths of the groups, N (the gradient's sum), K (its columns): N and K apart
CASES = [([1], 32, 48), ([5, 0, 2], 64, 160), ([0, 70, 3, 0], 96, 40), ([300, 1, 129], 544, 1000), ([900, 700], 1056, 520)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths,N,K", CASES)
def test_gradient_of_groups(monkeypatch, kind, lengths, N, K):
    """Whole codes and powers of two (sums below 2^24): every bit of the
    definition's, through the entry point of the gradient."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"[backward] {kind} {lengths} {N} {K}", flush=True)
    M, E = sum(lengths), len(lengths)
    offsets = [0]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(N + K)

    def integers(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda")

    recorder = Recorder(w8.library())
    monkeypatch.setattr(w8, "_lib", recorder)
    if kind == "mx":
        name = "mxfp4_linear_grouped_backward_dx"
        dq, wt = integers(0, 256, M, N // 2).to(torch.uint8), integers(0, 256, E, K, N // 2).to(torch.uint8)
        ds = integers(128, 130, M, ref.stride_of(N)).to(torch.uint8)
        ws = integers(128, 130, E, K, ref.stride_of(N)).to(torch.uint8)
        d, w = ref.values(dq, ds), ref.values(wt, ws)
    else:
        name = "w8a8_linear_grouped_backward_dx"
        code = torch.int8 if kind == "int8" else torch.float8_e4m3fn
        dq, wt = integers(-8, 9, M, N).float().to(code), integers(-8, 9, E, K, N).float().to(code)
        ds, ws = torch.pow(2.0, integers(-3, 4, M).float()), torch.pow(2.0, integers(-3, 4, E).float())
        d, w = dq.double() * ds.double()[:, None], wt.double() * ws.double()[:, None, None]
    out = torch.full((M, K), 7.25, dtype=torch.bfloat16, device="cuda")
    dx = getattr(w8, name)(dq, ds, wt, ws, off, out=out)
    want, _, inside = ref.grouped(d, w, offsets, M)
    assert bool(inside.all()) and dx is out and torch.equal(dx, want.float().bfloat16())
    assert torch.equal(dx, getattr(w8, name)(dq, ds, wt, ws, off))
    assert [c[0] for c in recorder.calls] == [name] * 2
    if kind == "mx" and E == 1:
        recorder.calls.clear()
        assert torch.equal(dx, w8.mxfp4_linear_backward_dx(dq, ds, wt[0], ws[0]))
        assert [c[0] for c in recorder.calls] == ["mxfp4_linear_backward_dx"]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 64, 1000), (33, 1056, 40), (700, 544, 520)])
def test_gradient_of_the_4_bit_linear(monkeypatch, M, N, K):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(M)
    recorder = Recorder(w8.library())
    monkeypatch.setattr(w8, "_lib", recorder)
    dq, ds = ref.random_mx(g, (M, N), 128, 130)
    wt, ws = ref.random_mx(g, (K, N), 128, 130)
    dx = w8.mxfp4_linear_backward_dx(dq, ds, wt, ws)
    assert dx.shape == (M, K) and [c[0] for c in recorder.calls] == ["mxfp4_linear_backward_dx"]
    assert torch.equal(dx, (ref.values(dq, ds) @ ref.values(wt, ws).T).float().bfloat16())


@pytest.mark.gpu
def test_refusals_name_the_gradients_operands():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    i8 = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    one = torch.ones(4, device="cuda")
    f = w8.w8a8_linear_grouped_backward_dx
    with pytest.raises(ValueError, match="share N"):
        f(i8, one, i8[None, :, :16].contiguous(), one[:1], off)
    with pytest.raises(TypeError, match="wq_t must hold"):
        f(i8, one, i8[None].float(), one[:1], off)
    with pytest.raises(ValueError, match="w_scale must have"):
        f(i8, one, i8[None], one, off)
    with pytest.raises(ValueError, match="dy_scale"):
        f(i8, one[:3], i8[None], one[:1], off)
    with pytest.raises(ValueError, match="offsets"):
        f(i8, one, i8[None], one[:1], off[:1])
    with pytest.raises(ValueError, match="out"):
        f(i8, one, i8[None], one[:1], off, out=torch.zeros(4, 5, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(w8.W8A8Error):
        f(i8, one, i8[None], None, off)
    q, s = ref.random_mx(torch.Generator().manual_seed(0), (4, 64))
    for call in (lambda *a: w8.mxfp4_linear_backward_dx(*a), lambda *a: w8.mxfp4_linear_grouped_backward_dx(*a, off)):
        with pytest.raises(ValueError, match="dyq must be"):
            call(q, s, *ref.random_mx(torch.Generator().manual_seed(0), (1, 4, 96)))
        with pytest.raises(ValueError, match="dy_scale must have"):
            call(q, s[:3].contiguous(), q, s)
        with pytest.raises(TypeError, match="wq_t and w_scale_t"):
            call(q, s, q.float(), s)
