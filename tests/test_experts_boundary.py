"""The C ABI of include/w8a8_experts.h without a GPU: exports, sizes, and
refusals before anything is launched."""
import random

import pytest
import torch

import experts_helpers as ref
import w8a8_quantized_linear_quant_amd as w8

lib = w8.library()
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED = range(5)
A = 1 << 20       # a 16-byte aligned fake address (never dereferenced)
MIS = A + 4
NULL = None


def test_exports_match_header():
    names = w8.exported_names_in_header(w8.EXPERTS_HEADER)
    assert names == ["mxfp4_dequantize", "mxfp4_linear", "mxfp4_linear_backward_dx", "mxfp4_linear_grouped",
                     "mxfp4_linear_grouped_backward_dx", "mxfp4_quantize", "mxfp4_quantize_transposed",
                     "mxfp4_scale_stride", "w8a8_linear_grouped", "w8a8_linear_grouped_backward_dx",
                     "w8a8_probe_grouped_kernel"]
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("K,want", [(-1, 0), (0, 0), (1, 16), (32, 16), (512, 16), (513, 32), (544, 32), (4096, 128)])
def test_scale_stride(K, want):
    assert lib.mxfp4_scale_stride(K) == want
    if K >= 0:
        assert w8.mxfp4_scale_stride(K) == want


def _quantize(xt=0, x=A, M=4, K=64, ldx=64, xq=A, ldq=64, xs=A):
    return lib.mxfp4_quantize(xt, x, M, K, ldx, xq, ldq, xs, NULL)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(M=0)), (OK, dict(M=0, x=NULL, xq=NULL, xs=NULL)), (INVALID, dict(xt=2)), (INVALID, dict(M=-1)),
    (INVALID, dict(x=NULL)), (INVALID, dict(xq=NULL)), (INVALID, dict(xs=NULL)), (ALIGN, dict(x=MIS)),
    (ALIGN, dict(xq=MIS)), (ALIGN, dict(xs=MIS)), (SHAPE, dict(K=0)), (SHAPE, dict(K=65)), (SHAPE, dict(ldx=63)),
    (SHAPE, dict(ldq=48)), (SHAPE, dict(ldq=32)), (SHAPE, dict(M=(1 << 30) + 1)), (SHAPE, dict(ldx=(1 << 24) + 1)),
    (SHAPE, dict(K=(1 << 22) + 1, ldx=1 << 23, ldq=(1 << 22) + 32)), (SHAPE, dict(M=1 << 28)),
])
def test_quantize_refusals(want, kw):
    assert _quantize(**kw) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(M=0)), (INVALID, dict(yt=5)), (INVALID, dict(y=NULL)), (INVALID, dict(xs=NULL)), (ALIGN, dict(y=MIS)),
    (SHAPE, dict(ldy=63)), (SHAPE, dict(K=65)), (SHAPE, dict(ldq=40)), (INVALID, dict(M=-2)),
])
def test_dequantize_refusals(want, kw):
    a = dict(xq=A, xs=A, M=4, K=64, ldq=64, yt=0, y=A, ldy=64)
    a.update(kw)
    assert lib.mxfp4_dequantize(a["xq"], a["xs"], a["M"], a["K"], a["ldq"], a["yt"], a["y"], a["ldy"], NULL) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(B=0)), (INVALID, dict(B=-1)), (SHAPE, dict(B=65536)), (SHAPE, dict(N=0)), (SHAPE, dict(K=0)),
    (SHAPE, dict(ldx=95)), (SHAPE, dict(ldq=32)), (SHAPE, dict(ldq=72)), (INVALID, dict(w=NULL)),
    (INVALID, dict(wq=NULL)), (INVALID, dict(ws=NULL)), (ALIGN, dict(w=MIS)), (ALIGN, dict(ws=MIS)),
    (SHAPE, dict(B=65535, N=1 << 20, K=1 << 20, ldx=1 << 20, ldq=1 << 20)), (INVALID, dict(wt=-1)),
    (SHAPE, dict(N=1 << 22, K=1 << 18, ldx=1 << 18, ldq=1 << 22)),
])
def test_quantize_transposed_refusals(want, kw):
    a = dict(wt=1, w=A, B=2, N=64, K=96, ldx=96, wq=A, ldq=64, ws=A)
    a.update(kw)
    assert lib.mxfp4_quantize_transposed(a["wt"], a["w"], a["B"], a["N"], a["K"], a["ldx"], a["wq"], a["ldq"], a["ws"],
                                         NULL) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(M=0)), (OK, dict(N=0)), (OK, dict(M=0, xq=NULL, y=NULL)), (INVALID, dict(M=-1)), (INVALID, dict(K=-32)),
    (SHAPE, dict(K=0)), (SHAPE, dict(K=48)), (SHAPE, dict(K=(1 << 22) + 32)), (SHAPE, dict(M=1 << 30, N=1 << 30)),
    (INVALID, dict(xq=NULL)), (INVALID, dict(xs=NULL)), (INVALID, dict(wq=NULL)), (INVALID, dict(ws=NULL)),
    (INVALID, dict(y=NULL)), (ALIGN, dict(xq=MIS)), (ALIGN, dict(xs=MIS)), (ALIGN, dict(ws=MIS)), (ALIGN, dict(y=MIS)),
    (ALIGN, dict(bias=MIS)),
])
def test_mx_linear_refusals(want, kw):
    a = dict(xq=A, xs=A, wq=A, ws=A, bias=NULL, M=4, N=8, K=64, y=A)
    a.update(kw)
    assert lib.mxfp4_linear(*a.values(), NULL) == want
    if "K" not in kw and "N" not in kw and "bias" not in kw:
        # the backward product reduces over N = 64 to K = 8 columns
        b = dict(a, N=a["K"], K=a["N"])
        assert lib.mxfp4_linear_backward_dx(b["xq"], b["xs"], b["wq"], b["ws"], b["M"], b["N"], b["K"], b["y"],
                                            NULL) == want


GROUPED = [
    (OK, dict(M=0)), (OK, dict(N=0)), (INVALID, dict(M=-1)), (INVALID, dict(X=-1)), (SHAPE, dict(E=0)),
    (SHAPE, dict(E=4097)), (SHAPE, dict(X=5, rows=NULL)), (INVALID, dict(offsets=NULL)), (ALIGN, dict(offsets=MIS)),
    (ALIGN, dict(rows=MIS)), (INVALID, dict(xq=NULL)), (INVALID, dict(xs=NULL)), (INVALID, dict(wq=NULL)),
    (INVALID, dict(ws=NULL)), (INVALID, dict(y=NULL)), (ALIGN, dict(xq=MIS)), (ALIGN, dict(wq=MIS)),
    (ALIGN, dict(xs=MIS)), (ALIGN, dict(ws=MIS)), (ALIGN, dict(bias=MIS)), (ALIGN, dict(y=MIS)),
    (SHAPE, dict(X=(1 << 30) + 1)), (SHAPE, dict(M=1 << 30, N=1 << 20)),
    (SHAPE, dict(X=1 << 20, K=1 << 13)),                       # 2^33 bytes (2^32 in 4 bits) to gather from
]


@pytest.mark.parametrize("want,kw", GROUPED + [(SHAPE, dict(K=8)), (SHAPE, dict(K=0)), (SHAPE, dict(K=24)),
                                               (INVALID, dict(qt=2)), (INVALID, dict(K=-16))])
def test_grouped_refusals(want, kw):
    a = dict(qt=0, xq=A, X=6, xs=A, wq=A, ws=A, per_channel=0, bias=NULL, offsets=A, E=3, rows=A, M=4, N=8, K=64, y=A)
    a.update(kw)
    assert lib.w8a8_linear_grouped(*a.values(), NULL) == want


@pytest.mark.parametrize("want,kw", GROUPED + [(SHAPE, dict(K=16)), (SHAPE, dict(K=48)), (INVALID, dict(K=-32))])
def test_mx_grouped_refusals(want, kw):
    a = dict(xq=A, X=6, xs=A, wq=A, ws=A, bias=NULL, offsets=A, E=3, rows=A, M=4, N=8, K=64, y=A)
    a.update(kw)
    assert lib.mxfp4_linear_grouped(*a.values(), NULL) == want


@pytest.mark.parametrize("want,kw", [(OK, dict(M=0)), (SHAPE, dict(E=0)), (SHAPE, dict(N=8)), (INVALID, dict(offsets=NULL)),
                                     (ALIGN, dict(wq=MIS)), (INVALID, dict(y=NULL))])
def test_grouped_backward_refusals(want, kw):
    a = dict(xq=A, xs=A, wq=A, ws=A, offsets=A, E=3, M=4, N=64, K=8, y=A)
    a.update(kw)
    assert lib.w8a8_linear_grouped_backward_dx(1, *a.values(), NULL) == want
    assert lib.mxfp4_linear_grouped_backward_dx(*a.values(), NULL) == want


def test_binding_wants_gpu_tensors():
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    s = torch.zeros(4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        w8.mxfp4_quantize(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="GPU tensor"):
        w8.mxfp4_quantize_transposed(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="GPU tensor"):
        w8.mxfp4_dequantize(u8, s)
    with pytest.raises(ValueError, match="GPU tensor"):
        w8.mxfp4_linear(u8, s, u8, s)
    with pytest.raises(TypeError, match="torch.uint8"):
        w8.mxfp4_linear(u8.float(), s, u8, s)
    with pytest.raises(TypeError, match="torch.Tensor"):
        w8.mxfp4_linear(u8, None, u8, s)
    with pytest.raises(TypeError):
        w8.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.float16))
    i8 = torch.zeros(4, 32, dtype=torch.int8)
    with pytest.raises(ValueError, match="GPU tensor"):
        w8.w8a8_linear_grouped(i8, None, i8[None], None, None)
    with pytest.raises(TypeError, match="torch.Tensor"):
        w8.w8a8_linear_grouped([1], None, i8[None], None, None)
    with pytest.raises(TypeError):
        w8.w8a8_linear_grouped(u8, None, u8[None], None, None)
    with pytest.raises(ValueError, match="w_scale must be"):
        w8.w8a8_linear_grouped_backward_dx(i8, None, i8[None], torch.zeros(1, 4), None)


def test_the_kernels_that_the_gpu_tests_name():
    for kind, kernel, M, E, N, K in ref.KERNELS:
        assert w8.probe_grouped_kernel(kind, M, N, K, E) == kernel, (kind, kernel, M, E, N, K)
    assert {k[:2] for k in ref.KERNELS} == {(t, k) for t in ("int8", "e4m3", "mx") for k in range(8)}


def test_probe_rejects():
    for args in ((0, 0, 8, 64, 1), (0, 8, 0, 64, 1), (0, 8, 8, 0, 1), (0, 8, 8, 64, 0), (3, 8, 8, 64, 1), (-1, 8, 8, 64, 1),
                 (0, 8, 8, 64, 4097), (2, (1 << 30) + 1, 8, 64, 1)):
        assert lib.w8a8_probe_grouped_kernel(*args) == -1, args


def test_few_rows_take_one_launch():
    """Kernels 0 to 3 have a workgroup a tile, column tiles in eights: 2^23 at most (2^31 threads), whatever the sizes."""
    rng, edge = random.Random(4), {0: (16, 16), 1: (16, 32), 2: (32, 32), 3: (64, 64)}
    for _ in range(20000):
        kind = rng.choice(("int8", "e4m3", "mx"))
        E, M, N, K = (int(2 ** rng.uniform(lo, hi)) for lo, hi in ((0, 12), (0, 30), (4, 30), (0, 17)))
        kernel = w8.probe_grouped_kernel(kind, M, N, 32 * K, E)
        if kernel in edge:
            rows, columns = edge[kernel]
            assert (M // rows + min(E, M)) * (-(-N // (8 * columns)) * 8) <= 2 ** 23, (kind, M, N, K, E)
