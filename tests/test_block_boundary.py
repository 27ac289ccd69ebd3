"""The C ABI of include/w8a8_block.h without a GPU: exports, the plan that the
host builds, workspace sizes, and refusals before anything is launched."""
import ctypes

import pytest
import torch

import w8a8_quantized_linear_quant_amd as w8

lib = w8.library()
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED = range(5)
A = 1 << 20       # a 16-byte aligned fake address (never dereferenced)
MIS = A + 2
NULL = None
TILE = 64


def test_exports_match_header():
    names = w8.exported_names_in_header(w8.BLOCK_HEADER)
    assert names == ["layer_norm_backward", "layer_norm_backward_workspace_bytes", "layer_norm_forward",
                     "lora_backward", "lora_backward_workspace_bytes", "lora_forward",
                     "lora_forward_workspace_bytes", "lora_plan", "w8a8_quant_act_rowwise_layer_norm"]
    for n in names:
        assert hasattr(lib, n), n


def _plan(lengths, adapters, L):
    p = w8.lora_plan(lengths, adapters, L, device="cpu")
    d = p.data.tolist()
    tiles = [tuple(d[4 * t:4 * t + 4]) for t in range(p.tiles)]
    return p, tiles, d[4 * p.tiles:]


def test_plan_of_uneven_requests():
    lengths, adapters = [0, 1, 64, 65, 3, 200, 0, 63], [1, 2, 0, -1, 2, 0, 0, 1]
    p, tiles, first = _plan(lengths, adapters, 4)
    assert p.rows == sum(lengths) and p.adapters == 4
    # row ranges by request, tile by tile, ordered by adapter and row
    want, row = [], 0
    for n, l in zip(lengths, adapters):
        want += [(row + i, min(TILE, n - i), l, 0) for i in range(0, n, TILE)]
        row += n
    want.sort(key=lambda t: (t[2], t[0]))
    assert tiles == want
    assert len(first) == 5
    for l in range(4):
        assert all(t[2] == l for t in tiles[first[l]:first[l + 1]])
    assert first[4] == p.tiles and all(t[2] == -1 for t in tiles[:first[0]])
    assert first[3] == first[4]                                     # an adapter that nobody uses


@pytest.mark.parametrize("lengths,adapters,tiles", [([], [], 0), ([0, 0], [0, -1], 0), ([5], [-1], 1), ([1] * 70, [0] * 70, 70)])
def test_plan_small(lengths, adapters, tiles):
    p, t, first = _plan(lengths, adapters, 1)
    assert p.tiles == tiles and first[-1] == tiles and sum(e[1] for e in t) == sum(lengths)


def test_plan_refusals():
    with pytest.raises(ValueError):
        w8.lora_plan([1, 2], [0], 1, device="cpu")
    with pytest.raises(ValueError):
        w8.lora_plan([1], [1], 1, device="cpu")
    with pytest.raises(ValueError):
        w8.lora_plan([1], [-2], 1, device="cpu")
    with pytest.raises(w8.W8A8Error):
        w8.lora_plan([-1], [0], 1, device="cpu")
    with pytest.raises(w8.W8A8Error):
        w8.lora_plan([1 << 30, 1], [0, 0], 1, device="cpu")          # more than 2^30 rows
    f = lib.lora_plan
    n, l, t = (ctypes.c_int64 * 1)(65), (ctypes.c_int32 * 1)(0), ctypes.c_int64()
    assert f(n, l, 1, 1, None, 0, ctypes.byref(t)) == OK and t.value == 2
    out = (ctypes.c_int32 * 10)()
    assert f(n, l, 1, 1, out, 9, ctypes.byref(t)) == SHAPE           # one integer short
    assert f(n, l, 1, 1, out, 10, ctypes.byref(t)) == OK
    assert list(out) == [0, 64, 0, 0, 64, 1, 0, 0, 0, 2]
    assert f(n, l, 1, 0, None, 0, ctypes.byref(t)) == SHAPE          # no pool
    assert f(n, l, 1, 65536, None, 0, ctypes.byref(t)) == SHAPE
    assert f(NULL, l, 1, 1, None, 0, ctypes.byref(t)) == INVALID
    assert f(n, l, -1, 1, None, 0, ctypes.byref(t)) == INVALID


def _forward(M=64, K=64, ldx=64, L=2, N=64, R=16, T=1, ldb=64, ldo=64, x=A, a=A, b=A, plan=A, base=A, out=A, u=A, ws=A,
             ranks=A):
    return lib.lora_forward(x, M, K, ldx, a, b, L, N, R, A, ranks, plan, T, base, ldb, out, ldo, u, ws, NULL)


def _backward(M=64, K=64, N=64, R=16, L=2, T=1, lddy=64, ldx=64, dy=A, x=A, u=A, base=A, ldb=64, dx=A, lddx=64, da=A,
              db=A, ws=A):
    return lib.lora_backward(dy, M, N, lddy, x, K, ldx, u, A, A, L, R, A, A, A, T, base, ldb, dx, lddx, da, db, ws,
                             NULL)


@pytest.mark.parametrize("f", [_forward, _backward])
def test_lora_refuses_sizes(f):
    assert f(R=0) == INVALID and f(R=136) == INVALID and f(R=4) == INVALID
    assert f(R=12) == SHAPE
    assert f(K=60) == SHAPE and f(N=60) == SHAPE and f(N=0) == SHAPE and f(K=(1 << 22) + 8, ldx=(1 << 22) + 8) == SHAPE
    assert f(ldx=56) == SHAPE and f(ldx=68) == SHAPE and f(ldb=60) == SHAPE
    assert f(L=0) == INVALID and f(L=65536) == SHAPE
    assert f(M=-1) == INVALID and f(T=-1) == INVALID and f(M=(1 << 30) + 1) == SHAPE


def test_lora_refuses_pointers():
    assert _forward(x=NULL) == INVALID and _forward(out=NULL) == INVALID and _forward(plan=NULL) == INVALID
    assert _forward(u=NULL, ws=NULL) == INVALID and _forward(a=NULL) == INVALID and _forward(ws=MIS) == ALIGN
    assert _forward(x=MIS) == ALIGN and _forward(out=MIS) == ALIGN and _forward(u=MIS) == ALIGN
    assert _forward(base=MIS) == ALIGN and _forward(ranks=MIS) == ALIGN and _forward(plan=MIS) == ALIGN
    assert _forward(ldo=60) == SHAPE
    assert _forward(M=0, x=NULL, out=NULL) == OK and _forward(T=0) == OK
    assert _backward(dy=NULL) == INVALID and _backward(u=NULL) == INVALID and _backward(x=NULL) == INVALID
    assert _backward(da=NULL) == INVALID and _backward(db=NULL) == INVALID           # both or neither
    assert _backward(dy=MIS) == ALIGN and _backward(dx=MIS) == ALIGN and _backward(da=MIS) == ALIGN
    assert _backward(lddy=56) == SHAPE and _backward(lddx=60) == SHAPE
    assert _backward(ws=NULL) == INVALID and _backward(ws=MIS) == ALIGN


def test_lora_workspace_sizes():
    assert w8.lora_forward_workspace_bytes(0, 16) == 0 and w8.lora_forward_workspace_bytes(5, 16) == 5 * 16 * 4
    assert lib.lora_forward_workspace_bytes(-1, 16) == 0 and lib.lora_forward_workspace_bytes(1, 129) == 0
    one, many = (w8.lora_backward_workspace_bytes(64 * t, t, 64, 64, 16, 1) for t in (1, 100))
    assert 64 * 16 * 4 <= one < many
    assert lib.lora_backward_workspace_bytes(64, 1, 64, 64, 16, 0) == 0


def _norm(xt=0, x=A, M=4, K=64, ldx=64, wt=0, w=A, b=A, eps=1e-5, y=A, ldy=64, mean=A, rstd=A):
    return lib.layer_norm_forward(xt, x, M, K, ldx, wt, w, b, eps, y, ldy, mean, rstd, NULL)


def _norm_backward(xt=0, dy=A, lddy=64, x=A, ldx=64, mean=A, rstd=A, M=4, K=64, wt=0, w=A, dx=A, lddx=64, dw=A, db=A,
                   ws=A):
    return lib.layer_norm_backward(xt, dy, lddy, x, ldx, mean, rstd, M, K, wt, w, dx, lddx, dw, db, ws, NULL)


def _norm_quant(qt=0, xt=0, x=A, M=4, K=64, ldx=64, wt=0, w=A, b=A, eps=1e-5, xq=A, ldq=64, sx=A, mean=A, rstd=A):
    return lib.w8a8_quant_act_rowwise_layer_norm(qt, xt, x, M, K, ldx, wt, w, b, eps, xq, ldq, sx, mean, rstd, NULL)


@pytest.mark.parametrize("f", [_norm, _norm_backward, _norm_quant])
def test_layer_norm_refuses(f):
    assert f(xt=2) == INVALID and f(wt=-1) == INVALID and f(M=-1) == INVALID
    assert f(K=0) == SHAPE and f(ldx=63) == SHAPE and f(K=(1 << 24) + 16, ldx=(1 << 24) + 16) == SHAPE
    assert f(x=NULL) == INVALID and f(x=MIS) == ALIGN and f(w=MIS) == ALIGN and f(mean=MIS) == ALIGN


def test_layer_norm_refuses_the_rest():
    assert _norm(eps=-1.0) == INVALID and _norm(eps=float("nan")) == INVALID and _norm(eps=float("inf")) == INVALID
    assert _norm(ldy=63) == SHAPE and _norm(y=NULL) == INVALID and _norm(y=MIS) == ALIGN
    assert _norm(M=0, x=NULL, y=NULL) == OK
    assert _norm_backward(mean=NULL) == INVALID and _norm_backward(dy=NULL) == INVALID
    assert _norm_backward(ws=NULL) == INVALID and _norm_backward(lddx=63) == SHAPE
    assert _norm_backward(dx=MIS) == ALIGN and _norm_backward(dw=MIS) == ALIGN
    assert _norm_quant(qt=2) == INVALID and _norm_quant(ldq=48) == SHAPE and _norm_quant(ldq=72) == SHAPE
    assert _norm_quant(sx=NULL) == INVALID and _norm_quant(xq=MIS) == ALIGN
    assert _norm_quant(M=0, x=NULL, xq=NULL, sx=NULL) == OK
    assert lib.layer_norm_backward_workspace_bytes(4, 0) == 0 and lib.layer_norm_backward_workspace_bytes(4, 64) > 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    a, b = torch.zeros(1, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 64, 8, dtype=torch.bfloat16)
    plan = w8.lora_plan([4], [0], 1, device="cpu")
    with pytest.raises(ValueError):
        w8.lora_forward(x, a, b, plan)
    with pytest.raises(ValueError):
        w8.lora_backward(x, x, None, a, b, plan)
    with pytest.raises(ValueError):
        w8.layer_norm_forward(x)
    with pytest.raises(ValueError):
        w8.layer_norm_backward(x, x, x, x)
    with pytest.raises(ValueError):
        w8.w8a8_quant_act_rowwise_layer_norm(x)


@pytest.mark.parametrize("f", [_forward, _backward])
def test_lora_refuses_more_tiles_than_a_plan_has(f):
    assert f(M=1 << 30, T=(1 << 24) + 1) == SHAPE
