"""Host side of the packed-row operators, on the CPU: what the calls refuse, workspace sizes, and the torch binding's
description of matrices.  Addresses are made up and never used: a refused call launches nothing."""
import ctypes

import pytest
import torch

import zero_partitioned_mixed_reduce_amd as zpm
from zero_partitioned_mixed_reduce_amd import _abi
from zero_partitioned_mixed_reduce_amd.packed import ZeroPacked, matrix

F16, BF16, F32 = _abi.ZERO_F16, _abi.ZERO_BF16, _abi.ZERO_F32
POW2, MAX = _abi.ZERO_SCALE_POW2, _abi.ZERO_SCALE_MAX
GELU, SILU = _abi.ZERO_ACT_GELU, _abi.ZERO_ACT_SILU
GB = 1 << 30


def mat(at, rows, cols, dtype=BF16, pitch=None):
    return _abi.zero_matrix_t(at, rows, cols, cols if pitch is None else pitch, dtype)


def pack(at, rows, cols, rule=POW2, pitch=None, scale=None):
    return _abi.zero_packed_t(at, at + GB // 2 if scale is None else scale, rows, cols,
                              max(16, (cols + 15) // 16 * 16) if pitch is None else pitch, rule)


def refused(needle, call, *args):
    with pytest.raises(zpm.ZeroError) as e:
        call(*args, None)
    assert e.value.status == _abi.ZERO_EINVAL and needle in str(e.value), str(e.value)


X, P, W, Y, Z = GB, 2 * GB, 3 * GB, 4 * GB, 5 * GB


@pytest.mark.parametrize("x, needle", [
    (mat(X, 8, 32, 0), "dtype"), (mat(X, 8, 32, 4), "dtype"), (mat(X, -1, 32), "rows"), (mat(X, 8, -1), "rows"),
    (mat(X, 8, (1 << 30) + 1), "rows"), (mat(X, 8, 32, pitch=31), "pitch"), (mat(X, 8, 32, pitch=(1 << 30) + 1), "pitch"),
    (mat(0, 8, 32), "null address"), (mat(X + 1, 8, 32), "aligned"), (mat(X + 2, 8, 32, F32), "aligned"),
    (mat(X, 8, 31), "same size"), (mat(X, 9, 32), "same size"), (None, "null x"),
    (mat(P + 64, 8, 32), "shares memory"), (mat(P + GB // 2, 8, 32), "shares memory")])
def test_write_refuses(x, needle):
    refused(needle, zpm.zero_packed_write, x, pack(P, 8, 32))


@pytest.mark.parametrize("p, needle", [
    (pack(P, 8, 32, 0), "rule"), (pack(P, 8, 32, 3), "rule"), (pack(P, -8, 32), "rows"), (pack(P, 8, (1 << 20) + 1), "cols"),
    (pack(P, 8, 32, pitch=24), "pitch"), (pack(P, 8, 32, pitch=40), "pitch"), (pack(P, 8, 32, pitch=(1 << 22) + 16), "pitch"),
    (pack(P + 8, 8, 32), "16-byte"), (pack(0, 8, 32, scale=P), "null address"), (pack(P, 8, 32, scale=0), "scales"),
    (pack(P, 8, 32, scale=P + GB // 2 + 2), "aligned"), (pack(P, 8, 32, scale=P + 16), "scales shares"), (None, "null p")])
def test_packed_rows_refused(p, needle):
    refused(needle, zpm.zero_packed_write, mat(X, 8, 32), p)
    if needle != "scales shares":
        refused(needle, zpm.zero_packed_read, p, mat(X, 8, 32))


def test_read_refuses():
    refused("same size", zpm.zero_packed_read, pack(P, 8, 32), mat(X, 8, 33))
    refused("shares memory", zpm.zero_packed_read, pack(P, 8, 32), mat(P + 128, 8, 32))
    refused("scales", zpm.zero_packed_read, pack(P, 8, 32), mat(P + GB // 2 - 64, 8, 32))
    refused("null out", zpm.zero_packed_read, pack(P, 8, 32), None)


def linear(x, w, bias, y, ws=None, cap=0):
    return zpm.zero_packed_linear, x, w, bias, y, ws, cap


@pytest.mark.parametrize("call, needle", [
    (linear(pack(X, 8, 32), pack(W, 16, 48), None, mat(Y, 8, 16)), "same number of columns"),
    (linear(pack(X, 8, 131057), pack(W, 16, 131057), None, mat(Y, 8, 16)), "131056"),
    (linear(pack(X, 8, 32), pack(W, 16, 32), None, mat(Y, 8, 17)), "y must be"),
    (linear(pack(X, 8, 32), pack(W, 16, 32), None, mat(Y, 16, 8)), "y must be"),
    (linear(pack(X, 8, 32), pack(W, 16, 32), mat(Z, 1, 15), mat(Y, 8, 16)), "bias must be"),
    (linear(pack(X, 8, 32), pack(W, 16, 32), mat(Z, 16, 1), mat(Y, 8, 16)), "bias must be"),
    (linear(pack(X, 8, 32), pack(W, 16, 32), mat(Y + 8, 1, 16), mat(Y, 8, 16)), "shares memory with bias"),
    (linear(pack(X, 8, 32), pack(W, 16, 32), None, mat(X + 32, 8, 16)), "shares memory with x"),
    (linear(pack(X, 8, 32), pack(W, 16, 32), None, mat(W + GB // 2, 8, 16)), "w's scales"),
    (linear(pack(X, 8, 32), pack(W, 16, 32), None, None), "null y"),
    (linear(pack(X, 8, 32), None, None, mat(Y, 8, 16)), "null w"),
    (linear(pack(X, 128, 65536), pack(W, 128, 65536), None, mat(Y, 128, 128)), "workspace must be non-null"),
    (linear(pack(X, 128, 65536), pack(W, 128, 65536), None, mat(Y, 128, 128), Z + 8, GB), "256-byte"),
    (linear(pack(X, 128, 65536), pack(W, 128, 65536), None, mat(Y, 128, 128), Z, 100), "workspace_capacity"),
    (linear(pack(X, 128, 65536), pack(W, 128, 65536), None, mat(Y, 128, 128), X, GB // 4), "workspace shares"),
    (linear(pack(1 << 40, 1 << 30, 16), pack(1 << 41, 1 << 30, 16), None, mat(1 << 50, 1 << 30, 1 << 30), Z, GB), "tiles"),
])
def test_linear_refuses(call, needle):
    refused(needle, *call)


@pytest.mark.parametrize("dy, q, dw, db, needle", [
    (mat(X, 8, 16, F32), pack(P, 8, 32), mat(Y, 16, 32), None, "dy must be ZERO_F16"),
    (mat(X, 9, 16), pack(P, 8, 32), mat(Y, 16, 32), None, "number of rows"),
    (mat(X, 8, 16), pack(P, 8, 32), mat(Y, 32, 16), None, "dw must be"),
    (mat(X, 8, 16), pack(P, 8, 32), mat(Y, 16, 32), mat(Z, 1, 32), "db must be"),
    (mat(X, 8, 16), pack(P, 8, 32), mat(X, 16, 32), None, "dw shares memory with dy"),
    (mat(X, 8, 16), pack(P, 8, 32), mat(P, 16, 32), None, "dw shares memory with the packed rows"),
    (mat(X, 8, 16), pack(P, 8, 32), mat(Y, 16, 32), mat(Y + 64, 1, 16), "dw shares memory with db"),
    (mat(X, 8, 16), pack(P, 8, 32), mat(Y, 16, 32), mat(X, 1, 16), "db shares memory with dy"),
    (mat(X, 8, 16), pack(P, 8, 32), mat(Y, 16, 32), mat(Z, 1, 16), "workspace must be non-null"),
    (None, pack(P, 8, 32), mat(Y, 16, 32), None, "null dy"), (mat(X, 8, 16), None, mat(Y, 16, 32), None, "null x"),
])
def test_weight_grad_refuses(dy, q, dw, db, needle):
    refused(needle, zpm.zero_packed_weight_grad, dy, q, dw, db, 0, None, 0)


@pytest.mark.parametrize("dy, q, dx, needle", [
    (mat(X, 8, 16, F32), pack(P, 16, 32), mat(Y, 8, 32), "dy must be ZERO_F16"),
    (mat(X, 8, 17), pack(P, 16, 32), mat(Y, 8, 32), "as many columns"),
    (mat(X, 8, 16), pack(P, 16, 32), mat(Y, 16, 32), "dx must be"),
    (mat(X, 8, 16), pack(P, 16, 32), mat(X + 16, 8, 32), "dx shares memory with dy"),
    (mat(X, 8, 16), pack(P, 16, 32), None, "null dx"), (mat(X, 8, 16), None, mat(Y, 8, 32), "null w"),
])
def test_input_grad_refuses(dy, q, dx, needle):
    refused(needle, zpm.zero_packed_input_grad, dy, q, dx, 0, None, 0)


@pytest.mark.parametrize("args, needle", [
    ((0, 0, mat(X, 8, 32), pack(P, 8, 32), mat(Y, 8, 32), None), "kind"),
    ((3, 0, mat(X, 8, 32), pack(P, 8, 32), mat(Y, 8, 32), None), "kind"),
    ((GELU, 0, mat(X, 8, 32), None, None, None), "no result"),
    ((GELU, 1, mat(X, 8, 33), pack(P, 8, 33), mat(Y, 8, 16), None), "even number"),
    ((SILU, 1, mat(X, 8, 32), pack(P, 8, 16), mat(Y, 8, 16), None), "xp must have"),
    ((SILU, 1, mat(X, 8, 32), pack(P, 8, 32), mat(Y, 8, 32), None), "y must be"),
    ((SILU, 0, mat(X, 8, 32), pack(P, 8, 32), None, pack(W, 8, 16)), "yp must be"),
    ((SILU, 0, mat(X, 8, 32), pack(P, 8, 32), mat(X, 8, 32), None), "y shares memory with x"),
    ((SILU, 0, mat(X, 8, 32), pack(P, 8, 32), None, pack(P + 64, 8, 32)), "yp shares memory with xp"),
    ((SILU, 0, mat(X, 8, 32), pack(P, 8, 32), mat(P + GB // 2, 8, 32), None), "y shares memory with xp's scales"),
])
def test_act_refuses(args, needle):
    refused(needle, zpm.zero_packed_act, *args)


@pytest.mark.parametrize("args, needle", [
    ((7, 0, pack(P, 8, 32), mat(X, 8, 32), mat(Y, 8, 32)), "kind"),
    ((GELU, 1, pack(P, 8, 31), mat(X, 8, 15), mat(Y, 8, 31)), "even number"),
    ((GELU, 1, pack(P, 8, 32), mat(X, 8, 32), mat(Y, 8, 32)), "dy must be"),
    ((GELU, 1, pack(P, 8, 32), mat(X, 8, 16), mat(Y, 8, 16)), "dx must have"),
    ((GELU, 0, pack(P, 8, 32), mat(X, 8, 32), mat(P, 8, 32)), "dx shares memory with xp"),
    ((GELU, 0, pack(P, 8, 32), mat(X, 8, 32), mat(X + 2, 8, 32)), "dx shares memory with dy"),
    ((GELU, 0, pack(P, 8, 32), mat(X, 8, 32), mat(X, 8, 32, F16)), "dx shares memory with dy"),
    ((GELU, 1, pack(P, 8, 32), mat(X, 8, 16, pitch=32), mat(X, 8, 32)), "dx shares memory with dy"),
])
def test_act_grad_refuses(args, needle):
    refused(needle, zpm.zero_packed_act_grad, *args)


def test_empty_calls_launch_nothing():
    none = mat(0, 0, 32)
    zpm.zero_packed_write(none, pack(0, 0, 32, scale=0), None)
    zpm.zero_packed_read(pack(0, 0, 32, scale=0), none, None)
    zpm.zero_packed_read(pack(0, 8, 0, scale=P), mat(0, 8, 0), None)
    zpm.zero_packed_linear(pack(0, 0, 32, scale=0), pack(W, 16, 32), None, mat(0, 0, 16), None, 0, None)
    zpm.zero_packed_input_grad(mat(0, 0, 16), pack(W, 16, 32), mat(0, 0, 32), 0, None, 0, None)
    zpm.zero_packed_weight_grad(mat(0, 8, 0), pack(W, 8, 32), mat(0, 0, 32), None, 0, None, 0, None)
    zpm.zero_packed_act(GELU, 0, none, pack(0, 0, 32, scale=0), none, None, None)
    zpm.zero_packed_act_grad(GELU, 0, pack(0, 0, 32, scale=0), none, none, None)


def test_workspace():
    ws = zpm.zero_packed_workspace
    assert ws(_abi.ZERO_PACKED_LINEAR, 16384, 4096, 11008) == 0          # tiles enough
    assert ws(_abi.ZERO_PACKED_LINEAR, 0, 4096, 11008) == 0
    few = ws(_abi.ZERO_PACKED_WEIGHT_GRAD, 65536, 64, 64)
    assert few >= 2 * 64 * 64 * 4 and few % 256 == 0
    assert ws(_abi.ZERO_PACKED_INPUT_GRAD, 8192, 4096, 4096) % 256 == 0
    for args in ((0, 1, 1, 1), (4, 1, 1, 1), (1, -1, 1, 1), (1, 1, (1 << 20) + 1, 1), (1, (1 << 30) + 1, 1, 1)):
        with pytest.raises(zpm.ZeroError):
            ws(*args)
    with pytest.raises(zpm.ZeroError):
        _abi._call("zero_packed_workspace", 1, 1, 1, 1, None)


def test_struct_layout():
    assert ctypes.sizeof(_abi.zero_matrix_t) == 40 and ctypes.sizeof(_abi.zero_packed_t) == 48


def test_matrix_descriptions():
    x = torch.zeros(6, 40, dtype=torch.bfloat16)
    d = matrix(x[1:4, 3:20], "x")
    assert (d.data, d.rows, d.cols, d.pitch, d.dtype) == (x.data_ptr() + 2 * 43, 3, 17, 40, BF16)
    d = matrix(x[0], "x")
    assert (d.rows, d.cols) == (1, 40)
    d = matrix(x[:, :1], "x")
    assert (d.rows, d.cols, d.pitch) == (6, 1, 40)
    assert matrix(x[:0], "x").rows == 0 and matrix(x[:, :0], "x").cols == 0
    for t in (x.t(), x[:, ::2], x[:1, ::2], x[0, ::2], x[0].expand(6, 40), x.view(2, 3, 40), x.to(torch.int8), x.double(),
              x.to_sparse(), torch._neg_view(x), 3, None):
        with pytest.raises(ValueError):
            matrix(t, "x")
    with pytest.raises(ValueError, match="packed rows are on"):
        matrix(x, "x", torch.device("cuda", 0))


def test_binding_refuses():
    with pytest.raises(ValueError, match="GPU"):
        ZeroPacked(4, 4, device="cpu")
    with pytest.raises(ValueError, match="negative"):
        ZeroPacked(-1, 4)
    q, s = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    for args in ((q.float(), s), (q[0], s), (q.t(), s), (q, s[:3]), (q, s.double()), (q, s.repeat(2)[::2]),
                 (q, s), (q, None)):
        with pytest.raises(ValueError):
            ZeroPacked.of(*args)


def test_lazily_negated_rows_refused():
    """Their memory holds the opposite of their values."""
    q, s = torch.ones(4, 32, dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError, match="negated"):
        ZeroPacked.of(torch._neg_view(q), s)
    with pytest.raises(ValueError, match="scale must be"):
        ZeroPacked.of(q, torch._neg_view(s))
