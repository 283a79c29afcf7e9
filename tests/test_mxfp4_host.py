"""MXFP4 without a GPU: the oracle's own pins, the packed sizes, and the statuses of calls that are refused
before anything is launched."""
import ctypes
import re
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest

from moe_hadamard128_act_b200 import build as qbuild
from oracle import mxfp4 as X

ROOT = Path(__file__).resolve().parents[1]
A = 1 << 20  # an aligned address that no call below reads
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def Q():
    qbuild.build()
    from moe_hadamard128_act_b200 import qlinear
    qlinear.lib()
    return qlinear


# ---- the oracle ----------------------------------------------------------------------------------------
def test_oracle_codes_are_e2m1():
    for c in range(16):
        s, e, m = c >> 3, (c >> 1) & 3, c & 1
        v = m * 0.5 if e == 0 else (1 + m * 0.5) * 2.0 ** (e - 1)
        assert X.CODE_VALUES[c] == (-v if s else v)


def test_oracle_rounds_to_nearest_ties_to_even_and_saturates():
    v = np.zeros((1, 32), np.float32)
    v[0, :16] = [7.9, 0.25, 0.2500001, 0.75, 0.7499999, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0000005, 6.5, -0.75, -2.5, -0.1, 0.0]
    n, b = X.quantise(v)
    assert b[0, 0] == 127  # floor(log2 7.9) - 2 = 0
    assert X.CODE_VALUES[n[0, :16]].tolist() == [6, 0, 0.5, 1, 0.5, 1, 2, 2, 4, 4, 6, 6, -1, -2, 0, 0]
    assert n[0, 14] == 8  # the sign of a zero is kept


@pytest.mark.parametrize("power", [-149, -133, -126, -125, -124, -3, 0, 100, 127])
def test_oracle_scale_of_a_power_of_two(power):
    v = np.zeros((1, 32), np.float32)
    v[0, 3] = np.ldexp(np.float32(1), power)
    n, b = X.quantise(v)
    assert b[0, 0] == max(power - 2, -127) + 127
    # exact while it is a multiple of the smallest step, half of 2^-127: a power above -128, or rounded to zero
    assert X.values(n, b)[0, 3] == (float(v[0, 3]) if power > -129 else 0.0)


def test_oracle_zero_and_nonfinite_blocks():
    v = np.ones((1, 128), np.float32)
    v[0, :32] = 0
    v[0, 40], v[0, 70], v[0, 100] = np.inf, np.nan, -np.inf
    n, b = X.quantise(v)
    assert b[0].tolist() == [0, 255, 255, 255] and not n[0].any()


def test_oracle_layout_round_trip():
    rng = np.random.default_rng(0)
    n, b = rng.integers(0, 16, (200, 384), dtype=np.uint8), rng.integers(0, 256, (200, 12), dtype=np.uint8)
    codes, scales = X.pack(n, b)
    assert codes.size == X.packed_sizes(200, 384)[0] and scales.size == X.packed_sizes(200, 384)[1]
    assert np.array_equal(codes & 15, n[:, 0::2]) and np.array_equal(codes >> 4, n[:, 1::2])
    back = scales.transpose(0, 3, 2, 1, 4).reshape(256, 12)
    assert np.array_equal(back[:200], b) and not back[200:].any()


# ---- the library -----------------------------------------------------------------------------------------
def test_constants_match_header(Q):
    text = (ROOT / "include" / "qlinear.h").read_text()
    for name in ("MXFP4_G32", "MXFP4A4_G32"):
        assert int(re.search(rf"QL_{name}\s*=\s*(\d+)", text).group(1)) == getattr(Q, name) == getattr(X, name)
        assert getattr(Q, name) in Q.FORMATS


@pytest.mark.parametrize("fmt", [16, 17])
@pytest.mark.parametrize("N,K", [(1, 128), (128, 128), (129, 256), (21504, 5376)])
def test_packed_sizes(Q, fmt, N, K):
    assert Q.qlinear_packed_sizes(fmt, N, K) == X.packed_sizes(N, K)


def test_sizes_refuse_bad_arguments(Q):
    for fmt, N, K in ((15, 8, 128), (18, 8, 128), (16, 0, 128), (17, 8, 64), (16, 8, 200)):
        with pytest.raises(Q.QLError) as e:
            Q.qlinear_packed_sizes(fmt, N, K)
        assert e.value.status == 1
    with pytest.raises(Q.QLError):
        Q.qlinear_workspace_size(16, 4, 1, 8, 128)
    for fmt, per in ((16, 2 * 5376), (17, 5376 // 2)):  # the parts or codes of 300 rows and their scales
        assert Q.qlinear_workspace_size(fmt, 0, 300, 64, 5376) >= 300 * (per + 5376 // 32)
    assert Q.qlinear_grouped_workspace_size(8, 64, 256, 17, 0, 100) >= 100 * (128 + 8)
    with pytest.raises(Q.QLError) as e:
        Q.qlinear_grouped_workspace_size(8, 64, 256, 1, 0, 100)  # int8 experts go by moe_gate_up
    assert e.value.status == 2


def test_forward_statuses(Q):
    f = Q.lib().qlinear_forward

    def call(x=P(A), W=P(A), s=P(A), fmt=16, flags=0, M=4, N=64, K=256, y=P(A), ws=P(A), wsb=1 << 30):
        return f(x, W, s, None, fmt, flags, M, N, K, y, ws, wsb, None)

    for fmt in (16, 17):
        assert call(fmt=fmt, K=200) == 1
        assert call(fmt=fmt, M=0) == 1
        assert call(fmt=fmt, flags=4) == 1
        assert call(fmt=fmt, x=None) == 1
        assert call(fmt=fmt, s=None) == 1
        assert call(fmt=fmt, x=P(A + 8)) == 3
        assert call(fmt=fmt, W=P(A + 16)) == 3  # codes: 32 bytes
        assert call(fmt=fmt, s=P(A + 8)) == 3
        assert call(fmt=fmt, y=P(A + 4)) == 3
        assert call(fmt=fmt, ws=None) == 4
        assert call(fmt=fmt, wsb=16) == 4
        assert call(fmt=fmt, ws=P(A + 8)) == 3
        assert call(fmt=fmt, K=32768 + 128, wsb=16) == 4  # no limit on K
        assert call(fmt=fmt, M=(1 << 30) + 1) == 2 and call(fmt=fmt, N=(1 << 30) + 1) == 2
    assert call(fmt=15) == 1 and call(fmt=18) == 1


def test_pack_quantise_and_dequant_statuses(Q):
    L = Q.lib()
    p = L.qlinear_pack
    for fmt in (16, 17):
        assert p(P(A), P(A), P(A), None, fmt, 0, 8, 128, P(A), P(A), None, None) == 1  # two sources
        assert p(None, P(A), None, None, fmt, 0, 8, 128, P(A), P(A), None, None) == 1  # codes without scales
        assert p(P(A + 4), None, None, None, fmt, 0, 8, 128, P(A), P(A), None, None) == 3
        assert p(P(A), None, None, None, fmt, 2, 8, 128, P(A), P(A), None, None) == 2  # the search is for int8
    q = L.act_quant_mxfp4
    assert q(P(A), 4, 100, 0, P(A), P(A), None) == 1
    assert q(P(A), 0, 128, 0, P(A), P(A), None) == 1
    assert q(P(A), 4, 128, 0, None, P(A), None) == 1
    assert q(P(A), 4, 128, 0, P(A), P(A + 4), None) == 3
    d = L.mxfp4_dequant
    assert d(P(A), P(A), 4, 64, P(A), None) == 1
    assert d(P(A), None, 4, 128, P(A), None) == 1
    assert d(P(A), P(A), 4, 128, P(A + 2), None) == 3
    many = Q.MXFP4_MAX_ROWS + 1
    assert many == (1 << 30) + 1
    assert d(P(A), P(A), many, 128, P(A), None) == 2 and q(P(A), many, 128, 0, P(A), P(A), None) == 2
    assert p(P(A), None, None, None, 16, 0, many, 128, P(A), P(A), None, None) == 2
    assert L.qlinear_gemm_a8(P(A), P(A), P(A), P(A), 17, 4, 64, 256, P(A), 0, None) == 1  # int8 and E4M3 only


def test_grouped_and_gate_up_statuses(Q):
    L = Q.lib()

    def grouped(x=P(A), off=P(A), ex=None, R=4, y=P(A), ws=P(A), wsb=1 << 30, **kw):
        a = dict(E=8, N=64, K=256, fmt=17, flags=0, codes=A, scales=A)
        a.update(kw)
        ex = Q.ql_experts(*a.values())
        return L.qlinear_grouped(x, off, ctypes.byref(ex), R, y, ws, wsb, None)

    assert L.qlinear_grouped(P(A), P(A), None, 4, P(A), P(A), 1 << 30, None) == 1
    assert grouped(R=0) == 1
    assert grouped(E=0) == 1 and grouped(E=1025) == 1
    assert grouped(K=200) == 1
    assert grouped(flags=4) == 1
    assert grouped(x=None) == 1 and grouped(off=None) == 1 and grouped(y=None) == 1 and grouped(codes=0) == 1
    assert grouped(R=(1 << 30) + 1) == 2 and grouped(E=1024, N=(1 << 20) + 1) == 2
    assert grouped(fmt=1) == 2 and grouped(fmt=7) == 2 and grouped(fmt=4) == 2
    assert grouped(codes=A + 16) == 3 and grouped(scales=A + 8) == 3
    assert grouped(off=P(A + 4)) == 3 and grouped(x=P(A + 2)) == 3 and grouped(y=P(A + 4)) == 3
    assert grouped(ws=None) == 4 and grouped(wsb=16) == 4 and grouped(ws=P(A + 8)) == 3
    ex = Q.ql_experts(8, 64, 256, 16, 1, A, A)
    g = L.moe_gate_up
    assert g(P(A), P(A), None, ctypes.byref(ex), 4, 65, P(A), P(A), 1 << 30, None) == 1
    assert g(P(A), P(A), None, ctypes.byref(ex), 4, 8, P(A), None, 0, None) == 4
    assert g(P(A), P(A), None, ctypes.byref(ex), 4, 8, P(A), P(A), 64, None) == 4
    bad = Q.ql_experts(8, 64, 256, 16, 0, A + 16, A)
    assert g(P(A), P(A), None, ctypes.byref(bad), 4, 8, P(A), P(A), 1 << 30, None) == 3
    assert Q.moe_workspace_size(8, 64, 256, 16, 0, 100, 2) >= 200 * (2 * 256 + 8 + 4)


def test_binding_refuses_wrong_tensors(Q):
    import torch
    x = torch.zeros(4, 128, dtype=torch.float16)
    u8 = torch.zeros(64, dtype=torch.uint8)
    for call in (lambda: Q.act_quant_mxfp4(x),
                 lambda: Q.mxfp4_dequant(u8, u8, 4, 128),
                 lambda: Q.qlinear_grouped(x, u8, u8, u8, 2, 64),
                 lambda: Q.qlinear_grouped(x.to(torch.bfloat16), torch.zeros(3), u8, u8, 2, 64),
                 lambda: Q.qlinear_grouped(x.to(torch.bfloat16), torch.zeros(3, dtype=torch.int32), u8, u8, 2, 64)):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_tensors_of_other_sizes(Q):
    import torch
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    c, sc = torch.zeros(64 * 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    y = torch.zeros(4, 63)
    for fmt in (Q.MXFP4_G32, Q.MXFP4A4_G32):
        for call in (lambda: Q.qlinear_forward(x, c[:-1], sc, None, fmt, 64),
                     lambda: Q.qlinear_forward(x, c, sc[:-1], None, fmt, 64),
                     lambda: Q.qlinear_forward(x, c, sc, None, fmt, 64, y=y),
                     lambda: Q.moe_gate_up(x, ids, c, sc, 2, 64, fmt=fmt),
                     lambda: Q.moe_gate_up(x, ids.long(), c, sc, 1, 64, fmt=fmt),
                     lambda: Q.moe_gate_up(x, ids[:3], c, sc, 1, 64, fmt=fmt),
                     lambda: Q.moe_gate_up(x.float(), ids, c, sc, 1, 64, fmt=fmt),
                     lambda: Q.moe_gate_up(x, ids, c, sc, 1, 64, fmt=fmt, y=y),
                     lambda: Q.qlinear_pack(fmt, 64, 128, W=torch.zeros(64, 128, dtype=torch.float16)),
                     lambda: Q.qlinear_pack(fmt, 64, 128, codes=torch.zeros(64 * 128 - 1, dtype=torch.uint8), scales=sc),
                     lambda: Q.qlinear_pack(fmt, 64, 128, codes=torch.zeros(64 * 128, dtype=torch.uint8), scales=sc)):
            with pytest.raises(ValueError, match="take|must be"):
                call()


def test_binding_refuses_stacked_weights_that_are_not_contiguous(Q):
    import torch
    E, N, K = 2, 128, 256
    x, ids = torch.zeros(4, K, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32)
    c, sc = torch.zeros(E, N * K // 2, dtype=torch.uint8), torch.zeros(E, 1024, dtype=torch.uint8)
    for fmt in (Q.MXFP4_G32, Q.MXFP4A4_G32):
        for codes, scales in ((c.t(), sc), (c, sc.t()), (c.repeat(1, 2)[:, ::2], sc), (c, sc[:1].expand(E, -1))):
            for call in (lambda: Q.qlinear_grouped(x, off, codes, scales, E, N, fmt),
                         lambda: Q.moe_gate_up(x, ids, codes, scales, E, N, fmt=fmt)):
                with pytest.raises(ValueError, match="contiguous"):
                    call()


def test_binding_refuses_tensors_of_two_devices(Q, monkeypatch):
    import torch
    E, N, K = 2, 128, 256

    def on(device, *size, dtype=torch.uint8):
        t = torch.zeros(*size, dtype=dtype)
        places[id(t)] = device
        kept.append(t)
        return t

    places, kept = {}, []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: places[id(t)])
    x, ids = on(0, 4, K, dtype=torch.bfloat16), on(0, 4, 2, dtype=torch.int32)
    off, y = on(0, E + 1, dtype=torch.int32), on(0, 4, N, dtype=torch.float32)
    c, sc, ws = on(0, E, N * K // 2), on(0, E, 1024), on(0, 1 << 20)
    c1, sc1, out = on(0, N * K // 2), on(0, 1024), on(0, N, K, dtype=torch.bfloat16)
    n, b = on(0, N, K), on(0, N, K // 32)
    for fmt in (Q.MXFP4_G32, Q.MXFP4A4_G32):
        for call, tensors in ((lambda: Q.qlinear_grouped(x, off, c, sc, E, N, fmt, y=y, ws=ws), (off, c, sc, y, ws)),
                              (lambda: Q.moe_gate_up(x, ids, c, sc, E, N, fmt=fmt, ws=ws), (ids, c, sc, ws)),
                              (lambda: Q.qlinear_forward(x, c1, sc1, None, fmt, N, y=y, ws=ws), (c1, sc1, y, ws)),
                              (lambda: Q.mxfp4_dequant(c1, sc1, N, K, out), (sc1, out)),
                              (lambda: Q.qlinear_pack(fmt, N, K, codes=n, scales=b), (b,))):
            for t in tensors:
                places[id(t)] = 1
                with pytest.raises(ValueError, match="the same device"):
                    call()
                places[id(t)] = 0


def test_binding_imports_beside_a_torch_without_cuda(Q):
    # such a torch lacks the CUDA parts of torch._C: names, constants and sizes are there all the same
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from moe_hadamard128_act_b200 import qlinear as Q
assert Q.qlinear_packed_sizes(Q.MXFP4_G32, 128, 256) == (128 * 128, 1024, 0)
assert Q.qlinear_workspace_size(Q.MXFP4A4_G32, 0, 1, 128, 256) > 0
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=300)
