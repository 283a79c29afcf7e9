"""MXFP4 on the GPU at the ends of its ranges: what 16-bit activations keep of every value, up to the largest
bf16, and calls that the operators' other tests do not make."""
import numpy as np
import pytest
import torch

from oracle import mxfp4 as X
from tests.gpu_util import dev, dev_bf16
from tests.test_gpu_mxfp4 import FMTS, close, weight, x_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Q():
    from moe_hadamard128_act_b200 import build as qbuild
    qbuild.build()
    from moe_hadamard128_act_b200 import qlinear
    qlinear.lib()
    yield qlinear
    assert qlinear.ql_get_device_error() == (0, 0)


# ---- one value of x an output ----------------------------------------------------------------------------
def one_hot(Q, N, K, byte=126):
    """A packed weight with one code 1.0 a row, under scales 2^(byte - 127), and the column it is in."""
    at = np.arange(N) * 37 % K
    n = np.zeros((N, K), np.uint8)
    n[np.arange(N), at] = 2
    c, s, _ = Q.qlinear_pack(16, N, K, codes=dev(n), scales=dev(np.full((N, K // 32), byte, np.uint8)))
    return c, s, at


def spread_rows(M, K, seed, tops):
    """bf16 bits: each block of 32 holds one value of a magnitude in [2^t, 2^(t + 1)), t one of `tops`, and others
    1 to 24 powers of two below that, all with mantissas and signs of their own."""
    rng = np.random.default_rng(seed)
    t = np.repeat(rng.choice(tops, (M, K // 32)), 32, axis=1)
    below = rng.integers(1, 25, (M, K))
    first = rng.integers(0, 32, (M, K // 32)) + 32 * np.arange(K // 32)
    np.put_along_axis(below, first, 0, axis=1)
    field = t - below + 127
    assert field.min() > 0 and field.max() < 255
    return (rng.integers(0, 2, (M, K)) << 15 | field << 7 | rng.integers(0, 128, (M, K))).astype(np.uint16)


def kept(got, x, fmt, at, scale=0.5):
    """Each output is one value of x~: 16-bit activations exact from 2^-14 of the largest magnitude of the value's
    32 up and within 2^-22 of that largest below, 4-bit ones what their codes stand for."""
    v = X.activations(x, fmt, False)
    got = got.cpu().numpy().astype(np.float64) / scale
    if fmt == X.MXFP4A4_G32:
        assert np.array_equal(got, v[:, at])
        return
    top = np.repeat(np.abs(v).reshape(len(v), -1, 32).max(-1), 32, axis=1)
    off, exact = np.abs(got - v[:, at]), (np.abs(v) >= top * 2.0 ** -14)[:, at]
    assert exact.any() and not exact.all()
    assert not off[exact].any()
    assert (off <= 2.0 ** -22 * top[:, at]).all()


# rows as digits: tiles cut along K, one block, whole tiles, several blocks; as parts: pairs of CTAs, with halved tiles
SHAPES = [(1, 512, 512), (3, 640, 256), (24, 512, 384), (8, 9600, 384), (100, 512, 384), (150, 512, 384), (200, 512, 512),
          (40, 9600, 256), (64, 9400, 2048)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_every_value_of_x_is_kept(Q, fmt, M, N, K):
    c, s, at = one_hot(Q, N, K)
    x = spread_rows(M, K, M, [0, 3, -40, 90, -90, 126])
    kept(Q.qlinear_forward(dev_bf16(x), c, s, None, fmt, N), x, fmt, at)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_every_value_of_x_is_kept_up_to_the_largest(Q, fmt, M, N, K):
    c, s, at = one_hot(Q, N, K)
    x = spread_rows(M, K, M, [0, 126, 127])
    x[0, 5] = 0xFF7F  # the lowest bf16, as masks use it
    kept(Q.qlinear_forward(dev_bf16(x), c, s, None, fmt, N), x, fmt, at)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[1, 0, 5, 2], [60, 0, 30, 6], [200, 1, 40, 3]])  # digits (16-bit x), parts, parts
def test_every_value_of_x_is_kept_by_experts(Q, fmt, counts):
    N, K, E = 300, 384, len(counts)
    c, s, at = one_hot(Q, N, K)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(offsets[-1])
    x = spread_rows(R, K, R, [0, -60, 70, 127])
    kept(Q.qlinear_grouped(dev_bf16(x), dev(offsets), c.repeat(E), s.repeat(E), E, N, fmt), x, fmt, at)
    ids = np.repeat(np.arange(E, dtype=np.int32), counts)[:, None]
    kept(Q.moe_gate_up(dev_bf16(x), dev(ids), c.repeat(E), s.repeat(E), E, N, fmt=fmt, flags=0)[:, 0], x, fmt, at)


@pytest.mark.parametrize("M", [3, 200])
def test_blocks_of_small_magnitude_in_a_row_that_reaches_2_to_minus_64(Q, M):
    # As digits (3 rows) a block below 2^-105 beside a value of 2^-64 or more is held in multiples of 2^-127.  So it is as
    # parts (200 rows): the block's largest, 255 * 2^-113, lies in [2^-106, 2^-105), so hi has the scale 2^(-106 - 7) and
    # lo, E4M3 in steps of 2^-9 and 2^-5 below hi, steps of 2^-127.  The weight's scale keeps the outputs in fp32's
    # normal range.
    N = K = 256
    c, s, at = one_hot(Q, N, K, 127 + 60)
    x = np.zeros((M, K), np.uint16)
    x[:, 0] = 63 << 7  # 2^-64
    x[:, 32:38] = [1, 2, 0x40, 0x7F, 7 << 7 | 0x35, 0x8000 | 21 << 7 | 0x7F]  # 2^-133 .. -255 * 2^-113
    v = X.bf16_values(x).astype(np.float64)
    got = Q.qlinear_forward(dev_bf16(x), c, s, None, 16, N).cpu().numpy().astype(np.float64) * 2.0 ** -60
    v[:, 32:64] = np.rint(v[:, 32:64] * 2.0 ** 127) * 2.0 ** -127
    assert np.array_equal(got, v[:, at])


# ---- segments of experts beside a bad one -------------------------------------------------------------------
def bad_offsets():
    yield [0, 10, 20, -1, 40], 40
    yield [0, 10, -3, 30, 40], 40
    yield [0, 10, 1 << 30, 20, 40], 40
    for bad in (-5, 1 << 20, 0):  # among many experts, where the search for a row's expert takes strides
        for e in (4, 48, 50, 99):
            offsets = [3 * i for i in range(101)]
            offsets[e] = bad
            yield offsets, 300


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offsets,R", list(bad_offsets()))
def test_grouped_sound_segments_beside_bad_offsets(Q, fmt, offsets, R):
    E, N, K = len(offsets) - 1, 130, 256
    x = x_bits(R, K, seed=3)
    c, s, W = weight(Q, N, K, seed=1)
    y = torch.full((R, N), 7.0, device="cuda")
    ws = torch.full((Q.qlinear_grouped_workspace_size(E, N, K, fmt, 0, R),), 0x7F, dtype=torch.uint8, device="cuda")
    Q.qlinear_grouped(dev_bf16(x), dev(np.array(offsets, np.int32)), c.repeat(E), s.repeat(E), E, N, fmt, y=y, ws=ws)
    assert Q.ql_get_device_error() == (6, Q.DEVERR_BOUNDS)
    got = y.cpu().numpy().astype(np.float64)
    claims = np.zeros(R, int)
    for a, b in zip(offsets, offsets[1:]):
        if 0 <= a <= b <= R:
            claims[a:b] += 1
    ref, bound = X.forward(x, W, fmt)
    one = claims == 1
    close(got[one], ref[one], bound[one])
    assert (got[claims == 0] == 7.0).all()


# ---- waits that run out -------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("limit", [1, 1500, 6000])
def test_pairs_that_gave_up_leave_nothing_behind(Q, fmt, limit):
    # pairs of CTAs give up at once or some way into the product (or, with the longest bound, perhaps not at all); the
    # calls that follow on the same SMs are right
    M, N, K = 200, 5000, 2176
    x = x_bits(M, K, seed=9)
    c, s, W = weight(Q, N, K)
    xd, ref = dev_bf16(x), X.forward(x, W, fmt)
    few = X.forward(x[:3], W, fmt)
    close(Q.qlinear_forward(xd, c, s, None, fmt, N), *ref)
    for _ in range(3):
        Q.ql_set_wait_limit(limit)
        try:
            Q.qlinear_forward(xd, c, s, None, fmt, N)
        finally:
            Q.ql_set_wait_limit(0)
        y = [Q.qlinear_forward(xd, c, s, None, fmt, N), Q.qlinear_forward(xd[:3], c, s, None, fmt, N)]
        status = Q.ql_get_device_error()
        assert status in ((6, Q.DEVERR_TIMEOUT), (0, 0)) and (limit > 1 or status[0] == 6)
        close(y[0], *ref)
        close(y[1], *few)


# ---- streams ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
def test_results_of_a_side_stream_outlive_what_the_current_stream_does_with_them(Q, fmt):
    # the current stream reads a result late; later calls on the side stream, which wait for nothing, take other memory
    N, K, M = 300, 512, 40
    c, s, W = weight(Q, N, K)
    inputs = [x_bits(M, K, seed=20 + i) for i in range(4)]
    xs = [dev_bf16(x) for x in inputs]
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    read = []
    for xd in xs:
        y = Q.qlinear_forward(xd, c, s, None, fmt, N, stream=side)
        codes, scales = Q.act_quant_mxfp4(xd, stream=side)
        main.wait_stream(side)
        torch.cuda._sleep(5_000_000)
        read.append((y.clone(), codes.clone(), scales.clone()))
        del y, codes, scales
    torch.cuda.synchronize()
    for x, xd, (y, codes, scales) in zip(inputs, xs, read):
        close(y, *X.forward(x, W, fmt))
        again = Q.act_quant_mxfp4(xd)
        assert torch.equal(codes, again[0]) and torch.equal(scales, again[1])
