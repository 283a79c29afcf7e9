"""MXFP4 on the GPU against the fp64 oracle: quantisers and packers bit for bit, the products within the bound
that the oracle derives for fp32 sums, over one weight and over rows grouped by expert."""
import numpy as np
import pytest
import torch

from moe_hadamard128_act_b200 import synth
from oracle import mxfp4 as X
from oracle import oracle as O
from tests.gpu_util import dev, dev_bf16, host_u16, host_u8

pytestmark = pytest.mark.gpu
FMTS = (X.MXFP4_G32, X.MXFP4A4_G32)


@pytest.fixture(scope="module")
def Q():
    from moe_hadamard128_act_b200 import build as qbuild
    qbuild.build()
    from moe_hadamard128_act_b200 import qlinear
    qlinear.lib()
    yield qlinear
    assert qlinear.ql_get_device_error() == (0, 0)


def x_bits(M, K, seed=0, outliers=0.01):
    return synth.activations(seed, f"mx{M}x{K}", M, K, outlier_frac=outliers)


def weight(Q, N, K, seed=0, fmt=16):
    """A packed Gaussian weight on the device and its values in fp64."""
    n, b = X.quantise(synth.weight_rows(seed, f"mxw{N}x{K}", K, 0, N))
    c, s, _ = Q.qlinear_pack(fmt, N, K, codes=dev(n), scales=dev(b))
    return c, s, X.values(n, b)


def close(got, ref, bound, what=""):
    got = got.cpu().numpy().astype(np.float64) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    fine = np.isfinite(ref)
    off = np.abs(got - ref)[fine] - bound[fine]
    assert off.size == 0 or off.max() <= 0, f"{what}: {off.max():.3e} past the bound at {np.argmax(off)}"


# ---- quantisers ----------------------------------------------------------------------------------------
def special_rows(K):
    """Rows with zeros, ties, subnormals, the largest values, infinities and NaN."""
    v = np.zeros((6, K), np.float64)
    v[1, :10] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, -0.125]
    v[2, :4] = [2.0 ** -133, -(2.0 ** -130), 2.0 ** -127, 0.0]
    v[3, :4] = [3.3895313892515355e38, -1.0, 2.0 ** 126, -(2.0 ** 124)]
    bits = O.bf16_encode(v.ravel()).reshape(v.shape)
    bits[4, :2] = [0x7F80, 0x3F80]  # infinity
    bits[4, K - 1] = 0xFF80
    bits[5, 33 % K] = 0x7FC0  # NaN
    return bits


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("M,K", [(1, 128), (3, 384), (16, 5376), (129, 256), (300, 1152)])
def test_act_quant_bitexact(Q, M, K, rotate):
    x = x_bits(M, K)
    n, b = X.quantise(X.bf16_values(x), rotate)
    c_ref, s_ref = X.pack(n, b)
    c, s = Q.act_quant_mxfp4(dev_bf16(x), rotate)
    assert np.array_equal(host_u8(c), c_ref.ravel()) and np.array_equal(host_u8(s), s_ref.ravel())


@pytest.mark.parametrize("K", [128, 640])
def test_act_quant_special_values(Q, K):
    x = special_rows(K)
    c_ref, s_ref = X.pack(*X.quantise(X.bf16_values(x)))
    c, s = Q.act_quant_mxfp4(dev_bf16(x))
    assert np.array_equal(host_u8(c), c_ref.ravel()) and np.array_equal(host_u8(s), s_ref.ravel())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("had", [0, 1])
@pytest.mark.parametrize("N,K", [(1, 128), (130, 384), (256, 1024)])
def test_pack_weight_bitexact(Q, fmt, had, N, K):
    W = synth.weight_rows(3, f"mxp{N}", K, 0, N)
    W[0, :64] = 0.0
    if not had:
        W[0, 64:70] = [3e38, -1e-44, 1e-38, np.inf, 1.0, 2.0]
        W[0, 96:99] = [1e-40, -3e-39, 5e-45]
    c_ref, s_ref = X.pack(*X.quantise(W, bool(had)))
    c, s, z = Q.qlinear_pack(fmt, N, K, W=dev(W), flags=had)
    assert z is None
    assert np.array_equal(host_u8(c), c_ref.ravel()) and np.array_equal(host_u8(s), s_ref.ravel())


def test_pack_given_codes(Q):
    rng = np.random.default_rng(1)
    N, K = 150, 640
    n, b = rng.integers(0, 16, (N, K), dtype=np.uint8), rng.integers(0, 256, (N, K // 32), dtype=np.uint8)
    c_ref, s_ref = X.pack(n, b)
    c, s, _ = Q.qlinear_pack(16, N, K, codes=dev(n), scales=dev(b))
    assert np.array_equal(host_u8(c), c_ref.ravel()) and np.array_equal(host_u8(s), s_ref.ravel())
    n[7, 9] = 16  # packed as 0 and flagged
    c, _, _ = Q.qlinear_pack(16, N, K, codes=dev(n), scales=dev(b))
    assert Q.ql_get_device_error() == (6, Q.DEVERR_CODE_RANGE)
    n[7, 9] = 0
    assert np.array_equal(host_u8(c), X.pack(n, b)[0].ravel())


def test_dequant_every_code_and_scale(Q):
    N, K = 256, 1024  # row r: every block has scale byte r, every code twice a block
    n = np.tile(np.arange(16, dtype=np.uint8), (N, K // 16))
    b = np.repeat(np.arange(256, dtype=np.uint8)[:, None], K // 32, 1)
    c, s, _ = Q.qlinear_pack(17, N, K, codes=dev(n), scales=dev(b))
    got = Q.mxfp4_dequant(c, s, N, K).float().cpu().numpy()
    with np.errstate(over="ignore"):
        ref = X.values(n, b).astype(np.float32)  # 4 * 2^127 and more: infinite
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[:255], ref[:255])
    assert np.array_equal(np.signbit(got[:255]), np.signbit(ref[:255]))


# ---- one weight ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,had", [
    (1, 64, 128, 0), (1, 1000, 5376, 0), (2, 1, 256, 1), (3, 129, 384, 0), (4, 4096, 1152, 1), (15, 128, 640, 0),
    (16, 2048, 5376, 1), (17, 333, 256, 0), (33, 200, 1024, 0), (64, 300, 384, 1), (65, 127, 512, 0),
    (130, 384, 896, 0), (193, 500, 128, 0), (300, 1000, 640, 1), (511, 257, 384, 0), (1290, 640, 256, 0),
    (2, 19000, 256, 0), (40, 130, 8192, 0), (24, 200, 256, 1), (25, 200, 256, 0), (63, 300, 384, 0), (64, 300, 384, 0),
    (192, 130, 256, 0), (256, 300, 512, 0), (257, 300, 384, 0), (5, 9473, 128, 0), (70, 9473, 128, 1), (1, 128, 33280, 0)])
def test_forward(Q, fmt, M, N, K, had):
    x = x_bits(M, K)
    c, s, W = weight(Q, N, K)
    y = Q.qlinear_forward(dev_bf16(x), c, s, None, fmt, N, flags=had)
    ref, bound = X.forward(x, W, fmt, bool(had))
    close(y, ref, bound)
    again = Q.qlinear_forward(dev_bf16(x), c, s, None, fmt, N, flags=had)
    assert torch.equal(y, again)  # the sums are bit-reproducible


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [5, 40, 200])
def test_forward_nonfinite_stays_in_its_row_and_column(Q, fmt, M):
    N, K = 300, 512
    x = x_bits(M, K)
    x[2, 100], x[4, 511] = 0x7FC0, 0xFF80
    x[3] = 0
    n, b = X.quantise(synth.weight_rows(2, "mxnan", K, 0, N))
    b[7, 5] = 255
    b[8, :] = 0  # the smallest scales
    c, s, _ = Q.qlinear_pack(fmt, N, K, codes=dev(n), scales=dev(b))
    y = Q.qlinear_forward(dev_bf16(x), c, s, None, fmt, N).cpu().numpy()
    ref, bound = X.forward(x, X.values(n, b), fmt)
    assert np.isnan(ref[2]).all() and np.isnan(ref[4]).all() and np.isnan(ref[:, 7]).all()
    assert np.isnan(ref).sum() == 2 * N + M - 2
    # fp32 atomic adds flush numbers below 2^-126: two partial sums of an output and their sum
    close(y.astype(np.float64), ref, bound + 3 * 2.0 ** -126)
    assert not y[3, [0, 1, 299]].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_forward_far_exponents(Q, fmt):
    # tiny activations times huge weights and the other way round: the products are ordinary numbers
    N, K = 256, 256
    rng = np.random.default_rng(5)
    n = rng.integers(0, 16, (N, K), dtype=np.uint8)
    for xe, we in ((-120, 115), (110, -112), (-133, 126)):
        x = O.bf16_encode((np.ldexp(rng.standard_normal((20, K)), xe)).ravel()).reshape(20, K)
        b = np.full((N, K // 32), 127 + we, np.uint8)
        c, s, _ = Q.qlinear_pack(fmt, N, K, codes=dev(n), scales=dev(b))
        y = Q.qlinear_forward(dev_bf16(x), c, s, None, fmt, N)
        ref, bound = X.forward(x, X.values(n, b), fmt)
        # a block at the least exponent has steps of 2^-127 halves: what the format keeps of x is in ref already
        # for 4-bit activations; the 16-bit parts' steps of 2^-136 hold every bf16 value
        close(y, ref, bound)


@pytest.mark.parametrize("fmt", FMTS)
def test_forward_exact_small_integers(Q, fmt):
    # codes of x and W are small integers under scale 1: every sum is exact in fp32
    rng = np.random.default_rng(9)
    M, N, K = 50, 200, 768
    xi = rng.choice([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], (M, K)).astype(np.float64)
    xi[:, ::32] = 4.0  # every block's scale is 1
    x = O.bf16_encode(xi.ravel()).reshape(M, K)
    n = rng.integers(0, 16, (N, K), dtype=np.uint8)
    b = np.full((N, K // 32), 127, np.uint8)
    c, s, _ = Q.qlinear_pack(fmt, N, K, codes=dev(n), scales=dev(b))
    y = Q.qlinear_forward(dev_bf16(x), c, s, None, fmt, N).cpu().numpy()
    assert np.array_equal(y.astype(np.float64), xi @ X.values(n, b).T)


# ---- grouped by expert -----------------------------------------------------------------------------------
COUNTS = [
    [1], [0, 3, 0, 0, 17, 1, 0, 64], [5] * 7, [0, 0, 0], [200, 1, 0, 33], [16, 32, 48, 64, 80, 96, 112, 128, 144],
    [1] * 40, [0] * 100 + [2] + [0] * 20, [513, 0, 2], [15, 17, 31, 33, 63, 65, 127, 129, 191, 193],
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K,had", [(200, 384, 1), (128, 256, 0)])
@pytest.mark.parametrize("counts", COUNTS, ids=[f"c{i}" for i in range(len(COUNTS))])
def test_grouped(Q, fmt, N, K, had, counts):
    E, lead, tail = len(counts), 3, 5
    offsets = lead + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(offsets[-1]) + tail
    x = x_bits(R, K, seed=1)
    x[:lead], x[R - tail:] = 0x7FC0, 0x7FC0  # rows of no expert are not read
    packed = [weight(Q, N, K, seed=e) for e in range(min(E, 6))]
    c, s = (torch.cat([packed[e % 6][i] for e in range(E)]) for i in (0, 1))
    y = torch.full((R, N), 7.0, device="cuda")
    ws = torch.full((Q.qlinear_grouped_workspace_size(E, N, K, fmt, had, R),), 0xFF, dtype=torch.uint8, device="cuda")
    off = torch.zeros(E + 4, dtype=torch.int32, device="cuda")
    off[:E + 1] = dev(offsets)
    Q.qlinear_grouped(dev_bf16(x), off[:E + 1], c, s, E, N, fmt, had, y=y, ws=ws)
    got = y.cpu().numpy()
    assert (got[:lead] == 7.0).all() and (got[R - tail:] == 7.0).all()  # left as they were
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        ref, bound = X.forward(x[a:b], packed[e % 6][2], fmt, bool(had))
        close(got[a:b].astype(np.float64), ref, bound, f"expert {e}")


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_flags_offsets_out_of_order(Q, fmt):
    E, N, K, R = 4, 130, 256, 40
    x = x_bits(R, K, seed=2)
    c, s, W = weight(Q, N, K, seed=1)
    for offsets in ([0, 10, 5, 20, 40], [0, 10, 20, 30, 41], [-3, 10, 20, 30, 40]):
        y = torch.full((R, N), 7.0, device="cuda")
        Q.qlinear_grouped(dev_bf16(x), dev(np.array(offsets, np.int32)), c.repeat(E), s.repeat(E), E, N, fmt, y=y)
        assert Q.ql_get_device_error() == (6, Q.DEVERR_BOUNDS)
        got = y.cpu().numpy()
        ref, bound = X.forward(x, W, fmt)
        sound = [e for e in range(E) if 0 <= offsets[e] <= offsets[e + 1] <= R]
        rows = [r for e in sound for r in range(offsets[e], offsets[e + 1])]
        if offsets[2] != 5:  # segments that do not overlap
            close(got[rows].astype(np.float64), ref[rows], bound[rows])
            left = [r for r in range(R) if r not in rows]
            assert (got[left] == 7.0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,topk,E,N,K,had", [(1, 8, 128, 200, 256, 1), (3, 2, 5, 130, 384, 0), (16, 8, 128, 256, 256, 1),
                                              (70, 4, 6, 128, 640, 0), (300, 8, 16, 200, 128, 1)])
def test_gate_up(Q, fmt, T, topk, E, N, K, had):
    ids, _ = synth.routing(T, T, E, topk)
    ids = ids.copy()
    if T == 3:
        ids[1, 0], ids[2, 1] = -1, E  # of no expert: zero rows, flagged
    if T == 70:
        ids[:] = 2  # every pair the same expert
    x = x_bits(T, K, seed=3)
    packed = [weight(Q, N, K, seed=e) for e in range(min(E, 5))]
    c, s = (torch.cat([packed[e % 5][i] for e in range(E)]) for i in (0, 1))
    y = torch.full((T, topk, N), float("nan"), device="cuda")
    Q.moe_gate_up(dev_bf16(x), dev(ids), c, s, E, N, fmt=fmt, flags=had, y=y)
    got = y.cpu().numpy().astype(np.float64)
    for e in range(-1, E + 1):
        t, j = np.nonzero(ids == e)
        if 0 <= e < E:
            ref, bound = X.forward(x[t], packed[e % 5][2], fmt, bool(had))
            close(got[t, j], ref, bound, f"expert {e}")
        else:
            assert not got[t, j].any()
    if T == 3:
        assert Q.ql_get_device_error() == (6, Q.DEVERR_EXPERT_ID)


@pytest.mark.parametrize("T,topk,E", [(16, 8, 3), (43, 3, 130), (2, 64, 100), (128, 1, 1024), (700, 4, 37), (513, 1, 9)])
def test_gate_up_at_the_limit_of_fused_routing(Q, T, topk, E):
    # 128 and 129 pairs; ids at random, so that a token may name an expert twice, some of no expert
    N, K, fmt = 130, 256, 16
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E + 1, (T, topk)).astype(np.int32)
    x = x_bits(T, K, seed=5)
    c, s, W = weight(Q, N, K, seed=2)
    c2, s2, W2 = weight(Q, N, K, seed=3)
    codes, scales = torch.cat([c, c2] * E)[: E * c.numel()], torch.cat([s, s2] * E)[: E * s.numel()]
    y = torch.full((T, topk, N), float("nan"), device="cuda")
    Q.moe_gate_up(dev_bf16(x), dev(ids), codes.contiguous(), scales.contiguous(), E, N, fmt=fmt, flags=0, y=y)
    assert Q.ql_get_device_error() == (6, Q.DEVERR_EXPERT_ID)
    got = y.cpu().numpy().astype(np.float64)
    for parity, w in ((0, W), (1, W2)):
        t, j = np.nonzero((ids >= 0) & (ids < E) & (ids % 2 == parity))
        close(got[t, j], *X.forward(x[t], w, fmt))
    t, j = np.nonzero((ids < 0) | (ids >= E))
    assert not got[t, j].any()


# ---- alignment, small magnitudes, waits ------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
def test_activations_and_weights_16_bytes_off_a_32_byte_boundary(Q, fmt):
    M, N, K = 9, 140, 384
    x = x_bits(M, K, seed=8)
    room = torch.empty(M * K + 8, dtype=torch.bfloat16, device="cuda")
    xd = room[8:].view(M, K)
    assert xd.data_ptr() % 32 == 16
    xd.copy_(dev_bf16(x))
    n, b = X.quantise(X.bf16_values(x), True)
    c_ref, s_ref = X.pack(n, b)
    cq, sq = Q.act_quant_mxfp4(xd, True)
    assert np.array_equal(host_u8(cq), c_ref.ravel()) and np.array_equal(host_u8(sq), s_ref.ravel())
    W = synth.weight_rows(3, "mxoff", K, 0, N)
    wide = torch.empty(N * K + 4, dtype=torch.float32, device="cuda")
    wd = wide[4:].view(N, K)
    wd.copy_(dev(W))
    c, s, _ = Q.qlinear_pack(fmt, N, K, W=wd)
    c_ref, s_ref = X.pack(*X.quantise(W))
    assert np.array_equal(host_u8(c), c_ref.ravel()) and np.array_equal(host_u8(s), s_ref.ravel())
    close(Q.qlinear_forward(xd, c, s, None, fmt, N), *X.forward(x, X.values(*X.quantise(W)), fmt))


@pytest.mark.parametrize("rotate", [0, 1])
@pytest.mark.parametrize("M", [8, 30])
def test_rows_of_small_magnitude(Q, M, rotate):
    # 16-bit activations keep what the bound allows from every block of a row, however small the row
    N, K = 200, 512
    rng = np.random.default_rng(4)
    v = rng.standard_normal((M, K))
    v[1] = np.ldexp(v[1], -110)
    v[2] = np.ldexp(v[2], -100)
    v[2, :32] = 0
    v[3] = np.ldexp(v[3], -126)
    v[3, 64:96] = np.ldexp(rng.standard_normal(32), -70)
    v[4, 128:160] = np.ldexp(v[4, 128:160], -120)
    v[5] = np.ldexp(v[5], -131)
    v[6] = 0
    v[7] = np.ldexp(v[7], 100)
    x = O.bf16_encode(v.ravel()).reshape(M, K)
    n = rng.integers(0, 16, (N, K), dtype=np.uint8)
    for scale in (127, 220):
        W = X.values(n, np.full((N, K // 32), scale, np.uint8))
        c, s, _ = Q.qlinear_pack(16, N, K, codes=dev(n), scales=dev(np.full((N, K // 32), scale, np.uint8)))
        ref, bound = X.forward(x, W, 16, bool(rotate))
        small = np.abs(ref) < 2.0 ** 126  # larger sums overflow fp32 on the way
        got = Q.qlinear_forward(dev_bf16(x), c, s, None, 16, N, flags=rotate).cpu().numpy().astype(np.float64)
        # fp32 atomic adds flush numbers below 2^-126: two partial sums of an output, each off by less than that,
        # and their sum once more, so 3 * 2^-126 at most
        off = np.abs(got - ref)[small] - bound[small] - 3 * 2.0 ** -126
        assert off.max() <= 0


def test_waits_that_run_out_are_reported(Q):
    # one row (a tile cut between two CTAs) and many (pairs of CTAs), both formats: with a bound that no wait
    # meets the calls return and say so, and the same calls are right again afterwards
    N, K = 600, 640
    c, s, W = weight(Q, N, K)
    for fmt in FMTS:
        for M in (1, 200):
            x = x_bits(M, K, seed=9)
            xd = dev_bf16(x)
            Q.qlinear_forward(xd, c, s, None, fmt, N)
            assert Q.ql_get_device_error() == (0, 0)
            Q.ql_set_wait_limit(1)
            try:
                Q.qlinear_forward(xd, c, s, None, fmt, N)
                st, bits = Q.ql_get_device_error()
            finally:
                Q.ql_set_wait_limit(0)
            assert st == 6 and bits == Q.DEVERR_TIMEOUT
            close(Q.qlinear_forward(xd, c, s, None, fmt, N), *X.forward(x, W, fmt))


# ---- together, streams, graphs -----------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
def test_experts_block(Q, fmt):
    """Pack, route, sort, multiply, activate and combine, as a mixture-of-experts block would."""
    T, topk, E, I, K = 24, 2, 4, 64, 256
    N = 2 * I
    Ws = [synth.weight_rows(11, f"mxb{e}", K, 0, N) for e in range(E)]
    packed = [Q.qlinear_pack(fmt, N, K, W=dev(w), flags=Q.HADAMARD) for w in Ws]
    c, s = torch.cat([p[0] for p in packed]), torch.cat([p[1] for p in packed])
    ids, w = synth.routing(5, T, E, topk)
    x = x_bits(T, K, seed=4)
    wd = synth.to_bf16_bits(synth.weight_rows(12, "mxd", I, 0, E * K)).reshape(E, K, I)
    h = Q.moe_gate_up(dev_bf16(x), dev(ids), c, s, E, N, fmt=fmt, flags=Q.HADAMARD)
    _, offsets, perm = Q.moe_permute(dev(ids), E)
    rows = dev_bf16(x)[(perm // topk).long()]
    sorted_h = Q.qlinear_grouped(rows, offsets.clone(), c, s, E, N, fmt, Q.HADAMARD)
    assert torch.equal(h.reshape(T * topk, N)[perm.long()], sorted_h)  # the same sums, row by row
    ref = np.zeros((T, topk, N))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        ref[t, j], bound = X.forward(x[t], X.values(*X.quantise(Ws[e], True)), fmt, True)
        close(h.cpu().numpy()[t, j].astype(np.float64), ref[t, j], bound)
    out = Q.moe_down_combine(h, dev(ids), dev(w), dev(wd.view(np.int16)), E).cpu().numpy()
    want = O.moe_down_combine(h.cpu().numpy(), ids, w, wd, E)
    assert np.linalg.norm(out - want) <= 1e-5 * np.linalg.norm(want)


@pytest.mark.parametrize("fmt", FMTS)
def test_two_streams_at_once(Q, fmt):
    N, K = 2000, 1024
    c, s, W = weight(Q, N, K)
    streams = [torch.cuda.Stream() for _ in range(2)]
    inputs = [x_bits(M, K, seed=10 + M) for M in (4, 150)]
    xs = [dev_bf16(x) for x in inputs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(Q.qlinear_forward(xs[i], c, s, None, fmt, N))
    torch.cuda.synchronize()
    for x, ys in zip(inputs, got):
        close(ys[0], *X.forward(x, W, fmt))
        assert all(torch.equal(ys[0], y) for y in ys[1:])


@pytest.mark.parametrize("fmt", FMTS)
def test_side_stream_and_graphs_that_share_a_workspace(Q, fmt):
    N, K = 700, 640
    c, s, W = weight(Q, N, K)
    sizes = (3, 100)
    ws = torch.empty(max(Q.qlinear_workspace_size(fmt, 0, M, N, K) for M in sizes), dtype=torch.uint8, device="cuda")
    xs = [dev_bf16(x_bits(M, K, seed=6)) for M in sizes]
    ys = [torch.empty(M, N, device="cuda") for M in sizes]
    side = torch.cuda.Stream()
    graphs = []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x, y in zip(xs, ys):
            Q.qlinear_forward(x, c, s, None, fmt, N, y=y, ws=ws)  # sets the launch attributes
        for x, y in zip(xs, ys):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                Q.qlinear_forward(x, c, s, None, fmt, N, y=y, ws=ws)
            graphs.append(g)
    torch.cuda.synchronize()
    for seed in (7, 8):
        new = [x_bits(M, K, seed=seed) for M in sizes]
        for x, b, y in zip(xs, new, ys):
            x.copy_(dev_bf16(b))
            y.fill_(float("nan"))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for b, y in zip(new, ys):
            close(y, *X.forward(b, W, fmt))


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_many_overlapping_segments(Q, fmt):
    # every second expert claims every row: flagged, and nothing outside y is touched
    E, N, K, R = 64, 130, 128, 600
    c, s, _ = weight(Q, N, K)
    y = torch.full((R + 1, N), 7.0, device="cuda")
    offsets = np.array([0, R] * (E // 2) + [0], np.int32)
    Q.qlinear_grouped(dev_bf16(x_bits(R, K)), dev(offsets), c.repeat(E), s.repeat(E), E, N, fmt, y=y[:R])
    assert Q.ql_get_device_error() == (6, Q.DEVERR_BOUNDS)
    assert (y[R] == 7.0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_and_gate_up_of_long_rows(Q, fmt):
    E, N, K, R = 2, 40, 32896, 5
    x, offsets = x_bits(R, K), [0, 2, 5]
    c, s, W = weight(Q, N, K)
    got = Q.qlinear_grouped(dev_bf16(x), dev(np.array(offsets, np.int32)), c.repeat(E), s.repeat(E), E, N, fmt)
    close(got, *X.forward(x, W, fmt))
    ids = dev(np.arange(R, dtype=np.int32).reshape(R, 1) % E)
    close(Q.moe_gate_up(dev_bf16(x), ids, c.repeat(E), s.repeat(E), E, N, fmt=fmt, flags=0)[:, 0], *X.forward(x, W, fmt))


@pytest.mark.parametrize("fmt", FMTS)
def test_gate_up_most_pairs_of_no_expert(Q, fmt):
    T, topk, E, N, K = 500, 4, 8, 260, 256
    ids = np.full((T, topk), -1, np.int32)
    ids[::50, 2] = 5
    x = x_bits(T, K)
    c, s, W = weight(Q, N, K)
    y = torch.full((T, topk, N), float("nan"), device="cuda")
    Q.moe_gate_up(dev_bf16(x), dev(ids), c.repeat(E), s.repeat(E), E, N, fmt=fmt, flags=0, y=y)
    assert Q.ql_get_device_error() == (6, Q.DEVERR_EXPERT_ID)
    close(y[::50, 2], *X.forward(x[::50], W, fmt))
    y[::50, 2] = 0
    assert not y.any()


@pytest.mark.parametrize("fmt", FMTS)
def test_stream_argument_owns_what_the_call_allocates(Q, fmt):
    # memory that the call took on a busy side stream is not handed to the current stream when the call returns
    N, K, M = 300, 1024, 40
    x = x_bits(M, K)
    c, s, W = weight(Q, N, K)
    side, xd = torch.cuda.Stream(), dev_bf16(x)
    need = Q.qlinear_workspace_size(fmt, 0, M, N, K)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    y = Q.qlinear_forward(xd, c, s, None, fmt, N, stream=side)
    codes, scales = Q.act_quant_mxfp4(xd, stream=side)
    for _ in range(4):
        torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    close(y, *X.forward(x, W, fmt))
    n, b = X.quantise(O.bf16_decode(x.ravel()).reshape(M, K))
    rc, rs = X.pack(n, b)
    assert np.array_equal(host_u8(codes).ravel(), rc.ravel()) and np.array_equal(host_u8(scales).ravel(), rs.ravel())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,had", [(65, 300, 2048, 0), (100, 1000, 2176, 1), (130, 2600, 2304, 0), (200, 520, 4224, 0),
                                       (300, 6500, 2048, 0), (700, 5130, 2176, 0)])
def test_forward_last_tiles_cut_along_k(Q, fmt, M, N, K, had):
    x = x_bits(M, K, seed=4)
    c, s, W = weight(Q, N, K, seed=4)
    xd = dev_bf16(x)
    y = torch.full((M, N), float("nan"), device="cuda")
    Q.qlinear_forward(xd, c, s, None, fmt, N, flags=had, y=y)
    close(y, *X.forward(x, W, fmt, bool(had)))
    for _ in range(5):
        assert torch.equal(Q.qlinear_forward(xd, c, s, None, fmt, N, flags=had), y)


@pytest.mark.parametrize("M,N,K", [(25, 9473, 256), (64, 9400, 2048), (100, 19000, 2176), (300, 9000, 1152), (90, 2000, 640),
                                   (144, 500, 384), (145, 500, 384)])
def test_forward_16_bit_either_side_of_digits(Q, M, N, K):
    # few rows of a large weight and many of a small one: as parts, some tiles halved, or as digits of several blocks
    x = x_bits(M, K, seed=8)
    c, s, W = weight(Q, N, K, seed=8)
    xd = dev_bf16(x)
    y = torch.full((M, N), float("nan"), device="cuda")
    Q.qlinear_forward(xd, c, s, None, 16, N, y=y)
    close(y, *X.forward(x, W, 16))
    assert torch.equal(Q.qlinear_forward(xd, c, s, None, 16, N), y)
