"""The microscaled 4-bit operators: what they compute, in plain form, and the calls that a user makes of them.

MXFP4 holds 32 consecutive values of a row as E2M1 codes (sign, two exponent bits, one mantissa bit: 0, 0.5, 1,
1.5, 2, 3, 4, 6 and their negatives) under one power-of-two scale 2^e, stored as the byte e + 127:

    e = max(floor(log2(max |v|)) - 2, -127),   code = E2M1 nearest to v / 2^e, ties to the even code, at most 6.

Packed: two codes a byte, the even column in the low nibble, [rows][K / 2]; scales in blocks of 128 rows x 128
columns, [ceil(rows / 128)][K / 128][32][4][4], where byte [r % 32][r % 128 / 32][k % 128 / 32] of a block is the
scale of row r at column k.

Kinds of cases:
  quantise  activations (bf16) to MXFP4, rotated by the 128-wide Walsh-Hadamard transform first or not, and the
            values that the codes stand for
  pack      a weight (fp32) to MXFP4 and the values that its codes stand for
  forward   y = x . W^T of a packed weight: "w4a16" takes x in bf16, "w4a4" quantises x to MXFP4 first
  grouped   the same over rows sorted by expert with ragged counts (offsets), one weight per expert
  gate_up   the same from (token, slot) pairs and their expert ids, as a mixture-of-experts block calls it
"""
import math

import numpy as np
import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ROTATION = float(np.float32(1.0) / np.sqrt(np.float32(128.0)))  # 0x3DB504F3


def listed():
    return [
        # One decode step's activations of the dense layer, with the drafted tokens that are checked together.
        {"name": "quantise 16 rows rotated", "kind": "quantise", "M": 16, "K": 5376, "rotate": True},
        # A long prompt's activations.
        {"name": "quantise 16384 rows", "kind": "quantise", "M": 16384, "K": 5376, "rotate": False},
        # Packing the dense layer's weight into the rotated domain, once per checkpoint.
        {"name": "pack 21504x5376 rotated", "kind": "pack", "N": 21504, "K": 5376, "rotate": True},
        # Decode of one sequence, 4-bit activations.
        {"name": "w4a4 1 row", "kind": "forward", "fmt": "w4a4", "M": 1, "N": 21504, "K": 5376, "rotate": False},
        # Decode with 15 drafted tokens, rotated domain.
        {"name": "w4a4 16 rows rotated", "kind": "forward", "fmt": "w4a4", "M": 16, "N": 21504, "K": 5376, "rotate": True},
        # Decode of one sequence, 16-bit activations.
        {"name": "w4a16 1 row", "kind": "forward", "fmt": "w4a16", "M": 1, "N": 21504, "K": 5376, "rotate": False},
        # A chunk of a prompt, an odd number of rows, 16-bit activations.
        {"name": "w4a16 300 rows", "kind": "forward", "fmt": "w4a16", "M": 300, "N": 21504, "K": 5376, "rotate": False},
        # Prefill of 2048 batched tokens, 4-bit activations.
        {"name": "w4a4 2048 rows", "kind": "forward", "fmt": "w4a4", "M": 2048, "N": 21504, "K": 5376, "rotate": False},
        # The routed experts of one token, 16-bit activations in the rotated domain.
        {"name": "gate_up 1 token w4a16", "kind": "gate_up", "fmt": "w4a16", "T": 1, "topk": 8, "E": 128, "N": 1408, "K": 2816, "rotate": True},
        # The routed experts of a decode batch whose rows a caller has sorted.
        {"name": "grouped 128 rows w4a4", "kind": "grouped", "fmt": "w4a4", "T": 16, "topk": 8, "E": 128, "N": 1408, "K": 2816, "rotate": False},
        # A batch between decode and prefill, 16-bit activations: most experts have a dozen rows.
        {"name": "grouped 1600 rows w4a16", "kind": "grouped", "fmt": "w4a16", "T": 200, "topk": 8, "E": 128, "N": 1408, "K": 2816, "rotate": False},
        # The routed experts of 2048 batched tokens.
        {"name": "gate_up 2048 tokens w4a4", "kind": "gate_up", "fmt": "w4a4", "T": 2048, "topk": 8, "E": 128, "N": 1408, "K": 2816, "rotate": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("quantise", "pack", "forward", "forward", "forward", "grouped", "grouped", "gate_up"))
    K = 128 * _spread(rng, 1, 42)
    rotate = rng.random() < 0.5
    if kind == "quantise":
        return {"kind": kind, "M": _spread(rng, 1, 16384), "K": K, "rotate": rotate}
    if kind == "pack":
        return {"kind": kind, "N": _spread(rng, 64, 21504), "K": K, "rotate": rotate}
    fmt = rng.choice(("w4a16", "w4a4"))
    if kind == "forward":
        return {"kind": kind, "fmt": fmt, "M": _spread(rng, 1, 2048), "N": _spread(rng, 64, 21504), "K": K, "rotate": rotate}
    E = _spread(rng, 2, 128)
    return {"kind": kind, "fmt": fmt, "T": _spread(rng, 1, 2048), "topk": rng.randint(1, min(8, E)), "E": E,
            "N": _spread(rng, 64, 1408), "K": 128 * _spread(rng, 1, 22), "rotate": rotate}


def work(case):
    K = case["K"]
    values = lambda rows: rows * K * 2  # noqa: E731  bf16 rows
    packed = lambda rows: rows * (K // 2 + K // 32)  # noqa: E731
    if case["kind"] == "quantise":  # x in, codes and scales out; those in again, the values out
        return {"bytes": 2 * values(case["M"]) + 2 * packed(case["M"]), "flops": 0}
    if case["kind"] == "pack":
        return {"bytes": 3 * values(case["N"]) + 2 * packed(case["N"]), "flops": 0}
    if case["kind"] == "forward":
        M, N = case["M"], case["N"]
        return {"bytes": values(M) + packed(N) + 4 * M * N, "flops": 2 * M * N * K}
    T, topk, E, N = case["T"], case["topk"], case["E"], case["N"]
    touched = E * (1.0 - (1.0 - topk / E) ** T)  # experts that T random choices reach
    rows = T * topk
    x = values(rows if case["kind"] == "grouped" else T)
    return {"bytes": x + touched * packed(N) + 4 * rows * N + 4 * (E + 1 if case["kind"] == "grouped" else rows), "flops": 2 * rows * N * K}


# ---- the plain form ------------------------------------------------------------------------------------
def _power(e):
    """2^e of whole numbers -127 <= e <= 127, exact in fp32."""
    return torch.where(e == -127, torch.full_like(e, 0x00400000), (e + 127) << 23).view(torch.float32)


def _rotated(v):
    """The orthonormal 128-point Walsh-Hadamard transform of each 128 columns, every step rounded to fp32."""
    shape = v.shape
    for s in (1, 2, 4, 8, 16, 32, 64):
        v = v.reshape(-1, 64 // s, 2, s)
        v = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), 2)
    return v.reshape(shape) * ROTATION


def _quantised(v):
    """(code numbers 0..15, scale exponents) of fp32 rows."""
    g = v.reshape(*v.shape[:-1], -1, 32)
    amax = g.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp_min(-127).to(torch.int32)
    a = g.abs() * _power(-e)
    n = (a > 0.25).to(torch.uint8)
    for border, above in ((0.75, a.ge), (1.25, a.gt), (1.75, a.ge), (2.5, a.gt), (3.5, a.ge), (5.0, a.gt)):
        n += above(border)
    n += torch.signbit(g).to(torch.uint8) * 8
    return n.reshape(v.shape), e.squeeze(-1)


def _values(n, e):
    """fp32 values of code numbers and exponents."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=n.device)
    return (grid[n.long()].reshape(*e.shape, 32) * _power(e)[..., None]).reshape(n.shape)


def _pack(n, e):
    """Code numbers and exponents to the packed layout."""
    codes = n[..., 0::2] | (n[..., 1::2] << 4)
    rows, blocks = e.shape[0], -(-e.shape[0] // 128)
    s = torch.zeros(blocks * 128, e.shape[1], dtype=torch.uint8, device=e.device)
    s[:rows] = (e + 127).to(torch.uint8)
    return codes.contiguous(), s.reshape(blocks, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous()


def _unpacked(codes, scales, rows, K):
    """fp32 values of the packed layout."""
    codes = codes.reshape(rows, K // 2)
    n = torch.stack((codes & 15, codes >> 4), -1).reshape(rows, K)
    e = scales.reshape(-1, K // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, K // 32)[:rows].to(torch.int32) - 127
    return _values(n, e)


def _activations(x, fmt, rotate):
    """What the product sees of bf16 rows, in fp32."""
    v = x.float()
    if rotate:
        v = _rotated(v)
    if fmt == "w4a4":
        return _values(*_quantised(v))
    return v.to(torch.bfloat16).float()


def _by_expert(rows, expert, place, weights, most):
    """Row r times the transposed weight of its expert; `place`: its number among that expert's rows, under `most`."""
    E, N, K = weights.shape
    held = torch.zeros(E, most, K, device=rows.device)
    held[expert, place] = rows
    return torch.bmm(held, weights.transpose(1, 2))[expert, place]


def _expert_weights(s):
    E, N, K = s["E"], s["N"], s["K"]
    blocks = -(-N // 128) * (K // 128) * 512
    e = s["scales"].reshape(E, blocks).reshape(E, -1, K // 128, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, -1, K // 32)[:, :N].to(torch.int32) - 127
    codes = s["codes"].reshape(E, N, K // 2)
    n = torch.stack((codes & 15, codes >> 4), -1).reshape(E, N, K)
    return _values(n, e)


# ---- the cases -----------------------------------------------------------------------------------------
def _x(rows, K, gen):
    """Activations with one column in a hundred twenty times as large."""
    x = torch.randn(rows, K, device="cuda", generator=gen)
    x[:, torch.randperm(K, device="cuda", generator=gen)[: K // 100]] *= 20.0
    return x.to(torch.bfloat16)


def _weight(rows, K, gen):
    return _pack(*_quantised(torch.randn(rows, K, device="cuda", generator=gen) * 0.02))


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    K = case["K"]
    if case["kind"] == "quantise":
        s["x"] = _x(case["M"], K, gen)
    elif case["kind"] == "pack":
        s["W"] = torch.randn(case["N"], K, device="cuda", generator=gen) * 0.02
    elif case["kind"] == "forward":
        s["x"] = _x(case["M"], K, gen)
        s["codes"], s["scales"] = _weight(case["N"], K, gen)
    else:
        T, topk, E = case["T"], case["topk"], case["E"]
        packed = [_weight(case["N"], K, gen) for _ in range(E)]
        s["codes"], s["scales"] = (torch.stack(p) for p in zip(*packed))
        s["ids"] = (torch.randn(T, E, device="cuda", generator=gen) * 2.0).topk(topk).indices.to(torch.int32)
        if case["kind"] == "gate_up":
            s["x"] = _x(T, K, gen)
        else:
            s["x"] = _x(T * topk, K, gen)
            counts = torch.bincount(s["ids"].flatten().long(), minlength=E)
            s["offsets"] = torch.cat((counts.new_zeros(1), counts.cumsum(0))).to(torch.int32)
    return s


def _own(s):
    from moe_hadamard128_act_b200 import qlinear as Q

    flags = Q.HADAMARD if s["rotate"] else 0
    K = s["K"]
    if s["kind"] == "quantise":
        codes, scales = Q.act_quant_mxfp4(s["x"], s["rotate"])
        return Q.mxfp4_dequant(codes, scales, s["M"], K)
    if s["kind"] == "pack":
        codes, scales, _ = Q.qlinear_pack(Q.MXFP4_G32, s["N"], K, W=s["W"], flags=flags)
        return Q.mxfp4_dequant(codes, scales, s["N"], K)
    fmt = Q.MXFP4A4_G32 if s["fmt"] == "w4a4" else Q.MXFP4_G32
    if s["kind"] == "forward":
        return Q.qlinear_forward(s["x"], s["codes"], s["scales"], None, fmt, s["N"], flags)
    if s["kind"] == "grouped":
        return Q.qlinear_grouped(s["x"], s["offsets"], s["codes"], s["scales"], s["E"], s["N"], fmt, flags)
    return Q.moe_gate_up(s["x"], s["ids"], s["codes"], s["scales"], s["E"], s["N"], fmt, flags)


def run(s):
    if own:
        return _own(s)
    K = s["K"]
    if s["kind"] in ("quantise", "pack"):
        v = (s["x"] if s["kind"] == "quantise" else s["W"]).float()
        return _values(*_quantised(_rotated(v) if s["rotate"] else v)).to(torch.bfloat16)
    x = _activations(s["x"], s["fmt"], s["rotate"])
    if s["kind"] == "forward":
        return x @ _unpacked(s["codes"], s["scales"], s["N"], K).T
    W = _expert_weights(s)
    if s["kind"] == "grouped":
        r = torch.arange(x.shape[0], device=x.device, dtype=torch.int32)
        expert = torch.searchsorted(s["offsets"], r, right=True) - 1
        return _by_expert(x, expert, (r - s["offsets"][expert]).long(), W, s["T"])
    ids = s["ids"].long()  # a token reaches an expert at most once: its own number is its place
    token = torch.arange(s["T"], device=x.device)[:, None].expand_as(ids)
    return _by_expert(x.repeat_interleave(s["topk"], 0), ids.flatten(), token.flatten(), W, s["T"]).reshape(s["T"], s["topk"], s["N"])


# ---- the definition in 64 bits -------------------------------------------------------------------------
def _pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_rotation(v):
    """The rotation's roundings are part of its definition: fp32 after every butterfly and after the factor."""
    index = torch.arange(128, device=v.device)
    v = v.float().reshape(-1, 128)
    for bit in range(7):
        partner = v[:, index ^ (1 << bit)]
        v = torch.where((index >> bit & 1).bool(), partner - v, v + partner)
    return (v.double() * torch.tensor(0x3DB504F3, dtype=torch.int32, device=v.device).view(torch.float32).double()).float()


def _exact_mxfp4(v):
    """The values that each 32 of a row are held as, in 64 bits."""
    g = v.double().reshape(-1, 32)
    m = g.abs().amax(1, keepdim=True)
    e = ((m.view(torch.int64) >> 52) - 1023 - 2).clamp(min=-127)
    a = g.abs() * _pow2(-e)
    # Spacing of the grid: 0.5 below 2, 1 below 4, 2 above; torch.round takes ties to even, which is the even code.
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0) * _pow2(e), g)


def _exact_weight(codes, scales, N, K):
    c = codes.reshape(N, K // 2).long()
    n = torch.empty(N, K, dtype=torch.int64, device=c.device)
    n[:, 0::2], n[:, 1::2] = c % 16, c // 16
    mag, exp = n % 2, n // 2 % 4  # value: m / 2 for exponent 0, else (1 + m / 2) 2^(exponent - 1)
    v = torch.where(exp == 0, mag * 0.5, (1 + mag * 0.5) * _pow2(exp - 1)) * (1 - 2 * (n // 8)).double()
    r, k = torch.arange(N, device=c.device)[:, None], 32 * torch.arange(K // 32, device=c.device)[None, :]
    at = ((r // 128) * (K // 128) + k // 128) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 128 // 32
    return (v.reshape(N, -1, 32) * _pow2(scales.reshape(-1)[at].long() - 127)[..., None]).reshape(N, K)


def exact(case, seed):
    s = prepare(case, seed)
    N, K = case.get("N"), case["K"]
    src = s["W"] if case["kind"] == "pack" else s["x"]
    v = (_exact_rotation(src) if case["rotate"] else src.float()).reshape(src.shape)
    if case["kind"] in ("quantise", "pack"):
        return _exact_mxfp4(v).reshape(v.shape)
    v = _exact_mxfp4(v).reshape(v.shape) if case["fmt"] == "w4a4" else v.to(torch.bfloat16).double()
    if case["kind"] == "forward":
        return v @ _exact_weight(s["codes"], s["scales"], N, K).T
    if case["kind"] == "gate_up":
        y = torch.zeros(case["T"], case["topk"], N, dtype=torch.float64, device=v.device)
    else:
        y = torch.zeros(v.shape[0], N, dtype=torch.float64, device=v.device)
    for e in range(case["E"]):
        W = _exact_weight(s["codes"][e], s["scales"][e], N, K)
        if case["kind"] == "gate_up":
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            y[t, j] = v[t] @ W.T
        else:
            a, b = (int(o) for o in s["offsets"][e : e + 2])
            y[a:b] = v[a:b] @ W.T
    return y
