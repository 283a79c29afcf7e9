// mx_layout.cuh -- where the MXFP4 operands lie, shared by the quantisers
// (k_mxfp4.cu) and the product (k_mxfp4_gemm.cu).
//
// The product's tensor-core instructions take their block scales from tensor
// memory, 32 rows to a column and four scales (128 of K) to a column's word, so
// scales are kept in 512-byte blocks of 128 rows x 128 of K,
// [row % 32][row % 128 / 32][k % 128 / 32], which one copy brings to shared
// memory and one tcgen05.cp to tensor memory.
//
// Activations are quantised into the order of the product's tiles.  Rows are
// cut, expert by expert, into token blocks of at most nt rows; block i of
// expert e gets the slot number offsets[e] / nt + e + i, which no other block
// has (an expert of c rows starts at most c / nt + 1 slots before the next), so
// nothing has to be counted beforehand.  A token is one or more operand rows of
// its block (MxMode):
//   kMxA4      its MXFP4 codes: row c.
//   kMxDigits  16-bit activations as eight E2M1 digits: rows 8 c .. 8 c + 7.
//   kMxParts   16-bit activations as two E4M3 parts: row c, and the low part's
//              row n + c, n the block's tokens rounded up to 16.
#pragma once

#include "ql_device.cuh"
#include "ql_internal.h"

namespace ql {

// Byte of row r's scale word for 128-column block kb within a run of 512-byte blocks, `nblk` blocks per kb.
__host__ __device__ __forceinline__ long long mx_scale_at(long long slot, int G, int kb, int nblk, int r) {
    return ((slot * G + kb) * nblk + (r >> 7)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}


__host__ __device__ __forceinline__ int mx_pad16(int rows) { return (rows + 15) & ~15; }

// Segment of expert e in the sorted rows; empty when its offsets are out of order or out of [0, R].
__device__ __forceinline__ bool mx_segment(const int32_t* offsets, int e, int R, int& a, int& b) {
    a = __ldg(offsets + e);
    b = __ldg(offsets + e + 1);
    if (a >= 0 && a <= b && b <= R) return true;
    a = b = 0;
    return false;
}

// The largest e in [0, E) with key(e) <= v for a non-decreasing key, by a whole warp (E <= 1024:
// two rounds of 32 probes); -1 if there is none.
template <typename Key>
__device__ __forceinline__ int mx_warp_search(int E, int v, Key key) {
    const int lane = threadIdx.x & 31;
    const int step = (E + 31) >> 5;
    unsigned m = __ballot_sync(kFull, lane * step < E && key(lane * step) <= v);
    if (!m) return -1;
    const int base = (31 - __clz(m)) * step;
    m = __ballot_sync(kFull, lane < step && base + lane < E && key(base + lane) <= v);
    return base + 31 - __clz(m | 1u);
}

// The expert whose segment row r lies in, and the segment, by a whole warp; -1: none.  Among offsets in order it is the
// last that starts at or before r.  Beside offsets that are not, the search may miss it: then all experts are looked at.
__device__ __forceinline__ int mx_expert_of(const int32_t* offsets, int E, int R, int r, int& a, int& b) {
    const int e = mx_warp_search(E, r, [&](int i) { return __ldg(offsets + i); });
    if (e >= 0 && mx_segment(offsets, e, R, a, b) && r >= a && r < b) return e;
    int found = E;  // the lane's, of those that it looks at; the loads wait for nothing
#pragma unroll 4
    for (int i = threadIdx.x & 31; i < E; i += 32) {
        const int first = __ldg(offsets + i), end = __ldg(offsets + i + 1);
        if (first >= 0 && first <= r && r < end && end <= R) found = min(found, i);
    }
    found = __reduce_min_sync(kFull, found);
    if (found < E && mx_segment(offsets, found, R, a, b)) return found;
    a = b = 0;
    return -1;
}

// Eight fp32 values to E2M1 by the hardware conversion (round to nearest even, saturating to +-6), the first in
// the low nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float v[8]) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// Largest magnitude of three, a NaN if there is one.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two E2M1 codes (low byte of c) to f16x2, exact.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t c) {
    uint32_t r;
    asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(r) : "r"(c));
    return r;
}
// 2^(b - 127) of a scale byte: exact (a subnormal for 0), NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FFFFFFFu : b << 23);
}

// ---- 128 columns of a row held 16 neighbouring values a lane by 8 lanes (a quarter of a warp) -------------
// The Walsh-Hadamard transform of fwht128_warp, bit for bit: the same butterflies in the same order, strides
// 1 .. 8 inside the lane and 16 .. 64 across lanes.
__device__ __forceinline__ void mx_fwht128(float v[16], int lane) {
#pragma unroll
    for (int s = 1; s < 16; s <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (!(i & s)) {
                const float a = v[i], b = v[i | s];
                v[i] = __fadd_rn(a, b);
                v[i | s] = __fsub_rn(a, b);
            }
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) {
        const float sgn = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float o = __shfl_xor_sync(kFull, v[i], m);
            v[i] = __fmaf_rn(sgn, v[i], o);
        }
    }
    const float c = fwht_scale();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(v[i], c);
}

// A 32-block's largest magnitude (2 lanes) as fp32 bits without the sign: unsigned order puts infinities and
// NaN (exponent field 255) above every finite value.
__device__ __forceinline__ uint32_t mx_block_max(const float v[16]) {
    float a = max3_abs(v[0], v[1], v[2]);
#pragma unroll
    for (int i = 3; i < 15; i += 2) a = max3_abs(a, v[i], v[i + 1]);
    const uint32_t m = __float_as_uint(max3_abs(a, v[15], v[15]));
    return max(m, __shfl_xor_sync(kFull, m, 1));
}
// The four blocks' scale bytes as one word, in all 8 lanes.
__device__ __forceinline__ uint32_t mx_scale_word(uint32_t byte, int lane) {
    uint32_t w = byte << (8 * ((lane >> 1) & 3));
    w |= __shfl_xor_sync(kFull, w, 2);
    return w | __shfl_xor_sync(kFull, w, 4);
}

// MXFP4 of a 32-block: the lane's sixteen codes (low nibble first) and the scale byte.  floor(log2 amax) is the
// exponent field, so the byte e + 127 with e = floor(log2 amax) - 2 is the field less 2, clamped at 0; the
// division by 2^e is an exact product.
__device__ __forceinline__ uint2 mx_quant16(const float v[16], uint32_t& byte) {
    const uint32_t ex = mx_block_max(v) >> 23;
    byte = ex > 2 ? ex - 2 : 0;
    const float inv = __uint_as_float((254u - byte) << 23);
    float s[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = v[i] * inv;
    uint2 c = make_uint2(cvt_e2m1x8(s), cvt_e2m1x8(s + 8));
    if (ex == 255) {  // an infinity or a NaN
        byte = 255;
        c = make_uint2(0, 0);
    }
    return c;
}

// A 32-block of bf16 values as eight E2M1 digits, v = 2^e sum_p d_p 8^-p: e puts the block's largest magnitude
// into [1, 2), v / 2^e is rounded to a multiple of 8^-7, and that number's digits in base 8 from -4 to 3 are all
// E2M1 values.  So v is off by at most 2^-22 of the largest magnitude, and not at all down to 2^-14 of it.
// byte: the first digit's scale; digit p's is byte - 3 p, so it is held at 21 or more: a block below 2^-105
// loses its last digits, unless its whole row is small and was scaled up by 2^up (see k_mx_act).
// The digits are taken in integers: 4 in every digit makes them 0 .. 7, three bits each, which are spread to
// nibbles; a byte permute then looks four of them up at once, and two more rounds of permutes turn one
// value's digits into one digit's values (digit p of eight values: d[p], low nibble first).
__device__ __forceinline__ uint32_t mx_digits_byte(uint32_t ex, int up) {
    return ex == 255 ? 255u : (uint32_t)max((int)ex + up, 21);  // 255: an infinity or a NaN
}
__device__ __forceinline__ void mx_digits8(const float* v, uint32_t byte, int up, uint32_t d[8]) {
    // 2^-e has the exponent field f: 0, a subnormal, for blocks that reach 2^127, and up to 254, for those below 2^-126 of a
    // row scaled up, so 8^7 = 2^21 is a factor of its own.
    const uint32_t f = 254u + (uint32_t)up - byte;
    const float inv = __uint_as_float(f == 0 ? 0x00400000u : f << 23);
    constexpr uint32_t kLow = 0x0A0C0D0Eu, kHigh = 0x05040200u;  // E2M1 of -4 .. -1 and 0 .. 3
    uint32_t lo[4], hi[4];  // values 2 j and 2 j + 1 in a byte; digits 7 .. 4 and 3 .. 0 from the low byte up
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t u = (uint32_t)(__float2int_rn(v[i] * inv * 0x1p21f) + 0x924924);
        // Fields moved up by multiply-adds (u + 15 f is u with its field f shifted by 4), which the integer pipe,
        // the busiest one here, does not see.
        u += (u & 0xFFF000u) * 15u;
        u += (u & 0x0FC00FC0u) * 3u;
        u += u & 0x38383838u;
        const uint32_t l = __byte_perm(kLow, kHigh, u & 0xFFFFu), h = __byte_perm(kLow, kHigh, u >> 16);
        lo[i >> 1] = (i & 1) ? lo[i >> 1] + l * 16u : l;
        hi[i >> 1] = (i & 1) ? hi[i >> 1] + h * 16u : h;
    }
    auto turn = [](const uint32_t a[4], uint32_t& b0, uint32_t& b1, uint32_t& b2, uint32_t& b3) {
        const uint32_t p = __byte_perm(a[0], a[1], 0x5140), q = __byte_perm(a[2], a[3], 0x5140);  // bytes 0 and 1
        const uint32_t r = __byte_perm(a[0], a[1], 0x7362), t = __byte_perm(a[2], a[3], 0x7362);  // bytes 2 and 3
        b0 = __byte_perm(p, q, 0x5410);
        b1 = __byte_perm(p, q, 0x7632);
        b2 = __byte_perm(r, t, 0x5410);
        b3 = __byte_perm(r, t, 0x7632);
    };
    turn(lo, d[7], d[6], d[5], d[4]);
    turn(hi, d[3], d[2], d[1], d[0]);
    if (byte == 255) {
#pragma unroll
        for (int p = 0; p < 8; ++p) d[p] = 0;
    }
}

// A 32-block of bf16 values as two E4M3 parts (low byte first), v = 2^e (hi + lo / 32): e puts the block's
// largest magnitude into [128, 256), hi is v / 2^e rounded to E4M3's four significant bits, and what is left of
// bf16's eight fits four more, so the sum is exact unless the value is so far below the largest that lo's
// spacing 2^-9 cuts it: exact from 2^-14 of the largest up, within 2^-22 of it below.  byte: hi's scale; lo's
// is byte - 5 (e is held at -122 or more for that), or 255 with it.
__device__ __forceinline__ void mx_split16(const float v[16], uint4& hi, uint4& lo, uint32_t& byte) {
    const uint32_t ex = mx_block_max(v) >> 23;
    byte = ex > 12 ? ex - 7 : 5;
    const float inv = __uint_as_float((254u - byte) << 23);
    uint32_t h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = v[2 * i] * inv, b = v[2 * i + 1] * inv;
        h[i] = cvt_e4m3x2(b, a);
        const uint32_t f = e4m3x2_to_f16x2(h[i]);
        l[i] = cvt_e4m3x2((b - f16_bits_to_float((uint16_t)(f >> 16))) * 32.0f,
                          (a - f16_bits_to_float((uint16_t)f)) * 32.0f);
    }
    hi = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    lo = make_uint4(l[0] | l[1] << 16, l[2] | l[3] << 16, l[4] | l[5] << 16, l[6] | l[7] << 16);
    if (ex == 255) {  // an infinity or a NaN
        byte = 255;
        hi = lo = make_uint4(0, 0, 0, 0);
    }
}

}  // namespace ql
