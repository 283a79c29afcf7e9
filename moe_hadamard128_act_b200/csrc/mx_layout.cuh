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
// nothing has to be counted beforehand.  A slot's operand rows are its rows in
// order, and for 16-bit activations the low parts of the same rows after them,
// starting at the block's row count rounded up to 16.
#pragma once

#include "ql_device.cuh"

namespace ql {

// Byte of row r's scale word for 128-column block kb within a run of 512-byte blocks, `nblk` blocks per kb.
__host__ __device__ __forceinline__ long long mx_scale_at(long long slot, int G, int kb, int nblk, int r) {
    return ((slot * G + kb) * nblk + (r >> 7)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

__host__ __device__ __forceinline__ int mx_pad16(int rows) { return (rows + 15) & ~15; }

// One token block: rows [row0, row0 + rows) of the sorted order.
struct MxBlock {
    int expert, row0, rows;  // rows = 0: an empty slot
};

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

// Two fp32 values to E2M1 by the hardware conversion (round to nearest even, saturating to +-6): the low
// nibble holds `lo`, the high nibble `hi`.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float hi, float lo) {
    uint32_t r;
    asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
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

// Largest magnitude of a 32-block held 4 values per lane by 8 neighbouring lanes, as fp32 bits without the
// sign: unsigned order puts infinities and NaN above every finite value.
__device__ __forceinline__ uint32_t mx_block_amax(const float v[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(kFull, m, d));
    return m;
}

// MXFP4 of a 32-block (4 values per lane): the lane's four codes (low nibble first) and the scale byte.
// floor(log2 amax) is the exponent field, so the byte e + 127 with e = floor(log2 amax) - 2 is the field
// less 2, clamped at 0; the division by 2^e is an exact product.
__device__ __forceinline__ uint32_t mx_quant4(const float v[4], uint32_t& byte) {
    const uint32_t ex = mx_block_amax(v) >> 23;
    if (ex == 255) {  // an infinity or a NaN
        byte = 255;
        return 0;
    }
    byte = ex > 2 ? ex - 2 : 0;
    const float inv = __uint_as_float((254u - byte) << 23);
    return cvt_e2m1x2(v[1] * inv, v[0] * inv) | cvt_e2m1x2(v[3] * inv, v[2] * inv) << 8;
}

// A 32-block of bf16 values as two E4M3 parts (4 values per lane, low byte first), v = 2^e (hi + lo / 32):
// e puts the block's largest magnitude into [128, 256), hi is v / 2^e rounded to E4M3's four significant
// bits, and what is left of bf16's eight fits four more, so the sum is exact unless the value is so far below
// the largest that lo's spacing 2^-9 cuts it: exact from 2^-14 of the largest up, within 2^-22 of it below.
// byte: hi's scale; lo's is byte - 5 (e is held at -122 or more for that).
__device__ __forceinline__ void mx_split4(const float v[4], uint32_t& hi, uint32_t& lo, uint32_t& byte) {
    const uint32_t ex = mx_block_amax(v) >> 23;
    hi = lo = 0;
    if (ex == 255) {
        byte = 255;
        return;
    }
    byte = ex > 12 ? ex - 7 : 5;
    const float inv = __uint_as_float((254u - byte) << 23);
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = v[i] * inv;
    hi = cvt_e4m3x2(s[1], s[0]) | cvt_e4m3x2(s[3], s[2]) << 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t h = e4m3x2_to_f16x2(hi >> (16 * i));
        s[2 * i] -= f16_bits_to_float((uint16_t)h);
        s[2 * i + 1] -= f16_bits_to_float((uint16_t)(h >> 16));
    }
    lo = cvt_e4m3x2(s[1] * 32.0f, s[0] * 32.0f) | cvt_e4m3x2(s[3] * 32.0f, s[2] * 32.0f) << 16;
}

}  // namespace ql
