// k_mxfp4.cu -- microscaled 4-bit floating point (MXFP4): the quantisers of
// weights and activations, the packer of given codes, and the values that
// packed codes stand for.
//
// One warp takes one row's 128 columns, 4 neighbouring values a lane, as the
// other quantisers of this library do: the rotation's shuffles stay inside the
// warp, a 32-block is 8 lanes, and the 128 columns' four scale bytes are one
// word of the scale layout (mx_layout.cuh).  Bound by HBM: 2 (bf16) or 4 (fp32)
// bytes in and 17/32 byte out per value.
#include "mx_layout.cuh"
#include "ql_internal.h"

namespace ql {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void load4(const float* p, float v[4]) {
    const float4 r = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float v[4]) { load4_bf16(p, v); }

// The warp's four scale bytes (one per 8 lanes) as the word that lane 0 stores.
__device__ __forceinline__ uint32_t scale_word(uint32_t byte) {
    uint32_t w = byte;
#pragma unroll
    for (int b = 1; b < 4; ++b) w |= __shfl_sync(kFull, byte, 8 * b) << (8 * b);
    return w;
}

// Rows [0, N) of W to packed MXFP4; rows up to the next multiple of 128 get zero scales.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_mx_quant(const T* W, int N, int K, int rotate, uint8_t* codes,
                                                          uint8_t* scales) {
    const int lane = threadIdx.x & 31;
    const int G = K / 128;
    const long long units = (long long)((N + 127) / 128 * 128) * G;
    const long long nw = (long long)gridDim.x * kWarps;
    for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += nw) {
        const int r = (int)(u / G), g = (int)(u - (long long)r * G);
        uint32_t word = 0;
        if (r < N) {
            float v[4];
            load4(W + (long long)r * K + g * 128 + 4 * lane, v);
            if (rotate) fwht128_warp(v, lane);
            uint32_t byte;
            const uint32_t c = mx_quant4(v, byte);
            *reinterpret_cast<uint16_t*>(codes + (long long)r * (K / 2) + g * 64 + 2 * lane) = (uint16_t)c;
            word = scale_word(byte);
        }
        if (lane == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_at(r >> 7, G, g, 1, r & 127)) = word;
    }
}

// Activations into the order of the product's tiles (mx_layout.cuh): sorted row r of `offsets` (null: one
// expert owning every row) reads x row r, or perm[r] / topk.  A16: two E4M3 parts per value.
template <bool A16>
__global__ void __launch_bounds__(kWarps * 32) k_mx_act(const MxAct a) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // let the product start its weight stream
    const int lane = threadIdx.x & 31;
    const int G = a.K / 128, r = blockIdx.x;
    int first = 0, count = a.R, e = 0;
    if (a.offsets) {
        e = mx_warp_search(a.E, r, [&](int i) { return __ldg(a.offsets + i); });
        if (e < 0) return;
        int end;
        mx_segment(a.offsets, e, a.R, first, end);
        if (r < first || r >= end) return;  // a row of no expert
        count = end - first;
    }
    long long src = r;
    if (a.perm) {
        const int p = __ldg(a.perm + r);
        if (p < 0 || p >= a.R) return;
        src = p / a.topk;
    }
    const int i = (r - first) / a.nt, c = (r - first) - i * a.nt;
    const int rows = min(a.nt, count - i * a.nt);
    const long long slot = first / a.nt + e + i;
    for (int g = blockIdx.y * kWarps + (threadIdx.x >> 5); g < G; g += gridDim.y * kWarps) {
        float v[4];
        load4_bf16(a.x + src * a.K + g * 128 + 4 * lane, v);
        if (a.rotate) fwht128_warp(v, lane);
        uint32_t byte;
        if constexpr (A16) {
            if (a.rotate) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = __bfloat162float(__float2bfloat16_rn(v[k]));
            }
            uint32_t hi, lo;
            mx_split4(v, hi, lo, byte);
            const long long at = (long long)r * a.K + g * 128 + 4 * lane;
            *reinterpret_cast<uint32_t*>(a.codes + at) = hi;
            *reinterpret_cast<uint32_t*>(a.codes + (long long)a.R * a.K + at) = lo;
            const uint32_t word = scale_word(byte);
            const uint32_t low = scale_word(byte == 255 ? 255 : byte - 5);
            if (lane == 0) {
                *reinterpret_cast<uint32_t*>(a.scales + mx_scale_at(slot, G, g, a.nblk, c)) = word;
                *reinterpret_cast<uint32_t*>(a.scales + mx_scale_at(slot, G, g, a.nblk, mx_pad16(rows) + c)) = low;
            }
        } else {
            const uint32_t q = mx_quant4(v, byte);
            *reinterpret_cast<uint16_t*>(a.codes + (long long)r * (a.K / 2) + g * 64 + 2 * lane) = (uint16_t)q;
            const uint32_t word = scale_word(byte);
            if (lane == 0) *reinterpret_cast<uint32_t*>(a.scales + mx_scale_at(slot, G, g, a.nblk, c)) = word;
        }
    }
}

// Given code numbers (one byte each) two to a byte; numbers above 15 are packed as 0 and flagged.
__global__ void __launch_bounds__(256) k_mx_pack_codes(const uint8_t* in, long long n8, uint8_t* out, unsigned* err) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n8) return;
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(in) + i);
    bool bad = false;
    uint32_t p = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t c = ((k < 4 ? w.x : w.y) >> (8 * (k & 3))) & 0xFFu;
        bad |= c > 15;
        p |= (c > 15 ? 0u : c) << (4 * k);
    }
    reinterpret_cast<uint32_t*>(out)[i] = p;
    if (bad) atomicOr(err, (unsigned)QL_DEVERR_CODE_RANGE);
}

// Row-major scale bytes [N][K / 32] into blocks.
__global__ void __launch_bounds__(256) k_mx_pack_scales(const uint8_t* in, int N, int K, uint8_t* out) {
    const int G = K / 128;
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= (long long)((N + 127) / 128 * 128) * G) return;
    const int r = (int)(u / G), g = (int)(u - (long long)r * G);
    *reinterpret_cast<uint32_t*>(out + mx_scale_at(r >> 7, G, g, 1, r & 127)) =
        r < N ? __ldg(reinterpret_cast<const uint32_t*>(in) + u) : 0u;
}

// 8 codes a thread: 4 bytes in, 16 bytes of bf16 out.  The f16 value of a code times a power of two has two
// significant bits, so the fp32 product and its rounding to bf16 are exact.
__global__ void __launch_bounds__(256) k_mx_dequant(const uint8_t* codes, const uint8_t* scales, int K, long long n8,
                                                    __nv_bfloat16* out) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n8) return;
    const int per = K / 8;
    const int r = (int)(i / per), k = (int)(i - (long long)r * per) * 8;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
    const float s = mx_scale(__ldg(scales + mx_scale_at(r >> 7, K / 128, k >> 7, 1, r & 127) + ((k >> 5) & 3)));
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t h = e2m1x2_to_f16x2((w >> (8 * j)) & 0xFFu);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f16_bits_to_float((uint16_t)h) * s,
                                                       f16_bits_to_float((uint16_t)(h >> 16)) * s);
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    reinterpret_cast<uint4*>(out)[i] = make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T>
cudaError_t quant(const T* W, int N, int K, int rotate, uint8_t* codes, uint8_t* scales, cudaStream_t s) {
    const long long units = (long long)((N + 127) / 128 * 128) * (K / 128);
    const long long blocks = (units + kWarps - 1) / kWarps;
    k_mx_quant<T><<<(unsigned)(blocks < 148 * 64 ? blocks : 148 * 64), kWarps * 32, 0, s>>>(W, N, K, rotate, codes,
                                                                                          scales);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_quant_weight(const float* W, int N, int K, int rotate, uint8_t* codes, uint8_t* scales,
                                   cudaStream_t s) {
    return quant(W, N, K, rotate, codes, scales, s);
}
cudaError_t launch_mx_quant_rows(const void* x, int M, int K, int rotate, uint8_t* codes, uint8_t* scales,
                                 cudaStream_t s) {
    return quant(static_cast<const __nv_bfloat16*>(x), M, K, rotate, codes, scales, s);
}

cudaError_t launch_mx_act(const MxAct& a, bool a16, cudaStream_t s) {
    const dim3 grid((unsigned)a.R, (unsigned)((a.K / 128 + kWarps - 1) / kWarps));
    if (a16) k_mx_act<true><<<grid, kWarps * 32, 0, s>>>(a);
    else k_mx_act<false><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_mx_pack(const uint8_t* codes_in, const uint8_t* scales_in, int N, int K, uint8_t* codes,
                           uint8_t* scales, unsigned* err, cudaStream_t s) {
    const long long n8 = (long long)N * (K / 8);
    k_mx_pack_codes<<<(unsigned)((n8 + 255) / 256), 256, 0, s>>>(codes_in, n8, codes, err);
    const long long words = (long long)((N + 127) / 128 * 128) * (K / 128);
    k_mx_pack_scales<<<(unsigned)((words + 255) / 256), 256, 0, s>>>(scales_in, N, K, scales);
    return cudaGetLastError();
}

cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int N, int K, void* out, cudaStream_t s) {
    const long long n8 = (long long)N * (K / 8);
    k_mx_dequant<<<(unsigned)((n8 + 255) / 256), 256, 0, s>>>(codes, scales, K, n8, static_cast<__nv_bfloat16*>(out));
    return cudaGetLastError();
}

}  // namespace ql
