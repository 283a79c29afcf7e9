// k_mxfp4_gemm.cu -- the product of MXFP4 weights: y = x~ . dequant(W)^T over
// one weight or, rows sorted by expert, over one weight per expert.
//
// A CTA takes 64 weight rows by one token block, dequantising both operands
// into shared memory 32 columns at a time.
#include "mx_layout.cuh"
#include "ql_internal.h"

namespace ql {
namespace {

constexpr int TN = 64, TK = 32;

template <bool A16>
__global__ void __launch_bounds__(256) k_mx_gemm(const MxGemm a) {
    __shared__ float sw[TK][TN + 1], sx[TK][kMxTokens + 1], fw[TN], fx[kMxTokens];
    const int slot = blockIdx.y, n0 = blockIdx.x * TN;
    MxBlock b{0, slot * a.nt, min(a.nt, a.R - slot * a.nt)};
    if (a.offsets) {  // the slot's expert: the largest e with offsets[e] / nt + e <= slot
        b.expert = mx_warp_search(a.E, slot, [&](int e) { return __ldg(a.offsets + e) / a.nt + e; });
        if (b.expert < 0) return;
        int lo, hi;
        if (!mx_segment(a.offsets, b.expert, a.R, lo, hi) && threadIdx.x == 0)
            atomicOr(a.err, (unsigned)QL_DEVERR_BOUNDS);
        b.row0 = lo + (slot - (lo / a.nt + b.expert)) * a.nt;
        b.rows = min(a.nt, hi - b.row0);
    }
    if (b.rows <= 0) return;
    const int G = a.K / 128, NB = (a.N + 127) / 128;
    const uint8_t* codes = a.codes + (long long)b.expert * a.N * (a.K / 2);
    const uint8_t* scales = a.scales + (long long)b.expert * NB * G * 512;
    const int tn = threadIdx.x % 16, tm = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += TK) {
        const int kb = k0 >> 7, j = (k0 >> 5) & 3;
        for (int i = threadIdx.x; i < TN * TK / 2; i += 256) {
            const int r = n0 + i / (TK / 2), k = 2 * (i % (TK / 2));
            uint32_t h = 0;
            if (r < a.N) h = e2m1x2_to_f16x2(__ldg(codes + (long long)r * (a.K / 2) + (k0 + k) / 2));
            if (k == 0) fw[r - n0] = r < a.N ? mx_scale(__ldg(scales + mx_scale_at(r >> 7, G, kb, 1, r & 127) + j)) : 0.0f;
            sw[k][r - n0] = f16_bits_to_float((uint16_t)h);
            sw[k + 1][r - n0] = f16_bits_to_float((uint16_t)(h >> 16));
        }
        for (int i = threadIdx.x; i < kMxTokens * TK / 2; i += 256) {
            const int c = i / (TK / 2), k = 2 * (i % (TK / 2));
            float v0 = 0.0f, v1 = 0.0f;
            if (c < b.rows) {
                const long long r = b.row0 + c;
                if constexpr (A16) {
                    const uint32_t hi = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(a.xq + r * a.K + k0 + k));
                    const uint32_t lo = e4m3x2_to_f16x2(
                        *reinterpret_cast<const uint16_t*>(a.xq + (long long)a.R * a.K + r * a.K + k0 + k));
                    v0 = f16_bits_to_float((uint16_t)hi) + f16_bits_to_float((uint16_t)lo) * 0.03125f;
                    v1 = f16_bits_to_float((uint16_t)(hi >> 16)) + f16_bits_to_float((uint16_t)(lo >> 16)) * 0.03125f;
                } else {
                    const uint32_t h = e2m1x2_to_f16x2(__ldg(a.xq + r * (a.K / 2) + (k0 + k) / 2));
                    v0 = f16_bits_to_float((uint16_t)h);
                    v1 = f16_bits_to_float((uint16_t)(h >> 16));
                }
                if (k == 0) fx[c] = mx_scale(__ldg(a.xs + mx_scale_at(slot, G, kb, a.nblk, c) + j));
            }
            sx[k][c] = v0;
            sx[k + 1][c] = v1;
        }
        __syncthreads();
        // The block's codes first, then both scales: neither operand alone has to be an fp32 number.
        float part[4][4] = {};
        for (int k = 0; k < TK; ++k)
            for (int m = 0; m < 4; ++m)
                for (int n = 0; n < 4; ++n) part[m][n] += sx[k][tm + 16 * m] * sw[k][tn + 16 * n];
        for (int m = 0; m < 4; ++m)
            for (int n = 0; n < 4; ++n) acc[m][n] += part[m][n] * (fx[tm + 16 * m] * fw[tn + 16 * n]);
        __syncthreads();
    }
    for (int m = 0; m < 4; ++m) {
        const int c = tm + 16 * m;
        if (c >= b.rows) break;
        long long row = b.row0 + c;
        if (a.perm) {
            row = __ldg(a.perm + row);
            if (row < 0 || row >= a.R) continue;
        }
        for (int n = 0; n < 4; ++n)
            if (n0 + tn + 16 * n < a.N) a.y[row * a.N + n0 + tn + 16 * n] = acc[m][n];
    }
}

}  // namespace

int mx_tokens(bool a16, int R, int E) {
    (void)a16; (void)R; (void)E;
    return kMxTokens;
}

cudaError_t launch_mx_gemm(const MxGemm& a, bool a16, cudaStream_t s) {
    const dim3 grid((unsigned)((a.N + TN - 1) / TN), (unsigned)mx_slots(a.R, a.offsets ? a.E : 0, a.nt));
    if (a16) k_mx_gemm<true><<<grid, 256, 0, s>>>(a);
    else k_mx_gemm<false><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ql
