// k_mxfp4.cu -- microscaled 4-bit floating point (MXFP4): the quantisers of
// weights and activations, the packer of given codes, and the values that
// packed codes stand for.
//
// Eight lanes take one row's 128 columns, 16 neighbouring values a lane (one
// 32-byte load of bf16): the rotation's shuffles stay inside the eight, a
// 32-block is 2 lanes, and the 128 columns' four scale bytes are one word of
// the scale layout (mx_layout.cuh).  With half as many values a lane the work
// around the values, not the memory, set the time (16384 x 5376 and back 82 us
// against 77).  Bound by HBM: 2 (bf16) or 4 (fp32) bytes in and 17/32 byte out
// per value; with the way back 5.8 TB/s.
#include "mx_layout.cuh"
#include "ql_internal.h"

namespace ql {
namespace {

constexpr int kWarps = 8;
// Warps of the activations' kernel (8: 1 to 2 us slower from 1600 rows on, with the last pass half empty).
constexpr int kActWarps = 4;

// 32 bytes, read once; one load if the tensor is 32-byte aligned (rows are whole multiples of that), else two.
__device__ __forceinline__ void ldg32(const void* p, bool wide, uint32_t w[8]) {
    if (wide) {
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}
__device__ __forceinline__ bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
// A lane's 16 values as they are loaded, and in fp32.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    uint32_t w[16];
    __device__ __forceinline__ void load(const float* p, bool wide) {
        ldg32(p, wide, w);
        ldg32(p + 8, wide, w + 8);
    }
    __device__ __forceinline__ void get(float v[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
    }
};
template <>
struct Raw<__nv_bfloat16> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const __nv_bfloat16* p, bool wide) { ldg32(p, wide, w); }
    __device__ __forceinline__ void get(float v[16]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

// Rows [0, N) of W to packed MXFP4; rows up to the next multiple of 128 get zero scales.  A CTA takes kRows
// rows and walks them 128 columns to eight lanes, all rows' loads of a column first.
constexpr int kRows = 2;  // 4: registers halve the warps, pack 121 us against 103 at 21504 x 5376
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_mx_quant(const T* W, int N, int K, int rotate, uint8_t* codes,
                                                          uint8_t* scales) {
    const int lane = threadIdx.x & 7, G = K / 128;
    const bool wide = aligned32(W);
    const int r0 = blockIdx.x * kRows;
    // every lane of a warp goes through the same iterations (the shuffles want all of them)
    for (int g0 = (blockIdx.y * kWarps + (threadIdx.x >> 5)) * 4; g0 < G; g0 += gridDim.y * kWarps * 4) {
        const int g = g0 + ((threadIdx.x >> 3) & 3);
        const int gl = min(g, G - 1);
        Raw<T> raw[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) raw[i].load(W + (long long)min(r0 + i, N - 1) * K + gl * 128 + 16 * lane, wide);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i;
            float v[16];
            raw[i].get(v);
            if (rotate) mx_fwht128(v, lane);
            uint32_t byte;
            const uint2 c = mx_quant16(v, byte);
            uint32_t word = mx_scale_word(byte, lane);
            if (g >= G) continue;
            if (r < N) *reinterpret_cast<uint2*>(codes + (long long)r * (K / 2) + g * 64 + 8 * lane) = c;
            else word = 0;
            if (lane == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_at(r >> 7, G, g, 1, r & 127)) = word;
        }
    }
}

// Activations into the order of the product's tiles (mx_layout.cuh).  A CTA takes 128-column units of one row
// of x, quantised once and written to every place that the row has among the sorted rows: its own (offsets
// null, or sorted rows given), or one for each of the token's topk pairs, at the pair's position inv[] in its
// expert's segment.  Up to kMxFusedPairs pairs come without a permutation: every CTA counts its pairs' places
// from the ids and flags those with an id outside [0, E).  The outputs of pairs of no expert are zeroed here.
struct Place {
    uint8_t *codes, *scale, *low;  // where the row's codes, its scales and its low part's scales begin
    float* y;                      // its output
    int row, c;                    // sorted row (-1: none), token of its block
};

// Digits: 32, and a factor of 2^-32 on the row's sums, if no magnitude of the row (rotated and rounded as the
// quantiser sees it) reaches 2^-64, else 0; by a whole warp.  The digits' scales end at 2^-127, which rounds a
// block below 2^-105 to multiples of that; beside a value of 2^-64 the loss is at most 2^-64 of it, and without one the
// row is moved up.
constexpr uint32_t kSmallRow = 63u << 23;  // 2^-64
__device__ __noinline__ int row_up(const __nv_bfloat16* x, int G, int rotate) {
    const int lane = threadIdx.x & 7;
    uint32_t m = 0;
    for (int g0 = 0; g0 < G; g0 += 4) {
        Raw<__nv_bfloat16> raw;
        raw.load(x + min(g0 + (int)((threadIdx.x >> 3) & 3), G - 1) * 128 + 16 * lane, aligned32(x));
        float v[16];
        raw.get(v);
        if (rotate) mx_fwht128(v, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(__bfloat162float(__float2bfloat16_rn(v[i]))) & 0x7FFFFFFFu);
    }
    return __reduce_max_sync(kFull, m) < kSmallRow ? 32 : 0;
}

template <int MODE>
__global__ void __launch_bounds__(kActWarps * 32) k_mx_act(const MxAct a) {
    // Launched while the kernel before it ends: nothing is read or written before that one is done, and only then
    // may the product start its weight stream, which waits for nothing else.
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    __shared__ Place places[kMxTopk];
    const int G = a.K / 128, x = blockIdx.x, nt = a.plan.nt, nblk = a.plan.nblk;
    const int dests = a.ids ? a.topk : 1;
    const int lane = threadIdx.x & 7;
    const __nv_bfloat16* const xr = a.x + (long long)x * a.K;
    const bool wide = aligned32(a.x);
    int g0 = (blockIdx.y * kActWarps + (threadIdx.x >> 5)) * 4;
    Raw<__nv_bfloat16> raw;  // the next unit's values: on their way while the places are worked out
    auto load = [&]() { raw.load(xr + min(g0 + (int)((threadIdx.x >> 3) & 3), G - 1) * 128 + 16 * lane, wide); };
    load();
    // Place j: pair (or row) y, at sorted row r of expert e's segment [first, end); r < 0: none.
    auto place = [&](int j, long long y, int r, int e, int first, int end) {
        if (r < first || r >= end) r = -1;
        const int i = r < 0 ? 0 : (r - first) / nt, c = r < 0 ? 0 : (r - first) - i * nt;
        const long long slot = first / nt + e + i;
        const int low = mx_pad16(min(nt, end - first - i * nt)) + c;
        const long long at = MODE == kMxA4 ? (long long)r * (a.K / 2)
                                           : MODE == kMxDigits ? 4LL * r * a.K : (long long)r * a.K;
        places[j] = Place{a.codes + at, a.scales + mx_scale_at(slot, G, 0, nblk, MODE == kMxDigits ? 0 : c),
                          a.scales + mx_scale_at(slot, G, 0, nblk, low), a.y + y * a.N, r, c};
    };
    if (a.ids && a.inv) {  // a thread a pair
        if ((int)threadIdx.x < dests) {
            const long long y = (long long)x * a.topk + threadIdx.x;
            int r = __ldg(a.inv + y), first = 0, end = 0;
            const int e = __ldg(a.ids + y);
            if (e >= 0 && e < a.E) mx_segment(a.offsets, e, a.R, first, end);
            place(threadIdx.x, y, r, e, first, end);
        }
    } else if (a.ids) {  // few pairs: a warp a pair, its place among all by counting
        for (int j = threadIdx.x >> 5; j < dests; j += kActWarps) {
            const long long y = (long long)x * a.topk + j;
            const int e = __ldg(a.ids + y);
            int below = 0, size = 0, rank = 0;
            for (int i = threadIdx.x & 31; i < a.R; i += 32) {
                const int o = __ldg(a.ids + i);
                below += o >= 0 && o < e;
                size += o == e;
                rank += o == e && i < y;
            }
            const int first = __reduce_add_sync(kFull, below), end = first + __reduce_add_sync(kFull, size);
            rank = __reduce_add_sync(kFull, rank);
            const bool ok = e >= 0 && e < a.E;
            if ((threadIdx.x & 31) == 0) place(j, y, ok ? first + rank : -1, e, first, end);
            if (!ok && (threadIdx.x & 31) == 0) atomicOr(a.err, (unsigned)QL_DEVERR_EXPERT_ID);
        }
    } else if (threadIdx.x < 32) {
        int e = 0, first = 0, end = a.R;
        if (a.offsets) e = mx_expert_of(a.offsets, a.E, a.R, x, first, end);
        if (threadIdx.x == 0) place(0, x, x, e, first, end);
    }
    __syncthreads();
    for (int j = 0; j < dests; ++j) {
        // Zeroed: what the product adds into, and the rows of pairs that no expert takes.
        const bool none = places[j].row < 0;
        if (none && !a.ids) continue;
        float* const y = places[j].y;
        for (int n = (none ? 0 : a.plan.zero) + blockIdx.y * blockDim.x + threadIdx.x; n < a.N; n += gridDim.y * blockDim.x) y[n] = 0.0f;
    }
    if (dests == 1 && places[0].row < 0) return;
    while (g0 < G) {
        const int g = g0 + ((threadIdx.x >> 3) & 3);
        const bool first_unit = g0 == 0;
        float v[16];
        raw.get(v);
        g0 += gridDim.y * kActWarps * 4;
        if (g0 < G) load();  // the next unit's values are on their way while this one is worked on
        if (a.rotate) {
            mx_fwht128(v, lane);
            if constexpr (MODE != kMxA4) {
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __bfloat162float(__float2bfloat16_rn(v[k]));
            }
        }
        uint32_t byte, d0[8], d1[8];
        uint2 c;
        uint4 hi, lo;
        if constexpr (MODE == kMxA4) {
            c = mx_quant16(v, byte);
        } else if constexpr (MODE == kMxParts) {
            mx_split16(v, hi, lo, byte);
        } else {
            const uint32_t m = mx_block_max(v);
            // Blocks of ordinary size settle that the row is not a small one; zeros fit any factor.  The row's
            // first block answers for the row, whatever it holds.
            int up = 0;
            if (__any_sync(kFull, m < kSmallRow && (m || first_unit))) up = row_up(xr, G, a.rotate);
            if (first_unit && (threadIdx.x & 31) == 0)
                for (int j = 0; j < dests; ++j)
                    if (places[j].row >= 0) a.factors[places[j].row] = up ? 0x1p-32f : 1.0f;
            byte = mx_digits_byte(m >> 23, up);
            mx_digits8(v, byte, up, d0);
            mx_digits8(v + 8, byte, up, d1);
        }
        const uint32_t word = mx_scale_word(byte, lane);
        const uint32_t lword = MODE == kMxParts ? mx_scale_word(byte == 255 ? 255u : byte - 5u, lane) : 0u;
        uint32_t dword = 0;  // digits: lane p holds digit p's four scales, each 3 p below the first's
        if constexpr (MODE == kMxDigits) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t b = (word >> (8 * k)) & 0xFFu;
                dword |= (b == 255 ? 255u : b - 3u * lane) << (8 * k);
            }
        }
        if (g >= G) continue;
        for (int j = 0; j < dests; ++j) {
            const Place p = places[j];
            if (p.row < 0) continue;
            const long long sf = (long long)g * nblk * 512;
            if constexpr (MODE == kMxA4) {
                *reinterpret_cast<uint2*>(p.codes + g * 64 + 8 * lane) = c;
                if (lane == 0) *reinterpret_cast<uint32_t*>(p.scale + sf) = word;
            } else if constexpr (MODE == kMxParts) {
                uint8_t* const at = p.codes + g * 128 + 16 * lane;
                *reinterpret_cast<uint4*>(at) = hi;
                *reinterpret_cast<uint4*>(at + (long long)a.R * a.K) = lo;
                if (lane == 0) *reinterpret_cast<uint32_t*>(p.scale + sf) = word;
                if (lane == 1) *reinterpret_cast<uint32_t*>(p.low + sf) = lword;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint2*>(p.codes + (long long)k * (a.K / 2) + g * 64 + 8 * lane) =
                        make_uint2(d0[k], d1[k]);
                *reinterpret_cast<uint32_t*>(p.scale + sf + mx_scale_at(0, G, 0, nblk, 8 * p.c + lane)) = dword;
            }
        }
    }
}

// The (token, slot) pairs in (expert, pair) order: offsets[E + 1], perm[P], inv[P], as moe_permute makes them, without
// its counts, chunks and tiles.  A CTA an expert, and one more for the pairs of no expert, which flags them and
// fills the tail of perm with -1.  Every CTA reads all ids, each warp a run of them 128 at a time:
// first it counts its expert's pairs and those of the experts before, then, knowing the other warps' counts, it
// writes.  Bound by latency: 16384 pairs of 128 experts take 6 us less than moe_permute's histogram.
constexpr int kRouteWarps = 16;
__global__ void __launch_bounds__(kRouteWarps * 32) k_mx_route(const int32_t* ids, int P, int E, int32_t* offsets,
                                                               int32_t* perm, int32_t* inv, unsigned* err) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // the quantiser may stand by
    __shared__ int mine_of[kRouteWarps], below_of[kRouteWarps];
    const int e = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = (P + kRouteWarps * 128 - 1) / (kRouteWarps * 128) * 128;
    const int p0 = warp * run, p1 = min(P, p0 + run);
    // This lane's four ids of the 128 from p on (E: none, or of no expert; E + 1: past the end).
    auto load = [&](int p, int id[4]) {
        const int q = p + 4 * lane;
        if (q + 3 < P) {
            const int4 v = __ldg(reinterpret_cast<const int4*>(ids + q));
            id[0] = v.x; id[1] = v.y; id[2] = v.z; id[3] = v.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) id[k] = q + k < P ? __ldg(ids + q + k) : E + 1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (q + k < P && (id[k] < 0 || id[k] >= E)) id[k] = E;
    };
    int mine = 0, below = 0;
#pragma unroll 4
    for (int p = p0; p < p1; p += 128) {
        int id[4];
        load(p, id);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mine += id[k] == e;
            below += id[k] < e;
        }
    }
    mine = __reduce_add_sync(kFull, mine);
    below = __reduce_add_sync(kFull, below);
    if (lane == 0) {
        mine_of[warp] = mine;
        below_of[warp] = below;
    }
    __syncthreads();
    int at = 0;  // the sorted row of this warp's first pair
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) at += below_of[w] + (w < warp ? mine_of[w] : 0);
    if (threadIdx.x == 0) offsets[e] = at;  // warp 0: the expert's first row; of E: the number of routed pairs
    if (mine) {
        int next = at;
        for (int p = p0; p < p1; p += 128) {
            int id[4], n = 0;
            load(p, id);
#pragma unroll
            for (int k = 0; k < 4; ++k) n += id[k] == e;
            if (!__any_sync(kFull, n)) continue;
            int incl = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(kFull, incl, d);
                if (lane >= d) incl += up;
            }
            int r = next + incl - n;
            next += __shfl_sync(kFull, incl, 31);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (id[k] != e) continue;
                const int q = p + 4 * lane + k;
                if (e < E) {
                    perm[r] = q;
                    inv[q] = r++;
                } else {
                    inv[q] = -1;
                }
            }
        }
    }
    if (e == E) {
        int bad = 0, first = 0;
#pragma unroll
        for (int w = 0; w < kRouteWarps; ++w) {
            bad += mine_of[w];
            first += below_of[w];
        }
        if (bad && threadIdx.x == 0) atomicOr(err, (unsigned)QL_DEVERR_EXPERT_ID);
        for (int i = first + threadIdx.x; i < P; i += kRouteWarps * 32) perm[i] = -1;
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

// 8 codes of kRows rows a thread: 4 bytes in, 16 bytes of bf16 out.  The f16 value of a code times a power of
// two has two significant bits, so the fp32 product and its rounding to bf16 are exact.
__global__ void __launch_bounds__(256) k_mx_dequant(const uint8_t* codes, const uint8_t* scales, int N, int K,
                                                    __nv_bfloat16* out) {
    const int r0 = blockIdx.x * kRows, G = K / 128;
    for (int u = threadIdx.x; u < K / 8; u += 256) {
        uint32_t w[kRows], b[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = min(r0 + i, N - 1);
            w[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + (long long)r * (K / 2)) + u);
            b[i] = __ldg(scales + mx_scale_at(r >> 7, G, u >> 4, 1, r & 127) + ((u >> 2) & 3));
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float s = mx_scale(b[i]);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t h = e2m1x2_to_f16x2((w[i] >> (8 * j)) & 0xFFu);
                const __nv_bfloat162 p = __floats2bfloat162_rn(f16_bits_to_float((uint16_t)h) * s,
                                                               f16_bits_to_float((uint16_t)(h >> 16)) * s);
                o[j] = *reinterpret_cast<const uint32_t*>(&p);
            }
            if (r0 + i < N)
                reinterpret_cast<uint4*>(out + (long long)(r0 + i) * K)[u] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

int cuts(int passes) { return passes < 65535 ? passes : 65535; }  // the grid's limit

template <typename T>
cudaError_t quant(const T* W, int N, int K, int rotate, uint8_t* codes, uint8_t* scales, cudaStream_t s) {
    const int blocks = (N + 127) / 128 * (128 / kRows), passes = (K / 128 + 4 * kWarps - 1) / (4 * kWarps);
    const dim3 grid((unsigned)blocks, (unsigned)(blocks < 148 ? cuts(passes) : 1));  // few rows: cut along K too
    k_mx_quant<T><<<grid, kWarps * 32, 0, s>>>(W, N, K, rotate, codes, scales);
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

cudaError_t launch_mx_route(const int32_t* ids, int P, int E, int32_t* offsets, int32_t* perm, int32_t* inv,
                            unsigned* err, cudaStream_t s) {
    // Not as a dependent launch: its blocks, waiting beside the product before them, cost that 6 of 87 us.
    k_mx_route<<<E + 1, kRouteWarps * 32, 0, s>>>(ids, P, E, offsets, perm, inv, err);
    return cudaGetLastError();
}

cudaError_t launch_mx_act(const MxAct& a, cudaStream_t s) {
    // One CTA a row; few rows are cut along K instead, so that their columns are not walked one after another.
    const int rows = a.ids ? a.R / a.topk : a.R, passes = (a.K / 128 + 4 * kActWarps - 1) / (4 * kActWarps);
    const dim3 grid((unsigned)rows, (unsigned)(rows < 148 ? cuts(passes) : 1));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kActWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, a.plan.mode == kMxA4       ? k_mx_act<kMxA4>
                                                   : a.plan.mode == kMxDigits ? k_mx_act<kMxDigits>
                                                                              : k_mx_act<kMxParts>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
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
    k_mx_dequant<<<(unsigned)((N + kRows - 1) / kRows), 256, 0, s>>>(codes, scales, N, K,
                                                                   static_cast<__nv_bfloat16*>(out));
    return cudaGetLastError();
}

}  // namespace ql
