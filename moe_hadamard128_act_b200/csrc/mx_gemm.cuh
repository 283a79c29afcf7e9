// mx_gemm.cuh -- what the two MXFP4 product kernels share: descriptors of the
// block-scaled tensor-core instructions, the list of tiles that every role of a
// kernel walks, and the epilogue.
#pragma once

#include "mx_layout.cuh"

namespace ql {
namespace {

constexpr int TM = 128;              // weight rows per CTA and tile: tensor-memory lanes
constexpr int A_BYTES = TM * 128;    // a step's weight codes
constexpr int BIG = 64, SMALL = 16;  // rows of the activation boxes
constexpr int kMaxStages = 12;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int CW = 16;  // accumulator columns per tensor-memory read
constexpr int kSmemMax = 215 * 1024;  // dynamic shared memory of a CTA at most

__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
    // K-major, 128-byte swizzle: 8-row atoms 1024 bytes apart (SBO), version 1.
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
    // No swizzle: 8 rows of 16 bytes, 128 bytes apart.
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (8ull << 32) | (1ull << 46);
}
// Block-scaled kinds: A format at bits 7-9, B format at 10-12, N >> 3 at 17-22, scales UE8M0 (bit 23), M >> 7 at
// 27-28; the scales' byte within a tensor-memory word at 4-5 (B) and 29-30 (A).
template <int MODE>
__device__ __forceinline__ uint32_t idesc(int m, int n) {
    const uint32_t fmt = MODE == kMxParts ? (5u << 7) : (1u << 7) | (1u << 10);  // E2M1 x E4M3, or E2M1 x E2M1
    return fmt | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27);
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t r[CW]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }

// One lane of a converged warp, the same every time.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kFull, v, 0); }

struct Tile {
    int expert, row0, rows, wb, slot;
    int k0, k1;  // its steps
};

// What the CTA knows of the experts' segments.
struct Routing {
    int cum[1025];             // token blocks of the experts before e
    int offsets[1025];         // of ids: the segments,
    int perm[kMxFusedPairs];   // and the pairs in sorted order
    int ids[kMxFusedPairs];
};
__device__ __forceinline__ bool grouped(const MxGemm& g) { return g.offsets || g.ids; }
__device__ __forceinline__ void segment(const MxGemm& g, const Routing& rt, int e, int& a, int& b) {
    if (g.ids) {
        a = rt.offsets[e];
        b = rt.offsets[e + 1];
    } else {
        mx_segment(g.offsets, e, g.R, a, b);
    }
}

// The tiles of unit `id` of `units` (a CTA, or a pair of them), each role walking the same list: weight block (of
// TR rows) by weight block within an expert so that its token blocks share the weights in L2.  With `split` tiles may be
// cut along K between two units.  Pairs cut those from g.plan.halves on in half along K.
template <int TR>
struct Tiles {
    static constexpr bool PAIR = TR > TM;
    const MxGemm& g;
    const Routing& rt;
    int NB, KS, units, total, t, whole;  // pairs: t counts halves from `whole` on
    long long u, end;  // split: the unit's run of steps
    __device__ Tiles(const MxGemm& g_, const Routing& rt_, int KS_, int id, int units_, bool split)
        : g(g_), rt(rt_), NB((g_.N + TR - 1) / TR), KS(KS_), units(units_), t(id), u(-1), end(0) {
        total = NB * (grouped(g) ? rt.cum[g.E] : (g.R + g.plan.nt - 1) / g.plan.nt);
        if constexpr (PAIR) {
            whole = min(total, g.plan.halves);
            total += total - whole;
        }
        // Runs of whole tiles lose up to a tile's time in the last round; past eight rounds that is little.
        if (split && (2 * total <= units || (total > units && total < 8 * units && total % units))) {
            const int parts = 2 * total <= units ? 2 * total : units;
            const long long steps = (long long)total * KS, c = id;
            u = c < parts ? c * steps / parts : 0;
            end = c < parts ? (c + 1) * steps / parts : 0;
        }
    }
    __device__ bool next(Tile& o) {
        int tile = t;
        o.k0 = 0;
        o.k1 = KS;
        if (u >= 0) {
            if (u >= end) return false;
            tile = (int)(u / KS);
            o.k0 = (int)(u - (long long)tile * KS);
            o.k1 = (int)min((long long)KS, o.k0 + (end - u));
            u += o.k1 - o.k0;
        } else {
            if (t >= total) return false;
            if (PAIR && t >= whole) {
                tile = whole + ((t - whole) >> 1);
                if ((t - whole) & 1) o.k0 = KS >> 1;
                else o.k1 = KS >> 1;
            }
            t += units;
        }
        int e = 0, i, first = 0, count = g.R;
        if (grouped(g)) {
            int hi = g.E;  // the largest e with cum[e] * NB <= tile
            while (hi - e > 1) {
                const int m = (e + hi) >> 1;
                if (rt.cum[m] * NB <= tile) e = m;
                else hi = m;
            }
            const int nb = rt.cum[e + 1] - rt.cum[e], local = tile - rt.cum[e] * NB;
            o.wb = local / nb;
            i = local - o.wb * nb;
            int last;
            segment(g, rt, e, first, last);
            count = last - first;
        } else {
            const int nb = (g.R + g.plan.nt - 1) / g.plan.nt;
            o.wb = tile / nb;
            i = tile - o.wb * nb;
        }
        o.expert = e;
        o.row0 = first + i * g.plan.nt;
        o.rows = min(g.plan.nt, count - i * g.plan.nt);
        o.slot = first / g.plan.nt + e + i;
        return true;
    }
};

// Token blocks of each expert, then their exclusive sums: cum[e], e <= E; of ids, the segments and the sorted order
// first (stable: by expert, then by pair).  By the whole CTA; the sums are there after the caller's next barrier.
__device__ __forceinline__ void route(const MxGemm& g, Routing& rt, int warp, int lane) {
    int* const cum = rt.cum;
    if (g.ids) {
        // ids in shared memory, 128 of them with the missing ones out of range; each thread counts for its experts,
        // then for its pair.
        if (threadIdx.x < kMxFusedPairs) {
            const int e = threadIdx.x < g.R ? __ldg(g.ids + threadIdx.x) : -1;
            rt.ids[threadIdx.x] = e >= 0 && e < g.E ? e : g.E;
        }
        __syncthreads();
        const int n = (g.R + 7) & ~7;
        for (int e = threadIdx.x; e <= g.E; e += kThreads) {
            int below = 0, size = 0;
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                below += rt.ids[i] < e;
                size += rt.ids[i] == e;
            }
            rt.offsets[e] = below;
            if (e < g.E) cum[e] = (size + g.plan.nt - 1) / g.plan.nt;
        }
        if (threadIdx.x < g.R) {
            const int p = threadIdx.x, e = rt.ids[p];
            int r = 0;
#pragma unroll 8
            for (int i = 0; i < n; ++i) r += rt.ids[i] < e || (rt.ids[i] == e && i < p);
            if (e < g.E) rt.perm[r] = p;
        }
    } else {
        for (int e = threadIdx.x; e < g.E; e += kThreads) {
            int a, b;
            if (!mx_segment(g.offsets, e, g.R, a, b)) atomicOr(g.err, (unsigned)QL_DEVERR_BOUNDS);
            cum[e] = (b - a + g.plan.nt - 1) / g.plan.nt;
        }
    }
    __syncthreads();
    if (warp != 3) return;
    // A lane adds up a run of experts.  Sound segments make no more than `most` blocks.  Overlapping ones (offsets out
    // of order) could make more tiles than a count holds: then there are none.
    const int most = g.R / g.plan.nt + g.E, run = (g.E + 31) >> 5, e0 = min(lane * run, g.E), e1 = min(e0 + run, g.E);
    long long own = 0;
    for (int e = e0; e < e1; ++e) own += cum[e];
    const int mine = (int)min(own, (long long)most + 1);
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl = min(incl + up, most + 1);
    }
    const int sum = __shfl_sync(kFull, incl, 31);
    int at = sum > most ? 0 : incl - mine;
    for (int e = e0; e < e1; ++e) {
        const int v = sum > most ? 0 : cum[e];
        cum[e] = at;
        at += v;
    }
    if (lane == 0) cum[g.E] = sum > most ? 0 : sum;
}

// The epilogue of one tile in two halves, for warp kEpiWarp0 + w: lanes 32 (w % 4) .. + 31 of the accumulator are
// weight rows, i.e. consecutive outputs of a token; the two warps of a lane quarter take every second read.
// ROWS: operand rows of a block at most.
template <int MODE, int ROWS>
struct Epilogue {
    static constexpr bool PARTS = MODE == kMxParts;
    static constexpr int TW = MODE == kMxDigits ? CW / 8 : CW;        // tokens of a tensor-memory read
    static constexpr int READS = ROWS / mx_planes(MODE) / TW / 2;     // this warp's
    static constexpr int REGS = (READS * TW + 31) / 32;
    int to[REGS];
    float factor[REGS];

    // Before the sums are ready: lane l fetches the output rows (-1: none) of the tokens number 32 i + l of this
    // warp's.
    __device__ __forceinline__ void fetch(const MxGemm& g, const Routing& rt, const Tile& ti, int h, int lane) {
#pragma unroll
        for (int i = 0; i < REGS; ++i) {
            const int m = 32 * i + lane, c = (2 * (m / TW) + h) * TW + m % TW;
            to[i] = -1;
            factor[i] = 1.0f;
            if (c < ti.rows) {
                to[i] = ti.row0 + c;
                if constexpr (MODE == kMxDigits) factor[i] = g.xf[to[i]];
                if (g.ids) {
                    to[i] = rt.perm[to[i]];
                } else if (g.perm) {
                    to[i] = __ldg(g.perm + to[i]);
                    if (to[i] >= g.R) to[i] = -1;
                }
            }
        }
    }

    // This warp's sums of the accumulator whose first column in its lanes is d, as bits: sum[j][i] is that of its
    // token number TW j + i.  The accumulator is free once every warp has returned.
    uint32_t sum[READS][TW];
    __device__ __forceinline__ void drain(const Tile& ti, uint32_t d, int h) {
        const int n16 = mx_pad16(ti.rows);
#pragma unroll
        for (int j = 0; j < READS; ++j) {
            const int c0 = (2 * j + h) * TW;
            if (c0 >= ti.rows) break;
            if constexpr (MODE == kMxA4) {
                tmem_ld16(d + c0, sum[j]);  // there after the wait below
            } else if constexpr (PARTS) {
                uint32_t v[CW], lo[CW];
                tmem_ld16(d + c0, v);
                tmem_ld16(d + n16 + c0, lo);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < TW; ++i) sum[j][i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(lo[i]));
            } else {
                uint32_t v[CW];
                tmem_ld16(d + 8 * c0, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < TW; ++i) {  // small digits first
                    const uint32_t* w = v + 8 * i;
                    sum[j][i] = __float_as_uint((__uint_as_float(w[0]) + __uint_as_float(w[1])) +
                                                ((__uint_as_float(w[2]) + __uint_as_float(w[3])) +
                                                 ((__uint_as_float(w[4]) + __uint_as_float(w[5])) +
                                                  (__uint_as_float(w[6]) + __uint_as_float(w[7])))));
                }
            }
        }
        if constexpr (MODE == kMxA4) tmem_wait_ld();
    }

    // n: this lane's output; add: the sums are of a part of K.
    __device__ __forceinline__ void store(const MxGemm& g, const Tile& ti, int h, int n, bool add) const {
#pragma unroll
        for (int j = 0; j < READS; ++j) {
            if ((2 * j + h) * TW >= ti.rows) break;
#pragma unroll
            for (int i = 0; i < TW; ++i) {
                const int m = j * TW + i;
                const int row = __shfl_sync(kFull, to[m / 32], m % 32);
                float s = __uint_as_float(sum[j][i]);
                if constexpr (MODE == kMxDigits) s *= __shfl_sync(kFull, factor[m / 32], m % 32);
                float* const y = g.y + (long long)row * g.N + n;
                if (row >= 0 && n < g.N) {
                    if (add) atomicAdd(y, s);
                    else *y = s;
                }
            }
        }
    }
};

}  // namespace
}  // namespace ql
