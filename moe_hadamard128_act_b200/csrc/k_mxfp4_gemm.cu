// k_mxfp4_gemm.cu -- the product of MXFP4 weights, y = x~ . dequant(W)^T, over
// one weight or, rows sorted by expert, over one weight per expert, on the
// fifth-generation tensor cores' block-scaled instructions.
//
// The hardware multiplies the codes as they are stored: every 32 products along
// K share the two operands' power-of-two scales, which the instruction reads
// from tensor memory, so nothing is dequantised and one fp32 accumulator takes
// the whole K.
//   4-bit activations (kind::mxf4): both operands packed E2M1, K = 64 a step.
//   16-bit activations (kind::mxf8f6f4): the weights' codes are spread to bytes
//     by the copy engine (16 codes to 16 bytes) on their way into shared memory,
//     and x enters as two E4M3 parts with scales of their own, x = hi + lo, the
//     low parts being further operand rows: column c of the accumulator is the
//     high part's sum of token c, column n16 + c the low part's, and the
//     epilogue adds them.  A weight tile is thus read once for both.
//
// A tile is 128 weight rows (the MMA's M, tensor-memory lanes) by one token
// block (its N: the block's rows rounded up to 16, for each part), so a decode
// batch and a prefill differ in N alone.  A step is 128 bytes of every operand
// row: 256 columns of K, or 128.  A ring slot holds the step's weight codes
// (16 KB), its activation codes and both scale blocks; as many slots as shared
// and tensor memory allow keep the weights streaming.  Each slot has its own
// tensor-memory columns for its scales: they are rewritten only when the slot
// is, after the MMAs that read them have finished.  Two accumulators let the
// epilogue of one tile run under the MMAs of the next.
//
// Warp roles: warp 0 brings in the weights, which wait for nothing, warp 2 the
// activations, once the quantiser before this kernel is done (programmatic
// dependent launch); warp 1 issues the scale copies and MMAs; warps 4..7 store the sums, 32 consecutive outputs of a token
// per warp and instruction.
//
// All waits are bounded; on a timeout the CTA sets QL_DEVERR_TIMEOUT and winds
// down without leaving tensor memory allocated, MMAs running or copies in
// flight.
#include "mx_layout.cuh"
#include "ql_internal.h"

namespace ql {
namespace {

constexpr int TM = 128;              // weight rows per tile
constexpr int A_BYTES = TM * 128;    // a slot's weight codes
constexpr int BIG = 64, SMALL = 16;  // rows of the activation boxes
constexpr int kMaxStages = 12;
constexpr int kEpiWarp0 = 4, kEpiWarps = 4;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int CW = 16;  // accumulator columns per tensor-memory read
constexpr int B_FULL = 0, B_EMPTY = kMaxStages, B_ACCF = 2 * kMaxStages, B_ACCE = B_ACCF + 2, B_DRAIN = B_ACCE + 2,
              NBARS = B_DRAIN + 1;
constexpr int kSmemMax = 227 * 1024;

struct MxParams {
    CUtensorMap tmW;         // weight codes: [E * N rows], box [128 rows][128 bytes of shared memory]
    CUtensorMap tmX, tmXb;   // activation codes: [R or 2 R rows], boxes of 16 and 64 rows x 128 bytes
    MxGemm g;
    int stages, stage_bytes;  // ring
    int acc_cols, sf0, sf_cols;  // tensor memory: accumulator stride, first scale column, scale columns per slot
};

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
template <bool A16>
__device__ __forceinline__ uint32_t idesc(int n) {
    const uint32_t fmt = A16 ? (5u << 7) : (1u << 7) | (1u << 10);  // E2M1 x E4M3, or E2M1 x E2M1
    return fmt | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(TM >> 7) << 27);
}
template <bool A16>
__device__ __forceinline__ void mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t sfa, uint32_t sfb,
                                    uint32_t acc_in) {
    if constexpr (A16)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(id), "r"(sfa), "r"(sfb), "r"(acc_in));
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(id), "r"(sfa), "r"(sfb), "r"(acc_in));
}
// 512 bytes of scales: 32 rows of 16 bytes to 4 columns, the same in all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t col, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(col), "l"(desc));
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
                 : "memory");
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
};

// The CTA's tiles, each role walking the same list: tile t of all, weight block by weight block within an
// expert so that its token blocks share the weights in L2.  cum[e]: token blocks of the experts before e.
struct Tiles {
    const MxGemm& g;
    const int* cum;
    int NB, total, t;
    __device__ Tiles(const MxGemm& g_, const int* cum_) : g(g_), cum(cum_), NB((g_.N + TM - 1) / TM), t(blockIdx.x) {
        total = NB * (g.offsets ? cum[g.E] : (g.R + g.nt - 1) / g.nt);
    }
    __device__ bool next(Tile& o) {
        if (t >= total) return false;
        int e = 0, i, first = 0, count = g.R;
        if (g.offsets) {
            int hi = g.E;  // the largest e with cum[e] * NB <= t
            while (hi - e > 1) {
                const int m = (e + hi) >> 1;
                if (cum[m] * NB <= t) e = m;
                else hi = m;
            }
            const int nb = cum[e + 1] - cum[e], local = t - cum[e] * NB;
            o.wb = local / nb;
            i = local - o.wb * nb;
            int end;
            mx_segment(g.offsets, e, g.R, first, end);
            count = end - first;
        } else {
            const int nb = (g.R + g.nt - 1) / g.nt;
            o.wb = t / nb;
            i = t - o.wb * nb;
        }
        o.expert = e;
        o.row0 = first + i * g.nt;
        o.rows = min(g.nt, count - i * g.nt);
        o.slot = first / g.nt + e + i;
        t += gridDim.x;
        return true;
    }
};

template <bool A16>
__global__ void __launch_bounds__(kThreads, 1) k_mx_gemm(const __grid_constant__ MxParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[NBARS];
    __shared__ uint32_t tmem_slot;
    __shared__ int cum[1025];
    constexpr int P = A16 ? 2 : 1;      // operand rows per token
    constexpr int KBS = A16 ? 1 : 2;    // 128-column blocks per step
    const MxGemm& g = p.g;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int G = g.K / 128, KS = (G + KBS - 1) / KBS;
    const int nblk = g.nblk;
    // A slot: weight codes, activation codes, weight scales (KBS blocks), activation scales (KBS x nblk blocks).
    const int b_off = A_BYTES, sa_off = p.stage_bytes - KBS * (1 + nblk) * 512, sb_off = sa_off + KBS * 512;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bar(B_FULL + s), 2);   // the two producers' expect_tx
            mbar_init(bar(B_EMPTY + s), 1);  // the step's MMA commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(B_ACCF + b), 1);          // the tile's last commit
            mbar_init(bar(B_ACCE + b), kEpiWarps);  // one arrive per epilogue warp
        }
        mbar_init(bar(B_DRAIN), 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_slot)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    if (g.offsets) {  // token blocks of each expert, then their exclusive sums
        for (int e = threadIdx.x; e < g.E; e += kThreads) {
            int a, b;
            if (!mx_segment(g.offsets, e, g.R, a, b)) atomicOr(g.err, (unsigned)QL_DEVERR_BOUNDS);
            cum[e] = (b - a + g.nt - 1) / g.nt;
        }
        __syncthreads();
        if (warp == 3) {
            int sum = 0;
            for (int e0 = 0; e0 < g.E; e0 += 32) {
                const int v = e0 + lane < g.E ? cum[e0 + lane] : 0;
                int incl = v;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int up = __shfl_up_sync(kFull, incl, d);
                    if (lane >= d) incl += up;
                }
                if (e0 + lane < g.E) cum[e0 + lane] = sum + incl - v;
                sum += __shfl_sync(kFull, incl, 31);
            }
            if (lane == 0) cum[g.E] = sum;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)tmem_slot);
    const unsigned long long lim = wait_limit(g.err);
    bool dead = false;
    Tiles tiles(g, cum);
    Tile ti;

    // The three issuing roles run as whole warps, with every operand the same in all lanes, and one elected lane
    // issues: the instructions take their operands from uniform registers, which a lone lane's values would have
    // to be moved to one by one for each of them.
    if (warp == 0) {  // ---- weights ----
        const bool leader = elect();
        if (leader) asm volatile("prefetch.tensormap [%0];\n" ::"l"(&p.tmW) : "memory");
        const int NB = (g.N + TM - 1) / TM;
        int step = 0, s = 0, ph = 1;
        while (!dead && tiles.next(ti)) {
            const int expert = uniform(ti.expert), wb = uniform(ti.wb);
            const int row = expert * g.N + wb * TM;
            const uint8_t* sf = g.scales + ((long long)expert * NB + wb) * G * 512;
            for (int k = 0; k < KS; ++k, ++step) {
                if (!__all_sync(kFull, mbar_wait(bar(B_EMPTY + s), ph, lim))) {
                    dead = true;
                    break;
                }
                const unsigned sfb = min(KBS, G - k * KBS) * 512;
                const uint32_t slot = base + s * p.stage_bytes, fb = bar(B_FULL + s);
                if (leader) {
                    mbar_expect_tx(fb, (A16 ? A_BYTES / 2 : A_BYTES) + sfb);  // spread copies count the packed bytes
                    tma_load_2d(slot, &p.tmW, k * 128, row, fb);
                    bulk_load(slot + sa_off, sf + (long long)k * KBS * 512, sfb, fb);
                }
                if (++s == p.stages) { s = 0; ph ^= 1; }
            }
        }
        // Copies still in flight must land before the CTA's shared memory is released.  A slot's phase also
        // takes the other producer's arrival: if that one gave up, this wait ends at its bound.
        for (int j = step > p.stages ? step - p.stages : 0; j < step; ++j)
            if (!__all_sync(kFull, mbar_wait(bar(B_FULL + j % p.stages), (j / p.stages) & 1))) break;
    } else if (warp == 2) {  // ---- activations ----
        const bool leader = elect();
        if (leader) {
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(&p.tmX) : "memory");
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(&p.tmXb) : "memory");
        }
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the quantiser's codes and scales
        int step = 0, s = 0, ph = 1;
        while (!dead && tiles.next(ti)) {
            const int n16 = uniform(mx_pad16(ti.rows)), row0 = uniform(ti.row0);
            const uint8_t* sf = g.xs + (long long)uniform(ti.slot) * G * nblk * 512;
            for (int k = 0; k < KS; ++k, ++step) {
                if (!__all_sync(kFull, mbar_wait(bar(B_EMPTY + s), ph, lim))) {
                    dead = true;
                    break;
                }
                const unsigned sfb = min(KBS, G - k * KBS) * nblk * 512;
                const uint32_t slot = base + s * p.stage_bytes, fb = bar(B_FULL + s);
                if (leader) {
                    mbar_expect_tx(fb, P * n16 * 128 + sfb);
                    for (int pl = 0; pl < P; ++pl) {
                        const int row = pl * g.R + row0;
                        const uint32_t dst = slot + b_off + pl * n16 * 128;
                        int r = 0;
                        for (; r + BIG <= n16; r += BIG) tma_load_2d(dst + r * 128, &p.tmXb, k * 128, row + r, fb);
                        for (; r < n16; r += SMALL) tma_load_2d(dst + r * 128, &p.tmX, k * 128, row + r, fb);
                    }
                    bulk_load(slot + sb_off, sf + (long long)k * KBS * nblk * 512, sfb, fb);
                }
                if (++s == p.stages) { s = 0; ph ^= 1; }
            }
        }
        for (int j = step > p.stages ? step - p.stages : 0; j < step; ++j)
            if (!__all_sync(kFull, mbar_wait(bar(B_FULL + j % p.stages), (j / p.stages) & 1))) break;
    } else if (warp == 1) {  // ---- scale copies and MMAs ----
        const bool leader = elect();
        int s = 0, ph = 0, tl = 0;
        while (!dead && tiles.next(ti)) {
            const int b = tl & 1;
            if (!__all_sync(kFull, mbar_wait(bar(B_ACCE + b), ((tl >> 1) & 1) ^ 1, lim))) {  // the epilogue is done
                dead = true;
                break;
            }
            const uint32_t d = tmem + b * p.acc_cols, id0 = idesc<A16>(P * uniform(mx_pad16(ti.rows)));
            for (int k = 0; k < KS; ++k) {
                if (!__all_sync(kFull, mbar_wait(bar(B_FULL + s), ph, lim))) {
                    dead = true;
                    break;
                }
                fence_after();
                const uint32_t slot = base + s * p.stage_bytes, sf = tmem + p.sf0 + s * p.sf_cols;
                const uint32_t sfb = sf + 4 * KBS;
                const int kbs = min(KBS, G - k * KBS);
                const uint64_t ad = desc_sw128(slot), bd = desc_sw128(slot + b_off);
                const uint64_t sad = desc_scales(slot + sa_off), sbd = desc_scales(slot + sb_off);
                if (leader) {
#pragma unroll
                    for (int q = 0; q < KBS; ++q) {  // 512 bytes a copy: +32 in the descriptors' address field
                        if (q < kbs) {
                            copy_scales(sf + 4 * q, sad + 32 * q);
                            copy_scales(sfb + 4 * nblk * q, sbd + 32 * nblk * q);
                            if (nblk > 1) copy_scales(sfb + 4 * (nblk * q + 1), sbd + 32 * (nblk * q + 1));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // 32 bytes of every row: +2 in the descriptors' address field
                        const int q = A16 ? 0 : j >> 1, byte = A16 ? j : 2 * (j & 1);  // its scales' block and byte
                        if (q < kbs)
                            mma<A16>(d, ad + 2 * j, bd + 2 * j, id0 | (uint32_t)byte << 4 | (uint32_t)byte << 29,
                                     sf + 4 * q, sfb + 4 * nblk * q, (k | j) ? 1u : 0u);
                    }
                    commit(bar(B_EMPTY + s));  // the slot and its scale columns may be refilled once these are done
                }
                __syncwarp();
                if (++s == p.stages) { s = 0; ph ^= 1; }
            }
            if (dead) break;
            if (leader) commit(bar(B_ACCF + b));
            ++tl;
        }
        // Every MMA issued must finish before tensor memory is freed.
        if (leader) commit(bar(B_DRAIN));
        __all_sync(kFull, mbar_wait(bar(B_DRAIN), 0));
    } else if (warp >= kEpiWarp0) {  // ---- epilogue ----
        const int q = warp & 3;
        int tl = 0;
        while (tiles.next(ti)) {
            const int b = tl & 1, n16 = mx_pad16(ti.rows);
            const int n = ti.wb * TM + 32 * q + lane;
            const uint32_t d = tmem + b * p.acc_cols + ((uint32_t)(32 * q) << 16);
            if (!__all_sync(kFull, mbar_wait(bar(B_ACCF + b), (tl >> 1) & 1, lim))) {  // together
                dead = true;
                break;
            }
            fence_after();
            for (int c0 = 0; c0 < ti.rows; c0 += CW) {
                uint32_t v[CW], lo[CW];
                tmem_ld16(d + c0, v);
                if constexpr (A16) tmem_ld16(d + n16 + c0, lo);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < CW; ++i) {
                    if (c0 + i >= ti.rows) break;
                    long long row = ti.row0 + c0 + i;
                    if (g.perm) {
                        row = __ldg(g.perm + row);
                        if (row < 0 || row >= g.R) continue;
                    }
                    float f = __uint_as_float(v[i]);
                    if constexpr (A16) f += __uint_as_float(lo[i]);
                    if (n < g.N) g.y[row * g.N + n] = f;
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) arrive(bar(B_ACCE + b));
            ++tl;
        }
    }
    if (dead) atomicOr(g.err, (unsigned)QL_DEVERR_TIMEOUT);

    fence_before();
    __syncthreads();
    if (warp == 2) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols));
    }
}

template <bool A16>
cudaError_t run(const MxGemm& g, cudaStream_t s) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    constexpr int P = A16 ? 2 : 1, KBS = A16 ? 1 : 2;
    MxParams p;
    p.g = g;
    const int rows = P * g.nt;  // operand rows of a full token block
    p.stage_bytes = (int)align_up(A_BYTES + rows * 128 + KBS * (1 + g.nblk) * 512, 1024);
    p.acc_cols = (int)align_up(rows, 32);
    p.sf0 = 2 * p.acc_cols;
    p.sf_cols = KBS * 4 * (1 + g.nblk);
    const int smem_max = (int)(di.smem_optin < (size_t)kSmemMax ? di.smem_optin : kSmemMax) - 8 * 1024;
    p.stages = (smem_max - 1024) / p.stage_bytes;
    if (p.stages > ((int)kTmemCols - p.sf0) / p.sf_cols) p.stages = ((int)kTmemCols - p.sf0) / p.sf_cols;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    if (p.stages < 2) return cudaErrorInvalidValue;
    const int smem = p.stages * p.stage_bytes + 1024;
    const long long wrows = (long long)g.E * g.N, xrows = (long long)P * g.R, xbytes = A16 ? g.K : g.K / 2;
    e = A16 ? make_tmap_u4_spread(g.codes, wrows, g.K, TM, &p.tmW)
            : make_tmap_2d(g.codes, wrows, g.K / 2, g.K / 2, 128, TM, CU_TENSOR_MAP_SWIZZLE_128B, &p.tmW);
    if (e == cudaSuccess) e = make_tmap_2d(g.xq, xrows, xbytes, xbytes, 128, SMALL, CU_TENSOR_MAP_SWIZZLE_128B, &p.tmX);
    if (e == cudaSuccess) e = make_tmap_2d(g.xq, xrows, xbytes, xbytes, 128, BIG, CU_TENSOR_MAP_SWIZZLE_128B, &p.tmXb);
    if (e != cudaSuccess) return e;

    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(k_mx_gemm<A16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax - 8 * 1024);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    const long long tiles = (long long)((g.N + TM - 1) / TM) * mx_slots(g.R, g.offsets ? g.E : 0, g.nt);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles < di.sm_count ? tiles : di.sm_count));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;  // after this library's quantiser
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_mx_gemm<A16>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Rows of a token block: the widest the accumulators allow, cut evenly over one weight's rows; for experts
// twice the average count, so that most experts are one block (a block costs its own rows alone, but a second
// one reads the weights again).
int mx_tokens(bool a16, int R, int E) {
    const int most = a16 ? kMxTokens / 2 : kMxTokens;
    if (!E) {
        const int blocks = (int)(((long long)R + most - 1) / most);
        return mx_pad16((int)(((long long)R + blocks - 1) / blocks));
    }
    const long long avg2 = (2LL * R + E - 1) / E;
    return avg2 >= most ? most : mx_pad16((int)avg2);
}

cudaError_t launch_mx_gemm(const MxGemm& g, bool a16, cudaStream_t s) { return a16 ? run<true>(g, s) : run<false>(g, s); }

}  // namespace ql
