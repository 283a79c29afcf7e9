// k_mxfp4_pair.cu -- the MXFP4 product (k_mxfp4_gemm.cu) for token blocks of many
// rows, two CTAs to a tile.
//
// With many tokens the operand stream into shared memory bounds the product: a
// CTA alone brings 16 KB of weights and up to 24 KB of activations for 256
// columns of K, twice the time that its MMAs take.  A pair of CTAs on
// neighbouring SMs (tcgen05 cta_group::2) multiplies 256 weight rows by the same
// token block: each brings its own 128 weight rows and half of the block's
// operand rows, and the hardware reads both halves, so every CTA brings 28 KB
// instead of 40.  Each CTA's tensor memory holds the sums of its own weight rows,
// so the epilogue is the single CTA's.
//
// 16-bit activations of many rows come here as two E4M3 parts with scales of their
// own (kind::mxf8f6f4), x = hi + lo, the low parts being further operand rows:
// column c of the accumulator is the high part's sum of token c, column n16 + c the
// low part's, and the epilogue adds them.  The weights' codes are spread to bytes by
// the copy engine (16 codes to 16 bytes) on their way into shared memory.  A quarter
// of the digits' tensor work at half its rate, but the spreading copy brings only
// half as many codes a second, which is what few rows wait for.
//
// The even CTA's warp 3 issues all copies of scales to tensor memory and its
// warp 1 all MMAs, a warp each because a step's six copies and four MMAs take one
// warp longer to issue (about 32 cycles each, 800 a step with the waits) than the
// tensor cores need for them; both CTAs' loads complete on its barriers, and
// its commits arrive at the barriers of both.
// Scale blocks: each CTA brings those of its own weight rows and all of the
// activations', which the copies to tensor memory put into both CTAs' columns.
// Token blocks of up to 192 operand rows have two accumulators, so that an
// epilogue runs under the next tile's MMAs.  A block of 256, which reads fewer
// operand bytes a product, fills half of the tensor memory with one: its epilogue
// takes the sums into registers, gives the accumulator back and then stores.
//
// The tiles of one weight's last round, if they would leave half of the pairs idle, may be cut in half along K between
// two pairs each (MxPlan::halves); as in k_mxfp4_gemm.cu both add into zeroed outputs, in either order.  The epilogue's two forms are
// apart because one that decides for every output costs 128 experts at 2048 tokens 103 us instead of 88.
//
// Waits are bounded as in k_mxfp4_gemm.cu.  Both CTAs leave together, once the
// commits of all steps have arrived at their barriers and, if one of them gave up,
// the copies that either started have landed.
#include "mx_gemm.cuh"

namespace ql {
namespace {

constexpr int PM = 2 * TM;  // weight rows of a pair's tile (MMA M)
constexpr int B_FULL = 0, B_EMPTY = kMaxStages, B_ACCF = 2 * kMaxStages, B_ACCE = B_ACCF + 2, B_DRAIN = B_ACCE + 2,
              B_SF = B_DRAIN + 1, NBARS = B_SF + kMaxStages;

struct PairParams {
    CUtensorMap tmW;        // weight codes: [E * N rows], box [128 rows][128 bytes of shared memory]
    CUtensorMap tmX, tmXb;  // activation codes: boxes of 16 and 64 rows x 128 bytes
    CUtensorMap tmSW, tmSX;  // scales as rows of 512 bytes, boxes of a step's blocks
    MxGemm g;
    int stages, stage_bytes;  // ring
    int nacc, acc_cols, sf0, sf_cols, sf_slots;  // tensor memory: accumulators and their stride, scales' first column, columns and slots
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;\n" : "=r"(r));
    return r;
}
// The address, in the even (0) or odd (1) CTA, of this CTA's shared-memory address.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t in_even(uint32_t addr) { return in_cta(addr, 0); }
// *p = v in one of the CTAs.
__device__ __forceinline__ void put(const int* p, int rank, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(in_cta(smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// A copy into this CTA that completes on a barrier of either CTA of the pair.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];\n" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int MODE>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t sfa, uint32_t sfb,
                                         uint32_t acc_in) {
    if constexpr (MODE == kMxParts)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(id), "r"(sfa), "r"(sfb), "r"(acc_in));
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(id), "r"(sfa), "r"(sfb), "r"(acc_in));
}
__device__ __forceinline__ void pair_copy_scales(uint32_t col, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(col), "l"(desc));
}
// Arrives at the barrier of this offset in both CTAs once everything issued before is done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    asm volatile(
        "{\n .reg .b16 m;\n mov.b16 m, 3;\n"
        " tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::"r"(bar)
        : "memory");
}
// mbar_wait for a barrier that the other CTA's threads arrive at.
__device__ __forceinline__ bool pair_try(uint32_t bar, unsigned phase) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(phase)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool pair_wait(uint32_t bar, unsigned phase, unsigned long long lim) {
    if (pair_try(bar, phase)) return true;
    if (lim <= 1) return false;
    const unsigned long long t0 = global_ns();
    for (unsigned it = 0;; ++it) {
        if (pair_try(bar, phase)) return true;
        if (((it & 255u) == 255u || lim < kWaitNs) && global_ns() - t0 > lim) return false;
    }
}
// The same for this CTA's barrier alone.
__device__ __forceinline__ void pair_commit_here(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_arrive(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_bar) : "memory");
}

// Wait until the barriers at `bar` of the ring's last steps before `steps` have completed those steps' phases.
__device__ __forceinline__ bool pair_wait_last(uint32_t bar, int steps, int stages, unsigned long long lim = kWaitNs) {
    for (int j = max(steps - stages, 0); j < steps; ++j)
        if (!__all_sync(kFull, mbar_wait(bar + 8 * (j % stages), (j / stages) & 1, lim))) return false;
    return true;
}

template <int MODE, int ROWS>  // ROWS: operand rows of a block at most
__global__ void __launch_bounds__(kThreads, 1) k_mx_pair(const __grid_constant__ PairParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[NBARS];
    __shared__ uint32_t tmem_slot;
    __shared__ Routing rt;
    __shared__ int gave_up;    // a wait of either CTA ran out (both CTAs' copies of it are set)
    __shared__ int brought[4];  // even CTA: the steps that each CTA's two producers started
    __shared__ int fed[2];      // the steps and tiles whose MMAs were committed
    constexpr bool PARTS = MODE == kMxParts;
    constexpr int KBS = PARTS ? 1 : 2;  // 128-column blocks per step
    const MxGemm& g = p.g;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int G = g.K / 128, KS = (G + KBS - 1) / KBS, NB = (g.N + TM - 1) / TM;
    const int nblk = g.plan.nblk;
    // A slot: weight codes, this CTA's half of the activation codes, weight scales (KBS blocks), activation scales
    // (KBS x nblk blocks).
    const int b_off = A_BYTES, sa_off = p.stage_bytes - KBS * (1 + nblk) * 512, sb_off = sa_off + KBS * 512;

    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // the next call's quantiser may stand by
    const unsigned long long lim = wait_limit(g.err);
    bool dead = false;
    Tile ti;
    if (threadIdx.x == 0) gave_up = 0;
    if (warp == 0 && elect()) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bar(B_FULL + s), 2);   // even CTA: its two producers' expect_tx, for both CTAs' copies
            mbar_init(bar(B_EMPTY + s), 1);  // the step's MMA commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(B_ACCF + b), 1);              // the tile's last commit
            mbar_init(bar(B_ACCE + b), 2 * kEpiWarps);  // even CTA: one arrive per epilogue warp of both
        }
        for (int q = 0; q < p.sf_slots; ++q) mbar_init(bar(B_SF + q), 1);  // even CTA: the step's scales are copied
        mbar_init(bar(B_DRAIN), 2);  // even CTA: the copies' and the MMAs' last commits
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_slot)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
    }
    if (grouped(g)) route(g, rt, warp, lane);
    fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are there
    fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)tmem_slot);
    Tiles<PM> tiles(g, rt, KS, blockIdx.x >> 1, gridDim.x >> 1, false);

    if (warp == 0) {  // ---- weights and their scales ----
        const bool leader = elect();
        int s = 0, ph = 1, step = 0;
        while (!dead && tiles.next(ti)) {
            const int e = uniform(ti.expert), wb = 2 * uniform(ti.wb) + rank;  // this CTA's 128 rows
            const int row = e * g.N + wb * TM;
            // Past the last row of all (an odd number of 128-row blocks) the scales are some block's: no output
            // comes of those rows.
            const int sf = (e * NB + min(wb, NB - 1)) * G;
            for (int k = uniform(ti.k0), k1 = uniform(ti.k1); k < k1; ++k, ++step) {
                if (!__all_sync(kFull, mbar_wait(bar(B_EMPTY + s), ph, lim))) {
                    dead = true;
                    break;
                }
                const uint32_t slot = base + s * p.stage_bytes, fb = in_even(bar(B_FULL + s));
                if (leader) {
                    // spread copies count the packed bytes; what lies past the last column or block counts too
                    if (rank == 0) mbar_expect_tx(bar(B_FULL + s), 2 * ((PARTS ? A_BYTES / 2 : A_BYTES) + KBS * 512));
                    pair_load_2d(slot, &p.tmW, k * 128, row, fb);
                    pair_load_2d(slot + sa_off, &p.tmSW, 0, sf + k * KBS, fb);
                }
                __syncwarp();
                if (++s == p.stages) { s = 0; ph ^= 1; }
            }
        }
        if (leader) put(&brought[2 * rank], 0, step);
        // The last steps' commits, which the other CTA's thread makes, arrive here before this CTA may leave.
        if (!dead && !pair_wait_last(bar(B_EMPTY), step, p.stages, lim)) dead = true;
    } else if (warp == 2) {  // ---- activations and their scales ----
        const bool leader = elect();
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the quantiser's codes and scales
        int s = 0, ph = 1, step = 0;
        while (!dead && tiles.next(ti)) {
            // the pair's columns: with 4-bit activations a multiple of 32, so that each half is whole 16-row boxes
            const int half = uniform(PARTS ? mx_pad16(ti.rows) : ((ti.rows + 31) & ~31) / 2);
            const int row = PARTS ? rank * g.R + uniform(ti.row0) : uniform(ti.row0) + rank * half;
            const int sf = uniform(ti.slot) * G * nblk;
            for (int k = uniform(ti.k0), k1 = uniform(ti.k1); k < k1; ++k, ++step) {
                if (!__all_sync(kFull, mbar_wait(bar(B_EMPTY + s), ph, lim))) {
                    dead = true;
                    break;
                }
                const uint32_t slot = base + s * p.stage_bytes, fb = in_even(bar(B_FULL + s));
                if (leader) {
                    if (rank == 0) mbar_expect_tx(bar(B_FULL + s), 2 * (half * 128 + KBS * nblk * 512));
                    int r = 0;
                    for (; r + BIG <= half; r += BIG)
                        pair_load_2d(slot + b_off + r * 128, &p.tmXb, k * 128, row + r, fb);
                    for (; r < half; r += SMALL) pair_load_2d(slot + b_off + r * 128, &p.tmX, k * 128, row + r, fb);
                    pair_load_2d(slot + sb_off, &p.tmSX, 0, sf + k * KBS * nblk, fb);
                }
                __syncwarp();
                if (++s == p.stages) { s = 0; ph ^= 1; }
            }
        }
        if (leader) put(&brought[2 * rank + 1], 0, step);
    } else if (warp == 3 && rank == 0) {  // ---- scales to tensor memory ----
        const bool leader = elect();
        int s = 0, ph = 0, q = 0;  // q: the step's scale columns
        int os = 0, oph = 0;       // ring slot (and its phase) of the step that had them before
        long long step = 0;
        while (!dead && tiles.next(ti)) {
            for (int k = uniform(ti.k0), k1 = uniform(ti.k1); k < k1; ++k, ++step) {
                bool ok = pair_wait(bar(B_FULL + s), ph, lim);
                // The MMAs that read these columns before are done: the load that filled the slot waited for them
                // if there are as many columns as slots.
                if (p.sf_slots < p.stages && step >= p.sf_slots) {
                    ok = ok && mbar_wait(bar(B_EMPTY + os), oph, lim);
                    if (++os == p.stages) { os = 0; oph ^= 1; }
                }
                if (!__all_sync(kFull, ok)) {
                    dead = true;
                    break;
                }
                fence_after();
                const uint32_t slot = base + s * p.stage_bytes, sf = tmem + p.sf0 + q * p.sf_cols;
                const uint32_t sfb = sf + 4 * KBS;
                const int kbs = min(KBS, G - k * KBS);
                const uint64_t sad = desc_scales(slot + sa_off), sbd = desc_scales(slot + sb_off);
                if (leader) {
#pragma unroll
                    for (int i = 0; i < KBS; ++i) {  // 512 bytes a copy: +32 in the descriptors' address field
                        if (i < kbs) {
                            pair_copy_scales(sf + 4 * i, sad + 32 * i);
                            pair_copy_scales(sfb + 4 * nblk * i, sbd + 32 * nblk * i);
                            if (nblk > 1) pair_copy_scales(sfb + 4 * (nblk * i + 1), sbd + 32 * (nblk * i + 1));
                        }
                    }
                    pair_commit_here(bar(B_SF + q));
                }
                __syncwarp();
                if (++s == p.stages) { s = 0; ph ^= 1; }
                if (++q == p.sf_slots) q = 0;
            }
        }
        if (leader) pair_commit_here(bar(B_DRAIN));
    } else if (warp == 1 && rank == 0) {  // ---- MMAs ----
        const bool leader = elect();
        int s = 0, q = 0, qph = 0, tl = 0, step = 0;
        while (!dead && tiles.next(ti)) {
            const int b = p.nacc == 2 ? tl & 1 : 0, use = p.nacc == 2 ? tl >> 1 : tl;
            if (!__all_sync(kFull, pair_wait(bar(B_ACCE + b), (use & 1) ^ 1, lim))) {  // both epilogues are done
                dead = true;
                break;
            }
            const int cols = uniform(PARTS ? 2 * mx_pad16(ti.rows) : (ti.rows + 31) & ~31);
            const uint32_t d = tmem + b * p.acc_cols, id0 = idesc<MODE>(PM, cols);
            const int k0 = uniform(ti.k0), k1 = uniform(ti.k1);
            for (int k = k0; k < k1; ++k, ++step) {
                // the scales are in place, and with them the operands, which their copier waited for
                if (!__all_sync(kFull, mbar_wait(bar(B_SF + q), qph, lim))) {
                    dead = true;
                    break;
                }
                fence_after();
                const uint32_t slot = base + s * p.stage_bytes, sf = tmem + p.sf0 + q * p.sf_cols;
                const uint32_t sfb = sf + 4 * KBS;
                const int kbs = min(KBS, G - k * KBS);
                const uint64_t ad = desc_sw128(slot), bd = desc_sw128(slot + b_off);
                if (leader) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // 32 bytes of every row: +2 in the descriptors' address field
                        const int i = PARTS ? 0 : j >> 1, byte = PARTS ? j : 2 * (j & 1);  // its scales' block and byte
                        if (i < kbs)
                            pair_mma<MODE>(d, ad + 2 * j, bd + 2 * j, id0 | (uint32_t)byte << 4 | (uint32_t)byte << 29,
                                           sf + 4 * i, sfb + 4 * nblk * i, (k > k0 || j) ? 1u : 0u);
                    }
                    pair_commit(bar(B_EMPTY + s));  // both CTAs' slots may be refilled once these are done
                }
                __syncwarp();
                if (++s == p.stages) s = 0;
                if (++q == p.sf_slots) { q = 0; qph ^= 1; }
            }
            if (dead) break;
            if (leader) pair_commit(bar(B_ACCF + b));
            __syncwarp();
            ++tl;
        }
        // Every copy and MMA issued must finish before tensor memory is freed.
        if (leader) {
            pair_commit_here(bar(B_DRAIN));
            for (int r = 0; r < 2; ++r) {
                put(&fed[0], r, step);
                put(&fed[1], r, tl);
            }
        }
        __syncwarp();
        mbar_wait(bar(B_DRAIN), 0);
    } else if (warp >= kEpiWarp0) {  // ---- epilogue ----
        const int q = warp & 3, h = (warp - kEpiWarp0) >> 2;
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        int tl = 0;
        while (tiles.next(ti)) {
            const int b = p.nacc == 2 ? tl & 1 : 0, use = p.nacc == 2 ? tl >> 1 : tl;
            Epilogue<MODE, ROWS> epi;
            epi.fetch(g, rt, ti, h, lane);
            if (!__all_sync(kFull, mbar_wait(bar(B_ACCF + b), use & 1, lim))) {  // together
                dead = true;
                break;
            }
            fence_after();
            epi.drain(ti, tmem + b * p.acc_cols + ((uint32_t)(32 * q) << 16), h);
            fence_before();
            __syncwarp();
            if (lane == 0) pair_arrive(in_even(bar(B_ACCE + b)));
            const int n = (2 * ti.wb + rank) * TM + 32 * q + lane;
            if (ti.k1 - ti.k0 == KS) epi.store(g, ti, h, n, false);
            else epi.store(g, ti, h, n, true);
            ++tl;
        }
    }
    if (dead) {
        atomicOr(g.err, (unsigned)QL_DEVERR_TIMEOUT);
        if (lane == 0) {
            put(&gave_up, 0, 1);
            put(&gave_up, 1, 1);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    cluster_sync();
    // All copies were consumed unless a wait ran out.  Then those in flight, and commits, have to arrive before the CTAs'
    // shared memory is released.  A step that not all four producers started ends this at the wait's bound.
    if (*const_cast<volatile int*>(&gave_up)) {
        if (warp == 0) {
            pair_wait_last(bar(B_EMPTY), fed[0], p.stages);
            pair_wait_last(bar(B_ACCF), fed[1], p.nacc);
            if (rank == 0)
                pair_wait_last(bar(B_FULL), max(max(brought[0], brought[1]), max(brought[2], brought[3])), p.stages);
        }
        __syncthreads();
        cluster_sync();
    }
    if (warp == 2) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols));
    }
}

template <int MODE, int ROWS>
cudaError_t run(const MxGemm& g, cudaStream_t s) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    if (di.smem_optin < (size_t)kSmemMax + 12 * 1024) return cudaErrorInvalidValue;
    constexpr bool PARTS = MODE == kMxParts;
    constexpr int P = mx_planes(MODE), KBS = PARTS ? 1 : 2;
    PairParams p;
    p.g = g;
    const int nblk = g.plan.nblk, rows = (P * g.plan.nt + 31) / 32 * 32;  // operand rows of a full token block
    if (rows > ROWS) return cudaErrorInvalidValue;
    p.stage_bytes = (int)align_up(A_BYTES + rows / 2 * 128 + KBS * (1 + nblk) * 512, 1024);
    p.acc_cols = rows;
    p.nacc = rows <= kMxRows2 ? 2 : 1;
    p.sf0 = p.nacc * p.acc_cols;
    p.sf_cols = KBS * 4 * (1 + nblk);
    p.stages = (kSmemMax - 1024) / p.stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    p.sf_slots = ((int)kTmemCols - p.sf0) / p.sf_cols;
    if (p.sf_slots > p.stages) p.sf_slots = p.stages;
    if (p.stages < 2 || p.sf_slots < 2) return cudaErrorInvalidValue;
    const long long wrows = (long long)g.E * g.N, xrows = (long long)P * g.R, xbytes = PARTS ? g.K : g.K / 2;
    const long long G = g.K / 128, wblocks = (long long)g.E * ((g.N + TM - 1) / TM) * G;
    const long long xblocks = mx_slots(g.R, g.offsets || g.ids ? g.E : 0, g.plan.nt) * G * nblk;
    e = PARTS ? make_tmap_u4_spread(g.codes, wrows, g.K, TM, &p.tmW)
              : make_tmap_2d(g.codes, wrows, g.K / 2, g.K / 2, 128, TM, CU_TENSOR_MAP_SWIZZLE_128B, &p.tmW);
    if (e == cudaSuccess) e = make_tmap_2d(g.xq, xrows, xbytes, xbytes, 128, SMALL, CU_TENSOR_MAP_SWIZZLE_128B, &p.tmX);
    if (e == cudaSuccess) e = make_tmap_2d(g.xq, xrows, xbytes, xbytes, 128, BIG, CU_TENSOR_MAP_SWIZZLE_128B, &p.tmXb);
    if (e == cudaSuccess) e = make_tmap_blocks(g.scales, wblocks, KBS, &p.tmSW);
    if (e == cudaSuccess) e = make_tmap_blocks(g.xs, xblocks, KBS * nblk, &p.tmSX);
    if (e != cudaSuccess) return e;

    static int pairs_of[64] = {};  // pairs that run at once
    int dev = 0;
    cudaGetDevice(&dev);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.stages * p.stage_bytes + 1024;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;  // after this library's quantiser
    cfg.attrs = attr;
    int pairs = dev < 64 ? pairs_of[dev] : 0;
    if (!pairs) {
        e = cudaFuncSetAttribute(k_mx_pair<MODE, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(di.sm_count / 2 * 2);
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&pairs, k_mx_pair<MODE, ROWS>, &cfg);
        if (e != cudaSuccess) return e;
        if (pairs > di.sm_count / 2) pairs = di.sm_count / 2;
        if (pairs < 1) return cudaErrorInvalidValue;
        if (dev < 64) pairs_of[dev] = pairs;
    }
    long long tiles = (long long)((g.N + PM - 1) / PM) * mx_slots(g.R, g.offsets || g.ids ? g.E : 0, g.plan.nt);
    if (tiles > g.plan.halves) tiles += tiles - g.plan.halves;
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, k_mx_pair<MODE, ROWS>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_pair(const MxGemm& g, cudaStream_t s) {
    const bool wide = mx_planes(g.plan.mode) * g.plan.nt > 128;
    if (g.plan.mode == kMxParts) return wide ? run<kMxParts, kMxRows>(g, s) : run<kMxParts, 128>(g, s);
    return wide ? run<kMxA4, kMxRows>(g, s) : run<kMxA4, 128>(g, s);
}

}  // namespace ql
