// k_mxfp4_gemm.cu -- the product of MXFP4 weights, y = x~ . dequant(W)^T, over
// one weight or, rows sorted by expert, over one weight per expert, on the
// fifth-generation tensor cores' block-scaled instructions.
//
// The hardware multiplies the codes as they are stored: every 32 products along
// K share the two operands' power-of-two scales, which the instruction reads
// from tensor memory, so nothing is dequantised and one fp32 accumulator takes
// the whole K.
//   4-bit activations (kind::mxf4): both operands packed E2M1, K = 64 a step.
//   16-bit activations, few rows (kind::mxf4): a token enters as eight rows of
//     E2M1 digits in base 8, each with scales of its own, whose products the
//     epilogue adds up.  The weights stream as fast as with 4-bit activations.
//   16-bit activations, many rows: as two parts, on pairs of CTAs alone
//     (k_mxfp4_pair.cu).
//
// A tile is 128 weight rows (the MMA's M, tensor-memory lanes) by one token
// block (its N: the block's operand rows rounded up to 16), so a decode batch and
// a prefill differ in N alone.  A step is 128 bytes of every operand
// row, 256 columns of K.  A ring slot holds the step's weight codes
// (16 KB), its activation codes and both scale blocks; as many slots as shared
// and tensor memory allow keep the weights streaming.  Each slot has its own
// tensor-memory columns for its scales: they are rewritten only when the slot
// is, after the MMAs that read them have finished.  Two accumulators let the
// epilogue of one tile run under the MMAs of the next.
//
// With few tiles the sums of a tile may be cut along K between two CTAs
// (MxPlan::split): the work is one row of steps, tile after tile, dealt out in
// equal runs, none shorter than a tile or else exactly half of one, so that at
// most two CTAs meet in a tile.  Both add into y, which the quantiser zeroed:
// 0 + a + b is the same in either order, so the result does not depend on which
// comes first.
//
// Warp roles: warp 0 brings in the weights, which wait for nothing, warp 2 the
// activations, once the quantiser before this kernel is done (programmatic
// dependent launch); warp 1 issues the scale copies and MMAs; warps 4..11 store
// the sums, 32 consecutive outputs of a token per warp and instruction.
//
// All waits are bounded; on a timeout the CTA sets QL_DEVERR_TIMEOUT and winds
// down without leaving tensor memory allocated, MMAs running or copies in
// flight.
#include "mx_gemm.cuh"

namespace ql {
namespace {

constexpr int kFirst = 8;  // weight steps ahead of the activations (12, 6, 4: 0.1 to 0.7 us slower at 1 row)
constexpr int B_FULL = 0, B_EMPTY = kMaxStages, B_ACCF = 2 * kMaxStages, B_ACCE = B_ACCF + 2, B_DRAIN = B_ACCE + 2,
              NBARS = B_DRAIN + 1;

struct MxParams {
    CUtensorMap tmW;         // weight codes: [E * N rows], box [128 rows][128 bytes of shared memory]
    CUtensorMap tmX, tmXb;   // activation codes: [R or 8 R rows], boxes of 16 and 64 rows x 128 bytes
    MxGemm g;
    int stages, stage_bytes;     // ring
    int acc_cols, sf0, sf_cols;  // tensor memory: accumulator stride, first scale column, scale columns per slot
};

__device__ __forceinline__ void mma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t sfa, uint32_t sfb,
                                    uint32_t acc_in) {
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
// ROWS: operand rows of a block at most.  The epilogue is written out for them, and a decode call waits for the
// instructions of a long one.
template <int MODE, int ROWS>
__global__ void __launch_bounds__(kThreads, 1) k_mx_gemm(const __grid_constant__ MxParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[NBARS];
    __shared__ uint32_t tmem_slot;
    __shared__ Routing rt;
    constexpr int KBS = 2;  // 128-column blocks per step
    const MxGemm& g = p.g;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int G = g.K / 128, KS = (G + KBS - 1) / KBS;
    const int nblk = g.plan.nblk;
    // A slot: weight codes, activation codes, weight scales (KBS blocks), activation scales (KBS x nblk blocks).
    const int b_off = A_BYTES, sa_off = p.stage_bytes - KBS * (1 + nblk) * 512, sb_off = sa_off + KBS * 512;

    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // the next call's quantiser may stand by
    const unsigned long long lim = wait_limit(g.err);
    bool dead = false;
    Tile ti;
    // One step of a tile's weights into ring slot s.
    auto load_weights = [&](const Tile& t, int k, int s, bool leader) {
        const int NB = (g.N + TM - 1) / TM;
        const unsigned sfb = min(KBS, G - k * KBS) * 512;
        const uint32_t slot = base + s * p.stage_bytes, fb = bar(B_FULL + s);
        const uint8_t* sf = g.scales + (((long long)t.expert * NB + t.wb) * G + k * KBS) * 512;
        if (leader) {
            mbar_expect_tx(fb, A_BYTES + sfb);
            tma_load_2d(slot, &p.tmW, k * 128, t.expert * g.N + t.wb * TM, fb);
            bulk_load(slot + sa_off, sf, sfb, fb);
        }
    };
    int ahead = 0;  // steps of the first tile that warp 0 has issued before the block's first barrier

    if (warp == 0) {
        const bool leader = elect();
        if (leader) {
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
        __syncwarp();
        if (!grouped(g)) {  // one weight: its stream starts at once
            Tiles<TM> first(g, rt, KS, blockIdx.x, gridDim.x, g.plan.split);
            if (first.next(ti)) {
                ahead = min(kFirst, min(p.stages, ti.k1 - ti.k0));
                for (int k = 0; k < ahead; ++k) load_weights(ti, ti.k0 + k, k, leader);
            }
        }
    } else if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_slot)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    if (grouped(g)) route(g, rt, warp, lane);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)tmem_slot);
    Tiles<TM> tiles(g, rt, KS, blockIdx.x, gridDim.x, g.plan.split);

    // The three issuing roles run as whole warps, with every operand the same in all lanes, and one elected lane
    // issues: the instructions take their operands from uniform registers, which a lone lane's values would have
    // to be moved to one by one for each of them.
    if (warp == 0) {  // ---- weights ----
        const bool leader = elect();
        int step = 0, s = 0, ph = 1;
        while (!dead && tiles.next(ti)) {
            ti.expert = uniform(ti.expert);
            ti.wb = uniform(ti.wb);
            for (int k = uniform(ti.k0), k1 = uniform(ti.k1); k < k1; ++k, ++step) {
                if (step >= ahead) {
                    // The first steps' weights are enough until the activations are there, whose copies would
                    // queue behind any more.
                    if (step == (grouped(g) ? kFirst : ahead)) asm volatile("griddepcontrol.wait;\n" ::: "memory");
                    if (!__all_sync(kFull, mbar_wait(bar(B_EMPTY + s), ph, lim))) {
                        dead = true;
                        break;
                    }
                    load_weights(ti, k, s, leader);
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
            const int cols = uniform(mx_pad16(mx_planes(MODE) * ti.rows)), row = mx_planes(MODE) * uniform(ti.row0);
            const uint8_t* sf = g.xs + (long long)uniform(ti.slot) * G * nblk * 512;
            for (int k = uniform(ti.k0), k1 = uniform(ti.k1); k < k1; ++k, ++step) {
                if (!__all_sync(kFull, mbar_wait(bar(B_EMPTY + s), ph, lim))) {
                    dead = true;
                    break;
                }
                const unsigned sfb = min(KBS, G - k * KBS) * nblk * 512;
                const uint32_t slot = base + s * p.stage_bytes, fb = bar(B_FULL + s);
                if (leader) {
                    mbar_expect_tx(fb, cols * 128 + sfb);
                    const uint32_t dst = slot + b_off;
                    int r = 0;
                    for (; r + BIG <= cols; r += BIG) tma_load_2d(dst + r * 128, &p.tmXb, k * 128, row + r, fb);
                    for (; r < cols; r += SMALL) tma_load_2d(dst + r * 128, &p.tmX, k * 128, row + r, fb);
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
            const uint32_t d = tmem + b * p.acc_cols, id0 = idesc<MODE>(TM, uniform(mx_pad16(mx_planes(MODE) * ti.rows)));
            const int k0 = uniform(ti.k0), k1 = uniform(ti.k1);
            for (int k = k0; k < k1; ++k) {
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
                        const int q = j >> 1, byte = 2 * (j & 1);  // its scales' block and byte
                        if (q < kbs)
                            mma(d, ad + 2 * j, bd + 2 * j, id0 | (uint32_t)byte << 4 | (uint32_t)byte << 29, sf + 4 * q,
                                sfb + 4 * nblk * q, (k > k0 || j) ? 1u : 0u);
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
        const int q = warp & 3, h = (warp - kEpiWarp0) >> 2;
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the quantiser's factors and zeroed outputs
        int tl = 0;
        while (tiles.next(ti)) {
            const int b = tl & 1;
            Epilogue<MODE, ROWS> epi;
            epi.fetch(g, rt, ti, h, lane);
            if (!__all_sync(kFull, mbar_wait(bar(B_ACCF + b), (tl >> 1) & 1, lim))) {  // together
                dead = true;
                break;
            }
            fence_after();
            epi.drain(ti, tmem + b * p.acc_cols + ((uint32_t)(32 * q) << 16), h);
            fence_before();
            __syncwarp();
            if (lane == 0) arrive(bar(B_ACCE + b));
            epi.store(g, ti, h, ti.wb * TM + 32 * q + lane, ti.k1 - ti.k0 < KS);
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

template <int MODE, int ROWS>
cudaError_t run(const MxGemm& g, cudaStream_t s) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    constexpr int P = mx_planes(MODE), KBS = 2;
    MxParams p;
    p.g = g;
    const int nblk = g.plan.nblk, rows = P * g.plan.nt;  // operand rows of a full token block
    if (rows > ROWS) return cudaErrorInvalidValue;
    p.stage_bytes = (int)align_up(A_BYTES + rows * 128 + KBS * (1 + nblk) * 512, 1024);
    p.acc_cols = (int)align_up(rows, 32);
    p.sf0 = 2 * p.acc_cols;
    p.sf_cols = KBS * 4 * (1 + nblk);
    if (di.smem_optin < (size_t)kSmemMax + 12 * 1024) return cudaErrorInvalidValue;
    p.stages = (kSmemMax - 1024) / p.stage_bytes;
    if (p.stages > ((int)kTmemCols - p.sf0) / p.sf_cols) p.stages = ((int)kTmemCols - p.sf0) / p.sf_cols;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    if (p.stages < 2) return cudaErrorInvalidValue;
    const int smem = p.stages * p.stage_bytes + 1024;
    const long long wrows = (long long)g.E * g.N, xrows = (long long)P * g.R, xbytes = g.K / 2;
    e = make_tmap_2d(g.codes, wrows, xbytes, xbytes, 128, TM, CU_TENSOR_MAP_SWIZZLE_128B, &p.tmW);
    if (e == cudaSuccess) e = make_tmap_2d(g.xq, xrows, xbytes, xbytes, 128, SMALL, CU_TENSOR_MAP_SWIZZLE_128B, &p.tmX);
    p.tmXb = p.tmX;
    if (e == cudaSuccess && rows >= BIG)
        e = make_tmap_2d(g.xq, xrows, xbytes, xbytes, 128, BIG, CU_TENSOR_MAP_SWIZZLE_128B, &p.tmXb);
    if (e != cudaSuccess) return e;

    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(k_mx_gemm<MODE, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    const long long tiles = (long long)((g.N + TM - 1) / TM) * mx_slots(g.R, g.offsets || g.ids ? g.E : 0, g.plan.nt);
    const long long ctas = (g.plan.split ? 2 : 1) * tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas < di.sm_count ? ctas : di.sm_count));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;  // after this library's quantiser
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_mx_gemm<MODE, ROWS>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

namespace {

constexpr int kPlanSms = 148;  // a plan goes by this GPU's count, so that a workspace size does not depend on a device

constexpr int kPairs = kPlanSms / 2;

// Tokens of a block for weights of R rows each on pairs of CTAs, and how many of its tiles, the last ones, are halved
// along K: the cut with the least rounds of tiles times what a tile of so many operand rows takes.  Measured at 5376
// columns, 74 x 256 weight rows and 2048 rows of 4-bit x, a round of 64, 96, 128, 160, 192, 208 and 256 operand rows
// takes 5.4, 6.1, 6.1, 7.0, 8.4, 8.8 and 9.9 us, one of 16-bit parts half as much again, but no less than the spreading
// copies' 9.4.  Other widths are taken to go with K, which leaves out a tile's start and epilogue at small K.
// Halves, of one weight's tiles that leave half of the pairs without work, cost zeroed outputs and adding into them, 2 us
// and half a us for every MB: 5376 x 21504 at 128 rows takes 22.9 us with them and 29.3 without (4-bit x) and 38.9
// against 49.4 (parts), but 4096 x 4096 at 256 rows 15.3 against 12.8.  After full rounds only parts gain (21504 x 5376
// at 96 rows 28.5 against 32.3): 4-bit x finds more bandwidth in a round that is not full and takes 22.6 against 21.3.
int pair_tokens(int P, long long R, int N, int K, int E, int* halved) {
    const int wide = (int)min((R + 15) / 16 * 16, (long long)kMxRows / P);
    const long long blocks_n = (N + 2 * TM - 1) / (2 * TM) * (long long)(E ? E : 1);
    double best = 0;
    int nt = wide;
    *halved = 0;
    for (int t = wide; t == wide || P * t >= 64; t -= 16) {
        const int rows = P * t;
        const long long tiles = blocks_n * ((R + t - 1) / t), full = tiles / kPairs, tail = tiles % kPairs;
        double tile = rows <= 128 ? 4.9 + rows * 0.01 : 3.7 + rows * 0.0244;
        if (P > 1) tile = 1.5 * tile > 9.4 ? 1.5 * tile : 9.4;
        tile *= K / 5376.0;
        const double half = tile / 2 + 2 + 0.5e-6 * 4 * (2 * TM) * t * tail;
        const bool cut = E == 0 && 2 * tail <= kPairs && (P > 1 || full == 0) && K >= 512 && half < tile;
        const double cost = full * tile + (tail == 0 ? 0 : cut ? half : tile);
        if (t == wide || cost < best) {
            best = cost;
            nt = t;
            *halved = cut ? (int)tail : 0;
        }
    }
    return nt;
}

}  // namespace

MxPlan mx_plan(bool a16, int R, int N, int K, int E) {
    MxPlan p;
    int halved = 0;
    const long long per = E ? ((long long)R + E - 1) / E : R;  // rows an expert
    // Digits for one block of one weight (21504 x 5376 at 24 rows 18.7 us; at 25 rows parts take 22.3 and digits 24.4),
    // for more while there are two CTAs to a tile (2816 x 5376 at 72 rows 11.4 us against 13.1 as parts, at 96 rows 14.5
    // against 13.5), and up to 20 rows an expert (128 of 1408 x 2816 at 280 tokens 70.6 us against 76.7, at 384 tokens
    // 88.0 against 79.9).
    const long long most = kMxRows2 / mx_planes(kMxDigits), digit_tiles = (N + TM - 1) / TM * ((per + most - 1) / most);
    const bool digits = E ? per <= 20 : per <= most || (per <= 6 * most && 2 * digit_tiles <= kPlanSms);
    p.mode = !a16 ? kMxA4 : digits ? kMxDigits : kMxParts;
    const int P = mx_planes(p.mode);
    if (p.mode == kMxDigits) {
        // Cut evenly, an even number of tokens; for experts 1.6 times the average count, so that most are one block (a
        // block costs its own rows alone, but a second one reads the weights again) and few ring slots go to rows
        // that are not there (128 experts of 1408 x 2816, 200 tokens: 63.2 us against 65.2 at twice the average).
        const long long b = (R + most - 1) / most, nt = E ? (8 * per + 4) / 5 : (R + b - 1) / b;
        p.nt = (int)(((nt < most ? nt : most) + 1) / 2 * 2);
        p.pair = 0;
    } else if (E && per * P < kMxRows2) {
        const long long wide = kMxRows2 / P;
        p.nt = (int)((2 * per < wide ? 2 * per : wide) + 15) / 16 * 16;
        // Experts with 4-bit activations wait for their weights longer than for their rows: pairs of CTAs take 128 of
        // 1408 x 2816 at 400 tokens to 60.8 us from 58.9, at 2048 tokens to 91.5 from 94; parts gain everywhere (400
        // tokens 80 against 96).
        p.pair = p.mode == kMxParts || p.nt >= kMxRows2;
    } else {
        // Parts come from 25 rows on, so in blocks of 64 operand rows at least, and always go to pairs; 4-bit activations
        // do once a token block is wide enough for its operand stream to count: 21504 x 5376 at 64 rows 20.5 us
        // against 22.3, at 192 rows 27.1 against 30.6.
        p.nt = pair_tokens(P, per, N, K, E, &halved);
        p.pair = p.mode == kMxParts || p.nt >= 64;
    }
    p.nblk = (P * p.nt + 127) / 128;
    // Cutting tiles along K costs a zeroed y: worth it while y is small beside the weights.
    const long long tiles = (long long)((N + TM - 1) / TM) * mx_slots(R, 0, p.nt);
    p.split = !p.pair && (long long)R * N * 4 <= (4 << 20) && (E || tiles < 8LL * kPlanSms);
    p.zero = p.split ? 0 : N;
    p.halves = INT_MAX;
    if (p.pair && halved) {
        const long long nb = mx_slots(R, 0, p.nt);
        p.halves = (int)((N + 2 * TM - 1) / (2 * TM) * nb - halved);
        p.zero = (int)min(p.halves / nb * (2 * TM), (long long)N);
    }
    return p;
}

cudaError_t launch_mx_gemm(const MxGemm& g, cudaStream_t s) {
    if (g.plan.pair) return launch_mx_pair(g, s);
    switch (g.plan.mode) {
    case kMxA4: return g.plan.nt <= 64 ? run<kMxA4, 64>(g, s) : run<kMxA4, kMxRows2>(g, s);
    case kMxDigits: return g.plan.nt <= 8 ? run<kMxDigits, 64>(g, s) : run<kMxDigits, kMxRows2>(g, s);
    default: return cudaErrorInvalidValue;  // parts go to pairs
    }
}

}  // namespace ql
