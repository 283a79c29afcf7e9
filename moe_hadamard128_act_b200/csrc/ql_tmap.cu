// ql_tmap.cu -- host-side construction of TMA tensor maps for 2-D matrices of
// bytes (packed weights, int8 activations), of 4-bit codes that the copy
// spreads to bytes or of scale blocks, cached by (address, shape, box, swizzle,
// element) since the same weight is encoded again on every call.
#include <mutex>

#include <cudaTypedefs.h>

#include "ql_internal.h"

namespace ql {
namespace {

struct TmapKey {
    const void* ptr;
    long long rows, width, ld;
    int box_x, box_y, swz;
    CUtensorMapDataType type;
    bool operator==(const TmapKey& o) const {
        return ptr == o.ptr && rows == o.rows && width == o.width && ld == o.ld && box_x == o.box_x &&
               box_y == o.box_y && swz == o.swz && type == o.type;
    }
};

// One entry to a hash of the key: a call looks at one entry for each map, however many weights are in use.
constexpr int kEntries = 512;
std::mutex g_mu;
TmapKey g_keys[kEntries];
CUtensorMap g_vals[kEntries];
bool g_used[kEntries] = {};

int entry_of(const TmapKey& k) {
    uint64_t h = reinterpret_cast<uintptr_t>(k.ptr) >> 4;
    for (const uint64_t v : {(uint64_t)k.rows, (uint64_t)k.width, (uint64_t)k.ld,
                             (uint64_t)k.box_x << 32 | (uint64_t)k.box_y << 16 | (uint64_t)k.swz << 8 | (uint64_t)k.type})
        h = (h ^ v) * 0x9E3779B97F4A7C15ull;
    return (int)(h >> 55);
}
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// width and box_x in elements, ld in bytes.
cudaError_t make_tmap(const void* base, CUtensorMapDataType type, long long rows, long long width, long long ld_bytes,
                      int box_x, int box_y, int swz, CUtensorMap* out) {
    std::lock_guard<std::mutex> lock(g_mu);
    const TmapKey key{base, rows, width, ld_bytes, box_x, box_y, swz, type};
    const int at = entry_of(key);
    if (g_used[at] && g_keys[at] == key) {
        *out = g_vals[at];
        return cudaSuccess;
    }
    if (!g_encode) {
        cudaDriverEntryPointQueryResult q;
        void* fn = nullptr;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) {
            cudaGetLastError();
            return cudaErrorNotSupported;
        }
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)box_x, (cuuint32_t)box_y};
    const cuuint32_t estr[2] = {1u, 1u};
    CUtensorMap m;
    const CUresult r = g_encode(&m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, static_cast<CUtensorMapSwizzle>(swz),
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
    g_keys[at] = key;
    g_vals[at] = m;
    g_used[at] = true;
    *out = m;
    return cudaSuccess;
}

}  // namespace

cudaError_t make_tmap_2d(const void* base, long long rows, long long width_bytes, long long ld_bytes, int box_x,
                         int box_y, int swz, CUtensorMap* out) {
    return make_tmap(base, CU_TENSOR_MAP_DATA_TYPE_UINT8, rows, width_bytes, ld_bytes, box_x, box_y, swz, out);
}

cudaError_t make_tmap_u4_spread(const void* base, long long rows, long long K, int box_y, CUtensorMap* out) {
    return make_tmap(base, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, rows, K, K / 2, 128, box_y,
                     CU_TENSOR_MAP_SWIZZLE_128B, out);
}

cudaError_t make_tmap_blocks(const void* base, long long rows, int box_y, CUtensorMap* out) {
    return make_tmap(base, CU_TENSOR_MAP_DATA_TYPE_INT32, rows, 128, 512, 128, box_y, CU_TENSOR_MAP_SWIZZLE_NONE, out);
}

}  // namespace ql
