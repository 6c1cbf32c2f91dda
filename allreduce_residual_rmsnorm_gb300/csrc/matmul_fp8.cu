// Host side of the 8-bit products: tensor maps, the choice of kernel, and the
// status words of their bounded waits.
#include <mutex>

#include "ar_internal.h"
#include "matmul_internal.h"

namespace arf {
namespace {

// code and detail of the first wait that gave up, per device
__device__ int g_status[2];

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                               cudaEnableDefault, &r);
        return e == cudaSuccess && r == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<EncodeTiled>(p)
                   : nullptr;
    }();
    return fn;
}

// Looked up once per device
constexpr int kMaxDevices = 64;
std::mutex g_mu;
DeviceInfo g_info[kMaxDevices] = {};

cudaError_t device_info(DeviceInfo* out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_mu);
    DeviceInfo& d = g_info[dev];
    if (!d.status) {
        int sms = 0;
        void* p = nullptr;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaGetSymbolAddress(&p, g_status);
        if (e != cudaSuccess)
            return e;
        d.sms = sms;
        d.status = static_cast<int*>(p);
    }
    *out = d;
    return cudaSuccess;
}

}  // namespace

bool byte_tensor_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t depth,
                     uint32_t box_rows)
{
    const EncodeTiled fn = encode_tiled();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {depth, rows};
    const cuuint64_t strides[1] = {depth};
    const cuuint32_t box[2] = {128, box_rows};
    const cuuint32_t steps[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
              steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool out_tensor_map(CUtensorMap* map, void* base, uint64_t rows, uint64_t cols, int dtype,
                    uint32_t box_rows, uint32_t box_cols)
{
    const EncodeTiled fn = encode_tiled();
    if (!fn)
        return false;
    const CUtensorMapDataType type = dtype == AR_DT_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : dtype == AR_DT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * (uint64_t)elem_bytes(dtype)};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t steps[2] = {1, 1};
    return fn(map, type, 2, base, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_matmul(int dtype, const MatmulArgs& a, cudaStream_t s)
{
    DeviceInfo d;
    const cudaError_t e = device_info(&d);
    if (e != cudaSuccess)
        return e;
    const int per = (a.rows + a.experts - 1) / a.experts;
    const int tokens = per <= 16 ? 16 : per <= 32 ? 32 : per <= 64 ? 64 : 128;
    if (per > 128)
        return launch_matmul_wide(dtype, a, d, s);
    // blocks without a split, and the split that fills two blocks per SM
    const int64_t blocks = (int64_t)((a.cols + 127) / 128) *
                           (a.experts < a.rows ? a.experts : a.rows);
    int split = 1;
    while (split < 8 && blocks * split * 2 <= 2 * d.sms && split * 2 <= quant_blocks(a.depth))
        split *= 2;
    return launch_matmul_narrow(dtype, a, tokens, split, d, s);
}

}  // namespace arf

extern "C" int ar_fusion_matmul_status(void* stream, int* detail)
{
    using namespace arf;
    if (detail)
        *detail = -1;
    DeviceInfo d;
    cudaError_t e = device_info(&d);
    int st[2] = {0, 0};
    const int clear[2] = {0, 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(st, d.status, sizeof st, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && st[0] != 0) {
        e = cudaMemcpyAsync(d.status, clear, sizeof clear, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess)
            e = cudaStreamSynchronize(s);
    }
    if (e != cudaSuccess)
        return set_last_error(AR_ERR_CUDA, cudaGetErrorString(e));
    if (st[0] == 0)
        return AR_OK;
    if (detail)
        *detail = st[1];
    return set_last_error(st[0], "a product's device-side wait gave up");
}
