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

}  // namespace

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

// Which kernel, by the time that each would take, in microseconds of this device.
// Both advance in steps of 128 of the depth that are bound by latency where the
// blocks fit the device once, and in waves where they do not:
//   wide     a step of a pair of blocks 0.40, a wave 1 more; 256 x 256 outputs
//   narrow   a step 0.22, 0.31 or 0.55 with 16, 32 or 64 rows, a wave (two blocks
//            per SM) 1.3 more, the sum over a split 0.04 a row; 128 columns
// Measured against the model (rows x cols x depth: narrow best / wide):
//   16 x 7168 x 2048: 5.3 / 10.1     128 x 7168 x 2048: 8.7 / 10.8
//   256 x 7168 x 2048: 13.2 / 11.0   256 x 4096 x 4096: 14.2 / 17.0
//   512 x 2048 x 7168: 21.4 / 25.8   1003 x 2048 x 7168: 33.2 / 26.4
// Loads of experts differ: they are taken to reach twice the mean (64 experts,
// 2048 rows x 4096 x 2048: 99 / 131; 32 experts: 74 / 65).
Choice choose_matmul(const MatmulArgs& a, int sms)
{
    const auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    const int64_t active = a.experts < a.rows ? a.experts : a.rows;
    const int64_t per = up(a.rows, a.experts) * (a.experts > 1 ? 2 : 1);
    const int steps = quant_blocks(a.depth);
    Choice best{0, 0};
    float us = 4.5f - 1.0f + (float)up(active * up(per, 256) * up(a.cols, 256), sms / 2) *
                                 (0.40f * steps + 1.0f);
    const int tokens[3] = {16, 32, 64};
    const float step[3] = {0.22f, 0.31f, 0.55f};
    for (int i = 0; i < 3; ++i) {
        for (int split = 1; split <= 8 && split <= steps; split *= 2) {
            const int64_t blocks = active * up(per, tokens[i]) * up(a.cols, 128) * split;
            const float t = 2.5f + (float)up(blocks, 2 * sms) * (1.3f + step[i] * up(steps, split)) +
                            (split > 1 ? 0.04f * tokens[i] : 0.0f);
            if (t < us) {
                us = t;
                best = Choice{tokens[i], split};
            }
        }
    }
    return best;
}

cudaError_t launch_matmul(int dtype, const MatmulArgs& a, cudaStream_t s)
{
    DeviceInfo d;
    const cudaError_t e = device_info(&d);
    if (e != cudaSuccess)
        return e;
    const Choice c = choose_matmul(a, d.sms);
    return c.split ? launch_matmul_narrow(dtype, a, c.tokens, c.split, d, s)
                   : launch_matmul_wide(dtype, a, d, s);
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
