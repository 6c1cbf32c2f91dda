// Two threads that call the attention-layer entry points on one stream with one workspace, over a
// CUDA runtime of this file that notes the launches instead of making them.  What is noted must be
// each call's kernel with its own join behind it.  Prints what is not so; 0: all is.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstring>
#include <mutex>
#include <random>
#include <thread>
#include <vector>

#include "ar_fusion.h"
#include "matmul_internal.h"

namespace {

struct Launch {
    std::thread::id by;
    unsigned blocks, threads;
};
std::mutex g_mu;
std::vector<Launch> g_launches;
int g_status[8];

}  // namespace

// ------------------------------------------- of the runtime, what the calls use
extern "C" {
void** __cudaRegisterFatBinary(void*) { static void* handle; return &handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaSuccess; }
unsigned __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "error"; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*)
{
    memset(a, 0, sizeof *a);
    a->numRegs = 255;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void**)
{
    thread_local std::mt19937 rng((unsigned)std::hash<std::thread::id>()(std::this_thread::get_id()));
    {
        std::lock_guard<std::mutex> lk(g_mu);
        g_launches.push_back({std::this_thread::get_id(), c->gridDim.x, c->blockDim.x});
    }
    for (unsigned i = rng() % 4; i; --i)
        std::this_thread::yield();
    return cudaSuccess;
}
}

// ------------------------------------------- of the library, what the calls use
namespace arf {
int set_last_error(int code, const char* m) { printf("%d: %s\n", code, m); return code; }
cudaError_t device_info(DeviceInfo* d) { *d = DeviceInfo{152, g_status}; return cudaSuccess; }
bool rows_tensor_map(CUtensorMap*, int, const void*, const uint64_t (&)[4], const uint64_t (&)[3],
                     const uint32_t (&)[4])
{
    return true;
}
}  // namespace arf

int main()
{
    constexpr int kCalls = 2000;
    void* const p = reinterpret_cast<void*>(uintptr_t{1} << 20);
    const auto calls = [&](int keys, bool prompts) {
        const ar_kv_cache c = {p, p, 16 * 128, 128, 64, 16 * 128, 128, 64, AR_DT_BF16, 4096, 16, 2, 64, 3,
                               keys / 16, nullptr, static_cast<int32_t*>(p), static_cast<int32_t*>(p)};
        const ar_head_rows rows = {p, 512, 64};
        for (int i = 0; i < kCalls; ++i) {
            const int rc = prompts && i % 2
                               ? ar_fusion_prompt_attention(&c, &rows, &rows, nullptr, static_cast<int32_t*>(p),
                                                            5, 8, AR_DT_BF16, 0.1f, 0, 0, p, 32 << 20, nullptr)
                               : ar_fusion_decode_attention(&c, &rows, &rows, nullptr, 8, AR_DT_BF16, 0.1f, 0,
                                                            0, p, 32 << 20, nullptr);
            if (rc != AR_OK)
                exit(3);
        }
    };
    std::thread one(calls, 8192, false), two(calls, 4096, true);
    one.join();
    two.join();
    if (g_launches.size() != 4 * kCalls) {
        printf("%zu launches, expected %d\n", g_launches.size(), 4 * kCalls);
        return 1;
    }
    int turns = 0, apart = 0;
    for (size_t i = 0; i < g_launches.size(); i += 2) {
        const Launch &kernel = g_launches[i], &join = g_launches[i + 1];
        apart += kernel.by != join.by || kernel.blocks != join.blocks || kernel.threads == 256 ||
                 join.threads != 256;
        turns += i && g_launches[i - 1].by != kernel.by;
    }
    printf("%d changes of thread, %d kernels without their join behind them\n", turns, apart);
    return apart ? 1 : turns < 10 ? 4 : 0;      // 4: the threads hardly met
}
