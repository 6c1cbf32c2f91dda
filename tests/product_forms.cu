// The products' kernels with their form given rather than chosen, for the tests.
// Built twice: against the library, and (PRODUCT_FORMS_ALONE) with the kernels'
// sources under another namespace and a shorter limit of their waits.
#include <cuda_runtime.h>

#include "ar_internal.h"
#include "matmul_internal.h"
#include "tensor_core.cuh"

#ifdef PRODUCT_FORMS_ALONE
int arf::set_last_error(int code, const char*) { return code; }
#endif

using namespace arf;

namespace {

// A wait for an arrival that never comes, with nothing in flight: out[0] is its
// answer, out[1] that of a second wait once the block's flag is set, out[2] that of
// a wait for an arrival that came.
__global__ void wait_kernel(int* status, int where, int* out)
{
    __shared__ __align__(8) uint64_t bar;
    __shared__ int dead;
    dead = 0;
    bar_init(smem_u32(&bar), 1);
    __syncthreads();
    const Bail bail{smem_u32(&dead), status};
    out[0] = bar_wait(smem_u32(&bar), 0, bail, where);
    out[1] = bar_wait(smem_u32(&bar), 0, bail, where + 1);
    bar_arrive(smem_u32(&bar));
    out[2] = bar_wait(smem_u32(&bar), 0, bail, where + 2);
}

}  // namespace

// tokens 0: the kernel for many rows; else the one for few with that many rows at a
// time and the depth split over `split` blocks.
extern "C" int product_form(const void* a, const float* sa, const void* b, const float* sb,
                            const int* offsets, int experts, int rows, int cols, int depth,
                            int dtype, void* out, int tokens, int split, void* stream)
{
    const MatmulArgs m{static_cast<const uint8_t*>(a), sa, static_cast<const uint8_t*>(b), sb,
                       offsets, experts, rows, cols, depth, out};
    DeviceInfo d;
    const cudaError_t e = device_info(&d);
    if (e != cudaSuccess)
        return e;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return tokens ? launch_matmul_narrow(dtype, m, tokens, split, d, s)
                  : launch_matmul_wide(dtype, m, d, s);
}

extern "C" void product_choice(int experts, int rows, int cols, int depth, int sms, int* tokens,
                               int* split)
{
    const MatmulArgs m{nullptr, nullptr, nullptr, nullptr, nullptr, experts, rows, cols, depth, nullptr};
    const Choice c = choose_matmul(m, sms);
    *tokens = c.tokens;
    *split = c.split;
}

extern "C" int lone_wait(int where, int* out)
{
    DeviceInfo d;
    const cudaError_t e = device_info(&d);
    if (e != cudaSuccess)
        return e;
    wait_kernel<<<1, 1>>>(d.status, where, out);
    return cudaGetLastError();
}
