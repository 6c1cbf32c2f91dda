// The two kernels behind the 8-bit products and what they share on the host.
#pragma once

#include <cuda.h>

#include "expert_internal.h"

namespace arf {

// A byte matrix [rows][depth] read in boxes of box_rows x 128 bytes, 128-byte
// swizzle, zeros outside.  False if the driver refuses.
bool byte_tensor_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t depth,
                     uint32_t box_rows);

// The output [rows][cols] as a target of stores of box_rows x box_cols, in the
// 64-byte swizzle (box_cols elements are 64 bytes).  cols * elem is a multiple of 16.
bool out_tensor_map(CUtensorMap* map, void* base, uint64_t rows, uint64_t cols, int dtype,
                    uint32_t box_rows, uint32_t box_cols);

// Rows of 16-bit heads as boxes of 64 elements in the 128-byte swizzle, or (dtype AR_DT_E4M3) of
// codes as boxes as they lie; zeros outside.  Strides in bytes, of dimensions 1 to 3.
bool rows_tensor_map(CUtensorMap* map, int dtype, const void* base, const uint64_t (&dims)[4],
                     const uint64_t (&strides)[3], const uint32_t (&box)[4]);

constexpr int kStatusWords = 2;     // code, detail
struct DeviceInfo {
    int sms;
    int* status;                // device status words: of the products, then of attention
};
// The answer of the status calls; `which` 0: products, 1: attention.
int read_status(int which, void* stream, int* detail, const char* message);
// Of the current device.
cudaError_t device_info(DeviceInfo* out);

// The kernel of a call: the one for few rows with `tokens` (16, 32 or 64) of them at
// a time and the depth split over `split` blocks, or, split 0, the one for many.
struct Choice {
    int tokens, split;
};
Choice choose_matmul(const MatmulArgs& a, int sms);

// Tokens on the lanes of tensor memory, 256 x 256 outputs per pair of blocks: many rows.
cudaError_t launch_matmul_wide(int dtype, const MatmulArgs& a, const DeviceInfo& d,
                               cudaStream_t s);
// Weights on the lanes, `tokens` (16, 32 or 64) rows at a time, the depth
// split over `split` blocks of a cluster: few rows per expert.
cudaError_t launch_matmul_narrow(int dtype, const MatmulArgs& a, int tokens, int split,
                                 const DeviceInfo& d, cudaStream_t s);

}  // namespace arf
