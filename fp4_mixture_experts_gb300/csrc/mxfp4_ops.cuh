// Declarations shared by the MXFP4 operators' translation units.
#pragma once

#include <cuda_fp16.h>

#include "moe_fp4_internal.cuh"

namespace moe_fp4 {

constexpr int kMaxGroups = 1024;

// rows to quantise: row r is row (row_index ? row_index[r] / div : r) of x
struct MxRows {
  const void* x;
  int64_t x_rows, x_stride;
  const int32_t* row_index;
  const int32_t* offsets;  // groups (tiled scales): [groups + 1], or null
  int64_t rows;
  int K, div, groups;
  bool f32;
};

int check_mx_rows(const MxRows& R);  // a moe_fp4_status
cudaError_t launch_mxfp4_quantize(const MxRows& R, uint8_t* codes, uint8_t* scales, bool tiled, cudaStream_t st);
// the error words of the operators' kernels (one in each translation unit): read, or cleared
cudaError_t ops_quant_error(int32_t* word, bool clear, cudaStream_t st);
cudaError_t ops_mm_error(int32_t* word, bool clear, cudaStream_t st);
cudaError_t ops_mm2_error(int32_t* word, bool clear, cudaStream_t st);

#ifdef __CUDACC__

// The group that holds row r: the last e with off[e] <= r, if r < off[e + 1];
// -1 if none does.  Offsets are taken as they are; a row is given a group only
// if the group lies in [0, rows], so that tile indices stay in their range.
__device__ __forceinline__ int find_group(const int32_t* off, int groups, int64_t r, int64_t rows) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(off + mid) <= r)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t first = __ldg(off + lo), end = __ldg(off + lo + 1);
  return first >= 0 && first <= r && r < end && end <= rows ? lo : -1;
}

#endif

}  // namespace moe_fp4
