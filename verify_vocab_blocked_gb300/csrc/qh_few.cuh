// qh_few.cuh -- the dh contraction of up to kFewRows rows (qh_few.cu).
#pragma once

#include "qh_internal.cuh"

namespace qh {

constexpr int kFewRows = 16;

// Vocab ranges of the contraction: its partials are [ranges, kFewRows, H] fp32.
int few_splits(int64_t M, int64_t V, int H, int bits);

// dh [M, H] bf16 = (-geff[r] 2^-14) * sum_v coeff[pos[r], v] w[v, :], M <= kFewRows;
// coeff [>= M rows, ldc] fp16, 32-byte aligned rows, zero in the columns from V up
// to the next multiple of 64.  Inactive rows (pos < 0) are zeros.
cudaError_t launch_few_dh(const uint32_t* wq, const __half* scales, const __half* biases, int64_t V, int H,
                          int bits, const __half* coeff, int64_t ldc, int64_t M, const int* pos,
                          const float* geff, const int* err, float* part, void* dh, cudaStream_t st);

}  // namespace qh
