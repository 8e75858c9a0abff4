// qh_linear.cuh -- launchers of the matrix product with its epilogue and of its
// gradient (qh_linear.cu, qh_linear_few.cu, qh_linear_bwd.cu).
#pragma once

#include <cuda.h>

#include "qh_ops.cuh"

namespace qh {

// Activations (the values of QHEAD_ACT_* in the public header).
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;
// 8-bit operands (QHEAD_E4M3); kSb* are the other element types.
constexpr int kE4m3 = 3;

// The normal distribution beyond |z|: its mass h = Phi(-|z|), and its density at z.
// From erfc(x) = p(t) exp(-x^2), t = 1 / (1 + 0.3275911 x) with p of degree 5
// (Abramowitz and Stegun, 7.1.26; off by at most 1.5e-7, so gelu and its derivative by
// 0.8e-7 |z|), a third of erff's instructions.
__device__ __forceinline__ float2 normal_tail(float z) {
    const float x = fabsf(z) * 0.70710678f;
    const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f) * t;
    const float e = __expf(-x * x);
    return make_float2(0.5f * p * e, 0.39894228f * e);
}

// A matrix operand of the product: rows of `ld` elements whose starts are
// 16-byte aligned.  k_major: the reduction runs along a row; else down the rows.
struct LinOperand {
    const void* p;
    int64_t ld;
    bool k_major;
};

// D[m, n] = sum_k A[m, k] B[n, k] of m < M, n < N, k < K, then, where given,
//     z = D a_scale[m] b_scale[n] + bias[n];  pre = fp16(z);  y = act(z) + res[m, n]
struct LinArgs {
    LinOperand a, b;
    int type;          // element type of A and B
    int64_t M, N, K;
    const float* a_scale;
    const float* b_scale;
    const void* bias;
    int bias_type;
    int act;
    const void* res;
    int res_type;
    int64_t ldr;
    void* y;           // [M, N]
    int y_type;
    __half* pre;       // [M, N]
    float* part;       // LinPlan::part_bytes
    int stall;         // test switch: no loads are issued, the waits expire
};

// The kernel and its tile for a product.
struct LinPlan {
    bool few;          // tokens on the tile's short side (else CTA pairs)
    int tile;          // few: rows of A a tile (16 .. 128); pairs: columns a tile
    int split;         // few: CTAs (of a cluster) that share a tile's reduction; pairs:
                       // parts of the reduction of each tile past the last full round
    int pairs;         // pairs: CTA pairs a round
    size_t part_bytes; // pairs: the parts' sums, 32-byte aligned (LinArgs::part)
};
LinPlan plan_linear(const LinArgs& a, int sms);
cudaError_t launch_linear(const LinArgs& a, const LinPlan& p, cudaStream_t st);
cudaError_t launch_linear_few(const LinArgs& a, const LinPlan& p, cudaStream_t st);  // p.few

// Rows of 1- or 2-byte elements into rows whose starts are 16-byte aligned.
cudaError_t launch_pad_rows(const void* src, int64_t ld, int64_t rows, int64_t cols, int bytes,
                            void* dst, int64_t ldd, cudaStream_t st);

// dz = dy act'(pre), rounded to `type`, into rows of `ldz` (NULL: not wanted),
// and the column sums of the unrounded dz (db NULL: not wanted).
struct DzArgs {
    const void* dy;
    int dy_type;
    int64_t ldy;
    const __half* pre;   // [M, N]; not read where act is none
    int act;
    int64_t M, N;
    void* dz;
    int64_t ldz;
    int type;
    void* db;            // [N] of `type`
    float* part;         // [dz_chunks(M, N, dy_type), N]
};
int dz_chunks(int64_t M, int64_t N, int dy_type);
cudaError_t launch_dz(const DzArgs& a, cudaStream_t st);

}  // namespace qh
