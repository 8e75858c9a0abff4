// qh_linear.cuh -- launchers of the matrix product with its epilogue and of its
// gradient (qh_linear.cu, qh_linear_few.cu, qh_linear_bwd.cu).
#pragma once

#include <cuda.h>

#include "qh_ops.cuh"
#include "qh_tc.cuh"

namespace qh {

// Activations (the values of QHEAD_ACT_* in the public header).
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;
// 8-bit operands (QHEAD_E4M3); kSb* are the other element types.
constexpr int kE4m3 = 3;

// 1 / (1 + 2^a): an infinite power gives 0.
__device__ __forceinline__ float logistic2(float a) { return tc::rcp_approx(1.f + tc::ex2_approx(a)); }
// silu(z) / z, and (1 + tanh u) / 2 = 1 / (1 + exp(-2u)) of gelu's form with tanh, u =
// sqrt(2 / pi) (z + 0.044715 z^3); log2(e) in the constants.
__device__ __forceinline__ float silu_gate(float z) { return logistic2(z * -1.4426950409f); }
__device__ __forceinline__ float tanh_gate(float z, float z2) {
    return logistic2(z * fmaf(z2, -0.10294324f, -2.3022082f));
}

// The normal distribution beyond |z|: its mass h = Phi(-|z|), and exp(-z^2 / 2).
// From erfc(x) = p(t) exp(-x^2), t = 1 / (1 + 0.3275911 x) with p of degree 5
// (Abramowitz and Stegun, 7.1.26; off by at most 1.5e-7, so gelu and its derivative by
// 0.8e-7 |z|), a third of erff's instructions.  Here x = |z| / sqrt(2) and h = erfc / 2.
__device__ __forceinline__ float2 normal_tail(float z, float z2) {
    const float t = tc::rcp_approx(fmaf(0.23164189f, fabsf(z), 1.f));
    float p = fmaf(0.5307027145f, t, -0.7265760135f);
    p = fmaf(p, t, 0.7107068705f);
    p = fmaf(p, t, -0.142248368f);
    p = fmaf(p, t, 0.127414796f) * t;
    const float e = tc::ex2_approx(z2 * -0.7213475204f);
    return make_float2(p * e, e);
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
    bool sums;         // pairs: the reduction in sums of sum_steps stages
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
    void* db;            // [N] of db_type
    int db_type;
    float* part;         // [dz_chunks(M, N, dy_type), N]
};
int dz_chunks(int64_t M, int64_t N, int dy_type);
cudaError_t launch_dz(const DzArgs& a, cudaStream_t st);

}  // namespace qh
