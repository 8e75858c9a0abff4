// qh_linear_bwd.cu -- what the gradient of the matrix product needs beside its
// two products: the activation's derivative and the bias gradient.
//
//     dz = dy act'(pre);   db[n] = sum_m dz[m, n]
//
// One pass over dy and pre, bound by its bytes.  dz is an operand of the tensor
// cores, which take one 16-bit type: it is rounded to x's (the products' own
// outputs are rounded to it too).  db is summed in fp32 from the unrounded
// values: each block sums a strip of 256 columns over a run of rows, a second
// launch adds the blocks' sums in order (deterministic).
#include "qh_linear.cuh"
#include "qh_tc.cuh"

#include <algorithm>

namespace qh {

namespace {

constexpr int kCols = 256, kWarps = 8;

__device__ __forceinline__ float act_grad(float z, int act) {
    switch (act) {
        case kActRelu: return z > 0.f ? 1.f : z != z ? z : 0.f;
        case kActSilu: {
            const float p = __fdividef(1.f, 1.f + __expf(-z));
            return p * fmaf(z, 1.f - p, 1.f);
        }
        case kActGelu: return fmaf(z * 0.39894228f, __expf(-0.5f * z * z), 0.5f * (1.f + erff(z * 0.70710678f)));
        case kActGeluTanh: {  // s = (1 + tanh u) / 2;  s + z u' 2 s (1 - s)
            const float z2 = z * z;
            const float s = __fdividef(1.f, 1.f + __expf(-1.5957691216f * fmaf(0.044715f * z2, z, z)));
            return fmaf(z * 1.5957691216f * fmaf(0.134145f, z2, 1.f), s * (1.f - s), s);
        }
        default: return 1.f;
    }
}

// A thread's 8 columns: in a row (VEC: 16-byte accesses), or 32 apart.
template <bool VEC>
__global__ void __launch_bounds__(32 * kWarps) dz_kernel(const DzArgs a, int64_t run) {
    __shared__ float sums[kWarps][kCols];
    tc::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = (int64_t)blockIdx.x * kCols + (VEC ? 8 * lane : lane);
    const int64_t r1 = min(a.M, ((int64_t)blockIdx.y + 1) * run);
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    if (c0 < a.N) {
#pragma unroll 2
        for (int64_t r = blockIdx.y * run + warp; r < r1; r += kWarps) {
            float g[8], z[8];
            if constexpr (VEC) {
                load8_as(a.dy, r * a.ldy + c0, a.dy_type, g);
                if (a.act != kActNone) load8(a.pre + r * a.N + c0, z);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool in = c0 + 32 * e < a.N;
                    g[e] = in ? sb_elem(a.dy, r * a.ldy + c0 + 32 * e, a.dy_type) : 0.f;
                    z[e] = in && a.act != kActNone ? __half2float(a.pre[r * a.N + c0 + 32 * e]) : 0.f;
                }
            }
            if (a.act != kActNone) {
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] *= act_grad(z[e], a.act);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += g[e];
            if (a.dz) {
                if constexpr (VEC) {
                    store8_as(a.dz, r * a.ldz + c0, a.type, g);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (c0 + 32 * e >= a.N) continue;
                        const int64_t at = r * a.ldz + c0 + 32 * e;
                        if (a.type == kSbBf16) static_cast<__nv_bfloat16*>(a.dz)[at] = __float2bfloat16_rn(g[e]);
                        else static_cast<__half*>(a.dz)[at] = __float2half_rn(g[e]);
                    }
                }
            }
        }
    }
    if (!a.db) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[warp][VEC ? 8 * lane + e : lane + 32 * e] = acc[e];
    __syncthreads();
    const int64_t n = (int64_t)blockIdx.x * kCols + threadIdx.x;
    if (n >= a.N) return;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][threadIdx.x];
    a.part[blockIdx.y * a.N + n] = s;
}

__global__ void __launch_bounds__(256) db_join_kernel(const float* part, int chunks, int64_t N, void* db, int type) {
    tc::grid_dep_wait();
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float s = 0.f;
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) s += part[c * N + n];
    if (type == kSbBf16) static_cast<__nv_bfloat16*>(db)[n] = __float2bfloat16_rn(s);
    else static_cast<__half*>(db)[n] = __float2half_rn(s);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

int dz_chunks(int64_t M, int64_t N) {
    const int64_t strips = (N + kCols - 1) / kCols;
    // about six blocks to each of 152 SMs, of 16 rows at least
    return (int)std::max<int64_t>(1, std::min<int64_t>((M + 15) / 16, (6 * 152 + strips - 1) / strips));
}

cudaError_t launch_dz(const DzArgs& a, cudaStream_t st) {
    const int chunks = dz_chunks(a.M, a.N);
    const int64_t run = (a.M + chunks - 1) / chunks;
    const dim3 grid((unsigned)((a.N + kCols - 1) / kCols), (unsigned)chunks);
    const bool vec = a.N % 8 == 0 && a.ldy % 8 == 0 && aligned16(a.dy) && aligned16(a.pre) && aligned16(a.dz) &&
                     (!a.dz || a.ldz % 8 == 0);
    cudaError_t e = vec ? launch_after(dz_kernel<true>, grid, dim3(32 * kWarps), st, a, run)
                        : launch_after(dz_kernel<false>, grid, dim3(32 * kWarps), st, a, run);
    if (e || !a.db) return e;
    return launch_after(db_join_kernel, dim3((unsigned)((a.N + 255) / 256)), dim3(256), st, a.part, chunks, a.N, a.db,
                        a.type);
}

}  // namespace qh
