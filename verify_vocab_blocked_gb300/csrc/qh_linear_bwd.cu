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
            const float p = silu_gate(z);
            return p * fmaf(z, 1.f - p, 1.f);
        }
        case kActGelu: {  // Phi(z) + z phi(z)
            const float2 n = normal_tail(z, z * z);
            return fmaf(z * 0.39894228f, n.y, z < 0.f ? n.x : 1.f - n.x);
        }
        case kActGeluTanh: {  // s = (1 + tanh u) / 2;  s + z u' 2 s (1 - s)
            const float z2 = z * z, s = tanh_gate(z, z2);
            return fmaf(z * 1.5957691216f * fmaf(0.134145f, z2, 1.f), s * (1.f - s), s);
        }
        default: return 1.f;
    }
}

// Eight elements as they lie in memory, BYTES each.
template <int BYTES>
struct Piece {
    uint4 u[BYTES / 2];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * BYTES);
#pragma unroll
        for (int k = 0; k < BYTES / 2; ++k) u[k] = q[k];
    }
    __device__ __forceinline__ void get(int type, float (&v)[8]) const {
        if constexpr (BYTES == 4) load8(reinterpret_cast<const float*>(u), v);
        else if (type == kSbBf16) load8(reinterpret_cast<const __nv_bfloat16*>(u), v);
        else load8(reinterpret_cast<const __half*>(u), v);
    }
};

template <int ACT>
__device__ __forceinline__ void times_grad(float (&g)[8], const float (&z)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] *= act_grad(z[e], ACT);
}
__device__ __forceinline__ void times_grad(float (&g)[8], const float (&z)[8], int act) {
    switch (act) {
        case kActRelu: times_grad<kActRelu>(g, z); break;
        case kActSilu: times_grad<kActSilu>(g, z); break;
        case kActGelu: times_grad<kActGelu>(g, z); break;
        case kActGeluTanh: times_grad<kActGeluTanh>(g, z); break;
        default: break;
    }
}

// The block's column sums from its warps', in order: sums[w][c] of column c.
__device__ __forceinline__ void write_sums(const DzArgs& a, const float (*sums)[kCols]) {
    __syncthreads();
    const int64_t n = (int64_t)blockIdx.x * kCols + threadIdx.x;
    if (n >= a.N) return;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][threadIdx.x];
    a.part[blockIdx.y * a.N + n] = s;
}

// 16-byte accesses: a lane's 8 columns of kRows rows at a time, all of whose loads
// are in flight together.  DB: bytes of dy's elements.  One round of blocks on the SMs:
// 8192 x 10240 bf16 with silu 95 us, 5.3 TB/s (107 with four rows and blocks as many as
// six to an SM, of which two fit).
constexpr int dz_blocks(int bytes) { return bytes == 4 ? 3 : 4; }  // to an SM
template <int DB>
__global__ void __launch_bounds__(32 * kWarps, dz_blocks(DB)) dz_kernel(const DzArgs a, int64_t run) {
    __shared__ float sums[kWarps][kCols];
    constexpr int kRows = DB == 4 ? 2 : 3;
    tc::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = (int64_t)blockIdx.x * kCols + 8 * lane;
    const int64_t r1 = min(a.M, ((int64_t)blockIdx.y + 1) * run);
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    if (c0 < a.N) {
        for (int64_t r = blockIdx.y * run + warp; r < r1; r += kRows * kWarps) {
            Piece<DB> pg[kRows];
            Piece<2> pz[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int64_t m = r + k * kWarps;
                if (m >= r1) continue;
                pg[k].load(a.dy, m * a.ldy + c0);
                if (a.act != kActNone) pz[k].load(a.pre, m * a.N + c0);
            }
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int64_t m = r + k * kWarps;
                if (m >= r1) continue;
                float g[8], z[8];
                pg[k].get(a.dy_type, g);
                if (a.act != kActNone) {
                    pz[k].get(kSbF16, z);
                    times_grad(g, z, a.act);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += g[e];
                if (a.dz) store8_as(a.dz, m * a.ldz + c0, a.type, g);
            }
        }
    }
    tc::grid_dep_trigger();
    if (!a.db) return;
#pragma unroll
    for (int e = 0; e < 8; e += 4)
        *reinterpret_cast<float4*>(&sums[warp][8 * lane + e]) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    write_sums(a, sums);
}

// Any alignment and width: a lane's columns are 32 apart.
__global__ void __launch_bounds__(32 * kWarps) dz_elem_kernel(const DzArgs a, int64_t run) {
    __shared__ float sums[kWarps][kCols];
    tc::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = (int64_t)blockIdx.x * kCols + lane;
    const int64_t r1 = min(a.M, ((int64_t)blockIdx.y + 1) * run);
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int64_t r = blockIdx.y * run + warp; r < r1; r += kWarps) {
        float g[8], z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool in = c0 + 32 * e < a.N;
            g[e] = in ? sb_elem(a.dy, r * a.ldy + c0 + 32 * e, a.dy_type) : 0.f;
            z[e] = in && a.act != kActNone ? __half2float(a.pre[r * a.N + c0 + 32 * e]) : 0.f;
        }
        times_grad(g, z, a.act);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[e] += g[e];
            if (!a.dz || c0 + 32 * e >= a.N) continue;
            const int64_t at = r * a.ldz + c0 + 32 * e;
            if (a.type == kSbBf16) static_cast<__nv_bfloat16*>(a.dz)[at] = __float2bfloat16_rn(g[e]);
            else static_cast<__half*>(a.dz)[at] = __float2half_rn(g[e]);
        }
    }
    tc::grid_dep_trigger();
    if (!a.db) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[warp][lane + 32 * e] = acc[e];
    write_sums(a, sums);
}

// 32 columns a block of 32 x 16: chunks y, y + 16, ... a thread, then the 16 in order.
constexpr int kJoinRows = 16;
__global__ void __launch_bounds__(32 * kJoinRows) db_join_kernel(const float* part, int chunks, int64_t N, void* db,
                                                                 int type) {
    __shared__ float sh[kJoinRows][33];
    tc::grid_dep_wait();
    const int64_t n = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const int y = threadIdx.y;
    float s = 0.f;
    if (n < N) {
#pragma unroll 4
        for (int c = y; c < chunks; c += kJoinRows) s += part[c * N + n];
    }
    sh[y][threadIdx.x] = s;
    __syncthreads();
    if (y > 0 || n >= N) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) s += sh[i][threadIdx.x];
    if (type == kSbF32) static_cast<float*>(db)[n] = s;
    else if (type == kSbBf16) static_cast<__nv_bfloat16*>(db)[n] = __float2bfloat16_rn(s);
    else static_cast<__half*>(db)[n] = __float2half_rn(s);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

int dz_chunks(int64_t M, int64_t N, int dy_type) {
    // the blocks that 152 SMs hold (the query of the size needs no device), of 16 rows at least
    const int64_t strips = (N + kCols - 1) / kCols, most = dz_blocks(type_bytes(dy_type)) * 152 / strips;
    return (int)std::max<int64_t>(1, std::min<int64_t>((M + 15) / 16, most));
}

cudaError_t launch_dz(const DzArgs& a, cudaStream_t st) {
    const int chunks = dz_chunks(a.M, a.N, a.dy_type);
    const int64_t run = (a.M + chunks - 1) / chunks;
    const dim3 grid((unsigned)((a.N + kCols - 1) / kCols), (unsigned)chunks);
    const bool vec = a.N % 8 == 0 && a.ldy % 8 == 0 && aligned16(a.dy) && aligned16(a.pre) && aligned16(a.dz) &&
                     (!a.dz || a.ldz % 8 == 0);
    const dim3 block(32 * kWarps);
    cudaError_t e = !vec                        ? launch_after(dz_elem_kernel, grid, block, st, a, run)
                    : type_bytes(a.dy_type) == 4 ? launch_after(dz_kernel<4>, grid, block, st, a, run)
                                                 : launch_after(dz_kernel<2>, grid, block, st, a, run);
    if (e || !a.db) return e;
    return launch_after(db_join_kernel, dim3((unsigned)((a.N + 31) / 32)), dim3(32, kJoinRows), st, (const float*)a.part,
                        chunks, a.N, a.db, a.db_type);
}

}  // namespace qh
