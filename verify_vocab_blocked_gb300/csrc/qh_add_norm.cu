// qh_add_norm.cu -- the residual's addition and the norm behind it, and the norm
// with an 8-bit output.
//
//     t = x + r;   y = norm(t) w + b   (qh_norm.cu's norm, of the unrounded t)
//     8 bits: scale = max |y| / 448 over the row, code = e4m3(y / scale)
//
// One pass: x and r are read once, t and y (or its codes) written once; the row
// stays in registers as fp32 between its sums.  The gradient is the norm's at the
// stored t plus what arrives at t itself.
#include <cuda_fp8.h>

#include "qh_norm.cuh"

namespace qh {

namespace {

constexpr float kE4m3Max = 448.f;

// Blocks of single-element rows to an SM (each within 65536 registers: five arrays of NE).
constexpr int elem_add_blocks(int nt, int ne) { return nt > 256 ? 1 : ne <= 8 ? 768 / elem_block(nt) : 2; }

// Largest over the G warps that share a row (every lane gets it; NaN is passed over).
template <int G>
__device__ __forceinline__ float row_max(float v, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (G > 1) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < G; ++w) v = fmaxf(v, red[w]);
        __syncthreads();
    }
    return v;
}

// Scale of a row whose largest magnitude is `top`, and its reciprocal for the codes.
// (A row of zeros has a scale too small to matter instead of a division by 0.)
__device__ __forceinline__ float2 scale_of(float top) {
    top = fmaxf(top, 1e-30f);
    return make_float2(top / kE4m3Max, kE4m3Max / top);
}

// Eight elements as they lie in memory, BYTES each, and widened.
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

// Bound by bytes: 32768 x 1536, x and y bf16, a float32 residual, centred: 89 us, 6.8
// TB/s; 8192 x 2560 bf16 to 8 bits: 23 us in the kernel, 6.4 TB/s.
//
// Rows in 16-byte accesses.  G warps a row (G = 1: several rows a block), NV pieces
// of 8 a thread, all of whose loads are in flight at once; XB, RB: bytes of x's and
// r's elements (RB = 0: no residual).
template <int XB, int RB, int NV, int G>
__global__ void __launch_bounds__(G == 1 ? 128 : 32 * G) add_norm_kernel(const AddNormArgs a) {
    __shared__ float red[G];
    const int t = G == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t r = G == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    if (G == 1 && r >= a.M) return;  // (whole warps)
    float v[NV][8];
    {
        Piece<XB> px[NV];
        Piece<RB ? RB : 2> pr[RB ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = (t + 32 * G * i) * 8;
            if (d >= a.H) continue;
            px[i].load(a.x, r * a.ldx + d);
            if constexpr (RB) pr[i].load(a.res, r * a.ldr + d);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = (t + 32 * G * i) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
            if (d >= a.H) continue;
            px[i].get(a.x_type, v[i]);
            if constexpr (RB) {
                float w[8];
                pr[i].get(a.r_type, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] += w[e];
                store8_as(a.total, r * a.H + d, a.r_type, v[i]);
            }
        }
    }
    const float inv = 1.f / (float)a.H;
    float mean = 0.f;
    if (a.center) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[i][e];
        mean = row_sum<G>(sum, red) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] -= mean;
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((t + 32 * G * i) * 8 >= a.H) continue;  // (centred, what lies past the row is not 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(v[i][e], v[i][e], sq);
    }
    const float rstd = 1.f / sqrtf(row_sum<G>(sq, red) * inv + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (t + 32 * G * i) * 8;
        if (d >= a.H) continue;
        float w[8], b[8];
        load8_as(a.w, d, a.w_type, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = 0.f;
        if (a.b) load8_as(a.b, d, a.w_type, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[i][e] = fmaf(v[i][e] * rstd, w[e], b[e]);
            top = fmaxf(top, fabsf(v[i][e]));
        }
        if (!a.scale) store8_as(a.y, r * a.H + d, a.y_type, v[i]);
    }
    if (!a.scale) return;
    const float2 s = scale_of(row_max<G>(top, red));
    if (t == 0) a.scale[r] = s.x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (t + 32 * G * i) * 8;
        if (d >= a.H) continue;
        uint32_t q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[i][4 * k] * s.y, v[i][4 * k + 1] * s.y),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[i][4 * k + 2] * s.y, v[i][4 * k + 3] * s.y),
                                                         __NV_SATFINITE, __NV_E4M3);
            q[k] = lo | hi << 16;
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + r * a.H + d) = make_uint2(q[0], q[1]);
    }
}

// Rows of any width and alignment, one element an access: a block of NT threads (a
// warp) a row, thread t's elements t + NT i, i < NE.  A thread keeps its columns'
// parameters over all the rows that its block walks, and the next row is on its way,
// held as it lies in memory, while a row's sums are joined.  The issue rate bounds
// these: 20001 x 2563 bf16 with a bf16 residual 100 us, 4.1 TB/s (114 with a row a
// block), float32 both 124 us, 5.8 TB/s.
template <int NT, int NE>
__global__ void __launch_bounds__(elem_block(NT), elem_add_blocks(NT, NE)) add_norm_elem_kernel(const AddNormArgs a) {
    __shared__ float red[2][3][64];
    constexpr int warps = NT / 32, rows = NT == 32 ? kElemWarps : 1;
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    const int t = threadIdx.x % NT;
    const float inv = 1.f / (float)a.H;
    const int left = a.H - t;  // element i exists: NT i < left
    float w[NE], b[NE];
    uint32_t x[NE], q[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        w[i] = b[i] = 0.f;
        q[i] = 0u;
        if (NT * i < left) {
            w[i] = sb_elem(a.w, t + NT * i, a.w_type);
            if (a.b) b[i] = sb_elem(a.b, t + NT * i, a.w_type);
        }
    }
    const auto raw = [&](const void* p, int type, int64_t at, uint32_t (&u)[NE]) {
        if (type == kSbF32) {
            const uint32_t* s = static_cast<const uint32_t*>(p) + at + t;
#pragma unroll
            for (int i = 0; i < NE; ++i) u[i] = NT * i < left ? s[NT * i] : 0u;
        } else {
            const unsigned short* s = static_cast<const unsigned short*>(p) + at + t;
#pragma unroll
            for (int i = 0; i < NE; ++i) u[i] = NT * i < left ? s[NT * i] : 0u;
        }
    };
    const auto fetch = [&](int64_t r) {
        if (r >= a.M) return;
        raw(a.x, a.x_type, r * a.ldx, x);
        if (a.res) raw(a.res, a.r_type, r * a.ldr, q);
    };
    const int64_t step = (int64_t)gridDim.x * rows;
    int64_t r = (int64_t)blockIdx.x * rows + threadIdx.x / NT;
    fetch(r);
    int flip = 0;
    for (; r < a.M; r += step, flip ^= 1) {
        float v[NE], mean = 0.f, sum = 0.f, sq = 0.f;
        as_type(a.x_type, [&](auto* tag) {
            using X = std::remove_pointer_t<decltype(tag)>;
#pragma unroll
            for (int i = 0; i < NE; ++i) v[i] = value_of<X>(x[i]);
        });
        if (a.res) {
            as_type(a.r_type, [&](auto* tag) {
                using R = std::remove_pointer_t<decltype(tag)>;
                R* p = static_cast<R*>(a.total) + r * a.H + t;
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    v[i] += value_of<R>(q[i]);
                    if (NT * i < left) p[NT * i] = (R)v[i];
                }
            });
        }
        fetch(r + step);
        if (a.center) {
#pragma unroll
            for (int i = 0; i < NE; ++i) sum += v[i];
            mean = block_sum1(sum, red[flip][0], warps) * inv;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (NT * i < left) v[i] -= mean;
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) sq = fmaf(v[i], v[i], sq);
        const float rstd = 1.f / sqrtf(block_sum1(sq, red[flip][1], warps) * inv + a.eps);
        if (t == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {  // (past the row: 0)
            v[i] = fmaf(v[i] * rstd, w[i], b[i]);
            if (NT * i < left) top = fmaxf(top, fabsf(v[i]));
        }
        if (!a.scale) {
            as_type(a.y_type, [&](auto* tag) {
                using Y = std::remove_pointer_t<decltype(tag)>;
                Y* y = static_cast<Y*>(a.y) + r * a.H + t;
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    if (NT * i < left) y[NT * i] = (Y)v[i];
            });
            continue;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) red[flip][2][threadIdx.x >> 5] = top;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < warps; ++k) top = fmaxf(top, red[flip][2][k]);
        }
        const float2 s = scale_of(top);
        if (t == 0) a.scale[r] = s.x;
        uint8_t* y = static_cast<uint8_t*>(a.y) + r * a.H + t;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (NT * i < left) y[NT * i] = __nv_cvt_float_to_fp8(v[i] * s.y, __NV_SATFINITE, __NV_E4M3);
    }
}

template <int XB, int RB, int NV, int G>
cudaError_t go(const AddNormArgs& a, cudaStream_t st) {
    // (few rows: one warp per block, spread over the SMs)
    const int rows = G > 1 || a.M < 2048 ? 1 : 4;
    return launch_after(add_norm_kernel<XB, RB, NV, G>, dim3((unsigned)((a.M + rows - 1) / rows)),
                        dim3(32 * (G > 1 ? G : rows)), st, a);
}

template <int XB, int RB>
cudaError_t pick(const AddNormArgs& a, cudaStream_t st) {
    const int H = a.H;
    if (H <= 256) return go<XB, RB, 1, 1>(a, st);
    if (H <= 512) return go<XB, RB, 2, 1>(a, st);
    if (H <= 1024) return go<XB, RB, 4, 1>(a, st);
    if (H <= 1536) return go<XB, RB, 3, 2>(a, st);
    if (H <= 2560) return go<XB, RB, 5, 2>(a, st);
    if (H <= 4096) return go<XB, RB, 4, 4>(a, st);
    return go<XB, RB, 4, 8>(a, st);
}

}  // namespace

cudaError_t launch_add_norm(const AddNormArgs& a, cudaStream_t st) {
    const bool vec = a.H % 8 == 0 && a.ldx % 8 == 0 && aligned16(a.x) && aligned16(a.y) && aligned16(a.w) &&
                     (!a.b || aligned16(a.b)) &&
                     (!a.res || (a.ldr % 8 == 0 && aligned16(a.res) && aligned16(a.total)));
    if (!vec)
        return elem_shape(a.H, [&](auto nt, auto ne) {
            constexpr int NT = decltype(nt)::value, NE = decltype(ne)::value;
            const int64_t blocks = NT == 32 ? (a.M + kElemWarps - 1) / kElemWarps : a.M;
            const int64_t most = device_sms() * (int64_t)elem_add_blocks(NT, NE);
            return launch_after(add_norm_elem_kernel<NT, NE>, dim3((unsigned)(blocks < most ? blocks : most)),
                                dim3(elem_block(NT)), st, a);
        });
    const int rb = !a.res ? 0 : type_bytes(a.r_type);
    if (type_bytes(a.x_type) == 4) return rb == 0 ? pick<4, 0>(a, st) : rb == 2 ? pick<4, 2>(a, st) : pick<4, 4>(a, st);
    return rb == 0 ? pick<2, 0>(a, st) : rb == 2 ? pick<2, 2>(a, st) : pick<2, 4>(a, st);
}

cudaError_t launch_add_norm_bwd(const NormBwdArgs& a, cudaStream_t st) { return launch_bwd<true>(a, st); }

}  // namespace qh
