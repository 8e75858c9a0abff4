// qh_linear_epi.cuh -- what the two kernels of the matrix product share: the
// epilogue's arithmetic, the operands' descriptors and tensor maps, the launch.
#pragma once

#include <algorithm>

#include "qh_linear.cuh"
#include "qh_tc.cuh"
#include "qh_tmap.h"

namespace qh {

namespace {

constexpr int kRowBytes = 128;   // bytes of a K-major row a stage: 64 or 128 elements
// Stages of a tensor-core sum of a float32 output (see SUMS), a power of two: 8-bit products
// have few bits to lose.
__host__ __device__ constexpr int sum_steps(bool f8) { return f8 ? 32 : 8; }

// ----------------------------------------------------------------- epilogue

__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case kActRelu: return z < 0.f ? 0.f : z;  // (keeps NaN)
        case kActSilu: return z * silu_gate(z);
        case kActGelu: {
            const float h = normal_tail(z, z * z).x;
            return z * (z < 0.f ? h : 1.f - h);
        }
        case kActGeluTanh: return z * tanh_gate(z, z * z);
        default: return z;
    }
}

// The pre-activation as it is kept for the gradient, in fp16: beyond fp16's range every
// activation's derivative is what it is at the range's end, so that it saturates (NaN
// stays); below it, a value that is not 0 keeps its sign (relu's derivative is that) as
// fp16's smallest, 2^-24.
__device__ __forceinline__ float in_half(float z) {
    float m = fabsf(z);
    asm("max.NaN.f32 %0, %0, 0f33800000;\n\tmin.NaN.f32 %0, %0, 0f477FE000;" : "+f"(m));  // 2^-24, 65504
    return z == 0.f ? z : copysignf(m, z);
}
__device__ __forceinline__ __half pre_of(float z) { return __float2half_rn(in_half(z)); }

__device__ __forceinline__ void put(void* p, int64_t i, int type, float v) {
    if (type == kSbF32) static_cast<float*>(p)[i] = v;
    else if (type == kSbBf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// What a kernel needs of LinArgs beside its tensor maps.
struct Epi {
    int64_t M, N;
    const float* a_scale;
    const float* b_scale;
    const void* bias;
    const void* res;
    void* y;
    __half* pre;
    int64_t ldr;
    int bias_type, act, res_type, y_type;
    int vec;           // the rows of y, pre and res are all aligned to 16 bytes
};

// One output of row m and column n, whose column's scale and bias are at hand.
__device__ __forceinline__ void finish(const Epi& e, int64_t m, int64_t n, float v, float bs, float bias) {
    if (e.a_scale) v *= e.a_scale[m];
    v = fmaf(v, bs, bias);
    const int64_t at = m * e.N + n;
    if (e.pre) e.pre[at] = pre_of(v);
    v = activate(v, e.act);
    if (e.res) v += sb_elem(e.res, m * e.ldr + n, e.res_type);
    put(e.y, at, e.y_type, v);
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int type) {
    if (type == kSbBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}


// One lane of a converged warp.  (The loops around it are run by the whole warp: the
// compiler then keeps descriptors and barriers in uniform registers.)
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Descriptor of an operand at `addr`: K-major rows of 128 bytes in 8-row atoms, or
// MN-major blocks of 64 elements 8 KB apart (64 rows of K each).
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return MN ? tc::sdesc_sw128(addr, 8192, 1024) : tc::sdesc_sw128(addr, 0, 1024);
}
// Its advance (in 16 bytes) per MMA: 32 bytes of K, or 16 rows of K.
template <bool MN>
constexpr uint32_t kStep = MN ? 128u : 2u;


// -------------------------------------------------------------------- host

// Instruction descriptor: fp32 accumulate; operand formats at bits 7 and 10
// (kind::f16: 0 fp16, 1 bf16; kind::f8f6f4: 0 e4m3).
inline uint32_t idesc_of(int type, int M, int N, bool amn, bool bmn) {
    const uint32_t f = type == kSbBf16 ? 1u : 0u;
    return tc::idesc_f16_f32(M, N, amn, bmn) | f << 7 | f << 10;
}

// The tensor map of an operand with `rows` of the output's side and `k` of the reduction.
inline bool map_operand(CUtensorMap* map, const LinOperand& o, int type, int64_t rows, int64_t k, int box_rows) {
    const int bytes = type == kE4m3 ? 1 : 2;
    return o.k_major ? tmap_rows_sw128(map, o.p, bytes, k, rows, o.ld * bytes, box_rows)
                     : tmap_rows_sw128(map, o.p, bytes, rows, k, o.ld * bytes, 64);
}

inline Epi epi_of(const LinArgs& a) {
    const auto rows = [](const void* p, int64_t ld, int type) {
        return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * type_bytes(type) % 16 == 0);
    };
    const bool vec = rows(a.y, a.N, a.y_type) && rows(a.pre, a.N, kSbF16) && rows(a.res, a.ldr, a.res_type);
    return Epi{a.M, a.N, a.a_scale, a.b_scale, a.bias, a.res, a.y, a.pre, a.ldr, a.bias_type, a.act, a.res_type, a.y_type,
               vec};
}

template <typename... P, typename... A>
cudaError_t launch_cluster(void (*fn)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t st, A... a) {
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), smem)) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(a)...);
}

// Whether the output asks for the tensor cores' sums to be short: see SUMS.
inline bool in_sums(const LinArgs& a) { return a.y_type == kSbF32; }

inline int steps(const LinArgs& a, int* step) {
    *step = a.type == kE4m3 ? 128 : 64;
    return (int)((a.K + *step - 1) / *step);
}

// Few rows: the columns of a CTA's accumulators at most, and the accumulators that `share`
// stages of the reduction take: one, or for float32 one for each sum_steps stages.
constexpr int few_tmem(int tile) { return tile <= 16 ? 128 : 256; }
inline int few_accs(const LinArgs& a, int share) {
    const int most = sum_steps(a.type == kE4m3);
    return in_sums(a) ? (share + most - 1) / most : 1;
}
inline bool few_fits(const LinArgs& a, int tile, int share) { return few_accs(a, share) * tile <= few_tmem(tile); }

}  // namespace

}  // namespace qh
