// qh_ops.cuh -- launchers of the operators beside the head (qh_embed.cu,
// qh_norm.cu) and their typed 8-element loads and stores.
#pragma once

#include "qh_internal.cuh"

namespace qh {

// Eight consecutive elements widened to fp32 (the address 16-byte aligned).
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        v[2 * i] = f.x; v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// One rounding to the element type.
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
    __half2 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(o);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    __nv_bfloat162 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(o);
}
// Eight fp32 in one 32-byte access (the address 32-byte aligned).
__device__ __forceinline__ void load8_wide(const float* p, float (&v)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                   "=f"(v[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store8_wide(float* p, const float (&v)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
                 "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
// The same on a pointer whose element type (kSb*) is known at run time only.
__device__ __forceinline__ void load8_as(const void* p, int64_t i, int type, float (&v)[8]) {
    if (type == kSbF32) load8(static_cast<const float*>(p) + i, v);
    else if (type == kSbBf16) load8(static_cast<const __nv_bfloat16*>(p) + i, v);
    else load8(static_cast<const __half*>(p) + i, v);
}
__device__ __forceinline__ void store8_as(void* p, int64_t i, int type, const float (&v)[8]) {
    if (type == kSbF32) store8(static_cast<float*>(p) + i, v);
    else if (type == kSbBf16) store8(static_cast<__nv_bfloat16*>(p) + i, v);
    else store8(static_cast<__half*>(p) + i, v);
}

// Two fp32 lanes per instruction (one issue slot for two products or sums).
__device__ __forceinline__ unsigned long long f2_bits(float2 a) {
    return *reinterpret_cast<unsigned long long*>(&a);
}
__device__ __forceinline__ float2 bits_f2(unsigned long long a) { return *reinterpret_cast<float2*>(&a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
    return bits_f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return bits_f2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return bits_f2(r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Code e (0 .. 7) of an 8-element unit (4 bits: one word, 8 bits: two) as fp32:
// placed in the mantissa of 2^23, which is subtracted exactly (a conversion
// instruction runs at an eighth of this rate).
template <int BITS>
__device__ __forceinline__ float code_f32(uint32_t w0, uint32_t w1, int e) {
    const uint32_t q = BITS == 4 ? (w0 >> (4 * e)) & 15u : ((e < 4 ? w0 : w1) >> (8 * (e & 3))) & 255u;
    return __uint_as_float(q | 0x4B000000u) - 8388608.f;
}

// Asynchronous copies global -> shared, of 16 bytes past L1, of fewer through it;
// of `bytes` < BYTES the rest is zeros.  The end of a group of them, and the wait
// that leaves the N youngest groups in flight.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int bytes) {
    static_assert(BYTES == 16, "cp.async size");
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

inline int type_bytes(int type) { return type == kSbF32 ? 4 : 2; }

// Launches fn as the programmatic dependent of the kernel before it on `st`: its
// blocks may start early and wait, with tc::grid_dep_wait() as their first
// statement (in every block, so that it ends only after that kernel).  What that
// kernel wrote is not read through const __restrict__ pointers: such loads may be
// moved above the wait.
template <typename... P, typename... A>
cudaError_t launch_after_smem(void (*fn)(P...), dim3 grid, dim3 block, int smem, cudaStream_t st, A... a) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(a)...);
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*fn)(P...), dim3 grid, dim3 block, cudaStream_t st, A... a) {
    return launch_after_smem(fn, grid, block, 0, st, a...);
}

// ---------------------------------------------------------------- embedding

cudaError_t launch_embed(const uint32_t* wq, SbView sb, int64_t V, int H, int bits,
                         const int32_t* tokens, const uint8_t* mask, int64_t M, float scale,
                         void* out, int out_type, cudaStream_t st);

// Workspace of the gradient: two buffers of sorted (token, row) pairs, the
// counts of live rows and of joins, two partial rows per chunk of sorted rows and
// the list of joins.
struct EmbedBwdPlan {
    int chunk = 0;       // sorted rows per block
    int64_t n_chunks = 0;
    size_t off_info = 0, off_a = 0, off_b = 0, off_part = 0, off_joins = 0, total = 0;
};
EmbedBwdPlan plan_embed_bwd(int64_t M, int H);
cudaError_t launch_embed_bwd(const EmbedBwdPlan& p, void* ws, int64_t V, int H,
                             const int32_t* tokens, const uint8_t* mask, int64_t M, float scale,
                             const void* dy, int dy_type, float* dw, bool accumulate,
                             cudaStream_t st);

// --------------------------------------------------------------- layer norm

struct NormArgs {
    const void* x;
    int x_type;
    int64_t ldx;
    int64_t M;
    int H;
    const void* w;
    const void* b;   // NULL: none
    int w_type;
    float eps;
    bool center;
    void* y;
    int y_type;
    float* mean;     // NULL unless center
    float* rstd;
};
cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st);

struct NormBwdArgs {
    const void* x;
    int x_type;
    int64_t ldx;
    int64_t M;
    int H;
    const void* w;
    int w_type;
    const float* mean;  // NULL: uncentred
    const float* rstd;
    const void* dy;
    int dy_type;
    int64_t ldy;
    void* dx;           // x's type, contiguous
    float* dw;
    float* db;          // NULL: not wanted
    float* part;        // [grid, 2, H]
    int grid;
    const void* add;    // x's type, rows of ldadd: added to dx (launch_add_norm_bwd)
    int64_t ldadd;
};
int norm_bwd_grid(int64_t M, int H);
cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t st);
cudaError_t launch_add_norm_bwd(const NormBwdArgs& a, cudaStream_t st);  // adds a.add into dx

// The norm of x + res (res NULL: of x), whose sum goes to `total`; scale: y is
// e4m3 codes, their row scales go there.
struct AddNormArgs {
    const void* x;
    int x_type;
    int64_t ldx;
    const void* res;
    int r_type;         // of res and total
    int64_t ldr;
    int64_t M;
    int H;
    const void* w;
    const void* b;      // NULL: none
    int w_type;
    float eps;
    bool center;
    void* total;        // [M, H] contiguous
    void* y;            // [M, H] contiguous
    int y_type;
    float* scale;       // NULL: y is of y_type
    float* mean;        // NULL: not wanted
    float* rstd;        // NULL: not wanted
};
cudaError_t launch_add_norm(const AddNormArgs& a, cudaStream_t st);

// ------------------------------------------------------------ gradient norm

struct GradTensors {
    const void* const* p;   // host arrays
    void* const* out;       // NULL: none are written; may be p
    const int64_t* n;
    const int* type;
    const int* out_type;
    int count;
};
size_t grad_norm_workspace(int count);
cudaError_t launch_grad_norm(const GradTensors& t, float max_norm, float* norm, void* ws, cudaStream_t st);

}  // namespace qh
