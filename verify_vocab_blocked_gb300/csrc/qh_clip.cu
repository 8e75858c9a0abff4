// qh_clip.cu -- the global norm of many gradient tensors, and clipping.
//
//     norm = sqrt(sum over tensors and elements of g^2)
//     out  = g min(1, max_norm / (norm + 1e-6))
//
// Bound by bytes: every tensor is read once for the norm and, where it has to be
// scaled, read again and written.  The tensors' addresses travel as kernel
// parameters (no copy to the device, so that a call can be captured), in tables of
// up to 480; the elements are dealt to the blocks in chunks of 8192, whichever
// tensor they belong to.  The second pass takes the chunks in the opposite order,
// so that what the first left in L2 is read from there.
//
// Squares are summed in fp32 over a thread's 32 elements of a chunk and in fp64
// beyond; a thread whose fp32 sum overflowed or is so small that squares may have
// been lost sums its elements of that chunk in fp64.  The blocks' sums are added in
// a fixed order by every block of the second pass: deterministic, no atomics.
#include <algorithm>

#include "qh_norm.cuh"

namespace qh {

namespace {

constexpr int kThreads = 256, kChunk = 8192;
constexpr int kNormBlocks = 152 * 6;  // partial sums of a launch, at most

template <int MOST>
struct Table {
    const void* p[MOST];
    void* out[MOST];
    int64_t n[MOST];
    int first[MOST + 1];  // chunks before tensor i
    uint8_t type[MOST], out_type[MOST];
    int count;
};

// The tensor that chunk c belongs to.
template <typename Tab>
__device__ __forceinline__ int owner(const Tab& t, int c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Calls f(i, v, k) for a block's share of n elements at p: v holds k of them from
// index i on -- 8 at a time where 16-byte accesses reach, else one.
template <typename T, typename F>
__device__ __forceinline__ void for_elements(const T* p, int n, F&& f) {
    const int mis = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T);
    const int head = mis ? min(n, 16 / (int)sizeof(T) - mis) : 0;
    if ((int)threadIdx.x < head) f((int)threadIdx.x, p + threadIdx.x, 1);
    const int pieces = (n - head) / 8;
#pragma unroll 4
    for (int i = threadIdx.x; i < pieces; i += kThreads) f(head + 8 * i, p + head + 8 * i, 8);
    const int done = head + 8 * pieces;
    if ((int)threadIdx.x < n - done) f(done + (int)threadIdx.x, p + done + threadIdx.x, 1);
}

template <typename T>
__device__ __forceinline__ float one_of(const T* p) {
    return value_of<T>(raw_of(p));
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int n) {
    float s = 0.f, top = 0.f;
    for_elements(p, n, [&](int, const T* q, int k) {
        if (k == 8) {
            float v[8];
            load8(q, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s = fmaf(v[e], v[e], s);
                top = fmaxf(top, fabsf(v[e]));
            }
        } else {
            const float v = one_of(q);
            s = fmaf(v, v, s);
            top = fmaxf(top, fabsf(v));
        }
    });
    // 2^-80: squares lost below 2^-149 are then 2^-64 of the sum
    if ((s >= 8.3e-25f && s <= 3.4e38f) || (top == 0.f && s == 0.f)) return s;
    double d = 0.0;
    for_elements(p, n, [&](int, const T* q, int k) {
        for (int e = 0; e < k; ++e) {
            const double v = one_of(q + e);
            d = fma(v, v, d);
        }
    });
    return d;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += red[w];
    return v;
}

template <int MOST>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<MOST> t, double* part) {
    __shared__ double red[kThreads / 32];
    tc::grid_dep_wait();
    const int chunks = t.first[t.count];
    double sum = 0.0;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = owner(t, c);
        const int64_t at = (int64_t)(c - t.first[i]) * kChunk;
        const int n = (int)min((int64_t)kChunk, t.n[i] - at);
        as_type(t.type[i], [&](auto* tag) {
            using T = std::remove_pointer_t<decltype(tag)>;
            sum += chunk_squares(static_cast<const T*>(t.p[i]) + at, n);
        });
    }
    tc::grid_dep_trigger();  // (earlier, the next kernel's blocks would crowd some SMs)
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ double norm_of(const double* part, int parts, double* red) {
    double v = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) v += part[i];
    return sqrt(block_sum(v, red));
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* part, int parts, float* norm) {
    __shared__ double red[kThreads / 32];
    tc::grid_dep_wait();
    const double v = norm_of(part, parts, red);
    if (threadIdx.x == 0) *norm = (float)v;
}

template <typename T, typename O>
__device__ __forceinline__ void scale_chunk(const T* p, O* out, int n, float coef) {
    // 8 at a time where both sides' accesses are 16-byte aligned at the same elements
    const int mis = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T);
    const int head = mis ? 16 / (int)sizeof(T) - mis : 0;
    if ((reinterpret_cast<uintptr_t>(out + head) & 15) == 0) {
        for_elements(p, n, [&](int i, const T* q, int k) {
            if (k == 8) {
                float v[8];
                load8(q, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= coef;
                store8(out + i, v);
            } else {
                out[i] = (O)(one_of(q) * coef);
            }
        });
    } else {
#pragma unroll 8
        for (int i = threadIdx.x; i < n; i += kThreads) out[i] = (O)(one_of(p + i) * coef);
    }
}

template <int MOST>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<MOST> t, const double* part,
                                                         int parts, float max_norm, float* norm) {
    __shared__ double red[kThreads / 32];
    tc::grid_dep_wait();
    const double v = norm_of(part, parts, red);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
    float coef = (float)((double)max_norm / (v + 1e-6));
    if (coef > 1.f) coef = 1.f;  // (NaN stays)
    const int chunks = t.first[t.count];
    for (int c = chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
        const int i = owner(t, c);
        if (coef == 1.f && t.p[i] == t.out[i]) continue;  // in place, within the limit
        const int64_t at = (int64_t)(c - t.first[i]) * kChunk;
        const int n = (int)min((int64_t)kChunk, t.n[i] - at);
        as_type(t.type[i], [&](auto* tag) {
            using T = std::remove_pointer_t<decltype(tag)>;
            const T* p = static_cast<const T*>(t.p[i]) + at;
            as_type(t.out_type[i], [&](auto* otag) {
                using O = std::remove_pointer_t<decltype(otag)>;
                scale_chunk(p, static_cast<O*>(t.out[i]) + at, n, coef);
            });
        });
    }
}

constexpr int kFewTensors = 48, kManyTensors = 480;

// Fills a table with the tensors from `at` on; the chunks it holds.
template <int MOST>
int fill(Table<MOST>& tab, const GradTensors& t, int at) {
    tab.count = std::min(MOST, t.count - at);
    int chunks = 0;
    for (int i = 0; i < tab.count; ++i) {
        const int k = at + i;
        tab.p[i] = t.p[k];
        tab.out[i] = t.out ? t.out[k] : nullptr;
        tab.n[i] = t.n[k];
        tab.type[i] = (uint8_t)t.type[k];
        tab.out_type[i] = (uint8_t)(t.out ? t.out_type[k] : t.type[k]);
        tab.first[i] = chunks;
        chunks += (int)((t.n[k] + kChunk - 1) / kChunk);
    }
    tab.first[tab.count] = chunks;
    return chunks;
}

int blocks_of(int chunks) { return std::max(1, std::min(chunks, kNormBlocks)); }

template <int MOST>
cudaError_t run(const GradTensors& t, float max_norm, float* norm, double* part, cudaStream_t st) {
    Table<MOST> tab;
    int parts = 0;
    for (int at = 0; at < t.count; at += MOST) {
        const int blocks = blocks_of(fill(tab, t, at));
        if (cudaError_t e = launch_after(squares_kernel<MOST>, dim3((unsigned)blocks), dim3(kThreads), st, tab, part + parts))
            return e;
        parts += blocks;
    }
    if (!t.out) return launch_after(norm_kernel, dim3(1), dim3(kThreads), st, part, parts, norm);
    // (the last tables first, and the last chunks of each)
    for (int at = (t.count - 1) / MOST * MOST; at >= 0; at -= MOST) {
        const int blocks = blocks_of(fill(tab, t, at));
        if (cudaError_t e = launch_after(scale_kernel<MOST>, dim3((unsigned)blocks), dim3(kThreads), st, tab,
                                         (const double*)part, parts, max_norm, at == 0 ? norm : (float*)nullptr))
            return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t grad_norm_workspace(int count) {
    const int tables = count <= kFewTensors ? 1 : (count + kManyTensors - 1) / kManyTensors;
    return sizeof(double) * (size_t)kNormBlocks * tables;
}

cudaError_t launch_grad_norm(const GradTensors& t, float max_norm, float* norm, void* ws, cudaStream_t st) {
    double* part = static_cast<double*>(ws);
    return t.count <= kFewTensors ? run<kFewTensors>(t, max_norm, norm, part, st)
                                  : run<kManyTensors>(t, max_norm, norm, part, st);
}

}  // namespace qh
