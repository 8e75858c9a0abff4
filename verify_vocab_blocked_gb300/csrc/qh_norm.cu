// qh_norm.cu -- layer norm (and its uncentred, root-mean-square form) before
// the head, and its gradient.
//
//     xc = x - mean(x)  (or x),  rstd = 1 / sqrt(mean(xc^2) + eps),  xh = xc rstd
//     y  = xh w + b
//     g  = dy w;  dx = rstd (g - [mean(g)] - xh mean(g xh));  dw = sum dy xh;  db = sum dy
//
// Bound by bytes: x is read once and y written once (the row stays in
// registers between its statistics and its output); backward x and dy once
// and dx once.  Statistics, sums and parameter gradients are fp32; the variance
// is taken from the centred values, so rows with a large mean lose nothing.
//
// dw and db: every block keeps its threads' columns in registers over all its
// rows and writes one partial row; a second launch adds the partial rows in
// order.  Deterministic, no atomics.
#include "qh_ops.cuh"
#include "qh_tc.cuh"

namespace qh {

namespace {

// V consecutive elements at element index i (V = 8: one or two 16-byte loads).
template <int V, typename T>
__device__ __forceinline__ void loadv(const T* p, float (&v)[V]) {
    if constexpr (V == 8) load8(p, v);
    else if constexpr (sizeof(T) == 4) v[0] = (float)*p;
    else v[0] = sb_elem(p, 0, std::is_same<T, __half>::value ? kSbF16 : kSbBf16);
}
template <int V>
__device__ __forceinline__ void loadv_as(const void* p, int64_t i, int type, float (&v)[V]) {
    if constexpr (V == 8) load8_as(p, i, type, v);
    else v[0] = sb_elem(p, i, type);
}
template <int V>
__device__ __forceinline__ void storev_as(void* p, int64_t i, int type, const float (&v)[V]) {
    if constexpr (V == 8) store8_as(p, i, type, v);
    else store_as(p, i, type, v[0]);
}

// Sum over the G warps that share a row (every lane gets it): shuffles, then,
// for a whole block on one row, the warps' sums in order.
template <int G>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (G > 1) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < G; ++w) v += red[w];
        __syncthreads();
    }
    return v;
}

// One row per G warps (G = 1: blockDim / 32 rows per block), NV pieces of V
// elements per thread held in registers: thread t of the row takes elements
// (t + 32 G i) V.
template <typename T, int V, int NV, int G>
__global__ void __launch_bounds__(G == 1 ? 256 : 32 * G) norm_fwd_kernel(const NormArgs a) {
    __shared__ float red[G];
    const int t = G == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t r = G == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (G == 1 && r >= a.M) return;  // (whole warps)
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    float v[NV][V];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (t + 32 * G * i) * V;
        if (d < a.H) {
            loadv<V>(x + d, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = 0.f;
        }
    }
    float mean = 0.f;
    const float inv = 1.f / (float)a.H;
    if (a.center) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) sum += v[i][e];
        mean = row_sum<G>(sum, red) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((t + 32 * G * i) * V < a.H) {
#pragma unroll
                for (int e = 0; e < V; ++e) v[i][e] -= mean;
            }
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) sq = fmaf(v[i][e], v[i][e], sq);
    const float rstd = 1.f / sqrtf(row_sum<G>(sq, red) * inv + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[r] = mean;
        a.rstd[r] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (t + 32 * G * i) * V;
        if (d >= a.H) continue;
        float w[V], b[V];
        loadv_as<V>(a.w, d, a.w_type, w);
#pragma unroll
        for (int e = 0; e < V; ++e) b[e] = 0.f;
        if (a.b) loadv_as<V>(a.b, d, a.w_type, b);
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] = fmaf(v[i][e] * rstd, w[e], b[e]);
        storev_as<V>(a.y, r * a.H + d, a.y_type, v[i]);
    }
}

// Two sums of R rows over the block: sums[2 r], sums[2 r + 1] in, totals out.
template <int N>
__device__ __forceinline__ void block_sums(float (&s)[N], float* red, int warps) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) red[k * 32 + warp] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        s[k] = lane < warps ? red[k * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    }
    __syncthreads();
}

// Block = R rows at a time, all columns; thread t takes elements
// (t + blockDim i) V.  The block's columns of dw and db stay in registers.
template <typename T, int V, int NV, int R, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormBwdArgs a) {
    __shared__ float red[2 * R * 32];
    const int t = threadIdx.x, nt = blockDim.x, warps = nt >> 5;
    const float inv = 1.f / (float)a.H;
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (t + nt * i) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.f;
        if (d < a.H) loadv_as<V>(a.w, d, a.w_type, w[i]);
    }
    for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.M; r0 += (int64_t)gridDim.x * R) {
        float x[R][NV][V], g[R][NV][V];
        float mean[R], rstd[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = r0 + k;
            const bool live = r < a.M;
            mean[k] = live && a.mean ? a.mean[r] : 0.f;
            rstd[k] = live ? a.rstd[r] : 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int d = (t + nt * i) * V;
                if (live && d < a.H) {
                    loadv<V>(static_cast<const T*>(a.x) + r * a.ldx + d, x[k][i]);
                    loadv_as<V>(a.dy, r * a.ldy + d, a.dy_type, g[k][i]);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        x[k][i][e] = mean[k];  // (its xh is 0)
                        g[k][i][e] = 0.f;
                    }
                }
            }
        }
        float s[2 * R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float c1 = 0.f, c2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (x[k][i][e] - mean[k]) * rstd[k];
                    const float dy = g[k][i][e];
                    dw[i][e] = fmaf(dy, xh, dw[i][e]);
                    db[i][e] += dy;
                    const float gw = dy * w[i][e];
                    c1 += gw;
                    c2 = fmaf(gw, xh, c2);
                    x[k][i][e] = xh;
                    g[k][i][e] = gw;
                }
            s[2 * k] = c1;
            s[2 * k + 1] = c2;
        }
        block_sums(s, red, warps);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = r0 + k;
            if (r >= a.M) break;
            const float c1 = a.mean ? s[2 * k] * inv : 0.f, c2 = s[2 * k + 1] * inv;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int d = (t + nt * i) * V;
                if (d >= a.H) continue;
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o[e] = rstd[k] * (g[k][i][e] - c1 - x[k][i][e] * c2);
                storev_as<V>(a.dx, r * a.H + d, a.x_type, o);
            }
        }
    }
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (t + nt * i) * V;
        if (d >= a.H) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            part[d + e] = dw[i][e];
            part[a.H + d + e] = db[i][e];
        }
    }
}

// 32 columns per block of 32 x 16: partial rows y, y + 16, ... per thread, then
// the 16 sums in order.  blockIdx.y: dw, db.
constexpr int kJoinRows = 16;
__global__ void __launch_bounds__(32 * kJoinRows) norm_join_kernel(const float* __restrict__ part,
                                                                   int n, int H,
                                                                   float* __restrict__ dw,
                                                                   float* __restrict__ db) {
    __shared__ float sh[kJoinRows][33];
    const int d = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
    float s = 0.f;
    if (d < H) {
        const float* p = part + (int64_t)blockIdx.y * H + d;
#pragma unroll 4
        for (int i = y; i < n; i += kJoinRows) s += p[(int64_t)i * 2 * H];
    }
    sh[y][threadIdx.x] = s;
    __syncthreads();
    if (y == 0 && d < H) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) s += sh[i][threadIdx.x];
        (blockIdx.y == 0 ? dw : db)[d] = s;
    }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T, int V, int NV, int G>
cudaError_t go_fwd(const NormArgs& a, cudaStream_t st) {
    if (G == 1) {
        const int rows = a.M >= 2048 ? 8 : 1;
        norm_fwd_kernel<T, V, NV, G><<<(unsigned)((a.M + rows - 1) / rows), 32 * rows, 0, st>>>(a);
    } else {
        norm_fwd_kernel<T, V, NV, G><<<(unsigned)a.M, 32 * G, 0, st>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick_fwd(const NormArgs& a, cudaStream_t st) {
    const bool vec = a.H % 8 == 0 && a.ldx % 8 == 0 && aligned16(a.x) && aligned16(a.y) &&
                     aligned16(a.w) && (!a.b || aligned16(a.b));
    const int H = a.H;
    if (vec) {
        if (H <= 256) return go_fwd<T, 8, 1, 1>(a, st);
        if (H <= 512) return go_fwd<T, 8, 2, 1>(a, st);
        if (H <= 1024) return go_fwd<T, 8, 4, 1>(a, st);
        if (H <= 1536) return go_fwd<T, 8, 6, 1>(a, st);
        if (H <= 2048) return go_fwd<T, 8, 8, 1>(a, st);
        if (H <= 2560) return go_fwd<T, 8, 10, 1>(a, st);
        if (H <= 4096) return go_fwd<T, 8, 2, 8>(a, st);
        return go_fwd<T, 8, 4, 8>(a, st);
    }
    if (H <= 1024) return go_fwd<T, 1, 4, 8>(a, st);
    if (H <= 2048) return go_fwd<T, 1, 8, 8>(a, st);
    if (H <= 4096) return go_fwd<T, 1, 16, 8>(a, st);
    return go_fwd<T, 1, 32, 8>(a, st);
}

template <typename T, int V, int NV, int R, int MAXT>
cudaError_t go_bwd(const NormBwdArgs& a, cudaStream_t st) {
    const int pieces = (a.H + V * NV - 1) / (V * NV);
    const int threads = (pieces + 31) / 32 * 32;
    norm_bwd_kernel<T, V, NV, R, MAXT><<<(unsigned)a.grid, threads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick_bwd(const NormBwdArgs& a, cudaStream_t st) {
    const bool vec = a.H % 8 == 0 && a.ldx % 8 == 0 && a.ldy % 8 == 0 && aligned16(a.x) &&
                     aligned16(a.dy) && aligned16(a.dx) && aligned16(a.w);
    const int H = a.H;
    if (vec) return H <= 4096 ? go_bwd<T, 8, 1, 2, 512>(a, st) : go_bwd<T, 8, 1, 1, 1024>(a, st);
    if (H <= 2048) return go_bwd<T, 1, 4, 2, 512>(a, st);
    if (H <= 4096) return go_bwd<T, 1, 8, 1, 512>(a, st);
    return go_bwd<T, 1, 16, 1, 512>(a, st);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
    if (a.x_type == kSbF32) return pick_fwd<float>(a, st);
    if (a.x_type == kSbBf16) return pick_fwd<__nv_bfloat16>(a, st);
    return pick_fwd<__half>(a, st);
}

int norm_bwd_grid(int64_t M, int H) {
    const int64_t want = 152 * (H <= 1024 ? 4 : 2);  // (GB300's SMs: the workspace query needs no device)
    return (int)(M < want ? (M < 1 ? 1 : M) : want);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
    cudaError_t e = a.x_type == kSbF32    ? pick_bwd<float>(a, st)
                    : a.x_type == kSbBf16 ? pick_bwd<__nv_bfloat16>(a, st)
                                          : pick_bwd<__half>(a, st);
    if (e) return e;
    norm_join_kernel<<<dim3((unsigned)((a.H + 31) / 32), a.db ? 2 : 1), dim3(32, kJoinRows), 0, st>>>(
        a.part, a.grid, a.H, a.dw, a.db);
    return cudaGetLastError();
}

}  // namespace qh
