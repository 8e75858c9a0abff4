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

#include <type_traits>

namespace qh {

namespace {

// ------------------------------------------------------------------ forward

// A thread's 8 elements of a row as they lie in memory.
template <typename T>
struct Raw {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        load8(reinterpret_cast<const T*>(u), v);
    }
};

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

// One row per G warps (G = 1: blockDim / 32 rows per block), NV pieces of 8
// elements per thread held in registers as they were loaded, so that all of a
// row's loads are in flight at once and many rows fit an SM: thread t of the row
// takes elements 8 (t + 32 G i) ...  65536 x 1536 bf16: 65 us, 6.2 TB/s (82 us
// with the row held as fp32).
template <typename T, int NV, int G>
__global__ void __launch_bounds__(G == 1 ? 256 : 32 * G) norm_fwd_kernel(const NormArgs a) {
    __shared__ float red[G];
    const int t = G == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t r = G == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (G == 1 && r >= a.M) return;  // (whole warps)
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    Raw<T> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (t + 32 * G * i) * 8;
        if (d < a.H) raw[i].load(x + d);
    }
    float mean = 0.f;
    const float inv = 1.f / (float)a.H;
    if (a.center) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((t + 32 * G * i) * 8 >= a.H) continue;
            float v[8];
            raw[i].get(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[e];
        }
        mean = row_sum<G>(sum, red) * inv;
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((t + 32 * G * i) * 8 >= a.H) continue;
        float v[8];
        raw[i].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(v[e] - mean, v[e] - mean, sq);
    }
    const float rstd = 1.f / sqrtf(row_sum<G>(sq, red) * inv + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[r] = mean;
        a.rstd[r] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int d = (t + 32 * G * i) * 8;
        if (d >= a.H) continue;
        float v[8], w[8], b[8];
        raw[i].get(v);
        load8_as(a.w, d, a.w_type, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = 0.f;
        if (a.b) load8_as(a.b, d, a.w_type, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf((v[e] - mean) * rstd, w[e], b[e]);
        store8_as(a.y, r * a.H + d, a.y_type, v);
    }
}

// ------------------------------------------------------------ single elements
//
// Rows of any width and alignment.  A row belongs to a block of NT threads, or
// (NT = 32) to a warp; thread t of the row takes elements t + NT i, i < NE, and keeps
// its columns' parameters over all the rows the block walks.  The next row is
// on its way while a row's sums are joined, held as it lies in memory: a
// conversion at its load would wait for it (20000 x 2563 bf16: forward 251 us,
// 72 with raw rows; backward 218, 87).  The issue rate bounds these (an element
// is an instruction of each kind): NT is a constant, so that a row's accesses
// are one address and immediate offsets, the type switches stand outside the
// loops over elements, and NE is 8 to 16, so that the reductions of a row are
// shared by many elements (20001 x 2563 fp32 forward: 172 us with NE = 4 and 672
// threads, 94 us with 256; 73 us, 5.6 TB/s, with four blocks to an SM).

// Totals of two sums over the block's `warps` warps, deterministic; one
// barrier, so `red` (64 floats) alternates between calls.
__device__ __forceinline__ float2 block_sum2(float c1, float c2, float* red, int warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool hi = lane & 16;  // the halves of the warp carry one sum each
    float v = (hi ? c2 : c1) + __shfl_xor_sync(0xffffffffu, hi ? c1 : c2, 16);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps > 1) {
        if ((lane & 15) == 0) red[2 * warp + (lane >> 4)] = v;
        __syncthreads();
        // lane: sum lane >> 4, warp lane & 15
        v = (lane & 15) < warps ? red[2 * (lane & 15) + (lane >> 4)] : 0.f;
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float block_sum1(float v, float* red, int warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps > 1) {
        if (lane == 0) red[warp] = v;
        __syncthreads();
        v = lane < warps ? red[lane] : 0.f;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// Calls f with a null pointer of the element type of code `type`.
template <typename F>
__device__ __forceinline__ void as_type(int type, F&& f) {
    if (type == kSbF32) f(static_cast<float*>(nullptr));
    else if (type == kSbBf16) f(static_cast<__nv_bfloat16*>(nullptr));
    else f(static_cast<__half*>(nullptr));
}

// An element as it lies in memory, and its value.
template <typename T>
__device__ __forceinline__ uint32_t raw_of(const T* p) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const uint32_t*>(p);
    else return *reinterpret_cast<const unsigned short*>(p);
}
template <typename T>
__device__ __forceinline__ float value_of(uint32_t u) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u);
    else if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)u));
    else return __uint_as_float(u << 16);
}

constexpr int kElemWarps = 8;  // rows of a block at NT = 32
constexpr int elem_block(int nt) { return nt == 32 ? 32 * kElemWarps : nt; }

// Blocks to an SM (each within 65536 registers).
constexpr int elem_fwd_blocks(int nt, int ne) {
    return nt > 256 ? 1 : ne <= 8 ? 1024 / elem_block(nt) : 48 / ne;
}
constexpr int elem_bwd_blocks(int nt) { return nt > 256 ? 1 : 512 / elem_block(nt); }

template <typename T, int NT, int NE>
__global__ void __launch_bounds__(elem_block(NT), elem_fwd_blocks(NT, NE))
    norm_fwd_elem_kernel(const NormArgs a) {
    __shared__ float red[2][64];
    constexpr int warps = NT / 32, rows = NT == 32 ? kElemWarps : 1;
    static_assert(warps <= 16, "block_sum2");
    const int t = threadIdx.x % NT, mine = threadIdx.x / NT;
    const float inv = 1.f / (float)a.H;
    const int left = a.H - t;  // element i exists: NT i < left
    const T* xp = static_cast<const T*>(a.x) + t;
    float w[NE], b[NE];
    uint32_t raw[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        w[i] = b[i] = 0.f;
        if (NT * i < left) {
            w[i] = sb_elem(a.w, t + NT * i, a.w_type);
            if (a.b) b[i] = sb_elem(a.b, t + NT * i, a.w_type);
        }
    }
    const int64_t step = (int64_t)gridDim.x * rows;
    int64_t r = (int64_t)blockIdx.x * rows + mine;
    auto fetch = [&](int64_t at) {
        if (at >= a.M) return;
        const T* p = xp + at * a.ldx;
#pragma unroll
        for (int i = 0; i < NE; ++i) raw[i] = NT * i < left ? raw_of(p + NT * i) : 0u;
    };
    fetch(r);
    int flip = 0;
    for (; r < a.M; r += step) {
        float mean = 0.f, sum = 0.f, sq = 0.f, x[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = value_of<T>(raw[i]);
        fetch(r + step);
        if (a.center) {
#pragma unroll
            for (int i = 0; i < NE; ++i) sum += x[i];
            mean = block_sum1(sum, red[flip], warps) * inv;
            flip ^= 1;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (NT * i < left) x[i] -= mean;
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) sq = fmaf(x[i], x[i], sq);
        const float rstd = 1.f / sqrtf(block_sum1(sq, red[flip], warps) * inv + a.eps);
        flip ^= 1;
        if (t == 0) {
            if (a.mean) a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
        as_type(a.y_type, [&](auto* tag) {
            using Y = std::remove_pointer_t<decltype(tag)>;
            Y* y = static_cast<Y*>(a.y) + r * a.H + t;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (NT * i < left) y[NT * i] = (Y)fmaf(x[i] * rstd, w[i], b[i]);
        });
    }
}

template <typename T, int NT, int NE>
__global__ void __launch_bounds__(elem_block(NT), elem_bwd_blocks(NT))
    norm_bwd_elem_kernel(const NormBwdArgs a) {
    __shared__ float red[2][64];
    extern __shared__ float cols[];  // NT = 32: the warps' columns at the end
    constexpr int warps = NT / 32, rows = NT == 32 ? kElemWarps : 1;
    static_assert(warps <= 16, "block_sum2");
    const int t = threadIdx.x % NT, mine = threadIdx.x / NT;
    const float inv = 1.f / (float)a.H;
    const int left = a.H - t;  // element i exists: NT i < left
    float w[NE], dw[NE], db[NE], mean = 0.f, rstd = 0.f;
    uint32_t xr[NE], gr[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        w[i] = dw[i] = db[i] = 0.f;
        if (NT * i < left) w[i] = sb_elem(a.w, t + NT * i, a.w_type);
    }
    const T* xp = static_cast<const T*>(a.x) + t;
    T* dxp = static_cast<T*>(a.dx) + t;
    auto fetch = [&](int64_t at) {
        if (at >= a.M) return;
        mean = a.mean ? a.mean[at] : 0.f;
        rstd = a.rstd[at];
        const T* p = xp + at * a.ldx;
#pragma unroll
        for (int i = 0; i < NE; ++i) xr[i] = NT * i < left ? raw_of(p + NT * i) : 0u;
        if (a.dy_type == kSbF32) {
            const float* y = static_cast<const float*>(a.dy) + at * a.ldy + t;
#pragma unroll
            for (int i = 0; i < NE; ++i) gr[i] = NT * i < left ? raw_of(y + NT * i) : 0u;
        } else {
            const __half* y = static_cast<const __half*>(a.dy) + at * a.ldy + t;  // (16 bits)
#pragma unroll
            for (int i = 0; i < NE; ++i) gr[i] = NT * i < left ? raw_of(y + NT * i) : 0u;
        }
    };
    int flip = 0;
    const int64_t step = (int64_t)gridDim.x * rows;
    int64_t r = (int64_t)blockIdx.x * rows + mine;
    fetch(r);
    for (; r < a.M; r += step) {
        float c1 = 0.f, c2 = 0.f, x[NE], g[NE];
        as_type(a.dy_type, [&](auto* tag) {
            using Y = std::remove_pointer_t<decltype(tag)>;
#pragma unroll
            for (int i = 0; i < NE; ++i) g[i] = value_of<Y>(gr[i]);
        });
#pragma unroll
        for (int i = 0; i < NE; ++i) {  // (past the row g is 0)
            const float xh = (value_of<T>(xr[i]) - mean) * rstd;
            dw[i] = fmaf(g[i], xh, dw[i]);
            db[i] += g[i];
            const float gw = g[i] * w[i];
            c1 += gw;
            c2 = fmaf(gw, xh, c2);
            x[i] = xh;
            g[i] = gw;
        }
        const float rs = rstd;
        fetch(r + step);
        const float2 sum = block_sum2(c1, c2, red[flip], warps);
        flip ^= 1;
        // rstd (g - c1 - xh c2)
        const float k1 = a.mean ? -rs * (sum.x * inv) : 0.f, k2 = -rs * (sum.y * inv);
        T* p = dxp + r * a.H;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (NT * i < left) p[NT * i] = (T)fmaf(x[i], k2, fmaf(g[i], rs, k1));
    }
    tc::grid_dep_trigger();
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.H;
    if constexpr (NT == 32) {
        // the warps' columns in order
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int d = t + 32 * i;
            if (d < a.H) {
                cols[(2 * mine) * a.H + d] = dw[i];
                cols[(2 * mine + 1) * a.H + d] = db[i];
            }
        }
        __syncthreads();
        for (int d = threadIdx.x; d < 2 * a.H; d += blockDim.x) {
            float s = 0.f;
            for (int k = 0; k < rows; ++k) s += cols[k * 2 * a.H + d];
            part[d] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int d = t + NT * i;
            if (d < a.H) {
                part[d] = dw[i];
                part[a.H + d] = db[i];
            }
        }
    }
}

// ------------------------------------------------------ backward, 16-byte path
//
// Thread t owns 8 columns of every row of its block, so a row's x and dy go
// through a ring of kStages x R rows in shared memory of which each thread fills
// (cp.async) and reads only its own slots: no barrier guards the ring, and the
// loads of the next kStages - 1 steps are in flight while a step's sums go
// through the block's one barrier per step.  (With the loads in registers, a
// step at a time, the kernel ran at 1.6 TB/s: 381 us at 65536 x 1536 bf16, 90 us
// with the ring, 6.7 TB/s.)  Two fp32 lanes per instruction: what bounds it beside
// the bytes is the issue rate.
//
// The columns come as pieces of PW: 8 (16 bytes of a 2-byte type), or with a
// 4-byte operand twice 4, blockDim x 4 apart, so that a warp's copies fill whole
// sectors (16-byte pieces 32 bytes apart fetch every sector twice: 255 us at
// 20000 x 4096 fp32, 149 us, 6.6 TB/s, without).
constexpr int kStages = 3;

// PW consecutive elements as pairs.
template <typename T, int PW>
__device__ __forceinline__ void get_pairs(const unsigned char* p, float2* v) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        v[0] = make_float2(a.x, a.y);
        v[1] = make_float2(a.z, a.w);
    } else {
        uint32_t u[PW / 2];
        if constexpr (PW == 8) {
            const uint4 q = *reinterpret_cast<const uint4*>(p);
            u[0] = q.x; u[1] = q.y; u[2] = q.z; u[3] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            u[0] = q.x; u[1] = q.y;
        }
#pragma unroll
        for (int i = 0; i < PW / 2; ++i) {
            if constexpr (std::is_same<T, __half>::value)
                v[i] = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            else
                v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
        }
    }
}
template <typename T, int PW>
__device__ __forceinline__ void put_pairs(T* p, const float2* v) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    } else {
        uint32_t u[PW / 2];
#pragma unroll
        for (int i = 0; i < PW / 2; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(v[i].x, v[i].y);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        if constexpr (PW == 8) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    }
}

// Totals of N = 2 R sums over the block (at most 64 / N warps); one barrier, so
// `red` alternates between calls.  Each level halves the values with the lanes
// where it can: N = 4: 6 shuffles down, 7 up, instead of 5 per value and level.
template <int N>
__device__ __forceinline__ void block_sums(float (&s)[N], float* red, int warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float v;
    if constexpr (N == 4) {
        const bool h16 = lane & 16, h8 = lane & 8;
        const float p = (h16 ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, h16 ? s[0] : s[2], 16);
        const float q = (h16 ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, h16 ? s[1] : s[3], 16);
        v = (h8 ? q : p) + __shfl_xor_sync(0xffffffffu, h8 ? p : q, 8);
    } else {
        const bool h16 = lane & 16;
        v = (h16 ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, h16 ? s[0] : s[1], 16);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
    }
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    // this lane's value: 2 (lane >> 4) + (lane >> 3 & 1) of 4, lane >> 4 of 2
    if (N == 4 ? (lane & 7) == 0 : (lane & 15) == 0) red[warp * N + (N == 4 ? lane >> 3 : lane >> 4)] = v;
    __syncthreads();
    const int n = warps * N;  // <= 64; value of entry i: i % N
    v = lane < n ? red[lane] : 0.f;
    if (lane + 32 < n) v += red[lane + 32];
#pragma unroll
    for (int o = 16; o >= N; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = __shfl_sync(0xffffffffu, v, k);
}

template <typename T, typename DT, int R, bool CENTER, int REGS>
__global__ void __maxnreg__(REGS) norm_bwd_ring_kernel(const NormBwdArgs a) {
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float red[2][64];
    constexpr int PW = sizeof(T) == 4 || sizeof(DT) == 4 ? 4 : 8, NP = 8 / PW;
    constexpr int BX = PW * sizeof(T), BD = PW * sizeof(DT);  // bytes of a piece
    const int t = threadIdx.x, nt = blockDim.x, warps = nt >> 5;
    const int row_bytes = NP * (BX + BD) * nt, stage_bytes = R * row_bytes;
    // within a row's slots: the x pieces (NP planes), then the dy pieces
    const int off_d = NP * BX * nt;
    const float inv = 1.f / (float)a.H;
    bool on[NP];
    float2 w[4], dw[4], db[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = dw[e] = db[e] = both(0.f);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int d = PW * (t + nt * p);
        on[p] = d < a.H;
        if (on[p]) {
#pragma unroll
            for (int e = 0; e < PW / 2; ++e)
                w[p * PW / 2 + e] = make_float2(sb_elem(a.w, d + 2 * e, a.w_type),
                                                sb_elem(a.w, d + 2 * e + 1, a.w_type));
        }
    }
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t r0 = (int64_t)blockIdx.x * R;
    const uint32_t ring_s = tc::smem_u32(ring);
    // the next rows to fetch
    int64_t rf = r0;
    const T* xf = static_cast<const T*>(a.x) + r0 * a.ldx + PW * t;
    const DT* gf = static_cast<const DT*>(a.dy) + r0 * a.ldy + PW * t;
    auto fetch = [&](int stage) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const uint32_t dst = ring_s + stage * stage_bytes + k * row_bytes;
            if (rf + k < a.M) {
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    if (on[p]) {
                        cp_async<BX>(dst + BX * (t + nt * p), xf + k * a.ldx + PW * nt * p);
                        cp_async<BD>(dst + off_d + BD * (t + nt * p), gf + k * a.ldy + PW * nt * p);
                    }
            }
        }
        cp_async_commit();  // (an empty group keeps the count)
        rf += step;
        xf += step * a.ldx;
        gf += step * a.ldy;
    };
    float mean[R], rstd[R];  // this step's, loaded one step ahead
    auto stats = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const bool live = r + k < a.M;
            mean[k] = CENTER && live ? a.mean[r + k] : 0.f;
            rstd[k] = live ? a.rstd[r + k] : 0.f;
        }
    };
    stats(r0);
    for (int s = 0; s < kStages - 1; ++s) fetch(s);
    int stage = 0, flip = 0;
    T* dx = static_cast<T*>(a.dx) + r0 * a.H + PW * t;
    for (; r0 < a.M; r0 += step, dx += step * a.H) {
        // into the slots whose values the step before took into registers
        fetch(stage == 0 ? kStages - 1 : stage - 1);
        cp_async_wait<kStages - 1>();
        float2 x[R][4], g[R][4];
        float s[2 * R], rs[R];
        const unsigned char* src = ring + stage * stage_bytes;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            rs[k] = rstd[k];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                float2 *xq = x[k] + p * PW / 2, *gq = g[k] + p * PW / 2;
                if (on[p] && r0 + k < a.M) {
                    get_pairs<T, PW>(src + k * row_bytes + BX * (t + nt * p), xq);
                    get_pairs<DT, PW>(src + k * row_bytes + off_d + BD * (t + nt * p), gq);
                } else {
#pragma unroll
                    for (int e = 0; e < PW / 2; ++e) xq[e] = gq[e] = both(0.f);
                }
            }
            float2 c1 = both(0.f), c2 = both(0.f);
            const float2 nm = both(-mean[k]), rr = both(rstd[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // (where there is no column or row, dy is 0)
                const float2 xh = mul2(CENTER ? add2(x[k][e], nm) : x[k][e], rr);
                const float2 dy = g[k][e];
                dw[e] = fma2(dy, xh, dw[e]);
                db[e] = add2(db[e], dy);
                const float2 gw = mul2(dy, w[e]);
                if (CENTER) c1 = add2(c1, gw);
                c2 = fma2(gw, xh, c2);
                x[k][e] = xh;
                g[k][e] = gw;
            }
            s[2 * k] = c1.x + c1.y;
            s[2 * k + 1] = c2.x + c2.y;
        }
        stats(r0 + step);
        block_sums(s, red[flip], warps);
        flip ^= 1;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (r0 + k >= a.M) continue;
            // rs (g - c1 - xh c2)
            const float2 p = both(rs[k]), q = both(-rs[k] * (s[2 * k + 1] * inv));
            const float2 c = both(CENTER ? -rs[k] * (s[2 * k] * inv) : 0.f);
            float2 o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = fma2(x[k][e], q, CENTER ? fma2(g[k][e], p, c) : mul2(g[k][e], p));
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (on[i]) put_pairs<T, PW>(dx + k * a.H + PW * nt * i, o + i * PW / 2);
        }
        if (++stage == kStages) stage = 0;
    }
    cp_async_wait<0>();
    tc::grid_dep_trigger();
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.H + PW * t;
#pragma unroll
    for (int i = 0; i < NP; ++i)
        if (on[i]) {
            put_pairs<float, 4>(part + PW * nt * i, dw + i * PW / 2);
            put_pairs<float, 4>(part + a.H + PW * nt * i, db + i * PW / 2);
            if constexpr (PW == 8) {
                put_pairs<float, 4>(part + 4, dw + 2);
                put_pairs<float, 4>(part + a.H + 4, db + 2);
            }
        }
}

// 32 columns per block of 32 x 16: partial rows y, y + 16, ... per thread, then
// the 16 sums in order.  blockIdx.y: dw, db.
constexpr int kJoinRows = 16;
__global__ void __launch_bounds__(32 * kJoinRows) norm_join_kernel(const float* part,
                                                                   int n, int H,
                                                                   float* __restrict__ dw,
                                                                   float* __restrict__ db) {
    __shared__ float sh[kJoinRows][33];
    tc::grid_dep_wait();  // (launched as the dependent of the rows' kernel)
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

// Threads and elements per thread of a row of single elements.
template <typename F>
cudaError_t elem_shape(int H, F&& f) {
#define QH_SHAPE(nt, ne) f(std::integral_constant<int, nt>{}, std::integral_constant<int, ne>{})
    if (H <= 256) return QH_SHAPE(32, 8);
    if (H <= 512) return QH_SHAPE(64, 8);
    if (H <= 1024) return QH_SHAPE(128, 8);
    if (H <= 2048) return QH_SHAPE(256, 8);
    if (H <= 3072) return QH_SHAPE(256, 12);
    if (H <= 4096) return QH_SHAPE(256, 16);
    if (H <= 6144) return QH_SHAPE(512, 12);
    return QH_SHAPE(512, 16);
#undef QH_SHAPE
}

template <typename T, int NV, int G>
cudaError_t go_fwd(const NormArgs& a, cudaStream_t st) {
    if (G == 1) {
        const int rows = a.M >= 2048 ? 8 : 1;  // (few rows: one warp per block, spread over the SMs)
        norm_fwd_kernel<T, NV, G><<<(unsigned)((a.M + rows - 1) / rows), 32 * rows, 0, st>>>(a);
    } else {
        norm_fwd_kernel<T, NV, G><<<(unsigned)a.M, 32 * G, 0, st>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick_fwd(const NormArgs& a, cudaStream_t st) {
    const bool vec = a.H % 8 == 0 && a.ldx % 8 == 0 && aligned16(a.x) && aligned16(a.y) &&
                     aligned16(a.w) && (!a.b || aligned16(a.b));
    const int H = a.H;
    if (vec) {
        if (H <= 256) return go_fwd<T, 1, 1>(a, st);
        if (H <= 512) return go_fwd<T, 2, 1>(a, st);
        if (H <= 1024) return go_fwd<T, 4, 1>(a, st);
        if (H <= 1536) return go_fwd<T, 6, 1>(a, st);
        if (H <= 2048) return go_fwd<T, 8, 1>(a, st);
        if (H <= 2560) return go_fwd<T, 10, 1>(a, st);
        if (H <= 4096) return go_fwd<T, 2, 8>(a, st);
        return go_fwd<T, 4, 8>(a, st);
    }
    return elem_shape(H, [&](auto nt, auto ne) {
        constexpr int NT = decltype(nt)::value, NE = decltype(ne)::value, B = elem_block(NT);
        const int64_t blocks = NT == 32 ? (a.M + kElemWarps - 1) / kElemWarps : a.M;
        const int64_t most = device_sms() * (int64_t)elem_fwd_blocks(NT, NE);
        norm_fwd_elem_kernel<T, NT, NE><<<(unsigned)(blocks < most ? blocks : most), B, 0, st>>>(a);
        return cudaGetLastError();
    });
}

// The backward's rows are dealt to the blocks in equal shares, so the blocks are as
// many as the device's SMs hold at once (at most a.grid, which the partial rows are
// planned for).  `a.grid` becomes that number.
void fit_grid(NormBwdArgs& a, int per_sm) {
    const int n = device_sms() * (per_sm < 1 ? 1 : per_sm);
    if (a.grid > n) a.grid = n;
}

template <typename T, typename DT, int R, int REGS>
cudaError_t go_ring(NormBwdArgs& a, cudaStream_t st) {
    const int threads = (a.H / 8 + 31) / 32 * 32;
    const int smem = kStages * R * threads * 8 * (int)(sizeof(T) + sizeof(DT));
    const int by_regs = 65536 / (REGS * threads), by_smem = 227 * 1024 / (smem + 1024 + 512);
    fit_grid(a, by_regs < by_smem ? by_regs : by_smem);
    auto go = [&](auto center) {
        auto* fn = norm_bwd_ring_kernel<T, DT, R, decltype(center)::value, REGS>;
        if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), smem)) return e;
        fn<<<(unsigned)a.grid, threads, smem, st>>>(a);
        return cudaGetLastError();
    };
    return a.mean ? go(std::true_type{}) : go(std::false_type{});
}

// Two rows a step while their threads fit 512 (a step's barrier is shared by
// both), one above.
template <typename T, typename DT>
cudaError_t pick_ring(NormBwdArgs& a, cudaStream_t st) {
    return a.H <= 4096 ? go_ring<T, DT, 2, 80>(a, st) : go_ring<T, DT, 1, 64>(a, st);
}

template <typename T>
cudaError_t pick_bwd(NormBwdArgs& a, cudaStream_t st) {
    const bool vec = a.H % 8 == 0 && a.ldx % 8 == 0 && a.ldy % 8 == 0 && aligned16(a.x) &&
                     aligned16(a.dy) && aligned16(a.dx);
    if (vec)
        return a.dy_type == kSbF32    ? pick_ring<T, float>(a, st)
               : a.dy_type == kSbBf16 ? pick_ring<T, __nv_bfloat16>(a, st)
                                      : pick_ring<T, __half>(a, st);
    return elem_shape(a.H, [&](auto nt, auto ne) {
        constexpr int NT = decltype(nt)::value, NE = decltype(ne)::value;
        const int smem = NT == 32 ? 2 * kElemWarps * a.H * (int)sizeof(float) : 0;
        fit_grid(a, elem_bwd_blocks(NT));
        norm_bwd_elem_kernel<T, NT, NE><<<(unsigned)a.grid, elem_block(NT), smem, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
    if (a.x_type == kSbF32) return pick_fwd<float>(a, st);
    if (a.x_type == kSbBf16) return pick_fwd<__nv_bfloat16>(a, st);
    return pick_fwd<__half>(a, st);
}

int norm_bwd_grid(int64_t M, int H) {
    // The most blocks the partial rows are planned for: as many as 80 registers a
    // thread leave (H / 8 threads), at most 8 an SM -- 16 for narrow rows -- since
    // each adds a partial row.  (The workspace query needs no device.)
    const int threads = H < 256 ? 32 : (H / 8 + 31) / 32 * 32;
    const int most = H <= 512 ? 16 : 8;
    int per_sm = 65536 / (80 * threads);
    per_sm = per_sm < 1 ? 1 : per_sm > most ? most : per_sm;
    constexpr int64_t kPlannedSms = 152;  // (a GB300's; a larger device leaves some idle)
    const int64_t want = kPlannedSms * per_sm;
    return (int)(M < want ? (M < 1 ? 1 : M) : want);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& args, cudaStream_t st) {
    NormBwdArgs a = args;
    cudaError_t e = a.x_type == kSbF32    ? pick_bwd<float>(a, st)
                    : a.x_type == kSbBf16 ? pick_bwd<__nv_bfloat16>(a, st)
                                          : pick_bwd<__half>(a, st);
    if (e) return e;
    const float* part = a.part;
    int n = a.grid, H = a.H;
    float *dw = a.dw, *db = a.db;
    void* ptrs[] = {&part, &n, &H, &dw, &db};
    return launch_dependent(reinterpret_cast<const void*>(norm_join_kernel),
                            dim3((unsigned)((a.H + 31) / 32), a.db ? 2 : 1), dim3(32, kJoinRows), 0, st,
                            ptrs);
}

}  // namespace qh
