// qh_few.cu -- the contraction dh[m, :] = sum_v c[m, v] w[v, :] for up to 16 rows.
//
// The tensor-core contraction (qh_tc_dh.cu) takes 128 token rows a tile, so its
// cost does not fall below theirs (200 us at 262144 x 2560 whatever the rows).
// For few rows the packed table's bytes are the floor (56 us there), and next to
// it the issue rate of unpacking: here the weights are unpacked in registers,
// straight into mma.sync operands.
//
// mma.m16n8k16: M = hidden columns, K = vocab rows, N = tokens (one tile of 8, or
// two).  A warp owns 128 columns; lane (g, t) = (lane / 4, lane % 4).  The vocab
// rows of a block of 32 are dealt so that lane t holds rows 8 t .. 8 t + 7, four to
// each of the block's two steps: its coefficients are 16 contiguous bytes per
// token, and its codes of a row (columns 16 g .. 16 g + 15) one read of 8 (4 bits)
// or 16 bytes (8 bits).  Column tile i of the warp is codes i and i + 8 of each
// lane g, so two rows' words give the A operand's pairs by byte permutation: (row 0
// code i, row 1 code i).  w = fma(q, s, b) in fp16, one rounding, as in the
// tensor-core kernels.
//
// Each warp copies its codes, scales and coefficients through a ring of its own in
// shared memory (cp.async): no block barrier, and no registers for loads in flight.
// With them in registers (a block of 64 rows ahead) two CTAs held an SM where now
// four do, and the kernel took 104 us at up to 8 rows and 135 at up to 16 (262144 x
// 2560, 4 bits); it takes 74 and 93 (61 at 13 rows of 131072 x 2560, 8 bits: 80).
// Pointers that advance by a block, against a product per row, are 8 us of that.
// The issue of the unpacking (58 % of the slots) and mma.sync (20 us a token tile,
// the most frequent stall) bound it; DRAM stands at 53 %.
// With the tokens as M, 16 whatever their number, up to 16 rows took 148 us; 64
// columns a warp, for more warps, 160 and 197 (loads of 4 bytes).
//
// Each warp keeps its sums in registers over the CTA's vocab range and writes them
// once; the ranges are added in order by a second launch.
#include "qh_dequant.cuh"
#include "qh_few.cuh"
#include "qh_ops.cuh"
#include "qh_tc.cuh"

namespace qh {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kColsWarp = 128, kColsCta = kColsWarp * kWarps;
constexpr int kBlockRows = 32, kLaneRows = kBlockRows / 4;

// One stage of a warp's ring: codes (8 rows and 32 bytes of pad at a time: the
// lanes' reads, 8 rows apart, fall on distinct banks), coefficients [token][row],
// scales and biases [row][group of 2].
template <int BITS, int NT>
struct Stage {
    static constexpr int kRowBytes = kColsWarp * BITS / 8;
    static constexpr int kPitch = kLaneRows * kRowBytes + 32;
    static constexpr int kCoeff = 4 * kPitch, kScale = kCoeff + 8 * NT * kBlockRows * 2;
    static constexpr int kBytes = kScale + 2 * 4 * kBlockRows;
    static constexpr int kStages = BITS == 4 ? 3 : 2;
    static constexpr int kCta = kWarps * kStages * kBytes;
};

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The codes of one row in this lane's 16 columns.
template <int BITS>
struct Codes {
    uint32_t w[BITS / 2];
    __device__ __forceinline__ void load(const uint32_t* p) {
        if constexpr (BITS == 4) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x; w[1] = x.y;
        } else {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        }
    }
};

// Codes 8 half + 4 quad .. + 3 of rows a and b as fp16 pairs.
template <int BITS>
__device__ __forceinline__ void pairs4(const Codes<BITS>& a, const Codes<BITS>& b, int half, int quad,
                                       uint32_t s2, uint32_t b2, uint32_t (&p)[4]) {
    if constexpr (BITS == 4) {
        deq4_word(__byte_perm(a.w[half], b.w[half], quad ? 0x7632 : 0x5410), s2, b2, p);
    } else {
        const uint32_t x = a.w[2 * half + quad], y = b.w[2 * half + quad];
        const uint32_t lo = __byte_perm(x, y, 0x5140), hi = __byte_perm(x, y, 0x7362);
        p[0] = deq8(lo, 0x4140u, s2, b2);
        p[1] = deq8(lo, 0x4342u, s2, b2);
        p[2] = deq8(hi, 0x4140u, s2, b2);
        p[3] = deq8(hi, 0x4342u, s2, b2);
    }
}

// CTAs to an SM, by the registers of the sums.
constexpr int ctas_per_sm(int bits, int nt) { return bits == 4 && nt == 1 ? 5 : 4; }

template <int BITS, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(BITS, NT)) few_dh_kernel(
    const uint32_t* __restrict__ wq, const __half* __restrict__ scales, const __half* __restrict__ biases,
    int64_t V, int H, const __half* coeff, int64_t ldc, int n_rows, float* __restrict__ part,
    int S) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    using St = Stage<BITS, NT>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int col0 = blockIdx.x * kColsCta + warp * kColsWarp;  // of the warp
    if (col0 >= H) return;                                      // (H: whole warps' columns)
    unsigned char* ring = smem + warp * St::kStages * St::kBytes;
    const int G = H / 64;
    const int64_t nb = (V + kBlockRows - 1) / kBlockRows;
    const int sp = blockIdx.y;
    const int64_t b0 = nb * sp / S, b1 = nb * (sp + 1) / S;
    constexpr int kChunks = St::kRowBytes / 16;                // 16-byte copies of a row,
    constexpr int kCopies = kBlockRows * kChunks / 32;         // of a lane, of rows kStep apart
    constexpr int kStep = 32 / kChunks;
    const int r0 = lane / kChunks, c0 = lane % kChunks;
    const int64_t wrow = (int64_t)H * BITS / 8;  // bytes
    const unsigned char* wbase = reinterpret_cast<const unsigned char*>(wq) + col0 * BITS / 8 + 16 * c0;
    const uint32_t ring_w = tc::smem_u32(ring) + r0 / kLaneRows * St::kPitch + r0 % kLaneRows * St::kRowBytes + 16 * c0;
    const uint32_t ring_c = tc::smem_u32(ring) + St::kCoeff + 64 * g + 16 * t;
    const uint32_t ring_s = tc::smem_u32(ring) + St::kScale + 4 * lane;
    // sources of the next block
    const unsigned char* wp = wbase + (b0 * kBlockRows + r0) * wrow;
    const __half* cp = coeff + (int64_t)(g < n_rows ? g : 0) * ldc + b0 * kBlockRows + 8 * t;
    const int64_t c8 = g + 8 < n_rows ? 8 * ldc : 0;  // to the second tile's token
    const int cn[2] = {g < n_rows ? 16 : 0, g + 8 < n_rows ? 16 : 0};
    int64_t so = (b0 * kBlockRows + lane) * G + col0 / 64;
    // scale of the lane's group in both halves' rows: bytes 0-1 or 2-3 of each word
    const uint32_t sel = g >> 2 ? 0x7632u : 0x5410u;

    float acc[8][NT][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;

    // Rows past V copy row V - 1: their coefficients are zero.
    auto issue = [&](int64_t blk, int slot) {
        if (blk < b1) {
            const uint32_t at = slot * St::kBytes;
            const int64_t v0 = blk * kBlockRows;
            if (v0 + kBlockRows <= V) {
#pragma unroll
                for (int k = 0; k < kCopies; ++k) {
                    const int r = k * kStep;
                    cp_async<16>(ring_w + at + r / kLaneRows * St::kPitch + r % kLaneRows * St::kRowBytes,
                                 wp + r * wrow);
                }
                cp_async<4>(ring_s + at, scales + so);
                cp_async<4>(ring_s + at + 4 * kBlockRows, biases + so);
            } else {
                const int64_t last = V - 1;
#pragma unroll
                for (int k = 0; k < kCopies; ++k) {
                    const int r = k * kStep;
                    const int64_t v = v0 + r0 + r < last ? v0 + r0 + r : last;
                    cp_async<16>(ring_w + at + r / kLaneRows * St::kPitch + r % kLaneRows * St::kRowBytes,
                                 wbase + v * wrow);
                }
                const int64_t o = (v0 + lane < last ? v0 + lane : last) * G + col0 / 64;
                cp_async<4>(ring_s + at, scales + o);
                cp_async<4>(ring_s + at + 4 * kBlockRows, biases + o);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) cp_async<16>(ring_c + at + 512 * n, cp + n * c8, cn[n]);
            wp += kBlockRows * wrow;
            cp += kBlockRows;
            so += kBlockRows * G;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < St::kStages - 1; ++s) issue(b0 + s, s);
    int slot = 0;
    for (int64_t blk = b0; blk < b1; ++blk) {
        cp_async_wait<St::kStages - 2>();
        __syncwarp();  // the block is in for every lane; every lane has read the one before
        issue(blk + St::kStages - 1, slot == 0 ? St::kStages - 1 : slot - 1);
        const unsigned char* src = ring + slot * St::kBytes;
        uint32_t cv[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + St::kCoeff + 64 * (g + 8 * n) + 16 * t);
            cv[n][0] = x.x; cv[n][1] = x.y; cv[n][2] = x.z; cv[n][3] = x.w;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const unsigned char* sp4 = src + St::kScale + 4 * (kLaneRows * t + 4 * s);
            const uint4 su = *reinterpret_cast<const uint4*>(sp4);
            const uint4 bu = *reinterpret_cast<const uint4*>(sp4 + 4 * kBlockRows);
            const uint32_t s01 = __byte_perm(su.x, su.y, sel), s23 = __byte_perm(su.z, su.w, sel);
            const uint32_t b01 = __byte_perm(bu.x, bu.y, sel), b23 = __byte_perm(bu.z, bu.w, sel);
            Codes<BITS> w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e].load(reinterpret_cast<const uint32_t*>(src + t * St::kPitch + (4 * s + e) * St::kRowBytes) +
                          g * (BITS / 2));
#pragma unroll
            for (int quad = 0; quad < 2; ++quad) {
                uint32_t p[2][4], q[2][4];  // rows (0, 1) and (2, 3), codes of either half
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    pairs4<BITS>(w[0], w[1], half, quad, s01, b01, p[half]);
                    pairs4<BITS>(w[2], w[3], half, quad, s23, b23, q[half]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a[4] = {p[0][i], p[1][i], q[0][i], q[1][i]};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma(acc[4 * quad + i][n], a, cv[n][2 * s], cv[n][2 * s + 1]);
                }
            }
        }
        if (++slot == St::kStages) slot = 0;
    }
    // Tile i, lane (g, t): columns 16 g + i and 16 g + i + 8, tokens 2 t and 2 t + 1.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = 8 * n + 2 * t + e;
            if (tok >= n_rows) continue;
            float* dst = part + ((int64_t)sp * kFewRows + tok) * H + col0 + 16 * g;
#pragma unroll
            for (int hi = 0; hi < 2; ++hi)
#pragma unroll
                for (int i = 0; i < 8; i += 4)
                    *reinterpret_cast<float4*>(dst + 8 * hi + i) =
                        make_float4(acc[i][n][2 * hi + e], acc[i + 1][n][2 * hi + e],
                                    acc[i + 2][n][2 * hi + e], acc[i + 3][n][2 * hi + e]);
        }
}

// dh[r, :] = (-geff[r] 2^-14) * sum of the ranges' partials, in order, in bf16:
// block (column block of 128, row); 16 groups of 16 threads take a contiguous
// share of the ranges each.
constexpr int kJoinGroups = 16;
__global__ void __launch_bounds__(16 * kJoinGroups) few_join_kernel(
    const float* part, int S, int H, const int* __restrict__ pos,
    const float* geff, const int* err, __nv_bfloat16* __restrict__ dh) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    __shared__ float sh[kJoinGroups][16][8];
    const int64_t r = blockIdx.y;
    const int i = pos[r];
    const int u = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int d = blockIdx.x * 128 + 8 * u;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    if (i >= 0) {
        const int s0 = S * grp / kJoinGroups, s1 = S * (grp + 1) / kJoinGroups;
#pragma unroll 4
        for (int s = s0; s < s1; ++s) {
            float x[8];
            load8_wide(part + ((int64_t)s * kFewRows + i) * H + d, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += x[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sh[grp][u][e] = acc[e];
    __syncthreads();
    if (grp != 0) return;
    for (int k = 1; k < kJoinGroups; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += sh[k][u][e];
    const float scale = i < 0 ? 0.f : *err != 0 ? __int_as_float(0x7fc00000) : -geff[r] * (1.f / 16384.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = i < 0 ? 0.f : acc[e] * scale;
    store8(dh + r * (int64_t)H + d, acc);
}

}  // namespace

int few_splits(int64_t M, int64_t V, int H, int bits) {
    const int gx = (H + kColsCta - 1) / kColsCta;
    const int64_t nb = (V + kBlockRows - 1) / kBlockRows;
    const int64_t want = ctas_per_sm(bits, M <= 8 ? 1 : 2) * (int64_t)device_sms() / gx;  // one wave
    return (int)(nb < want ? nb : want < 1 ? 1 : want);
}

cudaError_t launch_few_dh(const uint32_t* wq, const __half* scales, const __half* biases, int64_t V, int H,
                          int bits, const __half* coeff, int64_t ldc, int64_t M, const int* pos,
                          const float* geff, const int* err, float* part, void* dh, cudaStream_t st) {
    const int S = few_splits(M, V, H, bits);
    const dim3 grid((unsigned)((H + kColsCta - 1) / kColsCta), (unsigned)S);
    auto* fn = bits == 4 ? (M <= 8 ? few_dh_kernel<4, 1> : few_dh_kernel<4, 2>)
                         : (M <= 8 ? few_dh_kernel<8, 1> : few_dh_kernel<8, 2>);
    const int smem = bits == 4 ? (M <= 8 ? Stage<4, 1>::kCta : Stage<4, 2>::kCta)
                               : (M <= 8 ? Stage<8, 1>::kCta : Stage<8, 2>::kCta);
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), smem)) return e;
    if (cudaError_t e = launch_after_smem(fn, grid, dim3(kThreads), smem, st, wq, scales, biases, V, H, coeff, ldc, (int)M,
                                     part, S))
        return e;
    return launch_after(few_join_kernel, dim3((unsigned)(H / 128), (unsigned)M), dim3(16 * kJoinGroups), st,
                        part, S, H, pos, geff, err, static_cast<__nv_bfloat16*>(dh));
}

}  // namespace qh
