// qh_distill.cu -- the distillation loss of the quantized head against a
// teacher's top logits: everything around the two tensor-core kernels.
//
// Per active row, over the row's valid entries k (ids[k] in [0, V)) and the
// whole vocabulary v, at temperature T:
//     p_k  = softmax_k(t_k / T)          the teacher
//     z_v  = softcap(h . w_v)            the student
//     lse  = log sum_v exp(z_v / T),  q_v = exp(z_v / T - lse)
//     loss = sum_k p_k (log p_k - z_k / T + lse)
//     dh   = (dloss / T) sum_v (q_v - p_v) sech2_v w_v
//
// The [M, V] logits come from the same fp16-operand tensor-core kernels as the
// target-per-row loss (qh_tc_fwd.cu, qh_tc_dh.cu).  An fp16-rounded operand
// moves a logit by about 3e-4, which is no matter in the tail of the softmax
// but shows in a loss of a few tenths where the teacher's tokens hold most of
// the mass, and cancels badly in q_k - p_k.  So the teacher's K logits are
// computed exactly (fp32, weights widened) once, in the forward, and kept:
//   * the softmax epilogue leaves the teacher's columns out of its sum and the
//     finalize adds their exact terms and replaces those of the largest other
//     columns (a thousandth of the sum or more, up to kOthers), whose exact logits
//     are kept as well; it finds them by the maxima that the epilogue writes for
//     every 32 columns;
//   * the backward's coefficient block gets (q_k - p_k) sech2_k, formed in
//     fp32 from the exact logits, in the K teacher's and the kept other columns
//     of each row before the contraction with W, so the one-hot part of the
//     gradient needs no gather of head rows of its own.  (The other
//     columns belong to it: with their exact terms in lse but the tensor-core
//     logits in q, a row with mass there came out 1e-2 off, 1.7e-3 -- bf16's
//     rounding -- with both.)
//
// kept [M, ld] holds, per row, the K exact capped logits, the others' and their
// vocab rows plus one (as integer bits, 0: none), and while they fit 4 GiB the
// row's V logits, with the coefficients themselves, times kMark, in the teacher's
// and the others' columns: the backward then forms its coefficients from them in
// one pass instead of running the logit kernel again and a pass over the tokens.
// A row without others' columns marks in the first's logit what its gradient is:
// -inf, zero (nothing to learn from), +inf, NaN (a bad teacher).  Up to kFewM
// rows the weight-streaming kernel writes them, whose cost follows the rows (the
// tensor-core kernel's does not: 227 us from 1 to 128 rows of the 262144 x 2560
// head), and a softmax pass of its own reads them.
#include "qh_dequant.cuh"
#include "qh_distill.cuh"
#include "qh_ops.cuh"
#include "qh_tc.cuh"

#include <type_traits>

namespace qh {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kDotsPerWarp = 4;  // teacher logits of one row that a warp forms together

// A kept coefficient's factor (exact), and the size from which on a kept value is
// one: coefficients below kMarked / kMark = 2^-41 would be zeros in fp16 and are
// kept as -inf, and no logit comes near 2^85.
constexpr float kMark = 0x1p126f, kMarked = 0x1p85f;

__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }

__device__ __forceinline__ void prefetch_l1(const void* p) {
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p) : "memory");
}

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v = fmaxf(v, red[w]);
    __syncthreads();
    return v;
}

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += red[w];
    __syncthreads();
    return v;
}

// This thread's part of the exact fp32 logits of N vocab rows v[] (-1: none,
// its part means nothing) under one row of h: the 8-element units u0, u0 + stride,
// ..., U of them at a time with all their loads issued together.  w =
// fma(scale, code, bias) in fp32, two lanes per instruction; a code becomes fp32 as
// a byte in the mantissa of 2^23.  The issue rate bounds it, so the rows'
// addresses are formed once and the scales' type is a parameter.
template <int BITS, int SBT, int N, int U>
__device__ __forceinline__ void exact_parts_of(const __nv_bfloat16* __restrict__ hrow,
                                               const uint32_t* __restrict__ wq, const SbView& sb,
                                               const int (&v)[N], int H, int u0, int stride,
                                               float (&dot)[N]) {
    using ST = std::conditional_t<SBT == kSbF32, float, unsigned short>;
    using WT = std::conditional_t<BITS == 4, uint32_t, uint2>;
    const int units = H / 8;
    float2 acc[N];
    const WT* wr[N];
    const ST *sr[N], *br[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t row = v[i] < 0 ? 0 : v[i];
        acc[i] = both(0.f);
        wr[i] = reinterpret_cast<const WT*>(wq + row * (H * BITS / 32));
        sr[i] = static_cast<const ST*>(sb.s) + row * (H / 64);
        br[i] = static_cast<const ST*>(sb.b) + row * (H / 64);
    }
    auto widen = [](ST x) {
        if constexpr (SBT == kSbF32) return x;
        else if constexpr (SBT == kSbBf16) return __uint_as_float((uint32_t)x << 16);
        else return __half2float(__ushort_as_half(x));
    };
    for (int ub = u0; ub < units; ub += U * stride) {
        uint4 h[U];
        WT w[U][N];
        ST s[U][N], b[U][N];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int u = ub + k * stride;
            if (u >= units) continue;
            h[k] = *reinterpret_cast<const uint4*>(hrow + 8 * u);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                w[k][i] = wr[i][u];
                s[k][i] = sr[i][u / 8];
                b[k][i] = br[i][u / 8];
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (ub + k * stride >= units) continue;
            const uint32_t hw[4] = {h[k].x, h[k].y, h[k].z, h[k].w};
            float2 hp[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                hp[e] = make_float2(__uint_as_float(hw[e] << 16), __uint_as_float(hw[e] & 0xffff0000u));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 s2 = both(widen(s[k][i])), b2 = both(widen(b[k][i]));
                // 4 bits: elements 2 e in the bytes of lo, 2 e + 1 in those of hi
                uint32_t lo, hi;
                if constexpr (BITS == 4) {
                    lo = w[k][i] & 0x0f0f0f0fu;
                    hi = w[k][i] >> 4 & 0x0f0f0f0fu;
                } else {
                    lo = w[k][i].x;
                    hi = w[k][i].y;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 q;
                    if constexpr (BITS == 4) {
                        q.x = __uint_as_float(__byte_perm(lo, 0x4B000000u, 0x7650u | e));
                        q.y = __uint_as_float(__byte_perm(hi, 0x4B000000u, 0x7650u | e));
                    } else {
                        const uint32_t x = e < 2 ? lo : hi;
                        q.x = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7650u | (2 * (e & 1))));
                        q.y = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7650u | (2 * (e & 1) + 1)));
                    }
                    q = add2(q, both(-8388608.f));
                    acc[i] = fma2(hp[e], fma2(s2, q, b2), acc[i]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) dot[i] = acc[i].x + acc[i].y;
}

template <int BITS, int N, int U>
__device__ __forceinline__ void exact_parts(const __nv_bfloat16* __restrict__ hrow,
                                            const uint32_t* __restrict__ wq, const SbView& sb,
                                            const int (&v)[N], int H, int u0, int stride,
                                            float (&dot)[N]) {
    if (sb.type == kSbF16) exact_parts_of<BITS, kSbF16, N, U>(hrow, wq, sb, v, H, u0, stride, dot);
    else if (sb.type == kSbBf16) exact_parts_of<BITS, kSbBf16, N, U>(hrow, wq, sb, v, H, u0, stride, dot);
    else exact_parts_of<BITS, kSbF32, N, U>(hrow, wq, sb, v, H, u0, stride, dot);
}

// Row r of the compact list of left-out columns and the exact capped logits
// of the row's teacher tokens.  Grid (M, K split): block (r, y) computes the
// logits k in [16 y, 16 y + 16), four to a warp; block (r, 0) also writes the
// list: the distinct valid ids in ascending order (each id's rank by counting:
// K^2 / 128 steps per thread), INT32_MAX behind them.  With the logits given
// (zout; no list then) it takes the teacher's out of them itself.  The gathered rows' bytes
// bound it, then the issue rate (one dot at a time and a conversion per code:
// 234 us at 5744 rows of 1536, K = 32).
template <int BITS>
__global__ void __launch_bounds__(kThreads) distill_prep_kernel(
    const uint32_t* __restrict__ wq, SbView sb, int64_t V, int H, float cap,
    const __nv_bfloat16* __restrict__ h, const int* pos,
    const int32_t* __restrict__ ids, int K, int* __restrict__ sid, float* kept, int64_t ld,
    float* zout) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    const int64_t r = blockIdx.x;
    const int i = pos[r];
    const int32_t* idr = ids + r * K;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int k0 = blockIdx.y * kWarps * kDotsPerWarp;
    kept += r * ld;
    if (i < 0) {
        for (int k = k0 + threadIdx.x; k < min(K, k0 + kWarps * kDotsPerWarp); k += kThreads) kept[k] = 0.f;
        return;
    }
    if (sid != nullptr && blockIdx.y == 0) {
        __shared__ int id_sh[kMaxTeacher];
        __shared__ uint8_t first_sh[kMaxTeacher];
        __shared__ int n_sh;
        if (threadIdx.x == 0) n_sh = 0;
        for (int k = threadIdx.x; k < K; k += kThreads) id_sh[k] = idr[k];
        __syncthreads();
        for (int k = threadIdx.x; k < K; k += kThreads) {
            const int id = id_sh[k];
            bool first = id >= 0 && (int64_t)id < V;
            for (int j = 0; j < k && first; ++j) first = id_sh[j] != id;
            first_sh[k] = first;
            if (first) atomicAdd(&n_sh, 1);
        }
        __syncthreads();
        int* out = sid + (int64_t)i * (K + 1);
        for (int k = threadIdx.x; k < K; k += kThreads) {
            if (!first_sh[k]) continue;
            const int id = id_sh[k];
            int rank = 0;
            for (int j = 0; j < K; ++j) rank += first_sh[j] && id_sh[j] < id;
            out[rank] = id;
        }
        for (int k = n_sh + threadIdx.x; k < K + 1; k += kThreads) out[k] = INT32_MAX;
    }
    const int kw = k0 + warp * kDotsPerWarp;
    if (kw >= K) return;
    int v[kDotsPerWarp];
#pragma unroll
    for (int d = 0; d < kDotsPerWarp; ++d) {
        const int id = kw + d < K ? idr[kw + d] : -1;
        v[d] = id >= 0 && (int64_t)id < V ? id : -1;
    }
    float z[kDotsPerWarp];
    exact_parts<BITS, kDotsPerWarp, 2>(h + r * (int64_t)H, wq, sb, v, H, lane, 32, z);
#pragma unroll
    for (int d = 0; d < kDotsPerWarp; ++d) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) z[d] += __shfl_xor_sync(0xffffffffu, z[d], o);
        if (lane == 0 && kw + d < K) {
            kept[kw + d] = v[d] >= 0 ? softcap_exact(z[d], cap) : 0.f;
            if (zout != nullptr && v[d] >= 0) zout[r * ld + v[d]] = -INFINITY;
        }
    }
}

// The teacher's side of a row, shared by the block: ids and scaled logits in
// shared memory.  bad: an id past V or a logit that is NaN or +inf.
struct Teacher {
    float tmax, tsum;  // largest t / T over the valid entries (-inf: none), sum of exponentials
    bool bad;
};

template <typename T>
__device__ __forceinline__ float load_t(const T* p) { return (float)*p; }
template <>
__device__ __forceinline__ float load_t(const __half* p) { return __half2float(*p); }
template <>
__device__ __forceinline__ float load_t(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <typename T>
__device__ __forceinline__ Teacher load_teacher(const int32_t* idr, const T* tr, int K, int64_t V,
                                                float inv_t, int* id_sh, float* t_sh, float* red) {
    Teacher te;
    float mx = -INFINITY;
    int bad = 0;
    for (int k = threadIdx.x; k < K; k += kThreads) {
        const int id = idr[k];
        float t = -INFINITY;
        if (id >= 0) {
            t = load_t(tr + k) * inv_t;
            if ((int64_t)id >= V || !(t < INFINITY)) bad = 1;
        }
        id_sh[k] = id;
        t_sh[k] = t;
        mx = fmaxf(mx, t);
    }
    te.bad = __syncthreads_or(bad) != 0;
    te.tmax = block_max(mx, red);
    float sum = 0.f;
    if (te.tmax > -INFINITY)
        for (int k = threadIdx.x; k < K; k += kThreads) sum += expf(t_sh[k] - te.tmax);
    te.tsum = block_sum(sum, red);
    return te;
}

// A logit as the tensor-core kernels form it but for their accumulation's rounding:
// fp16 operands, w = fma(code, scale, bias) rounded to fp16, summed here in fp32.  One
// lane computes one vocab row v.
template <int BITS>
__device__ float rounded_logit(const __nv_bfloat16* __restrict__ hrow, const uint32_t* __restrict__ wq,
                               const SbView& sb, int64_t v, int H) {
    const uint32_t* wr = wq + v * (int64_t)(H * BITS / 32);
    float acc[2] = {0.f, 0.f};
#pragma unroll 2
    for (int u = 0; u < H / 8; ++u) {
        const int64_t g = v * (int64_t)(H / 64) + u / 8;
        const uint32_t s2 = bcast_h(__float2half_rn(sb_elem(sb.s, g, sb.type)));
        const uint32_t b2 = bcast_h(__float2half_rn(sb_elem(sb.b, g, sb.type)));
        const uint4 hw = *reinterpret_cast<const uint4*>(hrow + 8 * u);
        const __nv_bfloat16* hp = reinterpret_cast<const __nv_bfloat16*>(&hw);
        uint32_t p[4];  // 4 bits: elements (k, k + 4); 8 bits: (2 k, 2 k + 1)
        if constexpr (BITS == 4) {
            deq4_word(wr[u], s2, b2, p);
        } else {
            const uint2 w = reinterpret_cast<const uint2*>(wr)[u];
            p[0] = deq8(w.x, 0x4140u, s2, b2);
            p[1] = deq8(w.x, 0x4342u, s2, b2);
            p[2] = deq8(w.y, 0x4140u, s2, b2);
            p[3] = deq8(w.y, 0x4342u, s2, b2);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 w = __half22float2(u32_as_h2(p[k]));
            const int a = BITS == 4 ? k : 2 * k, b = BITS == 4 ? k + 4 : 2 * k + 1;
            acc[0] = fmaf(__half2float(__float2half_rn(__bfloat162float(hp[a]))), w.x, acc[0]);
            acc[1] = fmaf(__half2float(__float2half_rn(__bfloat162float(hp[b]))), w.y, acc[1]);
        }
    }
    return acc[0] + acc[1];
}

// One block per row: merges the row's partials at the temperature, adds the
// exact terms of the teacher's distinct tokens, replaces those of the largest
// other logits by exact ones, and forms the loss.  The others: the columns whose
// share of the sum is at least kShare (a tensor-core logit is 3e-4 off: below
// that share it moves lse by less than 3e-7), the kOthers largest if there are
// more.  They lie in the slices of 32 columns whose maxima reach that share, and
// the kOthers largest in the kOthers slices of the largest maxima; those slices are
// looked through: the kept logits, or where none are kept the logits formed again.
// (With one candidate a slice, lse and loss of a row whose mass lies on two adjacent
// tokens were up to 1.4e-3 off; 7e-6 and 1.5e-5 so, for 33 us at 512 rows of 262144
// and 104 us at 5744 of 131072, the listed tokens' terms and coefficients included;
// 187 us at 5736 of 262144 without kept logits.)
constexpr float kShare = 1e-3f;
constexpr int kMaxShares = 1024;  // at most 1 / kShare slices or columns have that share

// Of the n candidates (value, index) the kOthers largest, in order, by counting.
__device__ __forceinline__ void take_largest(const float2* cand, int n, float* v, int* at) {
    for (int k = threadIdx.x; k < n; k += kThreads) {
        const float2 q = cand[k];
        int rank = 0;
        for (int j = 0; j < n; ++j) {
            const float2 o = cand[j];
            rank += better(o.x, __float_as_int(o.y), q.x, __float_as_int(q.y));
        }
        if (rank < kOthers) {
            v[rank] = q.x;
            at[rank] = __float_as_int(q.y);
        }
    }
}

template <int BITS, typename T>
__global__ void __launch_bounds__(kThreads, 4) distill_finalize_kernel(
    const uint32_t* __restrict__ wq, SbView sb, int64_t V, int H, float cap,
    const __nv_bfloat16* __restrict__ h, const int* __restrict__ pos,
    const int32_t* __restrict__ ids, const T* __restrict__ tl, int K, float inv_t, float unbias,
    float* kept, int64_t ld, float* zout, const Partial* part, int S,
    const int* S_dev, const float* smax, const int* err, float* __restrict__ loss,
    float* __restrict__ lse) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    __shared__ float2 cand_sh[kMaxShares];  // slices, then columns (v, i) of enough share
    __shared__ int n_slices, n_cand;
    __shared__ float hot_v[kOthers];        // the slices that are looked through
    __shared__ int hot_i[kOthers];
    __shared__ float red[kWarps];
    __shared__ float2 red2[kWarps];
    __shared__ int id_sh[kMaxTeacher];
    __shared__ float t_sh[kMaxTeacher];
    __shared__ float other_v[kOthers], other_z[kOthers];  // the others' logits: kernel's (raw, unbiased), exact
    __shared__ int other_i[kOthers];
    const int64_t r = blockIdx.x;
    const int i = pos[r];
    float* zr = kept + r * ld;
    // No other columns: rows that are off, whose kernel gave up, or whose gradient
    // the mark tells.
    auto no_others = [&](float mark) {
        for (int c = threadIdx.x; c < kOthers; c += kThreads) {
            zr[K + c] = c == 0 ? mark : 0.f;
            zr[K + kOthers + c] = 0.f;
        }
    };
    if (i < 0) {
        if (threadIdx.x == 0) loss[r] = lse[r] = 0.f;
        no_others(0.f);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int k = 8 * threadIdx.x; k < K; k += 8 * kThreads) {  // (read behind the partials)
        prefetch_l1(ids + r * K + k);
        prefetch_l1(tl + r * K + k);
        prefetch_l1(zr + k);
    }
    const int n_sl = (int)((V + 31) / 32);
    const float* sm = smax + (int64_t)i * slice_columns(V);
    for (int k = 32 * threadIdx.x; k < n_sl; k += 32 * kThreads) prefetch_l1(sm + k);
    if (S_dev) S = *S_dev;
    // Without a cap the kernel's factor `unbias` stands in its exponent: m in its terms.
    const float mscale = cap > 0.f ? 1.f : unbias;
    float m = -INFINITY, s = 0.f;
    int bad = *err != 0;
    auto fold = [&](float om, float os) {
        const float nm = fmaxf(m, om);
        if (nm > -INFINITY) s = s * expf((m - nm) * inv_t) + os * expf((om - nm) * inv_t);
        m = nm;
    };
    const Partial* prow = part + (int64_t)i * S;
    for (int k = threadIdx.x; k < S; k += kThreads) {
        const Partial p = prow[k];
        bad |= p.status;
        fold(p.m * mscale, p.s);
    }
    if (threadIdx.x == 0) n_slices = n_cand = 0;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) loss[r] = lse[r] = nan_f();
        no_others(INFINITY);
        return;
    }
#pragma unroll
    for (int o = 1; o <= 16; o <<= 1) {
        // (the lower lane's state first, so that both partners end equal)
        const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
        const float am = lane & o ? om : m, as = lane & o ? os : s;
        const float bm = lane & o ? m : om, bs = lane & o ? s : os;
        m = am;
        s = as;
        fold(bm, bs);
    }
    if (lane == 0) red2[warp] = make_float2(m, s);
    __syncthreads();
    m = -INFINITY;
    s = 0.f;
    for (int w = 0; w < kWarps; ++w) fold(red2[w].x, red2[w].y);

    // The teacher's side, and its tokens' exact terms.
    const Teacher te = load_teacher(ids + r * K, tl + r * K, K, V, inv_t, id_sh, t_sh, red);
    float top = m;
    for (int k = threadIdx.x; k < K; k += kThreads)
        if (id_sh[k] >= 0 && (int64_t)id_sh[k] < V) top = fmaxf(top, zr[k]);
    top = block_max(top, red);
    float sum = 0.f, cross = 0.f;
    const float lsum = te.tsum > 0.f ? logf(te.tsum) : 0.f;
    for (int k = threadIdx.x; k < K; k += kThreads) {
        const int id = id_sh[k];
        if (id < 0 || (int64_t)id >= V) continue;
        bool first = true;  // a token listed twice is one term of the sum
        for (int j = 0; j < k && first; ++j) first = id_sh[j] != id;
        const float z = zr[k];
        if (first) sum += expf((z - top) * inv_t);
        const float lp = t_sh[k] - te.tmax - lsum;
        const float p = expf(lp);
        if (p > 0.f) cross += p * (lp - (z - top) * inv_t);  // (log p - z/T, from `top`)
    }
    sum = block_sum(sum, red);
    cross = block_sum(cross, red);
    float rest = m > -INFINITY ? s * expf((m - top) * inv_t) : 0.f;

    // The slices of enough share (in any order), then the largest of them by rank.
    // floor: the raw logit of that share (the cap is monotone).
    float floor = top + logf(kShare * (rest + sum)) / inv_t;
    if (cap > 0.f) {
        const float f = floor / cap;
        floor = f >= 1.f ? INFINITY : f <= -1.f ? -INFINITY : cap * atanhf(f);
    }
    auto enough = [&](float z) { return z > -INFINITY && z >= floor; };
    for (int k0 = 4 * threadIdx.x; k0 < n_sl; k0 += 16 * kThreads) {
        float4 q[4];  // (whole tiles of 8: the rest of a group of four is there)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = k0 + 4 * kThreads * e;
            q[e] = k < n_sl ? *reinterpret_cast<const float4*>(sm + k) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x[4] = {q[e].x, q[e].y, q[e].z, q[e].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = k0 + 4 * kThreads * e + j;
                if (k < n_sl && enough(x[j] * unbias)) {
                    const int n = atomicAdd(&n_slices, 1);
                    if (n < kMaxShares) cand_sh[n] = make_float2(x[j], __int_as_float(k));
                }
            }
        }
    }
    __syncthreads();
    const int all_hot = min(n_slices, kMaxShares), n_hot = min(all_hot, kOthers);
    take_largest(cand_sh, all_hot, hot_v, hot_i);
    __syncthreads();
    // Their columns, a slice to a warp.
    for (int c = warp; c < n_hot; c += kWarps) {
        const int col = 32 * hot_i[c] + lane;
        float x = -INFINITY;  // the kernel's raw logit, unbiased; -inf: a listed token, or past V
        if ((int64_t)col < V) {
            if (zout != nullptr) {
                x = zout[r * ld + col] * unbias;
            } else {
                x = rounded_logit<BITS>(h + r * (int64_t)H, wq, sb, col, H);
                if (enough(x))
                    for (int k = 0; k < K; ++k)
                        if (id_sh[k] == col) x = -INFINITY;
            }
        }
        if (enough(x)) {
            const int n = atomicAdd(&n_cand, 1);  // (at most 32 kOthers)
            cand_sh[n] = make_float2(x, __int_as_float(col));
        }
    }
    __syncthreads();
    const int n_all = n_cand, n_other = min(n_all, kOthers);
    take_largest(cand_sh, n_all, other_v, other_i);
    __syncthreads();
    // Their exact logits, two to a warp; the kernel's terms out.
#pragma unroll 1
    for (int c = 2 * warp; c < n_other; c += 2 * kWarps) {
        const int cv[2] = {other_i[c], c + 1 < n_other ? other_i[c + 1] : -1};
        float z[2];
        exact_parts<BITS, 2, 2>(h + r * (int64_t)H, wq, sb, cv, H, lane, 32, z);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) z[e] += __shfl_xor_sync(0xffffffffu, z[e], o);
            if (cv[e] >= 0 && lane == 0) other_z[c + e] = softcap_exact(z[e], cap);
        }
    }
    __syncthreads();
    if (warp == 0) {
        const bool have = lane < n_other;
        float out_of = 0.f, add = 0.f;  // the kernel's terms, the exact ones
        if (have) {
            out_of = expf((softcap_exact(other_v[lane], cap) - top) * inv_t);
            add = expf((other_z[lane] - top) * inv_t);
        }
        if (lane < kOthers) {
            zr[K + lane] = have ? other_z[lane] : 0.f;
            zr[K + kOthers + lane] = __int_as_float(have ? other_i[lane] + 1 : 0);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            out_of += __shfl_xor_sync(0xffffffffu, out_of, o);
            add += __shfl_xor_sync(0xffffffffu, add, o);
        }
        rest -= out_of;
        const float l = logf((rest < 0.f ? 0.f : rest) + add + sum);  // lse - top / T (NaN stays)
        if (lane == 0) {
            lse[r] = fmaf(top, inv_t, l);
            float out = cross + l;
            if (te.tmax == -INFINITY) out = 0.f;  // nothing to learn from
            if (te.bad) out = nan_f();
            loss[r] = out;
            red[0] = l;
        }
    }
    __syncthreads();
    if (te.bad || te.tmax == -INFINITY) {
        no_others(te.bad ? INFINITY : -INFINITY);
        return;
    }
    if (zout == nullptr) return;
    // The listed columns' coefficients (q - p) sech2 among the logits.
    zout += r * ld;
    const float l = red[0], rsum = 1.f / te.tsum;
    for (int k = threadIdx.x; k < K + n_other; k += kThreads) {
        const int id = k < K ? id_sh[k] : other_i[k - K];
        if (id < 0 || (int64_t)id >= V) continue;
        float p = 0.f;  // the token's teacher mass (every entry that lists it)
        if (k < K)
            for (int j = 0; j < K; ++j)
                if (id_sh[j] == id) p += expf(t_sh[j] - te.tmax) * rsum;
        const float z = k < K ? zr[k] : other_z[k - K];
        const float th = cap > 0.f ? z / cap : 0.f;
        const float c = (expf(fmaf(z - top, inv_t, -l)) - p) * fmaf(-th, th, 1.f) * kMark;
        zout[id] = fabsf(c) < kMarked ? -INFINITY : c;
    }
}

// Without kept logits: one block per row, after the coefficient pass of the vocab
// chunk [v_begin, v_begin + chunk): writes (q_k - p_k) sech2_k * 2^14 over the
// teacher's columns and the kept others (|q - p| <= 1: at most 16384 in
// fp16, one rounding) and
// the row's cotangent as the contraction kernel takes it, -dloss / T (0 for a
// row with nothing to learn from, NaN for a bad one).
template <typename T>
__global__ void __launch_bounds__(kThreads) distill_coeff_kernel(
    int64_t V, float cap, const int* pos, const int32_t* __restrict__ ids,
    const T* __restrict__ tl, int K, float inv_t, const float* __restrict__ kept, int64_t ld_kept,
    const float* __restrict__ lse, const float* __restrict__ dloss, float* __restrict__ geff,
    __half* coeff, int64_t ld, int64_t v_begin, int64_t chunk) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    const int64_t r = blockIdx.x;
    const int i = pos[r];
    if (i < 0) return;
    __shared__ float red[kWarps];
    __shared__ int id_sh[kMaxTeacher];
    __shared__ float t_sh[kMaxTeacher];
    const Teacher te = load_teacher(ids + r * K, tl + r * K, K, V, inv_t, id_sh, t_sh, red);
    if (threadIdx.x == 0 && v_begin == 0)
        geff[r] = te.bad ? nan_f() : te.tmax == -INFINITY ? 0.f : -dloss[r] * inv_t;
    if (te.bad || te.tmax == -INFINITY) return;
    const float rsum = 1.f / te.tsum, l = lse[r];
    const float* zr = kept + r * ld_kept;
    for (int k = threadIdx.x; k < K + kOthers; k += kThreads) {
        const int id = k < K ? id_sh[k] : __float_as_int(zr[k + kOthers]) - 1;
        if (id < v_begin || id >= v_begin + chunk || (int64_t)id >= V) continue;
        float p = 0.f;  // the token's teacher mass (every entry that lists it)
        if (k < K)
            for (int j = 0; j < K; ++j)
                if (id_sh[j] == id) p += expf(t_sh[j] - te.tmax) * rsum;
        const float z = zr[k];
        const float th = cap > 0.f ? z / cap : 0.f;
        const float c = (expf(fmaf(z, inv_t, -l)) - p) * fmaf(-th, th, 1.f);
        coeff[(int64_t)i * ld + (id - v_begin)] = __float2half_rn(c * 16384.f);
    }
}

// Softmax partials of the kept logits (few rows): block (s, r) takes split s of
// row r, whole slices of 32 columns; the largest capped logit, the sum at the
// temperature relative to it, and every slice's largest raw logit.
constexpr int kSplitThreads = 256;
__global__ void __launch_bounds__(kSplitThreads) distill_split_kernel(
    const float* z, int64_t ld, int64_t V, float cap, float inv_t,
    const int* pos, Partial* __restrict__ part, float* __restrict__ smax, int S) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    const int64_t r = blockIdx.y;
    const int i = pos[r], sp = blockIdx.x;
    if (i < 0) return;
    const int64_t n_sl = (V + 31) / 32;
    const int64_t v0 = 32 * (n_sl * sp / S), v1 = min(V, 32 * (n_sl * (sp + 1) / S));
    const float* zr = z + r * ld;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* sm = smax + (int64_t)i * slice_columns(V);
    float m = -INFINITY, s = 0.f;
    bool bad = false;  // a NaN logit
    for (int64_t base = v0; base < v1; base += 8 * kSplitThreads) {
        const int64_t vb = base + threadIdx.x;
        float x[8], y[8], top = -INFINITY;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = vb + k * kSplitThreads < v1 ? zr[vb + k * kSplitThreads] : -INFINITY;
        // The warp's 8 slices' maxima: each level halves the values with the lanes;
        // lane (a, b, c, ..) ends with slice 4 a + 2 b + c.
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = x[k];
#pragma unroll
        for (int n = 4, o = 16; n >= 1; n >>= 1, o >>= 1) {
#pragma unroll
            for (int k = 0; k < n; ++k) {
                const float give = lane & o ? y[k] : y[k + n];
                y[k] = fmaxf(lane & o ? y[k + n] : y[k], __shfl_xor_sync(0xffffffffu, give, o));
            }
        }
        y[0] = fmaxf(y[0], __shfl_xor_sync(0xffffffffu, y[0], 2));
        y[0] = fmaxf(y[0], __shfl_xor_sync(0xffffffffu, y[0], 1));
        const int64_t col = base + 32 * warp + (int64_t)(lane >> 2) * kSplitThreads;
        if ((lane & 3) == 0 && col < v1) sm[col / 32] = y[0];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            bad |= x[k] != x[k];
            if (x[k] > -INFINITY) {
                x[k] = softcap_exact(x[k], cap);
                top = fmaxf(top, x[k]);
            }
        }
        if (top == -INFINITY) continue;
        const float nm = fmaxf(m, top);
        s *= m > -INFINITY ? expf((m - nm) * inv_t) : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (x[k] > -INFINITY) s += expf((x[k] - nm) * inv_t);
        m = nm;
    }
    if (bad) {
        m = 0.f;
        s = nan_f();
    }
    __shared__ float2 red[kSplitThreads / 32];
    auto fold = [&](float om, float os) {
        const float nm = fmaxf(m, om);
        if (nm > -INFINITY) s = s * expf((m - nm) * inv_t) + os * expf((om - nm) * inv_t);
        m = nm;
    };
#pragma unroll
    for (int o = 1; o <= 16; o <<= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
        const float am = lane & o ? om : m, as = lane & o ? os : s;
        const float bm = lane & o ? m : om, bs = lane & o ? s : os;
        m = am;
        s = as;
        fold(bm, bs);
    }
    if (lane == 0) red[warp] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x != 0) return;
    m = -INFINITY;
    s = 0.f;
    for (int w = 0; w < kSplitThreads / 32; ++w) fold(red[w].x, red[w].y);
    RowState none;
    none.init();
    Partial p = none.to_partial();
    p.m = m;
    p.s = s;
    part[(int64_t)i * S + sp] = p;
}

// The coefficient block of the chunk [v_begin, v_begin + chunk) from the kept
// logits: q sech2 2^14 in fp16 (zeros past V) with the arithmetic of the logit
// kernel's own coefficient epilogue, or the kept coefficient; and the row's
// cotangent (see distill_coeff_kernel).  Thread = kPieces times 8 columns of one
// active row; the rows past the active ones are not written (nothing reads what the
// contraction makes of them).  Bound by bytes, 4 read and 2 written per logit: 6.8
// TB/s at 5744 x 131072 (666 us; 726 with 2 pieces, 899 with one: the loads of a
// block that lives for three dependent rounds are in flight in one of them).
constexpr int kPieces = 4;
__global__ void __launch_bounds__(256, 4) distill_from_logits_kernel(
    const float* __restrict__ z, const float* __restrict__ first_other, int64_t ld, int64_t V, float cap,
    float inv_t, float unbias, const int* rows, const int* count, const float* __restrict__ lse,
    const float* __restrict__ dloss, float* __restrict__ geff, __half* __restrict__ coeff, int64_t ldc,
    int64_t v_begin, int64_t chunk) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    constexpr float kL2e = 1.4426950408889634f;
    constexpr int kStep = 256 * 8;
    // blocks run along a row, row after row
    const int per_row = (int)((chunk + kPieces * kStep - 1) / (kPieces * kStep));
    const int i = blockIdx.x / per_row;
    const int64_t r = rows[i];  // (-1 past the active rows)
    if (i >= *count) return;
    const int64_t c0 = (int64_t)(blockIdx.x % per_row) * kPieces * kStep + threadIdx.x * 8;
    const float* zr = z + r * ld + v_begin;
    float x[kPieces][8];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        const int64_t c = c0 + p * kStep, v = v_begin + c;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[p][k] = -INFINITY;
        if (c >= chunk) continue;
        if (v + 8 <= V) {
            load8_wide(zr + c, x[p]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (v + k < V) x[p][k] = zr[c + k];
        }
    }
    if (v_begin + c0 == 0) {
        const float mark = first_other[r * ld];
        geff[r] = mark == INFINITY ? nan_f() : mark == -INFINITY ? 0.f : -dloss[r] * inv_t;
    }
    const float lsb = lse[r] * kL2e - 14.f;
    const float k2 = cap > 0.f ? 2.f * kL2e / cap * unbias : 0.f;
    const float l2e = kL2e * inv_t * (cap > 0.f ? 1.f : unbias);
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        if (c0 + p * kStep >= chunk) break;
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float xv = x[p][k];
            float zc = xv, sech2 = 1.f;
            if (cap > 0.f) {
                const float th = fmaf(-2.f, tc::rcp_approx(tc::ex2_approx(xv * k2) + 1.f), 1.f);
                zc = cap * th;
                sech2 = fmaf(-th, th, 1.f);
            }
            o[k] = tc::ex2_approx(fmaf(zc, l2e, -lsb)) * sech2;
            if (fabsf(xv) >= kMarked) o[k] = xv == -INFINITY ? 0.f : xv * (16384.f / kMark);
        }
        store8(coeff + (int64_t)i * ldc + c0 + p * kStep, o);
    }
}

// One block per row: the K slices of the contraction in order, rounded once to
// bf16.  Inactive rows are zeros; if a head kernel gave up, active rows NaN.
__global__ void __launch_bounds__(256) distill_dh_kernel(const float* dhp, int S,
                                                         int64_t Mpad, int H,
                                                         const int* __restrict__ pos,
                                                         const int* err,
                                                         __nv_bfloat16* __restrict__ dh) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    const int64_t r = blockIdx.x;
    const int i = pos[r];
    const bool bad = *err != 0;
    for (int u = threadIdx.x; u < H / 8; u += blockDim.x) {
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = i >= 0 && bad ? nan_f() : 0.f;
        if (i >= 0 && !bad) {
            for (int sl = 0; sl < S; ++sl) {
                const float4* src =
                    reinterpret_cast<const float4*>(dhp + ((int64_t)sl * Mpad + i) * H + 8 * u);
                const float4 a = src[0], b = src[1];
                acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
                acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
            }
        }
        __nv_bfloat162 o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __floats2bfloat162_rn(acc[2 * e], acc[2 * e + 1]);
        *reinterpret_cast<uint4*>(dh + r * (int64_t)H + 8 * u) = *reinterpret_cast<const uint4*>(o);
    }
}

// Calls f with a null pointer of the element type of code `type`.
template <typename F>
cudaError_t with_type(int type, F&& f) {
    if (type == kSbF16) return f(static_cast<const __half*>(nullptr));
    if (type == kSbBf16) return f(static_cast<const __nv_bfloat16*>(nullptr));
    return f(static_cast<const float*>(nullptr));
}

}  // namespace

cudaError_t launch_distill_prep(const uint32_t* wq, SbView sb, int64_t V, int H, int bits, float cap,
                                const __nv_bfloat16* h, const int* pos, int64_t M,
                                const int32_t* ids, int K, int* sid, float* kept, int64_t ld,
                                float* zout, cudaStream_t st) {
    constexpr int per = kWarps * kDotsPerWarp;
    const dim3 grid((unsigned)M, (unsigned)((K + per - 1) / per));
    auto* fn = bits == 4 ? distill_prep_kernel<4> : distill_prep_kernel<8>;
    return launch_after(fn, grid, dim3(kThreads), st, wq, sb, V, H, cap, h, pos, ids, K, sid, kept, ld, zout);
}

cudaError_t launch_distill_finalize(const uint32_t* wq, SbView sb, int64_t V, int H, int bits,
                                    float cap, const __nv_bfloat16* h, const int* pos, int64_t M,
                                    const int32_t* ids, const void* tl, int t_type, int K,
                                    float inv_t, float unbias, float* kept, int64_t ld, float* zout,
                                    const Partial* part, int S, const int* S_dev, const float* smax,
                                    const int* err, float* loss, float* lse, cudaStream_t st) {
    return with_type(t_type, [&](auto* tag) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        auto* fn = bits == 4 ? distill_finalize_kernel<4, T> : distill_finalize_kernel<8, T>;
        return launch_after(fn, dim3((unsigned)M), dim3(kThreads), st, wq, sb, V, H, cap, h, pos, ids,
                            static_cast<const T*>(tl), K, inv_t, unbias, kept, ld, zout, part, S, S_dev, smax,
                            err, loss, lse);
    });
}

cudaError_t launch_distill_coeff(int64_t V, float cap, const int* pos, int64_t M,
                                 const int32_t* ids, const void* tl, int t_type, int K, float inv_t,
                                 const float* kept, int64_t ld_kept, const float* lse,
                                 const float* dloss, float* geff, __half* coeff, int64_t ld,
                                 int64_t v_begin, int64_t chunk, cudaStream_t st) {
    return with_type(t_type, [&](auto* tag) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        return launch_after(distill_coeff_kernel<T>, dim3((unsigned)M), dim3(kThreads), st, V, cap, pos, ids,
                            static_cast<const T*>(tl), K, inv_t, kept, ld_kept, lse, dloss, geff, coeff, ld,
                            v_begin, chunk);
    });
}

cudaError_t launch_distill_split(const float* z, int64_t ld, int64_t V, float cap, float inv_t,
                                 const int* pos, int64_t M, Partial* part, float* smax,
                                 cudaStream_t st) {
    return launch_after(distill_split_kernel, dim3(kFewSplits, (unsigned)M), dim3(kSplitThreads), st, z, ld, V,
                        cap, inv_t, pos, part, smax, kFewSplits);
}

cudaError_t launch_distill_from_logits(const float* kept, int64_t K, int64_t ld, int64_t V, float cap,
                                       float inv_t, float unbias, const int* rows, const int* count, int64_t M,
                                       const float* lse, const float* dloss, float* geff, __half* coeff, int64_t ldc, int64_t v_begin,
                                       int64_t chunk, cudaStream_t st) {
    // (within 2^31 blocks: M V is at most 2^30 here, or M at most kFewM)
    constexpr int64_t per = 256 * 8 * kPieces;
    const dim3 grid((unsigned)((chunk + per - 1) / per * M));
    return launch_after(distill_from_logits_kernel, grid, dim3(256), st, kept + kept_logits_at(K), kept + K, ld, V,
                        cap, inv_t, unbias, rows, count, lse, dloss, geff, coeff, ldc, v_begin, chunk);
}

cudaError_t launch_distill_dh(const float* dhp, int S, int64_t Mpad, int H, const int* pos,
                              int64_t M, const int* err, void* dh, cudaStream_t st) {
    return launch_after(distill_dh_kernel, dim3((unsigned)M), dim3(256), st, dhp, S, Mpad, H, pos, err,
                        static_cast<__nv_bfloat16*>(dh));
}

}  // namespace qh
