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
#include "qh_norm.cuh"

namespace qh {

namespace {

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

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t st) { return launch_bwd<false>(a, st); }

}  // namespace qh
