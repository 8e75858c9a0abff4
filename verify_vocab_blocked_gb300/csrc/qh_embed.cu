// qh_embed.cu -- the other end of a tied quantized table: rows looked up and
// dequantized with a scale, and the gradient of the table.
//
//     y[m, :]   = scale * (s[t, d / 64] * q[t, d] + b[t, d / 64]),  t = tokens[m]
//     dW[v, :] (+)= scale * sum_{m : t_m = v} dy[m, :]
//
// Lookup: one fp32 FMA and one multiplication per element, rounded once to the
// output's type.  It is bound by bytes (the packed row once, the output once).
//
// Gradient: the live rows are sorted by token (stable, so every token's rows
// come in ascending order), then blocks of consecutive sorted rows sum the
// runs of equal tokens in registers.  A run inside one block is written to dW
// by that block; the parts of a run that crosses blocks go to the workspace
// and a further launch adds them in order.  So dW has no atomics, a frequent
// token's rows are spread over many blocks, and the result does not depend on
// the launch.  Bytes: dy once, dW's touched rows once (read too when added to).
// A fresh dW is filled with zeros by a launch that runs beside the sort:
// writing the touched rows twice costs less (30 of 2700 MB at 262144 x 2560)
// than picking the untouched ones out behind the sort (643 us for zeros and
// sums in one launch; 344 us for the zeros now, 7.8 TB/s).
#include "qh_ops.cuh"
#include "qh_tc.cuh"

namespace qh {

namespace {

// The packed codes of one 8-element unit.
struct Unit {
    uint32_t w0, w1;
    float s, b;
};

__device__ __forceinline__ Unit load_unit(const uint32_t* __restrict__ wq, const SbView& sb, int64_t t,
                                          int u, int H, int bits) {
    Unit x;
    const uint32_t* row = wq + t * (int64_t)(H * bits / 32);
    if (bits == 4) {
        x.w0 = row[u];
        x.w1 = 0u;
    } else {
        const uint2 w = reinterpret_cast<const uint2*>(row)[u];
        x.w0 = w.x;
        x.w1 = w.y;
    }
    const int64_t g = t * (int64_t)(H / 64) + u / 8;
    x.s = sb_elem(sb.s, g, sb.type);
    x.b = sb_elem(sb.b, g, sb.type);
    return x;
}

__device__ __forceinline__ void unit_values(const Unit& x, int bits, float scale, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = scale * fmaf(x.s, bits == 4 ? code_f32<4>(x.w0, 0u, e) : code_f32<8>(x.w0, x.w1, e), x.b);
}

// Thread = one 8-element unit of R consecutive rows; the R rows' loads are
// issued together (two dependent rounds: tokens, then packed units).
template <int R>
__global__ void __launch_bounds__(kMaxH / 8) embed_kernel(
    const uint32_t* __restrict__ wq, SbView sb, int64_t V, int H, int bits,
    const int32_t* __restrict__ tokens, const uint8_t* __restrict__ mask, int64_t M, float scale,
    void* __restrict__ out, int out_type, int wide) {
    const int u = threadIdx.x;
    if (u >= H / 8) return;
    const int64_t m0 = (int64_t)blockIdx.x * R;
    int t[R];
    bool on[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        on[i] = m0 + i < M && (mask == nullptr || mask[m0 + i] != 0);
        t[i] = m0 + i < M ? tokens[m0 + i] : 0;
    }
    Unit x[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (on[i] && t[i] >= 0 && (int64_t)t[i] < V) x[i] = load_unit(wq, sb, t[i], u, H, bits);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (m0 + i >= M) break;
        float v[8];
        if (!on[i]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
        } else if (t[i] < 0 || (int64_t)t[i] >= V) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __int_as_float(0x7fc00000);
        } else {
            unit_values(x[i], bits, scale, v);
        }
        // (fp32 in one 32-byte store: two of 16 bytes write every sector in halves)
        if (wide) store8_wide(static_cast<float*>(out) + (m0 + i) * H + 8 * u, v);
        else store8_as(out, (m0 + i) * H + 8 * u, out_type, v);
    }
}

// ------------------------------------------------------------------- sorting

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 512;    // 9 bits
constexpr int kSortCluster = 8;   // CTAs of the sorting cluster

struct SortSmem {
    uint32_t cnt[kSortWarps * kMaxDigit];  // per warp and digit: count, then offset
    uint32_t tot[kMaxDigit];               // this CTA's rows per digit
    uint32_t base[kMaxDigit];              // first sorted position of the CTA's rows per digit
    uint32_t warp_tot[kSortWarps];
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// Stable counting sort of the live rows by token, least-significant digit
// first, in one cluster: every warp owns a contiguous slice of the keys, counts
// its digits, and (after the CTAs have exchanged their totals through
// distributed shared memory) scatters its slice in order.  Rows that are
// masked or whose token lies outside [0, V) drop out in the first pass.
// info[0] = live rows, info[1] = 0.  One launch, no global atomics.  Latency bounds it: a
// slice of up to kHeld batches of 32 keys is loaded once a pass, all batches
// together, and stays in registers between the counting and the scatter.
constexpr int kHeld = 8;

// The lanes whose key has this lane's digit (of the lanes in `live`).
__device__ __forceinline__ uint32_t same_digit(uint32_t d, int width, uint32_t live) {
    uint32_t same = live;
#pragma unroll
    for (int b = 0; b < 9; ++b) {
        if (b >= width) break;
        const uint32_t bit = d >> b & 1u;
        const uint32_t bal = __ballot_sync(0xffffffffu, bit);
        same &= bit ? bal : ~bal;
    }
    return same;
}

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(
    const int32_t* __restrict__ tokens, const uint8_t* __restrict__ mask, int64_t M, int64_t V,
    int passes, int width, uint2* buf_a, uint2* buf_b, int* info) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SortSmem& sm = *reinterpret_cast<SortSmem*>(smem_raw);
    tc::grid_dep_trigger();  // (the zeros of a fresh dW may start)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int C = kSortCluster;
    const int c = (int)blockIdx.x;
    const int n_digit = 1 << width;
    int64_t n = M;
    uint32_t* cnt = sm.cnt + warp * kMaxDigit;
    for (int p = 0; p < passes; ++p) {
        const uint2* src = p & 1 ? buf_a : buf_b;  // (pass 0 reads the tokens)
        uint2* dst = p & 1 ? buf_b : buf_a;
        const int shift = p * width;
        // this warp's slice, whole batches of 32 keys
        int64_t len = (n + (int64_t)C * kSortWarps - 1) / ((int64_t)C * kSortWarps);
        len = (len + 31) / 32 * 32;
        const int64_t lo = ((int64_t)c * kSortWarps + warp) * len;
        const int64_t hi = lo + len < n ? lo + len : n;
        uint2 k[kHeld];
        uint32_t live = 0;  // bit j: this lane's key of batch j takes part
        auto load = [&](int64_t i0) {
            live = 0;
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                const int64_t i = i0 + 32 * j + lane;
                k[j] = make_uint2(0u, 0u);
                if (i >= hi) continue;
                if (p == 0) {
                    const int32_t t = tokens[i];
                    k[j] = make_uint2((uint32_t)t, (uint32_t)i);
                    if (t >= 0 && (int64_t)t < V && (mask == nullptr || mask[i] != 0)) live |= 1u << j;
                } else {
                    k[j] = src[i];
                    live |= 1u << j;
                }
            }
        };
        load(lo);
        for (int d = tid; d < kSortWarps * kMaxDigit / 4; d += kSortThreads)
            reinterpret_cast<uint4*>(sm.cnt)[d] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        for (int64_t i0 = lo; i0 < hi; i0 += 32 * kHeld) {
            if (i0 > lo) load(i0);
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                if (i0 + 32 * j >= hi) break;
                const bool ok = live >> j & 1u;
                const uint32_t d = (k[j].x >> shift) & (uint32_t)(n_digit - 1);
                const uint32_t same = same_digit(d, width, __ballot_sync(0xffffffffu, ok));
                if (ok && lane == __ffs(same) - 1) cnt[d] += __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        if (tid < n_digit) {  // counts -> offsets within the CTA's rows of the digit
            uint32_t run = 0;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t t = sm.cnt[w * kMaxDigit + tid];
                sm.cnt[w * kMaxDigit + tid] = run;
                run += t;
            }
            sm.tot[tid] = run;
        }
        tc::cluster_sync();
        uint32_t all = 0, before = 0;
        if (tid < n_digit) {
#pragma unroll
            for (int o = 0; o < kSortCluster; ++o) {
                const uint32_t t = ld_cluster_u32(tc::mapa_shared(&sm.tot[tid], o));
                if (o < c) before += t;
                all += t;
            }
        }
        // exclusive prefix over the digits
        uint32_t incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) sm.warp_tot[warp] = incl;
        __syncthreads();
        // (warps past the digits hold zeros)
        const uint32_t wt = sm.warp_tot[lane];
        uint32_t add = lane < warp ? wt : 0u, total = wt;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            add += __shfl_xor_sync(0xffffffffu, add, o);
            total += __shfl_xor_sync(0xffffffffu, total, o);
        }
        if (tid < n_digit) sm.base[tid] = add + incl - all + before;
        __syncthreads();
        for (int64_t i0 = lo; i0 < hi; i0 += 32 * kHeld) {
            if (len > 32 * kHeld) load(i0);  // (else still held)
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                if (i0 + 32 * j >= hi) break;
                const bool ok = live >> j & 1u;
                const uint32_t d = (k[j].x >> shift) & (uint32_t)(n_digit - 1);
                const uint32_t same = same_digit(d, width, __ballot_sync(0xffffffffu, ok));
                uint32_t at = 0;
                if (ok) at = sm.base[d] + cnt[d] + __popc(same & ((1u << lane) - 1u));
                __syncwarp();
                if (ok && lane == __ffs(same) - 1) cnt[d] += __popc(same);
                __syncwarp();
                if (ok) dst[at] = k[j];
            }
        }
        n = total;
        // The cluster's writes are visible and its totals read before the next pass.
        tc::cluster_sync();
    }
    if (c == 0 && tid == 0) {
        info[0] = (int)n;
        info[1] = 0;
    }
}

// The same order for up to kRankM rows by counting: a row's position is the number
// of live rows with a smaller token, or the same and an earlier row.  Every block
// holds all tokens in shared memory and a warp counts for a row at a time, so it
// is M^2 comparisons spread over the SMs against the radix sort's two passes of
// fixed cost: 2.5 us at 256 rows, 3.4 at 2048, 5.4 at 4096, 12.8 at 8192, where the
// radix sort, 12 to 14 us from the smallest on, meets it.
constexpr int kRankM = 8192;
constexpr int kRankThreads = 512;
__global__ void __launch_bounds__(kRankThreads) embed_rank_kernel(
    const int32_t* __restrict__ tokens, const uint8_t* __restrict__ mask, int M, int64_t V,
    uint2* __restrict__ out, int* __restrict__ info) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    int* tok = reinterpret_cast<int*>(smem_raw);  // dropped rows: INT32_MAX
    tc::grid_dep_trigger();
    const int n4 = (M + 3) / 4;
    int live = 0;
    for (int i = threadIdx.x; i < 4 * n4; i += kRankThreads) {
        int t = INT32_MAX;
        if (i < M) {
            const int x = tokens[i];
            if (x >= 0 && (int64_t)x < V && (mask == nullptr || mask[i] != 0)) t = x;
        }
        tok[i] = t;
        live += t != INT32_MAX;
    }
    if (blockIdx.x == 0) {
        __shared__ int total;
        if (threadIdx.x == 0) total = 0;
        __syncthreads();
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) live += __shfl_xor_sync(0xffffffffu, live, o);
        if ((threadIdx.x & 31) == 0) atomicAdd(&total, live);
        __syncthreads();
        if (threadIdx.x == 0) {
            info[0] = total;
            info[1] = 0;
        }
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4* tok4 = reinterpret_cast<const int4*>(tok);
    for (int r = blockIdx.x * (kRankThreads / 32) + warp; r < M; r += gridDim.x * (kRankThreads / 32)) {
        const int t = tok[r];
        if (t == INT32_MAX) continue;
        // groups of four before r's: not above t; r's own, exactly; behind: below t
        const int own = r >> 2;
        int n = 0;
        for (int j = lane; j < own; j += 32) {
            const int4 x = tok4[j];
            n += (x.x <= t) + (x.y <= t) + (x.z <= t) + (x.w <= t);
        }
        for (int j = own + 1 + lane; j < n4; j += 32) {
            const int4 x = tok4[j];
            n += (x.x < t) + (x.y < t) + (x.z < t) + (x.w < t);
        }
        if (lane < 4) {
            const int j = 4 * own + lane;
            n += j < r ? tok[j] <= t : tok[j] < t;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        if (lane == 0) out[n] = make_uint2((uint32_t)t, (uint32_t)r);
    }
}

// dW = 0, beside the sort (launched as its dependent): 32-byte stores, each block
// one contiguous piece, the blocks in order (with blocks that stay and stride the
// stores reach 6.4 to 6.6 TB/s, so 7.8).  The last block ends behind the sort, so
// that what waits for this launch waits for both.
constexpr int kZeroThreads = 256, kZeroUnroll = 4;
__global__ void __launch_bounds__(kZeroThreads) embed_zero_kernel(float* __restrict__ dw, int64_t n32) {
    tc::grid_dep_trigger();
    const uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    const int64_t i0 = (int64_t)blockIdx.x * kZeroThreads * kZeroUnroll + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kZeroUnroll; ++u)
        if (i0 + u * kZeroThreads < n32) tc::st_global_v8(dw + 8 * (i0 + u * kZeroThreads), z);
    if (blockIdx.x == gridDim.x - 1) tc::grid_dep_wait();
}

// ------------------------------------------------------------------- summing

constexpr int kMaxChunk = 64;

// Block = chunk sorted rows x all columns, thread = 8 columns.
template <typename T>
__global__ void __launch_bounds__(kMaxH / 8) embed_sum_kernel(
    const uint2* sorted, int* info, int chunk, int H, float scale,
    const T* __restrict__ dy, float* dw, int accumulate, float* __restrict__ part, int* __restrict__ joins) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    const int u = threadIdx.x;
    const int units = H / 8;
    __shared__ uint2 key[kMaxChunk + 2];  // the chunk's pairs, one before and one behind
    const int n = info[0];
    const int64_t c = blockIdx.x;
    const int64_t p0 = c * chunk;
    if (p0 >= n) return;
    const int len = (int)min((int64_t)chunk, n - p0);
    for (int i = threadIdx.x; i < len + 2; i += blockDim.x) {
        const int64_t p = p0 + i - 1;
        key[i] = p >= 0 && p < n ? sorted[p] : make_uint2(0xffffffffu, 0u);
    }
    __syncthreads();
    // (a run that begins here and goes on: its last key is the next chunk's first,
    // and it does not fill the chunk from one before)
    if (u == 0 && key[len].x == key[len + 1].x && (key[1].x != key[len].x || key[0].x != key[1].x))
        joins[atomicAdd(info + 1, 1)] = (int)c;
    if (u >= units) return;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    bool inside = key[0].x != key[1].x;  // the current run began in this chunk
    constexpr int U = 4;                 // rows whose loads are issued together
    for (int i0 = 0; i0 < len; i0 += U) {
        float x[U][8];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i0 + k < len) load8(dy + (int64_t)key[1 + i0 + k].y * H + 8 * u, x[k]);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + k;
            if (i >= len) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += x[k][e];
            const uint32_t t = key[1 + i].x;
            const bool ends = key[2 + i].x != t;
            if (ends && inside) {
                float* dst = dw + (int64_t)t * H + 8 * u;
                float o[8];
                if (accumulate) {
                    load8_wide(dst, o);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = fmaf(scale, acc[e], o[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = scale * acc[e];
                }
                store8_wide(dst, o);
            } else if (ends || i == len - 1) {
                // slot 0: a run from an earlier chunk; slot 1: one that goes on
                store8_wide(part + (2 * c + (inside ? 1 : 0)) * H + 8 * u, acc);
            }
            if (ends) {
                inside = true;
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = 0.f;
            }
        }
    }
}

// The listed runs (in any order: each is summed by itself) that begin in a chunk and
// go on past it: their parts, then dW.  Groups of threads take a contiguous share of
// the parts each and their sums are added in order (a frequent token has a part in
// every chunk of its run: 28 us at 32768 rows with one group).  Blocks as many as
// the SMs hold, not one a chunk, most of which would only look and return (32768
// rows of 1536, skewed: 101 us the whole, 98 so; of one token: 123, 110).
constexpr int kJoinGroups = 4;
__global__ void __launch_bounds__(1024) embed_join_kernel(
    const uint2* sorted, const int* info, int chunk, int H, float scale,
    const float* part, float* dw, int accumulate, const int* joins) {
    extern __shared__ __align__(16) float sums[];  // [groups - 1][H]
    tc::grid_dep_wait();
    const int n = info[0], n_joins = info[1];
    for (int at = blockIdx.x; at < n_joins; at += gridDim.x) {
        if (at != (int)blockIdx.x) __syncthreads();  // (the sums are read)
        const int64_t c = joins[at];
        const uint32_t t = sorted[(c + 1) * chunk].x;
        // chunks behind c whose first row belongs to the run (a prefix of them)
        int more = 0;
        for (int64_t q = c + 1;; q += blockDim.x) {
            const int64_t p = (q + threadIdx.x) * chunk;
            const int got = __syncthreads_count(p < n && sorted[p].x == t);
            more += got;
            if (got < (int)blockDim.x) break;
        }
        const int units = H / 8, groups = blockDim.x / units;
        const int g = threadIdx.x / units, u = threadIdx.x - g * units;
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        if (g < groups) {
            // parts 0 .. more: part 0 in slot 1 of chunk c, part k in slot 0 of chunk c + k
            const int k0 = (int)((int64_t)(more + 1) * g / groups);
            const int k1 = (int)((int64_t)(more + 1) * (g + 1) / groups);
#pragma unroll 4
            for (int k = k0; k < k1; ++k) {
                float x[8];
                load8_wide(part + (2 * (c + k) + (k == 0 ? 1 : 0)) * H + 8 * u, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += x[e];
            }
            if (g > 0) store8(sums + (g - 1) * H + 8 * u, acc);
        }
        __syncthreads();
        if (g != 0) continue;
        for (int k = 1; k < groups; ++k) {
            float x[8];
            load8(sums + (k - 1) * H + 8 * u, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += x[e];
        }
        float* dst = dw + (int64_t)t * H + 8 * u;
        float o[8];
        if (accumulate) load8_wide(dst, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = accumulate ? fmaf(scale, acc[e], o[e]) : scale * acc[e];
        store8_wide(dst, o);
    }
}

// The gradient of few rows in one launch (behind the zeros of a fresh dW): block m,
// if no live row before m has m's token, lists the rows that have it and sums them,
// groups of threads a contiguous share each.  A small call's time is its launches
// and their latency: 64 skewed rows of 1024 added take 6.2 us, 10.6 by the sort,
// and 21 us against 27 between two events around the call.  Up to 32 rows a group,
// so that a token's rows one after the other cost no more than the launches (128
// rows of one token, 2560 columns, 3 groups: 10.8 us against 12.4).
constexpr int kFewTokens = 128, kFewGroups = 8, kFewPerGroup = 32;
int few_groups(int H) {
    const int n = 1024 / (H / 8);
    return n > kFewGroups ? kFewGroups : n;
}
template <typename T>
__global__ void __launch_bounds__(kMaxH / 8) embed_few_kernel(
    const int32_t* __restrict__ tokens, const uint8_t* __restrict__ mask, int M, int64_t V, int H, float scale,
    const T* __restrict__ dy, float* dw, int accumulate, int groups) {
    extern __shared__ __align__(16) float sums[];  // [groups - 1][H]
    __shared__ int rows[kFewTokens];
    __shared__ int n_rows;
    const int m = blockIdx.x, lane = threadIdx.x;
    const int32_t t = tokens[m];
    if (lane < 32) {
        const bool on = t >= 0 && (int64_t)t < V && (mask == nullptr || mask[m] != 0);
        bool first = on;
        int n = 0;
        for (int j0 = 0; j0 < M; j0 += 32) {
            const int j = j0 + lane;
            const bool same = on && j < M && tokens[j] == t && (mask == nullptr || mask[j] != 0);
            if (__any_sync(0xffffffffu, same && j < m)) first = false;
            const uint32_t take = __ballot_sync(0xffffffffu, same && j >= m);
            if (take >> lane & 1u) rows[n + __popc(take & ((1u << lane) - 1u))] = j;
            n += __popc(take);
        }
        if (lane == 0) n_rows = first ? n : 0;
    }
    __syncthreads();
    tc::grid_dep_wait();  // (the zeros)
    const int n = n_rows;
    if (n == 0) return;
    const int g = threadIdx.x / (H / 8), u = threadIdx.x - g * (H / 8);
    const int end = g < groups ? n * (g + 1) / groups : 0;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    constexpr int U = 4;
    for (int i0 = n * g / groups; i0 < end; i0 += U) {
        float x[U][8];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i0 + k < end) load8(dy + (int64_t)rows[i0 + k] * H + 8 * u, x[k]);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i0 + k < end)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += x[k][e];
    }
    if (g > 0 && g < groups) store8(sums + (g - 1) * H + 8 * u, acc);
    __syncthreads();
    if (g != 0) return;
    for (int k = 1; k < groups; ++k) {
        float x[8];
        load8(sums + (k - 1) * H + 8 * u, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += x[e];
    }
    float* dst = dw + (int64_t)t * H + 8 * u;
    float o[8];
    if (accumulate) load8_wide(dst, o);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = accumulate ? fmaf(scale, acc[e], o[e]) : scale * acc[e];
    store8_wide(dst, o);
}

size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int unit_threads(int H) { return (H / 8 + 31) / 32 * 32; }

}  // namespace

// Rows a thread takes at once: 4 when there are blocks enough for every SM
// either way (8192 rows of 2560: 13.6 us with 1, 11.3 with 4), 1 for fewer, where
// a row's latency is the call's.
constexpr int64_t kEmbedWideM = 4096;

cudaError_t launch_embed(const uint32_t* wq, SbView sb, int64_t V, int H, int bits,
                         const int32_t* tokens, const uint8_t* mask, int64_t M, float scale,
                         void* out, int out_type, cudaStream_t st) {
    const int wide = out_type == kSbF32 && reinterpret_cast<uintptr_t>(out) % 32 == 0;
    if (M >= kEmbedWideM)
        embed_kernel<4><<<(unsigned)((M + 3) / 4), unit_threads(H), 0, st>>>(
            wq, sb, V, H, bits, tokens, mask, M, scale, out, out_type, wide);
    else
        embed_kernel<1><<<(unsigned)M, unit_threads(H), 0, st>>>(wq, sb, V, H, bits, tokens, mask, M,
                                                                 scale, out, out_type, wide);
    return cudaGetLastError();
}

EmbedBwdPlan plan_embed_bwd(int64_t M, int H) {
    EmbedBwdPlan p;
    // Shorter chunks while there are few (a block sums its rows one after the
    // other), longer ones while there are many (a run's parts are joined): 32768 x
    // 1536 rows take 105, 101 and 106 us with 16, 32 and 64, 131072 277, 251, 230.
    p.chunk = M <= 4096 ? 8 : M <= 16384 ? 16 : M <= 65536 ? 32 : kMaxChunk;
    p.n_chunks = (M + p.chunk - 1) / p.chunk;
    size_t off = 0;
    p.off_info = off; off = up(off + 16, 256);
    p.off_a = off;    off = up(off + 8 * (size_t)M, 256);
    p.off_b = off;    off = up(off + 8 * (size_t)M, 256);
    p.off_part = off; off = up(off + 2 * sizeof(float) * (size_t)p.n_chunks * H, 256);
    p.off_joins = off; off = up(off + 4 * (size_t)p.n_chunks, 256);
    p.total = off;
    return p;
}

template <typename T>
static cudaError_t launch_sum(const EmbedBwdPlan& p, const uint2* sorted, int* info, int H,
                              float scale, const void* dy, float* dw, int accumulate, float* part,
                              int* joins, cudaStream_t st) {
    int chunk = p.chunk;
    const T* y = static_cast<const T*>(dy);
    void* args[] = {&sorted, &info, &chunk, &H, &scale, &y, &dw, &accumulate, &part, &joins};
    return launch_dependent(reinterpret_cast<const void*>(embed_sum_kernel<T>), dim3((unsigned)p.n_chunks),
                            dim3(unit_threads(H)), 0, st, args);
}

template <typename T>
static cudaError_t launch_few(int64_t V, int H, const int32_t* tokens, const uint8_t* mask, int64_t M, float scale,
                              const void* dy, float* dw, bool accumulate, cudaStream_t st) {
    // (without zeros before it the kernel is launched in plain order: it reads the
    // tokens and the mask before it waits)
    const auto* y = static_cast<const T*>(dy);
    const int groups = few_groups(H);
    const dim3 block((unsigned)((groups * (H / 8) + 31) / 32 * 32));
    const int smem = (groups - 1) * H * (int)sizeof(float);
    if (!accumulate)
        return launch_after_smem(embed_few_kernel<T>, dim3((unsigned)M), block, smem, st, tokens, mask, (int)M, V, H,
                                 scale, y, dw, 0, groups);
    embed_few_kernel<T><<<(unsigned)M, block, smem, st>>>(tokens, mask, (int)M, V, H, scale, y, dw, 1, groups);
    return cudaGetLastError();
}

static cudaError_t launch_zero(float* dw, int64_t n32, bool beside, cudaStream_t st) {
    const int64_t per = kZeroThreads * kZeroUnroll;
    const dim3 grid((unsigned)((n32 + per - 1) / per));
    if (beside) return launch_after(embed_zero_kernel, grid, dim3(kZeroThreads), st, dw, n32);
    embed_zero_kernel<<<grid, kZeroThreads, 0, st>>>(dw, n32);
    return cudaGetLastError();
}

// sort -> (zeros beside it) -> sums -> joins, each launched as the dependent of
// the one before: it starts early and waits inside.
cudaError_t launch_embed_bwd(const EmbedBwdPlan& p, void* ws, int64_t V, int H,
                             const int32_t* tokens, const uint8_t* mask, int64_t M, float scale,
                             const void* dy, int dy_type, float* dw, bool accumulate,
                             cudaStream_t st) {
    char* w = static_cast<char*>(ws);
    int* info = reinterpret_cast<int*>(w + p.off_info);
    uint2* a = reinterpret_cast<uint2*>(w + p.off_a);
    uint2* b = reinterpret_cast<uint2*>(w + p.off_b);
    float* part = reinterpret_cast<float*>(w + p.off_part);
    int* joins = reinterpret_cast<int*>(w + p.off_joins);
    cudaError_t e;
    if (M <= kFewTokens && M <= kFewPerGroup * few_groups(H)) {
        if (!accumulate && (e = launch_zero(dw, V * H / 8, false, st))) return e;
        return dy_type == kSbF32    ? launch_few<float>(V, H, tokens, mask, M, scale, dy, dw, accumulate, st)
               : dy_type == kSbBf16 ? launch_few<__nv_bfloat16>(V, H, tokens, mask, M, scale, dy, dw, accumulate, st)
                                    : launch_few<__half>(V, H, tokens, mask, M, scale, dy, dw, accumulate, st);
    }
    const uint2* sorted;
    if (M <= kRankM) {
        const int smem = (int)(M + 3) / 4 * 16;
        // a row to each warp, as far as the SMs hold the blocks at once
        const int64_t blocks = (M + kRankThreads / 32 - 1) / (kRankThreads / 32);
        const int64_t most = 2 * (int64_t)device_sms();
        embed_rank_kernel<<<(unsigned)(blocks < most ? blocks : most), kRankThreads, smem, st>>>(
            tokens, mask, (int)M, V, a, info);
        if ((e = cudaGetLastError())) return e;
        sorted = a;
    } else {
        int nbits = 1;
        while (((int64_t)1 << nbits) < V) ++nbits;
        const int passes = (nbits + 8) / 9, width = (nbits + passes - 1) / passes;
        e = ensure_smem_limit(reinterpret_cast<const void*>(embed_sort_kernel), (int)sizeof(SortSmem));
        if (e) return e;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(kSortCluster);
        cfg.blockDim = dim3(kSortThreads);
        cfg.dynamicSmemBytes = sizeof(SortSmem);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kSortCluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, embed_sort_kernel, tokens, mask, M, V, passes, width, a, b, info);
        if (e) return e;
        sorted = passes & 1 ? a : b;
    }
    if (!accumulate && (e = launch_zero(dw, V * H / 8, true, st))) return e;
    int acc = accumulate ? 1 : 0;
    e = dy_type == kSbF32    ? launch_sum<float>(p, sorted, info, H, scale, dy, dw, acc, part, joins, st)
        : dy_type == kSbBf16 ? launch_sum<__nv_bfloat16>(p, sorted, info, H, scale, dy, dw, acc, part, joins, st)
                             : launch_sum<__half>(p, sorted, info, H, scale, dy, dw, acc, part, joins, st);
    if (e || p.n_chunks < 2) return e;
    int chunk = p.chunk, groups = 1024 / (H / 8);
    groups = groups < 1 ? 1 : groups > kJoinGroups ? kJoinGroups : groups;
    const int threads = (groups * (H / 8) + 31) / 32 * 32;
    void* args[] = {&sorted, &info, &chunk, &H, &scale, &part, &dw, &acc, &joins};
    const int64_t most = 2048 / threads * (int64_t)device_sms(), runs = p.n_chunks - 1;
    return launch_dependent(reinterpret_cast<const void*>(embed_join_kernel),
                            dim3((unsigned)(runs < most ? runs : most)), dim3(threads),
                            sizeof(float) * (size_t)(groups - 1) * H, st, args);
}

}  // namespace qh
