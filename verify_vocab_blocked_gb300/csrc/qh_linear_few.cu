// qh_linear_few.cu -- the matrix product of few rows (tokens).
//
// Its time is reading the weights once.  Their rows are the MMA's 128, the tokens its
// 16 to 128 columns, and the CTAs of a cluster share a tile's reduction, so that a small
// weight matrix is read by all SMs.  Each CTA finishes a share of the tokens: the others
// send it their sums by asynchronous stores into its shared memory, counted on its
// barrier, and it adds them in rank order (deterministic).  Reading them from there
// instead took 1 to 3 us more: a remote load waits for its way there and back, and the
// cluster had to stay until the last one.  What is sent moves at about 16 bytes a clock
// and SM, which keeps the splits of 64 and more tokens dear (64 x 2560 x 2560: 1.9 of 7.2
// us).  The weights K-major (the forward) or down their rows (dx = dz W).
//
// 5 x 2560 x 2560 bf16 from DRAM: 5.5 us a call in a graph, of which 2 are the bytes; the
// rest is the chain of launch, first loads, cluster barrier and the last stores.
// 5 x 2560 x 10240: 10.5 us, 5.0 TB/s; 128 x 10240 x 2560: 15.9.
#include "qh_linear_epi.cuh"

namespace qh {

namespace {

__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
        "r"(idesc), "r"(acc)
        : "memory");
}


// Epilogue warps: four, or two for a quadrant of the tensor memory's lanes where there are
// columns for both.  CTAs to an SM: its 512 columns of tensor memory hold the accumulators
// of them all (few_tmem), so that no CTA of a cluster waits for what another cluster holds.
constexpr int few_warps(int tile) { return tile <= 32 ? 4 : 8; }
constexpr int few_threads(int tile) { return 32 * (2 + few_warps(tile)); }
constexpr int few_per_sm(int tile) { return tile <= 16 ? 3 : 2; }

template <int T>
struct FewLayout {
    static constexpr int W_BYTES = 128 * kRowBytes;
    static constexpr int X_BYTES = T * kRowBytes;
    static constexpr int STAGE = W_BYTES + X_BYTES;
    static constexpr int NS = T == 32 ? 5 : T == 128 ? 3 : 4;
    static constexpr int OFF_BAR = NS * STAGE;
    static constexpr int BAR_BYTES = 8 * (2 * NS + 3) + 16;
    static constexpr int SMEM = OFF_BAR + BAR_BYTES + 1024;
    // The tokens in groups of G, a group's sums 16 (or 8) bytes a row; the share of a CTA of
    // `split` is every split-th group: split * ceil(NG / split) <= NG + 7 blocks of them.
    static constexpr int G = T <= 16 ? 2 : 4, NG = T / G;
    static_assert((NG + 7) * 128 * G * 4 <= OFF_BAR, "the parts of the share lie in the ring");
    static_assert(few_per_sm(T) * (SMEM + 1024) <= 228 * 1024, "CTAs to an SM");
    static_assert((few_per_sm(T) + 1) * (SMEM + 1024) > 228 * 1024 && few_per_sm(T) * few_tmem(T) <= 512,
                  "tensor memory for all that fit");
};

__device__ __forceinline__ void prefetch_l2(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// Four consecutive elements as they lie in memory (16 bits: two words), and widened.
__device__ __forceinline__ uint4 load4(const void* p, int64_t i, int type) {
    if (type == kSbF32) return *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __half*>(p) + i);  // (16 bits)
    return make_uint4(u.x, u.y, 0u, 0u);
}
__device__ __forceinline__ void add4(float (&v)[4], uint4 u, int type) {
    if (type == kSbF32) {
        v[0] += __uint_as_float(u.x), v[1] += __uint_as_float(u.y);
        v[2] += __uint_as_float(u.z), v[3] += __uint_as_float(u.w);
    } else if (type == kSbBf16) {
        v[0] += __uint_as_float(u.x << 16), v[1] += __uint_as_float(u.x & 0xffff0000u);
        v[2] += __uint_as_float(u.y << 16), v[3] += __uint_as_float(u.y & 0xffff0000u);
    } else {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
        v[0] += a.x, v[1] += a.y, v[2] += b.x, v[3] += b.y;
    }
}

// Stores into a CTA's shared memory, counted in bytes on its barrier.
__device__ __forceinline__ void st_async4(uint32_t to, uint32_t bar, const float* v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void st_async2(uint32_t to, uint32_t bar, const float* v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(to),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(bar)
                 : "memory");
}
// (load and wait in one: nothing reads the registers before)
__device__ __forceinline__ void tmem_ld_group(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_group(uint32_t addr, uint32_t (&r)[2]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(addr)
                 : "memory");
}
// Where a group's row r lies in its block: so that both 32 consecutive rows and every
// fourth one are read without bank conflicts.
__device__ __forceinline__ int slot(int r) { return r ^ (r >> 2 & 3) ^ (r >> 4 & 3) << 2; }

template <int ACT, int G>
__device__ __forceinline__ void activate_all(float (&v)[G][4]) {
#pragma unroll
    for (int u = 0; u < G; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[u][j] = activate(v[u][j], ACT);
    }
}

// The outputs of a CTA's share of the tokens (groups rank, rank + split, ...), a warp a
// group: a lane adds four columns' sums of all ranks, in order -- consecutive ones where
// the outputs' rows are aligned, else 32 apart.  parts: the share's blocks [rank][group],
// which `landed` waits for.
template <int T, typename Landed>
__device__ __forceinline__ void few_outputs(const Epi& e, uint32_t parts, int rank, int split, int warp, int64_t m0,
                                            int rows, int64_t n0, const float (&bs)[4], const float (&bias)[4],
                                            const Landed& landed) {
    using L = FewLayout<T>;
    constexpr int G = L::G, EW = few_warps(T);
    const int lane = threadIdx.x & 31;
    const bool vec = e.vec != 0;  // (then N is a multiple of 4)
    const int64_t n = n0 + (vec ? 4 * lane : lane);
    const int share = (L::NG + split - 1) / split;
    bool bad = false;
    for (int i = warp; (rank + split * i) * G < rows; i += EW) {
        const int t0 = (rank + split * i) * G;
        uint4 r[G];
        float as[G];
#pragma unroll
        for (int u = 0; u < G; ++u) {
            const bool in = t0 + u < rows && n < e.N;
            as[u] = e.a_scale && in ? e.a_scale[m0 + t0 + u] : 1.f;
            r[u] = make_uint4(0u, 0u, 0u, 0u);
            if (!e.res || !in) continue;
            const int64_t from = (m0 + t0 + u) * e.ldr + n;
            if (vec) {
                r[u] = load4(e.res, from, e.res_type);
            } else {
                r[u].x = __float_as_uint(sb_elem(e.res, from, e.res_type));
                if (n + 32 < e.N) r[u].y = __float_as_uint(sb_elem(e.res, from + 32, e.res_type));
                if (n + 64 < e.N) r[u].z = __float_as_uint(sb_elem(e.res, from + 64, e.res_type));
                if (n + 96 < e.N) r[u].w = __float_as_uint(sb_elem(e.res, from + 96, e.res_type));
            }
        }
        if (i == warp) bad = !landed();
        float v[G][4];
#pragma unroll 4
        for (int s = 0; s < split; ++s) {
            const uint32_t block = parts + (s * share + i) * (128 * G * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at = block + slot(vec ? 4 * lane + j : lane + 32 * j) * (4 * G);
                float x[G];
                if constexpr (G == 4)
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                                 : "r"(at));
                else
                    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "r"(at));
#pragma unroll
                for (int u = 0; u < G; ++u) v[u][j] = s == 0 ? x[u] : v[u][j] + x[u];
            }
        }
        if (bad) {
#pragma unroll
            for (int u = 0; u < G; ++u) v[u][0] = v[u][1] = v[u][2] = v[u][3] = __int_as_float(0x7fc00000);
        }
        const int live = n < e.N ? min(G, rows - t0) : 0;
        const int64_t at = (m0 + t0) * e.N + n;
#pragma unroll
        for (int u = 0; u < G; ++u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[u][j] = fmaf(v[u][j] * as[u], bs[j], bias[j]);
        }
        if (e.pre) {
#pragma unroll
            for (int u = 0; u < G; ++u) {
                __half h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = pre_of(v[u][j]);
                if (u >= live) continue;
                if (vec) {
                    *reinterpret_cast<uint2*>(e.pre + at + u * e.N) = *reinterpret_cast<const uint2*>(h);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + 32 * j < e.N) e.pre[at + u * e.N + 32 * j] = h[j];
                }
            }
        }
        switch (e.act) {
            case kActRelu: activate_all<kActRelu>(v); break;
            case kActSilu: activate_all<kActSilu>(v); break;
            case kActGelu: activate_all<kActGelu>(v); break;
            case kActGeluTanh: activate_all<kActGeluTanh>(v); break;
            default: break;
        }
        if (e.res) {
#pragma unroll
            for (int u = 0; u < G; ++u) add4(v[u], r[u], vec ? e.res_type : kSbF32);
        }
        if (!vec) {
#pragma unroll
            for (int u = 0; u < G; ++u) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (u < live && n + 32 * j < e.N) put(e.y, at + u * e.N + 32 * j, e.y_type, v[u][j]);
            }
        } else if (e.y_type == kSbF32) {
#pragma unroll
            for (int u = 0; u < G; ++u)
                if (u < live)
                    *reinterpret_cast<float4*>(static_cast<float*>(e.y) + at + u * e.N) =
                        make_float4(v[u][0], v[u][1], v[u][2], v[u][3]);
        } else {
#pragma unroll
            for (int u = 0; u < G; ++u)
                if (u < live)
                    *reinterpret_cast<uint2*>(static_cast<__half*>(e.y) + at + u * e.N) =  // (16 bits)
                        make_uint2(pack2(v[u][0], v[u][1], e.y_type), pack2(v[u][2], v[u][3], e.y_type));
        }
    }
}

// tw: the weights, whose rows (or, WMN, columns) are the tile's 128; tx: the tokens.
// blockIdx.x: 128-row tile and rank in the cluster of `split` (at most 8);
// blockIdx.y: token tile.  `sums`:
// the stages of an accumulator (a float32 output's reduction takes several, for the
// pairs' reason, added in registers at the end); `cols`: their columns.
template <int T, bool WMN>
__global__ void __launch_bounds__(few_threads(T), few_per_sm(T))
    linear_few_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
                      const __grid_constant__ Epi e, int n_k, int step_k, int split, int sums, int cols,
                      uint32_t idesc, int f8, int stall) {
    using L = FewLayout<T>;
    constexpr int NS = L::NS, EW = few_warps(T);
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint64_t* empty = full + NS;
    uint64_t* accf = empty + NS;
    uint64_t* mdrain = accf + 1;
    uint64_t* landed = mdrain + 1;  // the share's parts have
    uint32_t* tmem_base_sh = reinterpret_cast<uint32_t*>(landed + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_sh + 1);
    int* err = reinterpret_cast<int*>(tmem_base_sh + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)blockIdx.x % split;  // (= the rank in the cluster of `split`)
    const int n0 = (int)blockIdx.x / split * 128, m0 = (int)blockIdx.y * T;
    const int k0 = (int)((int64_t)n_k * rank / split), k1 = (int)((int64_t)n_k * (rank + 1) / split);
    const int rows = (int)min((int64_t)T, e.M - m0);
    const int groups = (rows + L::G - 1) / L::G, share = (L::NG + split - 1) / split;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        tc::mbar_init(accf, 1);
        tc::mbar_init(mdrain, 1);
        tc::mbar_init(landed, 1);
        *abort_flag = 0;
        *err = 0;
        tc::fence_mbar_init();
        // (groups of this rank x ranks x 128 rows; none: the arrival alone)
        tc::mbar_arrive_expect_tx(landed, (uint32_t)((groups - rank + split - 1) / split * split * (128 * L::G * 4)));
        tc::prefetch_tmap(&tw);
        tc::prefetch_tmap(&tx);
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_base_sh, cols);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem_base = *tmem_base_sh;
    // The ring's first tiles of the weights on their way into L2 while the kernel before ends
    // (a hint: what it may still write to them is written there, too).
    if (warp == 0 && stall == 0 && lane < NS && k0 + lane < k1) {
        const int k = (k0 + lane) * step_k;
        if constexpr (WMN) {
            prefetch_l2(&tw, n0, k);
            prefetch_l2(&tw, n0 + 64, k);
        } else {
            prefetch_l2(&tw, k, n0);
        }
    }
    tc::grid_dep_wait();
    tc::grid_dep_trigger();

    bool ok = true;
    float bs[4], bias[4];  // the scales and biases of a lane's columns
    if (warp == 0) {
        // (one thread's loops: the whole warp's with a lane elected for each stage's copies and
        // MMAs took 0.37 us a stage, so 0.23)
        if (elect_one()) {
            int stage = 0;
            uint32_t phase = 0, fills = 0;
            for (int kk = k0; kk < k1 && stall == 0; ++kk) {
                if (!tc::mbar_wait_cta(&empty[stage], phase ^ 1, abort_flag, err, tc::kErrTimeoutEmpty)) break;
                tc::mbar_arrive_expect_tx(&full[stage], L::STAGE);
                unsigned char* W = smem + stage * L::STAGE;
                if constexpr (WMN) {
                    tc::tma_load_2d(W, &tw, &full[stage], n0, kk * step_k);
                    tc::tma_load_2d(W + 8192, &tw, &full[stage], n0 + 64, kk * step_k);
                } else {
                    tc::tma_load_2d(W, &tw, &full[stage], kk * step_k, n0);
                }
                tc::tma_load_2d(W + L::W_BYTES, &tx, &full[stage], kk * step_k, m0);
                ++fills;
                if (++stage == NS) { stage = 0; phase ^= 1; }
            }
            tc::drain_ring(full, NS, fills, err);  // (every copy has landed, on any path)
        }
    } else if (warp == 1) {
        if (elect_one()) {
            int stage = 0, in = 0;
            uint32_t phase = 0, d = tmem_base;
            const uint64_t wd0 = operand_desc<WMN>(tc::smem_u32(smem));
            const uint64_t xd0 = operand_desc<false>(tc::smem_u32(smem + L::W_BYTES));
            for (int kk = k0; kk < k1; ++kk) {
                ok = tc::mbar_wait_cta(&full[stage], phase, abort_flag, err, tc::kErrTimeoutFull);
                if (!ok) break;
                tc::tc_fence_after();
                const uint64_t wd = wd0 + (uint32_t)(stage * (L::STAGE >> 4));
                const uint64_t xd = xd0 + (uint32_t)(stage * (L::STAGE >> 4));
                if (!WMN && f8) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) umma_f8(d, wd + 2 * s, xd + 2 * s, idesc, in | s);
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s) tc::umma_f16(d, wd + kStep<WMN> * s, xd + 2 * s, idesc, in | s);
                }
                tc::umma_commit(&empty[stage]);
                if (kk + 1 == k1) tc::umma_commit(accf);
                if (++stage == NS) { stage = 0; phase ^= 1; }
                if (++in == sums) in = 0, d += T;
            }
            if (!ok) {
                tc::umma_commit(mdrain);
                tc::mbar_drain(mdrain, 0, err);
            }
        }
    } else {
        // (their values are on their way while the accumulator fills)
        const bool vec = e.vec != 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = n0 + (vec ? 4 * lane + j : lane + 32 * j);
            bs[j] = e.b_scale && at < e.N ? e.b_scale[at] : 1.f;
            bias[j] = e.bias && at < e.N ? sb_elem(e.bias, at, e.bias_type) : 0.f;
        }
        ok = tc::mbar_wait_cta(accf, 0, abort_flag, err, tc::kErrTimeoutAccFull);
        tc::tc_fence_after();
    }
    // Every CTA's MMAs, and with them its copies, are done: the rings are free.
    __syncwarp();
    if (split > 1) tc::cluster_sync();
    if (warp >= 2) {
        // Lane: a weight row; the accumulator's columns: tokens, whose sums go to the CTA
        // that finishes them.
        const int sub = warp & 3, row = sub * 32 + lane;
        const int accs = (k1 - k0 + sums - 1) / sums;
        const uint32_t d = tmem_base + ((uint32_t)(sub * 32) << 16);
        const uint32_t parts = tc::smem_u32(smem) + rank * share * (128 * L::G * 4) + slot(row) * (4 * L::G);
        // Each CTA begins with its own share and goes on to the next CTA's: in one order for
        // all, they would all send to the same one at a time.  (EW / 4 warps a quadrant.)
        for (int o = 0; o < split; ++o) {
            const int owner = rank + o < split ? rank + o : rank + o - split;
            const uint32_t to = at_rank(parts, owner), bar = at_rank(tc::smem_u32(landed), owner);
#pragma unroll 2
            for (int i = (warp - 2) / 4; owner + split * i < groups; i += EW / 4) {
                float v[L::G];
                for (int a = 0; a < accs; ++a) {
                    uint32_t r[L::G];
                    tmem_ld_group(d + a * T + (owner + split * i) * L::G, r);
#pragma unroll
                    for (int j = 0; j < L::G; ++j)
                        v[j] = !ok ? __int_as_float(0x7fc00000) : a == 0 ? __uint_as_float(r[j]) : v[j] + __uint_as_float(r[j]);
                }
                if constexpr (L::G == 4) st_async4(to + i * (128 * L::G * 4), bar, v);
                else st_async2(to + i * (128 * L::G * 4), bar, v);
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem_base, cols);
    }
    if (warp >= 2) {
        // (past the cluster's barrier every CTA sends without a wait: the parts do land, and
        // none is under way to a CTA that has left)
        few_outputs<T>(e, tc::smem_u32(smem), rank, split, warp - 2, m0, rows, n0, bs, bias, [&]() {
            const bool all = tc::mbar_wait_cluster(landed, 0, abort_flag, err, tc::kErrTimeoutFull);
            if (!all) tc::mbar_drain(landed, 0, err);
            return all && ok;
        });
    }
}

template <int T, bool WMN>
cudaError_t go_few(const LinArgs& a, int split, cudaStream_t st) {
    using L = FewLayout<T>;
    CUtensorMap tw, tx;
    if (!map_operand(&tw, a.b, a.type, a.N, a.K, 128) || !map_operand(&tx, a.a, a.type, a.M, a.K, T))
        return cudaErrorInvalidValue;
    int step;
    const int n_k = steps(a, &step);
    const int share = (n_k + split - 1) / split, accs = few_accs(a, share);
    if (accs * T > few_tmem(T)) return cudaErrorInvalidValue;  // (no such plan)
    const int sums = (share + accs - 1) / accs;
    int cols = 32;
    while (cols < accs * T) cols *= 2;
    const dim3 grid((unsigned)((a.N + 127) / 128 * split), (unsigned)((a.M + T - 1) / T));
    return launch_cluster(linear_few_kernel<T, WMN>, grid, few_threads(T), L::SMEM, split, st, tw, tx,
                          epi_of(a), n_k, step, split, sums, cols, idesc_of(a.type, 128, T, WMN, false),
                          (int)(a.type == kE4m3), a.stall);
}

template <bool WMN>
cudaError_t pick_few(const LinArgs& a, const LinPlan& p, cudaStream_t st) {
    switch (p.tile) {
        case 16: return go_few<16, WMN>(a, p.split, st);
        case 32: return go_few<32, WMN>(a, p.split, st);
        case 64: return go_few<64, WMN>(a, p.split, st);
        default: return go_few<128, WMN>(a, p.split, st);
    }
}

}  // namespace

cudaError_t launch_linear_few(const LinArgs& a, const LinPlan& p, cudaStream_t st) {
    return a.b.k_major ? pick_few<false>(a, p, st) : pick_few<true>(a, p, st);
}

}  // namespace qh
