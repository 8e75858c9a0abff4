// qh_linear.cu -- matrix product with bias, activation and residual in its
// epilogue, on the fifth-generation tensor cores.
//
//     D[m, n] = sum_k A[m, k] B[n, k]
//     z = D a_scale[m] b_scale[n] + bias[n];   y = act(z) + res[m, n]
//
// A and B are bf16, fp16 or (K-major only) e4m3, fp32 accumulate; both may be
// K-major (the forward) or MN-major (the gradients: dx = dz W takes W down its
// rows, dW = dz^T x both operands).  Everything after the product is fp32 and
// rounded once.
//
// Two kernels:
//   * pairs: CTA pairs (cta_group::2), 256 x BN output tiles, persistent; one
//     thread streams both operands' 128-byte-swizzled tiles by TMA, one issues the
//     MMAs into two accumulators in turn, sixteen warps run the epilogue of one
//     while the other fills, the residual and the outputs going through shared
//     memory by TMA (8192 x 2560 x 10240 bf16: 226 us, 1 900 TFLOP/s; with K = 512, whose
//     tiles last as long as their epilogue, 59, with silu, residual and pre 127);
//   * few (qh_linear_few.cu): for up to 512 rows of A.
//
// A bounded wait that expires makes the tile NaN.
#include "qh_linear_epi.cuh"

namespace qh {

namespace {

constexpr uint16_t kPairMask = 0x3;

// What a pair walks: `full` whole tiles, then the others' parts, `split` of the
// reduction each (one after another), whose sums go to part[item - full].
struct Walk {
    int full, items, split;
    float* part;
};
__device__ __forceinline__ void item_of(const Walk& w, int i, int n_k, int& tile, int& k0, int& k1) {
    tile = i, k0 = 0, k1 = n_k;
    if (i < w.full) return;
    const int j = i - w.full, s = j % w.split;
    tile = w.full + j / w.split;
    k0 = (int)((int64_t)n_k * s / w.split);
    k1 = (int)((int64_t)n_k * (s + 1) / w.split);
}

template <int ACT>
__device__ __forceinline__ void activate32(float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = activate(v[j], ACT);
}

// One column's scale, and its bias as it lies in memory (a conversion at the load would
// wait for it); 1 and 0 where there is none.
struct Column {
    float scale;
    uint32_t bias;
    __device__ __forceinline__ void load(const Epi& e, int64_t n) {
        scale = e.b_scale && n < e.N ? e.b_scale[n] : 1.f;
        bias = 0u;
        if (!e.bias || n >= e.N) return;
        if (e.bias_type == kSbF32) bias = static_cast<const uint32_t*>(e.bias)[n];
        else bias = static_cast<const unsigned short*>(e.bias)[n];
    }
    __device__ __forceinline__ float bias_of(int type) const {
        if (type == kSbF32) return __uint_as_float(bias);
        return type == kSbBf16 ? __uint_as_float(bias << 16) : __half2float(__ushort_as_half((unsigned short)bias));
    }
};

__device__ __forceinline__ void activate32(float (&v)[32], int act) {
    switch (act) {
        case kActRelu: activate32<kActRelu>(v); break;
        case kActSilu: activate32<kActSilu>(v); break;
        case kActGelu: activate32<kActGelu>(v); break;
        case kActGeluTanh: activate32<kActGeluTanh>(v); break;
        default: break;
    }
}

// A warp's 32 rows x 64 bytes in shared memory as TMA lays them with the 64-byte
// swizzle: 32 columns of a 16-bit type or 16 of float32.  The address of row r's
// 16-byte piece q.
__device__ __forceinline__ uint32_t piece(uint32_t base, int r, int q) { return base + 64 * r + 16 * (q ^ (r >> 1 & 3)); }

__device__ __forceinline__ void sts128(uint32_t p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}

// v, or 16 of its values from `from` on as float32, to or from row r of such a tile.
__device__ __forceinline__ void put_half(uint32_t base, int r, const float (&v)[32], int type) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        sts128(piece(base, r, q), pack2(v[8 * q], v[8 * q + 1], type), pack2(v[8 * q + 2], v[8 * q + 3], type),
               pack2(v[8 * q + 4], v[8 * q + 5], type), pack2(v[8 * q + 6], v[8 * q + 7], type));
}
template <int FROM>
__device__ __forceinline__ void put_float(uint32_t base, int r, const float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        sts128(piece(base, r, q), __float_as_uint(v[FROM + 4 * q]), __float_as_uint(v[FROM + 4 * q + 1]),
               __float_as_uint(v[FROM + 4 * q + 2]), __float_as_uint(v[FROM + 4 * q + 3]));
}
template <int FROM>
__device__ __forceinline__ void add_float(uint32_t base, int r, float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 u = lds128(piece(base, r, q));
        v[FROM + 4 * q] += __uint_as_float(u.x), v[FROM + 4 * q + 1] += __uint_as_float(u.y);
        v[FROM + 4 * q + 2] += __uint_as_float(u.z), v[FROM + 4 * q + 3] += __uint_as_float(u.w);
    }
}
__device__ __forceinline__ void add_half(uint32_t base, int r, float (&v)[32], int type) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 u = lds128(piece(base, r, q));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 f;
            if (type == kSbBf16) f = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
            else f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            v[8 * q + 2 * j] += f.x;
            v[8 * q + 2 * j + 1] += f.y;
        }
    }
}

// z of row m and a thread's 32 consecutive columns, whose scales and biases the warp's
// lanes hold: through 256 bytes of shared memory.
__device__ __forceinline__ void scale32(const Epi& e, int64_t m, const Column& column, uint32_t sh, float (&v)[32]) {
    if (!e.bias && !e.b_scale) return;
    const int lane = threadIdx.x & 31;
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(sh + 4 * lane), "f"(column.scale) : "memory");
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(sh + 128 + 4 * lane), "f"(column.bias_of(e.bias_type)) : "memory");
    __syncwarp();
    if (e.b_scale) {
        const float as = m < e.M ? e.a_scale[m] : 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint4 u = lds128(sh + 16 * q);
            v[4 * q] *= as * __uint_as_float(u.x), v[4 * q + 1] *= as * __uint_as_float(u.y);
            v[4 * q + 2] *= as * __uint_as_float(u.z), v[4 * q + 3] *= as * __uint_as_float(u.w);
        }
    }
    if (e.bias) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint4 u = lds128(sh + 128 + 16 * q);
            v[4 * q] += __uint_as_float(u.x), v[4 * q + 1] += __uint_as_float(u.y);
            v[4 * q + 2] += __uint_as_float(u.z), v[4 * q + 3] += __uint_as_float(u.w);
        }
    }
    __syncwarp();
}

// A tile of a warp back to global memory: the warp's writes made visible to the copy,
// which one thread starts (rows and columns outside the matrix are not written), and
// the wait until such copies have read their tiles.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void tma_stores_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

constexpr int kEpiWarps = 16;
constexpr int kPairThreads = 32 * (2 + kEpiWarps);

template <int BN, bool AMN, bool BMN>
struct PairLayout {
    static constexpr int A_BYTES = 128 * kRowBytes;      // this CTA's 128 rows of A
    static constexpr int B_BYTES = BN / 2 * kRowBytes;   // and its half of B's columns
    static constexpr int STAGE = A_BYTES + B_BYTES;
    // 5 stages of 256 columns: 66 us at 8192 x 2560 x 2560, 71 with 4, 81 with 3
    static constexpr int NS = BN == 256 ? 5 : 6;
    static constexpr int OFF_E = NS * STAGE;             // an epilogue warp's tiles: residual, output
    static constexpr int E_TILE = 32 * 64, E_BYTES = 2 * E_TILE;
    static constexpr int OFF_BAR = OFF_E + kEpiWarps * E_BYTES;
    static constexpr int BAR_BYTES = 8 * (2 * NS + 5 + kEpiWarps) + 16;
    static constexpr int SMEM = OFF_BAR + BAR_BYTES + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// The tiles in groups of 8 rows of tiles, columns outer: what the pairs work on at
// a time is near-square, so that each operand's tiles are shared in L2.
__device__ __forceinline__ void tile_of(int t, int n_mt, int n_nt, int& mt, int& nt) {
    constexpr int G = 8;
    const int per = G * n_nt, g = t / per, in = t - g * per;
    const int rows = min(G, n_mt - g * G);
    nt = in / rows;
    mt = g * G + in - nt * rows;
}

__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void umma_f8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
        "r"(idesc), "r"(acc)
        : "memory");
}

// tc::tmem_wait_ld for a load issued earlier, whose registers nothing may read before.
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld_of8(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

// SUMS: for float32 outputs.  The tensor cores' accumulation truncates, up to a step of
// the running sum at each MMA; sum_steps stages are summed there, and these sums in
// registers, rounded to nearest.  (What is lost depends on the operands -- a product whose
// sums fp32 holds loses nothing -- so that no factor on the result could make up for it.)
// Error over the result's norm at K = 2560, operands of both signs and positive ones,
// bf16: 4.7e-7 and 8.5e-7 so, 9.2e-7 and 1.9e-6 with 16 stages, 2.4e-7 and 3.6e-7 with 4,
// an fp32 product 4.5e-7 and 6.4e-7; fp16, whose products have more bits to lose: 6.5e-7
// and 2.7e-6; e4m3, K = 10240: 2.1e-7 and 1.1e-6, in one sum 6.5e-7 and 5.0e-6.
// 8192 x 2560 x 10240 bf16: 278, 266 and 326 us (with 4 the epilogue sets the pace).
template <int BN, bool AMN, bool BMN, bool SUMS>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                       const __grid_constant__ CUtensorMap ty, const __grid_constant__ CUtensorMap tp,
                       const __grid_constant__ CUtensorMap tr,
                       const __grid_constant__ Epi e, const Walk walk, int n_k, int step_k, uint32_t idesc, int f8,
                       int stall) {
    using L = PairLayout<BN, AMN, BMN>;
    constexpr int NS = L::NS;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint64_t* empty = full + NS;
    uint64_t* accf = empty + NS;
    uint64_t* acce = accf + 2;
    uint64_t* mdrain = acce + 2;
    uint64_t* resf = mdrain + 1;   // an epilogue warp's residual tile has landed
    uint32_t* tmem_base_sh = reinterpret_cast<uint32_t*>(resf + kEpiWarps);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_sh + 1);
    int* err = reinterpret_cast<int*>(tmem_base_sh + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_ctarank();
    const int n_mt = (int)((e.M + 255) / 256), n_nt = (int)((e.N + BN - 1) / BN);
    const int first = (int)tc::cluster_id_x(), stride = (int)tc::nclusters_x();
    const int sum = sum_steps(f8 != 0);  // (of SUMS)

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&accf[i], 1);
            tc::mbar_init(&acce[i], 2 * kEpiWarps);
        }
        tc::mbar_init(mdrain, 1);
        for (int i = 0; i < kEpiWarps; ++i) tc::mbar_init(&resf[i], 1);
        *abort_flag = 0;
        *err = 0;
        tc::fence_mbar_init();
        tc::prefetch_tmap(&ta);
        tc::prefetch_tmap(&tb);
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tmem_base_sh, 2 * BN);
        tc::tmem_relinquish_pair();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem_base = *tmem_base_sh;
    tc::grid_dep_wait();

    if (warp == 0) {
        uint32_t fills = 0;
        bool ok = stall == 0;
        const uint32_t full_lead = tc::mapa_shared(full, 0);
        const bool leads = elect_one();
        if (leads) {
            int stage = 0;
            uint32_t phase = 0;
            for (int i = first; i < walk.items && ok; i += stride) {
                int t, mt, nt, k0, k1;
                item_of(walk, i, n_k, t, k0, k1);
                tile_of(t, n_mt, n_nt, mt, nt);
                const int m0 = mt * 256 + (int)rank * 128, n0 = nt * BN + (int)rank * (BN / 2);
                for (int kk = k0; kk < k1; ++kk) {
                    ok = tc::mbar_wait_cta(&empty[stage], phase ^ 1, abort_flag, err, tc::kErrTimeoutEmpty);
                    if (!ok) break;
                    // both CTAs' copies count on the even CTA's barrier
                    if (rank == 0) tc::mbar_arrive_expect_tx(&full[stage], 2 * L::STAGE);
                    unsigned char* A = smem + stage * L::STAGE;
                    unsigned char* B = A + L::A_BYTES;
                    const uint32_t bar = full_lead + 8 * stage;
                    const int k = kk * step_k;
                    if constexpr (AMN) {
                        tma_load_pair(A, &ta, bar, m0, k);
                        tma_load_pair(A + 8192, &ta, bar, m0 + 64, k);
                    } else {
                        tma_load_pair(A, &ta, bar, k, m0);
                    }
                    if constexpr (BMN) {
#pragma unroll
                        for (int q = 0; q < BN / 128; ++q) tma_load_pair(B + q * 8192, &tb, bar, n0 + 64 * q, k);
                    } else {
                        tma_load_pair(B, &tb, bar, k, n0);
                    }
                    ++fills;
                    if (++stage == NS) { stage = 0; phase ^= 1; }
                }
            }
        }
        __syncwarp();
        tc::grid_dep_trigger();  // (earlier, the next kernel's blocks would crowd some SMs)
        if (leads) {
            // The last stages are consumed (their commits reach both CTAs) before the CTA exits.
            for (uint32_t i = fills > NS ? fills - NS : 0; i < fills && ok; ++i)
                ok = tc::mbar_wait_cta(&empty[i % NS], (i / NS) & 1, abort_flag, err, tc::kErrTimeoutEmpty);
            // And on any path every copy has landed: the even CTA's barriers count both CTAs'.
            if (rank == 0) tc::drain_ring(full, NS, fills, err);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, aphase = 0;
            const uint64_t ad0 = operand_desc<AMN>(tc::smem_u32(smem));
            const uint64_t bd0 = operand_desc<BMN>(tc::smem_u32(smem + L::A_BYTES));
            bool ok = true;
            for (int i = first; i < walk.items && ok; i += stride) {
                int t, k0, k1;
                item_of(walk, i, n_k, t, k0, k1);
                for (int kk = k0; kk < k1; ++kk) {
                    const bool begins = kk == k0 || (SUMS && ((kk - k0) & (sum - 1)) == 0);
                    if (begins) {
                        ok = tc::mbar_wait_cluster(&acce[buf], aphase ^ 1, abort_flag, err, tc::kErrTimeoutAccEmpty);
                        if (!ok) break;
                        tc::tc_fence_after();
                    }
                    ok = tc::mbar_wait_cta(&full[stage], phase, abort_flag, err, tc::kErrTimeoutFull);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint32_t d = tmem_base + buf * BN;
                    const uint64_t ad = ad0 + (uint32_t)(stage * (L::STAGE >> 4));
                    const uint64_t bd = bd0 + (uint32_t)(stage * (L::STAGE >> 4));
                    const bool ends = kk + 1 == k1 || (SUMS && ((kk + 1 - k0) & (sum - 1)) == 0);
                    if (!AMN && !BMN && f8) {
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            umma_f8_pair(d, ad + 2 * s, bd + 2 * s, idesc, !begins || s != 0);
                    } else {
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            tc::umma_f16_pair(d, ad + kStep<AMN> * s, bd + kStep<BMN> * s, idesc, !begins || s != 0);
                    }
                    tc::umma_commit_pair(&empty[stage], kPairMask);
                    if (ends) tc::umma_commit_pair(&accf[buf], kPairMask);
                    if (++stage == NS) { stage = 0; phase ^= 1; }
                    if (ends && ++buf == 2) { buf = 0; aphase ^= 1; }
                }
            }
            if (!ok) {
                tc::umma_commit_pair(mdrain, 0x1);
                tc::mbar_drain(mdrain, 0, err);
            }
        }
    } else {
        // A warp's 32 accumulator rows (its quadrant of the lanes) and COLS columns, 32 at a
        // time: a row a lane.
        constexpr int COLS = BN * 4 / kEpiWarps, NC = COLS / 32;
        const int sub = warp & 3, group = (warp - 2) >> 2;
        const uint32_t acce_lead = tc::mapa_shared(acce, 0);
        unsigned char* tiles = smem + L::OFF_E + (warp - 2) * L::E_BYTES;
        const uint32_t res_tile = tc::smem_u32(tiles), out_tile = res_tile + L::E_TILE;
        uint64_t* resb = &resf[warp - 2];
        const float nan = __int_as_float(0x7fc00000);
        int buf = 0;
        uint32_t aphase = 0;
        // The residual's tiles in the order of their use, asked for by lane 0 one ahead, once
        // the warp has read the one before.
        const bool by_tma = e.vec != 0;
        const int res_cols = e.res_type == kSbF32 ? 16 : 32;
        int ask_i = first, ask_at = 0;
        const auto ask = [&]() {
            if (!by_tma || !e.res || lane != 0) return;
            for (; ask_i < walk.full; ask_i += stride, ask_at = 0) {
                int mt, nt;
                tile_of(ask_i, n_mt, n_nt, mt, nt);
                const int m = mt * 256 + (int)rank * 128 + sub * 32, n = nt * BN + group * COLS + ask_at;
                if (m < e.M && n < e.N && ask_at < COLS) {
                    tc::mbar_arrive_expect_tx(resb, L::E_TILE);
                    tc::tma_load_2d(tiles, &tr, resb, n, m);
                    ask_at += res_cols;
                    return;
                }
            }
        };
        // (an item's tiles into L2 while the one before is worked on: from DRAM, one tile ahead
        // does not cover the latency)
        const auto ask_l2 = [&](int i) {
            if (!by_tma || !e.res || lane * res_cols >= COLS || i >= walk.full) return;
            int mt, nt;
            tile_of(i, n_mt, n_nt, mt, nt);
            const int m = mt * 256 + (int)rank * 128 + sub * 32, n = nt * BN + group * COLS + res_cols * lane;
            if (m < e.M && n < e.N)
                asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(
                                 reinterpret_cast<uint64_t>(&tr)),
                             "r"(n), "r"(m)
                             : "memory");
        };
        ask_l2(first);
        ask();
        uint32_t rphase = 0;
        for (int i = first; i < walk.items; i += stride) {
            int t, mt, nt, k0, k1;
            item_of(walk, i, n_k, t, k0, k1);
            tile_of(t, n_mt, n_nt, mt, nt);
            const int64_t m0 = (int64_t)mt * 256 + rank * 128 + sub * 32;
            const int64_t n0 = (int64_t)nt * BN + group * COLS;
            float* part = i < walk.full ? nullptr
                                        : walk.part + (int64_t)(i - walk.full) * 256 * BN +
                                              (rank * 128 + sub * 32 + lane) * BN + group * COLS;
            const int rows = (int)min((int64_t)32, e.M - m0);  // (<= 0: none)
            const uint32_t d0 = tmem_base + ((uint32_t)(sub * 32) << 16) + group * COLS;
            ask_l2(i + stride);
            Column column;  // (of the next 32)
            column.load(e, n0 + lane);
            // The sums v of the columns' c-th 32.
            const auto out = [&](int c, float (&v)[32]) {
                const int64_t n = n0 + 32 * c;
                if (part) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tc::st_global_v8(part + 32 * c + 8 * q, reinterpret_cast<const uint32_t*>(v + 8 * q));
                    return;
                }
                if (rows <= 0 || n >= e.N) return;
                const Column col = column;
                if (c + 1 < NC) column.load(e, n + 32 + lane);
                if (!by_tma) {
                    // any alignment: through shared memory to rows of 32 lanes
                    scale32(e, m0 + lane, col, res_tile, v);
                    float* tr = reinterpret_cast<float*>(tiles);  // [row][column ^ row]
                    const int64_t at = m0 * e.N + n + lane;
                    const int live = n + lane < e.N ? rows : 0;
                    if (e.pre) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) tr[lane * 32 + (j ^ lane)] = in_half(v[j]);
                        __syncwarp();
#pragma unroll 8
                        for (int k = 0; k < live; ++k) e.pre[at + k * e.N] = __float2half_rn(tr[k * 32 + (lane ^ k)]);
                        __syncwarp();
                    }
                    activate32(v, e.act);
#pragma unroll
                    for (int j = 0; j < 32; ++j) tr[lane * 32 + (j ^ lane)] = v[j];
                    __syncwarp();
                    if (e.res) {
                        const int64_t from = m0 * e.ldr + n + lane;
#pragma unroll 8
                        for (int k = 0; k < live; ++k)
                            tr[k * 32 + (lane ^ k)] += sb_elem(e.res, from + k * e.ldr, e.res_type);
                    }
                    if (e.y_type == kSbF32) {
#pragma unroll 8
                        for (int k = 0; k < live; ++k) static_cast<float*>(e.y)[at + k * e.N] = tr[k * 32 + (lane ^ k)];
                    } else {
#pragma unroll 8
                        for (int k = 0; k < live; ++k) put(e.y, at + k * e.N, e.y_type, tr[k * 32 + (lane ^ k)]);
                    }
                    __syncwarp();
                    return;
                }
                // The warp's tile at `tile`, written before, to columns `at` on; and the wait
                // until the tiles sent have been read.
                const auto send = [&](const CUtensorMap* map, uint32_t tile, int64_t at) {
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tma_store(map, tile, (int)at, (int)m0);
                };
                const auto sent = [&]() {
                    if (lane == 0) tma_stores_read<0>();
                    __syncwarp();
                };
                sent();
                scale32(e, m0 + lane, col, out_tile, v);
                if (e.pre) {
                    float z[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) z[j] = in_half(v[j]);
                    put_half(out_tile, lane, z, kSbF16);
                    send(&tp, out_tile, n);
                }
                activate32(v, e.act);
                if (e.res) {
                    // (a failed wait: the copy is waited for all the same, and the outputs say so)
                    const auto landed = [&]() {
                        const bool ok = tc::mbar_wait_cta(resb, rphase, abort_flag, err, tc::kErrTimeoutFull);
                        if (!ok) tc::mbar_drain(resb, rphase, err);
                        rphase ^= 1;
                        return ok;
                    };
                    bool ok = landed();
                    if (e.res_type == kSbF32) {
                        add_float<0>(res_tile, lane, v);
                        __syncwarp();
                        ask();
                        if (n + 16 < e.N) {
                            ok &= landed();
                            add_float<16>(res_tile, lane, v);
                            __syncwarp();
                            ask();
                        }
                    } else {
                        add_half(res_tile, lane, v, e.res_type);
                        __syncwarp();
                        ask();
                    }
                    if (!ok) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = nan;
                    }
                }
                if (e.pre) sent();
                if (e.y_type == kSbF32) {
                    put_float<0>(out_tile, lane, v);
                    send(&ty, out_tile, n);
                    if (n + 16 < e.N) {
                        // (without a residual its tile is free)
                        if (e.res) sent();
                        put_float<16>(e.res ? out_tile : res_tile, lane, v);
                        send(&ty, e.res ? out_tile : res_tile, n + 16);
                    }
                } else {
                    put_half(out_tile, lane, v, e.y_type);
                    send(&ty, out_tile, n);
                }
            };
            // The accumulator has been read.  (Nothing in memory is handed over: a release would
            // wait for the warp's stores; 256 rows' dW of 2560 x 10240 took 36 us, 27 so.)
            const auto release = [&](int k) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster_relaxed(acce_lead + 8 * k);
            };
            if constexpr (!SUMS) {
                const bool ok = tc::mbar_wait_cta(&accf[buf], aphase, abort_flag, err, tc::kErrTimeoutAccFull);
                tc::tc_fence_after();
                const uint32_t d = d0 + buf * BN;
#pragma unroll 1
                for (int c = 0; c < NC; ++c) {
                    uint32_t r[32];
                    tc::tmem_ld32(d + 32 * c, r);
                    tmem_wait_ld_of(r);
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                    if (!ok) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = nan;
                    }
                    if (c + 1 == NC) release(buf);
                    out(c, v);
                }
                if (++buf == 2) { buf = 0; aphase ^= 1; }
            } else {
                float v[NC][32];
                for (int kk = k0; kk < k1; kk += sum) {
                    const bool ok = tc::mbar_wait_cta(&accf[buf], aphase, abort_flag, err, tc::kErrTimeoutAccFull);
                    tc::tc_fence_after();
#pragma unroll
                    for (int c = 0; c < 4 * NC; ++c) {
                        uint32_t r[8];
                        tmem_ld8(d0 + buf * BN + 8 * c, r);
                        tmem_wait_ld_of8(r);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float x = ok ? __uint_as_float(r[j]) : nan;
                            float& to = v[c / 4][8 * (c % 4) + j];
                            to = kk == k0 ? x : to + x;
                        }
                    }
                    release(buf);
                    if (++buf == 2) { buf = 0; aphase ^= 1; }
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) out(c, v[c]);
            }
        }
        if (lane == 0) tma_stores_done();
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem_base, 2 * BN);
    }
}

// The tiles whose reduction was shared: their parts' sums added in order, and the
// epilogue.  BN / 8 lanes a row of a tile, 8 columns each -- consecutive ones where the
// rows of the outputs are aligned, else BN / 8 apart; blockIdx.y: tile.
constexpr int kJoinThreads = 256;
template <int BN>
__global__ void __launch_bounds__(kJoinThreads) linear_join_kernel(const __grid_constant__ Epi e, const Walk walk) {
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    constexpr int kLanes = BN / 8, kRows = kJoinThreads / kLanes;
    const int n_mt = (int)((e.M + 255) / 256), n_nt = (int)((e.N + BN - 1) / BN);
    int mt, nt;
    tile_of(walk.full + blockIdx.y, n_mt, n_nt, mt, nt);
    const int row = blockIdx.x * kRows + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int64_t m = (int64_t)mt * 256 + row, n0 = (int64_t)nt * BN;
    if (m >= e.M) return;
    const float* p = walk.part + (int64_t)blockIdx.y * walk.split * 256 * BN + row * BN;
    if (!e.vec || n0 + BN > e.N) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = p[lane + kLanes * j];
#pragma unroll 2
        for (int s = 1; s < walk.split; ++s) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += p[(int64_t)s * 256 * BN + lane + kLanes * j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t n = n0 + lane + kLanes * j;
            if (n < e.N)
                finish(e, m, n, v[j], e.b_scale ? e.b_scale[n] : 1.f,
                       e.bias ? sb_elem(e.bias, n, e.bias_type) : 0.f);
        }
        return;
    }
    const int64_t n = n0 + 8 * lane;
    float v[8], r[8], u[8];
    load8_wide(p + 8 * lane, v);
    if (e.res) load8_as(e.res, m * e.ldr + n, e.res_type, r);
#pragma unroll 4
    for (int s = 1; s < walk.split; ++s) {
        load8_wide(p + (int64_t)s * 256 * BN + 8 * lane, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += u[j];
    }
    const float as = e.a_scale ? e.a_scale[m] : 1.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = fmaf(v[j] * as, e.b_scale ? e.b_scale[n + j] : 1.f, e.bias ? sb_elem(e.bias, n + j, e.bias_type) : 0.f);
    if (e.pre) {
        __half h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = pre_of(v[j]);
        *reinterpret_cast<uint4*>(e.pre + m * e.N + n) = *reinterpret_cast<const uint4*>(h);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = activate(v[j], e.act);
    if (e.res) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
    store8_as(e.y, m * e.N + n, e.y_type, v);
}

// -------------------------------------------------------------------- host

// The map of an output's or the residual's 32 x 32 tiles (not made where there is none).
bool map_tile(CUtensorMap* map, const void* p, int type, int64_t ld, const LinArgs& a, bool vec) {
    return !p || !vec ||
           tmap_tiles(map, p, type_bytes(type), (uint64_t)a.N, (uint64_t)a.M, (uint64_t)ld * type_bytes(type));
}

template <int BN, bool AMN, bool BMN, bool SUMS>
cudaError_t go_pair(const LinArgs& a, const LinPlan& p, cudaStream_t st) {
    using L = PairLayout<BN, AMN, BMN>;
    CUtensorMap ta, tb;
    if (!map_operand(&ta, a.a, a.type, a.M, a.K, 128) || !map_operand(&tb, a.b, a.type, a.N, a.K, BN / 2))
        return cudaErrorInvalidValue;
    int step;
    const int n_k = steps(a, &step);
    const int tiles = (int)((a.M + 255) / 256 * ((a.N + BN - 1) / BN));
    const int full = p.split > 1 ? tiles / p.pairs * p.pairs : tiles;
    const Walk walk{full, full + (tiles - full) * p.split, p.split, a.part};
    const int pairs = std::min(walk.items, p.pairs);
    const Epi e = epi_of(a);
    CUtensorMap ty{}, tp{}, tr{};
    if (!map_tile(&ty, a.y, a.y_type, a.N, a, e.vec) || !map_tile(&tp, a.pre, kSbF16, a.N, a, e.vec) ||
        !map_tile(&tr, a.res, a.res_type, a.ldr, a, e.vec))
        return cudaErrorInvalidValue;
    if (cudaError_t err = launch_cluster(linear_pair_kernel<BN, AMN, BMN, SUMS>, dim3((unsigned)(2 * pairs)),
                                         kPairThreads, L::SMEM, 2, st, ta, tb, ty, tp, tr, e, walk, n_k, step,
                                         idesc_of(a.type, 256, BN, AMN, BMN), (int)(a.type == kE4m3), a.stall))
        return err;
    if (full == tiles) return cudaSuccess;
    return launch_after(linear_join_kernel<BN>, dim3(256 * BN / 8 / kJoinThreads, (unsigned)(tiles - full)),
                        dim3(kJoinThreads), st, e, walk);
}

template <bool AMN, bool BMN>
cudaError_t pick_pair(const LinArgs& a, const LinPlan& p, cudaStream_t st) {
    if constexpr (!AMN && !BMN) {
        if (p.sums) return p.tile == 128 ? go_pair<128, AMN, BMN, true>(a, p, st) : go_pair<256, AMN, BMN, true>(a, p, st);
    }
    return p.tile == 128 ? go_pair<128, AMN, BMN, false>(a, p, st) : go_pair<256, AMN, BMN, false>(a, p, st);
}

// --------------------------------------------------------------- pad rows

// A thread's 16 bytes of a destination row, from the two 16-byte pieces that they lie
// across in the source (whose rows start anywhere); at a row's ends, where a piece
// reaches past the row, element by element.
template <typename E>
__global__ void __launch_bounds__(256) pad_rows_kernel(const E* src, int64_t ld, int64_t rows, int64_t cols, E* dst,
                                                       int64_t ldd) {
    constexpr int V = 16 / (int)sizeof(E);
    tc::grid_dep_wait();
    tc::grid_dep_trigger();
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (c >= cols) return;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const E* row = src + r * ld;
        const E* s = row + c;
        const int mis = (int)(reinterpret_cast<uintptr_t>(s) & 15);
        const E* base = s - mis / (int)sizeof(E);
        uint4 out;
        if (base >= row && base + (mis ? 2 * V : V) <= row + cols) {
            const uint4 a = *reinterpret_cast<const uint4*>(base);
            out = a;
            if (mis) {
                const uint4 b = *reinterpret_cast<const uint4*>(base + V);
                const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                const int k = mis >> 2, bits = 8 * (mis & 3);
                uint32_t u[5];  // (static indices: selects, not an array in memory)
#pragma unroll
                for (int j = 0; j < 5; ++j)
                    u[j] = k == 0 ? w[j] : k == 1 ? w[j + 1] : k == 2 ? w[j + 2] : j + 3 < 8 ? w[j + 3] : 0u;
                out = make_uint4(__funnelshift_r(u[0], u[1], bits), __funnelshift_r(u[1], u[2], bits),
                                 __funnelshift_r(u[2], u[3], bits), __funnelshift_r(u[3], u[4], bits));
            }
        } else {
            E v[V];
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = c + j < cols ? s[j] : E(0);
            out = *reinterpret_cast<const uint4*>(v);
        }
        *reinterpret_cast<uint4*>(dst + r * ldd + c) = out;  // (ldd is a whole number of pieces)
    }
}

}  // namespace

// Which kernel, tile and split: the least of their times, in us, by two formulas whose
// constants were fitted to 2000 measured plans (5 to 4096 rows on nine weights of 512 to
// 20000 columns and rows, read from DRAM).  The choice is 1.6 % above the best one measured
// in the mean and 20 % at the worst (float32 outputs, 24 shapes: 1 and 7 %); a rule by the
// number of rows alone left 1.7 times (301 x 1536 x 1536: 12.7 us on pairs, 7.4 in tiles of
// 64 rows; 192 x 6144 x 1536: 17.4 and 10.8).
LinPlan plan_linear(const LinArgs& a, int sms) {
    LinPlan p{};
    int step;
    const int n_k = steps(a, &step);
    p.pairs = std::max(1, sms / 2);
    p.sums = in_sums(a) && n_k > sum_steps(a.type == kE4m3);
    float best = 0.f;
    const auto better = [&](float cost) {
        if (p.tile && cost >= best) return false;
        best = cost;
        return true;
    };
    // Pairs: the rounds' stages (or their epilogues) and the epilogue of one tile.  The tiles past the last full
    // round may be shared by the idle pairs, in parts of 4 stages at least, whose sums a
    // second kernel joins.  Sums of 256 columns spill registers once a tile.
    for (const int tile : {256, 128}) {
        const int64_t tiles = (a.M + 255) / 256 * ((a.N + tile - 1) / tile);
        const int tail = (int)(tiles % p.pairs);
        const float stage = tile == 128 ? 0.21f : p.sums ? 0.36f : 0.30f;
        const float epilogue = tile == 128 ? 1.9f : 3.1f;
        const float rounds = 2.8f + epilogue + (float)(tiles / p.pairs) * std::max(epilogue, (float)n_k * stage);
        const int most = tail > 0 ? std::min(std::min(16, p.pairs / tail), n_k / 4) : 1;
        for (int split = 1; split <= std::max(1, most); ++split) {
            const float last = tail == 0    ? 0.f
                               : split == 1 ? (float)n_k * stage
                                            : (float)((n_k + split - 1) / split) * stage + 4.1f + 0.41f * (float)split;
            if (!better(rounds + last)) continue;
            p.tile = tile;
            p.split = split;
            p.part_bytes = split > 1 ? sizeof(float) * (size_t)tail * split * 256 * tile : 0;
        }
    }
    // Few rows: a CTA's stages, all CTAs' reads from L2, the weights from DRAM, and the sums
    // sent to and finished by the CTAs of a cluster.  The reduction is split for as many CTAs
    // as 0.8 to 0.9 of those that fit (two to an SM or, of 16 rows, three): fewer leave SMs
    // idle, more queue; a float32 output's in so many that a CTA's sums fit its accumulators
    // (else it is for the pairs).  Up to 128 rows in any number of rounds, up to 512 in one.
    if (!a.a.k_major || a.M > 512) return p;
    for (const int tile : {16, 32, 64, 128}) {
        if (tile > 16 ? tile > 2 * a.M - 1 : a.M > 16) continue;
        const int64_t strips = (a.N + 127) / 128, tiles = strips * ((a.M + tile - 1) / tile);
        const int64_t fit = tile == 16 ? sms * 8 / 3 : sms * 8 / 5;
        if (a.M > 128 && tiles > fit) continue;
        int split = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(8, n_k / 2), fit / tiles));
        while (split < 8 && !few_fits(a, tile, (n_k + split - 1) / split)) ++split;
        if (!few_fits(a, tile, (n_k + split - 1) / split)) continue;
        const float n = (float)(tiles * split), rows = (float)std::min<int64_t>(tile, a.M), s = (float)split;
        const float k = (float)((n_k + split - 1) / split), per_sm = std::max(1.f, n / (float)sms);
        const float cost = 2.9f + k * (tile == 128 ? 0.25f : 0.17f) * (float)((tiles * split + fit - 1) / fit) +
                           3.4e-9f * n * k * (float)(kRowBytes * (128 + tile)) +
                           1.2e-7f * (float)strips * (float)n_k * (float)(kRowBytes * 128) +
                           rows * per_sm * (0.024f * (s - 1.f) + 0.04f) / s;
        if (!better(cost)) continue;
        p.few = true;
        p.tile = tile;
        p.split = split;
        p.part_bytes = 0;
    }
    return p;
}

cudaError_t launch_linear(const LinArgs& a, const LinPlan& p, cudaStream_t st) {
    if (p.few) return launch_linear_few(a, p, st);
    if (!a.a.k_major) return pick_pair<true, true>(a, p, st);
    return a.b.k_major ? pick_pair<false, false>(a, p, st) : pick_pair<false, true>(a, p, st);
}

cudaError_t launch_pad_rows(const void* src, int64_t ld, int64_t rows, int64_t cols, int bytes, void* dst,
                            int64_t ldd, cudaStream_t st) {
    const int64_t pieces = (cols * bytes + 15) / 16;
    const dim3 grid((unsigned)((pieces + 255) / 256), (unsigned)std::min<int64_t>(rows, 16384));
    if (bytes == 1)
        return launch_after(pad_rows_kernel<uint8_t>, grid, dim3(256), st, static_cast<const uint8_t*>(src), ld, rows,
                            cols, static_cast<uint8_t*>(dst), ldd);
    return launch_after(pad_rows_kernel<uint16_t>, grid, dim3(256), st, static_cast<const uint16_t*>(src), ld, rows,
                        cols, static_cast<uint16_t*>(dst), ldd);
}

}  // namespace qh

