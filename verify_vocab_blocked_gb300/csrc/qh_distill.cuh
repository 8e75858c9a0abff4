// qh_distill.cuh -- launchers of the distillation loss (qh_distill.cu).
#pragma once

#include "qh_internal.cuh"

namespace qh {

constexpr int kMaxTeacher = 1024;  // teacher entries per row
constexpr int kOthers = 16;        // other vocab rows whose exact logits are kept, at most
constexpr int kKeptExtra = 2 * kOthers;  // kept values per row beyond the K logits
constexpr int64_t kFewM = 16;          // rows up to which the weight-streaming kernel forms them
constexpr int kFewSplits = 64;         // vocab splits of their softmax pass

// Whether the forward keeps its logits for the backward: up to 4 GiB, the budget of
// the backward's coefficient block, and always for few rows, whose softmax pass
// reads them.  The backward then forms its coefficients by one pass over them
// instead of running the logit kernel again (512 rows of the 262144 x 2560 head:
// see distill_from_logits_kernel).
constexpr int64_t kKeepBytes = (int64_t)4 << 30;
inline bool keeps_logits(int64_t M, int64_t V) { return M <= kFewM || M * V <= kKeepBytes / 4; }

// Columns of kept, and where a row's logits begin in it (whole 32-byte units;
// the logits in whole blocks of 32).
inline int64_t kept_logits_at(int64_t K) { return (K + kKeptExtra + 7) / 8 * 8; }
inline int64_t kept_columns(int64_t M, int64_t K, int64_t V) {
    return keeps_logits(M, V) ? kept_logits_at(K) + (V + 31) / 32 * 32 : K + kKeptExtra;
}

// The largest raw logit of every 32 vocab rows without the listed ones, per compact
// row, in whole tiles of 256 vocab rows.
__host__ __device__ inline int64_t slice_columns(int64_t V) { return (V + 255) / 256 * 8; }

// What a tensor-core logit is multiplied by to take its mean error out.  Its
// fp32 accumulation truncates: each of the H / 16 steps loses half an ulp of the
// partial sum on average.  Over mantissas an ulp is 0.72 * 2^-23 of its value
// in the mean, and the partial sum grows to the logit z evenly, so z comes out
// short by about (H / 16) * 0.36 * 2^-23 / 2 = (H / 16) * 2.1e-8 of itself.
// Measured from lse's mean error over 512 rows with three quarters of their mass on
// many unlisted logits (V = 32768, 4 and 8 bits, cap 30 and none): 1.4 to 1.9e-8 at
// 1024 to 8192 columns, 1.0 to 1.5e-8 at 512; at 128 the rows' spread hides it.  The
// factor takes that mean error from -2.5e-6 at 1024 columns, -6e-6 at 2560 and -2.0e-5
// at 8192 to within 1.4e-6 of zero at every width from 512 on.
inline float distill_unbias(int H) { return 1.f + 1.7e-8f * (float)(H / 16); }

// sid [Mpad, K + 1]: each compact row's distinct valid ids, ascending, then
// INT32_MAX; kept [M, ld]: in the first K the exact capped logits of
// the valid entries (0 for the others and for inactive rows).
cudaError_t launch_distill_prep(const uint32_t* wq, SbView sb, int64_t V, int H, int bits, float cap,
                                const __nv_bfloat16* h, const int* pos, int64_t M,
                                const int32_t* ids, int K, int* sid, float* kept, int64_t ld,
                                float* zout, cudaStream_t st);
cudaError_t launch_distill_finalize(const uint32_t* wq, SbView sb, int64_t V, int H, int bits,
                                    float cap, const __nv_bfloat16* h, const int* pos, int64_t M,
                                    const int32_t* ids, const void* tl, int t_type, int K,
                                    float inv_t, float unbias, float* kept, int64_t ld, float* zout,
                                    const Partial* part, int S, const int* S_dev, const float* smax,
                                    const int* err, float* loss, float* lse, cudaStream_t st);
cudaError_t launch_distill_coeff(int64_t V, float cap, const int* pos, int64_t M,
                                 const int32_t* ids, const void* tl, int t_type, int K, float inv_t,
                                 const float* kept, int64_t ld_kept, const float* lse,
                                 const float* dloss, float* geff, __half* coeff, int64_t ld,
                                 int64_t v_begin, int64_t chunk, cudaStream_t st);
cudaError_t launch_distill_split(const float* z, int64_t ld, int64_t V, float cap, float inv_t,
                                 const int* pos, int64_t M, Partial* part, float* smax,
                                 cudaStream_t st);
cudaError_t launch_distill_from_logits(const float* kept, int64_t K, int64_t ld, int64_t V, float cap,
                                       float inv_t, float unbias, const int* rows, const int* count, int64_t M,
                                       const float* lse, const float* dloss, float* geff, __half* coeff,
                                       int64_t ldc, int64_t v_begin, int64_t chunk, cudaStream_t st);
cudaError_t launch_distill_dh(const float* dhp, int S, int64_t Mpad, int H, const int* pos,
                              int64_t M, const int* err, void* dh, cudaStream_t st);

}  // namespace qh
