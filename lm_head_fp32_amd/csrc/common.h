// common.h -- internal declarations shared by the gfx950 kernels and the
// C-ABI layer of liblmhead.so.  Not installed; the public interface is
// include/lmhead.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lmh {

// Operand description for the generic contraction
//   D[c][r] (op)= sum_p A(r, p) * B(c, p)
// A(r, p) is at A[r * lda + p] when !a_trans (p contiguous) and at
// A[p * lda + r] when a_trans (r contiguous); B likewise with c.
// D is row-major [C x R] with leading dimension ldd (r contiguous).
struct GemmProblem {
    const uint16_t *A;
    int64_t lda;
    const uint16_t *B;
    int64_t ldb;
    void *D;
    int64_t ldd;
    int64_t R, C, P;
    // kStoreF32Stats only (the logits GEMM, R = vocabulary, C = tokens): the
    // tokens' targets and the per-256-row-block cross-entropy records
    // {m, d, X_y, own} written at part4[(r0 / 256) * part_stride4 + c].
    const int32_t *tgt = nullptr;
    int32_t ignore_index = 0;
    void *part4 = nullptr;
    int64_t part_stride4 = 0;
    // Split of the sum over p (gemm_big only): workgroup row blockIdx.y sums
    // p in [y * psplit, min(P, (y + 1) * psplit)) and stores its FP32 partial
    // tile at D + y * split_stride.  psplit == 0: no split.
    int64_t psplit = 0;
    int64_t split_stride = 0;
    // Output stores bypass the caches' normal allocation (nontemporal): a
    // GEMM's output is written once and not read back by this kernel, and
    // lines left dirty in L2 and the 256 MB MALL would otherwise be written
    // back during the next kernel's reads.  Off for partial sums that the
    // next kernel reads back at once.
    bool stream_out = true;
};

typedef float f32x4_nt __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_nt __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void store16(float *p, float4 v, bool stream)
{
    if (stream) {
        const f32x4_nt w = {v.x, v.y, v.z, v.w};
        __builtin_nontemporal_store(w, reinterpret_cast<f32x4_nt *>(p));
    } else {
        *reinterpret_cast<float4 *>(p) = v;
    }
}

typedef uint32_t u32x2_nt __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void store8(uint16_t *p, uint2 v, bool stream)
{
    if (stream) {
        const u32x2_nt w = {v.x, v.y};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2_nt *>(p));
    } else {
        *reinterpret_cast<uint2 *>(p) = v;
    }
}

__device__ __forceinline__ void store16(uint16_t *p, uint4 v, bool stream)
{
    if (stream) {
        const u32x4_nt w = {v.x, v.y, v.z, v.w};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_nt *>(p));
    } else {
        *reinterpret_cast<uint4 *>(p) = v;
    }
}

enum class Epi : int { kStoreF32 = 0, kStoreBF16 = 1, kAccumF32 = 2, kStoreF32Stats = 3 };

// Launchers (return the hipError_t of the launch).
hipError_t launch_gemm_logits(const GemmProblem &p, Epi epi, hipStream_t s);
// True when launch_gemm_logits runs kStoreF32Stats in its epilogue for p
// (the 256 x 256 eight-wave kernels); otherwise the caller computes the
// records from the stored logits.
bool gemm_logits_stats_in_epilogue(const GemmProblem &p);
hipError_t launch_gemm_dgrad(const GemmProblem &p, Epi epi, hipStream_t s);
// dgrad with the sum over V split `splits` ways (0 = the shape's default):
// FP32 partials in `ws`, then a reduction in split order into p.D.
int dgrad_default_splits(int64_t M, int64_t K, int64_t V);
int64_t dgrad_workspace_elems(int64_t M, int64_t K, int64_t V, int splits);
hipError_t launch_gemm_dgrad_split(const GemmProblem &p, bool bf16_out, int splits, float *ws,
                                   hipStream_t s);
hipError_t launch_gemm_wgrad(const GemmProblem &p, Epi epi, hipStream_t s);

hipError_t launch_xent_fwd(const float *logits, int64_t ld, int64_t n_rows, int64_t n_cols,
                           const int32_t *target, int32_t ignore_index, float *loss,
                           float *stats, hipStream_t s);
hipError_t launch_xent_partial(const float *logits, int64_t ld, int64_t n_rows, int64_t n_cols,
                               int64_t col0, int64_t block_cols, const int32_t *target,
                               int32_t ignore_index, float *part, int64_t part_stride,
                               hipStream_t s);
hipError_t launch_xent_merge(const float *part, int64_t n_parts, int64_t part_stride,
                             int64_t n_rows, const int32_t *target, int32_t ignore_index,
                             int64_t vocab, float *loss, float *stats, hipStream_t s);
hipError_t launch_xent_fused(const float *logits, int64_t ld, int64_t n_rows, int64_t n_cols,
                             const int32_t *target, int32_t ignore_index, const float *dloss,
                             int64_t dloss_stride, float *loss, float *stats, void *dlogits,
                             int64_t ldg, bool bf16_out, hipStream_t s);
hipError_t launch_xent_mean(const float *loss, const int32_t *target, int32_t ignore_index,
                            int64_t n_rows, float *mean_out, float *inv_out, hipStream_t s);
hipError_t launch_xent_bwd(const float *logits, int64_t ld, const float *stats,
                           const int32_t *target, int32_t ignore_index, const float *dloss,
                           int64_t dloss_stride, void *dlogits, int64_t ldg, bool bf16_out,
                           int64_t n_rows, int64_t n_cols, hipStream_t s);
// Register-only MFMA loop (diagnostic): 256-thread workgroups, one float per
// thread written to sink; all-ones or pseudo-random operands.
int mfma_loop_chains();
hipError_t launch_mfma_loop(int64_t iters, int64_t n_workgroups, bool random_operands,
                            float *sink, hipStream_t s);

// Low-rank adapters: A [n][r][K] and B [n][V][r] BF16, contiguous in K and r;
// token m uses adapter[m] (negative: none); scale [n] or null (1).
struct LoraAdapters {
    const uint16_t *A;
    int64_t lda, stride_a;
    const uint16_t *B;
    int64_t ldb, stride_b;
    const int32_t *adapter;
    const float *scale;
    int64_t n;
    int r;
};

// Gradients of the adapters' part of the logits; dX, dA, dB may be null.
struct LoraBwd {
    const uint16_t *g;
    int64_t ldg;
    const uint16_t *x;
    int64_t ldx;
    LoraAdapters ad;
    float *dX;
    int64_t lddx;
    float *dA;
    int64_t ldda, stride_da;
    float *dB;
    int64_t lddb, stride_db;
    bool accumulate;
    int64_t M, K, V;
};

int64_t lora_logits_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t r, bool bf16);
int64_t lora_bwd_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t r, int64_t n);
// p as for launch_gemm_logits (R = V, C = M, P = K), with D the final logits.
hipError_t launch_logits_lora(const GemmProblem &p, bool bf16, const LoraAdapters &ad, void *workspace,
                              hipStream_t s);
hipError_t launch_lora_bwd(const LoraBwd &p, void *workspace, hipStream_t s);

int64_t beam_segments(int64_t V);
int64_t beam_workspace_bytes(int64_t n_rows, int64_t V, int64_t n_out);
hipError_t launch_beam_select(const void *logits, int64_t ld, bool bf16, int64_t B, int64_t W,
                              int64_t V, const float *scores, const uint8_t *finished, int32_t eos,
                              int64_t n_out, float *out_scores, int32_t *out_parent,
                              int32_t *out_token, uint8_t *out_finished, void *workspace,
                              hipStream_t s);
// Strides in bytes: outer, row (beam), head.
hipError_t launch_beam_reorder(const void *src, void *dst, const int64_t (&src_strides)[3],
                               const int64_t (&dst_strides)[3], const int32_t *parent,
                               const int32_t *lengths, int64_t n_outer, int64_t B, int64_t W_in,
                               int64_t W_out, int64_t H, int64_t T, int64_t pos_bytes, hipStream_t s);

// Log-probabilities of given tokens; null outputs (and token, when nothing needs
// it) are skipped, k = 0 without alternatives.  Strides of the temperature and of
// the upstream gradients: 0 (one value) or 1 (one per row).
struct Logprobs {
    const void *logits;
    int64_t ld;
    bool bf16;
    int64_t n, V;
    const int32_t *token;
    int32_t ignore_index;
    const float *temperature;
    int64_t temperature_stride;
    int64_t k;
    float *logprob, *entropy;
    int32_t *rank;
    float *top_logprob;
    int32_t *top_token;
    float *stats;
};
struct LogprobsBwd {
    const void *logits;
    int64_t ld;
    bool bf16;
    const float *stats;
    const int32_t *token;
    int32_t ignore_index;
    const float *temperature;
    int64_t temperature_stride;
    const float *dlogprob;
    int64_t dlogprob_stride;
    const float *dentropy;
    int64_t dentropy_stride;
    void *dlogits;
    int64_t ldg;
    bool grad_bf16;
    int64_t n, V;
};
int64_t logprobs_workspace_bytes(int64_t n_rows, int64_t V, int64_t k);
hipError_t launch_logprobs(const Logprobs &p, void *workspace, hipStream_t s);
hipError_t launch_logprobs_bwd(const LogprobsBwd &p, hipStream_t s);

// Cross-entropy against a teacher's listed tokens (k of them per row).
constexpr int64_t kDistillMaxList = 256;
struct Distill {
    const void *logits;
    int64_t ld;
    bool bf16;
    int64_t n, V;
    const int32_t *token;
    int64_t ldt;
    const void *value;
    int64_t ldv;
    bool value_bf16;
    int64_t k;
    bool tail;
    const float *temperature;
    int64_t temperature_stride;
    float *loss;        // forward; may be null
    float *stats;       // written by the forward, read by the gradient
    const float *dloss; // gradient
    int64_t dloss_stride;
    void *dlogits;
    int64_t ldg;
    bool grad_bf16;
};
int64_t distill_workspace_bytes(int64_t n_rows, int64_t V);
hipError_t launch_distill_fwd(const Distill &p, void *workspace, hipStream_t s);
hipError_t launch_distill_bwd(const Distill &p, hipStream_t s);
hipError_t launch_distill_fused(const Distill &p, void *workspace, hipStream_t s);

// exp(z - m) as one hardware base-2 exponential; the same form everywhere the
// cross-entropy statistics are computed (CE kernels, logits GEMM epilogue).
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp_shifted(float z, float m)
{
    return __builtin_amdgcn_exp2f((z - m) * kLog2e);
}

// Merge two partial (m, d) pairs.  A pair with m = -inf is empty.
__device__ __forceinline__ void merge_md(float &m, float &d, float m2, float d2)
{
    const float mn = fmaxf(m, m2);
    if (mn == -INFINITY)
        return;  // both empty
    const float s1 = (m == -INFINITY) ? 0.0f : exp_shifted(m, mn);
    const float s2 = (m2 == -INFINITY) ? 0.0f : exp_shifted(m2, mn);
    d = d * s1 + d2 * s2;
    m = mn;
}

// FP32 -> BF16 bits, round to nearest, ties to even; NaN stays a quiet NaN.
// Written as a select (no branch), so that per-element use compiles to
// straight-line code.
__device__ __forceinline__ uint32_t f32_to_bf16_bits(float f)
{
    const uint32_t u = __float_as_uint(f);
    const uint32_t rounded = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
    const uint32_t quiet_nan = (u >> 16) | 0x40u;
    return ((u & 0x7fffffffu) > 0x7f800000u) ? quiet_nan : rounded;
}

}  // namespace lmh
