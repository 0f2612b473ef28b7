// beam.hip -- beam search over the output layer's logits on gfx950: the
// selection of the next beams (scan + merge) and the reordering of per-beam
// states that follows it.
//
// Selection, per request b with W beams over V tokens:
//   c(w, v) = s_w + (z_wv - m_w) - log d_w,  m_w = max_v z_wv,  d_w = sum_v exp(z_wv - m_w)
// and the n_out largest c in descending order, equal ones by ascending w, then
// descending z, then ascending v (by w V + v, then, unless logits differ by less
// than c resolves).  Within a beam the order of c is the order of z, so one pass over
// the logits suffices: every wave reads one segment of a row into registers
// and leaves the segment's {max, sum of exponentials} and its n_out largest
// logits; a second kernel folds the sums, turns the kept logits into scores
// and picks the winners.  Which candidate wins must not depend on rounding,
// so sums, logarithms and scores are FP64 (the logits enter exactly); only the
// returned score is rounded, once, to FP32.  The exponentials are taken about the
// row's maximum and log of their sum is kept apart from it, c = s_w + ((z_wv -
// m_w) - log d_w): the largest logit then adds exactly 1, so no candidate scores
// above its beam, a token that is the only one left scores exactly as its beam,
// and rows that differ by a constant (in FP32 exactly) give equal scores.  Scores
// that are equal by the mathematics alone, the same terms in another order say,
// can differ by the last bits of the sum.
//
// A candidate that is NaN counts as -inf.  The scan keeps values above -inf
// only; beams whose every candidate is -inf (a score that is not below +inf
// or is NaN or -inf, a row holding NaN or +inf, a row of -inf only) and the
// tokens a finished beam cannot take never reach a list.  Where fewer than
// n_out candidates lie above -inf, at most n_out - 1 of the first
// 2 n_out positions w V + v can be among them, so the rest is filled from
// those positions in order.
#include "common.h"

#include <math.h>

#include <algorithm>

namespace lmh {

namespace {

constexpr int64_t kMaxItems = int64_t{1} << 31;  // work-items per launch
constexpr int kBeamMax = 64;       // beams per request, and beams selected
constexpr int kSegCols = 2048;     // columns a wave holds at a time, 32 a lane
constexpr int kCandCap = 512;      // candidates a wave can hold

// What a wave leaves of its segment of a row, besides its list.
struct SegRecord {
    double d;  // sum over the segment of exp(z - m); NaN: it holds NaN or +inf
    double m;  // the segment's maximum; -inf: nothing above -inf
};
static_assert(sizeof(SegRecord) == 16, "one 16-byte record per segment");

// FP32 -> uint32 with the same order (-0 and +0 equal); 0 lies below -inf.
__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// exp(x) for x <= 0, relative error below 3e-10: x = n ln 2 + r with
// |r| <= ln 2 / 2, the Taylor sum of e^r to r^8 (the next term is
// 0.3466^9 / 9! = 2e-10), scaled by 2^n.
__device__ __forceinline__ double exp_nonpos(double x)
{
    x = fmax(x, -800.0);  // e^-800 underflows to 0, as e^-inf does
    const double n = rint(x * 1.4426950408889634);
    const double r = fma(-n, 0.6931471805599453, x);
    double p = 1.0 / 40320.0;
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return ldexp(p, static_cast<int>(n));
}

// Sum of exp(v[i] - m) for a finite m at least every v[i], in FP64.  y = (m - v[i]) /
// 512, one product and sum cut to [0, 1] by the instruction (a difference of 512
// and more, -inf too, counts as 512: e^-512 is nothing beside 1); 2^(-512 y log2 e)
// split into integer n and fraction f by adding 1.5 x 2^52 (n is then in the low
// word); 2^f from a polynomial that is 1 at f = 0 and whose relative error
// alternates below 2.0e-9 on [-1/2, 1/2] (fitted under that condition); 2^n by an
// integer add to the exponent: 12 full-rate instructions a value and one
// conversion.  The largest value adds exactly 1, and the same row moved by a
// constant has the same sum.
template <int PER>
__device__ __forceinline__ double sum_exp(const float (&v)[PER], double m)
{
    constexpr double kLog2E = 1.4426950408889634, kMagic = 6755399441055744.0;
    const double m512 = m / 512.0;
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const double y = fmin(fmax(fma(static_cast<double>(v[i]), -1.0 / 512.0, m512), 0.0), 1.0);
        const double t = fma(y, -512.0 * kLog2E, kMagic);
        const double f = fma(y, -512.0 * kLog2E, kMagic - t);
        double p = 0.00015353362227507272;
        p = fma(p, f, 0.0013398874406550455);
        p = fma(p, f, 0.009618437356465498);
        p = fma(p, f, 0.055503324711486945);
        p = fma(p, f, 0.2402264791363921);
        p = fma(p, f, 0.6931472028550582);
        p = fma(p, f, 1.0);
        const int n = static_cast<int>(__double_as_longlong(t));  // the low word
        d += __hiloint2double(__double2hiint(p) + (n << 20), __double2loint(p));
    }
    return d;
}

__device__ __forceinline__ double shfl_xor_f64(double v, int off)
{
    const uint64_t u = __double_as_longlong(v);
    const uint32_t lo = __shfl_xor(static_cast<uint32_t>(u), off, 64);
    const uint32_t hi = __shfl_xor(static_cast<uint32_t>(u >> 32), off, 64);
    return __longlong_as_double((static_cast<uint64_t>(hi) << 32) | lo);
}

__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t u, int off)
{
    const uint32_t lo = __shfl_xor(static_cast<uint32_t>(u), off, 64);
    const uint32_t hi = __shfl_xor(static_cast<uint32_t>(u >> 32), off, 64);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// Reductions over the wave, every lane getting the result: lanes of a row of
// 16 through DPP (quad permutations, then rotations by 4 and 8), the four rows
// through LDS permutes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v)
{
    const uint64_t u = __double_as_longlong(v);
    return __longlong_as_double((static_cast<uint64_t>(dpp<CTRL>(static_cast<uint32_t>(u >> 32))) << 32) |
                                dpp<CTRL>(static_cast<uint32_t>(u)));
}
constexpr int kQuadXor1 = 0xb1, kQuadXor2 = 0x4e, kRowRor4 = 0x124, kRowRor8 = 0x128;

__device__ __forceinline__ float wave_maximum(float m)  // NaN if any lane's is
{
    m = __builtin_elementwise_maximum(m, __uint_as_float(dpp<kQuadXor1>(__float_as_uint(m))));
    m = __builtin_elementwise_maximum(m, __uint_as_float(dpp<kQuadXor2>(__float_as_uint(m))));
    m = __builtin_elementwise_maximum(m, __uint_as_float(dpp<kRowRor4>(__float_as_uint(m))));
    m = __builtin_elementwise_maximum(m, __uint_as_float(dpp<kRowRor8>(__float_as_uint(m))));
    m = __builtin_elementwise_maximum(m, __shfl_xor(m, 16, 64));
    return __builtin_elementwise_maximum(m, __shfl_xor(m, 32, 64));
}

__device__ __forceinline__ double wave_sum(double d)
{
    d += dpp_f64<kQuadXor1>(d);
    d += dpp_f64<kQuadXor2>(d);
    d += dpp_f64<kRowRor4>(d);
    d += dpp_f64<kRowRor8>(d);
    d += shfl_xor_f64(d, 16);
    return d + shfl_xor_f64(d, 32);
}

// True when the beam can offer a candidate above -inf by its score alone.
__device__ __forceinline__ bool score_alive(float s)
{
    return s > -INFINITY && s < INFINITY;  // false for NaN
}

// A segment of a row on its way from memory: lane l holds columns
// j0 + (64 u + l) G + e, G per 16-byte load; columns at or past V read as -inf.
template <bool BF16>
struct Segment {
    static constexpr int G = BF16 ? 8 : 4, NQ = 32 / G;
    uint4 q[NQ];
    __device__ __forceinline__ void load(const void *row, int64_t V, int64_t j0, int lane)
    {
        if (j0 + kSegCols <= V) {
#pragma unroll
            for (int u = 0; u < NQ; ++u)
                q[u] = *reinterpret_cast<const uint4 *>(static_cast<const char *>(row) +
                                                        (j0 + (64 * u + lane) * G) * (16 / G));
            return;
        }
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            uint32_t w[4];
            const int64_t j = j0 + (64 * u + lane) * G;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (BF16) {
                    const uint16_t *p = static_cast<const uint16_t *>(row) + j + 2 * e;
                    const uint32_t lo = j + 2 * e < V ? p[0] : 0xff80u;
                    const uint32_t hi = j + 2 * e + 1 < V ? p[1] : 0xff80u;
                    w[e] = lo | (hi << 16);
                } else {
                    w[e] = j + e < V ? static_cast<const uint32_t *>(row)[j + e] : 0xff800000u;
                }
            }
            q[u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __device__ __forceinline__ void values(float (&v)[32]) const
    {
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (BF16) {
                    v[8 * u + 2 * e] = __uint_as_float(w[e] << 16);
                    v[8 * u + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                } else {
                    v[4 * u + e] = __uint_as_float(w[e]);
                }
            }
        }
    }
};

// One wave, a workgroup of its own, per (row, segment of 2048 columns).  Bound by
// the one read of the logits: the segment sits in registers, so the sum, the
// maximum and the candidates cost no second read; nothing is shared between
// waves, and six per SIMD cover each other's loads.  A wave goes first (priority)
// until its loads are out, so that they do not wait behind the some 600
// instructions with which the others treat theirs.  461 rows of 131072 FP32
// columns, 242 MB: 50 - 54 us, 4.5 - 4.8 TB/s; without the priority 53 - 54, in
// workgroups of four waves 56 - 59.
// Candidates: the k-th largest of the 64 lane maxima is a lower bound of the
// segment's k-th largest value (that many lanes hold a value at least as
// large), cut to its upper 16 bits so that 16 ballots find it; the few values
// at or above it are collected in LDS and ranked by counting.  The list is in
// descending value, equal values in ascending column.
template <bool BF16>
__global__ __launch_bounds__(64) void beam_scan_kernel(
    const void *__restrict__ logits, int64_t ld, int64_t V, uint32_t nseg,
    const float *__restrict__ scores, const uint8_t *__restrict__ finished, int32_t k,
    SegRecord *__restrict__ rec, uint64_t *__restrict__ lists)
{
    constexpr int G = Segment<BF16>::G;
    __shared__ uint64_t mine[kCandCap];
    __builtin_amdgcn_s_setprio(3);
    const int lane = threadIdx.x;
    const uint32_t id = blockIdx.x, row = id / nseg;  // below 2^25
    if (!score_alive(scores[row]) || (finished && finished[row]))
        return;  // the merge does not read this beam's records
    const int64_t j0 = static_cast<int64_t>(id - row * nseg) * kSegCols;
    float v[32];
    {
        Segment<BF16> sg;
        sg.load(static_cast<const char *>(logits) + static_cast<int64_t>(row) * ld * (16 / G), V, j0, lane);
        __builtin_amdgcn_s_setprio(0);
        sg.values(v);
    }
    float gm[8], lm = -INFINITY;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        gm[u] = __builtin_elementwise_maximum(__builtin_elementwise_maximum(v[4 * u], v[4 * u + 1]),
                                              __builtin_elementwise_maximum(v[4 * u + 2], v[4 * u + 3]));
        lm = __builtin_elementwise_maximum(lm, gm[u]);  // NaN stays NaN
    }
    const float m = wave_maximum(lm);
    uint64_t *out = lists + static_cast<int64_t>(id) * k;
    if (!(m < INFINITY) || m == -INFINITY) {
        // NaN or +inf somewhere (the whole row then offers nothing), or only
        // -inf: no candidates.
        if (lane == 0) {
            rec[id].d = (m == -INFINITY) ? 0.0 : static_cast<double>(NAN);
            rec[id].m = (m == -INFINITY) ? -INFINITY : 0.0;
        }
        if (lane < k)
            out[lane] = 0;
        return;
    }

    const double d = wave_sum(sum_exp(v, m));
    if (lane == 0) {
        rec[id].d = d;
        rec[id].m = m;
    }

    const uint32_t mykey = order_key(lm);
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b >= 16; --b) {
        const uint32_t c = t | (1u << b);
        if (__popcll(__ballot(mykey >= c)) >= k)
            t = c;
    }
    const float bound = key_value(max(t, order_key(-INFINITY) + 1u));
    const uint32_t rest = 0xffffffffu - (static_cast<uint32_t>(j0) + static_cast<uint32_t>(lane * G));
    auto key_of = [&](int i) {
        return (static_cast<uint64_t>(order_key(v[i])) << 32) | (rest - static_cast<uint32_t>(64 * (i / G) * G + i % G));
    };
    int n = 0;  // the same in every lane
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        if (!__ballot(gm[u] >= bound))
            continue;
#pragma unroll
        for (int i = 4 * u; i < 4 * u + 4; ++i) {
            const uint64_t mask = __ballot(v[i] >= bound);
            if (v[i] >= bound) {
                const int at = n + __popcll(mask & ((1ull << lane) - 1ull));
                if (at < kCandCap)
                    mine[at] = key_of(i);
            }
            n += __popcll(mask);
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (n <= kCandCap) {
        for (int i = lane; i < n; i += 64) {
            const uint64_t key = mine[i];
            int rank = 0;
            for (int q = 0; q < n; ++q)
                rank += mine[q] > key;
            if (rank < k)
                out[rank] = key;
        }
        if (n + lane < k)
            out[n + lane] = 0;
        return;
    }
    // Many equal values at the bound: k rounds, each taking the largest key
    // below the last one.
    uint64_t last = ~0ull;
    for (int r = 0; r < k; ++r) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint64_t key = key_of(i);
            if (v[i] > -INFINITY && key < last && key > best)
                best = key;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            best = max(best, shfl_xor_u64(best, off));
        if (lane == 0)
            out[r] = best;
        last = best;
    }
}

// A candidate: its score, its beam and its key in the beam's lists (larger: a
// larger logit, or an equal one of an earlier token).  `before`: larger score,
// equal scores by ascending beam, then descending key.  The scores of a beam
// whose logits are tiny can be equal where the logits are not; the lists hold
// the largest logits, so the logits decide.
struct Pick {
    double c;
    uint64_t key;
    int32_t w;
};
__device__ __forceinline__ bool before(const Pick &a, const Pick &b)
{
    return a.c > b.c || (a.c == b.c && (a.w < b.w || (a.w == b.w && a.key > b.key)));
}
__device__ __forceinline__ uint32_t key_token(uint64_t key)
{
    return 0xffffffffu - static_cast<uint32_t>(key);
}

constexpr int kMergeThreads = 512;
constexpr int kMergeCap = 1024;
constexpr double kMaskedOut = -0x1p126;

// One workgroup per request: the sum of every beam from its segments' records,
// then the n_out best of the W nseg sorted lists.  Latency-bound (a few
// thousand candidates): a lower bound on the n_out-th best score, from the
// lists' heads as in the scan, leaves a few dozen candidates to rank.
__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(
    const void *__restrict__ logits, int64_t ld, int32_t bf16, int32_t W, int64_t V, int32_t nseg,
    const float *__restrict__ scores, const uint8_t *__restrict__ finished, int32_t eos, int32_t k,
    const SegRecord *__restrict__ rec, const uint64_t *__restrict__ lists,
    float *__restrict__ out_scores, int32_t *__restrict__ out_parent,
    int32_t *__restrict__ out_token, uint8_t *__restrict__ out_finished)
{
    constexpr int NW = kMergeThreads / 64;
    __shared__ double logd[kBeamMax];     // NaN: no candidate above -inf
    __shared__ float top[kBeamMax];       // the row's maximum
    __shared__ float sc[kBeamMax];
    __shared__ uint8_t fin[kBeamMax];
    __shared__ uint32_t group[64];
    __shared__ double cs[kMergeCap];
    __shared__ uint64_t ck[kMergeCap];
    __shared__ int32_t cw[kMergeCap];
    __shared__ uint32_t n_cand;
    __shared__ Pick red[NW];

    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t row0 = b * W;
    // Lists 0 .. W nseg - 1 (beam l / nseg) and one candidate per finished beam;
    // list l is walked by thread (l % 64) * 8 + (l / 64) % 8, so that the 64
    // groups of eight threads share the lists evenly.  The head of the thread's
    // first list is on its way while the sums are folded.
    const int64_t n_lists = static_cast<int64_t>(W) * nseg;
    const int64_t l0 = (tid >> 3) + 64 * (tid & 7);
    const uint64_t head0 = l0 < n_lists ? lists[(row0 * nseg + l0) * k] : 0;
    if (tid < W) {
        sc[tid] = scores[row0 + tid];
        fin[tid] = finished ? (finished[row0 + tid] != 0) : 0;
    }
    if (tid < 64)
        group[tid] = 0;
    if (tid == 0)
        n_cand = 0;
    __syncthreads();

    for (int w = wave; w < W; w += NW) {
        double log_d = static_cast<double>(NAN), m = -INFINITY;
        if (!fin[w] && score_alive(sc[w])) {
            const SegRecord *r = rec + (row0 + w) * nseg;
            for (int s = lane; s < nseg; s += 64)
                m = fmax(m, r[s].m);
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1)
                m = fmax(m, shfl_xor_f64(m, off));
            if (m > -INFINITY) {
                double d = 0.0;  // NaN from any segment that holds NaN or +inf
                for (int s = lane; s < nseg; s += 64)
                    d += r[s].d * exp_nonpos(r[s].m - m);
                log_d = log(wave_sum(d));
                // Nothing but masks of the type's lowest value: not normalised
                // (m + log d is m in 64 bits).
                if (m < kMaskedOut && log_d == log_d)
                    log_d = 0.0;
            }
        }
        if (lane == 0) {
            logd[w] = log_d;
            top[w] = static_cast<float>(m);
        }
    }
    __syncthreads();

    auto score_of = [&](int w, uint64_t key) {
        const double z = static_cast<double>(key_value(static_cast<uint32_t>(key >> 32)));
        return static_cast<double>(sc[w]) + ((z - static_cast<double>(top[w])) - logd[w]);
    };
    // A finished beam's one candidate, at `eos`.
    const uint64_t held_key = 0xffffffffu - static_cast<uint32_t>(eos);
    auto held = [&](int w) { return fin[w] && score_alive(sc[w]) && eos >= 0 && eos < V; };

    double head = -INFINITY;
    for (int64_t l = l0; l < n_lists; l += kMergeThreads) {
        const int w = static_cast<int>(l / nseg);
        if (logd[w] == logd[w]) {
            const uint64_t key = l == l0 ? head0 : lists[(row0 * nseg + l) * k];
            if (key)
                head = fmax(head, score_of(w, key));
        }
    }
    if (tid < W && held(tid))
        head = fmax(head, static_cast<double>(sc[tid]));
    // Rounded down, so that a bound on the rounded heads bounds the scores; what
    // lies below the FP32 range becomes -inf, which is no bound.
    if (head > -INFINITY)
        atomicMax(&group[tid >> 3], order_key(__double2float_rd(head)));
    __syncthreads();
    uint32_t t = 0;
    {
        const uint32_t g = group[lane];
#pragma unroll
        for (int bit = 31; bit >= 8; --bit) {
            const uint32_t c = t | (1u << bit);
            if (__popcll(__ballot(g >= c)) >= k)
                t = c;
        }
    }
    // The bound is a finite FP32 value that k heads reach, or there is none: the
    // FP64 scores of fewer than k heads may lie in the FP32 range (or be all there
    // are), and one below it, -FLT_MAX plus a masked logit's -FLT_MAX say, still
    // comes before -inf.
    const double tv = t > order_key(-INFINITY) ? static_cast<double>(key_value(t)) : -INFINITY;
    auto append = [&](double c, int w, uint64_t key) {
        const uint32_t at = atomicAdd(&n_cand, 1u);
        if (at < kMergeCap) {
            cs[at] = c;
            ck[at] = key;
            cw[at] = w;
        }
    };
    if (head > -INFINITY && head >= tv) {
        for (int64_t l = l0; l < n_lists; l += kMergeThreads) {
            const int w = static_cast<int>(l / nseg);
            if (!(logd[w] == logd[w]))
                continue;
            const uint64_t *q = lists + (row0 * nseg + l) * k;
            // Four keys at a time: one wait for most lists.
            for (int i = 0; i < k; i += 4) {
                uint64_t key[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    key[e] = i + e < k ? q[i + e] : 0;
                bool more = true;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const double c = score_of(w, key[e]);
                    more = more && key[e] && c >= tv;
                    if (more)
                        append(c, w, key[e]);
                }
                if (!more)
                    break;
            }
        }
        if (tid < W && held(tid) && static_cast<double>(sc[tid]) >= tv)
            append(static_cast<double>(sc[tid]), tid, held_key);
    }
    __syncthreads();

    auto emit = [&](int i, double c, int w, int32_t tok) {
        const int64_t o = b * k + i;
        out_scores[o] = static_cast<float>(c);
        out_parent[o] = w;
        out_token[o] = tok;
        out_finished[o] = (fin[w] || tok == eos) ? 1 : 0;
    };
    const int n = static_cast<int>(n_cand);
    int found;
    if (n <= kMergeCap) {
        for (int i = tid; i < n; i += kMergeThreads) {
            const Pick me = {cs[i], ck[i], cw[i]};
            int rank = 0;
            for (int q = 0; q < n; ++q)
                rank += before(Pick{cs[q], ck[q], cw[q]}, me);
            if (rank < k)
                emit(rank, me.c, me.w, static_cast<int32_t>(key_token(me.key)));
        }
        found = min(n, k);
    } else {
        // Rows of ties: k rounds over every kept candidate, each taking the
        // best one after the last.
        Pick last = {INFINITY, 0, -1};
        found = 0;
        for (int rank = 0; rank < k; ++rank) {
            Pick best = {-INFINITY, 0, kBeamMax};
            auto offer = [&](const Pick &p) {
                if (before(last, p) && before(p, best))
                    best = p;
            };
            for (int64_t l = l0; l < n_lists; l += kMergeThreads) {
                const int w = static_cast<int>(l / nseg);
                if (!(logd[w] == logd[w]))
                    continue;
                const uint64_t *q = lists + (row0 * nseg + l) * k;
                for (int i = 0; i < k && q[i]; ++i)
                    offer(Pick{score_of(w, q[i]), q[i], w});
            }
            if (tid < W && held(tid))
                offer(Pick{static_cast<double>(sc[tid]), held_key, tid});
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1) {
                const Pick o = {shfl_xor_f64(best.c, off), shfl_xor_u64(best.key, off),
                                __shfl_xor(best.w, off, 64)};
                if (before(o, best))
                    best = o;
            }
            if (lane == 0)
                red[wave] = best;
            __syncthreads();
            best = red[0];
            for (int q = 1; q < NW; ++q)
                if (before(red[q], best))
                    best = red[q];
            __syncthreads();
            if (best.c == -INFINITY)
                break;
            if (tid == 0)
                emit(rank, best.c, best.w, static_cast<int32_t>(key_token(best.key)));
            last = best;
            ++found;
        }
    }
    if (found >= k || wave != 0)
        return;
    // The first positions whose candidate is -inf, in order.
    const uint32_t total = static_cast<uint32_t>(W * V);
    for (uint32_t f0 = 0; f0 < total && found < k; f0 += 64) {
        const uint32_t f = f0 + lane;
        bool none = false;
        const int w = f < total ? static_cast<int>(f / V) : 0;
        const int64_t v = f - static_cast<uint32_t>(w * V);
        if (f < total) {
            if (fin[w]) {
                none = v != eos || !score_alive(sc[w]);
            } else if (!(logd[w] == logd[w])) {
                none = true;
            } else {
                const int64_t at = (row0 + w) * ld + v;
                const float z = bf16 ? __uint_as_float(static_cast<uint32_t>(
                                           static_cast<const uint16_t *>(logits)[at]) << 16)
                                     : static_cast<const float *>(logits)[at];
                none = z == -INFINITY;
            }
        }
        const uint64_t mask = __ballot(none);
        const int pos = found + __popcll(mask & ((1ull << lane) - 1ull));
        if (none && pos < k)
            emit(pos, -INFINITY, w, static_cast<int32_t>(v));
        found += __popcll(mask);
    }
}

// ---------------------------------------------------------------------------
// Reordering.  dst row (o, b W_out + i, h) <- src row (o, b W_in + parent[b][i],
// h), the first live_b bytes of it (live_b = positions x bytes per position).
// A copy, bound by the bytes of the rows that move.  Rows need no alignment: a
// vector starts at any byte (the hardware takes unaligned global accesses),
// and the last live_b % 16 bytes go one by one.
//
// A row takes an odd number of workgroups.  Workgroups go round the eight XCDs
// in turn, so with an even number the same XCDs would always hold the rows'
// ends, which a request's length often cuts off (1 GB of [16][64][8][1024][64]
// BF16 with lengths of 1 .. 1024: 230 -> 159 us).
struct ReorderArgs {
    const char *src;
    char *dst;
    int64_t src_so, src_sr, src_sh;  // strides in bytes: outer, row, head
    int64_t dst_so, dst_sr, dst_sh;
    const int32_t *parent;
    const int32_t *lengths;
    int32_t W_in, W_out;
    int64_t T, pos_bytes;
};

template <int BYTES>
struct VecOf;
template <>
struct VecOf<16> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(1)));
};
template <>
struct VecOf<8> {
    typedef uint32_t type __attribute__((ext_vector_type(2), aligned(1)));
};
template <>
struct VecOf<4> {
    typedef uint32_t type __attribute__((aligned(1)));
};
template <>
struct VecOf<1> {
    typedef uint8_t type;
};

// The result is not read again by this kernel: its stores are marked as
// streamed once (1 GB cache: 219 -> 200 us; marking the loads as well lost what
// a small state's rows gain from the caches, 6.0 -> 8.5 us).
template <int VB>
__device__ __forceinline__ void store_vec(char *p, typename VecOf<VB>::type v)
{
    __builtin_nontemporal_store(v, reinterpret_cast<typename VecOf<VB>::type *>(p));
}

// Into other memory: a workgroup moves 8 KiB of one destination row, two
// vectors a thread.  The destination rows of a request that may share a parent
// are eight workgroups apart, on one XCD, whose L2 then serves the second
// reader.  Unit u = ((o H + h) B + b) blocks_per_row + block; each has W_out
// workgroups.  (1 GB as above: 150 us, 5.9 TB/s; 7 requests x 5 beams of some
// 6 MB: 6.4 us.  All rows of a request in one thread, as in place: 159 and
// 6.9 us; one vector a thread 260 and 8.8 us, four 161 and 6.1 us.)
constexpr int kCopyVecs = 2;

__global__ __launch_bounds__(256) void beam_copy_kernel(ReorderArgs a, uint32_t unit0, uint32_t units,
                                                        uint32_t blocks_per_row, uint32_t B, uint32_t H)
{
    typedef typename VecOf<16>::type vec;
    constexpr int kStep = 256 * 16;
    const uint32_t W = static_cast<uint32_t>(a.W_out);
    const uint32_t eight = blockIdx.x / (8 * W), at8 = blockIdx.x - eight * 8 * W;
    const uint32_t i = at8 / 8, unit = unit0 + eight * 8 + at8 % 8;
    if (unit >= units)
        return;
    const uint32_t ohb = unit / blocks_per_row, blk = unit - ohb * blocks_per_row;
    const uint32_t oh = ohb / B, b = ohb - oh * B;
    const uint32_t o = oh / H, h = oh - o * H;
    const int32_t p = a.parent[static_cast<int64_t>(b) * W + i];
    int64_t len = a.T;
    if (a.lengths)
        len = min(max(static_cast<int64_t>(a.lengths[b]), int64_t{0}), a.T);
    const int64_t at = static_cast<int64_t>(blk) * kStep * kCopyVecs + threadIdx.x * 16;
    const int64_t left = len * a.pos_bytes - at;
    if (left <= 0 || p < 0 || p >= a.W_in)
        return;
    const char *s = a.src + o * a.src_so + (static_cast<int64_t>(b) * a.W_in + p) * a.src_sr + h * a.src_sh + at;
    char *d = a.dst + o * a.dst_so + (static_cast<int64_t>(b) * W + i) * a.dst_sr + h * a.dst_sh + at;
    vec r[kCopyVecs];
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u)
        if (kStep * u + 16 <= left)
            r[u] = *reinterpret_cast<const vec *>(s + kStep * u);
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u) {
        if (kStep * u + 16 <= left)
            store_vec<16>(d + kStep * u, r[u]);
        else
            for (int64_t e = kStep * u; e < kStep * u + 16 && e < left; ++e)
                d[e] = s[e];
    }
}

// In place: one thread moves the same VB bytes of every beam of a request.  It
// reads all the rows it needs before it writes any, so rows may trade places
// with no second buffer, and rows that stay (or have no parent) are neither
// read nor written.
template <int WMAX, int VB>
__device__ __forceinline__ void move_column(char *d, int64_t sr, const int32_t *par, int32_t W)
{
    typedef typename VecOf<VB>::type vec;
    vec r[WMAX];
    uint64_t moves = 0;
#pragma unroll
    for (int i = 0; i < WMAX; ++i) {
        const int32_t p = i < W ? par[i] : -1;
        if (p >= 0 && p < W && p != i) {
            moves |= uint64_t{1} << i;
            r[i] = *reinterpret_cast<const vec *>(d + p * sr);
        }
    }
#pragma unroll
    for (int i = 0; i < WMAX; ++i)
        if ((moves >> i) & 1)
            store_vec<VB>(d + i * sr, r[i]);
}

template <int WMAX, int VB>
__global__ __launch_bounds__(256) void beam_permute_kernel(ReorderArgs a, uint32_t blocks_per_row,
                                                           uint32_t B, uint32_t H)
{
    // blockIdx.x = ((o * H + h) * B + b) * blocks_per_row + block, below 2^23
    const uint32_t slab = blockIdx.x / blocks_per_row, blk = blockIdx.x - slab * blocks_per_row;
    const uint32_t oh = slab / B, b = slab - oh * B;
    const uint32_t o = oh / H, h = oh - o * H;
    int64_t len = a.T;
    if (a.lengths)
        len = min(max(static_cast<int64_t>(a.lengths[b]), int64_t{0}), a.T);
    const int64_t live = len * a.pos_bytes;
    const int64_t at = (static_cast<int64_t>(blk) * 256 + threadIdx.x) * VB;
    if (at >= live)
        return;
    const int32_t *par = a.parent + static_cast<int64_t>(b) * a.W_out;
    char *d = a.dst + o * a.dst_so + static_cast<int64_t>(b) * a.W_out * a.dst_sr + h * a.dst_sh + at;
    if (at + VB <= live) {
        move_column<WMAX, VB>(d, a.dst_sr, par, a.W_out);
    } else {
        for (int64_t e = 0; at + e < live; ++e)
            move_column<WMAX, 1>(d + e, a.dst_sr, par, a.W_out);
    }
}

constexpr int64_t kMaxBlocks = kMaxItems / 256;  // workgroups of 256 per launch

// Workgroups of `bytes` each that a row takes (odd, see above).
int64_t row_blocks(const ReorderArgs &a, int64_t bytes)
{
    return ((a.T * a.pos_bytes + bytes - 1) / bytes) | 1;
}

hipError_t launch_copy(const ReorderArgs &a, int64_t B, int64_t H, int64_t n_outer, hipStream_t s)
{
    const int64_t per_row = row_blocks(a, 256 * 16 * kCopyVecs), per_outer = per_row * B * H;
    if (per_outer > kMaxBlocks)
        return hipErrorInvalidValue;  // refused by the caller's size check
    const int64_t outers = kMaxBlocks / per_outer, most = kMaxBlocks / (8 * a.W_out) * 8;
    for (int64_t o = 0; o < n_outer; o += outers) {
        ReorderArgs q = a;
        q.src += o * a.src_so;
        q.dst += o * a.dst_so;
        const int64_t units = std::min(outers, n_outer - o) * per_outer;
        for (int64_t u = 0; u < units; u += most) {
            const int64_t eights = (std::min(most, units - u) + 7) / 8;
            hipLaunchKernelGGL(beam_copy_kernel, dim3(static_cast<unsigned>(eights * 8 * a.W_out)), dim3(256), 0, s,
                               q, static_cast<uint32_t>(u), static_cast<uint32_t>(units),
                               static_cast<uint32_t>(per_row), static_cast<uint32_t>(B),
                               static_cast<uint32_t>(H));
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess)
                return e;
        }
    }
    return hipSuccess;
}

template <int WMAX, int VB>
hipError_t launch_permute(const ReorderArgs &a, int64_t B, int64_t H, int64_t n_outer, hipStream_t s)
{
    const int64_t per_row = row_blocks(a, 256 * VB), per_outer = per_row * B * H;
    if (per_outer > kMaxBlocks)
        return hipErrorInvalidValue;  // refused by the caller's size check
    const int64_t outers = kMaxBlocks / per_outer;
    for (int64_t o = 0; o < n_outer; o += outers) {
        ReorderArgs q = a;
        q.dst += o * a.dst_so;
        hipLaunchKernelGGL((beam_permute_kernel<WMAX, VB>),
                           dim3(static_cast<unsigned>(std::min(outers, n_outer - o) * per_outer)), dim3(256), 0, s, q,
                           static_cast<uint32_t>(per_row), static_cast<uint32_t>(B), static_cast<uint32_t>(H));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace

int64_t beam_segments(int64_t V)
{
    return (V + kSegCols - 1) / kSegCols;
}

int64_t beam_workspace_bytes(int64_t n_rows, int64_t V, int64_t n_out)
{
    return n_rows * beam_segments(V) * (static_cast<int64_t>(sizeof(SegRecord)) + 8 * n_out);
}

hipError_t launch_beam_select(const void *logits, int64_t ld, bool bf16, int64_t B, int64_t W,
                              int64_t V, const float *scores, const uint8_t *finished, int32_t eos,
                              int64_t n_out, float *out_scores, int32_t *out_parent,
                              int32_t *out_token, uint8_t *out_finished, void *workspace,
                              hipStream_t s)
{
    const int64_t nseg = beam_segments(V), waves = B * W * nseg;
    SegRecord *rec = static_cast<SegRecord *>(workspace);
    uint64_t *lists = reinterpret_cast<uint64_t *>(rec + waves);
    const dim3 grid(static_cast<unsigned>(waves)), block(64);
    const int32_t k = static_cast<int32_t>(n_out), nc = static_cast<int32_t>(nseg);
    if (bf16)
        hipLaunchKernelGGL((beam_scan_kernel<true>), grid, block, 0, s, logits, ld, V, static_cast<uint32_t>(nseg),
                           scores, finished, k, rec, lists);
    else
        hipLaunchKernelGGL((beam_scan_kernel<false>), grid, block, 0, s, logits, ld, V, static_cast<uint32_t>(nseg),
                           scores, finished, k, rec, lists);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    // A workgroup per request: more requests than one launch's work-items cover
    // take several.
    const int64_t most = kMaxItems / kMergeThreads, esz = bf16 ? 2 : 4;
    for (int64_t b = 0; b < B; b += most) {
        const int64_t r = b * W, o = b * n_out;
        hipLaunchKernelGGL(beam_merge_kernel, dim3(static_cast<unsigned>(std::min(most, B - b))),
                           dim3(kMergeThreads), 0, s, static_cast<const char *>(logits) + r * ld * esz, ld,
                           bf16 ? 1 : 0, static_cast<int32_t>(W), V, nc, scores + r,
                           finished ? finished + r : nullptr, eos, k, rec + r * nseg, lists + r * nseg * n_out,
                           out_scores + o, out_parent + o, out_token + o, out_finished + o);
        const hipError_t em = hipGetLastError();
        if (em != hipSuccess)
            return em;
    }
    return hipSuccess;
}

hipError_t launch_beam_reorder(const void *src, void *dst, const int64_t (&src_strides)[3],
                               const int64_t (&dst_strides)[3], const int32_t *parent,
                               const int32_t *lengths, int64_t n_outer, int64_t B, int64_t W_in,
                               int64_t W_out, int64_t H, int64_t T, int64_t pos_bytes, hipStream_t s)
{
    ReorderArgs a;
    a.src = static_cast<const char *>(src);
    a.dst = static_cast<char *>(dst);
    a.src_so = src_strides[0], a.src_sr = src_strides[1], a.src_sh = src_strides[2];
    a.dst_so = dst_strides[0], a.dst_sr = dst_strides[1], a.dst_sh = dst_strides[2];
    a.parent = parent;
    a.lengths = lengths;
    a.W_in = static_cast<int32_t>(W_in);
    a.W_out = static_cast<int32_t>(W_out);
    a.T = T;
    a.pos_bytes = pos_bytes;
    if (src != dst)
        return launch_copy(a, B, H, n_outer, s);
    // The rows of one column stay in registers: narrower columns for more beams.
    if (W_out <= 4)
        return launch_permute<4, 16>(a, B, H, n_outer, s);
    if (W_out <= 8)
        return launch_permute<8, 16>(a, B, H, n_outer, s);
    if (W_out <= 16)
        return launch_permute<16, 16>(a, B, H, n_outer, s);
    if (W_out <= 32)
        return launch_permute<32, 8>(a, B, H, n_outer, s);
    return launch_permute<64, 4>(a, B, H, n_outer, s);
}

}  // namespace lmh
