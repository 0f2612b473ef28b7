// beam.hip -- beam search over the output layer's logits on gfx950: the
// selection of the next beams (scan + merge) and the reordering of per-beam
// states that follows it.
//
// Selection, per request b with W beams over V tokens:
//   c(w, v) = s_w + (z_wv - logZ_w),  logZ_w = m_w + log sum_v exp(z_wv - m_w)
// and the n_out largest c in descending order, equal ones by ascending
// w V + v.  Within a beam the order of c is the order of z, so one pass over
// the logits suffices: every wave reads one segment of a row into registers
// and leaves the segment's {max, sum of exponentials} and its n_out largest
// logits; a second kernel folds the sums, turns the kept logits into scores
// and picks the winners.  Which candidate wins must not depend on rounding,
// so sums, logZ and scores are FP64 (the logits enter exactly); only the
// returned score is rounded, once, to FP32.
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

constexpr int kBeamMax = 64;       // beams per request, and beams selected
constexpr int kScanWaves = 4;      // waves per scan workgroup
constexpr int kCandCap = 512;      // candidates a wave can rank at once

struct SegRecord {
    double d;  // sum over the segment of exp(z - m); NaN: the row holds NaN or +inf
    float m;   // max of the segment
    float pad;
};
static_assert(sizeof(SegRecord) == 16, "one 16-byte record per segment");

// FP32 -> uint32 with the same order (-0 and +0 equal); 0 lies below -inf.
__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
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

// True when the beam can offer a candidate above -inf by its score alone.
__device__ __forceinline__ bool score_alive(float s)
{
    return s > -INFINITY && s < INFINITY;  // false for NaN
}

// Reads PER values of the segment [j0, j0 + 64 PER) of a row: lane l holds, in
// v[4 u + e] (FP32) or v[8 u + e] (BF16), column j0 + (64 u + l) * G + e with G
// values per 16-byte load; columns at or past V read as -inf.
template <bool BF16, int PER>
__device__ __forceinline__ void load_segment(const void *row, int64_t V, int64_t j0, int lane,
                                             float (&v)[PER])
{
    constexpr int G = BF16 ? 8 : 4;
    if (j0 + 64 * PER <= V) {
#pragma unroll
        for (int u = 0; u < PER / G; ++u) {
            const int64_t j = j0 + static_cast<int64_t>(64 * u + lane) * G;
            if constexpr (BF16) {
                const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + j);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[8 * u + 2 * e] = __uint_as_float(w[e] << 16);
                    v[8 * u + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                }
            } else {
                const float4 q = *reinterpret_cast<const float4 *>(static_cast<const float *>(row) + j);
                v[4 * u] = q.x, v[4 * u + 1] = q.y, v[4 * u + 2] = q.z, v[4 * u + 3] = q.w;
            }
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < PER / G; ++u) {
        const int64_t j = j0 + static_cast<int64_t>(64 * u + lane) * G;
#pragma unroll
        for (int e = 0; e < G; ++e) {
            float x = -INFINITY;
            if (j + e < V) {
                if constexpr (BF16)
                    x = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(row)[j + e]) << 16);
                else
                    x = static_cast<const float *>(row)[j + e];
            }
            v[G * u + e] = x;
        }
    }
}

// One wave per (row, segment of 64 PER columns).  Bound by the one read of the
// logits: the wave keeps its segment in registers, so the maximum, the
// exponentials and the candidates cost no second read, and nothing is shared
// between waves (no barrier).
// Candidates: the n_out-th largest of the 64 lane maxima is a lower bound of
// the segment's n_out-th largest value (that many lanes hold a value at least
// as large), cut to its upper 16 bits so that 16 ballots find it; the few
// values at or above it are collected in LDS and ranked by counting.  Lists
// are in descending value, equal values in ascending column.
template <bool BF16, int PER>
__global__ __launch_bounds__(kScanWaves * 64) void beam_scan_kernel(
    const void *__restrict__ logits, int64_t ld, int64_t n_rows, int64_t V, int32_t nseg,
    const float *__restrict__ scores, const uint8_t *__restrict__ finished, int32_t k,
    SegRecord *__restrict__ rec, uint64_t *__restrict__ lists)
{
    constexpr int G = BF16 ? 8 : 4;
    __shared__ uint64_t cand[kScanWaves][kCandCap];
    __shared__ uint32_t count[kScanWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kScanWaves + wave;
    if (id >= n_rows * nseg)
        return;
    const int64_t row = id / nseg;
    const int64_t j0 = (id - row * nseg) * (64 * PER);
    if (!score_alive(scores[row]) || (finished && finished[row]))
        return;  // the merge does not read this beam's records

    float v[PER];
    load_segment<BF16, PER>(static_cast<const char *>(logits) + row * ld * (BF16 ? 2 : 4), V, j0, lane, v);

    float lm = v[0];
#pragma unroll
    for (int i = 1; i < PER; ++i)
        lm = __builtin_elementwise_maximum(lm, v[i]);  // NaN stays NaN
    float m = lm;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        m = __builtin_elementwise_maximum(m, __shfl_xor(m, off, 64));
    uint64_t *out = lists + id * k;
    if (!(m < INFINITY) || m == -INFINITY) {
        // NaN or +inf somewhere (the whole row then offers nothing), or only
        // -inf: no candidates.
        if (lane == 0) {
            rec[id].m = m;
            rec[id].d = (m == -INFINITY) ? 0.0 : static_cast<double>(NAN);
        }
        for (int i = lane; i < k; i += 64)
            out[i] = 0;
        return;
    }

    const double md = static_cast<double>(m);
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        d += exp_nonpos(static_cast<double>(v[i]) - md);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        d += shfl_xor_f64(d, off);
    if (lane == 0) {
        rec[id].m = m;
        rec[id].d = d;
    }

    // Largest t (upper 16 bits) that at least k lane maxima reach, but above
    // the key of -inf.
    const uint32_t mykey = order_key(lm);
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b >= 16; --b) {
        const uint32_t c = t | (1u << b);
        if (__popcll(__ballot(mykey >= c)) >= k)
            t = c;
    }
    t = max(t, order_key(-INFINITY) + 1u);
    const float tv = key_value(t);

    if (lane == 0)
        count[wave] = 0;
    __builtin_amdgcn_wave_barrier();
    uint64_t *mine = cand[wave];
    if (lm >= tv) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (v[i] >= tv) {
                const uint32_t at = atomicAdd(&count[wave], 1u);
                const uint32_t col = static_cast<uint32_t>(j0) + (64 * (i / G) + lane) * G + i % G;
                if (at < kCandCap)
                    mine[at] = (static_cast<uint64_t>(order_key(v[i])) << 32) | (0xffffffffu - col);
            }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int n = static_cast<int>(__builtin_amdgcn_readfirstlane(count[wave]));
    if (n <= kCandCap) {
        for (int i = lane; i < n; i += 64) {
            const uint64_t key = mine[i];
            int rank = 0;
            for (int q = 0; q < n; ++q)
                rank += mine[q] > key;
            if (rank < k)
                out[rank] = key;
        }
        for (int i = n + lane; i < k; i += 64)
            out[i] = 0;
        return;
    }
    // Too many equal values at the bound (rows of ties): k rounds, each taking
    // the largest key below the last one.
    uint64_t last = ~0ull;
    for (int rank = 0; rank < k; ++rank) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t col = static_cast<uint32_t>(j0) + (64 * (i / G) + lane) * G + i % G;
            const uint64_t key = (static_cast<uint64_t>(order_key(v[i])) << 32) | (0xffffffffu - col);
            if (v[i] > -INFINITY && key < last && key > best)
                best = key;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            best = max(best, shfl_xor_u64(best, off));
        if (lane == 0)
            out[rank] = best;
        last = best;
    }
}

// (a, fa) before (b, fb): larger score, equal scores by ascending position.
__device__ __forceinline__ bool before(double a, uint32_t fa, double b, uint32_t fb)
{
    return a > b || (a == b && fa < fb);
}

constexpr int kMergeThreads = 256;
constexpr int kMergeCap = 1024;

// One workgroup per request: logZ of every beam from its segments' records,
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
    __shared__ double logz[kBeamMax];     // NaN: no candidate above -inf
    __shared__ float sc[kBeamMax];
    __shared__ uint8_t fin[kBeamMax];
    __shared__ uint32_t group[64];
    __shared__ double cs[kMergeCap];
    __shared__ uint32_t cf[kMergeCap];
    __shared__ uint32_t n_cand;
    __shared__ double red_c[NW];
    __shared__ uint32_t red_f[NW];

    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t row0 = b * W;
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
        double lz = static_cast<double>(NAN);
        if (!fin[w] && score_alive(sc[w])) {
            const SegRecord *r = rec + (row0 + w) * nseg;
            float m = -INFINITY;
            for (int s = lane; s < nseg; s += 64)
                m = __builtin_elementwise_maximum(m, r[s].m);
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1)
                m = __builtin_elementwise_maximum(m, __shfl_xor(m, off, 64));
            if (m > -INFINITY && m < INFINITY) {
                double d = 0.0;
                for (int s = lane; s < nseg; s += 64)
                    d += r[s].d * exp_nonpos(static_cast<double>(r[s].m) - static_cast<double>(m));
#pragma unroll
                for (int off = 32; off >= 1; off >>= 1)
                    d += shfl_xor_f64(d, off);
                lz = static_cast<double>(m) + log(d);
            }
        }
        if (lane == 0)
            logz[w] = lz;
    }
    __syncthreads();

    // Lists 0 .. W nseg - 1 (beam l / nseg), then one per finished beam; list l
    // is walked by thread (l % 64) * 4 + (l / 64) % 4, so that the 64 groups of
    // four threads share the lists evenly.
    const int64_t n_lists = static_cast<int64_t>(W) * nseg;
    const int64_t l0 = (tid >> 2) + 64 * (tid & 3);
    auto score_of = [&](int w, uint64_t key) {
        return static_cast<double>(sc[w]) +
               (static_cast<double>(key_value(static_cast<uint32_t>(key >> 32))) - logz[w]);
    };
    auto flat_of = [&](int w, uint64_t key) {
        return static_cast<uint32_t>(w * V) + (0xffffffffu - static_cast<uint32_t>(key));
    };
    // A finished beam's one candidate.
    auto held = [&](int w) { return fin[w] && score_alive(sc[w]) && eos >= 0 && eos < V; };

    double head = -INFINITY;
    for (int64_t l = l0; l < n_lists; l += kMergeThreads) {
        const int w = static_cast<int>(l / nseg);
        if (logz[w] == logz[w]) {
            const uint64_t key = lists[(row0 * nseg + l) * k];
            if (key)
                head = fmax(head, score_of(w, key));
        }
    }
    if (tid < W && held(tid))
        head = fmax(head, static_cast<double>(sc[tid]));
    // Rounded down, so that a bound on the rounded heads bounds the scores.
    if (head > -INFINITY)
        atomicMax(&group[tid >> 2], order_key(__double2float_rd(head)));
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
    t = max(t, order_key(-INFINITY) + 1u);
    const double tv = static_cast<double>(key_value(t));
    auto append = [&](double c, uint32_t f) {
        const uint32_t at = atomicAdd(&n_cand, 1u);
        if (at < kMergeCap) {
            cs[at] = c;
            cf[at] = f;
        }
    };
    if (head >= tv) {
        for (int64_t l = l0; l < n_lists; l += kMergeThreads) {
            const int w = static_cast<int>(l / nseg);
            if (!(logz[w] == logz[w]))
                continue;
            const uint64_t *q = lists + (row0 * nseg + l) * k;
            for (int i = 0; i < k; ++i) {
                const uint64_t key = q[i];
                if (!key)
                    break;
                const double c = score_of(w, key);
                if (c < tv)
                    break;
                append(c, flat_of(w, key));
            }
        }
        if (tid < W && held(tid) && static_cast<double>(sc[tid]) >= tv)
            append(static_cast<double>(sc[tid]), static_cast<uint32_t>(tid * V) + static_cast<uint32_t>(eos));
    }
    __syncthreads();

    auto emit = [&](int i, double c, uint32_t f) {
        const int w = static_cast<int>(f / V);
        const int32_t tok = static_cast<int32_t>(f - static_cast<uint32_t>(w * V));
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
            const double c = cs[i];
            const uint32_t f = cf[i];
            int rank = 0;
            for (int q = 0; q < n; ++q)
                rank += before(cs[q], cf[q], c, f);
            if (rank < k)
                emit(rank, c, f);
        }
        found = min(n, k);
    } else {
        // Rows of ties: k rounds over every kept candidate, each taking the
        // best one after the last.
        double lc = INFINITY;
        uint32_t lf = 0;
        found = 0;
        for (int rank = 0; rank < k; ++rank) {
            double bc = -INFINITY;
            uint32_t bf = 0xffffffffu;
            auto offer = [&](double c, uint32_t f) {
                if ((rank == 0 || before(lc, lf, c, f)) && before(c, f, bc, bf))
                    bc = c, bf = f;
            };
            for (int64_t l = l0; l < n_lists; l += kMergeThreads) {
                const int w = static_cast<int>(l / nseg);
                if (!(logz[w] == logz[w]))
                    continue;
                const uint64_t *q = lists + (row0 * nseg + l) * k;
                for (int i = 0; i < k && q[i]; ++i)
                    offer(score_of(w, q[i]), flat_of(w, q[i]));
            }
            if (tid < W && held(tid))
                offer(static_cast<double>(sc[tid]), static_cast<uint32_t>(tid * V) + static_cast<uint32_t>(eos));
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1) {
                const double oc = shfl_xor_f64(bc, off);
                const uint32_t of = __shfl_xor(bf, off, 64);
                if (before(oc, of, bc, bf))
                    bc = oc, bf = of;
            }
            if (lane == 0)
                red_c[wave] = bc, red_f[wave] = bf;
            __syncthreads();
            bc = red_c[0], bf = red_f[0];
            for (int q = 1; q < NW; ++q)
                if (before(red_c[q], red_f[q], bc, bf))
                    bc = red_c[q], bf = red_f[q];
            __syncthreads();
            if (bc == -INFINITY)
                break;
            if (tid == 0)
                emit(rank, bc, bf);
            lc = bc, lf = bf;
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
        if (f < total) {
            const int w = static_cast<int>(f / V);
            const int64_t v = f - static_cast<uint32_t>(w * V);
            if (fin[w]) {
                none = v != eos || !score_alive(sc[w]);
            } else if (!(logz[w] == logz[w])) {
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
            emit(pos, -INFINITY, f);
        found += __popcll(mask);
    }
}

// ---------------------------------------------------------------------------
// Reordering.  dst row (o, b W_out + i, h) <- src row (o, b W_in + parent[b][i],
// h), the first live_b bytes of it (live_b = positions x bytes per position).
// One thread moves the same 16 (8, 4) bytes of every beam of a request: in
// place it reads all the rows it needs before it writes any, so rows may trade
// places with no second buffer, and rows that stay are neither read nor
// written.  A copy, bound by the bytes of the rows that move.  Rows need no
// alignment: a vector starts at any byte (the hardware takes unaligned
// global accesses), and the last live_b % 16 bytes go one by one.
struct ReorderArgs {
    const char *src;
    char *dst;
    int64_t src_so, src_sr, src_sh;  // strides in bytes: outer, row, head
    int64_t dst_so, dst_sr, dst_sh;
    const int32_t *parent;
    const int32_t *lengths;
    int64_t B;
    int32_t W_in, W_out;
    int64_t H, T, pos_bytes;
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

template <int WMAX, int VB, bool IN_PLACE>
__device__ __forceinline__ void move_column(const char *s, char *d, int64_t ssr, int64_t dsr,
                                            const int32_t *par, int32_t W_in, int32_t W_out)
{
    typedef typename VecOf<VB>::type vec;
    if constexpr (IN_PLACE) {
        vec r[WMAX];
#pragma unroll
        for (int i = 0; i < WMAX; ++i) {
            const int32_t p = i < W_out ? par[i] : -1;
            if (p >= 0 && p < W_in && p != i)
                r[i] = *reinterpret_cast<const vec *>(s + p * ssr);
        }
#pragma unroll
        for (int i = 0; i < WMAX; ++i) {
            const int32_t p = i < W_out ? par[i] : -1;
            if (p >= 0 && p < W_in && p != i)
                *reinterpret_cast<vec *>(d + i * dsr) = r[i];
        }
    } else {
        for (int i0 = 0; i0 < W_out; i0 += 4) {
            vec r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t p = i0 + i < W_out ? par[i0 + i] : -1;
                if (p >= 0 && p < W_in)
                    r[i] = *reinterpret_cast<const vec *>(s + p * ssr);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t p = i0 + i < W_out ? par[i0 + i] : -1;
                if (p >= 0 && p < W_in)
                    *reinterpret_cast<vec *>(d + (i0 + i) * dsr) = r[i];
            }
        }
    }
}

template <int WMAX, int VB, bool IN_PLACE>
__global__ __launch_bounds__(256) void beam_reorder_kernel(ReorderArgs a, int64_t blocks_per_row)
{
    // blockIdx.x = ((o * H + h) * B + b) * blocks_per_row + block
    const int64_t id = blockIdx.x;
    const int64_t slab = id / blocks_per_row;
    const int64_t blk = id - slab * blocks_per_row;
    const int64_t oh = slab / a.B;
    const int64_t b = slab - oh * a.B;
    const int64_t o = oh / a.H;
    const int64_t h = oh - o * a.H;
    int64_t len = a.T;
    if (a.lengths)
        len = min(max(static_cast<int64_t>(a.lengths[b]), int64_t{0}), a.T);
    const int64_t live = len * a.pos_bytes;
    const int64_t at = (blk * 256 + threadIdx.x) * VB;
    if (at >= live)
        return;
    const int32_t *par = a.parent + b * a.W_out;
    const char *s = a.src + o * a.src_so + b * a.W_in * a.src_sr + h * a.src_sh + at;
    char *d = a.dst + o * a.dst_so + b * a.W_out * a.dst_sr + h * a.dst_sh + at;
    if (at + VB <= live) {
        move_column<WMAX, VB, IN_PLACE>(s, d, a.src_sr, a.dst_sr, par, a.W_in, a.W_out);
    } else {
        for (int64_t e = 0; at + e < live; ++e)
            move_column<WMAX, 1, IN_PLACE>(s + e, d + e, a.src_sr, a.dst_sr, par, a.W_in, a.W_out);
    }
}

template <int WMAX, int VB, bool IN_PLACE>
hipError_t launch_reorder(const ReorderArgs &a, int64_t n_outer, hipStream_t s)
{
    const int64_t per_row = (a.T * a.pos_bytes + 256 * VB - 1) / (256 * VB);
    const int64_t slabs = n_outer * a.H * a.B;
    constexpr int64_t kMaxBlocks = (int64_t{1} << 31) / 256;
    // Several launches over outer blocks where one would pass 2^31 work-items.
    if (per_row > kMaxBlocks || slabs / n_outer > kMaxBlocks / per_row)
        return hipErrorInvalidValue;  // refused by the caller's size check
    const int64_t per_launch = std::max<int64_t>(1, kMaxBlocks / (per_row * a.H * a.B));
    for (int64_t o = 0; o < n_outer; o += per_launch) {
        const int64_t no = std::min(per_launch, n_outer - o);
        ReorderArgs q = a;
        q.src += o * a.src_so;
        q.dst += o * a.dst_so;
        hipLaunchKernelGGL((beam_reorder_kernel<WMAX, VB, IN_PLACE>),
                           dim3(static_cast<unsigned>(no * a.H * a.B * per_row)), dim3(256), 0, s, q, per_row);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace

// Columns per scan segment (64 lanes x PER).
constexpr int kSegCols = 2048;

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
    const unsigned blocks = static_cast<unsigned>((waves + kScanWaves - 1) / kScanWaves);
    const int32_t k = static_cast<int32_t>(n_out), ns = static_cast<int32_t>(nseg);
    if (bf16)
        hipLaunchKernelGGL((beam_scan_kernel<true, kSegCols / 64>), dim3(blocks), dim3(kScanWaves * 64), 0, s,
                           logits, ld, B * W, V, ns, scores, finished, k, rec, lists);
    else
        hipLaunchKernelGGL((beam_scan_kernel<false, kSegCols / 64>), dim3(blocks), dim3(kScanWaves * 64), 0, s,
                           logits, ld, B * W, V, ns, scores, finished, k, rec, lists);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(beam_merge_kernel, dim3(static_cast<unsigned>(B)), dim3(kMergeThreads), 0, s, logits,
                       ld, bf16 ? 1 : 0, static_cast<int32_t>(W), V, ns, scores, finished, eos, k, rec,
                       lists, out_scores, out_parent, out_token, out_finished);
    return hipGetLastError();
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
    a.B = B;
    a.W_in = static_cast<int32_t>(W_in);
    a.W_out = static_cast<int32_t>(W_out);
    a.H = H;
    a.T = T;
    a.pos_bytes = pos_bytes;
    if (src != dst)
        return launch_reorder<4, 16, false>(a, n_outer, s);
    // In place the rows of one column stay in registers: narrower columns for
    // more beams.
    if (W_out <= 4)
        return launch_reorder<4, 16, true>(a, n_outer, s);
    if (W_out <= 8)
        return launch_reorder<8, 16, true>(a, n_outer, s);
    if (W_out <= 16)
        return launch_reorder<16, 16, true>(a, n_outer, s);
    if (W_out <= 32)
        return launch_reorder<32, 8, true>(a, n_outer, s);
    return launch_reorder<64, 4, true>(a, n_outer, s);
}

}  // namespace lmh
