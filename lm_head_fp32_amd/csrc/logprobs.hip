// logprobs.hip -- log-probabilities of given tokens on gfx950, with the rows'
// entropies, the tokens' ranks and the most likely alternatives, and their
// gradient.
//
// Per row, with the temperature T (1 unless given) and x_j = (z_j - m) / T:
//   m = max_j z_j,  d = sum_j exp(x_j),  s = sum_j x_j exp(x_j)
//   log p_j = x_j - log d,  H = -sum_j p_j log p_j = log d - s / d
// (both terms of H are at least 0, so nothing cancels).  d and s come from one
// pass, each lane's about its own running maximum, and are rescaled where it moves
// and where lanes and waves meet: d by f = exp((m_l - m) / T), s to
// f (s + (m_l - m) / T d).  A lane's and a wave's sums are FP32, from there on FP64.
// The order of the logits is the order of the log-probabilities, so ranks and
// alternatives are found on the logits themselves and no rounding decides them:
// equal logits rank by ascending column.
// Gradient of g log p_y + h H:
//   dz_j = (1 / T) [ g ([j == y] - p_j) - h p_j (log p_j + H) ].
#include "common.h"
#include "rows.h"

#include <math.h>

#include <algorithm>
#include <type_traits>

namespace lmh {

namespace {

constexpr int64_t kMaxItems = int64_t{1} << 31;  // work-items per launch
constexpr float kLn2 = 0.6931471805599453f;

// What a wave leaves of a segment of a row: y in place of x in units of log 2.
struct alignas(16) LogprobRecord {
    float m;       // maximum; -inf: nothing above -inf
    float d;       // sum of 2^y, y = (z - m) / T / ln 2; NaN: it holds NaN or +inf
    float s;       // sum of y 2^y
    uint32_t before;  // columns that rank before the row's token
};

// Running sums of a lane: d = sum 2^y, s = sum y 2^y about the lane's own maximum m
// (shift 0 while nothing lies above -inf), rescaled once per 32 values.
struct LaneSums {
    float m = -INFINITY, d = 0.0f, s = 0.0f;
    __device__ __forceinline__ void add(const float (&v)[32], float lm, float c)
    {
        const float mn = __builtin_elementwise_maximum(m, lm);
        const float ms = mn == -INFINITY ? 0.0f : mn;
        const float dy = __builtin_elementwise_maximum((m - ms) * c, kNoTerm);
        const float f = __builtin_amdgcn_exp2f(dy);
        float dn[2] = {0.0f, 0.0f}, sn[2] = {0.0f, 0.0f};  // two chains each
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float y = __builtin_elementwise_maximum((v[i] - ms) * c, kNoTerm);
            const float e = __builtin_amdgcn_exp2f(y);
            dn[i & 1] += e;
            sn[i & 1] = fmaf(e, y, sn[i & 1]);
        }
        s = fmaf(f, fmaf(dy, d, s), sn[0] + sn[1]);
        d = fmaf(d, f, dn[0] + dn[1]);
        m = mn;
    }
};

constexpr int kWaveCap = 256;  // candidates a wave keeps in LDS
constexpr int kListCap = 512;  // candidates of a workgroup that are ranked by counting

// The largest t with at least k of the wave's values (N a lane) >= t, cut to its
// upper 20 bits: a lower bound of the k-th largest, two bits a step.
template <int N>
__device__ __forceinline__ uint32_t kth_largest(const uint32_t (&mine)[N], int k)
{
    uint32_t t = 0;
    auto reach = [&](uint32_t c) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            n += __popcll(__ballot(mine[i] >= c));
        return n >= k;
    };
#pragma unroll
    for (int b = 30; b >= 12; b -= 2) {
        const uint32_t c1 = t | (1u << b), c2 = t | (2u << b), c3 = t | (3u << b);
        const bool r1 = reach(c1), r2 = reach(c2), r3 = reach(c3);
        t = r3 ? c3 : r2 ? c2 : r1 ? c1 : t;
    }
    return t;
}

// A workgroup's slots: 64, or 128 for more than 32 alternatives (the bound would
// have a rank of up to 64 ln 64 = 266 otherwise; of 128 slots it is 128 ln 2 = 89).
constexpr int kFewTop = 32;
__device__ __forceinline__ uint32_t slots_bound(const uint32_t *slot, int lane, int k)
{
    if (k <= kFewTop)
        return kth_largest<1>({slot[lane]}, k);
    return kth_largest<2>({slot[lane], slot[lane + 64]}, k);
}

// The k largest of n keys (n <= kWaveCap, all different) to the front of the
// list, by one wave; returns how many that are.
__device__ __forceinline__ int keep_k(uint64_t *list, int n, int k, int lane)
{
    uint64_t key[kWaveCap / 64];
    int rank[kWaveCap / 64];
#pragma unroll
    for (int i = 0; i < kWaveCap / 64; ++i) {
        key[i] = lane + 64 * i < n ? list[lane + 64 * i] : 0;
        rank[i] = 0;
    }
    for (int q = 0; q < n; ++q) {
        const uint64_t other = list[q];
#pragma unroll
        for (int i = 0; i < kWaveCap / 64; ++i)
            rank[i] += other > key[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < kWaveCap / 64; ++i)
        if (key[i] != 0 && rank[i] < k)
            list[rank[i]] = key[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return min(n, k);
}

// The keys of a segment that are at least `least` into the wave's list, however
// many they are (more equal values at the bound than are wanted, or a large k): read
// again, 64 columns at a time; a full list is cut to its k largest, which then bound
// what is still to come in the segment.  Rows that come here in every segment are slow: of
// 777 x 50001, ten alternatives, rows of masks at the type's lowest value but for five
// columns take 278 us, rows in ascending order 730, where others take 35.
template <bool BF16>
__device__ __forceinline__ int collect_all(const char *zr, int64_t V, int64_t j0, uint64_t least,
                                           uint64_t *list, int n, int k, int lane)
{
    for (int64_t j = j0 + lane; j < j0 + kSegCols; j += 64) {
        uint64_t key = 0;
        if (j < V)
            key = (static_cast<uint64_t>(order_key(row_element<BF16>(zr, j))) << 32) |
                  (0xffffffffu - static_cast<uint32_t>(j));
        uint64_t mask = __ballot(key >= least);
        if (n + __popcll(mask) > kWaveCap) {
            n = keep_k(list, n, k, lane);
            least = max(least, list[k - 1]);
            mask = __ballot(key >= least);
        }
        if (mask & (1ull << lane))
            list[n + __popcll(mask & ((1ull << lane) - 1ull))] = key;
        n += __popcll(mask);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    return n;
}

// A row's sums, folded by one wave; every lane holds them.
struct RowSums {
    float m;
    double d, s;
    uint32_t before;
};

__device__ __forceinline__ RowSums fold(const LogprobRecord *r, int32_t n, int lane, float c)
{
    float m = -INFINITY;
    for (int i = lane; i < n; i += 64)
        m = __builtin_elementwise_maximum(m, r[i].m);
    m = wave_maximum(m);
    double d = 0.0, s = 0.0;
    uint32_t before = 0;
    for (int i = lane; i < n; i += 64) {
        const LogprobRecord q = r[i];
        const float dy = __builtin_elementwise_maximum((q.m - m) * c, kNoTerm);
        const double f = __builtin_amdgcn_exp2f(dy);
        if (q.d != 0.0f) {  // NaN too
            d += f * q.d;
            s += f * (static_cast<double>(q.s) + static_cast<double>(dy) * q.d);
        }
        before += q.before;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        before += __shfl_xor(before, off, 64);
    return {m, wave_sum(d), wave_sum(s), before};
}

// What a row's sums say, written by one lane.
struct RowOutputs {
    float *logprob, *entropy;
    int32_t *rank;
    float4 *stats;
    float *top_logprob;
    int32_t *top_token;
};
__device__ __forceinline__ void write_row(const RowSums &q, float log_d, float inv_t, const char *zr,
                                          bool bf16, int64_t V, const int32_t *token, int32_t ignore_index,
                                          int64_t row, const RowOutputs &o)
{
    const float nan = __int_as_float(0x7fc00000);
    const bool bad = !(q.d > 0.0);
    const float entropy = bad ? nan : log_d - kLn2 * (static_cast<float>(q.s) / static_cast<float>(q.d));
    float lp = 0.0f;
    int32_t rank = -1;
    if (token) {
        const int32_t y = token[row];
        if (y == ignore_index) {
            lp = 0.0f;
        } else if (y < 0 || y >= V || bad) {
            lp = nan;
        } else {
            const float zy = bf16 ? row_element<true>(zr, y) : row_element<false>(zr, y);
            lp = static_cast<float>((static_cast<double>(zy) - q.m) * inv_t - log_d);
            if (o.rank) {
                rank = static_cast<int32_t>(q.before);
                for (int32_t j = y & (bf16 ? ~7 : ~3); j < y; ++j)
                    rank += (bf16 ? row_element<true>(zr, j) : row_element<false>(zr, j)) == zy;
            }
        }
    }
    o.stats[row] = make_float4(q.m, static_cast<float>(q.d), entropy, lp);
    if (o.logprob)
        o.logprob[row] = lp;
    if (o.entropy)
        o.entropy[row] = entropy;
    if (o.rank)
        o.rank[row] = rank;
}

// One workgroup of NW waves per (row, part of its segments of 2048 columns); a wave
// takes every NW-th segment of the part, the next one's loads under way.  With one
// part per row the workgroup writes the row's results, else a record and its k
// largest for the merge.  Bound by the one read of the logits where rows are many and
// long: 8192 x 131072 FP32 in 620 us, 6.9 TB/s (plain loads in place of non-temporal
// ones: 690); 2048 x 50001 with ten alternatives and ranks in 68 us, 6.0 TB/s.  A value
// takes 8.0 vector instructions a lane, with alternatives and a rank 12.2 (counted, the
// row's start and end among them); of BF16 rows of 16000 columns, two rounds a row, 10.8
// and 17.3, and these bound them: 8192 x 16000 take 46 - 48 us with the vector units
// busy all the while (the read is 36), with both 77 - 86, busy for 0.78 of it.  777 rows
// of 50001 are three to a CU and take 28 us, with both 35: 4.4 TB/s.  One row of 32768
// is the latency of one workgroup, 5 us, 8 with alternatives.  Many short rows are
// latency as well: 8192 x 1000 in 11 - 12 us, with ten alternatives 18, with 64 27 (the
// read is 4.6).
// Alternatives: slot[l] is the largest value that lane l of any wave has seen (for
// larger k two slots, for the halves of its values), so the k-th largest of the
// slots is a lower bound of the k-th largest value (k different values reach it),
// whatever the waves have read so far.  It is taken in the first, second, fourth, ...
// round of NW segments, still in registers (every round: 38.6 instead of 35.5 us for 777
// rows of 50001, ten alternatives); the few values that reach it are kept per wave, and at the end those
// that reach the last bound are ranked by counting.
template <bool BF16, bool TOP, bool RANK, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(4))) void logprobs_row_kernel(
    const void *__restrict__ logits, int64_t ld, int64_t V, uint32_t parts, int32_t part_segs,
    const int32_t *__restrict__ token, int32_t ignore_index, const float *__restrict__ temperature,
    int64_t temperature_stride, int32_t k, LogprobRecord *__restrict__ rec, uint64_t *__restrict__ lists,
    RowOutputs o)
{
    constexpr int G = Segment<BF16>::G;
    __shared__ uint64_t kept[TOP ? NW * kWaveCap : 1];
    __shared__ uint64_t cand[TOP ? kListCap : 1];
    __shared__ uint64_t red[NW];
    __shared__ uint32_t slot[128];
    __shared__ LogprobRecord part_rec[NW];
    __shared__ uint32_t cand_n;
    __shared__ float sh_log_d;
    __shared__ float sh_m;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t id = blockIdx.x, row = id / parts;
    const int32_t seg0 = static_cast<int32_t>(id - row * parts) * part_segs;
    const int32_t seg1 = min(seg0 + part_segs, static_cast<int32_t>((V + kSegCols - 1) / kSegCols));
    const char *zr = static_cast<const char *>(logits) + static_cast<int64_t>(row) * ld * (16 / G);

    Segment<BF16, true> next;
    int32_t seg = seg0 + wave;
    next.load(zr, V, static_cast<int64_t>(seg) * kSegCols, lane);
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const float c = kLog2e * inv_t;
    int32_t y = -1;
    float zy = INFINITY, above = INFINITY;  // above: the next FP32 value
    if constexpr (RANK) {
        y = token[row];
        if (y >= 0 && y < V) {
            zy = row_element<BF16>(zr, y);
            above = key_value(order_key(zy) + 1u);
        } else {
            y = -1;
        }
    }
    if constexpr (TOP) {
        for (int i = tid; i < 128; i += NW * 64)
            slot[i] = 0;
        for (int i = tid; i < kListCap; i += NW * 64)
            cand[i] = 0;
        if (tid == 0)
            cand_n = 0;
        __syncthreads();
    }
    uint64_t *mine = kept + wave * kWaveCap;
    uint32_t before = 0;
    LaneSums sums;
    int n_kept = 0;  // the same in every lane
    uint64_t least = 0;
    float bound = -INFINITY;
    // Every wave takes part in the first round (a segment past the row's end holds -inf
    // only), then each until its segments end.
    for (int32_t round = 0; round == 0 || seg < seg1; ++round, seg += NW) {
        float v[32], gm[8], lm = -INFINITY;
        next.values(v);
        if (seg + NW < seg1)
            next.load(zr, V, static_cast<int64_t>(seg + NW) * kSegCols, lane);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            gm[u] = __builtin_elementwise_maximum(
                __builtin_elementwise_maximum(__builtin_elementwise_maximum(v[4 * u], v[4 * u + 1]), v[4 * u + 2]),
                v[4 * u + 3]);
            if (u & 1)
                lm = __builtin_elementwise_maximum(__builtin_elementwise_maximum(lm, gm[u - 1]), gm[u]);  // NaN stays NaN
        }
        if constexpr (TOP) {  // a NaN only raises a slot: the row is NaN then
            if (k <= kFewTop) {
                atomicMax(&slot[lane], order_key(lm));
            } else {
                // Groups of four in turn, so that both have some where rows are short.
                float half[2] = {gm[0], gm[1]};
#pragma unroll
                for (int u = 2; u < 8; ++u)
                    half[u & 1] = __builtin_elementwise_maximum(half[u & 1], gm[u]);
                atomicMax(&slot[lane], order_key(half[0]));
                atomicMax(&slot[lane + 64], order_key(half[1]));
            }
        }
        sums.add(v, lm, c);
        if constexpr (RANK) {
            // Vectors before the token's count equal values, those behind it
            // larger ones only; its own vector's equal ones join in the end.
            const int32_t rel = y - seg * kSegCols - lane * G;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (!__ballot(gm[u] >= zy))
                    continue;
                const float least_ahead = 64 * (4 * u / G) * G + G <= rel ? zy : above;
#pragma unroll
                for (int i = 4 * u; i < 4 * u + 4; ++i)
                    before += __popcll(__ballot(v[i] >= least_ahead));
            }
        }
        if constexpr (TOP) {
            if (round == 0)
                __syncthreads();  // every wave's slots
            if (__ballot(lm >= bound)) {
                if ((round & (round + 1)) == 0) {
                    const uint32_t t = max(slots_bound(slot, lane, k), order_key(-INFINITY) + 1u);
                    least = max(least, static_cast<uint64_t>(t) << 32);
                    bound = key_value(static_cast<uint32_t>(least >> 32));
                }
                const int n_before = n_kept;
                const uint32_t rest = 0xffffffffu - (static_cast<uint32_t>(seg) * kSegCols + static_cast<uint32_t>(lane * G));
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (!__ballot(gm[u] >= bound))
                        continue;
#pragma unroll
                    for (int i = 4 * u; i < 4 * u + 4; ++i) {
                        const uint64_t mask = __ballot(v[i] >= bound);
                        if (!mask)
                            continue;
                        // The column's complement is formed here, not for all 32
                        // values ahead of the branches (64 registers).
                        uint32_t low = rest;
                        asm volatile("" : "+v"(low));
                        low -= static_cast<uint32_t>(64 * (i / G) * G + i % G);
                        const int at = n_kept + __popcll(mask & ((1ull << lane) - 1ull));
                        if (v[i] >= bound && at < kWaveCap)
                            mine[at] = (static_cast<uint64_t>(order_key(v[i])) << 32) | low;
                        n_kept += __popcll(mask);
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                if (n_kept > kWaveCap)
                    n_kept = collect_all<BF16>(zr, V, static_cast<int64_t>(seg) * kSegCols, least, mine, n_before, k, lane);
            }
        }
    }
    // The wave's sums, then the workgroup's.
    {
        const float m = wave_maximum(sums.m);
        const float ms = m == -INFINITY ? 0.0f : m;
        const float dy = __builtin_elementwise_maximum((sums.m - ms) * c, kNoTerm);
        const float f = __builtin_amdgcn_exp2f(dy);
        const float d = wave_sum(sums.d * f), s = wave_sum(f * fmaf(dy, sums.d, sums.s));
        if (lane == 0)
            part_rec[wave] = {m, d, s, before};
    }
    __syncthreads();
    if constexpr (TOP) {
        // What reaches the last bound: no slot changes any more, and none has since the
        // first round if it is the only one.
        if (seg1 - seg0 > NW)
            least = max(least, static_cast<uint64_t>(slots_bound(slot, lane, k)) << 32);
        for (int i = lane; i < n_kept; i += 64) {
            const uint64_t key = mine[i];
            if (key >= least) {
                const uint32_t at = atomicAdd(&cand_n, 1u);
                if (at < kListCap)
                    cand[at] = key;
            }
        }
    }
    RowSums q = {};
    float own_log_d = 0.0f;
    if (wave == 0) {
        q = fold(part_rec, NW, lane, c);
        own_log_d = q.d > 0.0 ? logf(static_cast<float>(q.d)) : __int_as_float(0x7fc00000);
        if (TOP && lane == 0) {
            sh_log_d = own_log_d;
            sh_m = q.m;
        }
    }
    if constexpr (TOP)
        __syncthreads();
    if (tid == 0) {  // behind the barrier: the token's logit may still be on its way
        if (parts == 1)
            write_row(q, own_log_d, inv_t, zr, BF16, V, token, ignore_index, row, o);
        else
            rec[id] = {q.m, static_cast<float>(q.d), static_cast<float>(q.s), q.before};
    }
    if constexpr (TOP) {
        uint64_t *out_keys = lists + static_cast<int64_t>(id) * k;
        float *lp = o.top_logprob + static_cast<int64_t>(row) * k;
        int32_t *tok = o.top_token + static_cast<int64_t>(row) * k;
        const float log_d = sh_log_d;
        const bool nan_row = parts == 1 && !(log_d == log_d);
        auto put = [&](int at, uint64_t key) {
            if (parts != 1) {
                out_keys[at] = key;
            } else if (key == 0 || nan_row) {
                lp[at] = nan_row ? __int_as_float(0x7fc00000) : -INFINITY;
                tok[at] = -1;
            } else {
                const float z = key_value(static_cast<uint32_t>(key >> 32));
                lp[at] = static_cast<float>((static_cast<double>(z) - sh_m) * inv_t - log_d);
                tok[at] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key));
            }
        };
        const int n = static_cast<int>(cand_n);
        if (nan_row) {
            if (tid < k)  // k <= 64 threads
                put(tid, 0);
        } else if (n <= kListCap) {
            for (int i = tid; i < n; i += NW * 64) {
                const uint64_t key = cand[i];
                int rank = 0;
                for (int q = 0; q < n; q += 8)  // zeros behind the n-th
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        rank += cand[q + j] > key;
                if (rank < k)
                    put(rank, key);
            }
            if (n + tid < k)  // fewer than k above -inf
                put(n + tid, 0);
        } else {
            // More than are ranked at once: k rounds, each taking the largest key
            // below the last one.
            uint64_t last = ~0ull;
            for (int r = 0; r < k; ++r) {
                uint64_t best = 0;
                for (int i = lane; i < n_kept; i += 64) {
                    const uint64_t key = mine[i];
                    if (key < last && key > best)
                        best = key;
                }
#pragma unroll
                for (int off = 32; off >= 1; off >>= 1)
                    best = max(best, shfl_xor_u64(best, off));
                if (lane == 0)
                    red[wave] = best;
                __syncthreads();
                for (int w = 0; w < NW; ++w)
                    best = max(best, red[w]);
                __syncthreads();
                if (tid == 0)
                    put(r, best);
                last = best;
            }
        }
    }
}

// Rows in parts without alternatives: one wave each.
__global__ __launch_bounds__(256) void logprobs_merge_kernel(
    const char *__restrict__ logits, int64_t ld_bytes, int32_t bf16, int64_t n_rows, int64_t V, int32_t parts,
    const int32_t *__restrict__ token, int32_t ignore_index, const float *__restrict__ temperature,
    int64_t temperature_stride, const LogprobRecord *__restrict__ rec, RowOutputs o)
{
    const int lane = threadIdx.x & 63;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (row >= n_rows)
        return;
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const RowSums q = fold(rec + row * parts, parts, lane, kLog2e * inv_t);
    if (lane == 0)
        write_row(q, logf(static_cast<float>(q.d)), inv_t, logits + row * ld_bytes, bf16 != 0, V, token, ignore_index, row, o);
}

constexpr int kTopThreads = 256;
constexpr int kTopCap = 2048;  // candidates of a row in LDS

// Rows in parts with alternatives: one workgroup each.  Of sorted lists of k keys, one
// per part, a lower bound of the k-th largest (from the lists' heads) leaves a few dozen
// candidates, which are ranked by counting.  Latency-bound: 64 rows in 4 parts, 20
// alternatives, 4 - 5 us; the first kernel's time falls by more (64 x 131072 BF16: 17 us
// in one kernel, 12 in two).
__global__ __launch_bounds__(kTopThreads) void logprobs_top_kernel(
    const char *__restrict__ logits, int64_t ld_bytes, int32_t bf16, int64_t V, int32_t parts,
    const int32_t *__restrict__ token, int32_t ignore_index, const float *__restrict__ temperature,
    int64_t temperature_stride, int32_t k, const LogprobRecord *__restrict__ rec,
    const uint64_t *__restrict__ lists, RowOutputs o)
{
    __shared__ uint64_t cand[kTopCap];
    __shared__ uint32_t n_cand, bound;
    __shared__ float sh_log_d;
    __shared__ float sh_m;
    __shared__ uint64_t red[kTopThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x;
    const uint64_t *keys = lists + row * parts * k;
    const int64_t n_keys = static_cast<int64_t>(parts) * k;
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const uint64_t first = tid < n_keys ? keys[tid] : 0;  // under way while the sums are folded
    RowSums q = {};
    if (wave == 0) {
        q = fold(rec + row * parts, parts, lane, kLog2e * inv_t);
        if (lane == 0) {
            sh_log_d = q.d > 0.0 ? logf(static_cast<float>(q.d)) : __int_as_float(0x7fc00000);
            sh_m = q.m;
            n_cand = 0;
        }
    } else if (wave == 1) {
        // 64 distinct entries, the lists' heads first: the k-th largest of them
        // is a bound that at least k keys reach.
        uint32_t mine = 0;
        if (parts >= 64) {
            for (int64_t l = lane; l < parts; l += 64)
                mine = max(mine, static_cast<uint32_t>(keys[l * k] >> 32));
        } else if (lane / parts < k) {
            mine = static_cast<uint32_t>(keys[static_cast<int64_t>(lane % parts) * k + lane / parts] >> 32);
        }
        const uint32_t t = kth_largest<1>({mine}, k);
        if (lane == 0)
            bound = t;
    }
    __syncthreads();
    const float log_d = sh_log_d;
    if (tid == 0)
        write_row(q, log_d, inv_t, logits + row * ld_bytes, bf16 != 0, V, token, ignore_index, row, o);
    float *lp = o.top_logprob + row * k;
    int32_t *tok = o.top_token + row * k;
    if (!(log_d == log_d)) {
        if (tid < k) {
            lp[tid] = __int_as_float(0x7fc00000);
            tok[tid] = -1;
        }
        return;
    }
    const uint64_t least = max(static_cast<uint64_t>(bound) << 32, uint64_t{1});
    for (int64_t i = tid; i < n_keys; i += kTopThreads) {
        const uint64_t key = i == tid ? first : keys[i];
        if (key >= least) {
            const uint32_t at = atomicAdd(&n_cand, 1u);
            if (at < kTopCap)
                cand[at] = key;
        }
    }
    __syncthreads();
    const uint32_t n = n_cand;
    auto put = [&](int at, uint64_t key) {
        const float z = key_value(static_cast<uint32_t>(key >> 32));
        lp[at] = static_cast<float>((static_cast<double>(z) - sh_m) * inv_t - log_d);
        tok[at] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key));
    };
    if (n <= kTopCap) {
        for (uint32_t i = tid; i < n; i += kTopThreads) {
            const uint64_t key = cand[i];
            int rank = 0;
            for (uint32_t q = 0; q < n; ++q)
                rank += cand[q] > key;
            if (rank < k)
                put(rank, key);
        }
        if (n + tid < static_cast<uint32_t>(k)) {  // fewer than k above -inf
            lp[n + tid] = -INFINITY;
            tok[n + tid] = -1;
        }
        return;
    }
    // More candidates than fit (many equal logits over many segments): k rounds,
    // each taking the largest key below the last one.
    uint64_t last = ~0ull;
    for (int r = 0; r < k; ++r) {
        uint64_t best = 0;
        for (int64_t i = tid; i < n_keys; i += kTopThreads) {
            const uint64_t key = keys[i];
            if (key < last && key > best)
                best = key;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            best = max(best, shfl_xor_u64(best, off));
        if (lane == 0)
            red[wave] = best;
        __syncthreads();
        for (int w = 0; w < kTopThreads / 64; ++w)
            best = max(best, red[w]);
        __syncthreads();
        if (tid == 0)
            put(r, best);  // n > kTopCap >= k: never 0
        last = best;
    }
}

// ------------------------------------------------------------------ gradient

constexpr int kBwdThreads = 128;
constexpr int kBwdVecs = 4;  // vectors per thread

// One chunk of 4 x 128 vectors of a row per workgroup.  With
// y = (z - m) / T / ln 2 and e = 2^y, dz = e a + (e y) b, b = -h ln 2 / (d T) and
// a = -(g + h (H - log d)) / (d T), and g / T more at the token.  Bound by the stream
// read and written: 4096 x 131072 FP32 to BF16 in 505 us, 6.4 TB/s (256 threads: 524;
// two vectors a thread: 503 - 531, the row's numbers weigh more).
template <bool ZBF16, bool GBF16, bool ENTROPY>
__global__ __launch_bounds__(kBwdThreads) void logprobs_bwd_kernel(
    const void *logits, int64_t ld, const float4 *__restrict__ stats, const int32_t *__restrict__ token,
    int32_t ignore_index, const float *__restrict__ temperature, int64_t temperature_stride,
    const float *__restrict__ dlogprob, int64_t dlogprob_stride, const float *__restrict__ dentropy,
    int64_t dentropy_stride, void *dlogits, int64_t ldg, int64_t V, uint32_t chunks)
{
    constexpr int G = kRowVec<ZBF16, GBF16>;
    using Vec = RowVec<ZBF16, G>;
    const uint32_t id = blockIdx.x, row = id / chunks, chunk = id - row * chunks;
    const int tid = threadIdx.x;
    const int64_t nv = V / G;
    const int32_t y = token ? token[row] : ignore_index;
    const bool ignored = !token || y == ignore_index;
    const bool bad = !ignored && (y < 0 || y >= V);
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const float g = (ignored || !dlogprob) ? 0.0f : dlogprob[row * dlogprob_stride];
    const float h = ENTROPY ? dentropy[row * dentropy_stride] : 0.0f;
    const float4 st = stats[row];
    const float nan = __int_as_float(0x7fc00000);
    float a = -(g + (ENTROPY ? h * (st.z - logf(st.y)) : 0.0f)) / st.y * inv_t;
    const float b = -h * kLn2 / st.y * inv_t, c = kLog2e * inv_t, at_token = g * inv_t;
    const bool nothing = !bad && g == 0.0f && h == 0.0f;  // the row is not read
    if (bad)
        a = nan;
    const char *zr = static_cast<const char *>(logits) + static_cast<int64_t>(row) * ld * (ZBF16 ? 2 : 4);
    char *gr = static_cast<char *>(dlogits) + static_cast<int64_t>(row) * ldg * (GBF16 ? 2 : 4);

    auto value = [&](float z, bool own) {
        const float e2 = __builtin_elementwise_maximum((z - st.x) * c, kNoTerm);
        const float e = __builtin_amdgcn_exp2f(e2);
        const float ea = own ? fmaf(e, a, at_token) : e * a;
        // e e2, which lies in (-0.54, 0], before b: b e2 passes FP32 where h / T is large,
        // and times e = 0 that would be NaN.
        return ENTROPY ? fmaf(e * e2, b, ea) : ea;
    };
    const int64_t first = static_cast<int64_t>(chunk) * kBwdThreads * kBwdVecs;
    Vec q[kBwdVecs];
    if (!nothing) {
#pragma unroll
        for (int u = 0; u < kBwdVecs; ++u) {
            const int64_t i = first + u * kBwdThreads + tid;
            if (i < nv)
                q[u].load(zr + i * Vec::kBytes);
        }
    }
#pragma unroll
    for (int u = 0; u < kBwdVecs; ++u) {
        const int64_t i = first + u * kBwdThreads + tid;
        if (i >= nv)
            continue;
        float o[G];
        const int64_t rel = static_cast<int64_t>(y) - i * G;
#pragma unroll
        for (int e = 0; e < G; ++e)
            o[e] = nothing ? 0.0f : value(q[u].value(e), !ignored && rel == e);
        store_row<GBF16>(gr, i, o);
    }
    // The last V % G columns, by the row's last chunk.
    if (chunk == chunks - 1 && tid < G) {
        const int64_t j = nv * G + tid;
        if (j < V) {
            store_element<GBF16>(gr, j, nothing ? 0.0f : value(row_element<ZBF16>(zr, j), !ignored && j == y));
        }
    }
}

}  // namespace

int64_t logprobs_workspace_bytes(int64_t n_rows, int64_t V, int64_t k)
{
    const int64_t parts = row_plan(n_rows, V, 1).parts;
    return parts == 1 ? 0 : n_rows * parts * (static_cast<int64_t>(sizeof(LogprobRecord)) + 8 * k);
}

hipError_t launch_logprobs(const Logprobs &p, void *workspace, hipStream_t s)
{
    const RowPlan plan = row_plan(p.n, p.V, 1);
    const int64_t parts = plan.parts, esz = p.bf16 ? 2 : 4;
    LogprobRecord *rec = static_cast<LogprobRecord *>(workspace);
    uint64_t *lists = reinterpret_cast<uint64_t *>(rec + p.n * parts);
    const int32_t k = static_cast<int32_t>(p.k);
    const int64_t chunk = std::max<int64_t>(1, kMaxItems / 1024 / parts);
    for (int64_t r0 = 0; r0 < p.n; r0 += chunk) {
        const int64_t nr = std::min(chunk, p.n - r0);
        const char *z = static_cast<const char *>(p.logits) + r0 * p.ld * esz;
        const int32_t *tok = p.token ? p.token + r0 : nullptr;
        const float *temp = p.temperature ? p.temperature + r0 * p.temperature_stride : nullptr;
        LogprobRecord *rc = rec + r0 * parts;
        uint64_t *ls = lists + r0 * parts * k;
        const RowOutputs o = {p.logprob ? p.logprob + r0 : nullptr, p.entropy ? p.entropy + r0 : nullptr,
                              p.rank ? p.rank + r0 : nullptr, reinterpret_cast<float4 *>(p.stats) + r0,
                              k ? p.top_logprob + r0 * k : nullptr, k ? p.top_token + r0 * k : nullptr};
        auto rows = [&](auto bf16, auto top, auto rank, auto waves) {
            constexpr int NW = decltype(waves)::value;
            hipLaunchKernelGGL(
                (logprobs_row_kernel<decltype(bf16)::value, decltype(top)::value, decltype(rank)::value, NW>),
                dim3(static_cast<unsigned>(nr * parts)), dim3(NW * 64), 0, s, z, p.ld, p.V,
                static_cast<uint32_t>(parts), plan.part_segs, tok, p.ignore_index, temp, p.temperature_stride, k,
                rc, ls, o);
        };
        const auto yes = std::true_type{};
        const auto no = std::false_type{};
        auto with_waves = [&](auto bf16, auto top, auto rank) {
            if (plan.waves == 1)
                rows(bf16, top, rank, std::integral_constant<int, 1>{});
            else if (plan.waves == 4)
                rows(bf16, top, rank, std::integral_constant<int, 4>{});
            else if (plan.waves == 8)
                rows(bf16, top, rank, std::integral_constant<int, 8>{});
            else
                rows(bf16, top, rank, std::integral_constant<int, 16>{});
        };
        auto with_rank = [&](auto bf16, auto top) { p.rank ? with_waves(bf16, top, yes) : with_waves(bf16, top, no); };
        auto with_top = [&](auto bf16) { k ? with_rank(bf16, yes) : with_rank(bf16, no); };
        p.bf16 ? with_top(yes) : with_top(no);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        if (parts == 1)
            continue;
        if (k)
            hipLaunchKernelGGL(logprobs_top_kernel, dim3(static_cast<unsigned>(nr)), dim3(kTopThreads), 0, s, z,
                               p.ld * esz, p.bf16 ? 1 : 0, p.V, static_cast<int32_t>(parts), tok, p.ignore_index,
                               temp, p.temperature_stride, k, rc, ls, o);
        else
            hipLaunchKernelGGL(logprobs_merge_kernel, dim3(static_cast<unsigned>((nr + 3) / 4)), dim3(256), 0, s, z,
                               p.ld * esz, p.bf16 ? 1 : 0, nr, p.V, static_cast<int32_t>(parts), tok,
                               p.ignore_index, temp, p.temperature_stride, rc, o);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_logprobs_bwd(const LogprobsBwd &p, hipStream_t s)
{
    const int64_t zsz = p.bf16 ? 2 : 4, gsz = p.grad_bf16 ? 2 : 4, G = zsz + gsz == 4 ? 8 : 4;
    const int64_t per = kBwdThreads * kBwdVecs;
    const int64_t chunks = std::max<int64_t>(1, (p.V / G + per - 1) / per);
    const int64_t rows = std::max<int64_t>(1, kMaxItems / kBwdThreads / chunks);
    for (int64_t r0 = 0; r0 < p.n; r0 += rows) {
        const int64_t nr = std::min(rows, p.n - r0);
        auto go = [&](auto zb, auto gb, auto ent) {
            hipLaunchKernelGGL((logprobs_bwd_kernel<decltype(zb)::value, decltype(gb)::value, decltype(ent)::value>),
                               dim3(static_cast<unsigned>(nr * chunks)), dim3(kBwdThreads), 0, s,
                               static_cast<const char *>(p.logits) + r0 * p.ld * zsz, p.ld,
                               reinterpret_cast<const float4 *>(p.stats) + r0, p.token ? p.token + r0 : nullptr,
                               p.ignore_index,
                               p.temperature ? p.temperature + r0 * p.temperature_stride : nullptr,
                               p.temperature_stride, p.dlogprob ? p.dlogprob + r0 * p.dlogprob_stride : nullptr,
                               p.dlogprob_stride, p.dentropy ? p.dentropy + r0 * p.dentropy_stride : nullptr,
                               p.dentropy_stride, static_cast<char *>(p.dlogits) + r0 * p.ldg * gsz, p.ldg, p.V,
                               static_cast<uint32_t>(chunks));
        };
        const auto yes = std::true_type{};
        const auto no = std::false_type{};
        auto with_ent = [&](auto zb, auto gb) { p.dentropy ? go(zb, gb, yes) : go(zb, gb, no); };
        auto with_grad = [&](auto zb) { p.grad_bf16 ? with_ent(zb, yes) : with_ent(zb, no); };
        p.bf16 ? with_grad(yes) : with_grad(no);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace lmh
