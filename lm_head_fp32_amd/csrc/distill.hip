// distill.hip -- cross-entropy against a teacher known by its top tokens, on
// gfx950: forward and gradient.
//
// Row i has a list of up to 256 tokens c_l with values v_l.  With the student's
// p = softmax(z / T):
//   logits mode: q = softmax(v / T) over the list,
//     loss = sum_l q_l (log q_l - log p_{c_l}),
//     dz_j = (1 / T) (p_j - q_j)                       (q_j = 0 off the list)
//   tail mode: q_l = exp(v_l), and what the list leaves, q_r = max(0, 1 - sum q),
//     belongs to all other tokens as one class with p_r = sum of their p:
//     loss += q_r (log q_r - log p_r),
//     dz_j = (1 / T) (Q p_j - q_j) on the list, Q = q_r + sum q,
//     dz_j = (1 / T) p_j (Q - q_r / p_r) off it.
// p_r is summed over the other tokens themselves: 1 - sum of the listed p would
// lose it where the list holds nearly everything.  So the scan of the logits leaves
// the listed columns out in tail mode (about their own maximum m_o), and the list's
// exponentials, read again by column, complete the row's sum d.  The gradient off
// the list is exp((z_j - m_o) / T) w with one number w per row, which neither
// overflows nor loses a small p_r.  A token that is listed twice counts twice in q
// and once in p.
#include "common.h"
#include "rows.h"

#include <math.h>

#include <algorithm>
#include <type_traits>

namespace lmh {

namespace {

constexpr int64_t kMaxItems = int64_t{1} << 31;  // work-items per launch
constexpr int kMaxList = kDistillMaxList;
constexpr int kListThreads = 256;
static_assert(kMaxList <= kListThreads, "one thread per entry of the list");

struct ListArgs {
    const int32_t *token;
    int64_t ldt;
    const void *value;
    int64_t ldv;
    int32_t k;
    bool bf16, tail;
};

// An entry of a row's list; one without a token or of value -inf is absent.
struct Entry {
    int32_t token;  // -1: absent
    float value;
};
__device__ __forceinline__ Entry entry(const ListArgs &t, int64_t row, int i)
{
    if (i >= t.k)
        return {-1, 0.0f};
    const int32_t id = t.token[row * t.ldt + i];
    const float v = t.bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(t.value)[row * t.ldv + i]) << 16)
                           : static_cast<const float *>(t.value)[row * t.ldv + i];
    return {id < 0 || v == -INFINITY ? -1 : id, v};
}

// A row's record, as lmhead_distill_fwd's stats.
struct alignas(16) RowStats {
    float m, d;          // of the whole row
    float loss;
    float weight;        // Q: 1, or 0 where the list is empty
    float other, w;      // gradient off the list: exp((z - other) / T) w / T
    float top, sum;      // q_l = exp((v_l - top) / T_v) / sum, T_v = T or (tail mode) 1
};
static_assert(sizeof(RowStats) == 32, "eight floats");

// What the list says of a row, in 64 bits: the teacher's total and entropy term
// (A = sum q log q), B = sum q (z - m_l) about the listed columns' maximum m_l, and the
// student's sum D over them, each once, about m_l too (tail mode).  B and (m_l - m) sum q
// have one sign; sum q z and m sum q would cancel where the logits have a large common
// part (a row of masks only, at the type's lowest value).
struct ListSums {
    double total, A, B, D, sum;
    float m_l, top;
    int32_t there;  // entries; 0: the list is empty
    bool off;       // one lies outside the columns
    bool twice;     // a token is listed more than once
};

struct ListShared {
    int32_t ids[kMaxList];
    float v_max[kListThreads / 64], z_max[kListThreads / 64];
    int32_t flags[kListThreads / 64];  // entries, 2^10 those outside, 2^20 those listed before
    double part[kListThreads / 64][4];
};

// What B is taken about: m_l, or any finite number where no listed column lies above -inf.
__device__ __forceinline__ float list_shift(float m_l)
{
    return m_l == -INFINITY ? 0.0f : m_l;
}

// Waves that hold entries of a list of k (one at least).
__device__ __forceinline__ int list_waves(int32_t k)
{
    return max((k + 63) / 64, 1);
}

// The sums of the shared parts; any thread, once list_part is through.
template <bool TAIL>
__device__ __forceinline__ ListSums list_sums(const ListShared &sh, int32_t k)
{
    const int NW = list_waves(k);
    ListSums r;
    r.top = sh.v_max[0];
    r.m_l = sh.z_max[0];
    int32_t flags = sh.flags[0];
    double s = sh.part[0][0];
    r.A = sh.part[0][1];
    r.B = sh.part[0][2];
    r.D = sh.part[0][3];
    for (int w = 1; w < NW; ++w) {
        r.top = __builtin_elementwise_maximum(r.top, sh.v_max[w]);
        r.m_l = __builtin_elementwise_maximum(r.m_l, sh.z_max[w]);
        flags += sh.flags[w];
        s += sh.part[w][0];
        r.A += sh.part[w][1];
        r.B += sh.part[w][2];
        r.D += sh.part[w][3];
    }
    r.there = flags & 0x3ff;
    r.off = ((flags >> 10) & 0x3ff) != 0;
    r.twice = (flags >> 20) != 0;
    r.sum = s;
    r.total = s;
    if constexpr (TAIL) {
        r.top = 0.0f;
        r.sum = 1.0;
    } else {
        r.total = s == s ? 1.0 : s;
        r.B /= s;
    }
    return r;
}

// By a workgroup whose first 256 threads hold an entry each (en, and z, the logit of
// its column; `again`: another entry may have its token).  Two barriers.  Returns the
// thread's own share of the teacher: with TAIL q itself, else q times the sum.
template <bool TAIL>
__device__ __forceinline__ double list_part(ListShared &sh, const Entry &en, float z, int64_t V, float inv_t,
                                            int32_t k, bool again, int tid)
{
    const int lane = tid & 63, wave = tid >> 6;
    const int NW = list_waves(k);
    const bool there = en.token >= 0;
    if (wave < NW) {
        const float vm = wave_maximum(there ? en.value : -INFINITY), zm = wave_maximum(z);
        const int32_t n = __popcll(__ballot(there)), off = __popcll(__ballot(there && en.token >= V)),
                      more = __popcll(__ballot(again));
        if (lane == 0) {
            sh.v_max[wave] = vm;
            sh.z_max[wave] = zm;
            sh.flags[wave] = n + (off << 10) + (more << 20);
        }
    }
    __syncthreads();
    double e = 0.0;
    if (wave < NW) {
        float top = sh.v_max[0], m_l = sh.z_max[0];
        int32_t flags = sh.flags[0];
        for (int w = 1; w < NW; ++w) {
            top = __builtin_elementwise_maximum(top, sh.v_max[w]);
            m_l = __builtin_elementwise_maximum(m_l, sh.z_max[w]);
            flags += sh.flags[w];
        }
        const double x = TAIL ? static_cast<double>(en.value) : (static_cast<double>(en.value) - top) * inv_t;
        e = there ? exp(x) : 0.0;
        const double s = wave_sum(e), a = wave_sum(e != 0.0 ? e * x : 0.0),
                     b = wave_sum(e != 0.0 ? e * (static_cast<double>(z) - list_shift(m_l)) : 0.0);
        double dl = 0.0;
        if constexpr (TAIL) {
            bool first = there;
            for (int i = 0; (flags >> 20) && i < min(tid, k); ++i)
                first = first && sh.ids[i] != en.token;
            dl = wave_sum(first && z != -INFINITY ? exp((static_cast<double>(z) - m_l) * inv_t) : 0.0);
        }
        if (lane == 0) {
            sh.part[wave][0] = s;
            sh.part[wave][1] = a;
            sh.part[wave][2] = b;
            sh.part[wave][3] = dl;
        }
    }
    __syncthreads();
    return e;
}

__device__ __forceinline__ double lane_value(double v, int lane)
{
    const uint64_t u = __double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(u), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(u >> 32), lane);
    return __longlong_as_double((static_cast<uint64_t>(hi) << 32) | lo);
}

// The row's numbers from the list's and the scanned columns' (m_o, d_o: all columns,
// or with TAIL those off the list); by a whole wave, every lane with the same
// arguments and the same result.  The two exponentials, the three logarithms and the
// three quotients are taken side by side, a lane each.
template <bool TAIL>
__device__ __forceinline__ RowStats finish_row(const ListSums &t, float m_o, double d_o, float inv_t, int lane)
{
    const double none = -static_cast<double>(INFINITY);
    float m = m_o;
    double d = d_o, shift = 0.0, scale = 1.0, q_r = 0.0;
    if constexpr (TAIL) {
        m = __builtin_elementwise_maximum(m_o, t.m_l);
        shift = (static_cast<double>(m_o) - m) * inv_t;
        const double x = lane == 0 ? (d_o != 0.0 ? shift : none)
                                   : (t.D != 0.0 ? (static_cast<double>(t.m_l) - m) * inv_t : none);
        const double f = exp(x);
        scale = lane_value(f, 0);
        d = (d_o != 0.0 ? d_o * scale : 0.0) + (t.D != 0.0 ? t.D * lane_value(f, 1) : 0.0);
        q_r = d_o != 0.0 ? fmax(0.0, 1.0 - t.total) : 0.0;  // no other column: that class is left out
    }
    const double logs = log(lane == 0 ? d : lane == 1 ? (TAIL ? d_o : t.sum) : (q_r != 0.0 ? q_r : 1.0));
    const double log_d = lane_value(logs, 0), log_2 = lane_value(logs, 1), log_qr = lane_value(logs, 2);
    const double weight0 = t.total + q_r;
    const double quot = (lane == 0 ? weight0 : lane == 1 ? q_r : t.A) / (lane == 0 ? d : lane == 1 ? d_o : t.sum);
    const double per_d = lane_value(quot, 0);
    // sum q log q: in logits mode of q = exp(x) / sum
    const double a = TAIL ? t.A : lane_value(quot, 2) - log_2;
    double l = a - (t.B + (static_cast<double>(list_shift(t.m_l)) - m) * t.total) * inv_t + log_d * t.total;
    double weight = weight0, w = per_d;
    if constexpr (TAIL) {
        if (q_r != 0.0)
            l += q_r * (log_qr - (shift + log_2 - log_d));
        w = d_o != 0.0 ? per_d * scale - (q_r != 0.0 ? lane_value(quot, 1) : 0.0) : 0.0;
    }
    if (t.off || !(d > 0.0) || !(t.total < INFINITY))
        l = w = weight = static_cast<double>(NAN);
    // No other column above -inf: any finite shift gives them exp(-inf) w = 0.
    const float other = m_o == -INFINITY ? m : m_o;
    return {m, static_cast<float>(d), static_cast<float>(l), static_cast<float>(weight),
            other, static_cast<float>(w), t.top, static_cast<float>(t.sum)};
}

// One workgroup of NW waves per (row, part of its segments of 2048 columns): {m, d}
// of the part, with TAIL of the columns that are not on the row's list; with one part
// per row also the loss and the record.  Of a row whose list is empty the first round of
// segments is read at most.  Bound by the read where rows are many and long (1024 x
// 131072 FP32: 83 us, 6.5 TB/s).  Many short rows are far from it (8192 x 1000, 16 listed:
// 30 us, with a class for the rest 35 - 37; the read is 4.6): the chain of list, barrier,
// scan, barrier and the row's numbers, in four waves of which one holds the segment and
// one the list.
template <bool BF16, bool TAIL, int NW>
__global__ __launch_bounds__(NW * 64) void distill_row_kernel(
    const void *__restrict__ logits, int64_t ld, int64_t V, uint32_t parts, int32_t part_segs, ListArgs list,
    const float *__restrict__ temperature, int64_t temperature_stride, float2 *__restrict__ rec,
    float *__restrict__ loss, RowStats *__restrict__ stats)
{
    constexpr int G = Segment<BF16>::G;
    extern __shared__ uint32_t listed[];  // TAIL: a bit per column of the part
    __shared__ ListShared sh;
    __shared__ float red_m[NW], red_d[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t id = blockIdx.x, row = id / parts;
    const int32_t seg0 = static_cast<int32_t>(id - row * parts) * part_segs;
    const int32_t seg1 = min(seg0 + part_segs, static_cast<int32_t>((V + kSegCols - 1) / kSegCols));
    const char *zr = static_cast<const char *>(logits) + static_cast<int64_t>(row) * ld * (16 / G);

    Entry en = {-1, 0.0f};
    if (tid < kMaxList)
        en = entry(list, row, tid);
    // The first round's loads do not wait for the list.
    Segment<BF16, true> next;
    int32_t seg = seg0 + wave;
    next.load(zr, V, static_cast<int64_t>(seg) * kSegCols, lane);
    if (__syncthreads_count(en.token >= 0) == 0) {
        if (tid == 0 && parts == 1) {
            stats[row] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (loss)
                loss[row] = 0.0f;
        }
        return;  // the merge of several parts does not read their records either
    }
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const float c = kLog2e * inv_t;
    float z = -INFINITY;
    if (parts == 1 && en.token >= 0 && en.token < V)
        z = row_element<BF16>(zr, en.token);
    if (tid < kMaxList)
        sh.ids[tid] = en.token;
    bool again = false;
    if constexpr (TAIL) {
        for (int i = tid; i < (seg1 - seg0) * (kSegCols / 32); i += NW * 64)
            listed[i] = 0;
        __syncthreads();
        const int64_t at = en.token - static_cast<int64_t>(seg0) * kSegCols;
        if (en.token >= 0 && at >= 0 && at < static_cast<int64_t>(seg1 - seg0) * kSegCols)
            again = (atomicOr(&listed[at >> 5], 1u << (at & 31)) >> (at & 31)) & 1u;
        __syncthreads();
    }
    if (parts == 1)
        list_part<TAIL>(sh, en, z, V, inv_t, list.k, again, tid);

    float m = -INFINITY, d = 0.0f;  // the lane's, rescaled once per 32 values
    for (; seg < seg1; seg += NW) {
        float v[32];
        next.values(v);
        if (seg + NW < seg1)
            next.load(zr, V, static_cast<int64_t>(seg + NW) * kSegCols, lane);
        if constexpr (TAIL) {
#pragma unroll
            for (int u = 0; u < 32 / G; ++u) {
                const int col = (seg - seg0) * kSegCols + (64 * u + lane) * G;
                const uint32_t bits = (listed[col >> 5] >> (col & 31)) & ((1u << G) - 1u);
                if (!__ballot(bits != 0))
                    continue;
#pragma unroll
                for (int e = 0; e < G; ++e)
                    v[u * G + e] = (bits >> e) & 1u ? -INFINITY : v[u * G + e];
            }
        }
        float lm = m;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            lm = __builtin_elementwise_maximum(lm, v[i]);  // NaN stays NaN
        const float ms = lm == -INFINITY ? 0.0f : lm;
        float dn[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 32; ++i)
            dn[i & 1] += __builtin_amdgcn_exp2f((v[i] - ms) * c);
        d = fmaf(d, __builtin_amdgcn_exp2f((m - ms) * c), dn[0] + dn[1]);
        m = lm;
    }
    {
        const float mw = wave_maximum(m), ms = mw == -INFINITY ? 0.0f : mw;
        d = wave_sum(d * __builtin_amdgcn_exp2f((m - ms) * c));
        if (lane == 0) {
            red_m[wave] = mw;
            red_d[wave] = d;
        }
    }
    __syncthreads();
    if (wave != 0)
        return;
    const float rm = lane < NW ? red_m[lane] : -INFINITY, rd = lane < NW ? red_d[lane] : 0.0f;
    const float m_o = wave_maximum(rm);
    const double d_o = wave_sum(rd != 0.0f ? static_cast<double>(rd) * __builtin_amdgcn_exp2f((rm - m_o) * c) : 0.0);
    if (parts == 1) {
        const RowStats st = finish_row<TAIL>(list_sums<TAIL>(sh, list.k), m_o, d_o, inv_t, lane);
        if (lane == 0) {
            stats[row] = st;
            if (loss)
                loss[row] = st.loss;
        }
    } else if (lane == 0) {
        rec[id] = make_float2(m_o, static_cast<float>(d_o));
    }
}

// Rows in several parts: one workgroup each, a thread per entry of its list.
template <bool TAIL>
__global__ __launch_bounds__(kListThreads) void distill_merge_kernel(
    const char *__restrict__ logits, int64_t ld_bytes, int32_t bf16, int64_t V, int32_t parts, ListArgs list,
    const float *__restrict__ temperature, int64_t temperature_stride, const float2 *__restrict__ rec,
    float *__restrict__ loss, RowStats *__restrict__ stats)
{
    constexpr int kBuckets = 1024;
    __shared__ ListShared sh;
    __shared__ uint32_t head[kBuckets], next[kMaxList];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x;
    const Entry en = entry(list, row, tid);
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const char *zr = logits + row * ld_bytes;
    float z = -INFINITY;
    if (en.token >= 0 && en.token < V)
        z = bf16 ? row_element<true>(zr, en.token) : row_element<false>(zr, en.token);
    sh.ids[tid] = en.token;
    bool again = false;
    if constexpr (TAIL) {  // entries of one token meet in one bucket
        for (int i = tid; i < kBuckets; i += kListThreads)
            head[i] = 0;
        __syncthreads();
        const uint32_t bucket = (static_cast<uint32_t>(en.token) * 2654435761u) >> 22;
        if (en.token >= 0)
            next[tid] = atomicExch(&head[bucket], static_cast<uint32_t>(tid) + 1u);
        __syncthreads();
        if (en.token >= 0)
            for (uint32_t e = head[bucket]; e != 0; e = next[e - 1])
                again = again || (sh.ids[e - 1] == en.token && static_cast<int>(e) - 1 != tid);
    }
    list_part<TAIL>(sh, en, z, V, inv_t, list.k, again, tid);
    const ListSums t = list_sums<TAIL>(sh, list.k);
    if (t.there == 0) {
        if (tid == 0) {
            stats[row] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (loss)
                loss[row] = 0.0f;
        }
        return;
    }
    if (tid >= 64)
        return;
    const float2 *r = rec + row * parts;
    float m_o = -INFINITY;
    for (int i = lane; i < parts; i += 64)
        m_o = __builtin_elementwise_maximum(m_o, r[i].x);
    m_o = wave_maximum(m_o);
    double d_o = 0.0;
    for (int i = lane; i < parts; i += 64) {
        const float2 p = r[i];
        if (p.y != 0.0f)  // NaN too
            d_o += static_cast<double>(p.y) * __builtin_amdgcn_exp2f((p.x - m_o) * (kLog2e * inv_t));
    }
    const RowStats st = finish_row<TAIL>(t, m_o, wave_sum(d_o), inv_t, lane);
    if (lane == 0) {
        stats[row] = st;
        if (loss)
            loss[row] = st.loss;
    }
}

// ------------------------------------------------------------------ gradient

// The upstream gradient per unit of z / T.  None is none at any temperature: 0 times the
// NaN of a temperature that is no temperature would make a row that asks for nothing NaN.
__device__ __forceinline__ float upstream(const float *dloss, int64_t i, float inv_t)
{
    const float g = dloss[i];
    return g == 0.0f ? 0.0f : g * inv_t;
}

constexpr int kBwdThreads = 128;
constexpr int kBwdVecs = 4;  // vectors per thread

// One chunk of 4 x 128 vectors of a row per workgroup.  Every
// column is first written as if it were off the list; the threads of the chunk's
// listed columns then write theirs over it.  Bound by the stream read and written:
// 2048 x 131072 FP32 to BF16 with 64 listed in 255 us, 6.3 TB/s.
template <bool ZBF16, bool GBF16>
__global__ __launch_bounds__(kBwdThreads) void distill_bwd_kernel(
    const void *logits, int64_t ld, const RowStats *__restrict__ stats, ListArgs list,
    const float *__restrict__ temperature, int64_t temperature_stride, const float *__restrict__ dloss,
    int64_t dloss_stride, void *dlogits, int64_t ldg, int64_t V, uint32_t chunks)
{
    constexpr int G = kRowVec<ZBF16, GBF16>;
    using Vec = RowVec<ZBF16, G>;
    constexpr int NW = kBwdThreads / 64, EPT = kMaxList / kBwdThreads;  // entries per thread
    __shared__ int32_t ids[kMaxList];
    __shared__ float qs[kMaxList];
    __shared__ int32_t counts[kMaxList / 64];
    const uint32_t id = blockIdx.x, row = id / chunks, chunk = id - row * chunks;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t nv = V / G;
    const RowStats st = stats[row];
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const float c = kLog2e * inv_t, up = upstream(dloss, row * dloss_stride, inv_t), w_up = st.w * up;
    const bool nothing = up == 0.0f || (st.weight == 0.0f && st.w == 0.0f);  // the row is not read
    const char *zr = static_cast<const char *>(logits) + static_cast<int64_t>(row) * ld * (ZBF16 ? 2 : 4);
    char *gr = static_cast<char *>(dlogits) + static_cast<int64_t>(row) * ldg * (GBF16 ? 2 : 4);

    const int64_t first = static_cast<int64_t>(chunk) * kBwdThreads * kBwdVecs;
    const bool last = chunk == chunks - 1;
    Vec q[kBwdVecs];
    float listed_grad[EPT];
    int32_t listed_at[EPT];
    if (!nothing) {
#pragma unroll
        for (int u = 0; u < kBwdVecs; ++u) {
            const int64_t i = first + u * kBwdThreads + tid;
            if (i < nv)
                q[u].load(zr + i * Vec::kBytes);
        }
        // The list's entries in this chunk, compacted by groups of 64.
        const int64_t end = last ? V : (first + kBwdThreads * kBwdVecs) * G;
        const float t_inv = list.tail ? 1.0f : inv_t;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const Entry en = entry(list, row, j * kBwdThreads + tid);
            const bool here = en.token >= first * G && en.token < end;
            const uint64_t mask = __ballot(here);
            const int group = j * NW + wave;
            listed_at[j] = here ? en.token : -1;
            if (here) {
                const int at = group * 64 + __popcll(mask & ((1ull << lane) - 1ull));
                ids[at] = en.token;
                qs[at] = __builtin_amdgcn_exp2f((en.value - st.top) * (kLog2e * t_inv)) / st.sum;
                const float z = row_element<ZBF16>(zr, en.token);
                listed_grad[j] = __builtin_amdgcn_exp2f((z - st.m) * c) * (st.weight / st.d);
            }
            if (lane == 0)
                counts[group] = __popcll(mask);
        }
        __syncthreads();  // the list's logits are read before the row is written (in place)
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            if (listed_at[j] < 0)
                continue;
            float sum = 0.0f;
            for (int v = 0; v < kMaxList / 64; ++v)
                for (int i = 0; i < counts[v]; ++i)
                    sum += ids[v * 64 + i] == listed_at[j] ? qs[v * 64 + i] : 0.0f;
            listed_grad[j] = (listed_grad[j] - sum) * up;
        }
    }
    auto value = [&](float z) { return __builtin_amdgcn_exp2f((z - st.other) * c) * w_up; };
#pragma unroll
    for (int u = 0; u < kBwdVecs; ++u) {
        const int64_t i = first + u * kBwdThreads + tid;
        if (i >= nv)
            continue;
        float o[G];
#pragma unroll
        for (int e = 0; e < G; ++e)
            o[e] = nothing ? 0.0f : value(q[u].value(e));
        store_row<GBF16>(gr, i, o);
    }
    // The last V % G columns, by the row's last chunk.
    if (last && tid < G) {
        const int64_t j = nv * G + tid;
        if (j < V)
            store_element<GBF16>(gr, j, nothing ? 0.0f : value(row_element<ZBF16>(zr, j)));
    }
    if (!nothing) {
        __syncthreads();  // the chunk is written
#pragma unroll
        for (int j = 0; j < EPT; ++j)
            if (listed_at[j] >= 0)
                store_element<GBF16>(gr, listed_at[j], listed_grad[j]);
    }
}

// ------------------------------------------- loss and gradient in one read

// A vector of -inf.
__device__ __attribute__((aligned(16))) uint32_t kNegInfFP32[4] = {0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u};
__device__ __attribute__((aligned(16))) uint32_t kNegInfBF16[4] = {0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};

// One workgroup per row, which sits in registers: VALS values per thread, V <= NT VALS.
// The list's part is worked out while the row's loads are under way.  head[i] names
// the first entry of the list (plus one) whose column lies in the row's vector i,
// next[] the others: so a thread finds the listed columns among its own, in
// tail mode to leave them out of the sums, in the end to write their gradients in
// their places.  Entries of the same token hold the same gradient, so that the order
// in which they are found does not matter.  1024 x 32768 FP32 to BF16, two rows to a CU,
// 64 listed and the rest as a class: 39 - 45 us (forward and gradient in two kernels: 56);
// a row that fills the CU's registers has nothing to cover its start and end (1024 x 50001:
// 74 - 86 us, 3.9 TB/s, against 88; two registers are spilled there in tail mode).  Rows of
// a thousand columns lose by the one read, as the list's chain is most of their time and
// a CU holds four of these workgroups (8192 x 1000, 16 listed and a class: 55 us, against
// 35 + 15); rows of 4096 gain (61, against 38 + 38).
template <bool ZBF16, bool GBF16, bool TAIL, int NT, int VALS>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(4))) void distill_fused_kernel(
    const void *logits, int64_t ld, int64_t V, ListArgs list, const float *__restrict__ temperature,
    int64_t temperature_stride, const float *__restrict__ dloss, int64_t dloss_stride, float *__restrict__ loss,
    RowStats *__restrict__ stats, void *dlogits, int64_t ldg)
{
    constexpr int G = kRowVec<ZBF16, GBF16>, PER = VALS / G, NW = NT / 64;
    using Vec = RowVec<ZBF16, G>;
    __shared__ uint32_t head[NT * PER + 1];
    __shared__ uint32_t next[kMaxList];
    __shared__ float grads[kMaxList];
    __shared__ ListShared sh;
    __shared__ float2 red[NW];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const char *zr = static_cast<const char *>(logits) + row * ld * (ZBF16 ? 2 : 4);
    char *gr = static_cast<char *>(dlogits) + row * ldg * (GBF16 ? 2 : 4);
    const int nv = static_cast<int>(V / G);  // whole vectors
    const int jt = nv * G + tid;             // a column behind them, for tid < G
    const bool has_tail = tid < G && jt < V;

    Entry en = {-1, 0.0f};
    if (tid < kMaxList)
        en = entry(list, row, tid);
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const float up = upstream(dloss, row * dloss_stride, inv_t), c = kLog2e * inv_t;
    auto zero_row = [&]() {
        const float o[G] = {};
        for (int i = tid; i < nv; i += NT)
            store_row<GBF16>(gr, i, o);
        if (has_tail)
            store_element<GBF16>(gr, jt, 0.0f);
    };
    if (__syncthreads_count(en.token >= 0) == 0) {
        if (tid == 0) {
            stats[row] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (loss)
                loss[row] = 0.0f;
        }
        zero_row();
        return;
    }

    // The list's logits are asked for first: they come back first, and the list's part
    // is done while the row is on its way.
    const bool inside = en.token >= 0 && en.token < V;
    const float z = row_element<ZBF16>(inside ? zr : reinterpret_cast<const char *>(ZBF16 ? kNegInfBF16 : kNegInfFP32),
                                       inside ? en.token : 0);
    // Every load is issued, past the row's end from a constant vector of -inf: loads
    // behind a condition cannot be counted, and the list would have to wait for all.
    const char *none = reinterpret_cast<const char *>(ZBF16 ? kNegInfBF16 : kNegInfFP32);
    Vec raw[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p)
        raw[p].load(p * NT + tid < nv ? zr + (p * NT + tid) * Vec::kBytes : none);
    float tv = row_element<ZBF16>(has_tail ? zr : none, has_tail ? jt : 0);
    if (tid < kMaxList)
        sh.ids[tid] = en.token;
#pragma unroll
    for (int p = 0; p < PER; ++p)
        head[p * NT + tid] = 0;
    if (tid == 0)
        head[nv] = 0;  // the columns behind the last whole vector
    __syncthreads();
    const int vec = inside ? en.token / G : 0;
    if (inside)
        next[tid] = atomicExch(&head[vec], static_cast<uint32_t>(tid) + 1u);
    __syncthreads();
    auto listed_in = [&](int i, auto use) {  // use(column within the vector, entry)
        for (uint32_t e = head[i]; e != 0; e = next[e - 1])
            use(sh.ids[e - 1] - i * G, static_cast<int>(e) - 1);
    };
    // Which of the thread's vectors hold listed columns (a bit each): read side by side,
    // where a test at each vector would wait for LDS.
    uint32_t hits = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p)
        hits |= (p * NT + tid < nv && head[p * NT + tid] != 0) ? 1u << p : 0u;
    bool again = false;
    if (inside)
        listed_in(vec, [&](int at, int e) { again = again || (at == en.token - vec * G && e != tid); });
    // What the gradient needs of it is read back from LDS when the row is through (kept
    // in registers it would be spilled).
    float q = static_cast<float>(list_part<TAIL>(sh, en, z, V, inv_t, list.k, again, tid));

    float v[VALS];
#pragma unroll
    for (int p = 0; p < PER; ++p)
#pragma unroll
        for (int e = 0; e < G; ++e)
            v[p * G + e] = raw[p].value(e);
    if constexpr (TAIL) {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            if (hits & (1u << p))
                listed_in(p * NT + tid, [&](int at, int) {
#pragma unroll
                    for (int e = 0; e < G; ++e)
                        v[p * G + e] = at == e ? -INFINITY : v[p * G + e];
                });
        }
        if (has_tail)
            listed_in(nv, [&](int at, int) { tv = at == tid ? -INFINITY : tv; });
    }
    // The thread's own maximum and sum, then the row's; v becomes exp((v - m_t) / T).
    float m_t = tv;
#pragma unroll
    for (int i = 0; i < VALS; ++i)
        m_t = __builtin_elementwise_maximum(m_t, v[i]);
    const float ms = m_t == -INFINITY ? 0.0f : m_t;
    tv = __builtin_amdgcn_exp2f((tv - ms) * c);
    float dn[4] = {tv, 0.0f, 0.0f, 0.0f};  // short chains of additions
#pragma unroll
    for (int i = 0; i < VALS; ++i) {
        v[i] = __builtin_amdgcn_exp2f((v[i] - ms) * c);
        dn[i & 3] += v[i];
    }
    float d = (dn[0] + dn[1]) + (dn[2] + dn[3]);
    float m_o = wave_maximum(m_t);
    {
        const float mw = m_o == -INFINITY ? 0.0f : m_o;
        d = wave_sum(d * __builtin_amdgcn_exp2f((m_t - mw) * c));
        if (lane == 0)
            red[wave] = make_float2(m_o, d);
    }
    __syncthreads();
    double d_o;
    {
        const float2 r = red[lane & (NW - 1)];
        m_o = wave_maximum(r.x);
        const float mw = m_o == -INFINITY ? 0.0f : m_o;
        d_o = wave_sum(lane < NW ? static_cast<double>(r.y) * __builtin_amdgcn_exp2f((r.x - mw) * c) : 0.0);
    }
    // What the gradient needs, in FP32 by every thread: weight / d, and the factor w of
    // exp((z - m_o) / T) off the list.
    float w;
    {
        const ListSums t = list_sums<TAIL>(sh, list.k);
        const float df = static_cast<float>(d_o);
        float m = m_o, wd;
        if constexpr (TAIL) {
            m = __builtin_elementwise_maximum(m_o, t.m_l);
            const float f = df != 0.0f ? __builtin_amdgcn_exp2f((m_o - m) * c) : 0.0f;
            const float dl = static_cast<float>(t.D);
            const float dw = (dl != 0.0f ? dl * __builtin_amdgcn_exp2f((t.m_l - m) * c) : 0.0f) + f * df;
            const float q_r = df != 0.0f ? static_cast<float>(fmax(0.0, 1.0 - t.total)) : 0.0f;
            wd = (static_cast<float>(t.total) + q_r) / dw;
            w = df != 0.0f ? wd * f - q_r / df : 0.0f;
            if (!(dw > 0.0f))
                wd = w = __int_as_float(0x7fc00000);
        } else {
            wd = w = static_cast<float>(t.total) / df;
            q /= static_cast<float>(t.sum);
            if (!(df > 0.0f))
                wd = w = __int_as_float(0x7fc00000);
        }
        if (t.off || !(t.total < INFINITY))
            wd = w = __int_as_float(0x7fc00000);
        if (t.twice) {  // the shares of the same token, in the list's order
            if (tid < kMaxList)
                grads[tid] = q;
            __syncthreads();
            float sum = 0.0f;
            for (int i = 0; inside && i < list.k; ++i)
                sum += sh.ids[i] == en.token ? grads[i] : 0.0f;
            q = sum;
            __syncthreads();
        }
        if (tid < kMaxList)
            grads[tid] = (__builtin_amdgcn_exp2f((z - m) * c) * wd - q) * up;
    }
    __syncthreads();
    if (up == 0.0f) {
        zero_row();
    } else {
        const float scale = m_t == -INFINITY && w == w ? 0.0f : __builtin_amdgcn_exp2f((m_t - m_o) * c) * (w * up);
        int t = tid;  // recomputed here: the addresses are not kept over the row's sums
        asm volatile("" : "+v"(t));
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int i = p * NT + t;
            if (i >= nv)
                break;
            float o[G];
#pragma unroll
            for (int e = 0; e < G; ++e)
                o[e] = v[p * G + e] * scale;
            if (hits & (1u << p))
                listed_in(i, [&](int at, int l) {
                    const float g = grads[l];
#pragma unroll
                    for (int e = 0; e < G; ++e)
                        o[e] = at == e ? g : o[e];
                });
            store_row<GBF16>(gr, i, o);
        }
        if (has_tail) {
            float o = tv * scale;
            listed_in(nv, [&](int at, int l) { o = at == tid ? grads[l] : o; });
            store_element<GBF16>(gr, jt, o);
        }
    }
    if (wave == 0) {
        const RowStats st = finish_row<TAIL>(list_sums<TAIL>(sh, list.k), m_o, d_o, inv_t, lane);
        if (lane == 0) {
            stats[row] = st;
            if (loss)
                loss[row] = st.loss;
        }
    }
}

}  // namespace

namespace {

// A part's listed columns are bits in LDS.
constexpr int64_t kMaxPartSegs = 128;

}  // namespace

int64_t distill_workspace_bytes(int64_t n_rows, int64_t V)
{
    const int64_t parts = row_plan(n_rows, V, 4, kMaxPartSegs).parts;
    return parts == 1 ? 0 : n_rows * parts * static_cast<int64_t>(sizeof(float2));
}

namespace {

ListArgs list_args(const Distill &p, int64_t r0)
{
    return {p.token + r0 * p.ldt, p.ldt, static_cast<const char *>(p.value) + r0 * p.ldv * (p.value_bf16 ? 2 : 4),
            p.ldv, static_cast<int32_t>(p.k), p.value_bf16, p.tail};
}

}  // namespace

hipError_t launch_distill_fwd(const Distill &p, void *workspace, hipStream_t s)
{
    const RowPlan plan = row_plan(p.n, p.V, 4, kMaxPartSegs);
    const int64_t parts = plan.parts, esz = p.bf16 ? 2 : 4;
    const int64_t chunk = std::max<int64_t>(1, kMaxItems / 1024 / parts);
    for (int64_t r0 = 0; r0 < p.n; r0 += chunk) {
        const int64_t nr = std::min(chunk, p.n - r0);
        const char *z = static_cast<const char *>(p.logits) + r0 * p.ld * esz;
        const float *temp = p.temperature ? p.temperature + r0 * p.temperature_stride : nullptr;
        float2 *rec = static_cast<float2 *>(workspace) + r0 * parts;
        float *loss = p.loss ? p.loss + r0 : nullptr;
        RowStats *stats = reinterpret_cast<RowStats *>(p.stats) + r0;
        const ListArgs list = list_args(p, r0);
        const unsigned bits = p.tail ? static_cast<unsigned>(std::min<int64_t>(plan.part_segs, row_segments(p.V))) * (kSegCols / 8) : 0;
        auto rows = [&](auto bf16, auto tail, auto waves) {
            constexpr int NW = decltype(waves)::value;
            hipLaunchKernelGGL((distill_row_kernel<decltype(bf16)::value, decltype(tail)::value, NW>),
                               dim3(static_cast<unsigned>(nr * parts)), dim3(NW * 64), bits, s, z, p.ld, p.V,
                               static_cast<uint32_t>(parts), plan.part_segs, list, temp, p.temperature_stride, rec,
                               loss, stats);
        };
        const auto yes = std::true_type{};
        const auto no = std::false_type{};
        auto with_waves = [&](auto bf16, auto tail) {
            if (plan.waves == 4)
                rows(bf16, tail, std::integral_constant<int, 4>{});
            else if (plan.waves == 8)
                rows(bf16, tail, std::integral_constant<int, 8>{});
            else
                rows(bf16, tail, std::integral_constant<int, 16>{});
        };
        auto with_tail = [&](auto bf16) { p.tail ? with_waves(bf16, yes) : with_waves(bf16, no); };
        p.bf16 ? with_tail(yes) : with_tail(no);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        if (parts == 1)
            continue;
        auto merge = [&](auto tail) {
            hipLaunchKernelGGL((distill_merge_kernel<decltype(tail)::value>), dim3(static_cast<unsigned>(nr)),
                               dim3(kListThreads), 0, s, z, p.ld * esz, p.bf16 ? 1 : 0, p.V,
                               static_cast<int32_t>(parts), list, temp, p.temperature_stride, rec, loss, stats);
        };
        p.tail ? merge(yes) : merge(no);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_distill_bwd(const Distill &p, hipStream_t s)
{
    const int64_t zsz = p.bf16 ? 2 : 4, gsz = p.grad_bf16 ? 2 : 4, G = zsz + gsz == 4 ? 8 : 4;
    const int64_t per = kBwdThreads * kBwdVecs;
    const int64_t chunks = std::max<int64_t>(1, (p.V / G + per - 1) / per);
    const int64_t rows = std::max<int64_t>(1, kMaxItems / kBwdThreads / chunks);
    for (int64_t r0 = 0; r0 < p.n; r0 += rows) {
        const int64_t nr = std::min(rows, p.n - r0);
        auto go = [&](auto zb, auto gb) {
            hipLaunchKernelGGL((distill_bwd_kernel<decltype(zb)::value, decltype(gb)::value>),
                               dim3(static_cast<unsigned>(nr * chunks)), dim3(kBwdThreads), 0, s,
                               static_cast<const char *>(p.logits) + r0 * p.ld * zsz, p.ld,
                               reinterpret_cast<const RowStats *>(p.stats) + r0, list_args(p, r0),
                               p.temperature ? p.temperature + r0 * p.temperature_stride : nullptr,
                               p.temperature_stride, p.dloss + r0 * p.dloss_stride, p.dloss_stride,
                               static_cast<char *>(p.dlogits) + r0 * p.ldg * gsz, p.ldg, p.V,
                               static_cast<uint32_t>(chunks));
        };
        const auto yes = std::true_type{};
        const auto no = std::false_type{};
        auto with_grad = [&](auto zb) { p.grad_bf16 ? go(zb, yes) : go(zb, no); };
        p.bf16 ? with_grad(yes) : with_grad(no);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// Rows of at most this many columns fit the registers of a workgroup; longer ones
// are read twice, by the forward and by the gradient.
constexpr int64_t kFusedMaxCols = 65536;

hipError_t launch_distill_fused(const Distill &p, void *workspace, hipStream_t s)
{
    if (p.V > kFusedMaxCols) {
        const hipError_t e = launch_distill_fwd(p, workspace, s);
        return e == hipSuccess ? launch_distill_bwd(p, s) : e;
    }
    const int64_t zsz = p.bf16 ? 2 : 4, gsz = p.grad_bf16 ? 2 : 4;
    const int64_t chunk = kMaxItems / 1024;
    for (int64_t r0 = 0; r0 < p.n; r0 += chunk) {
        const int64_t nr = std::min(chunk, p.n - r0);
        auto go = [&](auto zb, auto gb, auto tail, auto threads, auto vals) {
            constexpr int NT = decltype(threads)::value;
            hipLaunchKernelGGL((distill_fused_kernel<decltype(zb)::value, decltype(gb)::value, decltype(tail)::value,
                                                     NT, decltype(vals)::value>),
                               dim3(static_cast<unsigned>(nr)), dim3(NT), 0, s,
                               static_cast<const char *>(p.logits) + r0 * p.ld * zsz, p.ld, p.V, list_args(p, r0),
                               p.temperature ? p.temperature + r0 * p.temperature_stride : nullptr,
                               p.temperature_stride, p.dloss + r0 * p.dloss_stride, p.dloss_stride,
                               p.loss ? p.loss + r0 : nullptr, reinterpret_cast<RowStats *>(p.stats) + r0,
                               static_cast<char *>(p.dlogits) + r0 * p.ldg * gsz, p.ldg);
        };
        const auto yes = std::true_type{};
        const auto no = std::false_type{};
        auto with_size = [&](auto zb, auto gb, auto tail) {
            if (p.V <= 256 * 32)
                go(zb, gb, tail, std::integral_constant<int, 256>{}, std::integral_constant<int, 32>{});
            else if (p.V <= 512 * 32)
                go(zb, gb, tail, std::integral_constant<int, 512>{}, std::integral_constant<int, 32>{});
            else if (p.V <= 512 * 64 && p.n <= 256)
                // A CU per row: twice the waves take 11 instead of 12 us (128 rows of
                // 32768); two rows per CU in half the waves 42 instead of 49 us (1024).
                go(zb, gb, tail, std::integral_constant<int, 1024>{}, std::integral_constant<int, 32>{});
            else if (p.V <= 512 * 64)
                go(zb, gb, tail, std::integral_constant<int, 512>{}, std::integral_constant<int, 64>{});
            else
                go(zb, gb, tail, std::integral_constant<int, 1024>{}, std::integral_constant<int, 64>{});
        };
        auto with_tail = [&](auto zb, auto gb) { p.tail ? with_size(zb, gb, yes) : with_size(zb, gb, no); };
        auto with_grad = [&](auto zb) { p.grad_bf16 ? with_tail(zb, yes) : with_tail(zb, no); };
        p.bf16 ? with_grad(yes) : with_grad(no);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace lmh
