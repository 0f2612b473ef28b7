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

// A row's record, kDistillStats floats.
struct alignas(16) RowStats {
    float m, d;          // of the whole row
    float loss;
    float weight;        // Q: 1, or 0 where the list is empty
    float other, w;      // gradient off the list: exp((z - other) / T) w / T
    float top, sum;      // q_l = exp((v_l - top) / T_v) / sum, T_v = T or (tail mode) 1
};
static_assert(sizeof(RowStats) == 32, "eight floats");

// One wave, a workgroup of its own, per (row, segment of 2048 columns): {m, d},
// with TAIL of the columns that are not on the row's list.
template <bool BF16, bool TAIL>
__global__ __launch_bounds__(64) void distill_scan_kernel(
    const void *__restrict__ logits, int64_t ld, int64_t V, uint32_t nseg, ListArgs list,
    const float *__restrict__ temperature, int64_t temperature_stride, float2 *__restrict__ rec)
{
    constexpr int G = Segment<BF16>::G;
    const int lane = threadIdx.x;
    const uint32_t id = blockIdx.x, row = id / nseg;  // below 2^25
    const int64_t j0 = static_cast<int64_t>(id - row * nseg) * kSegCols;
    const char *zr = static_cast<const char *>(logits) + static_cast<int64_t>(row) * ld * (16 / G);
    Segment<BF16> sg;
    sg.load(zr, V, j0, lane);
    __shared__ uint32_t listed[TAIL ? kSegCols / 32 : 1];  // a bit per column
    if constexpr (TAIL) {
        listed[lane] = 0;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        for (int i = lane; i < list.k; i += 64) {
            const int64_t at = static_cast<int64_t>(entry(list, row, i).token) - j0;
            if (at >= 0 && at < kSegCols)
                atomicOr(&listed[at >> 5], 1u << (at & 31));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    float v[32];
    sg.values(v);
    if constexpr (TAIL) {
#pragma unroll
        for (int u = 0; u < 32 / G; ++u) {
            const int col = (64 * u + lane) * G;
            const uint32_t bits = listed[col >> 5] >> (col & 31);
#pragma unroll
            for (int e = 0; e < G; ++e)
                v[u * G + e] = (bits >> e) & 1u ? -INFINITY : v[u * G + e];
        }
    }
    const float c = kLog2e * inverse_temperature(temperature, row * temperature_stride);
    float lm = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        lm = __builtin_elementwise_maximum(lm, v[i]);  // NaN stays NaN
    const float m = wave_maximum(lm);
    float d = 0.0f;
    if (m != -INFINITY) {  // +inf or NaN make d NaN
#pragma unroll
        for (int i = 0; i < 32; ++i)
            d += __builtin_amdgcn_exp2f((v[i] - m) * c);
        d = wave_sum(d);
    }
    if (lane == 0)
        rec[id] = make_float2(m, d);
}

__device__ __forceinline__ double block_sum(double v, double *red, int wave, int lane)
{
    v = wave_sum(v);
    __syncthreads();
    if (lane == 0)
        red[wave] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kListThreads / 64; ++w)
        v += red[w];
    return v;
}

// One workgroup per row, a thread per entry of its list: the row's sums from its
// segments' records, the loss and what the gradient needs, in 64 bits.
__global__ __launch_bounds__(kListThreads) void distill_merge_kernel(
    const char *__restrict__ logits, int64_t ld_bytes, int32_t bf16, int64_t V, int32_t nseg, ListArgs list,
    const float *__restrict__ temperature, int64_t temperature_stride, const float2 *__restrict__ rec,
    float *__restrict__ loss, RowStats *__restrict__ stats)
{
    __shared__ int32_t ids[kMaxList];
    __shared__ double red[kListThreads / 64];
    __shared__ float red_f[kListThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x;
    const Entry en = entry(list, row, tid);
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const char *zr = logits + row * ld_bytes;
    const bool there = en.token >= 0;
    const bool off = there && en.token >= V;
    float z = -INFINITY;
    if (there && !off)
        z = bf16 ? row_element<true>(zr, en.token) : row_element<false>(zr, en.token);
    ids[tid] = en.token;
    const int n_there = __syncthreads_count(there);
    const bool any_off = __syncthreads_or(off);
    if (n_there == 0) {
        if (tid == 0) {
            stats[row] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (loss)
                loss[row] = 0.0f;
        }
        return;
    }
    auto block_max = [&](float v) {
        v = wave_maximum(v);
        __syncthreads();
        if (lane == 0)
            red_f[wave] = v;
        __syncthreads();
        v = red_f[0];
        for (int w = 1; w < kListThreads / 64; ++w)
            v = __builtin_elementwise_maximum(v, red_f[w]);
        return v;
    };
    // The student's sums over the scanned columns (all, or those off the list).
    const float2 *r = rec + row * nseg;
    float m_o = -INFINITY;
    for (int i = tid; i < nseg; i += kListThreads)
        m_o = __builtin_elementwise_maximum(m_o, r[i].x);
    m_o = block_max(m_o);
    double d_o = 0.0;
    for (int i = tid; i < nseg; i += kListThreads) {
        const float2 q = r[i];
        if (q.y != 0.0f)  // NaN too
            d_o += static_cast<double>(q.y) * exp((static_cast<double>(q.x) - m_o) * inv_t);
    }
    d_o = block_sum(d_o, red, wave, lane);
    float m = m_o;
    double d = d_o;
    if (list.tail) {
        // The list's columns join, each once.
        bool first = there && !off;
        for (int i = 0; i < tid && first; ++i)
            first = ids[i] != en.token;
        m = __builtin_elementwise_maximum(m_o, block_max(z));
        d = block_sum(first && z != -INFINITY ? exp((static_cast<double>(z) - m) * inv_t) : 0.0, red, wave, lane);
        if (d_o != 0.0)
            d += d_o * exp((static_cast<double>(m_o) - m) * inv_t);
    }
    // The teacher.
    float top = 0.0f;
    double log_q = -INFINITY, sum = 1.0;
    if (list.tail) {
        if (there)
            log_q = en.value;
    } else {
        top = block_max(there ? en.value : -INFINITY);
        const double x = there ? (static_cast<double>(en.value) - top) * inv_t : -static_cast<double>(INFINITY);
        sum = block_sum(there ? exp(x) : 0.0, red, wave, lane);
        log_q = x - log(sum);
    }
    const double q = there ? exp(log_q) : 0.0;
    const double log_d = log(d);
    const double log_p = (static_cast<double>(z) - m) * inv_t - log_d;
    const double total = block_sum(q, red, wave, lane);
    double l = block_sum(q != 0.0 ? q * (log_q - log_p) : 0.0, red, wave, lane);
    if (tid != 0)
        return;
    double weight = total, w = total / d;
    if (list.tail) {
        w = 0.0;
        if (d_o != 0.0) {  // there are other columns (or a NaN)
            const double shift = (static_cast<double>(m_o) - m) * inv_t;
            const double q_r = total == total ? fmax(0.0, 1.0 - total) : total;
            weight = total + q_r;
            if (q_r != 0.0)
                l += q_r * (log(q_r) - (shift + log(d_o) - log_d));
            w = weight * exp(shift) / d - q_r / d_o;
        }
    }
    if (any_off || !(d > 0.0) || !(total < INFINITY))
        l = w = weight = static_cast<double>(NAN);
    // No other column above -inf: any finite shift gives them exp(-inf) w = 0.
    const float other = m_o == -INFINITY ? m : m_o;
    stats[row] = {m, static_cast<float>(d), static_cast<float>(l), static_cast<float>(weight),
                  other, static_cast<float>(w), top, static_cast<float>(sum)};
    if (loss)
        loss[row] = static_cast<float>(l);
}

// ------------------------------------------------------------------ gradient

constexpr int kBwdThreads = kListThreads;
constexpr int kBwdVecs = 4;  // 16-byte loads per thread

// One chunk of kBwdVecs x 256 vectors of 16 bytes of a row per workgroup.  Every
// column is first written as if it were off the list; the threads of the chunk's
// listed columns then write theirs over it.
template <bool ZBF16, bool GBF16>
__global__ __launch_bounds__(kBwdThreads) void distill_bwd_kernel(
    const void *logits, int64_t ld, const RowStats *__restrict__ stats, ListArgs list,
    const float *__restrict__ temperature, int64_t temperature_stride, const float *__restrict__ dloss,
    int64_t dloss_stride, void *dlogits, int64_t ldg, int64_t V, uint32_t chunks)
{
    constexpr int G = ZBF16 ? 8 : 4;
    constexpr int NW = kBwdThreads / 64;
    __shared__ int32_t ids[kBwdThreads];
    __shared__ float qs[kBwdThreads];
    __shared__ int32_t counts[NW];
    const uint32_t id = blockIdx.x, row = id / chunks, chunk = id - row * chunks;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t nv = V / G;
    const RowStats st = stats[row];
    const float inv_t = inverse_temperature(temperature, row * temperature_stride);
    const float c = kLog2e * inv_t, up = dloss[row * dloss_stride] * inv_t, w_up = st.w * up;
    const bool nothing = up == 0.0f || (st.weight == 0.0f && st.w == 0.0f);  // the row is not read
    const char *zr = static_cast<const char *>(logits) + static_cast<int64_t>(row) * ld * (16 / G);
    char *gr = static_cast<char *>(dlogits) + static_cast<int64_t>(row) * ldg * (GBF16 ? 2 : 4);

    const int64_t first = static_cast<int64_t>(chunk) * kBwdThreads * kBwdVecs;
    const bool last = chunk == chunks - 1;
    uint4 q[kBwdVecs];
    float listed_grad = 0.0f;
    int64_t listed_at = -1;
    if (!nothing) {
#pragma unroll
        for (int u = 0; u < kBwdVecs; ++u) {
            const int64_t i = first + u * kBwdThreads + tid;
            if (i < nv)
                q[u] = load_row(zr, i);
        }
        // The list's entries in this chunk, compacted in each wave's quarter.
        const Entry en = entry(list, row, tid);
        const int64_t end = last ? V : (first + kBwdThreads * kBwdVecs) * G;
        const bool here = en.token >= first * G && en.token < end;
        const float t_inv = list.tail ? 1.0f : inv_t;
        const uint64_t mask = __ballot(here);
        if (here) {
            const int at = wave * 64 + __popcll(mask & ((1ull << lane) - 1ull));
            ids[at] = en.token;
            qs[at] = __builtin_amdgcn_exp2f((en.value - st.top) * (kLog2e * t_inv)) / st.sum;
            const float z = row_element<ZBF16>(zr, en.token);
            listed_grad = __builtin_amdgcn_exp2f((z - st.m) * c) * (st.weight / st.d);
            listed_at = en.token;
        }
        if (lane == 0)
            counts[wave] = __popcll(mask);
        __syncthreads();  // the list's logits are read before the row is written (in place)
        if (here) {
            float sum = 0.0f;
            for (int v = 0; v < NW; ++v)
                for (int i = 0; i < counts[v]; ++i)
                    sum += ids[v * 64 + i] == en.token ? qs[v * 64 + i] : 0.0f;
            listed_grad = (listed_grad - sum) * up;
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
            o[e] = nothing ? 0.0f : value(row_value<ZBF16>(q[u], e));
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
        if (listed_at >= 0)
            store_element<GBF16>(gr, listed_at, listed_grad);
    }
}

}  // namespace

int64_t distill_workspace_bytes(int64_t n_rows, int64_t V)
{
    return n_rows * row_segments(V) * static_cast<int64_t>(sizeof(float2));
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
    const int64_t nseg = row_segments(p.V), esz = p.bf16 ? 2 : 4;
    const int64_t chunk = std::max<int64_t>(1, kMaxItems / kListThreads / nseg);
    for (int64_t r0 = 0; r0 < p.n; r0 += chunk) {
        const int64_t nr = std::min(chunk, p.n - r0);
        const char *z = static_cast<const char *>(p.logits) + r0 * p.ld * esz;
        const float *temp = p.temperature ? p.temperature + r0 * p.temperature_stride : nullptr;
        float2 *rec = static_cast<float2 *>(workspace) + r0 * nseg;
        const ListArgs list = list_args(p, r0);
        auto scan = [&](auto bf16, auto tail) {
            hipLaunchKernelGGL((distill_scan_kernel<decltype(bf16)::value, decltype(tail)::value>),
                               dim3(static_cast<unsigned>(nr * nseg)), dim3(64), 0, s, z, p.ld, p.V,
                               static_cast<uint32_t>(nseg), list, temp, p.temperature_stride, rec);
        };
        const auto yes = std::true_type{};
        const auto no = std::false_type{};
        auto with_tail = [&](auto bf16) { p.tail ? scan(bf16, yes) : scan(bf16, no); };
        p.bf16 ? with_tail(yes) : with_tail(no);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        hipLaunchKernelGGL(distill_merge_kernel, dim3(static_cast<unsigned>(nr)), dim3(kListThreads), 0, s, z,
                           p.ld * esz, p.bf16 ? 1 : 0, p.V, static_cast<int32_t>(nseg), list, temp,
                           p.temperature_stride, rec, p.loss ? p.loss + r0 : nullptr,
                           reinterpret_cast<RowStats *>(p.stats) + r0);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_distill_bwd(const Distill &p, hipStream_t s)
{
    const int64_t zsz = p.bf16 ? 2 : 4, gsz = p.grad_bf16 ? 2 : 4, G = 16 / zsz;
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

hipError_t launch_distill_fused(const Distill &p, void *workspace, hipStream_t s)
{
    const hipError_t e = launch_distill_fwd(p, workspace, s);
    return e == hipSuccess ? launch_distill_bwd(p, s) : e;
}

}  // namespace lmh
