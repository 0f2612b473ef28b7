// lora.hip -- low-rank adapters of many requests beside the shared vocabulary
// weight, on gfx950: the adapters' part of the logits and their gradients.
//
// Token m uses adapter a = adapter[m] (a < 0: none), A_a [r][K], B_a [V][r]:
//   z[m][v]    = sum_k x[m][k] W[v][k] + sum_j u[m][j] B_a[v][j],
//   u[m][j]    = s_a sum_k x[m][k] A_a[j][k]
//   t[m][j]    = s_a sum_v g[m][v] B_a[v][j]          (g = dlogits)
//   dX[m][k]   = sum_j t[m][j] A_a[j][k]
//   dA_a[j][k] = sum over a's tokens of t[m][j] x[m][k]
//   dB_a[v][j] = sum over a's tokens of g[m][v] u[m][j]
//
// Every product runs on the BF16 matrix cores with FP32 accumulation.  u and t
// are FP32 sums that enter a second product; rounding them to BF16 would leave
// the FP32 logits and gradients with 2^-9 relative errors in the adapter's
// part, so each is cut into three BF16 pieces of 8 significant bits (hi + mid
// + lo = the FP32 value exactly, truncating) and the product runs over the
// three pieces: 3 r extra contraction steps against K or V of the main
// products.
//
// A batch mixes requests.  A tile's tokens may use different adapters, and one
// request's adapter must never touch another's result (0 x NaN included), so
// an adapter's product is formed for the whole tile into registers of its own
// and added only in the columns (tokens) that use it.
#include "common.h"

#include <algorithm>

namespace lmh {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int64_t kMaxItems = int64_t{1} << 31;  // work-items per launch

// 8 BF16 words at p, of which the first n (any value) are valid, the rest 0.
__device__ __forceinline__ uint4 load8(const uint16_t *p, int64_t n)
{
    if (n >= 8)
        return *reinterpret_cast<const uint4 *>(p);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n)
            w[e >> 1] |= static_cast<uint32_t>(p[e]) << ((e & 1) * 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ bf16x8 as_frag(const uint4 &v)
{
    return __builtin_bit_cast(bf16x8, v);
}

// The first n of 8 BF16 words, the rest 0.
__device__ __forceinline__ uint4 keep8(uint4 v, int64_t n)
{
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = n >= 2 * i + 2 ? in[i] : n == 2 * i + 1 ? (in[i] & 0xffffu) : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c)
{
    // Lane l: a row l % 16, b column l % 16, both at contraction 8 (l / 16) ..;
    // c rows 4 (l / 16) .. + 3, column l % 16.
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// FP32 -> three BF16 pieces whose sum is the value: each the upper 16 bits of
// what is left.  A non-finite value keeps it all in the first.
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3])
{
    const uint32_t hi = __float_as_uint(v) & 0xffff0000u;
    const bool finite = (hi & 0x7f800000u) != 0x7f800000u;
    const float r1 = v - __uint_as_float(hi);
    const uint32_t mid = __float_as_uint(r1) & 0xffff0000u;
    const float r2 = r1 - __uint_as_float(mid);
    p[0] = (v != v) ? 0x7fc0u : hi >> 16;
    p[1] = finite ? mid >> 16 : 0u;
    p[2] = finite ? __float_as_uint(r2) >> 16 : 0u;
}

// Adapters a tile's 16 tokens use: lane l holds token l % 16's id; bit t of the
// mask is token t.
__device__ __forceinline__ int32_t first_id(int32_t id, uint32_t todo)
{
    return __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
}
__device__ __forceinline__ uint32_t tokens_of(int32_t id, int32_t a)
{
    return static_cast<uint32_t>(__ballot(id == a)) & 0xffffu;
}

// Row length of the pieces of one token's u or t: [hi | mid | lo] of RP words
// each, RP the rank rounded up to 16, 32, 64 or 128; for RP = 16 one more
// group of 16 zeros makes whole 32-deep contraction steps.
__host__ __device__ constexpr int piece_row(int RP)
{
    return RP == 16 ? 64 : 3 * RP;
}

// Batches of at most kFewTokens tokens are walked by adapter instead of by
// blocks of 16 tokens: each adapter's weights are then read once per tile however
// the batch mixes its requests, the adapters spread over workgroups, and two
// launches do instead of three.  Shrink (and join) + expand at 256 tokens this
// way and at 257 the other, K = 4096, V = 32768: 32 mixed adapters of rank 16 40
// and 51 us, 4 in runs 34 and 33 us; 16 mixed of rank 64 50 and 65 us, 4 in runs
// 43 and 41 us.
constexpr int kFewTokens = 256;

// Such a batch in units of up to 16 tokens of one adapter: unit i holds tokens
// order[first .. first + count), ascending, of adapter id; count 0 past the
// last unit.  Tokens on none form units of id -1, all those whose id is no
// adapter units of id n.
struct FewUnit {
    int32_t id, first, count, pad;
};
struct FewUnits {
    FewUnit u[kFewTokens];
    int32_t order[kFewTokens];
};

// Fills `t` (LDS) from the ids; 1024 threads.  Every token's id is compared with
// all others, a quarter of them per thread (walking the distinct ids one after
// another took 0.5 us each).
__device__ __forceinline__ void group_few(const LoraAdapters &ad, int64_t M, FewUnits &t, int tid)
{
    __shared__ __attribute__((aligned(16))) int32_t ids[kFewTokens];
    __shared__ int32_t cnt[4][kFewTokens], ahead[4][kFewTokens], first[4][kFewTokens];
    __shared__ int32_t lead_start[kFewTokens], sums[2][4];
    if (tid < kFewTokens) {
        const int32_t v = tid < M ? ad.adapter[tid] : 0;
        ids[tid] = tid >= M ? -2 : v < 0 ? -1 : v >= ad.n ? static_cast<int32_t>(ad.n) : v;
        t.u[tid] = FewUnit{-1, 0, 0, 0};
    }
    __syncthreads();
    const int m = tid & (kFewTokens - 1), part = tid / kFewTokens, lane = tid & 63;
    const int32_t id = ids[m];
    int c = 0, before = 0, f = kFewTokens;
    const int quarter = (static_cast<int>(M) + 15) / 16 * 4;  // whole vectors; past M no id matches
    for (int i = quarter * part; i < min(quarter * part + quarter, kFewTokens); i += 4) {
        const int4 o = *reinterpret_cast<const int4 *>(ids + i);
        const int32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool same = w[e] == id;
            c += same;
            before += same && i + e < m;
            f = same ? min(f, i + e) : f;
        }
    }
    cnt[part][m] = c, ahead[part][m] = before, first[part][m] = f;
    __syncthreads();
    // Two scans in token order: the tokens of groups that began earlier (at a
    // group's first token), and the units that began earlier (at every 16th
    // token of a group).
    int lead = 0, unit = 0, lead_sum = 0, unit_sum = 0;
    if (tid < kFewTokens) {
        c = cnt[0][m] + cnt[1][m] + cnt[2][m] + cnt[3][m];
        before = ahead[0][m] + ahead[1][m] + ahead[2][m] + ahead[3][m];
        f = min(min(first[0][m], first[1][m]), min(first[2][m], first[3][m]));
        lead_sum = lead = id != -2 && before == 0 ? c : 0;
        unit_sum = unit = id != -2 && before % 16 == 0 ? 1 : 0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int ol = __shfl_up(lead_sum, off, 64), ou = __shfl_up(unit_sum, off, 64);
            lead_sum += lane >= off ? ol : 0;
            unit_sum += lane >= off ? ou : 0;
        }
        if (lane == 63)
            sums[0][tid >> 6] = lead_sum, sums[1][tid >> 6] = unit_sum;
    }
    __syncthreads();
    if (tid < kFewTokens) {
        lead_sum -= lead, unit_sum -= unit;
        for (int w = 0; w < (tid >> 6); ++w)
            lead_sum += sums[0][w], unit_sum += sums[1][w];
        if (lead)
            lead_start[m] = lead_sum;
    }
    __syncthreads();
    if (tid < kFewTokens && id != -2) {
        const int at = lead_start[f] + before;
        t.order[at] = m;
        if (unit)
            t.u[unit_sum] = FewUnit{id, at, min(16, c - before), 0};
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// The gradients' grouping of the tokens by adapter (stable): group g < n
// holds adapter g's tokens, group n the tokens on none, group n + 1 those
// whose id is not an adapter.  offset[g] is the group's first place in order[].
// Chunks of up to 64 tokens of one group are numbered too: those of group g
// start at chunk_base(offset[g], g), with some numbers unused, so that a
// workgroup can be given a chunk without knowing the counts.
__host__ __device__ __forceinline__ int64_t chunk_base(int64_t offset, int64_t g)
{
    // Room enough: floor((o + c) / 64) - floor(o / 64) + 1 >= ceil(c / 64).
    return offset / 64 + g;
}

struct Chunk {
    int32_t group, first, count, pad;  // its tokens are order[first .. first + count); group -1: unused
};

struct Grouping {
    int32_t *offset, *order;
    Chunk *chunks;
};

// The work of one workgroup of NT threads for group g: counts the ids below and
// in its group, then writes its tokens in order, and its chunks.  All groups
// together read the ids n + 2 times (they stay in L2); no workgroup waits for
// another.
template <int NT>
__device__ __forceinline__ void group_tokens(const int32_t *__restrict__ adapter, int64_t M, int64_t n,
                                             const Grouping &out, int64_t g)
{
    constexpr int NW = NT / 64;
    __shared__ int32_t part[2][NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto cls = [&](int32_t id) { return id < 0 ? n : id >= n ? n + 1 : static_cast<int64_t>(id); };
    int32_t less = 0, same = 0;
#pragma unroll 4
    for (int64_t m = tid; m < M; m += NT) {
        const int64_t c = cls(adapter[m]);
        less += c < g;
        same += c == g;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        less += __shfl_xor(less, off, 64);
        same += __shfl_xor(same, off, 64);
    }
    if (lane == 0)
        part[0][wave] = less, part[1][wave] = same;
    __syncthreads();
    int32_t first = 0, count = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        first += part[0][w], count += part[1][w];
    if (tid == 0) {
        out.offset[g] = first;
        if (g == n + 1)
            out.offset[n + 2] = static_cast<int32_t>(M);
    }
    const int64_t c0 = chunk_base(first, g), c1 = chunk_base(first + count, g + 1);
    for (int64_t c = c0 + tid; c < c1; c += NT) {
        const int32_t at = static_cast<int32_t>(64 * (c - c0));
        out.chunks[c] = at < count ? Chunk{static_cast<int32_t>(g), first + at, min(64, count - at), 0}
                                   : Chunk{-1, 0, 0, 0};
    }
    if (count == 0)
        return;
    int32_t done = 0;
    for (int64_t m0 = 0; m0 < M && done < count; m0 += NT) {
        const int64_t m = m0 + tid;
        const bool mine = m < M && cls(adapter[m]) == g;
        const uint64_t mask = __ballot(mine);
        __syncthreads();  // the round before has read part[0]
        if (lane == 0)
            part[0][wave] = __popcll(mask);
        __syncthreads();
        int32_t at = done + __popcll(mask & ((1ull << lane) - 1ull));
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            at += w < wave ? part[0][w] : 0;
            done += part[0][w];
        }
        if (mine)
            out.order[first + at] = static_cast<int32_t>(m);
    }
}

// The logits' order of more than kFewTokens tokens: by adapter within windows of
// kWindow tokens (then by place), tokens on none last, so that a block of 16 in
// that order has one adapter or two however the batch mixes its requests (320
// tokens mixing 16 adapters of rank 64, V = 32768: expand 131 -> 38 us; runs as
// before).  One
// workgroup of 256 per 64 tokens (lane: token), each wave counting the keys ahead
// of them in a quarter of the window.
constexpr int kWindow = 1024;

__device__ __forceinline__ void order_tokens(const int32_t *__restrict__ adapter, int64_t M,
                                             int32_t *__restrict__ order, int64_t block)
{
    __shared__ __attribute__((aligned(16))) uint32_t key[kWindow];
    __shared__ int32_t part[4][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t w0 = block * 64 / kWindow * kWindow;
    for (int i = tid; i < kWindow; i += 256)  // none: 2^31 and up; past M: the last
        key[i] = w0 + i < M ? static_cast<uint32_t>(adapter[w0 + i]) : 0xffffffffu;
    __syncthreads();
    const int me = static_cast<int>(block * 64 - w0) + lane;
    const uint32_t k = key[me];
    int ahead = 0;
#pragma unroll 4
    for (int i = wave * (kWindow / 4); i < (wave + 1) * (kWindow / 4); i += 4) {
        const uint4 o = *reinterpret_cast<const uint4 *>(key + i);
        const uint32_t v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            ahead += v[e] < k || (v[e] == k && i + e < me);
    }
    part[wave][lane] = ahead;
    __syncthreads();
    if (wave == 0 && w0 + me < M)
        order[w0 + part[0][lane] + part[1][lane] + part[2][lane] + part[3][lane]] =
            static_cast<int32_t>(w0 + me);
}

__global__ __launch_bounds__(256) void lora_group_kernel(const int32_t *__restrict__ adapter, int64_t M,
                                                         int64_t n, Grouping out)
{
    group_tokens<256>(adapter, M, n, out, blockIdx.x);
}

// ---------------------------------------------------------------------------
// u = s_a A_a x, 16 tokens by 16 ranks at a time; NW waves of a workgroup split
// K and are summed in order through LDS.  Written as pieces, rows
// [token][piece_row].
//
// The wave's part of the 16 x 16 result over K range [k, kend) (k a multiple of
// 32): pa and px point at the lane's row, its eight columns of a step.
__device__ __forceinline__ f32x4 shrink_wave(const uint16_t *pa, const uint16_t *px, int64_t k, int64_t kend,
                                             int64_t K, int q)
{
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (; k + 256 <= kend; k += 256) {
        uint4 va[8], vx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            va[i] = *reinterpret_cast<const uint4 *>(pa + k + 32 * i);
            vx[i] = *reinterpret_cast<const uint4 *>(px + k + 32 * i);
        }
        __builtin_amdgcn_sched_barrier(0);  // all sixteen in flight
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc = mfma16(as_frag(va[i]), as_frag(vx[i]), acc);
    }
    for (; k + 64 <= kend; k += 64) {
        uint4 va[2], vx[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            va[i] = *reinterpret_cast<const uint4 *>(pa + k + 32 * i);
            vx[i] = *reinterpret_cast<const uint4 *>(px + k + 32 * i);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            acc = mfma16(as_frag(va[i]), as_frag(vx[i]), acc);
    }
    for (; k < kend; k += 32) {
        const int64_t left = K - k - 8 * q;
        acc = mfma16(as_frag(load8(pa + k, left)), as_frag(load8(px + k, left)), acc);
    }
    return acc;
}

// The sum over the waves of rank tid / 16, token tid % 16 (threads below 256).
template <int NW>
__device__ __forceinline__ float shrink_sum(const f32x4 (&red)[NW][64], int tid)
{
    const int jj = tid >> 4, t16 = tid & 15;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        sum += red[w][(jj >> 2) * 16 + t16][jj & 3];
    return sum;
}

// At most kFewTokens tokens: one workgroup per unit (blockIdx.x) and 16 ranks,
// all of K in it -- latency-bound, and a second launch to join parts would cost
// more.  Leaves the units in `table` for the next kernel.  The first n_groups
// workgroups group the tokens for the gradients instead.
constexpr int kShrinkThreads = 1024;

__global__ void __launch_bounds__(kShrinkThreads) __attribute__((amdgpu_waves_per_eu(4, 4)))
lora_shrink_few_kernel(const uint16_t *__restrict__ x, int64_t ldx, int64_t M, int64_t K,
                       LoraAdapters ad, int RP, uint16_t *__restrict__ u3,
                       FewUnits *__restrict__ table, Grouping groups, unsigned n_groups)
{
    if (blockIdx.x < n_groups) {
        if (blockIdx.y == 0)
            group_tokens<kShrinkThreads>(ad.adapter, M, ad.n, groups, blockIdx.x);
        return;
    }
    constexpr int NW = kShrinkThreads / 64;
    __shared__ f32x4 red[NW][64];
    __shared__ FewUnits t;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t16 = lane & 15, q = lane >> 4;
    const int j0 = blockIdx.y * 16;
    group_few(ad, M, t, tid);
    if (table && blockIdx.x == 0 && blockIdx.y == 0 && tid < kFewTokens) {
        table->u[tid] = t.u[tid];
        table->order[tid] = t.order[tid];
    }
    const FewUnit u = t.u[blockIdx.x - n_groups];
    if (u.count == 0 || u.id < 0 || u.id >= ad.n)
        return;
    const float scale = ad.scale ? ad.scale[u.id] : 1.0f;
    const int64_t tok = t.order[u.first + min(t16, u.count - 1)];
    const int64_t per_wave = (K + 32 * NW - 1) / (32 * NW) * 32, k0 = wave * per_wave;
    red[wave][lane] = shrink_wave(
        ad.A + u.id * ad.stride_a + static_cast<int64_t>(min(j0 + t16, ad.r - 1)) * ad.lda + 8 * q,
        x + tok * ldx + 8 * q, k0, min(K, k0 + per_wave), K, q);
    __syncthreads();
    if (tid >= 256 || t16 >= u.count)
        return;
    const int j = j0 + (tid >> 4);
    const float sum = shrink_sum(red, tid);
    uint32_t p[3];
    split3(j < ad.r ? sum * scale : 0.0f, p);
    uint16_t *row = u3 + tok * piece_row(RP) + j;
    row[0] = static_cast<uint16_t>(p[0]);
    row[RP] = static_cast<uint16_t>(p[1]);
    row[2 * RP] = static_cast<uint16_t>(p[2]);
    if (RP == 16)
        row[48] = 0;
}

// Any number of tokens: each wave takes 16 neighbouring ones, all ranks and one
// of the S parts of K (blockIdx.x = (block S + part), four waves a block); the
// distinct adapters the tokens use, in token order, go round the blockIdx.y
// slots.  A CU draws some 20 - 50 GB/s, so what counts is how few bytes reach
// it and that every CU has some: x once for all ranks, A shared by the four
// waves through L1, K in parts whose sums [S][M][RP] lora_join_kernel adds.
// (M = 1024, K = 8192: rank 64 read 16 x 16 at a time 22 - 30 us.)  The first
// n_groups workgroups group the tokens for the gradients, or (no `offset`) put
// them in the logits' order, instead.
template <int RP>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const uint16_t *__restrict__ x, int64_t ldx,
                                                          int64_t M, int64_t K, LoraAdapters ad,
                                                          int S, int64_t part_k,
                                                          float *__restrict__ upart, Grouping groups,
                                                          unsigned n_groups)
{
    if (blockIdx.x < n_groups) {
        if (blockIdx.y != 0)
            return;
        if (groups.offset)
            group_tokens<256>(ad.adapter, M, ad.n, groups, blockIdx.x);
        else
            order_tokens(ad.adapter, M, groups.order, blockIdx.x);
        return;
    }
    constexpr int RB = RP / 16, UN = RB <= 2 ? 8 : RB == 4 ? 4 : 2;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t16 = lane & 15, q = lane >> 4;
    const int64_t wg = blockIdx.x - n_groups, part = wg % S;
    const int64_t tok = (wg / S * 4 + wave) * 16 + t16;
    const int32_t id = tok < M ? ad.adapter[tok] : -1;
    uint32_t todo = static_cast<uint32_t>(__ballot(id >= 0 && id < ad.n)) & 0xffffu;
    const int64_t k0 = part * part_k, kend = min(K, k0 + part_k);
    const uint16_t *px = x + min(tok, M - 1) * ldx + 8 * q;
    for (unsigned slot = 0; todo; ++slot) {
        const int32_t a = first_id(id, todo);
        todo &= ~tokens_of(id, a);
        if (slot % gridDim.y != blockIdx.y)
            continue;
        const uint16_t *pa[RB];
        f32x4 acc[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            pa[b] = ad.A + a * ad.stride_a + static_cast<int64_t>(min(16 * b + t16, ad.r - 1)) * ad.lda + 8 * q;
            acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        int64_t k = k0;
        for (; k + 32 * UN <= kend; k += 32 * UN) {
            uint4 vx[UN], va[UN][RB];
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                vx[i] = *reinterpret_cast<const uint4 *>(px + k + 32 * i);
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    va[i][b] = *reinterpret_cast<const uint4 *>(pa[b] + k + 32 * i);
            }
            __builtin_amdgcn_sched_barrier(0);  // all of them in flight
#pragma unroll
            for (int i = 0; i < UN; ++i)
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    acc[b] = mfma16(as_frag(va[i][b]), as_frag(vx[i]), acc[b]);
        }
        for (; k < kend; k += 32) {
            const int64_t left = K - k - 8 * q;
            const bf16x8 fx = as_frag(load8(px + k, left));
#pragma unroll
            for (int b = 0; b < RB; ++b)
                acc[b] = mfma16(as_frag(load8(pa[b] + k, left)), fx, acc[b]);
        }
        if (id == a) {
            float *p = upart + (part * M + tok) * RP + 4 * q;
#pragma unroll
            for (int b = 0; b < RB; ++b)
                *reinterpret_cast<f32x4 *>(p + 16 * b) = acc[b];
        }
    }
}

// u or t = s_a x the sum of its parts [n_parts][M][RP], in order per lane and
// then by lane: 16 lanes share one group of four ranks of one token.  Written
// as pieces; ranks past r are zero.
__global__ __launch_bounds__(256) void lora_join_kernel(const float *__restrict__ parts, int64_t n_parts,
                                                        int64_t M, int RP, LoraAdapters ad,
                                                        uint16_t *__restrict__ pieces)
{
    __shared__ f32x4 red[16][16];
    const int tid = threadIdx.x, col = tid & 15, part = tid >> 4;
    const int64_t n4 = M * RP / 4;
    const int64_t i4 = static_cast<int64_t>(blockIdx.x) * 16 + col;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (i4 < n4) {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(parts) + i4;
#pragma unroll 8
        for (int64_t b = part; b < n_parts; b += 16)
            sum += p[b * n4];
    }
    red[part][col] = sum;
    __syncthreads();
    if (part != 0 || i4 >= n4)
        return;
#pragma unroll
    for (int w = 1; w < 16; ++w)
        sum += red[w][col];
    const int64_t m = i4 * 4 / RP;
    const int j = static_cast<int>(i4 * 4 - m * RP);
    const int32_t a = ad.adapter[m];
    if (a < 0 || a >= ad.n)
        return;  // its parts were never written, and nothing reads its pieces
    const float s = ad.scale ? ad.scale[a] : 1.0f;
    uint32_t p[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        split3(j + e < ad.r ? sum[e] * s : 0.0f, p[e]);
    uint16_t *row = pieces + m * piece_row(RP) + j;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint2 *>(row + k * RP) =
            make_uint2(p[0][k] | (p[1][k] << 16), p[2][k] | (p[3][k] << 16));
    if (RP == 16)
        *reinterpret_cast<uint2 *>(row + 48) = make_uint2(0u, 0u);
}

// 8 words of a matrix row from column j (a multiple of 8), the row's length r
// (a row pitch is at least r rounded up to 8): words past r are zero.  Only the
// last row of the matrix may end where its storage does, so the others are read
// whole.
__device__ __forceinline__ uint4 load8_row(const uint16_t *row, int j, int r, bool last)
{
    if (j >= r)
        return make_uint4(0u, 0u, 0u, 0u);
    if (j + 8 <= r)
        return *reinterpret_cast<const uint4 *>(row + j);
    return last ? load8(row + j, r - j) : keep8(*reinterpret_cast<const uint4 *>(row + j), r - j);
}

// 16 tokens x 64 vocabulary rows of one adapter's part, turned from the matrix
// layout (lane: token t16, rows 16 i + 4 q ..) into row pieces (lane: token
// 4 i + q of the 16, columns 4 t16 ..) through 4 KiB of the wave's LDS: 16-byte
// chunk c of token t's 64 values sits at c ^ t.
__device__ __forceinline__ void turn_rows(f32x4 (&d)[4], float *own, int t16, int q)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4 *>(own + t16 * 64 + (((4 * i + q) ^ t16) << 2)) = d[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < 4; ++i)
        d[i] = *reinterpret_cast<const f32x4 *>(own + (4 * i + q) * 64 + ((t16 ^ (4 * i + q)) << 2));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Four values of an FP32 row at column v, zero past V.
__device__ __forceinline__ f32x4 load_piece(const float *p, int64_t v, int64_t V)
{
    if (v + 4 <= V)
        return *reinterpret_cast<const f32x4 *>(p + v);
    f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int e = 0; e < 4 && v + e < V; ++e)
        r[e] = p[v + e];
    return r;
}

template <bool BF16>
__device__ __forceinline__ void store_piece(void *out, int64_t row, int64_t v, int64_t V, f32x4 r)
{
    if constexpr (BF16) {
        uint16_t *p = static_cast<uint16_t *>(out) + row + v;
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = f32_to_bf16_bits(r[e]);
        if (v + 4 <= V)
            store8(p, make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16)), false);
        else
            for (int e = 0; e < 4 && v + e < V; ++e)
                p[e] = static_cast<uint16_t>(h[e]);
    } else {
        float *p = static_cast<float *>(out) + row + v;
        if (v + 4 <= V)
            *reinterpret_cast<f32x4 *>(p) = r;
        else
            for (int e = 0; e < 4 && v + e < V; ++e)
                p[e] = r[e];
    }
}

// logits += u B^T for at most kFewTokens tokens: one workgroup per 256
// vocabulary rows and share (blockIdx.y) of the units.  Bound by B of the
// adapters in use and by z, read and written once; many small workgroups hide
// the latency (128 tokens over 32 adapters, V = 32768, rank 16: 18 us at five
// waves per SIMD for 66 MB; 24 us by blocks of 16 neighbouring tokens).
template <int RP, bool BF16>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(RP <= 32 ? 5 : 3)))
lora_expand_few_kernel(const float *z, int64_t ldz, void *out, int64_t ldo, int64_t M, int64_t V,
                       LoraAdapters ad, const uint16_t *__restrict__ u3,
                       const FewUnits *__restrict__ table)
{
    constexpr int U = RP < 32 ? 1 : RP / 32, S = piece_row(RP) / 32;
    __shared__ __attribute__((aligned(16))) float turn[4][16 * 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t16 = lane & 15, q = lane >> 4;
    const int64_t v0 = static_cast<int64_t>(blockIdx.x) * 256 + wave * 64;
    if (v0 >= V)
        return;
    const int jq = RP == 16 ? 8 * (q & 1) : 8 * q;  // the lane's first rank of a step
    const int64_t v = v0 + 4 * t16;
    for (int i0 = blockIdx.y; i0 < kFewTokens; i0 += gridDim.y) {
        const FewUnit un = table->u[i0];
        const int32_t a = un.id;
        if (un.count == 0)
            return;
        if (!BF16 && a < 0)
            continue;  // z is in place
        const int32_t *list = table->order + un.first;
        const bool live = a >= 0 && a < ad.n;
        bf16x8 fb[U][4], fu[S];
        if (live) {
            const uint16_t *pb = ad.B + a * ad.stride_b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t vr = min(v0 + 16 * i + t16, V - 1);
#pragma unroll
                for (int uu = 0; uu < U; ++uu)
                    fb[uu][i] = as_frag(load8_row(pb + vr * ad.ldb, 32 * uu + jq, ad.r, vr == V - 1));
            }
        }
        int64_t row[4];  // the tokens of this lane's row pieces, -1 past the unit
        f32x4 zr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            row[i] = 4 * i + q < un.count ? list[4 * i + q] : -1;
            zr[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (row[i] >= 0)
                zr[i] = load_piece(z + row[i] * ldz, v, V);
        }
        f32x4 d[4];
        const float fill = a >= ad.n ? NAN : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = f32x4{fill, fill, fill, fill};
        if (live) {
            const uint16_t *pu = u3 + static_cast<int64_t>(list[min(t16, un.count - 1)]) * piece_row(RP) + 8 * q;
#pragma unroll
            for (int s = 0; s < S; ++s)
                fu[s] = as_frag(*reinterpret_cast<const uint4 *>(pu + 32 * s));
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    d[i] = mfma16(fb[s % U][i], fu[s], d[i]);
        }
        turn_rows(d, turn[wave], t16, q);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row[i] >= 0)
                store_piece<BF16>(out, row[i] * ldo, v, V, zr[i] + d[i]);
    }
}

// ---------------------------------------------------------------------------
// z = x W^T for outputs of few tiles, where the shared product's kernels leave
// most of the chip idle: a workgroup forms a T x T tile (tokens x vocabulary
// rows), its eight waves an eighth of K each, summed in order through LDS.
// Fragments come straight from memory, a batch of steps at a time; what bounds
// it is how fast they reach the CU (218 tokens, K = 8192, V = 1070: the whole call
// 59 us, 151 with the kernels of lmhead_logits).
constexpr int kBaseWaves = 8;

template <int T>
__global__ __launch_bounds__(kBaseWaves * 64) void lora_base_kernel(const uint16_t *__restrict__ x, int64_t ldx,
                                                                    const uint16_t *__restrict__ W, int64_t ldw,
                                                                    float *__restrict__ z, int64_t ldz, int64_t M,
                                                                    int64_t K, int64_t V)
{
    constexpr int NF = T / 16, UN = T == 32 ? 8 : 4;
    __shared__ f32x4 red[kBaseWaves][NF * NF][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t16 = lane & 15, q = lane >> 4;
    const int64_t v0 = static_cast<int64_t>(blockIdx.x) * T, m0 = static_cast<int64_t>(blockIdx.y) * T;
    const uint16_t *pw[NF], *px[NF];
    f32x4 acc[NF][NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        pw[i] = W + min(v0 + 16 * i + t16, V - 1) * ldw + 8 * q;
        px[i] = x + min(m0 + 16 * i + t16, M - 1) * ldx + 8 * q;
#pragma unroll
        for (int j = 0; j < NF; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int64_t per_wave = (K + 32 * kBaseWaves - 1) / (32 * kBaseWaves) * 32;
    int64_t k = wave * per_wave;
    const int64_t kend = min(K, k + per_wave);
    for (; k + 32 * UN <= kend; k += 32 * UN) {
        uint4 vw[UN][NF], vx[UN][NF];
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                vw[u][i] = *reinterpret_cast<const uint4 *>(pw[i] + k + 32 * u);
                vx[u][i] = *reinterpret_cast<const uint4 *>(px[i] + k + 32 * u);
            }
        __builtin_amdgcn_sched_barrier(0);  // all of them in flight
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    acc[i][j] = mfma16(as_frag(vw[u][i]), as_frag(vx[u][j]), acc[i][j]);
    }
    for (; k < kend; k += 32) {
        const int64_t left = K - k - 8 * q;
        uint4 vw[NF], vx[NF];
#pragma unroll
        for (int i = 0; i < NF; ++i) {
            vw[i] = load8(pw[i] + k, left);
            vx[i] = load8(px[i] + k, left);
        }
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j)
                acc[i][j] = mfma16(as_frag(vw[i]), as_frag(vx[j]), acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
            red[wave][i * NF + j][lane] = acc[i][j];
    __syncthreads();
    for (int f = wave; f < NF * NF; f += kBaseWaves) {
        f32x4 sum = red[0][f][lane];
#pragma unroll
        for (int w = 1; w < kBaseWaves; ++w)
            sum += red[w][f][lane];
        const int64_t m = m0 + 16 * (f % NF) + t16, v = v0 + 16 * (f / NF) + 4 * q;
        if (m < M)
            store_piece<false>(z, m * ldz, v, V, sum);
    }
}

// ---------------------------------------------------------------------------
// logits += u B^T: reads the FP32 product z, adds each token's adapter, stores
// FP32 (in place) or BF16 (rounded once).  A workgroup covers 256 vocabulary
// rows and `nb` blocks of 16 tokens of the logits' order, one after another;
// wave w holds rows 64 w .. + 63 as four 16 x 16 results per block.  B rows go
// straight from memory into matrix operands (a fragment is 16 contiguous bytes
// of a row) and stay there while the next block uses the same adapter; z and
// the result move in whole 256-byte row pieces, the products turned through 4
// KiB of LDS per wave.  Bound by z, read and written once, and by B of the
// adapters in use (M = 1024, V = 32768, four adapters of rank 64: 72 us for 285
// MB, 4.0 TB/s; a copy of these bytes reaches 4.7).
constexpr int kMostBlocks = 8;

template <int RP, bool BF16>
__global__ __launch_bounds__(256) void lora_expand_kernel(const float *z, int64_t ldz, void *out,
                                                          int64_t ldo, int64_t M, int64_t V,
                                                          LoraAdapters ad,
                                                          const uint16_t *__restrict__ u3,
                                                          const int32_t *__restrict__ order, int nb,
                                                          int64_t tok_groups, int64_t wg0)
{
    constexpr int U = RP < 32 ? 1 : RP / 32;     // distinct 32-deep steps over a rank
    constexpr int S = piece_row(RP) / 32;        // steps over the three pieces
    __shared__ __attribute__((aligned(16))) float turn[4][16 * 64];
    __shared__ int32_t toks[16 * kMostBlocks], ids[16 * kMostBlocks];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t16 = lane & 15, q = lane >> 4;
    // Workgroups b, b + 8, ... share an XCD: they take the token groups of one
    // vocabulary tile in turn, so that its B rows are read into one L2.
    const int64_t wg = wg0 + blockIdx.x;
    const int64_t vt = wg / 8 / tok_groups * 8 + wg % 8;
    const int64_t tg = wg / 8 % tok_groups;
    const int64_t v0 = vt * 256 + wave * 64;
    // The workgroup's tokens: toks -1 where z stays as it is or there is none.
    if (tid < 16 * nb) {
        const int64_t at = tg * nb * 16 + tid;
        const int32_t tok = at < M ? order[at] : -1;
        const int32_t id = tok >= 0 ? ad.adapter[tok] : -1;
        toks[tid] = BF16 || id >= 0 ? tok : -1;
        ids[tid] = id;
    }
    __syncthreads();
    if (v0 >= V)
        return;
    float *const own = turn[wave];
    const int jq = RP == 16 ? 8 * (q & 1) : 8 * q;  // the lane's first rank of a step
    bf16x8 fb[U][4];
    int32_t held = -1;  // the adapter whose B rows fb holds
    auto load_b = [&](int32_t a, bf16x8 (&f)[U][4]) {
        const uint16_t *pb = ad.B + a * ad.stride_b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t v = min(v0 + 16 * i + t16, V - 1);
            const bool last = v == V - 1;
#pragma unroll
            for (int uu = 0; uu < U; ++uu)
                f[uu][i] = as_frag(load8_row(pb + v * ad.ldb, 32 * uu + jq, ad.r, last));
        }
    };
    // One block of 16 tokens: ids, pieces of u, and row pieces of z (this lane's
    // four are tokens 4 i + q, columns v0 + 4 t16 .. + 3).  The next
    // block's are on their way before this one's results are stored: a wait for
    // loads issued after stores would wait for the stores too.
    const int64_t v = v0 + 4 * t16;
    struct Block {
        int32_t id;
        bf16x8 u[S];
        f32x4 z[4];
    };
    auto load_block = [&](Block &t, int b) {
        t.id = ids[16 * b + t16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t tok = toks[16 * b + 4 * i + q];
            t.z[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (tok >= 0)
                t.z[i] = load_piece(z + tok * ldz, v, V);
        }
        const uint16_t *pu = u3 + static_cast<int64_t>(max(toks[16 * b + t16], 0)) * piece_row(RP) + 8 * q;
#pragma unroll
        for (int s = 0; s < S; ++s)
            t.u[s] = as_frag(*reinterpret_cast<const uint4 *>(pu + 32 * s));
    };
    Block cur;
    load_block(cur, 0);
    for (int b = 0; b < nb; ++b) {
        if ((tg * nb + b) * 16 >= M)
            return;
        Block nxt;
        if (b + 1 < nb)
            load_block(nxt, b + 1);
        const int32_t id = cur.id;
        const bool bad = id >= ad.n;
        uint32_t todo = static_cast<uint32_t>(__ballot(id >= 0 && id < ad.n)) & 0xffffu;
        if (!BF16 && !todo && !__ballot(bad)) {
            cur = nxt;
            continue;
        }
        f32x4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        while (todo) {
            const int32_t a = first_id(id, todo);
            todo &= ~tokens_of(id, a);
            if (a != held)
                load_b(a, fb);
            held = a;
            f32x4 tmp[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                tmp[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tmp[i] = mfma16(fb[s % U][i], cur.u[s], tmp[i]);
            if (id == a) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] = tmp[i];
            }
        }
        if (bad) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = f32x4{NAN, NAN, NAN, NAN};
        }
        turn_rows(acc, own, t16, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t tok = toks[16 * b + 4 * i + q];
            if (tok >= 0)
                store_piece<BF16>(out, tok * ldo, v, V, cur.z[i] + acc[i]);
        }
        cur = nxt;
    }
}

// ---------------------------------------------------------------------------
// Gradients.
//
// Staged tiles: 64 rows (tokens, or ranks) of PITCH BF16 words, 16-byte chunk c
// of row p at chunk c ^ key(p).  Wide rows (16 chunks or more): the key
// separates the eight rows that a quarter of a row-wise fragment read touches,
// and the two groups of four rows that half of a transposing read touches.
// Rows of pieces take the three low bits only, so that a chunk stays within
// its eight.
template <int PITCH, bool PIECES>
__device__ __forceinline__ int tile_at(int p, int chunk)
{
    int key;
    if constexpr (PIECES)
        key = ((p & 3) << 1) ^ ((p >> 2) & 1);
    else
        key = ((p & 3) << 2) ^ ((p >> 2) & 1) ^ (((p >> 3) & 1) << 1);
    return p * PITCH + ((chunk ^ key) << 3);
}

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));

// Transposed fragment: lane l receives column n0 + l % 16 at rows p .. p + 7,
// p = the lane group's first row (a multiple of 8).  Within a group of 16
// lanes, lane 4 b + a addresses row b, columns 4 a .. 4 a + 3, and the
// transposing read hands lane i column i of the four rows.
template <int PITCH, bool PIECES>
__device__ __forceinline__ bf16x8 tile_column_frag(const uint16_t *tile, int p, int n0, int lane)
{
    typedef __attribute__((address_space(3))) v4i16 lds_v4;
    const int b = (lane >> 2) & 3, col = n0 + 4 * (lane & 3);
    auto at = [&](int row) { return tile + tile_at<PITCH, PIECES>(row, col >> 3) + (col & 7); };
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(at(p + b)));
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(at(p + 4 + b)));
    const v8i16 c = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, c);
}

// Row fragment: 8 columns from n (a multiple of 8) of row p.
template <int PITCH, bool PIECES>
__device__ __forceinline__ bf16x8 tile_row_frag(const uint16_t *tile, int p, int n)
{
    return *reinterpret_cast<const bf16x8 *>(tile + tile_at<PITCH, PIECES>(p, n >> 3));
}

// LDS pitch of a row of pieces: whole groups of eight chunks.
__host__ __device__ constexpr int piece_pitch(int RP)
{
    return RP == 32 ? 128 : piece_row(RP);
}

// One chunk of tokens on its way from memory in a workgroup of 256: 64 rows of
// 256 columns of a matrix, and the tokens' pieces.  Rows past the count are
// zero.  Row numbers come from LDS, two chunks ahead, so that no wait for a
// number or a piece stands behind the rows in flight (a wave's loads retire in
// order).
template <int RP>
struct ChunkLoad {
    static constexpr int PL = piece_row(RP), PP = piece_pitch(RP), NP = PL / 32;
    uint4 v[8], u[NP];

    __device__ __forceinline__ void load(const uint16_t *base, int64_t ld, int64_t col0, int64_t ncols,
                                         const uint16_t *pieces, const int32_t *rows, int64_t count,
                                         int tid)
    {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int at = 256 * i + tid, row = at / (PL / 8);
            u[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row < count)
                u[i] = *reinterpret_cast<const uint4 *>(
                    pieces + static_cast<int64_t>(rows[row]) * PL + 8 * (at - row * (PL / 8)));
        }
        const int64_t col = col0 + 8 * (tid & 31);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 8 * i + (tid >> 5);
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row < count && col < ncols)
                v[i] = load8(base + static_cast<int64_t>(rows[row]) * ld + col, ncols - col);
        }
    }
    __device__ __forceinline__ void store(uint16_t *tile, uint16_t *pieces, int tid) const
    {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int at = 256 * i + tid, row = at / (PL / 8);
            *reinterpret_cast<uint4 *>(pieces + tile_at<PP, true>(row, at - row * (PL / 8))) = u[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(tile + tile_at<256, false>(8 * i + (tid >> 5), tid & 31)) = v[i];
    }
};

// Walks a group's tokens 64 at a time through `tile` [64][256] and `pieces`
// [64][PP] in LDS: f(chunk's token numbers, count) between barriers.  rows:
// 2 x 64 numbers in LDS.
template <int RP, typename F>
__device__ __forceinline__ void for_each_chunk(const uint16_t *base, int64_t ld, int64_t col0, int64_t ncols,
                                               const uint16_t *pieces, const int32_t *order, int64_t count,
                                               uint16_t *tile, uint16_t *ptile, int32_t (&rows)[2][64],
                                               int tid, F &&f)
{
    auto number = [&](int64_t c) { return tid < 64 && c + tid < count ? order[c + tid] : 0; };
    if (tid < 64) {
        rows[0][tid] = number(0);
        rows[1][tid] = number(64);
    }
    __syncthreads();
    ChunkLoad<RP> nxt;
    nxt.load(base, ld, col0, ncols, pieces, rows[0], count, tid);
    int32_t ahead = 0;
    for (int64_t c = 0; c < count; c += 64) {
        const int b = (c >> 6) & 1;
        __syncthreads();  // the chunk before is read
        if (c > 0 && tid < 64)
            rows[b ^ 1][tid] = ahead;  // the chunk after this one
        nxt.store(tile, ptile, tid);
        __syncthreads();
        ahead = number(c + 128);
        if (c + 64 < count)
            nxt.load(base, ld, col0, ncols, pieces, rows[b ^ 1], count - c - 64, tid);
        f(rows[b], c, count - c);
    }
}

// Gradients are not read again by these kernels: their stores are marked as
// streamed once (M = 1024, K = 8192, V = 32768: v 20.4 -> 18 us, k 13.4 -> 11.9).
__device__ __forceinline__ void store_f32x4(float *p, f32x4 v, int64_t n, bool add)
{
    if (n >= 4) {
        if (add)
            v += *reinterpret_cast<const f32x4 *>(p);
        __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(p));
    } else {
        for (int e = 0; e < n; ++e)
            p[e] = add ? p[e] + v[e] : v[e];
    }
}

// One workgroup per (256 vocabulary columns, adapter): walks the adapter's
// tokens 64 at a time and takes both products from one read of g: its part of
// t (over these 256 columns; joined by lora_join_kernel) and dB (accumulated over
// the tokens in registers).  B^T sits in LDS.  Bound by the one read of g (M =
// 1024, V = 32768, 4 adapters of rank 16: 18 us, 3.7 TB/s with 3 us to start and
// drain and 4 us of dependent loads -- group, token numbers, rows -- before the
// stream); a second chunk in flight gained nothing (22 against 20.7 us).  The parts of t cost
// 8 RP bytes per token and block against 512 of g.  An adapter's tokens are not split
// over workgroups: few columns and few adapters leave most CUs idle.  u3 is written
// only for a call that wants dB: without it sU holds whatever the workspace did and
// must not be used.
template <int RP>
__global__ __launch_bounds__(256) void lora_bwd_v_kernel(
    const uint16_t *__restrict__ g, int64_t ldg, int64_t M, int64_t V, LoraAdapters ad,
    const int32_t *__restrict__ offset, const int32_t *__restrict__ order,
    const uint16_t *__restrict__ u3, float *__restrict__ tpart, float *__restrict__ dB, int64_t lddb,
    int64_t stride_db, int accumulate, int64_t nvb)
{
    constexpr int JF = RP / 16, LDB = 256 + 8, PP = piece_pitch(RP);
    __shared__ __attribute__((aligned(16))) uint16_t sG[64 * 256];
    __shared__ __attribute__((aligned(16))) uint16_t sU[64 * PP];
    __shared__ __attribute__((aligned(16))) uint16_t sBT[RP * LDB];
    __shared__ int32_t rows[2][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t16 = lane & 15, q = lane >> 4;
    const int64_t a = blockIdx.x / nvb, vb = blockIdx.x - a * nvb;
    const int64_t v0 = vb * 256;
    const int64_t o0 = offset[a], cnt = offset[a + 1] - o0;
    if (cnt == 0 && (accumulate || !dB))
        return;

    if (tpart && cnt > 0) {
        const int64_t v = v0 + tid;
        const uint16_t *pb = ad.B + a * ad.stride_b + v * ad.ldb;
#pragma unroll
        for (int j = 0; j < RP; j += 8) {
            const uint4 w = v < V ? load8_row(pb, j, ad.r, v == V - 1) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sBT[(j + e) * LDB + tid] = static_cast<uint16_t>(ws[e >> 1] >> (16 * (e & 1)));
        }
    }
    f32x4 accB[JF][4];
#pragma unroll
    for (int jf = 0; jf < JF; ++jf)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            accB[jf][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (cnt > 0)
        for_each_chunk<RP>(
            g, ldg, v0, V, u3, order + o0, cnt, sG, sU, rows, tid,
            [&](const int32_t *toks, int64_t, int64_t left) {
                if (tpart) {
                    // Ranks (rows) x this wave's 16 tokens, over the 256 columns.
                    f32x4 acc[JF];
#pragma unroll
                    for (int jf = 0; jf < JF; ++jf)
                        acc[jf] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const bf16x8 ft = tile_row_frag<256, false>(sG, 16 * wave + t16, 32 * s + 8 * q);
#pragma unroll
                        for (int jf = 0; jf < JF; ++jf)
                            acc[jf] = mfma16(*reinterpret_cast<const bf16x8 *>(
                                                 sBT + (16 * jf + t16) * LDB + 32 * s + 8 * q),
                                             ft, acc[jf]);
                    }
                    if (16 * wave + t16 < left) {
                        float *p = tpart + (vb * M + toks[16 * wave + t16]) * RP + 4 * q;
#pragma unroll
                        for (int jf = 0; jf < JF; ++jf)
                            *reinterpret_cast<f32x4 *>(p + 16 * jf) = acc[jf];
                    }
                }
                if (dB) {
                    // Ranks (rows) x this wave's 64 columns, over the 64 tokens.
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        bf16x8 fg[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            fg[i] = tile_column_frag<256, false>(sG, 32 * ks + 8 * q, 64 * wave + 16 * i, lane);
#pragma unroll
                        for (int jf = 0; jf < JF; ++jf)
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                const bf16x8 fu =
                                    tile_column_frag<PP, true>(sU, 32 * ks + 8 * q, p * RP + 16 * jf, lane);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    accB[jf][i] = mfma16(fu, fg[i], accB[jf][i]);
                            }
                    }
                }
            });
    if (!dB)
        return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t v = v0 + 64 * wave + 16 * i + t16;
        if (v >= V)
            continue;
        float *p = dB + a * stride_db + v * lddb;
#pragma unroll
        for (int jf = 0; jf < JF; ++jf) {
            const int j = 16 * jf + 4 * q;
            store_f32x4(p + j, accB[jf][i], ad.r - j, accumulate != 0);
        }
    }
}

// dX and dA, 256 columns of K per workgroup.  The first nkb n workgroups
// accumulate dA of one adapter over its tokens, 64 at a time, from one read of
// x; the others write dX = t A of one chunk of up to 64 tokens, A_a's block in
// LDS (tokens on no adapter get zeros, those whose id is none NaN).  One launch,
// so that the two share the chip: dA has few workgroups, dX many short ones.
// Bound by writing dX (M = 1024, K = 8192, 4 adapters of rank 16: 12 us for 17 MB
// read and 34 MB written, 4.2 TB/s).
template <int RP>
__global__ __launch_bounds__(256) void lora_bwd_k_kernel(
    const uint16_t *__restrict__ x, int64_t ldx, int64_t K, LoraAdapters ad,
    const int32_t *__restrict__ offset, const int32_t *__restrict__ order,
    const Chunk *__restrict__ chunks, const uint16_t *__restrict__ t3, float *__restrict__ dX,
    int64_t lddx, float *__restrict__ dA, int64_t ldda, int64_t stride_da, int accumulate, int64_t nkb)
{
    constexpr int JF = RP / 16, PP = piece_pitch(RP), PL = piece_row(RP);
    constexpr int U = RP < 32 ? 1 : RP / 32, S = PL / 32;
    constexpr int WIDE = RP > 64 ? RP * 256 : 64 * 256;  // x [64][256] or A [RP][256]
    __shared__ __attribute__((aligned(16))) uint16_t wide[WIDE];
    __shared__ __attribute__((aligned(16))) uint16_t pieces[64 * PP];
    __shared__ __attribute__((aligned(16))) float turn[4][16 * 64];
    __shared__ int32_t rows[2][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t16 = lane & 15, q = lane >> 4;
    const int64_t unit = blockIdx.x / nkb, kb = blockIdx.x - unit * nkb;
    const int64_t k0 = kb * 256;
    const int64_t n_da = dA ? ad.n : 0;

    if (unit < n_da) {
        const int64_t a = unit;
        const int64_t o0 = offset[a], cnt = offset[a + 1] - o0;
        if (cnt == 0 && accumulate)
            return;
        f32x4 acc[4][JF];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int jf = 0; jf < JF; ++jf)
                acc[i][jf] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (cnt > 0)
            for_each_chunk<RP>(
                x, ldx, k0, K, t3, order + o0, cnt, wide, pieces, rows, tid,
                [&](const int32_t *, int64_t, int64_t) {
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        bf16x8 fx[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            fx[i] = tile_column_frag<256, false>(wide, 32 * ks + 8 * q, 64 * wave + 16 * i, lane);
#pragma unroll
                        for (int jf = 0; jf < JF; ++jf)
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                const bf16x8 ft =
                                    tile_column_frag<PP, true>(pieces, 32 * ks + 8 * q, p * RP + 16 * jf, lane);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    acc[i][jf] = mfma16(fx[i], ft, acc[i][jf]);
                            }
                    }
                });
#pragma unroll
        for (int jf = 0; jf < JF; ++jf) {
            const int j = 16 * jf + t16;
            if (j >= ad.r)
                continue;
            float *p = dA + a * stride_da + j * ldda;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t k = k0 + 64 * wave + 16 * i + 4 * q;
                store_f32x4(p + k, acc[i][jf], K - k, accumulate != 0);
            }
        }
        return;
    }

    const Chunk ch = chunks[unit - n_da];
    if (ch.group < 0 || (ch.group == ad.n && accumulate))
        return;
    const int64_t kw = k0 + 64 * wave + 4 * t16;  // this lane's columns of a row piece
    if (ch.group >= ad.n) {
        const float fill = ch.group == ad.n ? 0.0f : NAN;
        for (int i = q; i < ch.count; i += 4)
            store_f32x4(dX + static_cast<int64_t>(order[ch.first + i]) * lddx + kw,
                        f32x4{fill, fill, fill, fill}, K - kw, false);
        return;
    }
    const int64_t a = ch.group;
    if (tid < 64)
        rows[0][tid] = tid < ch.count ? order[ch.first + tid] : 0;
    {
        const int64_t col = k0 + 8 * (tid & 31);
        const uint16_t *pa = ad.A + a * ad.stride_a;
#pragma unroll
        for (int i = 0; i < RP / 8; ++i) {
            const int j = 8 * i + (tid >> 5);
            const uint4 w = (j < ad.r && col < K) ? load8(pa + j * ad.lda + col, K - col)
                                                  : make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(wide + tile_at<256, false>(j, tid & 31)) = w;
        }
    }
    __syncthreads();
    bf16x8 fa[U][4];
#pragma unroll
    for (int uu = 0; uu < U; ++uu)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            fa[uu][i] = tile_column_frag<256, false>(wide, RP == 16 ? 8 * (q & 1) : 32 * uu + 8 * q,
                                                     64 * wave + 16 * i, lane);
    // This wave's 64 columns (rows) x 16 tokens at a time.
    for (int t0 = 0; t0 < ch.count; t0 += 16) {
        const uint16_t *pt = t3 + static_cast<int64_t>(rows[0][min(t0 + t16, ch.count - 1)]) * PL + 8 * q;
        f32x4 d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bf16x8 ft = as_frag(*reinterpret_cast<const uint4 *>(pt + 32 * s));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[i] = mfma16(fa[s % U][i], ft, d[i]);
        }
        turn_rows(d, turn[wave], t16, q);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t0 + 4 * i + q < ch.count)
                store_f32x4(dX + static_cast<int64_t>(rows[0][t0 + 4 * i + q]) * lddx + kw, d[i], K - kw,
                            accumulate != 0);
    }
}

int rank_bucket(int64_t r)
{
    return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128;
}

int64_t round256(int64_t b)
{
    return (b + 255) / 256 * 256;
}

// Units a batch of M <= kFewTokens tokens can have.
int64_t few_units(int64_t M, int64_t n)
{
    return std::min<int64_t>(M, M / 16 + n + 2);
}

// Parts of K of the shrink beyond kFewTokens tokens: enough for 512
// workgroups, at most 32, at least 256 columns each.
constexpr int64_t kShrinkWorkgroups = 512;
int64_t shrink_parts(int64_t M, int64_t K)
{
    const int64_t blocks = std::max<int64_t>(1, (M + 63) / 64);
    return std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(32, K / 256), kShrinkWorkgroups / blocks));
}

hipError_t launch_join(const float *parts, int64_t n_parts, int64_t M, int RP, const LoraAdapters &ad,
                       uint16_t *pieces, hipStream_t s)
{
    const int64_t n4 = M * RP / 4;  // blocks of 16; at most 2^31 work-items per launch
    const int64_t most = kMaxItems / 16;
    if (n4 > most)
        return hipErrorInvalidValue;  // refused by the caller's size check
    hipLaunchKernelGGL(lora_join_kernel, dim3(static_cast<unsigned>((n4 + 15) / 16)), dim3(256), 0, s, parts,
                       n_parts, M, RP, ad, pieces);
    return hipGetLastError();
}

// u3 from x; upart: [shrink_parts][M][RP] FP32 (M > kFewTokens only).  n_groups:
// workgroups that write `groups` beside it (ad.n + 2, one per group; (M + 63) /
// 64 where only the order is wanted, M > kFewTokens; 0: none).
hipError_t launch_shrink(const uint16_t *x, int64_t ldx, int64_t M, int64_t K, const LoraAdapters &ad,
                         uint16_t *u3, FewUnits *table, float *upart, const Grouping &groups,
                         int64_t n_groups, hipStream_t s)
{
    const int RP = rank_bucket(ad.r);
    const int64_t zr = RP / 16;
    if (M <= kFewTokens) {
        const dim3 grid(static_cast<unsigned>(n_groups + few_units(M, ad.n)), static_cast<unsigned>(zr));
        hipLaunchKernelGGL(lora_shrink_few_kernel, grid, dim3(kShrinkThreads), 0, s, x, ldx, M, K, ad, RP,
                           u3, table, groups, static_cast<unsigned>(n_groups));
        return hipGetLastError();
    }
    const int64_t S = shrink_parts(M, K), part_k = (K + 32 * S - 1) / (32 * S) * 32;
    const int64_t slots = std::max<int64_t>(1, std::min<int64_t>(ad.n, 4));
    const int64_t wgs = (M + 63) / 64 * S;  // < 2^17
    const dim3 grid(static_cast<unsigned>(n_groups + wgs), static_cast<unsigned>(slots));
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, x, ldx, M, K, ad, static_cast<int>(S), part_k, upart,
                           groups, static_cast<unsigned>(n_groups));
    };
    switch (RP) {
    case 16: run(lora_shrink_kernel<16>); break;
    case 32: run(lora_shrink_kernel<32>); break;
    case 64: run(lora_shrink_kernel<64>); break;
    default: run(lora_shrink_kernel<128>); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    return launch_join(upart, S, M, RP, ad, u3, s);
}

template <int RP>
hipError_t launch_expand(const float *z, int64_t ldz, void *out, int64_t ldo, bool bf16, int64_t M,
                         int64_t V, const LoraAdapters &ad, const uint16_t *u3,
                         const FewUnits *table, const int32_t *order, hipStream_t s)
{
    if (M <= kFewTokens) {
        // Shares of the units: as many as make 4096 workgroups.
        const int64_t vts = (V + 255) / 256;
        const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(few_units(M, ad.n), 4096 / vts));
        const dim3 grid(static_cast<unsigned>(vts), static_cast<unsigned>(parts));
        if (bf16)
            hipLaunchKernelGGL((lora_expand_few_kernel<RP, true>), grid, dim3(256), 0, s, z, ldz, out, ldo, M, V,
                               ad, u3, table);
        else
            hipLaunchKernelGGL((lora_expand_few_kernel<RP, false>), grid, dim3(256), 0, s, z, ldz, out, ldo, M,
                               V, ad, u3, table);
        return hipGetLastError();
    }
    // Token blocks per workgroup: up to eight (B rows kept across a request's
    // tokens, loads ahead of stores) while 1024 workgroups remain.  M = 1024, V =
    // 32768, four adapters of rank 64 in runs: 71 us; four blocks 81 us.
    const int64_t tb = (M + 15) / 16, vts = (V + 255) / 256;
    const int nb = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(kMostBlocks, tb * vts / 1024)));
    const int64_t groups = (tb + nb - 1) / nb;
    // Whole groups of eight vocabulary tiles (the tiles past V exit).
    const int64_t wgs = (vts + 7) / 8 * 8 * groups, most = kMaxItems / 256;
    for (int64_t w0 = 0; w0 < wgs; w0 += most) {
        const dim3 grid(static_cast<unsigned>(std::min(most, wgs - w0)));
        if (bf16)
            hipLaunchKernelGGL((lora_expand_kernel<RP, true>), grid, dim3(256), 0, s, z, ldz, out, ldo, M, V,
                               ad, u3, order, nb, groups, w0);
        else
            hipLaunchKernelGGL((lora_expand_kernel<RP, false>), grid, dim3(256), 0, s, z, ldz, out, ldo, M,
                               V, ad, u3, order, nb, groups, w0);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

constexpr int64_t kGroupsBeside = 1024;

// The gradients' workspace, in order.
struct BwdLayout {
    int64_t offset, order, chunks, u3, t3, parts, end;  // parts: of u, then of t
};

// Numbers of chunks: every group's start at chunk_base.
int64_t chunk_numbers(int64_t M, int64_t n)
{
    return chunk_base(M, n + 2);
}

BwdLayout bwd_layout(int64_t M, int64_t K, int64_t V, int64_t r, int64_t n)
{
    const int64_t RP = rank_bucket(r), nvb = (V + 255) / 256;
    const int64_t pieces = round256(2 * piece_row(static_cast<int>(RP)) * M);
    BwdLayout l;
    l.offset = 0;
    l.order = l.offset + round256(4 * (n + 3));
    l.chunks = l.order + round256(4 * M);
    l.u3 = l.chunks + round256(static_cast<int64_t>(sizeof(Chunk)) * chunk_numbers(M, n));
    l.t3 = l.u3 + pieces;
    l.parts = l.t3 + pieces;
    l.end = l.parts + round256(4 * std::max(nvb, shrink_parts(M, K)) * M * RP);
    return l;
}

template <int RP>
hipError_t launch_bwd_v(const LoraBwd &p, const BwdLayout &l, char *ws, hipStream_t s)
{
    const int64_t nvb = (p.V + 255) / 256;
    hipLaunchKernelGGL((lora_bwd_v_kernel<RP>), dim3(static_cast<unsigned>(nvb * p.ad.n)), dim3(256), 0, s,
                       p.g, p.ldg, p.M, p.V, p.ad, reinterpret_cast<const int32_t *>(ws + l.offset),
                       reinterpret_cast<const int32_t *>(ws + l.order),
                       reinterpret_cast<const uint16_t *>(ws + l.u3),
                       (p.dX || p.dA) ? reinterpret_cast<float *>(ws + l.parts) : nullptr, p.dB, p.lddb,
                       p.stride_db, p.accumulate ? 1 : 0, nvb);
    return hipGetLastError();
}

template <int RP>
hipError_t launch_bwd_k(const LoraBwd &p, const BwdLayout &l, char *ws, hipStream_t s)
{
    const int64_t nkb = (p.K + 255) / 256;
    const int64_t units = (p.dA ? p.ad.n : 0) + (p.dX ? chunk_numbers(p.M, p.ad.n) : 0);
    if (units == 0)
        return hipSuccess;  // dA of no adapters
    hipLaunchKernelGGL((lora_bwd_k_kernel<RP>), dim3(static_cast<unsigned>(nkb * units)), dim3(256), 0, s,
                       p.x, p.ldx, p.K, p.ad, reinterpret_cast<const int32_t *>(ws + l.offset),
                       reinterpret_cast<const int32_t *>(ws + l.order),
                       reinterpret_cast<const Chunk *>(ws + l.chunks),
                       reinterpret_cast<const uint16_t *>(ws + l.t3), p.dX, p.lddx, p.dA, p.ldda,
                       p.stride_da, p.accumulate ? 1 : 0, nkb);
    return hipGetLastError();
}

}  // namespace

// The forward's workspace, in order: a small batch's units or a larger one's
// order, u, and the FP32
// product of BF16 logits; the parts of u share the last one's place (they are
// joined before the product runs).
struct FwdLayout {
    int64_t table, u3, z, end;  // table: FewUnits, or the order of more tokens
};

static FwdLayout fwd_layout(int64_t M, int64_t K, int64_t V, int64_t r, bool bf16)
{
    const int64_t RP = rank_bucket(r);
    FwdLayout l;
    l.table = 0;
    l.u3 = round256(M <= kFewTokens ? sizeof(FewUnits) : 4 * M);
    l.z = l.u3 + round256(2 * piece_row(static_cast<int>(RP)) * M);
    l.end = l.z + round256(std::max<int64_t>(bf16 ? 4 * M * ((V + 3) / 4 * 4) : 0,
                                             M <= kFewTokens ? 0 : 4 * shrink_parts(M, K) * M * RP));
    return l;
}

int64_t lora_logits_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t r, bool bf16)
{
    return fwd_layout(M, K, V, r, bf16).end;
}

int64_t lora_bwd_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t r, int64_t n)
{
    return bwd_layout(M, K, V, r, n).end;
}

// Tile of lora_base_kernel for outputs of few tiles, or 0: the kernels of
// lmhead_logits, whose tiles are larger and whose workgroups walk all of K.  The
// whole call, theirs and this one's:
//   32 x 32, at most one workgroup per CU.  M 12, V 5000, K 7976: 67 and 35 us;
//     218, 1070, 8192: 151 and 59 us; 58, 3000, 976: 25 and 18 us.  Up to 16
//     tokens at K >= 8192 theirs split K as well: 16, 2549, 8192: 41.7 and 43.6.
//   64 x 64, M > 128, at most two per CU.  410, 2989, 7304: 192 and 114 us; 654,
//     2549, 2048: 59 and 53 us; past it 400, 5000, 2048: 59 and 65 us.
//   64 x 64 for fewer tokens, at most one per CU.  128, 5000, 4632: 74 and 49 us;
//     past it 128, 9000, 2048: 41 and 50 us.  Up to 64 tokens theirs are as fast
//     where K is long and a multiple of 64 and W is in the caches: 45, 9000, 8000:
//     64 and 76 us (from memory 90 and 80), but 45, 9000, 7976: 83 and 63 us.
static int64_t base_tile(int64_t M, int64_t K, int64_t V)
{
    auto tiles = [&](int64_t T) { return (M + T - 1) / T * ((V + T - 1) / T); };
    if (tiles(32) <= 256)
        return M <= 16 && K >= 8192 ? 0 : 32;
    if (M > 128)
        return tiles(64) <= 512 ? 64 : 0;
    return tiles(64) <= 256 && (M > 64 || K < 5120 || K % 64 != 0) ? 64 : 0;
}

// The shared product, FP32.
static hipError_t launch_base(const GemmProblem &f, hipStream_t s)
{
    const int64_t M = f.C, K = f.P, V = f.R, T = base_tile(M, K, V);
    if (T == 0)
        return launch_gemm_logits(f, Epi::kStoreF32, s);
    const dim3 grid(static_cast<unsigned>((V + T - 1) / T), static_cast<unsigned>((M + T - 1) / T));
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kBaseWaves * 64), 0, s, f.B, f.ldb, f.A, f.lda,
                           static_cast<float *>(f.D), f.ldd, M, K, V);
    };
    if (T == 32)
        run(lora_base_kernel<32>);
    else
        run(lora_base_kernel<64>);
    return hipGetLastError();
}

hipError_t launch_logits_lora(const GemmProblem &p, bool bf16, const LoraAdapters &ad, void *workspace,
                              hipStream_t s)
{
    const int64_t M = p.C, K = p.P, V = p.R;
    char *ws = static_cast<char *>(workspace);
    const FwdLayout l = fwd_layout(M, K, V, ad.r, bf16);
    FewUnits *table = reinterpret_cast<FewUnits *>(ws + l.table);  // M <= kFewTokens
    int32_t *order = reinterpret_cast<int32_t *>(ws + l.table);    // M > kFewTokens
    uint16_t *u3 = reinterpret_cast<uint16_t *>(ws + l.u3);
    GemmProblem f = p;  // the shared product, FP32: in place, or in the workspace for BF16 logits
    if (bf16) {
        f.D = ws + l.z;
        f.ldd = (V + 3) / 4 * 4;
    }
    f.stream_out = false;  // read back at once
    hipError_t e = launch_shrink(p.B, p.ldb, M, K, ad, u3, table, reinterpret_cast<float *>(ws + l.z),
                                 Grouping{nullptr, order, nullptr}, M <= kFewTokens ? 0 : (M + 63) / 64, s);
    if (e == hipSuccess)
        e = launch_base(f, s);
    if (e != hipSuccess)
        return e;
    const float *z = static_cast<const float *>(f.D);
    switch (rank_bucket(ad.r)) {
    case 16: return launch_expand<16>(z, f.ldd, p.D, p.ldd, bf16, M, V, ad, u3, table, order, s);
    case 32: return launch_expand<32>(z, f.ldd, p.D, p.ldd, bf16, M, V, ad, u3, table, order, s);
    case 64: return launch_expand<64>(z, f.ldd, p.D, p.ldd, bf16, M, V, ad, u3, table, order, s);
    default: return launch_expand<128>(z, f.ldd, p.D, p.ldd, bf16, M, V, ad, u3, table, order, s);
    }
}

hipError_t launch_lora_bwd(const LoraBwd &p, void *workspace, hipStream_t s)
{
    const BwdLayout l = bwd_layout(p.M, p.K, p.V, p.ad.r, p.ad.n);
    char *ws = static_cast<char *>(workspace);
    const int RP = rank_bucket(p.ad.r);
    uint16_t *t3 = reinterpret_cast<uint16_t *>(ws + l.t3);
    const int64_t nvb = (p.V + 255) / 256;
    const Grouping groups = {reinterpret_cast<int32_t *>(ws + l.offset),
                             reinterpret_cast<int32_t *>(ws + l.order),
                             reinterpret_cast<Chunk *>(ws + l.chunks)};
    const int64_t n_groups = p.ad.n + 2;
    const bool shrink = p.dB && p.ad.n > 0 && p.M > 0;
    // One launch for the grouping and u, neither of which needs the other (M =
    // 1024, K = 8192: 4.5 + 7.6 -> 8 us); beyond kGroupsBeside groups the
    // grouping is the longer of the two and goes by itself.
    const bool beside = shrink && n_groups <= kGroupsBeside;
    hipError_t e = hipSuccess;
    if (!beside) {
        hipLaunchKernelGGL(lora_group_kernel, dim3(static_cast<unsigned>(n_groups)), dim3(256), 0, s,
                           p.ad.adapter, p.M, p.ad.n, groups);
        e = hipGetLastError();
    }
    if (e == hipSuccess && shrink)
        e = launch_shrink(p.x, p.ldx, p.M, p.K, p.ad, reinterpret_cast<uint16_t *>(ws + l.u3), nullptr,
                          reinterpret_cast<float *>(ws + l.parts), groups, beside ? n_groups : 0, s);
    if (e == hipSuccess && p.ad.n > 0 && p.V > 0) {
        switch (RP) {
        case 16: e = launch_bwd_v<16>(p, l, ws, s); break;
        case 32: e = launch_bwd_v<32>(p, l, ws, s); break;
        case 64: e = launch_bwd_v<64>(p, l, ws, s); break;
        default: e = launch_bwd_v<128>(p, l, ws, s); break;
        }
    }
    if (e != hipSuccess || (!p.dX && !p.dA) || p.K == 0)
        return e;
    if (p.ad.n > 0 && p.M > 0) {
        e = launch_join(reinterpret_cast<const float *>(ws + l.parts), nvb, p.M, RP, p.ad, t3, s);
        if (e != hipSuccess)
            return e;
    }
    switch (RP) {
    case 16: return launch_bwd_k<16>(p, l, ws, s);
    case 32: return launch_bwd_k<32>(p, l, ws, s);
    case 64: return launch_bwd_k<64>(p, l, ws, s);
    default: return launch_bwd_k<128>(p, l, ws, s);
    }
}

}  // namespace lmh
