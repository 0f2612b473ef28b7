// rows.h -- device helpers of the kernels that read rows of logits by segments
// of 2048 columns, one wave each: loads, wave reductions, and the largest values
// of a segment.
#pragma once

#include "common.h"

#include <algorithm>

namespace lmh {

constexpr int kSegCols = 2048;     // columns a wave holds at a time, 32 a lane
constexpr int kCandCap = 512;      // candidates a wave can hold

inline int64_t row_segments(int64_t V)
{
    return (V + kSegCols - 1) / kSegCols;
}

// How the rows of a forward are shared out: a workgroup of 4 waves per row where
// there are rows enough for every CU, of 8 or 16 where there are fewer (no more than
// the row has segments; of one wave for many rows of one or two: 8192 rows of 1000
// took 27 us in four waves), and up to 128 rows in parts, 256 / rows of them and one round
// of segments at least each (129 rows of 131072, a workgroup each, take as long as 128 in
// two parts each: 13.5 us).  A part has at most max_segs segments (a multiple of 16).
struct RowPlan {
    int32_t waves, part_segs;
    int64_t parts;
};
inline RowPlan row_plan(int64_t n_rows, int64_t V, int32_t min_waves, int64_t max_segs = int64_t{1} << 30)
{
    const int64_t nseg = row_segments(V);
    const int32_t most = nseg <= 2 && n_rows >= 512 ? min_waves : nseg <= 4 ? 4 : nseg <= 8 ? 8 : 16;
    const int32_t waves = std::min<int32_t>(most, n_rows >= 512 ? 4 : n_rows > 256 ? 8 : 16);
    const int64_t rounds = (nseg + waves - 1) / waves;  // of a workgroup over the whole row
    const int64_t want = std::max<int64_t>(1, 256 / std::max<int64_t>(n_rows, 1));
    const int64_t per = std::min((rounds + want - 1) / want, max_segs / waves);
    return {waves, static_cast<int32_t>(waves * per), (rounds + per - 1) / per};
}

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

__device__ __forceinline__ float wave_sum(float d)
{
    d += __uint_as_float(dpp<kQuadXor1>(__float_as_uint(d)));
    d += __uint_as_float(dpp<kQuadXor2>(__float_as_uint(d)));
    d += __uint_as_float(dpp<kRowRor4>(__float_as_uint(d)));
    d += __uint_as_float(dpp<kRowRor8>(__float_as_uint(d)));
    d += __shfl_xor(d, 16, 64);
    return d + __shfl_xor(d, 32, 64);
}

// The 16 bytes at vector i of a row that is streamed once, as G values (4 FP32 or
// 8 BF16).
__device__ __forceinline__ uint4 load_row(const char *row, int64_t i)
{
    const u32x4_nt w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_nt *>(row) + i);
    return make_uint4(w.x, w.y, w.z, w.w);
}

// A segment of a row on its way from memory: lane l holds columns
// j0 + (64 u + l) G + e, G per 16-byte load; columns at or past V read as -inf.
// STREAM: the loads are non-temporal (rows that are read once).
template <bool BF16, bool STREAM = false>
struct Segment {
    static constexpr int G = BF16 ? 8 : 4, NQ = 32 / G;
    uint4 q[NQ];
    static __device__ __forceinline__ uint4 load16(const char *p)
    {
        return STREAM ? load_row(p, 0) : *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void load(const void *row, int64_t V, int64_t j0, int lane)
    {
        const char *base = static_cast<const char *>(row) + j0 * (16 / G);
        const uint32_t at = static_cast<uint32_t>(lane) * 16;
        if (j0 + kSegCols <= V) {
#pragma unroll
            for (int u = 0; u < NQ; ++u)
                q[u] = load16(base + at + 1024 * u);
            return;
        }
        const uint32_t none = BF16 ? 0xff80ff80u : 0xff800000u;
        const int32_t cols = static_cast<int32_t>(V - j0), whole = cols / G;
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            q[u] = make_uint4(none, none, none, none);
            if (64 * u + lane < whole)
                q[u] = load16(base + at + 1024 * u);
        }
        if (whole * G < cols) {  // the one vector that the row's end lies in
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (BF16) {
                    const uint16_t *p = reinterpret_cast<const uint16_t *>(base) + whole * G + 2 * e;
                    const uint32_t lo = whole * G + 2 * e < cols ? p[0] : 0xff80u;
                    const uint32_t hi = whole * G + 2 * e + 1 < cols ? p[1] : 0xff80u;
                    w[e] = lo | (hi << 16);
                } else {
                    w[e] = whole * G + e < cols ? reinterpret_cast<const uint32_t *>(base)[whole * G + e] : none;
                }
            }
#pragma unroll
            for (int u = 0; u < NQ; ++u)
                if (64 * u + lane == whole)
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

// Columns a thread takes at a time of a row that is read and written once: 16 bytes of
// the wider type (stores of 32 bytes a lane, in two halves, took 1.5 times as long).
template <bool ZBF16, bool GBF16>
constexpr int kRowVec = ZBF16 && GBF16 ? 8 : 4;

// G columns of such a row, 8 or 16 bytes.
template <bool BF16, int G>
struct RowVec {
    static constexpr int kBytes = G * (BF16 ? 2 : 4), kWords = kBytes / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const char *p)
    {
        if constexpr (kWords == 4) {
            const u32x4_nt q = __builtin_nontemporal_load(reinterpret_cast<const u32x4_nt *>(p));
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else {
            const u32x2_nt q = __builtin_nontemporal_load(reinterpret_cast<const u32x2_nt *>(p));
            w[0] = q.x, w[1] = q.y;
        }
    }
    __device__ __forceinline__ float value(int e) const
    {
        if constexpr (BF16)
            return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        else
            return __uint_as_float(w[e]);
    }
};

template <bool BF16>
__device__ __forceinline__ float row_element(const char *row, int64_t j)
{
    if constexpr (BF16)
        return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[j]) << 16);
    else
        return reinterpret_cast<const float *>(row)[j];
}

typedef float f32x2_cvt __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_cvt __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)  // nearest even
{
    const f32x2_cvt v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_cvt));
}

// G gradients at vector i of a row, FP32 or rounded once to BF16.
template <bool BF16, int G>
__device__ __forceinline__ void store_row(char *row, int64_t i, const float (&o)[G])
{
    if constexpr (BF16) {
        uint16_t *p = reinterpret_cast<uint16_t *>(row) + i * G;
        if constexpr (G == 8)
            store16(p, make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                                  pack_bf16(o[6], o[7])), true);
        else
            store8(p, make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])), true);
    } else {
        float *p = reinterpret_cast<float *>(row) + i * G;
#pragma unroll
        for (int e = 0; e < G; e += 4)
            store16(p + e, make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]), true);
    }
}
template <bool BF16>
__device__ __forceinline__ void store_element(char *row, int64_t j, float o)
{
    if constexpr (BF16)
        reinterpret_cast<uint16_t *>(row)[j] = static_cast<uint16_t>(f32_to_bf16_bits(o));
    else
        reinterpret_cast<float *>(row)[j] = o;
}

constexpr float kNoTerm = -200.0f;  // 2^-200 is 0 in FP32: what -inf is cut to

// A temperature that is not positive and finite makes the row NaN, and so does one below
// 4.3e-39: log2(e) / T, by which the exponents are formed, passes the FP32 range there,
// and (m - m) log2(e) / T is NaN (but not where every column is listed with a class for
// the rest, so it is decided here).
__device__ __forceinline__ float inverse_temperature(const float *t, int64_t i)
{
    if (!t)
        return 1.0f;
    const float v = t[i], inv = 1.0f / v;
    return (v > 0.0f && v < INFINITY && kLog2e * inv < INFINITY) ? inv : __int_as_float(0x7fc00000);
}

// The k largest of a segment's values (v, held as Segment loads them, some above
// -inf, none NaN or +inf; gm the maxima of four at a time, lm the lane's) into
// out[0 .. k), as keys: order_key above the complement of the column, so that a
// larger key is a larger value or an equal one of an earlier column; 0 where fewer
// lie above -inf.  Candidates: the k-th largest of the 64 lane maxima is a lower
// bound of the segment's k-th largest value (that many lanes hold a value at least
// as large), cut to its upper 16 bits so that 16 ballots find it; the few values
// at or above it are collected in LDS (mine[kCandCap], the wave's own) and ranked
// by counting.
template <int G>
__device__ __forceinline__ void keep_largest(const float (&v)[32], const float (&gm)[8], float lm,
                                             uint32_t j0, int lane, int k, uint64_t *mine,
                                             uint64_t *out)
{
    const uint32_t mykey = order_key(lm);
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b >= 16; --b) {
        const uint32_t c = t | (1u << b);
        if (__popcll(__ballot(mykey >= c)) >= k)
            t = c;
    }
    const float bound = key_value(max(t, order_key(-INFINITY) + 1u));
    const uint32_t rest = 0xffffffffu - (j0 + static_cast<uint32_t>(lane * G));
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

}  // namespace lmh
