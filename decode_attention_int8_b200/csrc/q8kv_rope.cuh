// q8kv_rope.cuh -- rotary positions with one to four axes, fused with the q8 cache write: the
// new tokens' query and key rows are rotated, the queries written as the fp32 rows the decode
// reads, the rotated keys and the values quantised and stored at their slots.
//
// What it computes, per token i and pair p of a rotated row (rotary_dim / 2 pairs): with
// (c, s) the cosine and sine of pair p at position positions[axis(p)][i] (a row of the table),
//   x1' = fl(fl(x1 c) - fl(x2 s)),   x2' = fl(fl(x2 c) + fl(x1 s)),
// every operation rounded to fp32 on its own, because the keys' codes are whole numbers that a
// contraction into an FMA would change. Pair p is (p, p + rotary_dim / 2), or (2p, 2p + 1)
// with adjacent pairing; channels past rotary_dim pass through. Images and video give time,
// height and width a position each: axis(p) says which of them turns pair p. Keys and values
// are then quantised by the row rule of q8kv_cache_write.cuh.
//
// What bounds it: HBM. A token reads (Hq + 2 Hk) D elements and writes 4 Hq D + 2 Hk (D + 4)
// bytes; a separate rotation would write and read the keys once more. The table rows are
// shared by a token's Hq + Hk rotated rows, so a warp takes the rows of one token one after
// the other and keeps the cosines and sines of its lanes' pairs in registers: a row has 8
// lanes (16 for head_dim 256) of 4-element chunks, as in the cache write, so 4 (or 2) rows
// go at once, and with rotary_dim = head_dim and pairs (p, p + D / 2) both members of a pair
// lie in one lane. Few tokens leave most of the machine empty when a warp takes a whole token,
// so a token's rows are then split over several warps (rope_parts).
#pragma once

#include <cuda_bf16.h>

#include "q8kv_cache_write.cuh"

namespace q8kv {

constexpr unsigned kErrPosition = 0x40u; // a position outside the table (clamped)
constexpr int kRopeAxes = 4;

// How a pair's two channels lie: both in one lane (rotary_dim = head_dim), anywhere in the
// row (a second load fetches the partner), or next to each other.
enum RopeMode { kRopeFull = 0, kRopeHalf = 1, kRopeAdjacent = 2 };

struct RopeParams {
    float *q_out;
    int8_t *k, *v;
    float *ks, *vs;
    const void *q_new, *k_new, *v_new;
    const int64_t *slots;
    const int32_t *pos;  // [n_axes][n_tokens]
    const float *table;  // [max_pos][rot]: cosines of the pairs, then sines
    long long n_tokens;
    long long q_stride, kv_stride; // elements from one token's rows to the next token's
    long long n_slots;
    int Hq, Hk, rot, max_pos, n_axes;
    int parts;      // warps per token
    unsigned *errors;
    uint8_t axis[128]; // axis of each pair
};

// Four consecutive elements as loaded, and as fp32 (exact).
template <typename T>
struct Raw4 {
    uint2 w;
};
template <>
struct Raw4<float> {
    float4 w;
};

template <typename T>
__device__ __forceinline__ Raw4<T> load_raw(const T *p)
{
    Raw4<T> r;
    if constexpr (sizeof(T) == 4)
        r.w = __ldcs(reinterpret_cast<const float4 *>(p));
    else
        r.w = __ldcs(reinterpret_cast<const uint2 *>(p));
    return r;
}

template <typename T>
__device__ __forceinline__ float4 widen(const Raw4<T> &r)
{
    if constexpr (sizeof(T) == 4) {
        return r.w;
    } else {
        if constexpr (std::is_same_v<T, __half>) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&r.w.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&r.w.y));
            return make_float4(a.x, a.y, b.x, b.y);
        } else { // bfloat16: the upper half of the fp32 bits
            return make_float4(__uint_as_float(r.w.x << 16), __uint_as_float(r.w.x & 0xffff0000u),
                               __uint_as_float(r.w.y << 16), __uint_as_float(r.w.y & 0xffff0000u));
        }
    }
}

// x1 c - x2 s and x2 c + x1 s, each operation rounded
__device__ __forceinline__ float rot_lo(float a, float b, float c, float s)
{
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rot_hi(float b, float a, float c, float s)
{
    return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
__device__ __forceinline__ float4 rot_lo4(float4 a, float4 b, float4 c, float4 s)
{
    return make_float4(rot_lo(a.x, b.x, c.x, s.x), rot_lo(a.y, b.y, c.y, s.y),
                       rot_lo(a.z, b.z, c.z, s.z), rot_lo(a.w, b.w, c.w, s.w));
}
__device__ __forceinline__ float4 rot_hi4(float4 b, float4 a, float4 c, float4 s)
{
    return make_float4(rot_hi(b.x, a.x, c.x, s.x), rot_hi(b.y, a.y, c.y, s.y),
                       rot_hi(b.z, a.z, c.z, s.z), rot_hi(b.w, a.w, c.w, s.w));
}

// A lane's cosines and sines for one token: kRopeFull keeps the pairs of its first C / 2
// chunks, kRopeHalf those of each chunk, kRopeAdjacent the two pairs of each chunk (in c4's
// x, y and s4's x, y).
template <int D, int MODE>
struct Angles {
    static constexpr int C = RowFrag<D>::C;
    static constexpr int N = MODE == kRopeFull ? C / 2 : C;
    float4 c[N], s[N];
};

__device__ __forceinline__ int axis_pos(const int (&pos)[kRopeAxes], int a)
{
    int r = pos[0];
#pragma unroll
    for (int i = 1; i < kRopeAxes; ++i)
        r = a == i ? pos[i] : r;
    return r;
}

// Cosines (and sines) of the 4 pairs p .. p + 3 (p a multiple of 4).
__device__ __forceinline__ void angles4(const RopeParams &p, const int (&pos)[kRopeAxes], int pair,
                                        float4 &c, float4 &s)
{
    const uint32_t a = *reinterpret_cast<const uint32_t *>(p.axis + pair);
    const int half = p.rot >> 1;
    if (a == (a & 0xffu) * 0x01010101u) { // one axis for all four
        const float *row = p.table + (long long)axis_pos(pos, a & 0xffu) * p.rot + pair;
        c = __ldg(reinterpret_cast<const float4 *>(row));
        s = __ldg(reinterpret_cast<const float4 *>(row + half));
        return;
    }
    float cc[4], ss[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float *row =
            p.table + (long long)axis_pos(pos, (a >> (8 * i)) & 0xffu) * p.rot + pair + i;
        cc[i] = __ldg(row);
        ss[i] = __ldg(row + half);
    }
    c = make_float4(cc[0], cc[1], cc[2], cc[3]);
    s = make_float4(ss[0], ss[1], ss[2], ss[3]);
}

template <int D, int MODE>
__device__ __forceinline__ Angles<D, MODE> load_angles(const RopeParams &p,
                                                       const int (&pos)[kRopeAxes], int sub)
{
    constexpr int LPR = write_lanes_per_row(D);
    Angles<D, MODE> a;
    const int half = p.rot >> 1;
#pragma unroll
    for (int i = 0; i < Angles<D, MODE>::N; ++i) {
        const int e = 4 * (sub + LPR * i); // first channel of the chunk
        a.c[i] = make_float4(1.f, 1.f, 1.f, 1.f);
        a.s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (MODE == kRopeAdjacent) {
            if (e < p.rot) {
                const int pair = e >> 1;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float *row =
                        p.table + (long long)axis_pos(pos, p.axis[pair + k]) * p.rot + pair + k;
                    const float c = __ldg(row), s = __ldg(row + half);
                    (k ? a.c[i].y : a.c[i].x) = c;
                    (k ? a.s[i].y : a.s[i].x) = s;
                }
            }
        } else {
            if (e < p.rot)
                angles4(p, pos, MODE == kRopeHalf && e >= half ? e - half : e, a.c[i], a.s[i]);
        }
    }
    return a;
}

// One row as loaded by its lanes: its chunks and, for kRopeHalf, the chunks of their partners.
template <int D, typename T, int MODE>
struct RopeRow {
    static constexpr int C = RowFrag<D>::C;
    Raw4<T> x[C];
    Raw4<T> y[MODE == kRopeHalf ? C : 1];
};

template <int D, typename T, int MODE>
__device__ __forceinline__ RopeRow<D, T, MODE> load_row(const T *row, int sub, int rot, bool turn)
{
    constexpr int LPR = write_lanes_per_row(D);
    RopeRow<D, T, MODE> r;
#pragma unroll
    for (int c = 0; c < RowFrag<D>::C; ++c) {
        const int e = 4 * (sub + LPR * c);
        r.x[c] = load_raw<T>(row + e);
        if constexpr (MODE == kRopeHalf) {
            const int half = rot >> 1;
            r.y[c] = r.x[c];
            if (turn && e < rot)
                r.y[c] = load_raw<T>(row + (e < half ? e + half : e - half));
        }
    }
    return r;
}

template <int D, typename T, int MODE>
__device__ __forceinline__ RowFrag<D> rotate(const RopeRow<D, T, MODE> &r,
                                             const Angles<D, MODE> &a, int sub, int rot, bool turn)
{
    constexpr int LPR = write_lanes_per_row(D);
    constexpr int C = RowFrag<D>::C;
    RowFrag<D> f;
#pragma unroll
    for (int c = 0; c < C; ++c)
        f.x[c] = widen<T>(r.x[c]);
    if (!turn)
        return f;
    if constexpr (MODE == kRopeFull) {
#pragma unroll
        for (int c = 0; c < C / 2; ++c) {
            const float4 lo = f.x[c], hi = f.x[c + C / 2];
            f.x[c] = rot_lo4(lo, hi, a.c[c], a.s[c]);
            f.x[c + C / 2] = rot_hi4(hi, lo, a.c[c], a.s[c]);
        }
    } else if constexpr (MODE == kRopeHalf) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = 4 * (sub + LPR * c);
            const float4 y = widen<T>(r.y[c]);
            if (e < (rot >> 1))
                f.x[c] = rot_lo4(f.x[c], y, a.c[c], a.s[c]);
            else if (e < rot)
                f.x[c] = rot_hi4(f.x[c], y, a.c[c], a.s[c]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (4 * (sub + LPR * c) < rot) {
                const float4 x = f.x[c], cc = a.c[c], ss = a.s[c];
                f.x[c] = make_float4(rot_lo(x.x, x.y, cc.x, ss.x), rot_hi(x.y, x.x, cc.x, ss.x),
                                     rot_lo(x.z, x.w, cc.y, ss.y), rot_hi(x.w, x.z, cc.y, ss.y));
            }
        }
    }
    return f;
}

// Iterations of a token: its query rows PPW at a time, then its key and value rows.
__host__ __device__ constexpr int rope_iters(int Hq, int Hk, int D)
{
    const int ppw = write_pairs_per_warp(D);
    return (Hq + ppw - 1) / ppw + (2 * Hk + ppw - 1) / ppw;
}

template <int D, typename T, int MODE>
__global__ void __launch_bounds__(kWriteThreads, 3)
    rope_cache_write_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int LPR = write_lanes_per_row(D);
    constexpr int PPW = write_pairs_per_warp(D);
    constexpr int C = RowFrag<D>::C;
    // the new rows may come from the kernel before this one on the stream
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, sub = lane % LPR, grp = lane / LPR;
    const long long items = p.n_tokens * p.parts;
    const long long step = (long long)gridDim.x * kWriteWarps;
    const int q_iters = (p.Hq + PPW - 1) / PPW;
    const int iters = rope_iters(p.Hq, p.Hk, D);
    unsigned err = 0;

    // this lane's row of iteration it of token `tok`: where it starts, whether it exists
    auto row_of = [&](long long tok, int it, bool &exists, bool &turn) -> const T * {
        if (it < q_iters) {
            const int h = it * PPW + grp;
            exists = h < p.Hq;
            turn = true;
            return static_cast<const T *>(p.q_new) + tok * p.q_stride +
                   (long long)(exists ? h : 0) * D;
        }
        const int r = (it - q_iters) * PPW + grp;
        exists = r < 2 * p.Hk;
        turn = r < p.Hk;
        const int h = !exists ? 0 : (turn ? r : r - p.Hk);
        return static_cast<const T *>(turn ? p.k_new : p.v_new) + tok * p.kv_stride +
               (long long)h * D;
    };

#pragma unroll 1
    for (long long item = (long long)blockIdx.x * kWriteWarps + (threadIdx.x >> 5); item < items;
         item += step) {
        const long long tok = item / p.parts;
        const int part = (int)(item - tok * p.parts);
        const int it0 = part * iters / p.parts, it1 = (part + 1) * iters / p.parts;
        bool exists, turn;
        RopeRow<D, T, MODE> cur;
        {
            const T *row = row_of(tok, it0, exists, turn);
            cur = load_row<D, T, MODE>(row, sub, p.rot, turn);
        }
        int pos[kRopeAxes];
#pragma unroll
        for (int a = 0; a < kRopeAxes; ++a) {
            int x = a < p.n_axes ? __ldg(p.pos + a * p.n_tokens + tok) : 0;
            if (x < 0 || x >= p.max_pos) {
                err |= kErrPosition;
                x = x < 0 ? 0 : p.max_pos - 1;
            }
            pos[a] = x;
        }
        long long slot = __ldg(p.slots + tok);
        if (slot >= p.n_slots) {
            err |= kErrSlot;
            slot = -1;
        }
        const Angles<D, MODE> ang = load_angles<D, MODE>(p, pos, sub);
#pragma unroll 1
        for (int it = it0; it < it1; ++it) {
            // the next rows are in flight while this iteration's are turned and stored
            bool next_exists = false, next_turn = false;
            RopeRow<D, T, MODE> next = cur;
            if (it + 1 < it1) {
                const T *row = row_of(tok, it + 1, next_exists, next_turn);
                next = load_row<D, T, MODE>(row, sub, p.rot, next_turn);
            }
            const RowFrag<D> f = rotate<D, T, MODE>(cur, ang, sub, p.rot, turn);
            if (it < q_iters) {
                if constexpr (MODE == kRopeHalf)
                    __syncwarp(); // in place: every lane has read its partners
                if (exists) {
                    float4 *dst = reinterpret_cast<float4 *>(
                        p.q_out + (tok * p.Hq + it * PPW + grp) * D);
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        dst[sub + LPR * c] = f.x[c];
                }
            } else {
                const int r = (it - q_iters) * PPW + grp;
                const bool store = exists && slot >= 0;
                const long long row = store ? slot * p.Hk + (turn ? r : r - p.Hk) : 0;
                bool bad;
                const float sc =
                    quantise_row<D>(f, (turn ? p.k : p.v) + row * D, store, sub, bad);
                if (store) {
                    if (sub == 0)
                        (turn ? p.ks : p.vs)[row] = sc;
                    if (bad)
                        err |= kErrNonFinite;
                }
            }
            cur = next;
            exists = next_exists;
            turn = next_turn;
        }
    }
    if (err)
        atomicOr(p.errors, err);
}

} // namespace q8kv
