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
// bytes; a separate rotation would write and read the keys once more. A block takes a tile of
// up to 4 tokens: the tile's cosines and sines are gathered into shared memory (one thread per
// pair, whatever its axis; positions two tiles ahead, table entries one tile ahead by cp.async),
// and its warps stream the tile's rows, D / 16 lanes a row and 16 elements a lane, each warp with
// the next rows in flight. A lane's four chunks of 4 elements lie D / 4 apart, so both members
// of a pair are in one lane where rotary_dim is D or D / 2; other widths load the partner too.
// Neighbouring warps take neighbouring rows, so the block reads and writes contiguous memory.
// (A first version gave a warp one token and kept its angles in registers: 24 warps per SM at
// distant addresses, waiting on every token's position -> table chain, ran the 32768-token fp32
// prompt in 632 us, this one in 229 in graph replays, 0.95 of the copy rate.) Other widths load
// their rotated chunks twice and spill: 340 us for that prompt at rotary_dim 32 of 128. Few tokens
// leave SMs empty, so a tile's rows are then split over several blocks.
#pragma once

#include <cuda_bf16.h>

#include "q8kv_cache_write.cuh"

namespace q8kv {

constexpr unsigned kErrPosition = 0x40u; // a position outside the table (clamped)
constexpr int kRopeAxes = 4;

// How a pair's two channels lie: two chunks of a lane apart (rotary_dim = head_dim), one chunk
// apart (head_dim / 2), anywhere in the row (a second load fetches the partner), or next to
// each other.
enum RopeMode { kRopeFull = 0, kRopeHalf = 1, kRopeAnywhere = 2, kRopeAdjacent = 3 };

constexpr int kRopeChunks = 4; // chunks of 4 elements per lane and row
__host__ __device__ constexpr int rope_lanes(int D)
{
    return D / 16; // lanes per row
}
__host__ __device__ constexpr int rope_rows(int D)
{
    return 32 / rope_lanes(D); // rows per warp and iteration
}

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
    int tile, parts; // tokens per block and step; blocks that share a tile
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

// One row as loaded by its lanes: its chunks and, for kRopeAnywhere, those of their partners.
template <typename T, int MODE>
struct RopeRow {
    Raw4<T> x[kRopeChunks];
    Raw4<T> y[MODE == kRopeAnywhere ? kRopeChunks : 1];
};

struct RopeFrag {
    float4 x[kRopeChunks];
};

template <int D, typename T, int MODE>
__device__ __forceinline__ RopeRow<T, MODE> load_row(const T *row, int sub, int rot, bool turn)
{
    RopeRow<T, MODE> r;
#pragma unroll
    for (int c = 0; c < kRopeChunks; ++c) {
        const int e = 4 * (sub + rope_lanes(D) * c);
        r.x[c] = load_raw<T>(row + e);
        if constexpr (MODE == kRopeAnywhere) {
            const int half = rot >> 1;
            r.y[c] = r.x[c];
            if (turn && e < rot)
                r.y[c] = load_raw<T>(row + (e < half ? e + half : e - half));
        }
    }
    return r;
}

// The rotated row; cosines of the token's pairs lie at cs, sines at cs + rot / 2.
template <int D, typename T, int MODE>
__device__ __forceinline__ RopeFrag rotate(const RopeRow<T, MODE> &r, const float *cs, int sub,
                                           int rot, bool turn)
{
    RopeFrag f;
#pragma unroll
    for (int c = 0; c < kRopeChunks; ++c)
        f.x[c] = widen<T>(r.x[c]);
    if (!turn)
        return f;
    if constexpr (MODE == kRopeFull || MODE == kRopeHalf) {
        constexpr int kApart = MODE == kRopeFull ? 2 : 1, kPairs = D / 4 * kApart;
#pragma unroll
        for (int c = 0; c < kApart; ++c) {
            const int e = 4 * (sub + rope_lanes(D) * c);
            const float4 co = *reinterpret_cast<const float4 *>(cs + e);
            const float4 si = *reinterpret_cast<const float4 *>(cs + kPairs + e);
            const float4 lo = f.x[c], hi = f.x[c + kApart];
            f.x[c] = rot_lo4(lo, hi, co, si);
            f.x[c + kApart] = rot_hi4(hi, lo, co, si);
        }
    } else if constexpr (MODE == kRopeAnywhere) {
        const int half = rot >> 1;
#pragma unroll
        for (int c = 0; c < kRopeChunks; ++c) {
            const int e = 4 * (sub + rope_lanes(D) * c);
            if (e >= rot)
                continue;
            const bool low = e < half;
            const float4 y = widen<T>(r.y[c]);
            const float4 co = *reinterpret_cast<const float4 *>(cs + (low ? e : e - half));
            const float4 si = *reinterpret_cast<const float4 *>(cs + (low ? e + half : e));
            f.x[c] = low ? rot_lo4(f.x[c], y, co, si) : rot_hi4(f.x[c], y, co, si);
        }
    } else {
        const float *sn = cs + (rot >> 1);
#pragma unroll
        for (int c = 0; c < kRopeChunks; ++c) {
            const int e = 4 * (sub + rope_lanes(D) * c);
            if (e >= rot)
                continue;
            const float4 x = f.x[c];
            const float2 co = *reinterpret_cast<const float2 *>(cs + (e >> 1));
            const float2 si = *reinterpret_cast<const float2 *>(sn + (e >> 1));
            f.x[c] = make_float4(rot_lo(x.x, x.y, co.x, si.x), rot_hi(x.y, x.x, co.x, si.x),
                                 rot_lo(x.z, x.w, co.y, si.y), rot_hi(x.w, x.z, co.y, si.y));
        }
    }
    return f;
}

// Quantise one row by the cache write's rule (q8kv_cache_write.cuh) with this kernel's lanes
// (all of the warp take part in the reductions); if `store`, write the lane's codes. Returns
// the row's scale and sets `bad` for a non-finite row.
template <int D>
__device__ __forceinline__ float rope_quantise(const RopeFrag &f, int8_t *dst, bool store, int sub,
                                               bool &bad)
{
    float m = 0.f;
    unsigned odd = 0;
#pragma unroll
    for (int c = 0; c < kRopeChunks; ++c) {
        const float a[4] = {fabsf(f.x[c].x), fabsf(f.x[c].y), fabsf(f.x[c].z), fabsf(f.x[c].w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            odd |= a[i] <= 3.402823466e38f ? 0u : 1u; // an infinity or a NaN
            m = fmaxf(m, a[i]);
        }
    }
#pragma unroll
    for (int o = rope_lanes(D) / 2; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        odd |= __shfl_xor_sync(0xffffffffu, odd, o);
    }
    bad = odd != 0u;
    if (m < 1e-6f)
        m = 1.0f;
    const float scale = bad ? __int_as_float(0x7fc00000) : __fmul_rn(m, 0x1.020408p-7f);
    const float inv = __fdiv_rn(127.0f, m);
    if (store) {
#pragma unroll
        for (int c = 0; c < kRopeChunks; ++c) {
            const float4 x = f.x[c];
            const uint32_t w = code_byte(x.x, inv) | (code_byte(x.y, inv) << 8) |
                               (code_byte(x.z, inv) << 16) | (code_byte(x.w, inv) << 24);
            reinterpret_cast<uint32_t *>(dst)[sub + rope_lanes(D) * c] = bad ? 0u : w;
        }
    }
    return scale;
}

// Iterations of a token: its query rows, rope_rows(D) at a time, then its key and value rows.
__host__ __device__ constexpr int rope_iters(int Hq, int Hk, int D)
{
    const int ppw = rope_rows(D);
    return (Hq + ppw - 1) / ppw + (2 * Hk + ppw - 1) / ppw;
}

constexpr int kRopeTile = 4; // tokens per block and step, at most
// Resident blocks per SM: a 16-bit row keeps fewer bytes in flight per warp and fewer registers,
// so there is room and need for a fourth block, except where a lane also holds its partners'
// chunks and would spill at 64 registers (13392 bf16 tokens, 32 / 8 heads of 128, with 3 / 4 blocks:
// rotary_dim 128 78.3 / 73.8 us, 64 77.7 / 74.2, 128 adjacent 78.6 / 75.8; kRopeAnywhere: 32 101.8
// / 107.4, 96 106.9 / 112.5; 4999 tokens of 32 40.5 / 44.6).
template <typename T>
__host__ __device__ constexpr int rope_blocks(int mode)
{
    return sizeof(T) == 2 && mode != kRopeAnywhere ? 4 : 3;
}

// A block's share of one step: a tile of tokens, or a part of its iterations.
struct RopeUnit {
    long long tok0;
    int nt, j, j1; // tokens; this warp's first iteration and the end of the block's
};

template <int D, typename T, int MODE>
__global__ void __launch_bounds__(kWriteThreads, rope_blocks<T>(MODE))
    rope_cache_write_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int LPR = rope_lanes(D);
    constexpr int PPW = rope_rows(D);
    constexpr int C = kRopeChunks;
    __shared__ __align__(16) float angle[2][kRopeTile][D]; // cosines, then sines, of a token
    __shared__ long long tile_slot[2][kRopeTile];
    // the new rows may come from the kernel before this one on the stream
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sub = lane % LPR, grp = lane / LPR;
    const int q_iters = (p.Hq + PPW - 1) / PPW;
    const int iters = rope_iters(p.Hq, p.Hk, D);
    const int half = p.rot >> 1;
    const long long units = (p.n_tokens + p.tile - 1) / p.tile * p.parts;
    unsigned err = 0;

    auto unit_at = [&](long long unit) {
        RopeUnit u;
        const long long tile = unit / p.parts;
        const int part = (int)(unit - tile * p.parts);
        u.tok0 = tile * p.tile;
        u.nt = p.n_tokens - u.tok0 < p.tile ? (int)(p.n_tokens - u.tok0) : p.tile;
        const int all = u.nt * iters; // iterations of the tile, token by token
        u.j = part * all / p.parts + warp;
        u.j1 = (part + 1) * all / p.parts;
        return u;
    };
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
    // Positions of a unit's tokens for this thread's pair, and (one thread per token) the slot:
    // loaded two units ahead; the table's entries follow one unit ahead by cp.async.
    int pos[kRopeTile];
    long long slot = -1;
    const int st = tid - (kWriteThreads - kRopeTile); // the token whose slot this thread takes
    const int axis = tid < half ? p.axis[tid] : 0;
    auto load_pos = [&](long long unit) {
        if (unit >= units)
            return;
        const RopeUnit u = unit_at(unit);
#pragma unroll
        for (int t = 0; t < kRopeTile; ++t)
            pos[t] = tid < half && t < u.nt ? __ldg(p.pos + axis * p.n_tokens + u.tok0 + t) : 0;
        if (st >= 0 && st < u.nt)
            slot = __ldg(p.slots + u.tok0 + st);
    };
    auto load_angles = [&](long long unit, int buf) {
        if (unit < units) {
            const int nt = unit_at(unit).nt;
            if (tid < half) {
                const uint32_t dst = smem_addr(&angle[buf][0][tid]);
#pragma unroll
                for (int t = 0; t < kRopeTile; ++t)
                    if (t < nt) {
                        int x = pos[t];
                        if (x < 0 || x >= p.max_pos) {
                            err |= kErrPosition;
                            x = x < 0 ? 0 : p.max_pos - 1;
                        }
                        const float *row = p.table + (long long)x * p.rot + tid;
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                         dst + (uint32_t)(t * D * 4)),
                                     "l"(row)
                                     : "memory");
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                         dst + (uint32_t)((t * D + half) * 4)),
                                     "l"(row + half)
                                     : "memory");
                    }
            }
            if (st >= 0 && st < nt) {
                if (slot >= p.n_slots) {
                    err |= kErrSlot;
                    slot = -1;
                }
                tile_slot[buf][st] = slot;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    long long unit = blockIdx.x;
    if (unit >= units)
        return;
    RopeUnit u = unit_at(unit);
    bool exists = false, turn = false;
    RopeRow<T, MODE> cur;
    int tk = u.j / iters, it = u.j - tk * iters;
    if (u.j < u.j1)
        cur = load_row<D, T, MODE>(row_of(u.tok0 + tk, it, exists, turn), sub, p.rot, turn);
    load_pos(unit);
    load_angles(unit, 0);
    load_pos(unit + gridDim.x);
    for (int buf = 0;; buf ^= 1) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads(); // this unit's angles are there, the last unit's are read no more
        const long long next_unit = unit + gridDim.x;
        load_angles(next_unit, buf ^ 1);
        load_pos(next_unit + gridDim.x);
        const bool more = next_unit < units;
        const RopeUnit nu = more ? unit_at(next_unit) : u;
        bool any = u.j < u.j1;
        if (!any && more && nu.j < nu.j1) { // nothing to do here: on to the next unit's rows
            tk = nu.j / iters;
            it = nu.j - tk * iters;
            cur = load_row<D, T, MODE>(row_of(nu.tok0 + tk, it, exists, turn), sub, p.rot, turn);
        }
        while (any) {
            // the next rows (the next unit's first, at the end) are in flight while this
            // iteration's are turned and stored
            const long long tok = u.tok0 + tk;
            const int t = tk, i = it;
            u.j += kWriteWarps;
            it += kWriteWarps;
            while (it >= iters) {
                it -= iters;
                ++tk;
            }
            any = u.j < u.j1;
            long long ntok = u.tok0 + tk;
            bool load = any;
            if (!any && more && nu.j < nu.j1) {
                tk = nu.j / iters;
                it = nu.j - tk * iters;
                ntok = nu.tok0 + tk;
                load = true;
            }
            bool next_exists = false, next_turn = false;
            RopeRow<T, MODE> next = cur;
            if (load)
                next = load_row<D, T, MODE>(row_of(ntok, it, next_exists, next_turn), sub, p.rot,
                                            next_turn);
            const RopeFrag f = rotate<D, T, MODE>(cur, angle[buf][t], sub, p.rot, turn);
            if (i < q_iters) {
                if constexpr (MODE == kRopeAnywhere)
                    __syncwarp(); // in place: every lane has read its partners
                if (exists) {
                    float4 *dst =
                        reinterpret_cast<float4 *>(p.q_out + (tok * p.Hq + i * PPW + grp) * D);
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        dst[sub + LPR * c] = f.x[c];
                }
            } else {
                const int r = (i - q_iters) * PPW + grp;
                const long long sl = tile_slot[buf][t];
                const bool store = exists && sl >= 0;
                const long long row = store ? sl * p.Hk + (turn ? r : r - p.Hk) : 0;
                bool bad;
                const float sc =
                    rope_quantise<D>(f, (turn ? p.k : p.v) + row * D, store, sub, bad);
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
        if (!more)
            break;
        unit = next_unit;
        u = nu;
    }
    if (err)
        atomicOr(p.errors, err);
}

} // namespace q8kv
