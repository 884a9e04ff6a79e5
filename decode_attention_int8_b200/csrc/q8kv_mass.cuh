// q8kv_mass.cuh -- accumulated attention weights of the cached tokens, the quantity an eviction
// policy ranks them by.
//
// What it computes, per sequence b, KV head kv and token t < L_b:
//   mass[b][kv][t] = decay * mass[b][kv][t] + sum over the head's query rows r of
//                    exp(s_rt - lse_r),
// with the decode's own scores s (int8 query blocks, exact block dots, q8kv_decode.cuh) and
// the log-sum-exp of each row that the decode left: one pass over K, no softmax to redo.
//
// What bounds it: HBM, at 132 bytes of K and 8 of mass per (token, KV head). A warp takes 16
// tokens of one head at a time: tokens are the M rows of mma.m16n8k32.s8, four query rows its N
// columns twice over. A lane owns 16 consecutive bytes of a token's row; with those as the MMA's
// k positions, lanes c = 0, 1 hold block 2h of the row (h: which half) and lanes c = 2, 3 block
// 2h + 1, and the query operand is zero where column group n / 4 and block differ. One
// accumulator so carries two blocks' exact dots side by side, every column is used, and two
// shuffles bring the halves together, each lane keeping two rows of one token.
//
// Every lane copies its own bytes (and its token's scale and old mass) ahead of use with
// cp.async into a ring of kMassStages tiles in shared memory that only it reads: the copies in
// flight cost no registers and no synchronisation. (With the next tile's operands in registers
// instead, the kernel spilled at 24 warps per SM and took 114 us on 48 ragged sequences of up
// to 16384 tokens, 64 / 8 heads; at 16 warps 107 us.) The tokens of all sequences form one list
// that the blocks share evenly; a block's warps take different heads of the same tokens,
// whose rows are neighbours in the pool. The block quantises a segment's query rows together,
// into shared memory, while the first tiles are on their way.
#pragma once

#include <cstdint>
#include <type_traits>

#include "q8kv_decode.cuh"

namespace q8kv {

constexpr int kMassMaxWarps = 8;
constexpr int kMassTile = 16;    // tokens per warp step
constexpr int kMassStages = 4;   // tiles in a warp's ring
constexpr int kMassMaxBatch = 16384;
constexpr int kMassMaxRows = 128; // query rows per KV head
constexpr int kMassStageBytes = 32 * (64 + 8); // per lane: 64 bytes of K, the scale, the mass

struct MassParams {
    float *mass;       // [B][Hk][cap]
    const float *q;    // [B][nq][Hq][128]
    const float *lse;  // [B][nq][Hq]
    const int8_t *k;
    const float *ks;
    const int32_t *table, *lens;
    int B, nq, Hq, Hk, Gq, R; // Gq: query heads per KV head; R = nq Gq rows per KV head
    int quads;         // R / 4, rounded up
    int bs_log2, mbps, num_blocks, cap;
    int heads_pass;    // heads the block's warps cover at once
    int subs;          // warps that share a head's tokens
    float scale_log2, decay;
    unsigned *errors;
};

// Dynamic shared memory: the rings, the segment's query rows, the tile prefixes.
struct MassLayout {
    uint32_t off_codes, off_zero, off_qs, off_lse, off_view, off_prefix, total;
};

__host__ __device__ inline MassLayout mass_layout(int warps, int heads, int quads, int B)
{
    MassLayout l;
    uint32_t o = (uint32_t)(warps * kMassStages * kMassStageBytes);
    l.off_codes = o; // [head][row][128]
    o += (uint32_t)(heads * quads * 4 * kD);
    l.off_zero = o;  // 128 bytes of zeros
    o += kD;
    l.off_qs = o;    // [head][quad][c][half][row]: scales in the order the lanes use them
    o += (uint32_t)(heads * quads * 16 * 4);
    l.off_lse = o;   // [head][row]: log-sum-exp, base 2 (+inf: no row)
    o += (uint32_t)(heads * quads * 4 * 4);
    l.off_view = o;  // [row]: index of the row's query token
    o += (uint32_t)(quads * 4 * 4);
    l.off_prefix = o;
    l.total = o + 4u * (uint32_t)(B + 1);
    return l;
}

// The query operand of four rows in the lane order described above, with the scales and
// log-sum-exp of the two rows whose scores this lane keeps.
struct MassQuad {
    uint4 b[2];      // [half]: the lane's 16 code bytes
    float qs[2][2];  // [half][row]: scale of the lane's block
    float lse2[2];
};

__device__ __forceinline__ void mass_cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void mass_cp4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// NQ: quads held in registers (all of a head's rows), 0: read from shared memory per tile.
template <int NQ>
__global__ void __launch_bounds__(kMassMaxWarps * 32, 3)
    attn_mass_kernel(const __grid_constant__ MassParams p)
{
    extern __shared__ __align__(16) uint8_t msm[];
    __shared__ int wsum[kMassMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nwarps = blockDim.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const MassLayout lay = mass_layout(nwarps, p.heads_pass, p.quads, p.B);
    int *prefix = reinterpret_cast<int *>(msm + lay.off_prefix); // tiles before each sequence
    // the query, its statistics and the cache come from kernels before this one
    grid_dep_wait();
    grid_dep_launch();

    // ---- tiles of every sequence, as prefix sums; the rows' query indices
    if (tid < kD / 4)
        reinterpret_cast<uint32_t *>(msm + lay.off_zero)[tid] = 0u;
    for (int r = tid; r < 4 * p.quads; r += blockDim.x)
        reinterpret_cast<int *>(msm + lay.off_view)[r] = r / p.Gq;
    int carry = 0;
#pragma unroll 1
    for (int base = 0; base < p.B; base += blockDim.x) {
        const int b = base + tid;
        int n = 0;
        if (b < p.B) {
            int L = __ldg(p.lens + b);
            if (L < 0 || L > p.cap) {
                atomicOr(p.errors, kErrSeqLen);
                L = L < 0 ? 0 : p.cap;
            }
            n = (L + kMassTile - 1) / kMassTile;
        }
        int v = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(kFullMask, v, o);
            if (lane >= o)
                v += t;
        }
        if (lane == 31)
            wsum[warp] = v;
        __syncthreads();
        int off = carry, total = 0;
        for (int w = 0; w < nwarps; ++w) {
            off += w < warp ? wsum[w] : 0;
            total += wsum[w];
        }
        if (b < p.B)
            prefix[b + 1] = off + v;
        carry += total;
        __syncthreads();
    }
    if (tid == 0)
        prefix[0] = 0;
    __syncthreads();
    const int N = carry;
    int t0 = (int)((long long)N * blockIdx.x / gridDim.x);
    const int t1 = (int)((long long)N * (blockIdx.x + 1) / gridDim.x);
    const int hw = warp % p.heads_pass, sub = warp / p.heads_pass;
    const int bs_mask = (1 << p.bs_log2) - 1;
    const int sel = c >> 1; // which half of the tile's tokens this lane keeps
    const bool writer = (c & 1) == 0;
    const unsigned row8 = 8u * (unsigned)p.Hk * kD; // bytes from token t's row to t + 8's
    const bool old = p.decay != 0.f;
    // this lane's part of the ring: 16-byte slots 512 bytes apart, then the 4-byte ones
    const uint32_t ring = smem_addr(msm) + (uint32_t)(warp * kMassStages * kMassStageBytes);
    const uint32_t mine16 = ring + 16u * lane, mine4 = ring + 2048u + 4u * lane;
    // this lane's query bytes of a quad: those of row g & 3 where its block is in column group
    // g / 4, else zeros
    const bool in_col = (c >> 1) == (g >> 2);

    while (t0 < t1) {
        // the sequence of tile t0: the last b with prefix[b] <= t0
        int b = 0, z = p.B - 1;
        while (b < z) {
            const int m = (b + z + 1) >> 1;
            if (prefix[m] <= t0)
                b = m;
            else
                z = m - 1;
        }
        const int first = prefix[b];
        const int t2 = min(t1, prefix[b + 1]);
        int L = __ldg(p.lens + b);
        L = L > p.cap ? p.cap : L;
        const int32_t *table = p.table + (long long)b * p.mbps;
        const int all_see = L - (p.nq - 1); // tokens that every row sees
#pragma unroll 1
        for (int kv0 = 0; kv0 < p.Hk; kv0 += p.heads_pass) {
            const int kv = kv0 + hw;
            float *mass = p.mass + ((long long)b * p.Hk + kv) * p.cap + g + 8 * sel;
            const int8_t *kbase = p.k + ((long long)g * p.Hk + kv) * kD + 16 * c;
            const float *sbase = p.ks + (long long)(g + 8 * sel) * p.Hk + kv;
            const int step = p.subs * kMassTile;
            const int tok1 = kv < p.Hk ? (t2 - first) * kMassTile : 0;
            int ti = (t0 - first + sub) * kMassTile; // first token of the next tile to fetch
            int blk = ti < tok1 ? __ldg(table + (ti >> p.bs_log2)) : 0;
            uint32_t usable = 0;                     // one bit per fetched tile, latest lowest
            uint32_t put = 0;                        // ring offset of the next tile
            auto fetch = [&]() {
                usable <<= 1;
                if (ti < tok1) {
                    const bool ok = (unsigned)blk < (unsigned)p.num_blocks;
                    if (ok) {
                        const int slot = (blk << p.bs_log2) + (ti & bs_mask);
                        const long long row = (long long)slot * p.Hk; // (slot, head 0)
                        const int8_t *k = kbase + row * kD;
                        mass_cp16(mine16 + put, k);
                        mass_cp16(mine16 + put + 512, k + 64);
                        mass_cp16(mine16 + put + 1024, k + row8);
                        mass_cp16(mine16 + put + 1536, k + row8 + 64);
                        mass_cp4(mine4 + put, sbase + row);
                        // (in bounds of the row: a tile never passes the table's last block)
                        if (old)
                            mass_cp4(mine4 + put + 128, mass + ti);
                        usable |= 1u;
                    } else if (lane == 0) {
                        atomicOr(p.errors, kErrBlockTable);
                    }
                    ti += step;
                    if (ti < tok1) // (the next tile's block, a step ahead)
                        blk = __ldg(table + (ti >> p.bs_log2));
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                put = put == (kMassStages - 1) * kMassStageBytes ? 0 : put + kMassStageBytes;
            };
            int t = ti; // first token of the tile in use
#pragma unroll
            for (int i = 0; i < kMassStages - 1; ++i)
                fetch();

            // ---- the segment's query rows, by the whole block: 16 lanes per row
            __syncthreads(); // the last segment's rows have been read
#pragma unroll 1
            for (int x0 = 2 * warp; x0 < p.heads_pass * 4 * p.quads; x0 += 2 * nwarps) {
                const int x = x0 + (lane >> 4);
                const int hd = x / (4 * p.quads), r = x - hd * 4 * p.quads;
                const int part = lane & 15; // block part / 4, its values 8 (part % 4) ..
                const bool live = r < p.R && kv0 + hd < p.Hk;
                float v[8];
                float l2 = INFINITY;
                if (live) {
                    const int i = reinterpret_cast<const int *>(msm + lay.off_view)[r];
                    const long long row = ((long long)b * p.nq + i) * p.Hq +
                                          (long long)(kv0 + hd) * p.Gq + (r - i * p.Gq);
                    const float4 *src =
                        reinterpret_cast<const float4 *>(p.q + row * kD + 8 * part);
                    const float4 y = __ldg(src), w = __ldg(src + 1);
                    v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
                    v[4] = w.x, v[5] = w.y, v[6] = w.z, v[7] = w.w;
                    l2 = __ldg(p.lse + row) * 1.44269504088896341f;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = 0.f;
                }
                uint32_t lo, hi;
                float qsc;
                quantize_block_quad(v, lo, hi, qsc);
                if (hd < p.heads_pass) { // (the last step may pass the last row)
                    *reinterpret_cast<uint2 *>(msm + lay.off_codes +
                                               (uint32_t)(x * kD + 8 * part)) =
                        make_uint2(lo, hi);
                    if ((part & 3) == 0) {
                        // block j = 2h + c / 2 of row 2 (c & 1) + e lies at [c][h][e]
                        const int j = part >> 2, rr = r & 3;
                        const int cc = 2 * (j & 1) + (rr >> 1);
                        reinterpret_cast<float *>(
                            msm + lay.off_qs)[((x >> 2) * 4 + cc) * 4 + (j >> 1) * 2 + (rr & 1)] =
                            qsc;
                    }
                    if (part == 0)
                        reinterpret_cast<float *>(msm + lay.off_lse)[x] = l2;
                }
            }
            __syncthreads();
            auto quad = [&](int n) {
                MassQuad q;
                const int row = (hw * p.quads + n) * 4;
                const uint8_t *codes = in_col ? msm + lay.off_codes + (row + (g & 3)) * kD
                                              : msm + lay.off_zero;
                q.b[0] = *reinterpret_cast<const uint4 *>(codes + 16 * c);
                q.b[1] = *reinterpret_cast<const uint4 *>(codes + 64 + 16 * c);
                const float4 s = *reinterpret_cast<const float4 *>(msm + lay.off_qs +
                                                                   (uint32_t)(row + c) * 16u);
                q.qs[0][0] = s.x, q.qs[0][1] = s.y, q.qs[1][0] = s.z, q.qs[1][1] = s.w;
                const float2 l = *reinterpret_cast<const float2 *>(
                    msm + lay.off_lse + (uint32_t)(row + 2 * (c & 1)) * 4u);
                q.lse2[0] = l.x, q.lse2[1] = l.y;
                return q;
            };
            MassQuad held[NQ > 0 ? NQ : 1];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
                held[n] = quad(n);

            // ---- the tiles
            uint32_t get = 0;
#pragma unroll 1
            for (; t < tok1; t += step) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kMassStages - 2) : "memory");
                const uint4 x0 = lds128(mine16 + get), x1 = lds128(mine16 + get + 512);
                const uint4 y0 = lds128(mine16 + get + 1024), y1 = lds128(mine16 + get + 1536);
                const float ksl = lds_f32(mine4 + get) * p.scale_log2;
                const float before = old ? lds_f32(mine4 + get + 128) : 0.f;
                get = get == (kMassStages - 1) * kMassStageBytes ? 0 : get + kMassStageBytes;
                fetch(); // into the tile consumed last
                if (!((usable >> (kMassStages - 1)) & 1u))
                    continue;
                const bool full = t + kMassTile <= all_see; // every row sees all its tokens
                const int tok = t + g + 8 * sel;
                // the sum of the two rows' weights of this lane in quad n
                auto weights = [&](const MassQuad &q, int n) {
                    float s[2][2]; // [token half][row]
                    int d[4];
                    mma_s8_16832_biased(d, x0.x, y0.x, x0.y, y0.y, q.b[0].x, q.b[0].y);
                    mma_s8_16832_acc(d, x0.z, y0.z, x0.w, y0.w, q.b[0].z, q.b[0].w, d);
                    int f[4];
                    mma_s8_16832_biased(f, x1.x, y1.x, x1.y, y1.y, q.b[1].x, q.b[1].y);
                    mma_s8_16832_acc(f, x1.z, y1.z, x1.w, y1.w, q.b[1].z, q.b[1].w, f);
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 2; ++e) // the biased views minus the bias: exact
                            s[u][e] = fmaf(__int_as_float(f[2 * u + e]) - kDotBiasF, q.qs[1][e],
                                           (__int_as_float(d[2 * u + e]) - kDotBiasF) *
                                               q.qs[0][e]);
                    // blocks 0, 2 lie in lanes c < 2 and blocks 1, 3 in lanes c >= 2 (of the
                    // same rows): each lane gives the token it does not keep
                    float a[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float give = sel ? s[0][e] : s[1][e];
                        const float keep = sel ? s[1][e] : s[0][e];
                        const float x = keep + __shfl_xor_sync(kFullMask, give, 2);
                        a[e] = fast_exp2(fmaf(x, ksl, -q.lse2[e]));
                    }
                    if (!full) {
                        const int2 v = *reinterpret_cast<const int2 *>(
                            msm + lay.off_view + (uint32_t)(4 * n + 2 * (c & 1)) * 4u);
                        a[0] = tok < all_see + v.x ? a[0] : 0.f;
                        a[1] = tok < all_see + v.y ? a[1] : 0.f;
                    }
                    return a[0] + a[1];
                };
                float w = 0.f;
                if constexpr (NQ > 0) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        w += weights(held[n], n);
                } else {
#pragma unroll 1
                    for (int n = 0; n < p.quads; ++n)
                        w += weights(quad(n), n);
                }
                w += __shfl_xor_sync(kFullMask, w, 1);
                if (writer && (full || tok < L))
                    mass[t] = old ? fmaf(p.decay, before, w) : w;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        t0 = t2;
    }
}

} // namespace q8kv
