// q8kv_mass.cuh -- accumulated attention weights of the cached tokens, the quantity an eviction
// policy ranks them by.
//
// What it computes, per sequence b, KV head kv and token t < L_b:
//   mass[b][kv][t] = decay * mass[b][kv][t] + sum over the head's query rows r of
//                    exp(s_rt - lse_r),
// with the decode's own scores s (int8 query blocks, exact block dots, q8kv_decode.cuh) and
// the log-sum-exp of each row that the decode left: one pass over K, no softmax to redo.
//
// What bounds it: HBM, at 132 bytes of K and 8 of mass per (token, KV head), so K goes straight
// from global memory into the registers of the MMA that needs it and nothing is staged. A warp
// takes 16 tokens of one head at a time: tokens are the M rows of mma.m16n8k32.s8, four query
// rows its N columns twice over. A lane loads 16 consecutive bytes of a token's row; with
// those as the MMA's k positions, lanes c = 0, 1 hold block 2h of the row (h: which half) and
// lanes c = 2, 3 block 2h + 1, and the query operand is zero where column group n / 4 and block
// differ. One accumulator so carries two blocks' exact dots side by side, every column is
// used, and two shuffles bring the halves together, each lane keeping two rows of one token.
// Two register sets alternate, so the next 16 tokens' rows, scale and mass are in flight while
// one set is used, and the first ones while the query is quantised. The tokens of all
// sequences form one list that the blocks share evenly; a block's warps take different heads of
// the same tokens, whose rows are neighbours in the pool.
#pragma once

#include <cstdint>

#include "q8kv_decode.cuh"

namespace q8kv {

constexpr int kMassMaxWarps = 8;
constexpr int kMassTile = 16;      // tokens per warp step
constexpr int kMassMaxBatch = 16384;

struct MassParams {
    float *mass;       // [B][Hk][cap]
    const float *q;    // [B][nq][Hq][128]
    const float *lse;  // [B][nq][Hq]
    const int8_t *k;
    const float *ks;
    const int32_t *table, *lens;
    int B, nq, Hq, Hk, Gq, R; // Gq: query heads per KV head; R = nq Gq rows per KV head
    int bs_log2, mbps, num_blocks, cap;
    int heads_pass;    // heads the block's warps cover at once
    int subs;          // warps that share a head's tokens
    float scale_log2, decay;
    unsigned *errors;
};

// The query operand of four rows: codes in the lane order described above, the scales and
// log-sum-exp (base 2) of the two rows whose scores this lane keeps.
struct MassQuad {
    uint32_t b[2][4];  // [half][words of the lane's 16 bytes]
    float qs[2][2];    // [half][row]: scale of the lane's block
    float lse2[2];
};

__device__ __forceinline__ MassQuad mass_query(const MassParams &p, int b, int kv, int row0, int g,
                                               int c)
{
    MassQuad f;
    const int r = row0 + (g & 3); // column g of the operand
    const bool mine = (c >> 1) == (g >> 2) && r < p.R;
    float qsc[2];
    const float *row = p.q;
    if (mine) {
        const int i = r / p.Gq;
        row += (((long long)b * p.nq + i) * p.Hq + (long long)kv * p.Gq + (r - i * p.Gq)) * kD;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v[16];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float4 x = mine ? __ldg(reinterpret_cast<const float4 *>(row + 64 * h + 16 * c) + w)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            v[4 * w] = x.x;
            v[4 * w + 1] = x.y;
            v[4 * w + 2] = x.z;
            v[4 * w + 3] = x.w;
        }
        float qm = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k)
            qm = fmaxf(qm, fabsf(v[k]));
        qm = fmaxf(qm, __shfl_xor_sync(kFullMask, qm, 1)); // lanes c, c ^ 1: one 32-block
        if (qm < 1e-6f)
            qm = 1.0f;
        qsc[h] = mine ? __fmul_rn(qm, 1.0f / 127.0f) : 0.f;
        const float iq = __fdiv_rn(127.0f, qm);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t word = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                int x = __float2int_rn(__fmul_rn(v[4 * w + k], iq));
                x = max(-127, min(127, x));
                word |= (uint32_t)(x & 0xff) << (8 * k);
            }
            f.b[h][w] = word;
        }
    }
    // accumulator columns 2c, 2c + 1: rows 2 (c & 1) and the next, block pair member c >> 1
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int from = (2 * c + e) * 4 + 2 * (c >> 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            f.qs[h][e] = __shfl_sync(kFullMask, qsc[h], from);
        const int rr = row0 + 2 * (c & 1) + e;
        f.lse2[e] = INFINITY; // a padding row weighs nothing: exp2(0 - inf)
        if (rr < p.R) {
            const int i = rr / p.Gq;
            f.lse2[e] = __ldg(p.lse + ((long long)b * p.nq + i) * p.Hq + (long long)kv * p.Gq +
                              (rr - i * p.Gq)) * 1.44269504088896341f;
        }
    }
    return f;
}

// One step's operands: rows of tokens g and g + 8 of the tile, the scale and the old mass of
// the token this lane keeps.
struct MassTile {
    uint4 k[2][2]; // [token half][row half]
    float ks, old;
    bool ok;
};

template <int NQ>
__global__ void __launch_bounds__(kMassMaxWarps * 32, NQ == 4 ? 2 : 3)
    attn_mass_kernel(const __grid_constant__ MassParams p)
{
    extern __shared__ int prefix[]; // [B + 1]: tiles before each sequence
    __shared__ int wsum[kMassMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nwarps = blockDim.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    // the query, its statistics and the cache come from kernels before this one
    grid_dep_wait();
    grid_dep_launch();

    // ---- tiles of every sequence, as prefix sums
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
        const int tok1 = (t2 - first) * kMassTile;
#pragma unroll 1
        for (int kv = hw; kv < p.Hk; kv += p.heads_pass) {
            float *mass = p.mass + ((long long)b * p.Hk + kv) * p.cap + g + 8 * sel;
            const int8_t *kbase = p.k + ((long long)g * p.Hk + kv) * kD + 16 * c;
            const float *sbase = p.ks + (long long)(g + 8 * sel) * p.Hk + kv;
#pragma unroll 1
            for (int row0 = 0; row0 < p.R; row0 += 4 * NQ) {
                const float decay = row0 == 0 ? p.decay : 1.f;
                const int step = p.subs * kMassTile;
                int t = (t0 - first + sub) * kMassTile; // first token of the tile

                auto load = [&](MassTile &m, int t) {
                    const int blk = __ldg(table + (t >> p.bs_log2));
                    m.ok = (unsigned)blk < (unsigned)p.num_blocks;
                    if (!m.ok && lane == 0)
                        atomicOr(p.errors, kErrBlockTable);
                    const int slot = ((m.ok ? blk : 0) << p.bs_log2) + (t & bs_mask);
                    const long long row = (long long)slot * p.Hk; // (slot, head 0)
                    const int8_t *k = kbase + row * kD;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            m.k[u][h] =
                                __ldcs(reinterpret_cast<const uint4 *>(k + u * row8 + 64 * h));
                    m.ks = __ldg(sbase + row);
                    m.old = 0.f;
                    if (decay != 0.f && writer && t + g + 8 * sel < L)
                        m.old = mass[t];
                };
                MassTile A, B;
                if (t < tok1)
                    load(A, t);
                MassQuad q[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                    q[n] = mass_query(p, b, kv, row0 + 4 * n, g, c);

                auto use = [&](const MassTile &m, int t) {
                    const float ksl = m.ks * p.scale_log2;
                    const int tok = t + g + 8 * sel;
                    float w = 0.f;
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        float s[2][2]; // [token half][row]
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            int d[4];
                            const uint4 x = m.k[0][h], y = m.k[1][h];
                            mma_s8_16832_biased(d, x.x, y.x, x.y, y.y, q[n].b[h][0], q[n].b[h][1]);
                            mma_s8_16832_acc(d, x.z, y.z, x.w, y.w, q[n].b[h][2], q[n].b[h][3], d);
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    // the biased view minus the bias: exact
                                    const float v = __int_as_float(d[2 * u + e]) - kDotBiasF;
                                    s[u][e] = h == 0 ? v * q[n].qs[0][e]
                                                     : fmaf(v, q[n].qs[1][e], s[u][e]);
                                }
                        }
                        // blocks 0, 2 lie in lanes c < 2 and blocks 1, 3 in lanes c >= 2 (of
                        // the same rows): each lane gives the token it does not keep
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float give = sel ? s[0][e] : s[1][e];
                            const float keep = sel ? s[1][e] : s[0][e];
                            const float x = keep + __shfl_xor_sync(kFullMask, give, 2);
                            const float a = fast_exp2(fmaf(x, ksl, -q[n].lse2[e]));
                            if (t + kMassTile <= all_see) {
                                w += a;
                            } else { // row r sees the tokens below L - (nq - 1 - r / Gq)
                                const int r = row0 + 4 * n + 2 * (c & 1) + e;
                                w += tok < all_see + r / p.Gq ? a : 0.f;
                            }
                        }
                    }
                    w += __shfl_xor_sync(kFullMask, w, 1);
                    if (writer && tok < L && m.ok)
                        mass[t] = decay == 0.f ? w : fmaf(decay, m.old, w);
                };
                while (t < tok1) {
                    int tn = t + step;
                    if (tn < tok1)
                        load(B, tn);
                    use(A, t);
                    t = tn;
                    if (t >= tok1)
                        break;
                    tn = t + step;
                    if (tn < tok1)
                        load(A, tn);
                    use(B, t);
                    t = tn;
                }
            }
        }
        t0 = t2;
    }
}

} // namespace q8kv
