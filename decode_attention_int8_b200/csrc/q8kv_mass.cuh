// q8kv_mass.cuh -- accumulated attention weights of the cached tokens, the quantity an eviction
// policy ranks them by.
//
// What it computes, per sequence b, KV head kv and token t < L_b:
//   mass[b][kv][t] = decay * mass[b][kv][t] + sum over the head's query rows r of
//                    exp(s_rt - lse_r),
// with the decode's own scores s (int8 query blocks, exact block dots, q8kv_decode.cuh) and
// the log-sum-exp of each row that the decode left: one pass over K, no softmax to redo.
//
// What bounds it: HBM, at 132 bytes of K and 8 of mass per (token, KV head), then the issue
// slots (48 ragged sequences of up to 16384 tokens, 64 / 8 heads: 73 us in graph replays, 0.85 of
// the copy rate; 16 x 4096, 32 / 8: 17 us, 0.67, the rest its start; calls from a loop on the host
// take up to 5 us more of the former). With more than 8 rows per head the operand is read again for
// every tile and the products and exponentials of the rows bound it (24 x 8192, 32 rows: 71 us,
// 0.48). A warp takes 16 tokens of one head at a
// time as the M rows of mma.m16n8k32.s8, query rows as its N columns:
//  * 5 or more rows per head: eight rows per MMA, one MMA per 32-channel block, K fragments by
//    ldmatrix.
//  * up to 4 rows (they would leave half the columns empty): four rows twice over. A lane takes
//    16 consecutive bytes of a token's row as its k positions, so lanes c = 0, 1 hold block 2h
//    of the row (h: which half) and lanes c = 2, 3 block 2h + 1; the query operand is zero where
//    column group n / 4 and block differ. One accumulator so carries two blocks' exact dots
//    side by side, and two shuffles bring the halves together, each lane keeping one token.
//
// A warp copies its tiles (rows, scales, old masses) ahead of use with cp.async into a ring of
// kMassStages tiles in shared memory that only it reads: the copies in flight cost no registers
// and no block-wide synchronisation. (With the next tile's operands in registers instead, the
// kernel spilled at 24 warps per SM and took 114 us on 48 ragged sequences of up to 16384
// tokens, 64 / 8 heads.) The tokens of all sequences form one list that the blocks share
// evenly, each for a few heads; the heads' rows of a token are neighbours in the pool. The block
// quantises a segment's query rows together, into shared memory, while the first tiles are on
// their way.
#pragma once

#include <cstdint>

#include "q8kv_decode.cuh"

namespace q8kv {

constexpr int kMassMaxWarps = 8;
constexpr int kMassTile = 16;    // tokens per warp step
constexpr int kMassStages = 4;   // tiles in a warp's ring
constexpr int kMassMaxBatch = 16384;
// A block that goes on to another sequence drains its rings, quantises the new query and fills
// them again, in about the time of this many of its tiles; the even split of the list counts
// them at every sequence's start. (48 ragged sequences, 64 / 8 heads: 79.6 us without.)
constexpr int kMassStartTiles = 6;
constexpr int kMassMaxRows = 128; // query rows per KV head
constexpr int kMassStageBytes = kMassTile * (kD + 8); // rows, then scales, then masses
constexpr int kMassLoads = 2;    // query rows of 16 lanes in flight
constexpr int kMassRowBytes = kD + 16; // a query row in shared memory (rows on distinct banks)

struct MassParams {
    float *mass;       // [B][Hk][cap]
    const float *q;    // [B][nq][Hq][128]
    const float *lse;  // [B][nq][Hq]
    const int8_t *k;
    const float *ks;
    const int32_t *table, *lens;
    int B, nq, Hq, Hk, Gq, R; // Gq: query heads per KV head; R = nq Gq rows per KV head
    int rows;          // R rounded up to 4 (one quad) or to a multiple of 8
    int bs_log2, mbps, num_blocks, cap;
    int heads_pass;    // heads of a block
    int passes;        // blocks that share a range of tokens, each with its heads
    int subs;          // warps that share a head's tokens
    float scale_log2, decay;
    unsigned *errors;
};

// Dynamic shared memory: the rings, the segment's query rows, the tile prefixes.
struct MassLayout {
    uint32_t off_codes, off_zero, off_qs, off_lse, off_view, off_prefix, total;
};

__host__ __device__ inline MassLayout mass_layout(int warps, int heads, int rows, int B)
{
    MassLayout l;
    uint32_t o = (uint32_t)(warps * kMassStages * kMassStageBytes);
    l.off_codes = o; // [head][row]
    o += (uint32_t)(heads * rows * kMassRowBytes);
    l.off_zero = o;  // 128 bytes of zeros
    o += kD;
    l.off_qs = o;    // scales in the order the lanes use them: a quad's [c][half][row], a
                     // group of eight's [c][block][row]
    o += (uint32_t)(heads * rows * kNB * 4);
    l.off_lse = o;   // [head][row]: log-sum-exp, base 2 (+inf: no row)
    o += (uint32_t)(heads * rows * 4);
    l.off_view = o;  // [row]: index of the row's query token
    o += (uint32_t)(rows * 4);
    l.off_prefix = o;
    l.total = o + 4u * (uint32_t)(B + 1);
    return l;
}

// Operand of four rows (kMassQuad): the lane's bytes, or zeros; of eight rows: column g's
// words. With the scales of the rows whose dots this lane holds, and their log-sum-exp.
struct MassOperand {
    uint32_t b[8];
    float qs[8]; // (a quad's: the first four)
    float lse2[2];
};

enum MassMode { kMassQuad = 0, kMassOct = 1, kMassOcts = 2 };

__device__ __forceinline__ void mass_cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void mass_cp4(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mass_ldsm_x4(uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3,
                                        uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

// MODE: kMassQuad for up to 4 rows per head, kMassOct for up to 8 (both held in registers),
// kMassOcts for more (read from shared memory per tile).
template <int MODE>
__global__ void __launch_bounds__(kMassMaxWarps * 32, 3)
    attn_mass_kernel(const __grid_constant__ MassParams p)
{
    extern __shared__ __align__(16) uint8_t msm[];
    __shared__ int wsum[kMassMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nwarps = blockDim.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const MassLayout lay = mass_layout(nwarps, p.heads_pass, p.rows, p.B);
    int *prefix = reinterpret_cast<int *>(msm + lay.off_prefix); // units before each sequence
    // the query, its statistics and the cache come from kernels before this one
    grid_dep_wait();
    grid_dep_launch();

    // ---- units of every sequence (its tiles and the charge for its start), as prefix sums; the
    // rows' query indices
    if (tid < kD / 4)
        reinterpret_cast<uint32_t *>(msm + lay.off_zero)[tid] = 0u;
    for (int r = tid; r < p.rows; r += blockDim.x)
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
            n = L > 0 ? (L + kMassTile - 1) / kMassTile + kMassStartTiles : 0;
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
    const int share = blockIdx.x / p.passes, shares = gridDim.x / p.passes;
    const int kv0 = (blockIdx.x - share * p.passes) * p.heads_pass; // this block's first head
    int u0 = (int)((long long)N * share / shares);
    const int u1 = (int)((long long)N * (share + 1) / shares);
    const int hw = warp % p.heads_pass, sub = warp / p.heads_pass;
    const unsigned bs_mask = (1u << p.bs_log2) - 1u;
    const int sel = c >> 1; // which half of the tile's tokens this lane ends up with
    const bool old = p.decay != 0.f;
    const unsigned hkd = (unsigned)p.Hk * kD; // bytes from token to token
    const unsigned long long row8 = 8ull * hkd;
    const unsigned long long kstep = (unsigned long long)(p.subs * kMassTile) * hkd;
    const uint32_t bytes4 = lane < 16 || old ? 4u : 0u; // (0: filled with zeros, nothing read)

    // The warp's ring. Copies: lane (g, c) moves 16-byte chunks c and c + 4 of rows g and g + 8,
    // to chunk positions XORed with the row (ldmatrix then meets every bank once; a lane that
    // reads its own chunks back finds them where it put them); lanes 0-15 move the tokens'
    // scales, lanes 16-31 their masses.
    const uint32_t ring = smem_addr(msm) + (uint32_t)(warp * kMassStages * kMassStageBytes);
    const uint32_t put_row = ring + (uint32_t)(g * kD);
    const uint32_t put0 = put_row + (uint32_t)((c ^ g) * 16), put1 = put_row + (uint32_t)(((c + 4) ^ g) * 16);
    const uint32_t put_s = ring + (uint32_t)(kMassTile * kD + 4 * lane);
    const uint32_t get_s = ring + (uint32_t)(kMassTile * kD + 4 * g);
    // ldmatrix addresses: lanes 0-7 rows 0-7, 8-15 rows 8-15 of a block's first 16 bytes, lanes
    // 16-31 the same of its last 16
    const uint32_t get_m = ring + (uint32_t)((lane & 15) * kD);
    const int get_c = (lane >> 4) ^ (lane & 7); // chunk 2j + lane / 16, XORed with the row

    while (u0 < u1) {
        // the sequence of unit u0: the last b with prefix[b] <= u0
        int b = 0, z = p.B - 1;
        while (b < z) {
            const int m = (b + z + 1) >> 1;
            if (prefix[m] <= u0)
                b = m;
            else
                z = m - 1;
        }
        const int first = prefix[b] + kMassStartTiles, end = prefix[b + 1];
        const int t0 = max(u0 - first, 0), t2 = min(u1, end) - first; // the block's tiles of it
        u0 = min(u1, end);
        if (t0 >= t2)
            continue;
        int L = __ldg(p.lens + b);
        L = L > p.cap ? p.cap : L;
        const int32_t *table = p.table + (long long)b * p.mbps;
        const int all_see = L - (p.nq - 1); // tokens that every row sees
        const int kv = kv0 + hw;
        float *mass_row = p.mass + ((long long)b * p.Hk + kv) * p.cap;
        float *mass = mass_row + g + 8 * sel;
        const int8_t *kbase = p.k + ((long long)g * p.Hk + kv) * kD + 16 * c;
        // this lane's 4-byte copy: a scale (by slot) or a mass (by position)
        const float *base4 = lane < 16 ? p.ks + (long long)lane * p.Hk + kv
                                       : mass_row + (lane - 16);
        const unsigned stride4 = lane < 16 ? (unsigned)p.Hk * 4u : 4u;
        const unsigned step4 = (unsigned)(p.subs * kMassTile) * stride4;
        const int step = p.subs * kMassTile;
        const int tok1 = kv < p.Hk ? t2 * kMassTile : 0;
        int t = (t0 + sub) * kMassTile; // first token of the tile in use
        // Tiles are fetched in order; within one block of the table the addresses only
        // advance, so the table and the products are left to the step into a new one.
        int ti = t;             // first token of the next tile to fetch
        int left = 0;           // tiles of its block still to fetch
        const int8_t *kp = kbase;
        const char *p4 = reinterpret_cast<const char *>(base4);
        unsigned ok = 0;        // the block is in the pool
        uint32_t usable = 0;    // `ok` of the fetched tiles, latest lowest
        int blk = ti < tok1 ? __ldg(table + (ti >> p.bs_log2)) : 0;
        auto fetch = [&](uint32_t put) {
            if (ti < tok1) {
                if (left == 0) {
                    ok = (unsigned)blk < (unsigned)p.num_blocks;
                    const unsigned in = (unsigned)ti & bs_mask;
                    const unsigned slot = ((ok ? (unsigned)blk : 0u) << p.bs_log2) + in;
                    left = (int)((bs_mask - in) / (unsigned)step) + 1;
                    kp = kbase + (unsigned long long)slot * hkd;
                    p4 = reinterpret_cast<const char *>(base4) +
                         (unsigned long long)(lane < 16 ? slot : (unsigned)ti) * stride4;
                    if (!ok && lane == 0)
                        atomicOr(p.errors, kErrBlockTable);
                    const int tn = ti + left * step; // the next block, one block ahead
                    if (tn < tok1)
                        blk = __ldg(table + (tn >> p.bs_log2));
                }
                mass_cp16(put0 + put, kp);
                mass_cp16(put1 + put, kp + 64);
                mass_cp16(put0 + put + 8 * kD, kp + row8);
                mass_cp16(put1 + put + 8 * kD, kp + row8 + 64);
                // (in bounds of the row: a tile never passes the table's last block)
                mass_cp4(put_s + put, p4, bytes4);
                kp += kstep;
                p4 += step4;
                ti += step;
                --left;
            }
            usable = usable * 2u + ok;
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // ---- the segment's query rows, by the whole block: 16 lanes per row, kMassLoads rows
        // of each in flight. The first of them are loaded before the copies wait for the
        // table, and quantised after.
        const int part = lane & 15; // block part / 4, its values 8 (part % 4) ..
        const int all_rows = p.heads_pass * p.rows;
        float vs[kMassLoads][8], ls[kMassLoads];
        auto load_query = [&](int x, float (&v)[8], float &l) {
            const int hd = MODE == kMassQuad ? x >> 2 : (MODE == kMassOct ? x >> 3 : x / p.rows);
            const int r = x - hd * p.rows;
            l = 3.402823466e38f; // no row: +inf in base 2, no weight
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = 0.f;
            if (r < p.R && x < all_rows && kv0 + hd < p.Hk) {
                const int i = reinterpret_cast<const int *>(msm + lay.off_view)[r];
                const long long row = ((long long)b * p.nq + i) * p.Hq +
                                      (long long)(kv0 + hd) * p.Gq + (r - i * p.Gq);
                const float4 *src =
                    reinterpret_cast<const float4 *>(p.q + row * kD + 8 * part);
                const float4 y = __ldg(src), w = __ldg(src + 1);
                v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
                v[4] = w.x, v[5] = w.y, v[6] = w.z, v[7] = w.w;
                l = __ldg(p.lse + row);
            }
        };
        auto load_queries = [&](int x0) {
#pragma unroll
            for (int i = 0; i < kMassLoads; ++i)
                load_query(x0 + 2 * nwarps * i + (lane >> 4), vs[i], ls[i]);
        };
        load_queries(2 * warp);
#pragma unroll
        for (int i = 0; i < kMassStages - 1; ++i)
            fetch(i * kMassStageBytes);
        __syncthreads(); // the last segment's rows have been read
        auto put_query = [&](int x, const float (&v)[8], float l) { // (whole warps)
            const int hd = MODE == kMassQuad ? x >> 2 : (MODE == kMassOct ? x >> 3 : x / p.rows);
            const int r = x - hd * p.rows;
            uint32_t lo, hi;
            float qsc;
            quantize_block_quad(v, lo, hi, qsc);
            // A NaN channel would leave the codes as a zero (the quantiser's maximum and conversion
            // drop it): the row's statistic takes it up instead, and with it every weight. (An
            // infinity is the block's scale, under codes of 0: the scores are NaN by themselves.) A
            // statistic of +inf would weigh nothing, like a row that is not there.
            bool bad = l == INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                bad |= v[i] != v[i];
            const float l2 = __ballot_sync(kFullMask, bad) & (0xffffu << (lane & 16))
                                 ? __int_as_float(0x7fc00000)
                                 : l * 1.44269504088896341f;
            if (x < all_rows) { // (the last step may pass the last row)
                *reinterpret_cast<uint2 *>(msm + lay.off_codes +
                                           (uint32_t)(x * kMassRowBytes + 8 * part)) =
                    make_uint2(lo, hi);
                if ((part & 3) == 0) {
                    float *qs = reinterpret_cast<float *>(msm + lay.off_qs);
                    const int j = part >> 2;
                    if constexpr (MODE == kMassQuad) {
                        // block j = 2h + c / 2 of row 2 (c & 1) + e lies at [c][h][e]
                        const int cc = 2 * (j & 1) + (r >> 1);
                        qs[(hd * 4 + cc) * 4 + (j >> 1) * 2 + (r & 1)] = qsc;
                    } else { // row 2c + e of its eight at [c][j][e]
                        qs[((x >> 3) * 4 + ((r & 7) >> 1)) * 8 + j * 2 + (r & 1)] = qsc;
                    }
                }
                if (part == 0)
                    reinterpret_cast<float *>(msm + lay.off_lse)[x] = l2;
            }
        };
#pragma unroll 1
        for (int x0 = 2 * warp;;) {
#pragma unroll
            for (int i = 0; i < kMassLoads; ++i)
                if (x0 + 2 * nwarps * i < all_rows)
                    put_query(x0 + 2 * nwarps * i + (lane >> 4), vs[i], ls[i]);
            x0 += 2 * nwarps * kMassLoads;
            if (x0 >= all_rows)
                break;
            load_queries(x0);
        }
        __syncthreads();
        auto operand = [&](int n) { // quad, or group n of eight, of this warp's head
            MassOperand q;
            if constexpr (MODE == kMassQuad) {
                const bool in_col = (c >> 1) == (g >> 2);
                const uint8_t *codes =
                    in_col ? msm + lay.off_codes + (hw * 4 + (g & 3)) * kMassRowBytes
                           : msm + lay.off_zero;
                const uint4 x = *reinterpret_cast<const uint4 *>(codes + 16 * c);
                const uint4 y = *reinterpret_cast<const uint4 *>(codes + 64 + 16 * c);
                q.b[0] = x.x, q.b[1] = x.y, q.b[2] = x.z, q.b[3] = x.w;
                q.b[4] = y.x, q.b[5] = y.y, q.b[6] = y.z, q.b[7] = y.w;
                const float4 s = *reinterpret_cast<const float4 *>(
                    msm + lay.off_qs + (uint32_t)(hw * 4 + c) * 16u);
                q.qs[0] = s.x, q.qs[1] = s.y, q.qs[2] = s.z, q.qs[3] = s.w;
                const float2 l = *reinterpret_cast<const float2 *>(
                    msm + lay.off_lse + (uint32_t)(hw * 4 + 2 * (c & 1)) * 4u);
                q.lse2[0] = l.x, q.lse2[1] = l.y;
            } else {
                const int row = hw * p.rows + 8 * n;
                const uint8_t *codes = msm + lay.off_codes + (row + g) * kMassRowBytes + 4 * c;
#pragma unroll
                for (int j = 0; j < kNB; ++j) {
                    q.b[2 * j] = *reinterpret_cast<const uint32_t *>(codes + 32 * j);
                    q.b[2 * j + 1] = *reinterpret_cast<const uint32_t *>(codes + 32 * j + 16);
                }
                const float4 *s = reinterpret_cast<const float4 *>(
                    msm + lay.off_qs + (uint32_t)((row >> 3) * 4 + c) * 32u);
                const float4 s0 = s[0], s1 = s[1];
                q.qs[0] = s0.x, q.qs[1] = s0.y, q.qs[2] = s0.z, q.qs[3] = s0.w;
                q.qs[4] = s1.x, q.qs[5] = s1.y, q.qs[6] = s1.z, q.qs[7] = s1.w;
                const float2 l = *reinterpret_cast<const float2 *>(
                    msm + lay.off_lse + (uint32_t)(row + 2 * c) * 4u);
                q.lse2[0] = l.x, q.lse2[1] = l.y;
            }
            return q;
        };
        MassOperand held;
        if constexpr (MODE != kMassOcts)
            held = operand(0);
        const int *view = reinterpret_cast<const int *>(msm + lay.off_view);

        // ---- the tiles
        uint32_t at = 0, last = (kMassStages - 1) * kMassStageBytes; // this tile, the one before
        float *out = mass + t;
#pragma unroll 1
        for (; t < tok1; t += step) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kMassStages - 2) : "memory");
            __syncwarp(); // (and every lane has read the tile that fetch() overwrites)
            const bool full = t + kMassTile <= all_see; // every row sees all its tokens
            float w;
            const float before = lds_f32(get_s + at + 64 + 32 * sel);
            if constexpr (MODE == kMassQuad) {
                const uint4 x0 = lds128(put0 + at), x1 = lds128(put1 + at);
                const uint4 y0 = lds128(put0 + at + 8 * kD), y1 = lds128(put1 + at + 8 * kD);
                const float ksl = lds_f32(get_s + at + 32 * sel) * p.scale_log2;
                fetch(last);
                int d[4], f[4];
                mma_s8_16832(d, x0.x, y0.x, x0.y, y0.y, held.b[0], held.b[1]);
                mma_s8_16832_acc(d, x0.z, y0.z, x0.w, y0.w, held.b[2], held.b[3], d);
                mma_s8_16832(f, x1.x, y1.x, x1.y, y1.y, held.b[4], held.b[5]);
                mma_s8_16832_acc(f, x1.z, y1.z, x1.w, y1.w, held.b[6], held.b[7], f);
                float s[2][2]; // [token half][row]
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        s[u][e] = fmaf((float)f[2 * u + e], held.qs[2 + e],
                                       (float)d[2 * u + e] * held.qs[e]);
                // blocks 0, 2 lie in lanes c < 2 and blocks 1, 3 in lanes c >= 2 (of the
                // same rows): each lane gives the token it does not keep
                float a[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float give = sel ? s[0][e] : s[1][e];
                    const float keep = sel ? s[1][e] : s[0][e];
                    const float x = keep + __shfl_xor_sync(kFullMask, give, 2);
                    a[e] = fast_exp2(fmaf(x, ksl, -held.lse2[e]));
                }
                if (!full) {
                    const int tok = t + g + 8 * sel;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        a[e] = tok < all_see + view[2 * (c & 1) + e] ? a[e] : 0.f;
                }
                w = a[0] + a[1];
            } else {
                uint32_t k[kNB][4];
#pragma unroll
                for (int j = 0; j < kNB; ++j)
                    mass_ldsm_x4(k[j][0], k[j][1], k[j][2], k[j][3],
                            get_m + at + (uint32_t)((get_c ^ (2 * j)) * 16));
                const float ks0 = lds_f32(get_s + at) * p.scale_log2;
                const float ks1 = lds_f32(get_s + at + 32) * p.scale_log2;
                fetch(last);
                float w0 = 0.f, w1 = 0.f;
                auto group = [&](const MassOperand &q, int n) {
                    float s[4];
#pragma unroll
                    for (int j = 0; j < kNB; ++j) {
                        int d[4];
                        mma_s8_16832(d, k[j][0], k[j][1], k[j][2], k[j][3], q.b[2 * j],
                                     q.b[2 * j + 1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[i] = j == 0 ? (float)d[i] * q.qs[i & 1]
                                          : fmaf((float)d[i], q.qs[2 * j + (i & 1)], s[i]);
                    }
                    float a[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        a[i] = fast_exp2(fmaf(s[i], i < 2 ? ks0 : ks1, -q.lse2[i & 1]));
                    if (!full) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            a[i] = t + g + 8 * (i >> 1) <
                                           all_see + view[8 * n + 2 * c + (i & 1)]
                                       ? a[i]
                                       : 0.f;
                    }
                    w0 += a[0] + a[1];
                    w1 += a[2] + a[3];
                };
                if constexpr (MODE == kMassOct) {
                    group(held, 0);
                } else {
#pragma unroll 1
                    for (int n = 0; n < p.rows >> 3; ++n)
                        group(operand(n), n);
                }
                w = (sel ? w1 : w0) + __shfl_xor_sync(kFullMask, sel ? w0 : w1, 2);
            }
            w += __shfl_xor_sync(kFullMask, w, 1);
            if ((c & 1) == 0 && (full || t + g + 8 * sel < L) &&
                ((usable >> (kMassStages - 1)) & 1u))
                *out = fmaf(p.decay, before, w); // (before is zero without decay)
            out += step;
            last = at;
            at = at == (kMassStages - 1) * kMassStageBytes ? 0 : at + kMassStageBytes;
        }
        // (a lane's own copies are done; the barrier is for the other lanes' reads of the last
        // tiles, whose places the next segment's first copies take)
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    }
}

} // namespace q8kv
