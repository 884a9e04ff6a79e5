// q8kv_evict.cuh -- eviction from the q8 cache by accumulated attention weight: per (sequence,
// KV head) keep a fixed number of tokens and move their rows, in order, to new blocks.
//
// What it computes, per sequence of L tokens and KV head: with L <= keep every token stays;
// otherwise the first `sink` tokens, the last `recent` ones and, of those between, the
// keep - sink - recent of largest mass (a NaN counts as the lowest value; equal masses go to
// the lowest position). Kept tokens stay in order: the j-th becomes token j of the sequence's
// new block table. Heads choose independently: attention is a sum over tokens, so head h's
// token j and head h + 1's need not come from the same position.
//
// evict_select_kernel finds the set. The threshold (the last mass that stays) comes from
// a radix selection over the order-preserving 32-bit key of the mass: three histograms (11, 11
// and 10 bits) instead of a sort; then one pass marks the positions above the threshold and those
// equal to it (two bits each), and one writes the former and the first of the latter. A block
// takes a (sequence, head), or a cluster of up to 8 when there are few of them or their keys
// do not fit one block's shared memory: the masses are read once, counted in the first
// histogram as they arrive and kept as keys, and the blocks' histograms are added up through
// distributed shared memory. Its time is issue slots and latency (barriers, dependent steps),
// so loads go 16 at a time and blocks are as large as they get. The first histogram, which
// counts every token, has several copies, so that equal digits of neighbouring tokens do not
// serialise on one counter; the others count the few tokens of one digit.
//
// evict_move_kernel copies. A warp takes 32 rows: each lane looks up one row's place (position,
// two table entries) and moves its scales, then the warp moves the rows, D / 16 lanes of 16 bytes
// a row, the places passed on by shuffles. Heads run fastest, so the rows written are contiguous
// for a whole token. It is bound by HBM: 2 (2 D + 8) bytes per kept row. Old and new blocks do
// not overlap, so the order of the copies does not matter.
#pragma once

#include <cooperative_groups.h>

#include <cstdint>

#include "q8kv_ptx.cuh"

namespace q8kv {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
static_assert(kEvictWarps == 32, "one lane per warp in the block-wide scans");
constexpr int kEvictCluster = 8;
constexpr int kEvictBins = 2048;
constexpr int kEvictCopies = 4; // histogram copies per block
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = kMoveThreads; // rows per block: one place per lane

struct EvictParams {
    const float *mass;      // [B][Hk][cap]
    const int32_t *table, *lens, *new_table;
    float *new_mass;        // [B][Hk][new_cap]
    int32_t *kept;          // [B][Hk][keep]
    int32_t *new_lens;      // [B]
    int8_t *k, *v;
    float *ks, *vs;
    int B, Hk, D, bs, mbps, new_mbps, num_blocks, keep, sink, recent;
    int cap, new_cap;       // tokens per row of mass and of new_mass
    int in_smem;            // a block's keys fit its shared memory
    unsigned *errors;
};

// Order-preserving key: larger masses have larger keys, -0 equals +0, NaN equals -inf.
__device__ __forceinline__ uint32_t mass_key(float x)
{
    if (!(x == x))
        x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictShared {
    uint32_t copies[kEvictCopies][kEvictBins]; // first counts; then the rows' marks
    uint32_t hist[2][kEvictBins]; // this block's counts, read by the cluster
    uint32_t warp_sum[kEvictWarps];
    uint32_t digit, rest;         // chosen digit; tokens still wanted within it
    uint32_t gt[kEvictWarps], eq[kEvictWarps];
    uint32_t total_gt, total_eq;  // this block's counts, read by the cluster
};

__device__ __forceinline__ void cluster_barrier(cooperative_groups::cluster_group &cluster, int cs)
{
    if (cs == 1)
        __syncthreads();
    else
        cluster.sync();
}

// Digit of the wanted-th largest key among the counted ones: the bin where the running count
// from the top reaches `wanted`. Every block of the cluster computes it from all histograms.
__device__ __forceinline__ void pick_digit(cooperative_groups::cluster_group &cluster,
                                           EvictShared &sh, int buf, int bins, uint32_t wanted,
                                           int tid)
{
    const int lane = tid & 31, warp = tid >> 5;
    const int cs = (int)cluster.num_blocks();
    constexpr int kPer = kEvictBins / kEvictThreads;
    uint32_t n[kPer];
    uint32_t sum = 0;
    // thread t: bins bins - 1 - kPer t - i, i = 0 .. kPer - 1
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        n[i] = 0;
    const int top = bins - 1 - kPer * tid;
    if (top >= 0) {
        if (cs == 1) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                n[i] = sh.hist[buf][top - i];
        } else {
            uint32_t v[kEvictCluster][kPer]; // all blocks' counts in flight at once
#pragma unroll
            for (int r = 0; r < kEvictCluster; ++r) {
                const uint32_t *h = cluster.map_shared_rank(&sh.hist[buf][0], r < cs ? r : 0);
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    v[r][i] = r < cs ? h[top - i] : 0;
            }
#pragma unroll
            for (int r = 0; r < kEvictCluster; ++r)
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    n[i] += v[r][i];
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        sum += n[i];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += t;
    }
    if (lane == 31)
        sh.warp_sum[warp] = incl;
    __syncthreads();
    // (one value per warp and lane: the warps' sums are added by one more warp scan)
    uint32_t ws = sh.warp_sum[lane];
    const uint32_t own = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, ws, o);
        if (lane >= o)
            ws += t;
    }
    uint32_t run = incl - sum + __shfl_sync(0xffffffffu, ws - own, warp);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (run < wanted && wanted <= run + n[i]) {
            sh.digit = (uint32_t)(top - i);
            sh.rest = wanted - run;
        }
        run += n[i];
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kEvictThreads)
    evict_select_kernel(const __grid_constant__ EvictParams p)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) uint8_t esm[];
    EvictShared &sh = *reinterpret_cast<EvictShared *>(esm);
    uint32_t *keys = reinterpret_cast<uint32_t *>(esm + sizeof(EvictShared));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int pair = blockIdx.x / cs;
    const int b = pair / p.Hk, h = pair - b * p.Hk;
    // the masses come from the kernel before this one on the stream
    grid_dep_wait();
    grid_dep_launch();
    int L = __ldg(p.lens + b);
    if (L < 0 || L > p.cap) {
        if (tid == 0)
            atomicOr(p.errors, 0x1u); // seq_len clamped
        L = L < 0 ? 0 : p.cap;
    }
    const float *mass = p.mass + (long long)pair * p.cap;
    float *new_mass = p.new_mass + (long long)pair * p.new_cap;
    int32_t *kept = p.kept + (long long)pair * p.keep;
    const int n_new = L < p.keep ? L : p.keep;
    const int stride = cs * kEvictThreads, first = rank * kEvictThreads + tid;
    if (h == 0 && rank == 0 && tid == 0)
        p.new_lens[b] = n_new;
    for (int j = n_new + first; j < p.new_cap; j += stride)
        new_mass[j] = 0.f;
    for (int j = n_new + first; j < p.keep; j += stride)
        kept[j] = -1;
    if (L <= p.keep) { // everything stays (all blocks of the cluster)
        for (int j = first; j < L; j += stride) {
            kept[j] = j;
            new_mass[j] = mass[j];
        }
        return;
    }

    // this block's positions [lo, hi); the chosen ones come from [mid0, mid1)
    const int per = ((L + cs - 1) / cs + 31) & ~31;
    const int lo = rank * per < L ? rank * per : L;
    const int hi = lo + per < L ? lo + per : L;
    const int n = hi - lo;
    // [a, z): the block's part of them, counted from lo
    const int a = min(max(p.sink - lo, 0), n), z = max(min(L - p.recent - lo, n), a);
    uint32_t wanted = (uint32_t)(p.keep - p.sink - p.recent);
    const float *src = mass + lo; // position lo + i at src[i]
    auto key_at = [&](int i) { return p.in_smem ? keys[i] : mass_key(__ldg(src + i)); };

    // ---- keys, and their first digits
#pragma unroll
    for (int i = 0; i < kEvictCopies * kEvictBins / 4 / kEvictThreads; ++i)
        reinterpret_cast<uint4 *>(&sh.copies[0][0])[i * kEvictThreads + tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    {
        constexpr int kBatch = 16;
        uint32_t *mine = sh.copies[lane % kEvictCopies];
#pragma unroll 1
        for (int i0 = tid; i0 < n; i0 += kBatch * kEvictThreads) {
            float v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u * kEvictThreads;
                v[u] = i < n ? __ldg(src + i) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u * kEvictThreads;
                const uint32_t key = mass_key(v[u]);
                if (p.in_smem && i < n)
                    keys[i] = key;
                if (i >= a && i < z)
                    atomicAdd(mine + (key >> 21), 1u);
            }
        }
    }
    __syncthreads();

    // ---- threshold key T, and how many tokens equal to it stay
    uint32_t T = 0xffffffffu, ties = 0;
    if (wanted > 0) { // (the same for every block)
#pragma unroll
        for (int i = tid; i < kEvictBins; i += kEvictThreads) {
            uint32_t s = 0;
#pragma unroll
            for (int c = 0; c < kEvictCopies; ++c)
                s += sh.copies[c][i];
            sh.hist[0][i] = s;
            sh.hist[1][i] = 0; // (for the second digit)
        }
        cluster_barrier(cluster, cs);
        pick_digit(cluster, sh, 0, 2048, wanted, tid);
        uint32_t prefix = sh.digit;
        wanted = sh.rest;
#pragma unroll 4
        for (int i = a + tid; i < z; i += kEvictThreads) {
            const uint32_t key = key_at(i);
            if ((key >> 21) == prefix)
                atomicAdd(&sh.hist[1][(key >> 10) & 2047u], 1u);
        }
        // (every block has passed the barrier below once the third counts begin, so the first
        // ones, whose place they take, are read no more: cleared after it)
        cluster_barrier(cluster, cs);
        pick_digit(cluster, sh, 1, 2048, wanted, tid);
        prefix = (prefix << 11) | sh.digit;
        wanted = sh.rest;
        if (tid < 1024)
            sh.hist[0][tid] = 0;
        __syncthreads();
#pragma unroll 4
        for (int i = a + tid; i < z; i += kEvictThreads) {
            const uint32_t key = key_at(i);
            if ((key >> 10) == prefix)
                atomicAdd(&sh.hist[0][key & 1023u], 1u);
        }
        cluster_barrier(cluster, cs);
        pick_digit(cluster, sh, 0, 1024, wanted, tid);
        T = (prefix << 10) | sh.digit;
        ties = sh.rest;
    }

    // ---- mark: warp w takes a contiguous run of rows of 32 positions; the marks of a row are two
    // words in the histogram copies' place (kEvictCopies * kEvictBins / 2 rows at most, else
    // worked out again)
    const int rows = (n + 31) >> 5;
    const bool marked = rows <= kEvictCopies * kEvictBins / 2;
    uint2 *marks = reinterpret_cast<uint2 *>(&sh.copies[0][0]);
    const int r0 = rows * warp / kEvictWarps, r1 = rows * (warp + 1) / kEvictWarps;
    auto mark = [&](int r) {
        const int i = r * 32 + lane;
        const bool in = i < n, held = in && (i < a || i >= z);
        const uint32_t key = in ? key_at(i) : 0u;
        const bool gt = held || (in && key > T);
        const bool eq = in && !held && ties > 0 && key == T;
        return make_uint2(__ballot_sync(0xffffffffu, gt), __ballot_sync(0xffffffffu, eq));
    };
    uint32_t ngt = 0, neq = 0;
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
        const uint2 m = mark(r);
        if (marked && lane == 0)
            marks[r] = m;
        ngt += __popc(m.x);
        neq += __popc(m.y);
    }
    if (lane == 0) {
        sh.gt[warp] = ngt;
        sh.eq[warp] = neq;
    }
    __syncthreads();
    // counts of the warps before this one, and of the block
    uint32_t wg = sh.gt[lane], we = sh.eq[lane];
    const uint32_t og = wg, oe = we;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, wg, o);
        const uint32_t y = __shfl_up_sync(0xffffffffu, we, o);
        if (lane >= o) {
            wg += x;
            we += y;
        }
    }
    if (tid == 31) {
        sh.total_gt = wg;
        sh.total_eq = we;
    }
    uint32_t gt_before = __shfl_sync(0xffffffffu, wg - og, warp);
    uint32_t eq_before = __shfl_sync(0xffffffffu, we - oe, warp);
    if (cs > 1) {
        cluster.sync();
        uint32_t tg[kEvictCluster], te[kEvictCluster];
#pragma unroll
        for (int r = 0; r < kEvictCluster; ++r) {
            tg[r] = te[r] = 0;
            if (r < rank) {
                tg[r] = *cluster.map_shared_rank(&sh.total_gt, r);
                te[r] = *cluster.map_shared_rank(&sh.total_eq, r);
            }
        }
#pragma unroll
        for (int r = 0; r < kEvictCluster; ++r) {
            gt_before += tg[r];
            eq_before += te[r];
        }
    }
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
        const uint2 m = marked ? marks[r] : mark(r);
        const uint32_t e = eq_before + __popc(m.y & below);
        const bool take = (m.x >> lane & 1u) || ((m.y >> lane & 1u) && e < ties);
        if (take) {
            const uint32_t pos = gt_before + __popc(m.x & below) + (e < ties ? e : ties);
            kept[pos] = lo + r * 32 + lane;
            new_mass[pos] = __ldg(src + r * 32 + lane);
        }
        gt_before += __popc(m.x);
        eq_before += __popc(m.y);
    }
    if (cs > 1)
        cluster.sync(); // no block leaves while its counts are read
}

// Rows of sequence blockIdx.y: row r is kept token r / Hk of head r % Hk. Quotients by the
// head count and the block size are taken once per row.
template <int D>
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const __grid_constant__ EvictParams p)
{
    constexpr int kLanes = D / 16;          // lanes per row
    constexpr int kAtOnce = 32 / kLanes;    // rows a warp moves per instruction
    constexpr int kBatch = kLanes < 4 ? kLanes : 4; // such steps in flight
    grid_dep_wait();
    grid_dep_launch();
    const int b = blockIdx.y;
    const int lane = threadIdx.x & 31, sub = lane % kLanes, grp = lane / kLanes;
    const unsigned rows = (unsigned)(p.keep * p.Hk); // < 2^30 (host check)
    const unsigned r = blockIdx.x * kMoveRows + threadIdx.x;
    long long src = -1, dst = 0; // this lane's row (slot * Hk + head); src < 0: none
    if (r < rows) {
        const unsigned j = r / (unsigned)p.Hk, h = r - j * (unsigned)p.Hk;
        const int t = __ldcg(p.kept + ((long long)b * p.Hk + h) * p.keep + j);
        if (t >= 0) {
            const unsigned tb = (unsigned)t / (unsigned)p.bs, jb = j / (unsigned)p.bs;
            const int from = __ldg(p.table + (long long)b * p.mbps + tb);
            const int to = __ldg(p.new_table + (long long)b * p.new_mbps + jb);
            if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks) {
                atomicOr(p.errors, 0x2u); // block-table entry outside the pool: skipped
            } else {
                src = ((long long)from * p.bs + ((unsigned)t - tb * p.bs)) * p.Hk + h;
                dst = ((long long)to * p.bs + (j - jb * p.bs)) * p.Hk + h;
                if (src == dst)
                    src = -1; // in place already
            }
        }
    }
    float ks = 0.f, vs = 0.f;
    if (src >= 0) {
        ks = p.ks[src];
        vs = p.vs[src];
    }
#pragma unroll 1
    for (int i0 = 0; i0 < kLanes; i0 += kBatch) {
        uint4 k[kBatch], v[kBatch];
        long long d[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int from = (i0 + i) * kAtOnce + grp;
            const long long s = __shfl_sync(0xffffffffu, src, from);
            d[i] = __shfl_sync(0xffffffffu, dst, from);
            if (s < 0) {
                d[i] = -1;
            } else {
                k[i] = __ldcs(reinterpret_cast<const uint4 *>(p.k + s * D) + sub);
                v[i] = __ldcs(reinterpret_cast<const uint4 *>(p.v + s * D) + sub);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (d[i] >= 0) {
                *(reinterpret_cast<uint4 *>(p.k + d[i] * D) + sub) = k[i];
                *(reinterpret_cast<uint4 *>(p.v + d[i] * D) + sub) = v[i];
            }
    }
    if (src >= 0) {
        p.ks[dst] = ks;
        p.vs[dst] = vs;
    }
}

} // namespace q8kv
