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
// and 10 bits) instead of a sort; then one pass counts the positions above the threshold and
// those equal to it, and one writes the former and the first of the latter. A block takes a
// (sequence, head), or a cluster of up to 8 when there are few of them or their keys do not
// fit one block's shared memory: the masses are read once, counted in the first histogram
// as they arrive and kept as keys, and the blocks' histograms are added up through distributed
// shared memory. What bounds it is issue slots (a few dozen instructions a position) and, for
// short sequences, barriers: so a thread takes four neighbouring positions at a time, and counts
// stay per lane until the end of a pass. The first histogram, which counts every token, has
// several copies, so that equal digits of neighbouring tokens do not serialise on one counter;
// the others count the few tokens of one digit. (16 x 8 heads of 16384 positions: 15 us; 22.3 us
// with one position per lane, ballots and three passes over copied histograms.)
//
// evict_move_kernel copies. A warp takes 32 rows: each lane looks up one row's place (position,
// two table entries) and moves its scales, then the warp moves the rows, D / 16 lanes of 16 bytes
// a row, the places passed on by shuffles. Heads run fastest, so the rows written are contiguous
// for a whole token. It is bound by HBM: 2 (2 D + 8) bytes per kept row (4096 rows of 16 x 8 heads:
// 47 us, 5.9 TB/s). Old and new blocks do not overlap, so the order of the copies does not
// matter.
#pragma once

#include <cooperative_groups.h>

#include <cstdint>

#include "q8kv_ptx.cuh"

namespace q8kv {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
static_assert(kEvictWarps <= 32 && kEvictThreads >= 256, "one lane per warp in the block-wide sums");
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
    uint32_t copies[kEvictCopies][kEvictBins];
    uint32_t hist[2][kEvictBins]; // this block's counts, read by the cluster
    uint32_t warp_sum[8];
    uint32_t slice[kEvictCluster]; // totals of the blocks' slices of the bins
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
// from the top reaches `wanted`. One block: 256 threads, 8 bins each, the highest bins first.
__device__ __forceinline__ void pick_digit(EvictShared &sh, int buf, int bins, uint32_t wanted,
                                           int tid)
{
    constexpr int kPer = 8, kThreads = kEvictBins / kPer, kWarps = kThreads / 32;
    const int lane = tid & 31, warp = tid >> 5;
    uint32_t n[kPer]; // n[i]: bin low + i
    uint32_t sum = 0, incl = 0;
    const int low = bins - kPer * (tid + 1);
    if (tid < kThreads) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            n[i] = 0;
        if (low >= 0) {
            const uint4 x = *reinterpret_cast<const uint4 *>(sh.hist[buf] + low);
            const uint4 y = *reinterpret_cast<const uint4 *>(sh.hist[buf] + low + 4);
            n[0] = x.x, n[1] = x.y, n[2] = x.z, n[3] = x.w;
            n[4] = y.x, n[5] = y.y, n[6] = y.z, n[7] = y.w;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            sum += n[i];
        incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += t;
        }
        if (lane == 31)
            sh.warp_sum[warp] = incl;
    }
    __syncthreads();
    if (tid < kThreads) {
        uint32_t run = incl - sum;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            run += w < warp ? sh.warp_sum[w] : 0;
        if (run < wanted && wanted <= run + sum) {
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i) {
                if (run < wanted && wanted <= run + n[i]) {
                    sh.digit = (uint32_t)(low + i);
                    sh.rest = wanted - run;
                }
                run += n[i];
            }
        }
    }
    __syncthreads();
}

// The same over a cluster: each block adds up its slice of the bins over all blocks' histograms
// (reading them whole in every block moved 64 KB per block and digit through distributed shared
// memory: 6.7 us a digit with 8 blocks), the blocks tell each other their slices' totals, and
// the one that holds the digit tells the others. The caller's barrier after the counts and the
// two here order every remote access.
__device__ __forceinline__ void pick_digit_cluster(cooperative_groups::cluster_group &cluster,
                                                   EvictShared &sh, int buf, int bins,
                                                   uint32_t wanted, int tid, int cs, int rank)
{
    const int lane = tid & 31, warp = tid >> 5;
    const int width = bins / cs; // <= kEvictThreads: two blocks at least
    // thread t: bin (rank + 1) * width - 1 - t, so running counts go downwards
    uint32_t n = 0;
    const int bin = (rank + 1) * width - 1 - tid;
    if (tid < width) {
        uint32_t v[kEvictCluster];
#pragma unroll
        for (int r = 0; r < kEvictCluster; ++r)
            v[r] = r < cs ? cluster.map_shared_rank(&sh.hist[buf][0], r)[bin] : 0u;
#pragma unroll
        for (int r = 0; r < kEvictCluster; ++r)
            n += v[r];
    }
    uint32_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += t;
    }
    if (lane == 31)
        sh.gt[warp] = incl;
    __syncthreads();
    const uint32_t w = lane < kEvictWarps ? sh.gt[lane] : 0u;
    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u);
    const uint32_t total = __reduce_add_sync(0xffffffffu, w);
    if (tid < cs)
        *cluster.map_shared_rank(&sh.slice[rank], tid) = total;
    cluster.sync();
    uint32_t run = before + incl - n;
#pragma unroll
    for (int r = 0; r < kEvictCluster; ++r)
        run += r > rank && r < cs ? sh.slice[r] : 0u;
    if (tid < width && run < wanted && wanted <= run + n) {
        for (int r = 0; r < cs; ++r) {
            *cluster.map_shared_rank(&sh.digit, r) = (uint32_t)bin;
            *cluster.map_shared_rank(&sh.rest, r) = wanted - run;
        }
    }
    cluster.sync();
}

// SMEM: the block's keys stay in shared memory; otherwise they are made again from the masses.
template <bool SMEM>
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

    // this block's positions [lo, lo + n); the chosen ones are among [a, z), counted from lo
    const int per = ((L + cs - 1) / cs + 31) & ~31;
    const int lo = rank * per < L ? rank * per : L;
    const int n = (lo + per < L ? lo + per : L) - lo;
    const int a = min(max(p.sink - lo, 0), n), z = max(min(L - p.recent - lo, n), a);
    uint32_t wanted = (uint32_t)(p.keep - p.sink - p.recent);
    const float *src = mass + lo; // position lo + i at src[i]
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15u) == 0; // 16-byte loads
    // masses of positions i .. i + 3 (i a multiple of 4); past the last one: NaN
    auto mass4 = [&](int i) {
        if (vec && i + 4 <= n)
            return __ldg(reinterpret_cast<const float4 *>(src + i));
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x[u] = i + u < n ? __ldg(src + i + u) : __int_as_float(0x7fc00000);
        return make_float4(x[0], x[1], x[2], x[3]);
    };
    auto load4 = [&](int i) {
        const float4 x = mass4(i);
        return make_uint4(mass_key(x.x), mass_key(x.y), mass_key(x.z), mass_key(x.w));
    };
    auto keys4 = [&](int i) {
        if constexpr (SMEM)
            return *reinterpret_cast<const uint4 *>(keys + i);
        else
            return load4(i);
    };

    // ---- keys, and their first digits
#pragma unroll
    for (int i = 0; i < kEvictCopies * kEvictBins / 4 / kEvictThreads; ++i)
        reinterpret_cast<uint4 *>(&sh.copies[0][0])[i * kEvictThreads + tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    {
        uint32_t *mine = sh.copies[lane % kEvictCopies];
        constexpr int kBatch = 4; // 16 loads in flight
#pragma unroll 1
        for (int i0 = 4 * tid; i0 < n; i0 += 4 * kBatch * kEvictThreads) {
            float4 v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                v[u] = mass4(i0 + 4 * u * kEvictThreads);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + 4 * u * kEvictThreads;
                if (i >= n)
                    break;
                const uint32_t x[4] = {mass_key(v[u].x), mass_key(v[u].y), mass_key(v[u].z),
                                       mass_key(v[u].w)};
                if constexpr (SMEM)
                    *reinterpret_cast<uint4 *>(keys + i) = make_uint4(x[0], x[1], x[2], x[3]);
                if (i >= a && i + 4 <= z) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        atomicAdd(mine + (x[e] >> 21), 1u);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i + e >= a && i + e < z)
                            atomicAdd(mine + (x[e] >> 21), 1u);
                }
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
        // counts of the keys whose bits from `above` up are `prefix`, by their bits from `shift`
        auto count = [&](uint32_t *hist, uint32_t prefix, int above, int shift) {
            const uint32_t from = prefix << above, width = 1u << above;
#pragma unroll 4
            for (int i = 4 * tid; i < z; i += 4 * kEvictThreads) {
                const uint4 k = keys4(i);
                const uint32_t x[4] = {k.x - from, k.y - from, k.z - from, k.w - from};
                if (min(min(x[0], x[1]), min(x[2], x[3])) < width) { // (few: one digit's keys)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (x[e] < width && i + e >= a && i + e < z)
                            atomicAdd(hist + (x[e] >> shift), 1u);
                }
            }
        };
        auto pick = [&](int buf, int bins) {
            if (cs == 1)
                pick_digit(sh, buf, bins, wanted, tid);
            else
                pick_digit_cluster(cluster, sh, buf, bins, wanted, tid, cs, rank);
        };
        cluster_barrier(cluster, cs);
        pick(0, 2048);
        uint32_t prefix = sh.digit;
        wanted = sh.rest;
        count(sh.hist[1], prefix, 21, 10);
        // (every block is past its reads of the first counts, whose place the third ones take,
        // once it has come to this barrier: they are cleared after it)
        cluster_barrier(cluster, cs);
        pick(1, 2048);
        prefix = (prefix << 11) | sh.digit;
        wanted = sh.rest;
        for (int i = tid; i < 1024; i += kEvictThreads)
            sh.hist[0][i] = 0;
        __syncthreads();
        count(sh.hist[0], prefix, 10, 0);
        cluster_barrier(cluster, cs);
        pick(0, 1024);
        T = (prefix << 10) | sh.digit;
        ties = sh.rest;
    }

    // ---- count, then write: warp w takes a contiguous run of chunks of 128 positions, a lane
    // four neighbours of each. Bits 0-3 of a mark: above the threshold (or held); bits 4-7:
    // equal to it.
    auto mark = [&](int i) {
        uint32_t m = 0;
        if (i < n) {
            const uint4 k = keys4(i);
            const uint32_t x[4] = {k.x, k.y, k.z, k.w};
            if (i >= a && i + 4 <= z) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    m |= (x[e] > T ? 1u << e : 0u) | (x[e] == T ? 16u << e : 0u);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i + e < n) {
                        if (i + e < a || i + e >= z)
                            m |= 1u << e;
                        else
                            m |= (x[e] > T ? 1u << e : 0u) | (x[e] == T ? 16u << e : 0u);
                    }
            }
        }
        return m;
    };
    const int chunks = (n + 127) >> 7;
    const int c0 = chunks * warp / kEvictWarps, c1 = chunks * (warp + 1) / kEvictWarps;
    uint32_t ngt = 0, neq = 0;
#pragma unroll 2
    for (int c = c0; c < c1; ++c) {
        const uint32_t m = mark(c * 128 + 4 * lane);
        ngt += __popc(m & 15u);
        neq += __popc(m >> 4);
    }
    ngt = __reduce_add_sync(0xffffffffu, ngt);
    neq = __reduce_add_sync(0xffffffffu, neq);
    if (lane == 0) {
        sh.gt[warp] = ngt;
        sh.eq[warp] = neq;
    }
    __syncthreads();
    // counts of the warps before this one, and of the block
    const uint32_t wg = lane < kEvictWarps ? sh.gt[lane] : 0u;
    const uint32_t we = lane < kEvictWarps ? sh.eq[lane] : 0u;
    uint32_t gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0u);
    uint32_t eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0u);
    if (cs > 1) {
        if (warp == kEvictWarps - 1 && lane == 0) {
            sh.total_gt = gt_before + ngt;
            sh.total_eq = eq_before + neq;
        }
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
#pragma unroll 2
    for (int c = c0; c < c1; ++c) {
        const int i = c * 128 + 4 * lane;
        const uint32_t m = mark(i);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (m) // (the masses themselves: a key has lost NaN and the sign of zero)
            x = mass4(i);
        // counts of the lanes before this one: above in the low half, equal in the high one
        const uint32_t own = __popc(m & 15u) | (__popc(m >> 4) << 16);
        uint32_t incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += t;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
        const uint32_t e = eq_before + ((incl - own) >> 16);
        uint32_t pos = gt_before + ((incl - own) & 0xffffu) + min(e, ties);
        // of those equal to the threshold, the first `ties` stay
        uint32_t take = m & 15u, eq = m >> 4;
        for (uint32_t k = e; eq && k < ties; ++k) {
            take |= eq & (0u - eq);
            eq &= eq - 1u;
        }
        const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if ((take >> u) & 1u) {
                kept[pos] = lo + i + u;
                new_mass[pos] = v[u];
                ++pos;
            }
        gt_before += all & 0xffffu;
        eq_before += all >> 16;
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
