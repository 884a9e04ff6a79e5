// q8kv_evict_api.cuh -- host side of q8kv_evict (include/q8kv.h): argument checks and the
// launches of evict_select_kernel and evict_move_kernel. Included at the end of q8kv_api.cu,
// whose device bookkeeping it uses.
#pragma once

#include "q8kv_evict.cuh"

namespace {

using namespace q8kv;

bool g_evict_attr[kMaxDevices];
int g_evict_clusters[kMaxDevices][4]; // clusters of 1 << i blocks, one block per SM, in one wave

// Sets the kernels' attributes and counts the clusters that run at once (the SMs that share a
// scheduler's cluster space need not be a multiple of the cluster's size).
q8kv_status evict_setup(DeviceInfo *dev, int d)
{
    Q8KV_CUDA(cudaFuncSetAttribute(evict_select_kernel<true>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, dev->smem_optin));
    Q8KV_CUDA(cudaFuncSetAttribute(evict_select_kernel<false>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, dev->smem_optin));
    for (int i = 0; (1 << i) <= kEvictCluster; ++i) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << i;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1u << i);
        cfg.blockDim = dim3(kEvictThreads);
        cfg.dynamicSmemBytes = (size_t)dev->smem_optin;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        Q8KV_CUDA(cudaOccupancyMaxActiveClusters(&g_evict_clusters[d][i],
                                                 evict_select_kernel<true>, &cfg));
    }
    g_evict_attr[d] = true;
    return Q8KV_OK;
}

template <int D>
q8kv_status launch_move(const EvictParams &p, cudaStream_t stream)
{
    constexpr int per_block = kMoveRows;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)p.keep * p.Hk + per_block - 1) / per_block),
                       (unsigned)p.B);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    Q8KV_CUDA(cudaLaunchKernelEx(&cfg, evict_move_kernel<D>, p));
    return Q8KV_OK;
}

} // namespace

extern "C" {

q8kv_status q8kv_evict(int8_t *k_blocks, int8_t *v_blocks, float *kscale, float *vscale,
                       float *new_mass, int32_t *kept, int32_t *new_lens, const float *mass,
                       const int32_t *block_table, const int32_t *seq_lens,
                       const int32_t *new_block_table, int B, int n_kv_heads, int head_dim,
                       int kv_block_size, int max_blocks_per_seq, int new_max_blocks_per_seq,
                       int num_kv_blocks, int keep, int sink, int recent, cudaStream_t stream)
{
    if (!k_blocks || !v_blocks || !kscale || !vscale || !new_mass || !kept || !new_lens || !mass ||
        !block_table || !seq_lens || !new_block_table)
        return Q8KV_ERR_INVALID_ARG;
    if (B <= 0 || n_kv_heads <= 0 || head_dim <= 0 || head_dim % 32 != 0 || kv_block_size <= 0 ||
        max_blocks_per_seq <= 0 || new_max_blocks_per_seq <= 0 || num_kv_blocks <= 0 ||
        keep <= 0 || sink < 0 || recent < 0 || (long long)sink + recent > keep ||
        keep > (long long)new_max_blocks_per_seq * kv_block_size)
        return Q8KV_ERR_INVALID_ARG;
    if (!aligned16(k_blocks) || !aligned16(v_blocks) || new_lens == seq_lens ||
        static_cast<const float *>(new_mass) == mass)
        return Q8KV_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(kscale) | reinterpret_cast<uintptr_t>(vscale) |
          reinterpret_cast<uintptr_t>(new_mass) | reinterpret_cast<uintptr_t>(kept) |
          reinterpret_cast<uintptr_t>(new_lens) | reinterpret_cast<uintptr_t>(mass) |
          reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
          reinterpret_cast<uintptr_t>(new_block_table)) & 3u) != 0)
        return Q8KV_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || B > 16384 ||
        (long long)max_blocks_per_seq * kv_block_size >= (1LL << 30) ||
        (long long)new_max_blocks_per_seq * kv_block_size >= (1LL << 30) ||
        (long long)num_kv_blocks * kv_block_size >= (1LL << 31) ||
        (long long)keep * n_kv_heads >= (1LL << 30) ||
        (long long)B * n_kv_heads * kEvictCluster >= (1LL << 31))
        return Q8KV_ERR_UNSUPPORTED;
    DeviceInfo *dev = nullptr;
    q8kv_status st;
    EvictParams p;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        st = device_info(&dev);
        if (st != Q8KV_OK)
            return st;
        const int d = (int)(dev - g_dev);
        if (!g_evict_attr[d]) {
            st = evict_setup(dev, d);
            if (st != Q8KV_OK)
                return st;
        }
    }
    p.mass = mass;
    p.table = block_table;
    p.lens = seq_lens;
    p.new_table = new_block_table;
    p.new_mass = new_mass;
    p.kept = kept;
    p.new_lens = new_lens;
    p.k = k_blocks;
    p.v = v_blocks;
    p.ks = kscale;
    p.vs = vscale;
    p.B = B;
    p.Hk = n_kv_heads;
    p.D = head_dim;
    p.bs = kv_block_size;
    p.mbps = max_blocks_per_seq;
    p.new_mbps = new_max_blocks_per_seq;
    p.num_blocks = num_kv_blocks;
    p.keep = keep;
    p.sink = sink;
    p.recent = recent;
    p.cap = max_blocks_per_seq * kv_block_size;
    p.new_cap = new_max_blocks_per_seq * kv_block_size;
    p.errors = dev->errors;
    // Blocks per (sequence, head): one for up to 16 masses per thread, more for longer rows
    // while all clusters run at once, a block per SM (18 rows of 140000 masses: clusters of 4,
    // 49.5 us with the move; of 8 they take two rounds, 63.2 us. 14 rows: 8, 37.7 us. Rows of
    // 16384 in 32 pairs: one block each 28.8 us, clusters of 2 32.3 us, whose barriers cost more
    // than the shares save).
    const long long pairs = (long long)B * n_kv_heads;
    const int *at_once = g_evict_clusters[dev - g_dev];
    int cs = 1;
    for (int i = 1; cs < kEvictCluster && pairs <= at_once[i] && p.cap > 16 * kEvictThreads * cs; ++i)
        cs *= 2;
    // and as many as it takes for a block's masses to fit its shared memory
    auto part = [&](int n) { return ((size_t)((p.cap + n - 1) / n + 31) & ~(size_t)31) * 4; };
    const size_t room = (size_t)dev->smem_optin - sizeof(EvictShared);
    while (cs < kEvictCluster && part(cs) > room)
        cs *= 2;
    const bool in_smem = part(cs) <= room;
    const size_t smem = sizeof(EvictShared) + (in_smem ? part(cs) : 0);
    st = launch_cluster(in_smem ? evict_select_kernel<true> : evict_select_kernel<false>, p,
                        (unsigned)pairs, cs, kEvictThreads, smem, stream);
    if (st != Q8KV_OK)
        return st;
    if (head_dim == 64)
        return launch_move<64>(p, stream);
    if (head_dim == 128)
        return launch_move<128>(p, stream);
    return launch_move<256>(p, stream);
}

} // extern "C"
