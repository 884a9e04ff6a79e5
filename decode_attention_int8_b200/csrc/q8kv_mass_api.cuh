// q8kv_mass_api.cuh -- host side of q8kv_attn_mass (include/q8kv.h): argument checks and the
// launch of attn_mass_kernel. Included at the end of q8kv_api.cu, whose device bookkeeping
// it uses.
#pragma once

#include "q8kv_mass.cuh"

namespace {

using namespace q8kv;

bool g_mass_attr[kMaxDevices][3];

template <int MODE>
q8kv_status launch_mass(const MassParams &p, DeviceInfo *dev, int warps, cudaStream_t stream)
{
    bool &set = g_mass_attr[dev - g_dev][MODE];
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        if (!set) {
            Q8KV_CUDA(cudaFuncSetAttribute(attn_mass_kernel<MODE>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           dev->smem_optin - 1024));
            set = true;
        }
    }
    const uint32_t smem = mass_layout(warps, p.heads_pass, p.rows, p.B).total;
    // as many blocks as one wave holds: 3 per SM (24 warps), fewer with many query rows or
    // sequences
    long long wave = (long long)(dev->smem_optin / (smem + 1024));
    wave = (wave < 1 ? 1 : (wave > 3 ? 3 : wave)) * dev->sms;
    const long long tiles = (long long)p.B * ((p.cap + kMassTile - 1) / kMassTile);
    const long long shares = wave / p.passes > 1 ? wave / p.passes : 1; // of the tokens
    return launch_pdl(attn_mass_kernel<MODE>, p,
                      (unsigned)((tiles < shares ? tiles : shares) * p.passes),
                      (unsigned)warps * 32u, smem, stream);
}

} // namespace

extern "C" {

q8kv_status q8kv_attn_mass(float *mass, const float *q, const float *lse, const int8_t *k_blocks,
                           const float *kscale, const int32_t *block_table,
                           const int32_t *seq_lens, int B, int n_queries, int n_q_heads,
                           int n_kv_heads, int head_dim, int kv_block_size,
                           int max_blocks_per_seq, int num_kv_blocks, float scale, float decay,
                           cudaStream_t stream)
{
    if (!mass || !q || !lse || !k_blocks || !kscale || !block_table || !seq_lens)
        return Q8KV_ERR_INVALID_ARG;
    if (B <= 0 || n_queries <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 ||
        head_dim % 32 != 0 || kv_block_size <= 0 || max_blocks_per_seq <= 0 ||
        num_kv_blocks <= 0 || n_q_heads % n_kv_heads != 0 || !std::isfinite(scale) ||
        !(decay >= 0.f && decay <= 1.f))
        return Q8KV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_blocks) ||
        ((reinterpret_cast<uintptr_t>(mass) | reinterpret_cast<uintptr_t>(lse) |
          reinterpret_cast<uintptr_t>(kscale) | reinterpret_cast<uintptr_t>(block_table) |
          reinterpret_cast<uintptr_t>(seq_lens)) & 3u) != 0)
        return Q8KV_ERR_INVALID_ARG;
    const long long R = (long long)n_queries * (n_q_heads / n_kv_heads);
    if (head_dim != kD || !is_pow2(kv_block_size) || kv_block_size < 16 || kv_block_size > 256 ||
        R > kMassMaxRows || B > kMassMaxBatch || n_kv_heads > 4096 ||
        (long long)num_kv_blocks * kv_block_size >= (1LL << 31) ||
        (long long)max_blocks_per_seq * kv_block_size >= (1LL << 30) ||
        (long long)B * max_blocks_per_seq * (kv_block_size / 16) >= (1LL << 30))
        return Q8KV_ERR_UNSUPPORTED;
    DeviceInfo *dev = nullptr;
    q8kv_status st;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        st = device_info(&dev);
    }
    if (st != Q8KV_OK)
        return st;
    MassParams p;
    p.mass = mass;
    p.q = q;
    p.lse = lse;
    p.k = k_blocks;
    p.ks = kscale;
    p.table = block_table;
    p.lens = seq_lens;
    p.B = B;
    p.nq = n_queries;
    p.Hq = n_q_heads;
    p.Hk = n_kv_heads;
    p.Gq = n_q_heads / n_kv_heads;
    p.R = (int)R;
    p.bs_log2 = ilog2(kv_block_size);
    p.mbps = max_blocks_per_seq;
    p.num_blocks = num_kv_blocks;
    p.cap = max_blocks_per_seq * kv_block_size;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.decay = decay;
    p.errors = dev->errors;
    // Up to 8 warps: a few heads' worth, the tokens split over the warps left; other blocks take
    // the other heads of the same tokens. A block quantises its heads' query rows at the start
    // of every sequence, so with many rows, or few tokens, fewer heads (us with 8 / 4 / 2 / 1):
    //   16 x 4096, 8 heads of 4 rows      17.3 / 16.9 / 17.4 / 17.7    256 x 100: 12.6 / 12.6 / 14.5 / 19.1
    //   16 x 500, 8 heads of 8 rows        7.9 /  7.3 /  6.8 /  7.6    1 x 256:    4.8 /  3.9 /  3.6 /  3.5
    //   24 x 8192, 8 heads of 32 rows     82.6 / 74.4 / 73.9 / 71.0    2 x 2388:  17.8 / 11.7 /  8.6 /  7.6
    // With more than 8 rows one head is not best everywhere: 512 x 100 of 32 rows takes 65.6 us with
    // one and 58.3 with four, 24 ragged sequences of up to 8192 tokens 47.6 and 51.8.
    p.rows = p.R <= 4 ? 4 : (p.R + 7) & ~7;
    const long long warp_tiles = (long long)B * (p.cap / kMassTile) * n_kv_heads;
    const int most = p.rows > 8 ? 1 : (warp_tiles <= 2LL * 3 * kMassMaxWarps * dev->sms ? 2 : 4);
    const int passes = (n_kv_heads + most - 1) / most;
    p.heads_pass = (n_kv_heads + passes - 1) / passes;
    p.passes = (n_kv_heads + p.heads_pass - 1) / p.heads_pass;
    p.subs = kMassMaxWarps / p.heads_pass;
    const int warps = p.heads_pass * p.subs;
    if (p.R <= 4)
        return launch_mass<kMassQuad>(p, dev, warps, stream);
    if (p.R <= 8)
        return launch_mass<kMassOct>(p, dev, warps, stream);
    return launch_mass<kMassOcts>(p, dev, warps, stream);
}

} // extern "C"
