// q8kv_rope_api.cuh -- host side of q8kv_rope_cache_write (include/q8kv.h): argument checks
// and the launch of rope_cache_write_kernel. Included at the end of q8kv_api.cu, whose
// device bookkeeping it uses.
#pragma once

#include "q8kv_rope.cuh"

namespace {

using namespace q8kv;

static_assert(kErrPosition == Q8KV_DEVERR_POSITION, "device error bits differ from the header");

// A launch of the rotary write or the attention mass: programmatic dependent launch.
template <typename Params>
q8kv_status launch_pdl(void (*fn)(Params), const Params &p, unsigned grid, unsigned threads,
                       size_t smem, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    Q8KV_CUDA(cudaLaunchKernelEx(&cfg, fn, p));
    return Q8KV_OK;
}

template <int D, typename T>
q8kv_status launch_rope(RopeParams &p, int mode, int sms, cudaStream_t stream)
{
    // Tokens per block step: the tile of 1 to 4 whose rounds over the wave of resident blocks take
    // least, a round costing its tokens and about a third of one (4999 bf16 tokens: 3, not 4
    // with a third round for 66 of 1250 tiles). A tile that leaves SMs empty is shared by
    // several blocks, of at least one row group per warp.
    const int iters = rope_iters(p.Hq, p.Hk, D);
    const long long wave = (long long)rope_blocks<T>(mode) * sms;
    p.tile = 1;
    long long least = 0;
    for (int t = 1; t <= kRopeTile; ++t) {
        const long long rounds = ((p.n_tokens + t - 1) / t + wave - 1) / wave;
        const long long cost = rounds * (3 * t + 1);
        if (t == 1 || cost <= least) {
            least = cost;
            p.tile = t;
        }
    }
    if (p.n_tokens <= wave)
        p.tile = 1;
    const long long tiles = (p.n_tokens + p.tile - 1) / p.tile;
    const long long most = (iters * p.tile + kWriteWarps - 1) / kWriteWarps;
    const long long parts = (wave + tiles - 1) / tiles;
    p.parts = (int)(parts < most ? parts : most);
    const long long blocks = tiles * p.parts;
    const unsigned grid = (unsigned)(blocks < wave ? blocks : wave);
    if (mode == kRopeFull)
        return launch_pdl(rope_cache_write_kernel<D, T, kRopeFull>, p, grid, kWriteThreads, 0,
                          stream);
    if (mode == kRopeHalf)
        return launch_pdl(rope_cache_write_kernel<D, T, kRopeHalf>, p, grid, kWriteThreads, 0,
                          stream);
    if (mode == kRopeAnywhere)
        return launch_pdl(rope_cache_write_kernel<D, T, kRopeAnywhere>, p, grid, kWriteThreads, 0,
                          stream);
    return launch_pdl(rope_cache_write_kernel<D, T, kRopeAdjacent>, p, grid, kWriteThreads, 0,
                      stream);
}

template <typename T>
q8kv_status launch_rope(RopeParams &p, int D, int mode, int sms, cudaStream_t stream)
{
    if (D == 64)
        return launch_rope<64, T>(p, mode, sms, stream);
    if (D == 128)
        return launch_rope<128, T>(p, mode, sms, stream);
    return launch_rope<256, T>(p, mode, sms, stream);
}

} // namespace

extern "C" {

q8kv_status q8kv_rope_cache_write(float *q_out, int8_t *k_blocks, int8_t *v_blocks,
                                  float *kscale, float *vscale, const void *q_new,
                                  const void *k_new, const void *v_new,
                                  const int64_t *slot_mapping, const int32_t *positions,
                                  const float *cos_sin, const uint8_t *pair_axis, int n_tokens,
                                  int n_axes, int n_q_heads, int n_kv_heads, int head_dim,
                                  int rotary_dim, int adjacent, int max_position,
                                  q8kv_dtype dtype, int kv_block_size, int num_kv_blocks,
                                  long long q_token_stride, long long kv_token_stride,
                                  cudaStream_t stream)
{
    if (!k_blocks || !v_blocks || !kscale || !vscale)
        return Q8KV_ERR_INVALID_ARG;
    if (n_tokens < 0 || n_axes <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 ||
        head_dim % 32 != 0 || rotary_dim <= 0 || rotary_dim > head_dim || rotary_dim % 8 != 0 ||
        max_position <= 0 || kv_block_size <= 0 || num_kv_blocks <= 0)
        return Q8KV_ERR_INVALID_ARG;
    if (dtype != Q8KV_F32 && dtype != Q8KV_F16 && dtype != Q8KV_BF16)
        return Q8KV_ERR_INVALID_ARG;
    const int per16 = dtype == Q8KV_F32 ? 4 : 8; // elements in 16 bytes
    const long long q_row = (long long)n_q_heads * head_dim;
    const long long kv_row = (long long)n_kv_heads * head_dim;
    if (q_token_stride == 0)
        q_token_stride = q_row;
    if (kv_token_stride == 0)
        kv_token_stride = kv_row;
    if (q_token_stride < q_row || q_token_stride % per16 != 0 || kv_token_stride < kv_row ||
        kv_token_stride % per16 != 0)
        return Q8KV_ERR_INVALID_ARG;
    if (!aligned16(k_blocks) || !aligned16(v_blocks) ||
        (reinterpret_cast<uintptr_t>(kscale) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(vscale) & 3u) != 0)
        return Q8KV_ERR_INVALID_ARG;
    if (pair_axis)
        for (int i = 0; i < rotary_dim / 2 && i < 128; ++i)
            if (pair_axis[i] >= n_axes)
                return Q8KV_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || n_axes > kRopeAxes ||
        n_q_heads > 4096 || n_kv_heads > 4096)
        return Q8KV_ERR_UNSUPPORTED;
    if (n_tokens == 0) // nothing to do (the row pointers may be null)
        return Q8KV_OK;
    if (!q_out || !q_new || !k_new || !v_new || !slot_mapping || !positions || !cos_sin ||
        !aligned16(q_out) || !aligned16(q_new) || !aligned16(k_new) || !aligned16(v_new) ||
        !aligned16(cos_sin) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0 ||
        (reinterpret_cast<uintptr_t>(positions) & 3u) != 0)
        return Q8KV_ERR_INVALID_ARG;
    // in place: the fp32 rows at exactly the rows they came from
    if (static_cast<const void *>(q_out) == q_new &&
        (dtype != Q8KV_F32 || q_token_stride != q_row))
        return Q8KV_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    q8kv_status st;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        st = device_info(&dev);
    }
    if (st != Q8KV_OK)
        return st;
    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    p.q_out = q_out;
    p.k = k_blocks;
    p.v = v_blocks;
    p.ks = kscale;
    p.vs = vscale;
    p.q_new = q_new;
    p.k_new = k_new;
    p.v_new = v_new;
    p.slots = slot_mapping;
    p.pos = positions;
    p.table = cos_sin;
    p.n_tokens = n_tokens;
    p.q_stride = q_token_stride;
    p.kv_stride = kv_token_stride;
    p.n_slots = (long long)num_kv_blocks * kv_block_size;
    p.Hq = n_q_heads;
    p.Hk = n_kv_heads;
    p.rot = rotary_dim;
    p.max_pos = max_position;
    p.n_axes = n_axes;
    p.errors = dev->errors;
    if (pair_axis)
        std::memcpy(p.axis, pair_axis, (size_t)rotary_dim / 2);
    const int mode = adjacent                     ? kRopeAdjacent
                     : rotary_dim == head_dim     ? kRopeFull
                     : 2 * rotary_dim == head_dim ? kRopeHalf
                                                  : kRopeAnywhere;
    if (dtype == Q8KV_F32)
        return launch_rope<float>(p, head_dim, mode, dev->sms, stream);
    if (dtype == Q8KV_F16)
        return launch_rope<__half>(p, head_dim, mode, dev->sms, stream);
    return launch_rope<__nv_bfloat16>(p, head_dim, mode, dev->sms, stream);
}

} // extern "C"
