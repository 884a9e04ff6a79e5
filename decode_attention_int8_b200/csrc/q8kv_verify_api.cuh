// q8kv_verify_api.cuh -- host side of q8kv_verify_draft (include/q8kv.h): argument checks and
// the launch of verify_kernel. Included at the end of q8kv_api.cu, whose device bookkeeping
// it uses.
#pragma once

#include "q8kv_verify.cuh"

namespace {

using namespace q8kv;

static_assert(kErrProbs == Q8KV_DEVERR_PROBS, "device error bits differ from the header");

// A launch of clusters of `cs` blocks (portable sizes), programmatic dependent launch.
template <typename Params>
q8kv_status launch_cluster(void (*fn)(Params), const Params &p, unsigned clusters, int cs,
                           unsigned threads, size_t smem, cudaStream_t stream)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * (unsigned)cs);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    Q8KV_CUDA(cudaLaunchKernelEx(&cfg, fn, p));
    return Q8KV_OK;
}

template <typename T>
q8kv_status launch_verify(const VerifyParams &p, int B, int sms, cudaStream_t stream)
{
    // the widest load that every row's start allows: 16 bytes, two elements (an even vocabulary),
    // or one
    constexpr int kVec = 16 / (int)sizeof(T);
    auto starts = [&](int n) {
        const uintptr_t bytes = (uintptr_t)n * sizeof(T);
        return (reinterpret_cast<uintptr_t>(p.target) % bytes) == 0 && p.target_stride % n == 0 &&
               (!p.draft || ((reinterpret_cast<uintptr_t>(p.draft) % bytes) == 0 &&
                             p.draft_stride % n == 0));
    };
    // Blocks per sequence: the fewest "waves times time of a block", where a wave holds 4 blocks
    // per SM and a block takes its share of the row plus the time of about 8192 weights (start,
    // accept test, exchange, search). Measured, fp32, 5 drafts, with 1 / 2 / 4 / 8 blocks: 128 rows
    // of 131075 57 / 36 / 29 / 32 us; 600 of them (a wave of 592 and one of 8, with one block
    // each) 129 / 111 / 108 / 120; 32 rows 50 / 29 / - / 13; 600 rows of 32000 42 / 39 / - / 68.
    const long long slots = 4LL * sms;
    int cs = 1;
    long long best = 0;
    for (int c = 1; c <= kVerifyCluster; c *= 2) {
        const long long cost = ((long long)B * c + slots - 1) / slots * (8192 + p.vocab / c);
        if (c == 1 || cost <= best) {
            best = cost;
            cs = c;
        }
    }
    if (starts(kVec))
        return launch_cluster(verify_kernel<T, kVec>, p, (unsigned)B, cs, kVerifyThreads, 0, stream);
    if (starts(2))
        return launch_cluster(verify_kernel<T, 2>, p, (unsigned)B, cs, kVerifyThreads, 0, stream);
    return launch_cluster(verify_kernel<T, 1>, p, (unsigned)B, cs, kVerifyThreads, 0, stream);
}

} // namespace

extern "C" {

q8kv_status q8kv_verify_draft(int32_t *n_accepted, int32_t *tokens, const void *target_probs,
                              const void *draft_probs, const int32_t *draft_tokens,
                              const int32_t *n_drafts, const float *uniforms, int B,
                              int max_drafts, int vocab, long long target_stride,
                              long long draft_stride, q8kv_dtype dtype, cudaStream_t stream)
{
    if (B < 0 || max_drafts < 0 || vocab <= 0)
        return Q8KV_ERR_INVALID_ARG;
    if (dtype != Q8KV_F32 && dtype != Q8KV_F16 && dtype != Q8KV_BF16)
        return Q8KV_ERR_INVALID_ARG;
    if (target_stride == 0)
        target_stride = vocab;
    if (draft_stride == 0)
        draft_stride = vocab;
    if (target_stride < vocab || draft_stride < vocab)
        return Q8KV_ERR_INVALID_ARG;
    const uintptr_t size = dtype == Q8KV_F32 ? 4 : 2;
    if (max_drafts > 1024 || B > (1 << 24) || vocab > (1 << 30))
        return Q8KV_ERR_UNSUPPORTED;
    if (B == 0)
        return Q8KV_OK;
    if (!n_accepted || !tokens || !target_probs || !uniforms || (max_drafts > 0 && !draft_tokens))
        return Q8KV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(target_probs) % size) != 0 ||
        (reinterpret_cast<uintptr_t>(draft_probs) % size) != 0 ||
        ((reinterpret_cast<uintptr_t>(n_accepted) | reinterpret_cast<uintptr_t>(tokens) |
          reinterpret_cast<uintptr_t>(draft_tokens) | reinterpret_cast<uintptr_t>(n_drafts) |
          reinterpret_cast<uintptr_t>(uniforms)) & 3u) != 0)
        return Q8KV_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    q8kv_status st;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        st = device_info(&dev);
    }
    if (st != Q8KV_OK)
        return st;
    VerifyParams p;
    p.accepted = n_accepted;
    p.tokens = tokens;
    p.target = target_probs;
    p.draft = draft_probs;
    p.drafted = draft_tokens;
    p.n_drafts = n_drafts;
    p.uniforms = uniforms;
    p.target_stride = target_stride;
    p.draft_stride = draft_stride;
    p.max_drafts = max_drafts;
    p.vocab = vocab;
    p.errors = dev->errors;
    if (dtype == Q8KV_F32)
        return launch_verify<float>(p, B, dev->sms, stream);
    if (dtype == Q8KV_F16)
        return launch_verify<__half>(p, B, dev->sms, stream);
    return launch_verify<__nv_bfloat16>(p, B, dev->sms, stream);
}

} // extern "C"
