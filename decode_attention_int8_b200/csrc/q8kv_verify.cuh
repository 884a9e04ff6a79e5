// q8kv_verify.cuh -- verification of drafted tokens against the target's probabilities from
// given random numbers (speculative sampling).
//
// What it computes, per sequence with drafts x_0 .. x_(n-1), draft probabilities q_i, target
// probabilities p_i (i = 0 .. n) and uniforms u_i: draft i is accepted while u_i q_i(x_i) <
// p_i(x_i). At the first refusal i the next token is drawn from the residual max(p_i - q_i, 0)
// and, when every draft is accepted, from p_n: the smallest x whose running sum exceeds
// u Z, Z the sum of all weights and u the sequence's last uniform.
//
// Products and sums carry fp64's precision. The answer is a whole number: a sum over 1e5 weights in
// fp32 is off by about 1e-7 of Z, and with that many borders in [0, Z) one draw in a few
// hundred would name a neighbour. With fp64 accumulators, and fp32 steps before them whose rounding
// errors are summed up too, a border moves by less than 1e-13 Z, beside the roundings of the fp64
// sums (2^-53 of the running sum for each of a lane's).
//
// What bounds it: HBM for large batches (one row of p, and one of q after a refusal, read
// once), latency for small ones. A cluster of up to 8 blocks takes a sequence: every block
// repeats the accept test (a gather of 2 n values), then sums its part of the row, each warp
// a contiguous piece; the blocks exchange their sums through distributed shared memory (one
// cluster barrier), and the one warp whose piece holds the border reads that piece again (from
// L2) to find the token. One launch, no workspace. (Timestamps with 128 rows of 131075 fp32
// weights: accept test 1.6 us, sums 19 us, the rate of HBM, waiting for the cluster's slowest
// block 2.5 us, the rest 4 us. Running sums left at 8 places of each piece, which spare the
// second reading, and 8 separate sums per warp were tried: 29.6 and 28.7 us, against 29.4.)
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "q8kv_ptx.cuh"

namespace q8kv {

constexpr unsigned kErrProbs = 0x80u; // a draft token, draft count or row of weights was unusable
constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;

struct VerifyParams {
    int32_t *accepted; // [B]
    int32_t *tokens;   // [B][max_drafts + 1]
    const void *target, *draft;
    const int32_t *drafted, *n_drafts;
    const float *uniforms; // [B][max_drafts + 1]
    long long target_stride, draft_stride; // elements between rows
    int max_drafts, vocab;
    unsigned *errors;
};

__device__ __forceinline__ float as_f32(float x)
{
    return x;
}
__device__ __forceinline__ float as_f32(__half x)
{
    return __half2float(x);
}
__device__ __forceinline__ float as_f32(__nv_bfloat16 x)
{
    return __bfloat162float(x);
}

// VEC consecutive elements by one load: 16 bytes, or as many as the rows' starts allow.
template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Pack {
    T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T *p)
{
    Pack<T, VEC> r;
    static_assert(VEC * sizeof(T) <= 16, "one load");
    if constexpr (VEC == 1)
        r.v[0] = *p;
    else if constexpr (VEC * sizeof(T) == 16)
        *reinterpret_cast<uint4 *>(r.v) = __ldg(reinterpret_cast<const uint4 *>(p));
    else if constexpr (VEC * sizeof(T) == 8)
        *reinterpret_cast<uint2 *>(r.v) = __ldg(reinterpret_cast<const uint2 *>(p));
    else
        *reinterpret_cast<uint32_t *>(r.v) = __ldg(reinterpret_cast<const uint32_t *>(p));
    return r;
}

// The weights a token is drawn from: the target's row, less the draft's (kResidual) or without
// one token (kWithout: a draft without probabilities is certain of its token). What is not
// above zero, NaN among it, weighs nothing.
enum VerifyMode { kPlain = 0, kResidual = 1, kWithout = 2 };

template <int MODE>
__device__ __forceinline__ double weight(float p, float q, int x, int without)
{
    double w = (double)p;
    if constexpr (MODE == kResidual)
        w -= (double)q;
    else if constexpr (MODE == kWithout)
        w = x == without ? 0.0 : w;
    return w > 0.0 ? w : 0.0;
}

__device__ __forceinline__ double warp_sum(double x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ double warp_scan(double x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double t = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += t;
    }
    return x;
}

// A weight as fp32 and what its rounding left out (added to err): p - q with p > q >= 0 is h
// plus (p - h) - q, exactly.
template <int MODE>
__device__ __forceinline__ float weight32(float p, float q, int x, int without, float &err)
{
    if constexpr (MODE == kResidual) {
        const float h = __fsub_rn(p, q), e = __fsub_rn(__fsub_rn(p, h), q);
        const bool on = p > q;
        err += on ? e : 0.f;
        return on ? h : 0.f;
    } else if constexpr (MODE == kWithout) {
        return p > 0.f && x != without ? p : 0.f;
    } else {
        return p > 0.f ? p : 0.f;
    }
}

// Sum of two weights as fp32 and what its rounding left out.
__device__ __forceinline__ float pair_sum(float a, float b, float &err)
{
    const float x = fmaxf(a, b), y = fminf(a, b), s = __fadd_rn(x, y);
    err += __fsub_rn(y, __fsub_rn(s, x));
    return s;
}

// Sum of the weights of tokens [lo, hi), one warp (lo a multiple of VEC). Two weights are added
// up in fp32 first, exactly: their sum goes to the fp64 accumulator, and the rounding errors, at
// most 2^-23 of it, to an fp32 one that is emptied into fp64 every turn. Its own errors are then
// those of 13 sums of at most 2^-23 of the turn's weights each, so below 13 * 2^-47 = 2^-43.3 of the
// total whatever the length. (Kept over the whole row, roundings of one sign put it off by 1e-12
// of the total after 8192 weights of a lane.) That takes little more than half a conversion and half
// an fp64 sum per weight instead of two and two (128 rows of 131072 bf16 weights: 20.6 us, 23.2
// us with fp64 differences; fp32: 25.7, 26.6).
template <typename T, int VEC, int MODE>
__device__ __forceinline__ double piece_sum_mode(const T *pr, const T *qr, int without, int lo,
                                                 int hi, int lane)
{
    // packs of each row in flight per lane
    constexpr int U = VEC <= 2 ? 8 : (VEC == 4 ? 4 : 2);
    constexpr int kStep = 32 * VEC;
    double acc[2] = {0.0, 0.0};
    int e0 = lo + lane * VEC;
#pragma unroll 1
    for (; e0 + (U - 1) * kStep + VEC <= hi; e0 += U * kStep) { // (lanes may differ by one turn)
        Pack<T, VEC> a[U], b[U];
        float err[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = load_pack<T, VEC>(pr + e0 + u * kStep);
            if constexpr (MODE == kResidual)
                b[u] = load_pack<T, VEC>(qr + e0 + u * kStep);
        }
#pragma unroll
        for (int k = 0; k < U * VEC; k += 2) {
            const int c = (k >> 1) & 1;
            float w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int u = (k + h) / VEC, i = (k + h) % VEC;
                w[h] = weight32<MODE>(as_f32(a[u].v[i]),
                                      MODE == kResidual ? as_f32(b[u].v[i]) : 0.f,
                                      e0 + u * kStep + i, without, err[c]);
            }
            acc[c] += (double)pair_sum(w[0], w[1], err[c]);
        }
        acc[0] += (double)(err[0] + err[1]);
    }
#pragma unroll 1
    for (; e0 < hi; e0 += kStep)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (e0 + i < hi)
                acc[i & 1] += weight<MODE>(as_f32(pr[e0 + i]),
                                           MODE == kResidual ? as_f32(qr[e0 + i]) : 0.f, e0 + i,
                                           without);
    double sum = warp_sum(acc[0] + acc[1]);
    if (!(sum < INFINITY)) { // weights near fp32's largest, whose pair overflows, or an infinity
        sum = 0.0;
#pragma unroll 1
        for (int e = lo + lane; e < hi; e += 32)
            sum += weight<MODE>(as_f32(pr[e]), MODE == kResidual ? as_f32(qr[e]) : 0.f, e, without);
        sum = warp_sum(sum);
    }
    return sum;
}

template <typename T, int VEC>
__device__ __forceinline__ double piece_sum(const T *pr, const T *qr, int mode, int without, int lo,
                                            int hi, int lane)
{
    if (mode == kResidual)
        return piece_sum_mode<T, VEC, kResidual>(pr, qr, without, lo, hi, lane);
    if (mode == kPlain)
        return piece_sum_mode<T, VEC, kPlain>(pr, qr, without, lo, hi, lane);
    return piece_sum_mode<T, VEC, kWithout>(pr, qr, without, lo, hi, lane);
}

// The token of piece [lo, hi) (at most kVerifyFind): the first whose running sum, counted from
// `base`, exceeds `goal`, or the last of any weight when rounding leaves none. One warp: the
// weights pass through shared memory, so the loads are coalesced and each lane still adds up
// consecutive tokens; then the lanes' sums are scanned, and the one that crosses the goal
// walks its tokens.
constexpr int kVerifyFind = 512;

template <typename T, int MODE>
__device__ __forceinline__ int piece_find_mode(const T *pr, const T *qr, int without, int lo, int hi,
                                               double base, double goal, int lane, double *sm)
{
    constexpr int N = kVerifyFind / 32;
    float x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lo + i * 32 + lane;
        x[i] = y[i] = 0.f;
        if (e < hi) {
            x[i] = as_f32(pr[e]);
            if constexpr (MODE == kResidual)
                y[i] = as_f32(qr[e]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) { // token k at k + k / N: lanes read without bank conflicts
        const int k = i * 32 + lane;
        sm[k + k / N] = weight<MODE>(x[i], y[i], lo + k, without);
    }
    __syncwarp();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        s += sm[lane * (N + 1) + i];
    const double incl = base + warp_scan(s, lane);
    const unsigned over = __ballot_sync(0xffffffffu, incl > goal && s > 0.0);
    const unsigned any = __ballot_sync(0xffffffffu, s > 0.0);
    const int sel = over ? __ffs(over) - 1 : (any ? 31 - __clz(any) : 0);
    int at = lo + sel * N;
    if (lane == sel) {
        double run = incl - s;
        bool found = false;
        for (int i = 0; i < N; ++i) {
            const double w = sm[lane * (N + 1) + i];
            run += w;
            if (w > 0.0 && !found) {
                at = lo + sel * N + i;
                found = run > goal;
            }
        }
    }
    return __shfl_sync(0xffffffffu, at, sel);
}

template <typename T>
__device__ __forceinline__ int piece_find(const T *pr, const T *qr, int mode, int without, int lo,
                                          int hi, double base, double goal, int lane, double *sm)
{
    if (mode == kResidual)
        return piece_find_mode<T, kResidual>(pr, qr, without, lo, hi, base, goal, lane, sm);
    if (mode == kPlain)
        return piece_find_mode<T, kPlain>(pr, qr, without, lo, hi, base, goal, lane, sm);
    return piece_find_mode<T, kWithout>(pr, qr, without, lo, hi, base, goal, lane, sm);
}

// Of consecutive pieces with these sums, the first whose running sum (from `base`, which moves to
// the piece's start) exceeds `goal`, or the last of any weight.
__device__ __forceinline__ int crossing(const double *sums, int n, double &base, double goal)
{
    double run = base, last_base = base;
    int last = 0;
    for (int i = 0; i < n; ++i) {
        if (sums[i] > 0.0) {
            last = i;
            last_base = run;
            if (run + sums[i] > goal)
                break;
        }
        run += sums[i];
    }
    base = last_base;
    return last;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kVerifyThreads, 4)
    verify_kernel(const __grid_constant__ VerifyParams p)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ double piece[kVerifyWarps]; // sums of this block's warps
    __shared__ double total[2];            // this block's sum (read by the cluster), by attempt
    __shared__ double find[kVerifyFind + 32];
    __shared__ int first_refused, count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const long long b = blockIdx.x / cs;
    // the probabilities may come from the kernel before this one on the stream
    grid_dep_wait();
    grid_dep_launch();
    const T *target = static_cast<const T *>(p.target) + b * (p.max_drafts + 1) * p.target_stride;
    const T *draft = p.draft ? static_cast<const T *>(p.draft) + b * p.max_drafts * p.draft_stride
                             : nullptr;
    const int32_t *drafted = p.drafted + b * p.max_drafts;
    const float *uni = p.uniforms + b * (p.max_drafts + 1);

    // ---- accept test, 32 drafts at a time (every block of the cluster: no exchange needed)
    if (warp == 0) {
        int n = p.n_drafts ? __ldg(p.n_drafts + b) : p.max_drafts;
        unsigned err = 0;
        if (n < 0 || n > p.max_drafts) {
            err |= kErrProbs;
            n = n < 0 ? 0 : p.max_drafts;
        }
        int refused = n;
#pragma unroll 1
        for (int i0 = 0; i0 < n && refused == n; i0 += 32) {
            const int i = i0 + lane;
            bool bad = false;
            if (i < n) {
                const int x = __ldg(drafted + i);
                bad = true;
                if (x >= 0 && x < p.vocab) {
                    const double pv = (double)as_f32(target[i * p.target_stride + x]);
                    const double qv = draft ? (double)as_f32(draft[i * p.draft_stride + x]) : 1.0;
                    bad = !((double)__ldg(uni + i) * qv < pv);
                } else {
                    err |= kErrProbs;
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, bad);
            if (m)
                refused = i0 + __ffs(m) - 1;
        }
        if (err)
            atomicOr(p.errors, err);
        if (lane == 0) {
            first_refused = refused;
            count = n;
        }
    }
    __syncthreads();
    const int at = first_refused;
    const bool refused = at < count;
    const T *pr = target + at * p.target_stride;
    const T *qr = refused && draft ? draft + at * p.draft_stride : pr;
    int mode = !refused ? kPlain : (draft ? kResidual : kWithout);
    const int without = refused ? __ldg(drafted + at) : -1;

    // ---- this block's part of the row, and this warp's piece of it
    constexpr int kUnit = 32 * VEC;
    const int units = (p.vocab + kUnit - 1) / kUnit;
    const int pieces = cs * kVerifyWarps;
    const int w = rank * kVerifyWarps + warp;
    const int u0 = (int)((long long)units * w / pieces);
    const int u1 = (int)((long long)units * (w + 1) / pieces);
    const int lo = u0 * kUnit < p.vocab ? u0 * kUnit : p.vocab;
    const int hi = u1 * kUnit < p.vocab ? u1 * kUnit : p.vocab;

    double Z = 0.0, before = 0.0; // all weights, those of the blocks before this one
    int owner = 0;                // block whose part crosses the goal
    double goal = 0.0;
    const double u = (double)__ldg(uni + p.max_drafts);
#pragma unroll 1
    for (int attempt = 0; attempt < 2; ++attempt) {
        const double s = piece_sum<T, VEC>(pr, qr, mode, without, lo, hi, lane);
        if (lane == 0)
            piece[warp] = s;
        __syncthreads();
        double mine = 0.0;
#pragma unroll
        for (int i = 0; i < kVerifyWarps; ++i)
            mine += piece[i];
        if (tid == 0)
            total[attempt] = mine;
        cluster.sync();
        double sums[kVerifyCluster];
#pragma unroll
        for (int r = 0; r < kVerifyCluster; ++r)
            sums[r] = r < cs ? *cluster.map_shared_rank(&total[attempt], r) : 0.0;
        Z = 0.0;
#pragma unroll
        for (int r = 0; r < kVerifyCluster; ++r)
            Z += sums[r];
        goal = u * Z;
        double run = 0.0;
        int last = 0;
        owner = -1;
#pragma unroll
        for (int r = 0; r < kVerifyCluster; ++r) {
            if (r == rank)
                before = run;
            run += sums[r];
            if (sums[r] > 0.0) {
                last = r;
                if (owner < 0 && run > goal)
                    owner = r;
            }
        }
        if (owner < 0)
            owner = last;
        // a residual without weight: the refused token was as likely as the target allows, and
        // the draw falls back to the target's own row
        if (Z > 0.0 || mode == kPlain)
            break;
        mode = kPlain;
        __syncthreads(); // piece[] is written again
    }
    cluster.barrier_arrive(); // (waited for below: no block leaves while its sums are read)

    int32_t *tokens = p.tokens + b * (p.max_drafts + 1);
    if (rank == 0) {
        if (tid == 0)
            p.accepted[b] = at;
#pragma unroll 1
        for (int i = tid; i <= p.max_drafts; i += kVerifyThreads)
            if (i != at)
                tokens[i] = i < at ? __ldg(drafted + i) : -1;
    }
    const bool drawn = Z > 0.0 && Z < INFINITY;
    if (rank == owner && !drawn && tid == 0) { // nothing to draw from
        tokens[at] = -1;
        atomicOr(p.errors, kErrProbs);
    }
    if (rank == owner && drawn) {
        // ---- the warp piece of this block that crosses the goal, divided among the block's warps
        // until one warp can finish it (every thread follows the same choice)
        double base = before;
        int sel = rank * kVerifyWarps + crossing(piece, kVerifyWarps, base, goal);
        int a = (int)((long long)units * sel / pieces) * kUnit;
        int z = (int)((long long)units * (sel + 1) / pieces) * kUnit;
        z = z < p.vocab ? z : p.vocab;
#pragma unroll 1
        while (z - a > kVerifyFind) {
            const int per = ((z - a + kVerifyWarps * kUnit - 1) / (kVerifyWarps * kUnit)) * kUnit;
            const int l = a + warp * per < z ? a + warp * per : z;
            const int h = l + per < z ? l + per : z;
            __syncthreads(); // piece[] has been read
            const double s = piece_sum<T, VEC>(pr, qr, mode, without, l, h, lane);
            if (lane == 0)
                piece[warp] = s;
            __syncthreads();
            sel = crossing(piece, kVerifyWarps, base, goal);
            a = a + sel * per;
            z = a + per < z ? a + per : z;
        }
        if (warp == 0) {
            const int x = piece_find<T>(pr, qr, mode, without, a, z, base, goal, lane, find);
            if (lane == 0)
                tokens[at] = x;
        }
    }
    cluster.barrier_wait();
}

} // namespace q8kv
