// ep_picksum.cu -- the weighted sum of the rows a receive row's picks have in
// the experts' output, which ep_combine reads as one row per receive slot
// (include/ep_ops.h).
//
// Bound by memory: every place's row is read once, every receive row written
// once.  A pick's place is found by searching its expert's rows, which are in
// increasing order; the searches of a row's picks run side by side, one to a
// lane, and the block's other rows' copies hide them.
#include "ep_ops.cuh"

namespace {

using namespace ep;

constexpr int kThreads = 256;

struct SumParams {
    int64_t rows, places;
    const __nv_bfloat16 *y;
    const int32_t *recv_topk_idx, *recv_base, *expert_off, *expert_count, *expert_rows;
    const float *recv_topk_weights;
    __nv_bfloat16 *out;
    int64_t y_stride, out_stride;
    int32_t *status;
    int hidden, topk, ranks, per_rank;
};

// Place of receive row r among expert e's rows, or -1.
__device__ int find_place(const SumParams &p, int e, int r) {
    int64_t lo = p.expert_off[e], hi = lo + p.expert_count[e];
    if (lo < 0 || hi < lo || hi > p.places) return -1;
    const int64_t end = hi;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (p.expert_rows[mid] < r) lo = mid + 1;
        else hi = mid;
    }
    return lo < end && p.expert_rows[lo] == r ? static_cast<int>(lo) : -1;
}

__global__ void __launch_bounds__(kThreads) pick_sum_kernel(SumParams p) {
    __shared__ int place[kMaxTopk];
    __shared__ float weight[kMaxTopk];
    __shared__ int picks;
    const int64_t r = blockIdx.x;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int at = -1;
        float w = 0.0f;
        const int local = lane < p.topk ? p.recv_topk_idx[r * p.topk + lane] : -1;
        if (local >= 0) {
            // the last rank whose window starts at or before this row
            int lo = 0, hi = p.ranks;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.recv_base[mid] <= r) lo = mid;
                else hi = mid;
            }
            if (local < p.per_rank) at = find_place(p, lo * p.per_rank + local, static_cast<int>(r));
            w = p.recv_topk_weights[r * p.topk + lane];
            if (at < 0 && p.status) set_error(p.status, EP_ERR_INVALID_ARG);
        }
        const uint32_t there = __ballot_sync(0xffffffffu, at >= 0);
        if (at >= 0) {
            const int n = __popc(there & ((1u << lane) - 1u));
            place[n] = at;
            weight[n] = w;
        }
        if (lane == 0) picks = __popc(there);
    }
    __syncthreads();
    const int n = picks;
    for (int v = threadIdx.x; v < p.hidden >> 3; v += kThreads) {
        float acc[8] = {};
        for (int k = 0; k < n; ++k) {
            float f[8];
            unpack8(*reinterpret_cast<const uint4 *>(p.y + place[k] * p.y_stride + v * 8), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = fmaf(weight[k], f[j], acc[j]);
        }
        *reinterpret_cast<uint4 *>(p.out + r * p.out_stride + v * 8) = pack8(acc);
    }
}

}  // namespace

extern "C" ep_status ep_pick_sum(int64_t rows, int64_t places, int32_t hidden, int32_t topk, int32_t ranks,
                                 int32_t experts, const void *y, int64_t y_stride, const int32_t *recv_topk_idx,
                                 const float *recv_topk_weights, const int32_t *recv_base, const int32_t *expert_off,
                                 const int32_t *expert_count, const int32_t *expert_rows, void *out,
                                 int64_t out_stride, int32_t *status, void *stream) {
    if (rows < 0 || rows >= (1ll << 31) || places < 0 || places >= (1ll << 31) || hidden < 8 || hidden % 8 != 0 ||
        topk < 1 || topk > kMaxTopk || ranks < 1 || ranks > kMaxRanks || experts < ranks || experts % ranks != 0 ||
        experts > 4096)
        return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    if (!recv_topk_idx || !recv_topk_weights || !recv_base || !expert_off || !expert_count || !out ||
        (places > 0 && (!y || !expert_rows)))
        return EP_ERR_INVALID_ARG;
    if (!aligned(y, 16) || y_stride % 8 != 0 || y_stride < hidden || !aligned(out, 16) || out_stride % 8 != 0 ||
        out_stride < hidden)
        return EP_ERR_INVALID_ARG;
    const Caller c;
    if (!c.ok) return EP_ERR_CUDA;
    if (!c.has_or_null(y) || !c.has(recv_topk_idx) || !c.has(recv_topk_weights) || !c.has(recv_base) ||
        !c.has(expert_off) || !c.has(expert_count) || !c.has_or_null(expert_rows) || !c.has(out) ||
        !c.has_or_null(status))
        return EP_ERR_INVALID_ARG;
    SumParams p{};
    p.rows = rows, p.places = places;
    p.y = static_cast<const __nv_bfloat16 *>(y), p.y_stride = y_stride;
    p.recv_topk_idx = recv_topk_idx, p.recv_topk_weights = recv_topk_weights, p.recv_base = recv_base;
    p.expert_off = expert_off, p.expert_count = expert_count, p.expert_rows = expert_rows;
    p.out = static_cast<__nv_bfloat16 *>(out), p.out_stride = out_stride, p.status = status;
    p.hidden = hidden, p.topk = topk, p.ranks = ranks, p.per_rank = experts / ranks;
    pick_sum_kernel<<<static_cast<unsigned>(rows), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launched();
}
