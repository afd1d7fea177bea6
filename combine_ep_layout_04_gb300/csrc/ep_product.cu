// ep_product.cu -- the experts' products of 8-bit rows and 8-bit matrices with
// a scale for each block of 128 columns (rows) and 128 x 128 (matrices), over
// the expert-major places of the expert layout (include/ep_ops.h).
#include "ep_ops.cuh"

namespace {

using namespace ep;

struct ProductParams {
    int64_t places, a_rows;
    const uint8_t *values, *w;
    const float *scales, *w_scales;
    const int32_t *expert_off, *expert_count, *rows;
    __nv_bfloat16 *out;
    uint8_t *out_values;
    float *out_scales;
    int32_t *status;
    int64_t value_stride, scale_stride, out_stride, out_value_stride, out_scale_stride;
    int experts, width, n, nb, kb;      // n: columns of an output; nb, kb: blocks of 128 in n and width
};

// Experts' counts as the kernels use them: a segment outside [0, places) is
// not touched.
__device__ __forceinline__ int count_of(const ProductParams &p, int e) {
    const int64_t off = p.expert_off[e], n = p.expert_count[e];
    return off < 0 || n < 0 || off + n > p.places ? 0 : static_cast<int>(n);
}
__device__ __forceinline__ bool bad_segment(const ProductParams &p, int e) {
    const int64_t off = p.expert_off[e], n = p.expert_count[e];
    return off < 0 || n < 0 || off + n > p.places;
}

__device__ __forceinline__ float fp8_value(uint8_t v) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

constexpr int kM = 32, kK = 32;

// 32 places x 128 columns a block (of both matrices where kGated), fp32
// products of 32 columns at a time through shared memory.  A warp holds four
// places, a lane four columns of each, so that a place's block maximum is one
// warp's.
template <bool kGated>
__global__ void __launch_bounds__(256) product_kernel(ProductParams p) {
    __shared__ float a[kM][kK + 1], b[kGated ? 2 : 1][kBlock][kK + 1];
    __shared__ int s_expert, s_tile;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        int left = blockIdx.y, e = 0;
        for (; e < p.experts; ++e) {
            const int tiles = (count_of(p, e) + kM - 1) / kM;
            if (bad_segment(p, e) && p.status) set_error(p.status, EP_ERR_INVALID_ARG);
            if (left < tiles) break;
            left -= tiles;
        }
        s_expert = e;
        s_tile = left;
    }
    __syncthreads();
    const int e = s_expert;
    if (e >= p.experts) return;
    const int n0 = blockIdx.x * kBlock;
    const int64_t first = p.expert_off[e] + static_cast<int64_t>(s_tile) * kM;
    const int here = min(kM, count_of(p, e) - s_tile * kM);
    float acc[kGated ? 2 : 1][4][4] = {};
    for (int k0 = 0; k0 < p.width; k0 += kK) {
        const int block = k0 / kBlock;
        for (int i = tid; i < kM * kK; i += 256) {
            const int m = i / kK, k = k0 + i % kK;
            float v = 0.0f;
            if (m < here && k < p.width) {
                const int64_t row = p.rows ? p.rows[first + m] : first + m;
                if (row >= 0 && row < p.a_rows)
                    v = fp8_value(p.values[row * p.value_stride + k]) * p.scales[row * p.scale_stride + block];
                else if (p.status)
                    set_error(p.status, EP_ERR_INVALID_ARG);
            }
            a[m][i % kK] = v;
        }
#pragma unroll
        for (int h = 0; h < (kGated ? 2 : 1); ++h) {
            const int64_t matrix = static_cast<int64_t>(e) * (kGated ? 2 : 1) + h;
            const float s = p.w_scales[(matrix * p.nb + blockIdx.x) * p.kb + block];
            for (int i = tid; i < kBlock * kK; i += 256) {
                const int n = n0 + i / kK, k = k0 + i % kK;
                b[h][i / kK][i % kK] =
                    n < p.n && k < p.width ? fp8_value(p.w[(matrix * p.n + n) * p.width + k]) * s : 0.0f;
            }
        }
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < kK; ++k) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = a[warp * 4 + i][k];
#pragma unroll
            for (int h = 0; h < (kGated ? 2 : 1); ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float y = b[h][j * 32 + lane][k];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[h][i][j] = fmaf(x[i], y, acc[h][i][j]);
                }
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int m = warp * 4 + i;
        if (m >= here) break;
        if (!kGated) {
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + j * 32 + lane;
                if (n < p.n) p.out[(first + m) * p.out_stride + n] = __float2bfloat16(acc[0][i][j]);
            }
        } else {
            float y[4], most = kFloor;
            for (int j = 0; j < 4; ++j) {
                const float g = acc[0][i][j];
                y[j] = n0 + j * 32 + lane < p.n ? g / (1.0f + expf(-g)) * acc[kGated ? 1 : 0][i][j] : 0.0f;
                most = max_nan(most, fabsf(y[j]));
            }
            for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
            const float inv = kFp8Max / most;
            if (lane == 0) p.out_scales[(first + m) * p.out_scale_stride + blockIdx.x] = most * (1.0f / kFp8Max);
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + j * 32 + lane;
                if (n < p.n)
                    p.out_values[(first + m) * p.out_value_stride + n] =
                        __nv_cvt_float_to_fp8(y[j] * inv, __NV_SATFINITE, __NV_E4M3);
            }
        }
    }
}

}  // namespace

extern "C" ep_status ep_expert_product(int64_t places, int64_t a_rows, int32_t experts, int32_t width, int32_t out,
                                       int32_t gated, const void *values, int64_t value_stride, const float *scales,
                                       int64_t scale_stride, const void *w, const float *w_scales,
                                       const int32_t *expert_off, const int32_t *expert_count, const int32_t *rows,
                                       void *out_bf16, int64_t out_stride, void *out_values, int64_t out_value_stride,
                                       float *out_scales, int64_t out_scale_stride, int32_t *status, void *stream) {
    if (places < 0 || places >= (1ll << 31) || a_rows < 0 || a_rows >= (1ll << 31) || experts < 1 ||
        experts > 4096 || width < 16 || width > 65536 || width % 16 != 0 || out < 8 || out > 65536 || out % 8 != 0 ||
        (gated != 0 && gated != 1))
        return EP_ERR_INVALID_ARG;
    if (places == 0) return EP_OK;
    const int nb = (out + kBlock - 1) / kBlock, kb = (width + kBlock - 1) / kBlock;
    if (!w || !w_scales || !expert_off || !expert_count || (a_rows > 0 && (!values || !scales)) ||
        (!rows && places > a_rows))
        return EP_ERR_INVALID_ARG;
    if (!aligned(values, 16) || value_stride % 16 != 0 || value_stride < width || !aligned(scales, 4) ||
        scale_stride < kb || !aligned(w, 16) || !aligned(w_scales, 4))
        return EP_ERR_INVALID_ARG;
    if (gated ? !out_values || !out_scales || out_bf16 || !aligned(out_values, 8) || out_value_stride % 8 != 0 ||
                    out_value_stride < out || !aligned(out_scales, 4) || out_scale_stride < nb
              : !out_bf16 || out_values || out_scales || !aligned(out_bf16, 16) || out_stride % 8 != 0 ||
                    out_stride < out)
        return EP_ERR_INVALID_ARG;
    const Caller c;
    if (!c.ok) return EP_ERR_CUDA;
    if (!c.has_or_null(values) || !c.has_or_null(scales) || !c.has(w) || !c.has(w_scales) || !c.has(expert_off) ||
        !c.has(expert_count) || !c.has_or_null(rows) || !c.has_or_null(out_bf16) || !c.has_or_null(out_values) ||
        !c.has_or_null(out_scales) || !c.has_or_null(status))
        return EP_ERR_INVALID_ARG;
    ProductParams p{};
    p.places = places, p.a_rows = a_rows;
    p.values = static_cast<const uint8_t *>(values), p.value_stride = value_stride;
    p.scales = scales, p.scale_stride = scale_stride;
    p.w = static_cast<const uint8_t *>(w), p.w_scales = w_scales;
    p.expert_off = expert_off, p.expert_count = expert_count, p.rows = rows;
    p.out = static_cast<__nv_bfloat16 *>(out_bf16), p.out_stride = out_stride;
    p.out_values = static_cast<uint8_t *>(out_values), p.out_value_stride = out_value_stride;
    p.out_scales = out_scales, p.out_scale_stride = out_scale_stride;
    p.status = status;
    p.experts = experts, p.width = width, p.n = out, p.nb = nb, p.kb = kb;
    // every expert may leave one tile short
    const int64_t tiles = places / kM + (places < experts ? places : experts);
    if (tiles > 65535) return EP_ERR_INVALID_ARG;
    const dim3 grid(nb, static_cast<unsigned>(tiles));
    if (gated)
        product_kernel<true><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    else
        product_kernel<false><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launched();
}
