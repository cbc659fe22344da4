// rmsnorm.cu -- the norm in front of an MoE block: residual addition, root-mean-square norm,
// outputs in bf16 and / or MXFP8, and the backward.
//
//   s = x + r                         (fp32; stored once as bf16: the residual stream)
//   rstd = 1 / sqrt(mean(s^2) + eps)  (fp32)
//   y = s rstd w                      (fp32, from the unrounded s; rounded once per output)
//
// Backward, with xhat = s rstd taken from the stored s:
//   dx = rstd (w dy - xhat mean(w dy xhat)) + d_s      (of x and of r alike)
//   dw = sum over rows of dy xhat
//
// Bound by memory: each tensor is read or written once.  One block per row, the row held in
// registers between the sum of squares and the scaling.
#include "common.cuh"
#include "mx.cuh"

namespace moe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormMaxVec = 16;      // 8-element vectors a thread holds: H <= 32768
constexpr int kNormBwdBlocks = 304;  // rows of partial weight gradients

__device__ __forceinline__ void unpack8(const uint4 &raw, float (&v)[8]) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(p[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint4 raw;
    __nv_bfloat162 *p = reinterpret_cast<__nv_bfloat162 *>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    return raw;
}

// Sum over the block, the same value in every thread; s_red holds one float per warp and is
// free again after the caller's next __syncthreads.
__device__ __forceinline__ float block_sum(float v, float *s_red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) s_red[warp] = v;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < nw; ++i) t += s_red[i];
    return t;
}

template <int V>
__global__ void __launch_bounds__(kNormThreads)
add_rmsnorm_kernel(const uint4 *__restrict__ x, const uint4 *__restrict__ res, const uint4 *__restrict__ weight,
                   float eps, int H, uint4 *__restrict__ sum, uint4 *__restrict__ y, uint8_t *__restrict__ y_q,
                   uint8_t *__restrict__ y_sf, float *__restrict__ rstd_out) {
    pdl_wait();
    __shared__ float s_red[kNormThreads / 32];
    const int nv = H / 8;
    const int64_t row = blockIdx.x;
    float v[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * kNormThreads + threadIdx.x;
        if (c < nv) {
            unpack8(x[row * nv + c], v[i]);
            if (res) {
                float r[8];
                unpack8(res[row * nv + c], r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += r[j];
                sum[row * nv + c] = pack8(v[i]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
        }
    }
    ss = block_sum(ss, s_red);
    const float rstd = 1.0f / sqrtf(ss / (float)H + eps);
    if (threadIdx.x == 0 && rstd_out) rstd_out[row] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * kNormThreads + threadIdx.x;
        float o[8] = {};
        if (c < nv) {
            float w[8];
            unpack8(weight[c], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = v[i][j] * rstd * w[j];
            if (y) y[row * nv + c] = pack8(o);
        }
        if (y_q) {
            // four neighbouring threads hold one block of 32
            float a = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(o[j]));
            a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
            const int X = mx::scale_exp(a);
            if (c < nv) {
                *reinterpret_cast<uint2 *>(y_q + row * H + (int64_t)c * 8) = mx::quantize8(o, X);
                if ((threadIdx.x & 3) == 0) y_sf[row * (H / 32) + c / 4] = (uint8_t)(X + 127);
            }
        }
    }
}

// dx of the rows blockIdx.x, blockIdx.x + gridDim.x, ..., and this block's share of dw.
template <int V>
__global__ void __launch_bounds__(kNormThreads)
add_rmsnorm_bwd_kernel(const uint4 *__restrict__ dy, const uint4 *__restrict__ d_sum, const uint4 *__restrict__ sum,
                       const uint4 *__restrict__ weight, const float *__restrict__ rstd_in, int64_t T, int H,
                       uint4 *__restrict__ dx, float *__restrict__ dw_part) {
    pdl_wait();
    __shared__ float s_red[2][kNormThreads / 32];
    const int nv = H / 8;
    float dw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    int par = 0;
    for (int64_t row = blockIdx.x; row < T; row += gridDim.x, par ^= 1) {
        const float rstd = rstd_in[row];
        float g[V][8], xh[V][8];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * kNormThreads + threadIdx.x;
            if (c < nv) {
                float w[8];
                unpack8(dy[row * nv + c], g[i]);
                unpack8(sum[row * nv + c], xh[i]);
                unpack8(weight[c], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh[i][j] *= rstd;
                    dw[i][j] += g[i][j] * xh[i][j];
                    g[i][j] *= w[j];
                    dot += g[i][j] * xh[i][j];
                }
            }
        }
        const float m = block_sum(dot, s_red[par]) / (float)H;   // the other half is free: one barrier a row
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * kNormThreads + threadIdx.x;
            if (c < nv) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = rstd * (g[i][j] - xh[i][j] * m);
                if (d_sum) {
                    float d[8];
                    unpack8(d_sum[row * nv + c], d);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] += d[j];
                }
                dx[row * nv + c] = pack8(o);
            }
        }
    }
    if (!dw_part) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * kNormThreads + threadIdx.x;
        if (c < nv) {
            float4 *p = reinterpret_cast<float4 *>(dw_part + (int64_t)blockIdx.x * H + (int64_t)c * 8);
            p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// dw[c] = sum over the blocks' partial rows, in block order (the same order every run).
__global__ void __launch_bounds__(kNormThreads)
rmsnorm_dw_kernel(const float *__restrict__ part, int blocks, int H, float *__restrict__ dw) {
    pdl_wait();
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= H) return;
    float s = 0.0f;
    for (int b = 0; b < blocks; ++b) s += part[(int64_t)b * H + c];
    dw[c] = s;
}

moe_status_t check_norm(int64_t T, int H) {
    if (T < 0 || H < 1) return MOE_ERR_INVALID_ARG;
    if (H % 8 != 0 || H > kNormThreads * 8 * kNormMaxVec || T > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_add_rmsnorm(const moe_bf16_t *x, const moe_bf16_t *residual, const moe_bf16_t *weight,
                                        float eps, int64_t T, int H, moe_bf16_t *sum, moe_bf16_t *y, uint8_t *y_q,
                                        uint8_t *y_sf, float *rstd, moe_stream_t stream) {
    MOE_NVTX_RANGE("moe_add_rmsnorm");
    using namespace moe;
    moe_status_t st = check_norm(T, H);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.0f) || (!y_q) != (!y_sf) || (residual && !sum)) return MOE_ERR_INVALID_ARG;
    if (y_q && H % 32 != 0) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!x || !weight || (!y && !y_q)) return MOE_ERR_INVALID_ARG;
    if (!all_aligned16({x, residual, weight, sum, y}) || reinterpret_cast<uintptr_t>(y_q) % 8)
        return MOE_ERR_UNSUPPORTED;
    const int per = (H / 8 + kNormThreads - 1) / kNormThreads;
#define MOE_NORM(V)                                                                                               \
    launch_k(add_rmsnorm_kernel<V>, dim3((unsigned)T), dim3(kNormThreads), 0, (cudaStream_t)stream,               \
             reinterpret_cast<const uint4 *>(x), reinterpret_cast<const uint4 *>(residual),                       \
             reinterpret_cast<const uint4 *>(weight), eps, H, reinterpret_cast<uint4 *>(sum),                     \
             reinterpret_cast<uint4 *>(y), y_q, y_sf, rstd)
    if (per <= 1) MOE_NORM(1);
    else if (per <= 2) MOE_NORM(2);
    else if (per <= 4) MOE_NORM(4);
    else if (per <= 8) MOE_NORM(8);
    else MOE_NORM(16);
#undef MOE_NORM
    return launch_status();
}

extern "C" size_t moe_rmsnorm_bwd_workspace_bytes(int64_t T, int H) {
    using namespace moe;
    if (check_norm(T, H) != MOE_OK) return 0;
    const int64_t blocks = T < kNormBwdBlocks ? (T > 0 ? T : 1) : kNormBwdBlocks;
    return (size_t)blocks * (size_t)H * sizeof(float);
}

extern "C" moe_status_t moe_add_rmsnorm_bwd(const moe_bf16_t *dy, const moe_bf16_t *d_sum, const moe_bf16_t *sum,
                                            const moe_bf16_t *weight, const float *rstd, int64_t T, int H,
                                            moe_bf16_t *dx, float *dweight, void *ws, size_t ws_bytes,
                                            moe_stream_t stream) {
    MOE_NVTX_RANGE("moe_add_rmsnorm_bwd");
    using namespace moe;
    moe_status_t st = check_norm(T, H);
    if (st != MOE_OK) return st;
    if (dweight && (!ws || ws_bytes < moe_rmsnorm_bwd_workspace_bytes(T, H))) return MOE_ERR_WORKSPACE;
    if (T > 0 && (!dy || !sum || !weight || !rstd || !dx)) return MOE_ERR_INVALID_ARG;
    if (!all_aligned16({dy, d_sum, sum, weight, dx, dweight ? ws : nullptr})) return MOE_ERR_UNSUPPORTED;
    cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) return dweight ? cuda_status(cudaMemsetAsync(dweight, 0, (size_t)H * sizeof(float), s)) : MOE_OK;
    const int blocks = T < kNormBwdBlocks ? (int)T : kNormBwdBlocks;
    float *part = dweight ? static_cast<float *>(ws) : nullptr;
    const int per = (H / 8 + kNormThreads - 1) / kNormThreads;
#define MOE_NORM_BWD(V)                                                                                           \
    launch_k(add_rmsnorm_bwd_kernel<V>, dim3((unsigned)blocks), dim3(kNormThreads), 0, s,                         \
             reinterpret_cast<const uint4 *>(dy), reinterpret_cast<const uint4 *>(d_sum),                         \
             reinterpret_cast<const uint4 *>(sum), reinterpret_cast<const uint4 *>(weight), rstd, T, H,           \
             reinterpret_cast<uint4 *>(dx), part)
    if (per <= 1) MOE_NORM_BWD(1);
    else if (per <= 2) MOE_NORM_BWD(2);
    else if (per <= 4) MOE_NORM_BWD(4);
    else if (per <= 8) MOE_NORM_BWD(8);
    else MOE_NORM_BWD(16);
#undef MOE_NORM_BWD
    if (dweight)
        launch_k(rmsnorm_dw_kernel, dim3((unsigned)((H + kNormThreads - 1) / kNormThreads)), dim3(kNormThreads), 0, s,
                 part, blocks, H, dweight);
    return launch_status();
}
