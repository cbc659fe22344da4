// decode.cu -- a whole MoE layer for a few tokens: routing, gate / up products, SwiGLU, down
// product and the weighted sum over the experts, on bf16 or MXFP8 expert weights.
//
//   idx, w = route(logits)                         (moe_route_topk / moe_route_topk_sigmoid)
//   h_tj   = silu(x_t Wg[e]) (x_t Wu[e]),  e = idx[t, j]
//   out_t  = bf16(sum_j w_tj h_tj Wd[e])           (fp32 sums, one rounding)
//
// MXFP8 weights enter as the values their codes stand for; x and h are not quantised.
#include "common.cuh"
#include "mx.cuh"

namespace moe {
namespace {

struct Clamp {
    float glo, ghi, ulo, uhi;
};

// Element (k, n) of expert e of a bf16 [E, K, N] tensor.
struct WeightsBf16 {
    const __nv_bfloat16 *w;
    int K, N;
    __device__ __forceinline__ float operator()(int e, int k, int n) const {
        return __bfloat162float(w[((int64_t)e * K + k) * N + n]);
    }
};

// The same of a tensor quantised by moe_quantize_weights_mxfp8.
struct WeightsMx {
    const uint8_t *q, *sf;
    int K, N;
    __device__ __forceinline__ float operator()(int e, int k, int n) const {
        const int64_t blk = ((int64_t)e * (K / 128) + k / 128) * (N / 128) + n / 128;
        const int m = n % 128, kk = k % 128;
        __nv_fp8_e4m3 c;
        c.__x = q[blk * 16384 + m * 128 + (((kk / 16) ^ (m % 8)) * 16) + kk % 16];
        const int X = (int)sf[blk * 512 + (m % 32) * 16 + (m / 32) * 4 + kk / 32] - 127;
        return ldexpf((float)c, X);
    }
};

// One block per route and 128 features.
template <typename W>
__global__ void __launch_bounds__(128)
decode_fc1_kernel(const __nv_bfloat16 *__restrict__ x, const int32_t *__restrict__ topk_idx, int k, W gate, W up,
                  Clamp cl, float *__restrict__ h) {
    pdl_wait();
    const int r = blockIdx.y, f = blockIdx.x * 128 + threadIdx.x, H = gate.K, F = gate.N;
    const int e = topk_idx[r];
    const __nv_bfloat16 *xr = x + (int64_t)(r / k) * H;
    float g = 0.0f, u = 0.0f;
    for (int i = 0; i < H; ++i) {
        const float v = __bfloat162float(xr[i]);
        g += v * gate(e, i, f);
        u += v * up(e, i, f);
    }
    g = fminf(fmaxf(g, cl.glo), cl.ghi);
    u = fminf(fmaxf(u, cl.ulo), cl.uhi);
    h[(int64_t)r * F + f] = g / (1.0f + expf(-g)) * u;
}

// One block per token and 128 output columns.
template <typename W>
__global__ void __launch_bounds__(128)
decode_fc2_kernel(const float *__restrict__ h, const int32_t *__restrict__ topk_idx, const float *__restrict__ topk_w,
                  int k, W down, __nv_bfloat16 *__restrict__ out) {
    pdl_wait();
    const int t = blockIdx.y, n = blockIdx.x * 128 + threadIdx.x, F = down.K, H = down.N;
    float acc = 0.0f;
    for (int j = 0; j < k; ++j) {
        const int e = topk_idx[t * k + j];
        const float *hr = h + (int64_t)(t * k + j) * F;
        float y = 0.0f;
        for (int f = 0; f < F; ++f) y += hr[f] * down(e, f, n);
        acc += topk_w[t * k + j] * y;
    }
    out[(int64_t)t * H + n] = __float2bfloat16_rn(acc);
}

size_t decode_workspace(int64_t T, int F, int k) { return kWsHeaderBytes + (size_t)(T * k) * (size_t)F * sizeof(float); }

bool interval_ok(float lo, float hi) { return lo <= hi; }   // false for a NaN bound

template <typename W>
moe_status_t launch_decode(const moe_bf16_t *x, const float *logits, const float *expert_bias, int score_fn,
                           int normalize, const Clamp &cl, const W &gate, const W &up, const W &down, int64_t T, int H,
                           int F, int E, int k, int32_t *topk_idx, float *topk_w, moe_bf16_t *out, void *ws,
                           cudaStream_t s) {
    const moe_status_t st =
        score_fn == MOE_SCORE_SIGMOID
            ? moe_route_topk_sigmoid(logits, expert_bias, T, E, k, normalize, topk_idx, topk_w, s)
            : moe_route_topk(logits, T, E, k, topk_idx, topk_w, s);
    if (st != MOE_OK) return st;
    float *h = reinterpret_cast<float *>(static_cast<char *>(ws) + kWsHeaderBytes);
    launch_k(decode_fc1_kernel<W>, dim3((unsigned)(F / 128), (unsigned)(T * k)), dim3(128), 0, s,
             reinterpret_cast<const __nv_bfloat16 *>(x), topk_idx, k, gate, up, cl, h);
    launch_k(decode_fc2_kernel<W>, dim3((unsigned)(H / 128), (unsigned)T), dim3(128), 0, s, h, topk_idx, topk_w, k,
             down, reinterpret_cast<__nv_bfloat16 *>(out));
    return launch_status();
}

moe_status_t check_decode(const void *x, const void *logits, int score_fn, const Clamp &cl, int64_t T, int H, int F,
                          int E, int k, const void *topk_idx, const void *topk_w, const void *out) {
    if (T < 0 || H < 1 || F < 1) return MOE_ERR_INVALID_ARG;
    if (score_fn != MOE_SCORE_SOFTMAX && score_fn != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (!interval_ok(cl.glo, cl.ghi) || !interval_ok(cl.ulo, cl.uhi)) return MOE_ERR_INVALID_ARG;
    if (T > MOE_DECODE_MAX_TOKENS || H % 128 != 0 || F % 128 != 0 || E < 1 || E > 1024 || k < 1 || k > 32 || k > E)
        return MOE_ERR_UNSUPPORTED;
    if (T > 0 && (!x || !logits || !topk_idx || !topk_w || !out)) return MOE_ERR_INVALID_ARG;
    if (!all_aligned16({x, out})) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_decode_workspace_bytes(int64_t T, int H, int F, int E, int k) {
    if (T < 0 || T > MOE_DECODE_MAX_TOKENS || H < 1 || F < 1 || H % 128 || F % 128 || E < 1 || E > 1024 || k < 1 ||
        k > 32 || k > E)
        return 0;
    return moe::decode_workspace(T, F, k);
}

extern "C" moe_status_t moe_decode_workspace_init(void *ws, size_t ws_bytes, moe_stream_t stream) {
    return moe_workspace_init(ws, ws_bytes, stream);
}

extern "C" moe_status_t moe_decode(const moe_bf16_t *x, const float *logits, const float *expert_bias, int score_fn,
                                   int normalize, float gate_lo, float gate_hi, float up_lo, float up_hi,
                                   const moe_bf16_t *W_gate, const moe_bf16_t *W_up, const moe_bf16_t *W_down,
                                   int64_t T, int H, int F, int E, int k, int32_t *topk_idx, float *topk_w,
                                   moe_bf16_t *out, void *ws, size_t ws_bytes, moe_stream_t stream) {
    MOE_NVTX_RANGE("moe_decode");
    using namespace moe;
    const Clamp cl{gate_lo, gate_hi, up_lo, up_hi};
    const moe_status_t st = check_decode(x, logits, score_fn, cl, T, H, F, E, k, topk_idx, topk_w, out);
    if (st != MOE_OK || T == 0) return st;
    if (!W_gate || !W_up || !W_down) return MOE_ERR_INVALID_ARG;
    if (!all_aligned16({W_gate, W_up, W_down})) return MOE_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < moe_decode_workspace_bytes(T, H, F, E, k)) return MOE_ERR_WORKSPACE;
    auto w = [](const moe_bf16_t *p, int K, int N) {
        return WeightsBf16{reinterpret_cast<const __nv_bfloat16 *>(p), K, N};
    };
    return launch_decode(x, logits, expert_bias, score_fn, normalize ? 1 : 0, cl, w(W_gate, H, F), w(W_up, H, F),
                         w(W_down, F, H), T, H, F, E, k, topk_idx, topk_w, out, ws, (cudaStream_t)stream);
}

extern "C" moe_status_t moe_decode_mxfp8(const moe_bf16_t *x, const float *logits, const float *expert_bias,
                                         int score_fn, int normalize, float gate_lo, float gate_hi, float up_lo,
                                         float up_hi, const uint8_t *Wg_q, const uint8_t *Wg_sf, const uint8_t *Wu_q,
                                         const uint8_t *Wu_sf, const uint8_t *Wd_q, const uint8_t *Wd_sf, int64_t T,
                                         int H, int F, int E, int k, int32_t *topk_idx, float *topk_w,
                                         moe_bf16_t *out, void *ws, size_t ws_bytes, moe_stream_t stream) {
    MOE_NVTX_RANGE("moe_decode_mxfp8");
    using namespace moe;
    const Clamp cl{gate_lo, gate_hi, up_lo, up_hi};
    const moe_status_t st = check_decode(x, logits, score_fn, cl, T, H, F, E, k, topk_idx, topk_w, out);
    if (st != MOE_OK || T == 0) return st;
    if (!Wg_q || !Wg_sf || !Wu_q || !Wu_sf || !Wd_q || !Wd_sf) return MOE_ERR_INVALID_ARG;
    if (!all_aligned16({Wg_q, Wg_sf, Wu_q, Wu_sf, Wd_q, Wd_sf})) return MOE_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < moe_decode_workspace_bytes(T, H, F, E, k)) return MOE_ERR_WORKSPACE;
    return launch_decode(x, logits, expert_bias, score_fn, normalize ? 1 : 0, cl, WeightsMx{Wg_q, Wg_sf, H, F},
                         WeightsMx{Wu_q, Wu_sf, H, F}, WeightsMx{Wd_q, Wd_sf, F, H}, T, H, F, E, k, topk_idx, topk_w,
                         out, ws, (cudaStream_t)stream);
}
