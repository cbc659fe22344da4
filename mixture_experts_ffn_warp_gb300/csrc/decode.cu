// decode.cu -- a whole MoE layer for a few tokens in one kernel: routing, gate / up products,
// SwiGLU, down product and the weighted sum over the experts, on bf16 or MXFP8 expert weights.
//
//   idx, w = route(logits)                         (moe_route_topk / moe_route_topk_sigmoid)
//   h_tj   = silu(x_t Wg[e]) (x_t Wu[e]),  e = idx[t, j]
//   out_t  = bf16(sum_j w_tj h_tj Wd[e])           (fp32 sums, one rounding)
//
// With at most 64 tokens the call is bound by reading the hit experts' weights once.  The
// kernel is built around that stream: one persistent CTA per SM (a cooperative launch), the
// weights as the M = 128 operand of tcgen05.mma and the tokens as its N columns, so that a
// weight element is used from shared memory by all tokens at once and never passes through
// registers.
//
// Work split.  Phase 1 (gate / up) has a unit for each (expert, 128 features, K chunk), phase
// 2 (down) one for each (256 output columns, expert, K chunk); a unit is 32 KB (bf16) or 33 KB
// (MXFP8) of weights.  Each phase's units form one line that is cut into equal contiguous
// ranges, one per CTA, whatever the sizes and the routing.  Where a cut falls inside a tile
// the CTAs concerned leave fp32 partial sums in the workspace: in phase 1 the last one to
// arrive adds them (always in CTA order) and applies SwiGLU, in phase 2 each of them adds a
// slice of the output tile.  No sum's order depends on timing.
//
// Between the phases h must be complete, but not the weight stream: a producer warp loads
// weights as long as the ring has room, so that the stages filled ahead cover the time in
// which the last partial sums are joined.  A second producer warp loads the small operand
// (x, then h) and is the only one that waits.
//
// Precision.  On bf16 weights h enters phase 2 as two bf16 terms hi + lo in separate columns
// (N is padded to 16 anyway), so no rounding below fp32 precedes the output's.  On MXFP8
// weights x and h enter as two E4M3 terms each, the second of the first's remainder with its
// own block scales: x is then exact but for elements 2^-15 below their block's largest, h has
// a relative rms error of 7e-4 an element (one bf16 rounding: 1.6e-3).
//
// The down product's columns are drained per expert and only for the tokens routed to it: an
// expert's infinities reach no other token.
#include "common.cuh"
#include "mx.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr int kDecThreads = 256;     // warps: weights, x / h, MMA, idle, 4 epilogue
constexpr int kDecMaxStages = 8;
constexpr int kDecMaxCtas = 160;
constexpr int kDecMaxExperts = 1024;
constexpr int kABytes = 16384;       // one weight block: 128 output columns x 64 (bf16) / 128 (MXFP8) of K
constexpr int kSfBytes = 512;        // scale atom of 128 rows x 128 of K
constexpr uint32_t kDecSmemMax = 232448;

// Workspace: header, counters, then data.  The counters are zero between calls.
constexpr size_t kDecCtrBytes = 4096;
struct Counters {
    uint32_t exited;                 // CTAs that have finished
    uint32_t tiles_done;             // phase 1 tiles whose h is written
    uint32_t x_ready;                // CTAs whose share of x is quantised (MXFP8)
    uint32_t pad;
    uint32_t split1[kDecMaxCtas];    // arrivals at the tile that continues past CTA i's range
    uint32_t split2[kDecMaxCtas];
};
static_assert(sizeof(Counters) <= kDecCtrBytes, "counters");

struct DecArgs {
    const __nv_bfloat16 *x;
    const float *logits, *bias;
    int sigmoid, normalize;
    float glo, ghi, ulo, uhi;
    const uint8_t *wq[3], *wsf[3];   // MXFP8: gate, up, down codes and scales
    int T, T16, H, F, E, k;
    int32_t *topk_idx;
    float *topk_w;
    __nv_bfloat16 *out;
    uint32_t *err;
    Counters *ctr;
    uint8_t *xq;                     // MXFP8: x as blocks of the MMA operand
    uint8_t *hq;                     // h as blocks of the MMA operand
    float *part;                     // partial sums, [CTA][2][T16 * 256]
    int stages;
    uint32_t stage_bytes;
    uint32_t off_acc, off_meta;      // shared memory behind the ring
    int nbuf;                        // accumulator buffers in TMEM
};

// ---------------------------------------------------------------- small device helpers

__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap *m, uint64_t *bar, int c0, int c1,
                                                 int c2, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(sm100::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(pol)
        : "memory");
}

__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar,
                                               uint64_t pol) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(sm100::smem_u32(bar)), "l"(pol)
        : "memory");
}

// Global-memory writes of the generic proxy <-> bulk copies that read them.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Bounded wait for *p == want (as mbar_wait).
__device__ __forceinline__ bool wait_count(const uint32_t *p, uint32_t want, volatile int *abort, uint32_t *err,
                                           uint64_t limit_ns) {
    if (ld_acquire(p) == want) return true;
    const uint64_t t0 = sm100::globaltimer_ns();
    while (true) {
        if (ld_acquire(p) == want) return true;
        if (*abort) return false;
        if (sm100::globaltimer_ns() - t0 > limit_ns) {
            *abort = 1;
            raise_device_error(err, MOE_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// Barrier of the four epilogue warps; true when `ok` holds in every thread.
__device__ __forceinline__ bool epi_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}
// Waits for this thread's TMEM loads; the registers pass through, so that no use moves ahead.
__device__ __forceinline__ void tmem_ld_wait8(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}

__device__ __forceinline__ uint32_t order_key(float v) {   // larger ranks first; NaN ranks below -inf; 0 = taken
    if (v != v) return 1u;
    const uint32_t b = __float_as_uint(v == 0.0f ? 0.0f : v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Contiguous range i of n equal shares of U units (every share non-empty when n <= U).
__device__ __forceinline__ int64_t share_begin(int64_t U, int i, int n) { return U * i / n; }
// The share that unit u falls in.
__device__ __forceinline__ int share_of(int64_t u, int64_t U, int n) { return (int)(((u + 1) * n - 1) / U); }

// E4M3 code of v / 2^X and the remainder v - code * 2^X; what is not finite becomes a NaN code.
__device__ __forceinline__ uint8_t e4m3_term(float v, int X, float &rem) {
    const __nv_fp8_storage_t c = __nv_cvt_float_to_fp8(v * mx::inv_pow2(X), __NV_SATFINITE, __NV_E4M3);
    __nv_fp8_e4m3 f;
    f.__x = c;
    rem = v - ldexpf((float)f, X);
    const bool finite = fabsf(v) <= 3.402823466e38f;
    if (!finite) rem = 0.0f;
    return finite ? (uint8_t)c : (uint8_t)0x7F;
}

// v of 32 lanes (one MX block) as two E4M3 terms: codes and scale bytes.
__device__ __forceinline__ void two_terms(float v, uint8_t (&code)[2], uint8_t (&sf)[2]) {
    float rem = v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(rem)));
        const int X = mx::scale_exp(__uint_as_float(amax));
        float next;
        code[i] = e4m3_term(rem, X, next);
        sf[i] = (uint8_t)(X + 127);
        rem = next;
    }
}

// Byte of (row n, byte column c) in a block of 128-byte rows under the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(uint32_t n, uint32_t c) { return n * 128 + ((c & ~15u) ^ ((n & 7) << 4)) + (c & 15u); }
// Byte of (row n, 32-block kb) in a scale atom.
__device__ __forceinline__ uint32_t sf_byte(uint32_t n, uint32_t kb) { return (n % 32) * 16 + (n / 32) * 4 + kb; }

__device__ __forceinline__ float swiglu(float g, float u, const DecArgs &a) {
    g = fminf(fmaxf(g, a.glo), a.ghi);
    u = fminf(fmaxf(u, a.ulo), a.uhi);
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// ---------------------------------------------------------------- the kernel

// Units of this CTA in one phase, cut at tile ends: next() gives (tile, first chunk, chunks).
struct Segments {
    int64_t u, end;
    int per;   // chunks per tile
    __device__ bool next(int64_t &tile, int &k0, int &n) {
        if (u >= end) return false;
        tile = u / per;
        k0 = (int)(u - tile * per);
        const int64_t left = end - u;
        n = left < per - k0 ? (int)left : per - k0;
        u += n;
        return true;
    }
};

template <bool MX>
__global__ void __launch_bounds__(kDecThreads, 1)
decode_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG,
              const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmD, const DecArgs a) {
    constexpr int KC = MX ? 128 : 64;                 // K elements of a chunk (128 bytes of an operand row)
    constexpr uint32_t B_OFF = 2 * kABytes + (MX ? 2 * kSfBytes : 0);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t full_w[kDecMaxStages], full_b[kDecMaxStages], empty[kDecMaxStages], tfull[2], tempty[2], drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_active_n;
    __shared__ volatile int s_abort;
    __shared__ uint32_t s_last;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem_base = sm100::smem_u32(smem);
    const int G = (int)gridDim.x, cta = (int)blockIdx.x;
    const int R = a.T * a.k, amax = R < a.E ? R : a.E;
    uint64_t *s_mask = reinterpret_cast<uint64_t *>(smem + a.off_meta);   // [E] tokens of each expert, a bit each
    float *s_w = reinterpret_cast<float *>(s_mask + a.E);                 // [T * k]
    int *s_row0 = reinterpret_cast<int *>(s_w + R);                       // [active] padded rows before the expert
    uint16_t *s_active = reinterpret_cast<uint16_t *>(s_row0 + amax);     // [active] expert ids, ascending
    uint16_t *s_idx = s_active + amax;                                    // [T * k]
    const uint64_t limit = device_wait_limit(a.err);
    volatile int *abort = &s_abort;

    // ------------------------------------------------------------ set-up
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            sm100::mbar_init(&full_w[s], 1);
            sm100::mbar_init(&full_b[s], 1);
            sm100::mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(&tfull[i], 1);
            sm100::mbar_init(&tempty[i], 128);
        }
        sm100::mbar_init(&drain, 1);
        s_abort = 0;
        sm100::fence_mbar_init();
    }
    if (warp == 2) {
        sm100::tmem_alloc(&s_tmem, 512);
        sm100::tmem_relinquish();
    }
    for (int e = threadIdx.x; e < a.E; e += kDecThreads) s_mask[e] = 0;

    if constexpr (MX) {
        // this CTA's share of x: blocks of 32 elements, a warp each, into [H / 128] blocks of
        // 2 T16 operand rows (first terms, then second) and a scale atom
        const int nb = a.H / 32;
        const uint32_t blk_bytes = (uint32_t)a.T16 * 256 + kSfBytes;
        for (int b = cta * 8 + warp; b < a.T * nb; b += G * 8) {
            const int t = b / nb, kb = b - t * nb;
            uint8_t code[2], sf[2];
            two_terms(__bfloat162float(a.x[(int64_t)t * a.H + kb * 32 + lane]), code, sf);
            uint8_t *blk = a.xq + (size_t)(kb / 4) * blk_bytes;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t n = t + i * a.T16;
                blk[sw128(n, (kb & 3) * 32 + lane)] = code[i];
                if (lane == 0) blk[a.T16 * 256 + sf_byte(n, kb & 3)] = sf[i];
            }
        }
        fence_proxy_async_global();
        __threadfence();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    if (MX && threadIdx.x == 0) atomicAdd(&a.ctr->x_ready, 1u);

    // ------------------------------------------------------------ routing, by every CTA for itself
    {
        uint32_t *key = reinterpret_cast<uint32_t *>(smem) + warp * a.E;   // the ring is not in use yet
        for (int t = warp; t < a.T; t += 8) {
            const float *row = a.logits + (int64_t)t * a.E;
            uint32_t bk = 0, be = 0;                       // this lane's best key and its expert
            for (int e = lane; e < a.E; e += 32) {
                float v = __ldg(row + e);
                if (a.sigmoid) {
                    v = 1.0f / (1.0f + expf(-v));
                    if (a.bias) v += __ldg(a.bias + e);
                }
                const uint32_t kk = order_key(v);
                key[e] = kk;
                if (kk > bk) { bk = kk; be = e; }
            }
            uint32_t mine = 0;                             // lane j keeps the expert of slot j
            for (int j = 0; j < a.k; ++j) {
                const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, bk);
                const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, bk == top ? be : 0xFFFFFFFFu);
                if (lane == j) mine = e;
                if ((e & 31) == (uint32_t)lane) {          // the winner's lane looks again
                    key[e] = 0;
                    bk = 0;
                    for (int i = lane; i < a.E; i += 32)
                        if (key[i] > bk) { bk = key[i]; be = i; }
                }
            }
            float w = 0.0f;
            if (a.sigmoid) {
                float sc = lane < a.k ? 1.0f / (1.0f + expf(-__ldg(row + mine))) : 0.0f;
                if (sc != sc) sc = 0.0f;                   // a NaN logit scores 0
                float S = sc;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) S += __shfl_xor_sync(0xFFFFFFFFu, S, off);
                w = a.normalize ? sc / (S + 1e-20f) : sc;
            } else {
                const float l = lane < a.k ? __ldg(row + mine) : 0.0f;
                const float l0 = __shfl_sync(0xFFFFFFFFu, l, 0);
                const float ex = (lane < a.k && l0 != -INFINITY) ? expf(l - l0) : 0.0f;
                float S = ex;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) S += __shfl_xor_sync(0xFFFFFFFFu, S, off);
                w = l0 == -INFINITY ? 0.0f : ex / S;
            }
            if (lane < a.k) {
                s_idx[t * a.k + lane] = (uint16_t)mine;
                s_w[t * a.k + lane] = w;
                atomicOr(reinterpret_cast<unsigned long long *>(&s_mask[mine]), 1ull << t);
                if (cta == 0) {
                    a.topk_idx[t * a.k + lane] = (int32_t)mine;
                    a.topk_w[t * a.k + lane] = w;
                }
            }
        }
    }
    __syncthreads();
    if (warp == 0) {
        // the experts that are hit, ascending, and the 16-row blocks of h before each
        int n = 0, rows = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const uint64_t m = e < a.E ? s_mask[e] : 0;
            const uint32_t hit = __ballot_sync(0xFFFFFFFFu, m != 0);
            if (!hit) continue;
            int c = (__popcll(m) + 15) & ~15, incl = c;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
                if (lane >= off) incl += o;
            }
            if (m) {
                const int i = n + __popc(hit & ((1u << lane) - 1));
                s_active[i] = (uint16_t)e;
                s_row0[i] = rows + incl - c;
            }
            n += __popc(hit);
            rows += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (lane == 0) s_active_n = n;
    }
    sm100::fence_proxy_async_smem();   // the ring's bytes were written as scratch above
    __syncthreads();

    const int A = s_active_n;
    const uint32_t tmem = s_tmem;
    const int FT = a.F / 128, K1 = a.H / KC, K2 = a.F / KC, NT = (a.H + 255) / 256;
    const int64_t U1 = (int64_t)A * FT * K1, U2 = (int64_t)NT * A * K2;
    const int G1 = U1 < G ? (int)U1 : G, G2 = U2 < G ? (int)U2 : G;
    // phase 2 tiles here are (output tile, expert) pairs: nt = tile / A, expert = tile % A
    const Segments none{0, 0, 1};
    const Segments ph1 = cta < G1 ? Segments{share_begin(U1, cta, G1), share_begin(U1, cta + 1, G1), K1} : none;
    const Segments ph2 = cta < G2 ? Segments{share_begin(U2, cta, G2), share_begin(U2, cta + 1, G2), K2} : none;
    const uint32_t row_bytes = MX ? 2u * a.F : 4u * a.F;   // bytes of h per 16-row-block row, both terms
    auto rows16 = [&](int ai) { return (__popcll(s_mask[s_active[ai]]) + 15) & ~15; };
    auto h_block = [&](int ai, int c16, int kc) {          // block kc of the expert's h
        const uint32_t bytes = (uint32_t)c16 * 256 + (MX ? kSfBytes : 0);
        return a.hq + (size_t)s_row0[ai] * row_bytes + (MX ? (size_t)ai * FT * kSfBytes : 0) + (size_t)kc * bytes;
    };

    if (warp == 0) {
        // ======================================================== weights
        if (lane == 0) {
            const uint64_t pol = evict_first_policy();
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            int64_t tile;
            int k0, n;
            for (int ph = 0; ph < 2 && ok; ++ph) {
                Segments sg = ph == 0 ? ph1 : ph2;
                while (ok && sg.next(tile, k0, n)) {
                    const int ai = ph == 0 ? (int)(tile / FT) : (int)(tile % A);
                    const int e = s_active[ai];
                    const int col = ph == 0 ? (int)(tile - (int64_t)ai * FT) : 2 * (int)(tile / A);   // 128-column block
                    const bool two = ph == 0 || (col + 1) * 128 < a.H;
                    const uint32_t bytes = (two ? 2u : 1u) * (kABytes + (MX ? kSfBytes : 0));
                    for (int kc = k0; kc < k0 + n; ++kc) {
                        if (!sm100::mbar_wait(&empty[stage], phase ^ 1u, abort, a.err, limit)) { ok = false; break; }
                        const uint32_t sa = smem_base + stage * a.stage_bytes;
                        uint64_t *fb = &full_w[stage];
                        sm100::mbar_arrive_expect_tx(fb, bytes);
                        if constexpr (MX) {
                            const int nblk = (ph == 0 ? a.F : a.H) / 128, K = ph == 0 ? K1 : K2;
                            const int64_t blk = ((int64_t)e * K + kc) * nblk + col;
                            for (int i = 0; i < (two ? 2 : 1); ++i) {
                                const int w = ph == 0 ? i : 2;
                                const int64_t b = ph == 0 ? blk : blk + i;
                                bulk_load_hint(sa + i * kABytes, a.wq[w] + b * kABytes, kABytes, fb, pol);
                                bulk_load_hint(sa + 2 * kABytes + i * kSfBytes, a.wsf[w] + b * kSfBytes, kSfBytes, fb, pol);
                            }
                        } else if (ph == 0) {
                            const int row = e * a.H + kc * KC;
                            tma_load_3d_hint(sa, &tmG, fb, 0, row, 2 * col, pol);
                            tma_load_3d_hint(sa + kABytes, &tmU, fb, 0, row, 2 * col, pol);
                        } else {
                            const int row = e * a.F + kc * KC;
                            tma_load_3d_hint(sa, &tmD, fb, 0, row, 2 * col, pol);
                            if (two) tma_load_3d_hint(sa + kABytes, &tmD, fb, 0, row, 2 * col + 2, pol);
                        }
                        ++issued;
                        if (++stage == a.stages) { stage = 0; phase ^= 1u; }
                    }
                }
            }
            if (!ok) {   // the copies already issued land before the CTA exits
                for (int i = 0; i < a.stages && i < issued; ++i) {
                    if (--stage < 0) { stage = a.stages - 1; phase ^= 1u; }
                    int dummy = 0;
                    sm100::mbar_wait(&full_w[stage], phase, &dummy, nullptr, 10000000ull);
                }
            }
        }
    } else if (warp == 1) {
        // ======================================================== x, then h
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            int64_t tile;
            int k0, n;
            for (int ph = 0; ph < 2 && ok; ++ph) {
                Segments sg = ph == 0 ? ph1 : ph2;
                if (sg.u >= sg.end) continue;
                if (MX && ph == 0) ok = wait_count(&a.ctr->x_ready, (uint32_t)G, abort, a.err, limit);
                if (ph == 1) ok = wait_count(&a.ctr->tiles_done, (uint32_t)(A * FT), abort, a.err, limit);
                fence_proxy_async_global();
                while (ok && sg.next(tile, k0, n)) {
                    const int ai = (int)(tile % A);        // phase 2's expert
                    const int c16 = ph == 0 ? 0 : rows16(ai);
                    for (int kc = k0; kc < k0 + n; ++kc) {
                        if (!sm100::mbar_wait(&empty[stage], phase ^ 1u, abort, a.err, limit)) { ok = false; break; }
                        const uint32_t sb = smem_base + stage * a.stage_bytes + B_OFF;
                        uint64_t *fb = &full_b[stage];
                        if (ph == 0) {
                            if constexpr (MX) {
                                const uint32_t bytes = (uint32_t)a.T16 * 256 + kSfBytes;
                                sm100::mbar_arrive_expect_tx(fb, bytes);
                                sm100::bulk_load(sb, a.xq + (size_t)kc * bytes, bytes, fb);
                            } else {
                                sm100::mbar_arrive_expect_tx(fb, (uint32_t)a.T16 * 128);
                                sm100::tma_load_2d(sb, &tmX, fb, kc * KC, 0);
                            }
                        } else {
                            const uint32_t bytes = (uint32_t)c16 * 256 + (MX ? kSfBytes : 0);
                            sm100::mbar_arrive_expect_tx(fb, bytes);
                            sm100::bulk_load(sb, h_block(ai, c16, kc), bytes, fb);
                        }
                        ++issued;
                        if (++stage == a.stages) { stage = 0; phase ^= 1u; }
                    }
                }
            }
            if (!ok) {
                for (int i = 0; i < a.stages && i < issued; ++i) {
                    if (--stage < 0) { stage = a.stages - 1; phase ^= 1u; }
                    int dummy = 0;
                    sm100::mbar_wait(&full_b[stage], phase, &dummy, nullptr, 10000000ull);
                }
            }
        }
    } else if (warp == 2) {
        // ======================================================== MMA issuer
        int stage = 0, buf = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true, issued_any = false;
        int64_t tile;
        int k0, n;
        const uint32_t half = 2u * a.T16;                  // columns between the two accumulators of a buffer
        for (int ph = 0; ph < 2 && ok; ++ph) {
            Segments sg = ph == 0 ? ph1 : ph2;
            while (ok && sg.next(tile, k0, n)) {
                const int N = ph == 0 ? (MX ? 2 * a.T16 : a.T16) : 2 * rows16((int)(tile % A));
                const bool two = ph == 0 || (2 * (int)(tile / A) + 1) * 128 < a.H;
                const uint32_t idesc = MX ? sm100::idesc_mxf8(128, N) : sm100::idesc_bf16(128, N, true, false);
                const bool got = sm100::mbar_wait(&tempty[buf], acc_phase ^ 1u, abort, a.err, limit);
                if (__any_sync(0xFFFFFFFFu, !got)) { ok = false; break; }
                sm100::tc_fence_after();
                const uint32_t d0 = tmem + (uint32_t)buf * 2 * half, d1 = d0 + half;
                for (int i = 0; i < n; ++i) {
                    const bool got_w = sm100::mbar_wait(&full_w[stage], phase, abort, a.err, limit) &&
                                       sm100::mbar_wait(&full_b[stage], phase, abort, a.err, limit);
                    if (__any_sync(0xFFFFFFFFu, !got_w)) { ok = false; break; }
                    sm100::tc_fence_after();
                    const uint32_t sa = smem_base + stage * a.stage_bytes;
                    const uint64_t ad = MX ? sm100::sdesc_sw128(sa, 16, 1024) : sm100::sdesc_sw128(sa, 8192, 1024);
                    const uint64_t bd = sm100::sdesc_sw128(sa + B_OFF, 16, 1024);
                    constexpr uint64_t A_STEP = MX ? (32 >> 4) : (2048 >> 4);   // a K step of 32 / 16 elements
                    if (sm100::elect_one()) {
                        if constexpr (MX) {
                            const uint32_t tsf = tmem + (uint32_t)a.nbuf * 2 * half + stage * 12;
                            sm100::tmem_cp_32x128b_x4(tsf, sm100::sdesc_plain(sa + 2 * kABytes));
                            if (two) sm100::tmem_cp_32x128b_x4(tsf + 4, sm100::sdesc_plain(sa + 2 * kABytes + kSfBytes));
                            sm100::tmem_cp_32x128b_x4(tsf + 8, sm100::sdesc_plain(sa + B_OFF + N * 128));
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                const uint32_t id = idesc | sm100::idesc_sf_ids(kk, kk);
                                sm100::mma_mxf8(d0, ad + kk * A_STEP, bd + kk * 2, id, tsf, tsf + 8, (i | kk) != 0);
                                if (two)
                                    sm100::mma_mxf8(d1, ad + (kABytes >> 4) + kk * A_STEP, bd + kk * 2, id, tsf + 4,
                                                    tsf + 8, (i | kk) != 0);
                            }
                        } else {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                sm100::mma_bf16(d0, ad + kk * A_STEP, bd + kk * 2, idesc, (i | kk) != 0);
                                if (two)
                                    sm100::mma_bf16(d1, ad + (kABytes >> 4) + kk * A_STEP, bd + kk * 2, idesc,
                                                    (i | kk) != 0);
                            }
                        }
                        sm100::mma_commit(&empty[stage]);
                    }
                    issued_any = true;
                    __syncwarp();
                    if (++stage == a.stages) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                if (sm100::elect_one()) sm100::mma_commit(&tfull[buf]);
                __syncwarp();
                if (++buf == a.nbuf) { buf = 0; acc_phase ^= 1u; }
            }
        }
        if (!ok && issued_any && sm100::elect_one()) {
            // the MMAs already issued finish before TMEM is released
            sm100::mma_commit(&drain);
            int dummy = 0;
            sm100::mbar_wait(&drain, 0, &dummy, nullptr, 10000000ull);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ======================================================== epilogue
        const int col = (warp - 4) * 32 + lane;            // TMEM lane: feature or output column of a 128 block
        const uint32_t lane_base = (uint32_t)(warp - 4) << 21;   // lane quarter in bits 16..31
        const bool lead = threadIdx.x == 128;
        const uint32_t half = 2u * a.T16;
        const int slot_floats = a.T16 * 256;
        int buf = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        int64_t tile;
        int k0, n;

        // h of token i (of the expert's c16 padded rows), features 128 ft + col
        auto store_h = [&](int ai, int c16, int ft, int i, float v) {
            if constexpr (MX) {
                uint8_t code[2], sf[2];
                two_terms(v, code, sf);
                uint8_t *blk = h_block(ai, c16, ft);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t r = i + m * c16;
                    blk[sw128(r, col)] = code[m];
                    if (lane == 0) blk[c16 * 256 + sf_byte(r, warp - 4)] = sf[m];
                }
            } else {
                const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                const float hf = __bfloat162float(hi);
                const __nv_bfloat16 lo = __float2bfloat16_rn(isinf(hf) ? 0.0f : v - hf);
                uint8_t *blk = h_block(ai, c16, 2 * ft + col / 64);
                *reinterpret_cast<__nv_bfloat16 *>(blk + sw128(i, (col % 64) * 2)) = hi;
                *reinterpret_cast<__nv_bfloat16 *>(blk + sw128(i + c16, (col % 64) * 2)) = lo;
            }
        };
        // the tile's h is written by all four warps: visible to the bulk copies, then counted
        auto tile_done = [&]() {
            fence_proxy_async_global();
            __threadfence();
            epi_all(true);
            if (lead) atomicAdd(&a.ctr->tiles_done, 1u);
        };

        // ---------------- phase 1
        Segments sg = ph1;
        while (ok && sg.next(tile, k0, n)) {
            const int ai = (int)(tile / FT), ft = (int)(tile - (int64_t)ai * FT);
            const int e = s_active[ai], c16 = rows16(ai);
            const uint64_t mask = s_mask[e];
            const int cnt = __popcll(mask);
            const bool whole = n == K1;
            const int slot = tile == ph1.u / K1 ? 0 : 1;   // the CTA's first tile, or its last
            float *part = a.part + ((size_t)cta * 2 + slot) * slot_floats;
            ok = epi_all(sm100::mbar_wait(&tfull[buf], acc_phase, abort, a.err, limit));
            if (!ok) break;
            sm100::tc_fence_after();
            const uint32_t dg = tmem + lane_base + (uint32_t)buf * 2 * half, du = dg + half;
            uint64_t m = mask;
            for (int i0 = 0; i0 < cnt; i0 += 8) {
                uint32_t g[8] = {}, u[8] = {}, g2[8] = {}, u2[8] = {};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i0 + j < cnt) {
                        const uint32_t t = __ffsll((long long)m) - 1;
                        m &= m - 1;
                        tmem_ld1(dg + t, g[j]);
                        tmem_ld1(du + t, u[j]);
                        if constexpr (MX) {
                            tmem_ld1(dg + a.T16 + t, g2[j]);
                            tmem_ld1(du + a.T16 + t, u2[j]);
                        }
                    }
                tmem_ld_wait8(g);
                tmem_ld_wait8(u);
                if constexpr (MX) {
                    tmem_ld_wait8(g2);
                    tmem_ld_wait8(u2);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i0 + j < cnt) {
                        float gv = __uint_as_float(g[j]), uv = __uint_as_float(u[j]);
                        if constexpr (MX) {
                            gv += __uint_as_float(g2[j]);
                            uv += __uint_as_float(u2[j]);
                        }
                        if (whole) {
                            store_h(ai, c16, ft, i0 + j, swiglu(gv, uv, a));
                        } else {
                            part[(i0 + j) * 256 + col] = gv;
                            part[(i0 + j) * 256 + 128 + col] = uv;
                        }
                    }
            }
            sm100::tc_fence_before();
            sm100::mbar_arrive(&tempty[buf]);
            if (++buf == a.nbuf) { buf = 0; acc_phase ^= 1u; }
            if (!whole) {
                // partial sums of CTAs c0..c1; the last to arrive adds them in that order
                const int c0 = share_of(tile * K1, U1, G1), c1 = share_of(tile * K1 + K1 - 1, U1, G1);
                __threadfence();
                epi_all(true);
                if (lead) {
                    const uint32_t old = atomicAdd(&a.ctr->split1[c0], 1u);
                    s_last = old == (uint32_t)(c1 - c0);
                    if (s_last) a.ctr->split1[c0] = 0;
                    __threadfence();
                }
                epi_all(true);
                if (!s_last) continue;
                __threadfence();
                for (int i = 0; i < cnt; ++i) {
                    float gv = 0.0f, uv = 0.0f;
                    for (int c = c0; c <= c1; ++c) {
                        const int cs = tile == share_begin(U1, c, G1) / K1 ? 0 : 1;
                        const float *p = a.part + ((size_t)c * 2 + cs) * slot_floats + i * 256 + col;
                        gv += __ldcg(p);
                        uv += __ldcg(p + 128);
                    }
                    store_h(ai, c16, ft, i, swiglu(gv, uv, a));
                }
            }
            tile_done();
        }

        // ---------------- phase 2
        float *acc = reinterpret_cast<float *>(smem + a.off_acc);   // [T][256]; a thread's two columns are its own
        sg = ph2;
        int64_t cur = -1;                                  // output tile that acc belongs to
        const int64_t per_nt = (int64_t)A * K2;
        const int64_t first_nt = ph2.u / per_nt;
        // leaves the output tile `nt`: written out, or left to the others as a partial sum
        auto flush = [&](int64_t nt) {
            const int cols = a.H - (int)nt * 256 < 256 ? 128 : 256;
            const int c0 = share_of(nt * per_nt, U2, G2), c1 = share_of(nt * per_nt + per_nt - 1, U2, G2);
            if (c0 == c1) {
                for (int t = 0; t < a.T; ++t) {
                    __nv_bfloat16 *o = a.out + (int64_t)t * a.H + nt * 256 + col;
                    o[0] = __float2bfloat16_rn(acc[t * 256 + col]);
                    if (cols == 256) o[128] = __float2bfloat16_rn(acc[t * 256 + 128 + col]);
                }
                return;
            }
            float *part = a.part + ((size_t)cta * 2 + (nt == first_nt ? 0 : 1)) * slot_floats;
            for (int t = 0; t < a.T; ++t) {
                part[t * 256 + col] = acc[t * 256 + col];
                if (cols == 256) part[t * 256 + 128 + col] = acc[t * 256 + 128 + col];
            }
            __threadfence();
            epi_all(true);
            if (lead) atomicAdd(&a.ctr->split2[c0], 1u);
        };
        while (ok && sg.next(tile, k0, n)) {
            const int64_t nt = tile / A;
            const int ai = (int)(tile - nt * A), e = s_active[ai], c16 = rows16(ai);
            const bool two = (2 * (int)nt + 1) * 128 < a.H;
            if (nt != cur) {
                if (cur >= 0) flush(cur);
                cur = nt;
                for (int t = 0; t < a.T; ++t) {
                    acc[t * 256 + col] = 0.0f;
                    acc[t * 256 + 128 + col] = 0.0f;
                }
            }
            ok = epi_all(sm100::mbar_wait(&tfull[buf], acc_phase, abort, a.err, limit));
            if (!ok) break;
            sm100::tc_fence_after();
            const uint32_t d0 = tmem + lane_base + (uint32_t)buf * 2 * half, d1 = d0 + half;
            uint64_t m = s_mask[e];
            const int cnt = __popcll(m);
            for (int i0 = 0; i0 < cnt; i0 += 8) {
                uint32_t y0[8] = {}, y1[8] = {}, z0[8] = {}, z1[8] = {};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i0 + j < cnt) {
                        const uint32_t i = i0 + j;
                        tmem_ld1(d0 + i, y0[j]);
                        tmem_ld1(d0 + c16 + i, z0[j]);
                        if (two) {
                            tmem_ld1(d1 + i, y1[j]);
                            tmem_ld1(d1 + c16 + i, z1[j]);
                        }
                    }
                tmem_ld_wait8(y0);
                tmem_ld_wait8(z0);
                tmem_ld_wait8(y1);
                tmem_ld_wait8(z1);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i0 + j < cnt) {
                        const int t = __ffsll((long long)m) - 1;
                        m &= m - 1;
                        const uint32_t at = __ballot_sync(
                            0xFFFFFFFFu, lane < a.k && s_idx[t * a.k + (lane < a.k ? lane : 0)] == e);
                        const float w = s_w[t * a.k + __ffs(at) - 1];
                        acc[t * 256 + col] += w * (__uint_as_float(y0[j]) + __uint_as_float(z0[j]));
                        acc[t * 256 + 128 + col] += w * (__uint_as_float(y1[j]) + __uint_as_float(z1[j]));
                    }
            }
            sm100::tc_fence_before();
            sm100::mbar_arrive(&tempty[buf]);
            if (++buf == a.nbuf) { buf = 0; acc_phase ^= 1u; }
        }
        if (ok && cur >= 0) {
            flush(cur);
            // the CTA's split tiles, its first and its last: each contributor adds a slice of the tile
            for (int i = 0; i < 2 && ok; ++i) {
                const int64_t nt = i == 0 ? first_nt : cur;
                if (i == 1 && cur == first_nt) break;
                const int c0 = share_of(nt * per_nt, U2, G2), c1 = share_of(nt * per_nt + per_nt - 1, U2, G2);
                if (c0 == c1) continue;
                bool got = true;
                if (lead) got = wait_count(&a.ctr->split2[c0], (uint32_t)(c1 - c0 + 1), abort, a.err, limit);
                ok = epi_all(got);
                if (!ok) break;
                __threadfence();
                const int quads = a.H - (int)nt * 256 < 256 ? 32 : 64, total = a.T * quads;   // 4 columns each
                const int nc = c1 - c0 + 1, rank = cta - c0;
                for (int v = total * rank / nc + col; v < total * (rank + 1) / nc; v += 128) {
                    const int t = v / quads, q = v - t * quads;
                    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int c = c0; c <= c1; ++c) {
                        const int cs = nt == share_begin(U2, c, G2) / per_nt ? 0 : 1;
                        const float4 p = __ldcg(reinterpret_cast<const float4 *>(
                            a.part + ((size_t)c * 2 + cs) * slot_floats + t * 256 + q * 4));
                        s.x += p.x;
                        s.y += p.y;
                        s.z += p.z;
                        s.w += p.w;
                    }
                    __nv_bfloat162 o[2] = {__floats2bfloat162_rn(s.x, s.y), __floats2bfloat162_rn(s.z, s.w)};
                    *reinterpret_cast<uint2 *>(a.out + (int64_t)t * a.H + nt * 256 + q * 4) =
                        *reinterpret_cast<const uint2 *>(o);
                }
            }
        }
    }

    // ------------------------------------------------------------ teardown
    sm100::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        __syncwarp();
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&a.ctr->exited, 1u) == (uint32_t)G - 1) {   // nobody waits any more: zero for the next call
            for (int i = 0; i < G; ++i) a.ctr->split2[i] = 0;
            a.ctr->tiles_done = 0;
            a.ctr->x_ready = 0;
            a.ctr->exited = 0;
            __threadfence();
        }
    }
}

// ---------------------------------------------------------------- host

struct Clamp {
    float glo, ghi, ulo, uhi;
};

struct DecLayout {
    size_t xq, hq, part, total;
};

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }
int tokens16(int64_t T) { return (int)((T + 15) / 16 * 16); }

DecLayout decode_layout(int64_t T, int H, int F, int E, int k) {
    const size_t T16 = (size_t)tokens16(T), R = (size_t)(T * k), act = R < (size_t)E ? R : (size_t)E;
    // rows of h padded to 16 per expert hit, two terms of 2 bytes (bf16); the MXFP8 blocks and atoms need less
    const size_t rows = R + 15 * act < act * T16 ? R + 15 * act : act * T16;
    DecLayout l;
    l.xq = kWsHeaderBytes + kDecCtrBytes;
    l.hq = l.xq + round_up((size_t)H / 128 * (T16 * 256 + kSfBytes), 1024);
    l.part = l.hq + round_up(rows * (size_t)F * 4, 1024);
    l.total = l.part + (size_t)kDecMaxCtas * 2 * T16 * 256 * sizeof(float);
    return l;
}

bool decode_sizes_ok(int64_t T, int H, int F, int E, int k) {
    return T >= 0 && T <= MOE_DECODE_MAX_TOKENS && H >= 128 && F >= 128 && H % 128 == 0 && F % 128 == 0 && E >= 1 &&
           E <= kDecMaxExperts && k >= 1 && k <= 32 && k <= E && (int64_t)E * H < (1ll << 31) &&
           (int64_t)E * F < (1ll << 31);
}

moe_status_t check_decode(const void *x, const void *logits, int score_fn, const Clamp &cl, int64_t T, int H, int F,
                          int E, int k, const void *topk_idx, const void *topk_w, const void *out) {
    if (T < 0 || H < 1 || F < 1) return MOE_ERR_INVALID_ARG;
    if (score_fn != MOE_SCORE_SOFTMAX && score_fn != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (!(cl.glo <= cl.ghi) || !(cl.ulo <= cl.uhi)) return MOE_ERR_INVALID_ARG;   // empty, or a NaN bound
    if (!decode_sizes_ok(T, H, F, E, k)) return MOE_ERR_UNSUPPORTED;
    if (T > 0 && (!x || !logits || !topk_idx || !topk_w || !out)) return MOE_ERR_INVALID_ARG;
    if (!all_aligned16({x, out})) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

template <bool MX>
moe_status_t launch_decode(DecArgs a, const moe_bf16_t *const (&W)[3], void *ws, cudaStream_t s) {
    CUtensorMap tm[4] = {};
    if (!MX) {
        const int H = a.H, F = a.F;
        if (!tmap_bf16_2d(&tm[0], a.x, H, a.T, H, 64, a.T16) ||
            !tmap_bf16_col_chunks(&tm[1], W[0], F, (uint64_t)a.E * H, F, 64) ||
            !tmap_bf16_col_chunks(&tm[2], W[1], F, (uint64_t)a.E * H, F, 64) ||
            !tmap_bf16_col_chunks(&tm[3], W[2], H, (uint64_t)a.E * F, H, 64))
            return MOE_ERR_CUDA;
    }
    const DecLayout l = decode_layout(a.T, a.H, a.F, a.E, a.k);
    char *base = static_cast<char *>(ws);
    a.err = ws_error_word(ws);
    a.ctr = reinterpret_cast<Counters *>(base + kWsHeaderBytes);
    a.xq = reinterpret_cast<uint8_t *>(base + l.xq);
    a.hq = reinterpret_cast<uint8_t *>(base + l.hq);
    a.part = reinterpret_cast<float *>(base + l.part);

    const int R = a.T * a.k, act = R < a.E ? R : a.E;
    const uint32_t b_bytes = (uint32_t)a.T16 * 256 + (MX ? 3 * kSfBytes : 0);   // x or h, all scale atoms
    a.stage_bytes = (uint32_t)round_up(2 * kABytes + b_bytes, 1024);
    const uint32_t acc = (uint32_t)a.T16 * 1024;
    const uint32_t meta = (uint32_t)a.E * 8 + R * 4 + act * 4 + act * 2 + R * 2;
    const uint32_t fixed = acc + (uint32_t)round_up(meta, 16) + 1024 /* alignment */ + 1024 /* static */;
    int stages = (int)((kDecSmemMax - fixed) / a.stage_bytes);
    a.stages = stages < kDecMaxStages ? stages : kDecMaxStages;
    if (a.stages < 2) return MOE_ERR_UNSUPPORTED;
    a.off_acc = a.stages * a.stage_bytes;
    a.off_meta = a.off_acc + acc;
    a.nbuf = 8 * a.T16 + (MX ? 12 * a.stages : 0) <= 512 ? 2 : 1;
    const uint32_t smem = a.off_meta + (uint32_t)round_up(meta, 16) + 1024;

    static PerDeviceOnce once;
    int sms = 0;
    const moe_status_t st = once.get(
        [](int *v) {
            if (cudaFuncSetAttribute(decode_kernel<MX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)kDecSmemMax - 1024) != cudaSuccess)
                return MOE_ERR_CUDA;
            *v = device_sm_count();
            return MOE_OK;
        },
        &sms);
    if (st != MOE_OK) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(sms < kDecMaxCtas ? sms : kDecMaxCtas));
    cfg.blockDim = dim3(kDecThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;   // the CTAs wait for one another's partial sums and h
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, decode_kernel<MX>, tm[0], tm[1], tm[2], tm[3], a) != cudaSuccess) {
        (void)cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return launch_status();
}

DecArgs decode_args(const moe_bf16_t *x, const float *logits, const float *bias, int score_fn, int normalize,
                    const Clamp &cl, int64_t T, int H, int F, int E, int k, int32_t *topk_idx, float *topk_w,
                    moe_bf16_t *out) {
    DecArgs a{};
    a.x = reinterpret_cast<const __nv_bfloat16 *>(x);
    a.logits = logits;
    a.bias = bias;
    a.sigmoid = score_fn == MOE_SCORE_SIGMOID;
    a.normalize = normalize;
    a.glo = cl.glo;
    a.ghi = cl.ghi;
    a.ulo = cl.ulo;
    a.uhi = cl.uhi;
    a.T = (int)T;
    a.T16 = tokens16(T);
    a.H = H;
    a.F = F;
    a.E = E;
    a.k = k;
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    a.out = reinterpret_cast<__nv_bfloat16 *>(out);
    return a;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_decode_workspace_bytes(int64_t T, int H, int F, int E, int k) {
    if (!moe::decode_sizes_ok(T, H, F, E, k)) return 0;
    return moe::decode_layout(T, H, F, E, k).total;
}

extern "C" moe_status_t moe_decode_workspace_init(void *ws, size_t ws_bytes, moe_stream_t stream) {
    const size_t n = moe::kWsHeaderBytes + moe::kDecCtrBytes;
    if (!ws || ws_bytes < n) return MOE_ERR_WORKSPACE;
    return moe::cuda_status(cudaMemsetAsync(ws, 0, n, (cudaStream_t)stream));
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
    if (!all_aligned16({W_gate, W_up, W_down, ws})) return MOE_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < moe_decode_workspace_bytes(T, H, F, E, k)) return MOE_ERR_WORKSPACE;
    const moe_bf16_t *const W[3] = {W_gate, W_up, W_down};
    return launch_decode<false>(decode_args(x, logits, expert_bias, score_fn, normalize, cl, T, H, F, E, k, topk_idx,
                                            topk_w, out),
                                W, ws, (cudaStream_t)stream);
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
    if (!all_aligned16({Wg_q, Wg_sf, Wu_q, Wu_sf, Wd_q, Wd_sf, ws})) return MOE_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < moe_decode_workspace_bytes(T, H, F, E, k)) return MOE_ERR_WORKSPACE;
    DecArgs a = decode_args(x, logits, expert_bias, score_fn, normalize, cl, T, H, F, E, k, topk_idx, topk_w, out);
    a.wq[0] = Wg_q;
    a.wsf[0] = Wg_sf;
    a.wq[1] = Wu_q;
    a.wsf[1] = Wu_sf;
    a.wq[2] = Wd_q;
    a.wsf[2] = Wd_sf;
    const moe_bf16_t *const W[3] = {nullptr, nullptr, nullptr};
    return launch_decode<true>(a, W, ws, (cudaStream_t)stream);
}
