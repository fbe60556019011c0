// gated.cuh -- the gated feed-forward's elementwise mathematics.
//
// With g and u the gate and up projections of a token (each the frozen 4-bit
// linear with its adapter), the block's hidden value and its gradients are
//   H  = act(g) u
//   dG = dH u act'(g),   dU = dH act(g)
// act is SiLU, g sigma(g) with act' = sigma(g) (1 + g (1 - sigma(g))), or the
// tanh form of GELU, g/2 (1 + t) with t = tanh(c (g + 0.044715 g^3)),
// c = sqrt(2 / pi), act' = (1 + t) / 2 + g/2 (1 - t^2) c (1 + 3 * 0.044715 g^2).
// All of it is formed in fp32.  Rounded to bf16 are H and the kept [g | u] (the
// outputs), and operands of the tensor-core products that follow: [dG | dU] for
// dX and dB, G for dX and dA, U in the forward.  Each rounding adds 1.7e-3 of
// the norm to what it reaches.  So that no gradient carries more than one
// besides its own, as in the linear's backward, G is formed from dG and dU in
// two bf16 halves each and dB from U in two.
#pragma once

#include <stdint.h>

#include <type_traits>

#include "common.cuh"
#include "dropout.cuh"
#include "gemm.cuh"

namespace qlora {

enum { ACT_SILU = 0, ACT_GELU_TANH = 1 };

// 1 / (1 + exp(-x)) with the hardware's base-2 exponential and reciprocal
// (each within 2^-22 of the value; the results are rounded to 8 bits next).
// Finite for every finite x: 2^y may overflow to infinity, whose reciprocal is
// the right 0.
__device__ __forceinline__ float sigmoid_f(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.0f));
    return r;
}

// g clamped to [-32, 32]; a NaN stays NaN (fminf and fmaxf would drop it).
__device__ __forceinline__ float clamp32(float g) {
    float x;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(g), "f"(-32.0f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(x), "f"(32.0f));
    return x;
}

// act(g) and act'(g).
__device__ __forceinline__ float act_value(int act, float g) {
    if (act == ACT_SILU) return g * sigmoid_f(g);
    // (1 + tanh y) / 2 = sigma(2 y); at |g| = 32 it is 0 or 1 in fp32, and the
    // clamp keeps the cubic finite for every g
    const float x = clamp32(g);
    return g * sigmoid_f(2.0f * 0.7978845608028654f * x * (1.0f + 0.044715f * x * x));
}
__device__ __forceinline__ void act_value_grad(int act, float g, float* v, float* dv) {
    if (act == ACT_SILU) {
        const float s = sigmoid_f(g);
        *v = g * s;
        *dv = s * (1.0f + g * (1.0f - s));
        return;
    }
    const float x = clamp32(g), g2 = x * x;
    const float s = sigmoid_f(2.0f * 0.7978845608028654f * x * (1.0f + 0.044715f * g2));
    *v = g * s;
    // d/dg g sigma(2 y) = sigma + g 2 y' sigma (1 - sigma), y' = c (1 + 3 * 0.044715 g^2)
    *dv = s + x * (2.0f * 0.7978845608028654f) * (1.0f + 0.134145f * g2) * s * (1.0f - s);
}

// Eight columns of dG and dU from dH, g and u, one after the other: dG and dU
// of columns 2 q and 2 q + 1 go to out(q, dG, dG', dU, dU').
template <int act, class Out>
__device__ __forceinline__ void gated_grad8(const uint4& hv, const uint4& gv, const uint4& uv, Out out) {
    const uint32_t h[4] = {hv.x, hv.y, hv.z, hv.w}, g[4] = {gv.x, gv.y, gv.z, gv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float v0, d0, v1, d1;
        act_value_grad(act, bf16_lo(g[q]), &v0, &d0);
        act_value_grad(act, bf16_hi(g[q]), &v1, &d1);
        const float h0 = bf16_lo(h[q]), h1 = bf16_hi(h[q]);
        out(q, h0 * bf16_lo(u[q]) * d0, h1 * bf16_hi(u[q]) * d1, h0 * v0, h1 * v1);
    }
}

// dGU[m] = [dH u act'(g) | dH act(g)] without adapters; eight columns a thread.
__global__ void __launch_bounds__(256) k_gated_grad(const uint16_t* dH, const uint16_t* GU, uint16_t* dGU, int64_t M,
                                                    int64_t F, int act) {
    pdl_trigger();
    pdl_wait();
    const int64_t f8 = F / 8;
    for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < M * f8;
         b += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = b / f8, c = b - m * f8;
        const uint4 hv = *reinterpret_cast<const uint4*>(dH + m * F + c * 8);
        const uint4 gv = *reinterpret_cast<const uint4*>(GU + m * 2 * F + c * 8);
        const uint4 uv = *reinterpret_cast<const uint4*>(GU + m * 2 * F + F + c * 8);
        uint32_t og[4], ou[4];
        auto out = [&](int q, float g0, float g1, float u0, float u1) {
            og[q] = pack_bf16x2(g0, g1);
            ou[q] = pack_bf16x2(u0, u1);
        };
        if (act == ACT_SILU)
            gated_grad8<ACT_SILU>(hv, gv, uv, out);
        else
            gated_grad8<ACT_GELU_TANH>(hv, gv, uv, out);
        *reinterpret_cast<uint4*>(dGU + m * 2 * F + c * 8) = make_uint4(og[0], og[1], og[2], og[3]);
        *reinterpret_cast<uint4*>(dGU + m * 2 * F + F + c * 8) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    }
}

// ---------------------------------------------------------------------------
// The gated backward's first pass with adapters: dGU = [dH u act'(g) | dH act(g)]
// as above, and sG = bf16(scale [dG B_gate | dU B_up]) from the tiles while
// they are in shared memory, so that the second product does not read dGU back
// (180 MB on LLaMA-65B at 2048 tokens) and can take the values to 16 bits: a
// tile is followed by the remainders of its rounding, multiplied onto the same
// sums.
//
// A CTA owns 128 tokens x a range of 64-column steps.  Per step sixteen warps
// form dG and dU [128 x 64] from dH, g and u, which they load into registers
// two steps ahead (96 KB in flight an SM: 2.2 us a step; with all three through
// a TMA ring in shared memory, three steps deep, it was 3.2 us), and write them
// with their remainders to one of two operand stages; one thread stores the two
// rounded tiles with TMA, one loads the two adapters' B rows and one issues the
// tcgen05 products onto two accumulators [128 x r].  The column range is split over S
// CTAs (about one CTA an SM in all), whose fp32 partial sums k_gated_sG adds in
// split order (deterministic) and rounds once (added by each token tile's last
// CTA instead, 590 KB through one SM, it took 26 us longer).
// Bound by HBM: dH and g, u read, dGU written, 10 B per token and hidden
// column (LLaMA-65B, 2048 tokens: 451 MB, 101 us under the profiler, 4.5 TB/s;
// LLaMA-7B, 1997 tokens: 54 us; 94 and 50 us without the remainders, in four
// stages).
// ---------------------------------------------------------------------------
struct GatedGradParams {
    CUtensorMap tmDGU;  // dGU [M][2F], box {64, 128}
    CUtensorMap tmB;    // B [2F][r], box {64, 64}
    const uint16_t* dH;  // [M][F]
    const uint16_t* GU;  // [M][2F]
    int M, F, r, act;
    int S;              // splits of the column range
    float scale;
    uint16_t* sG;       // [M][2r]
    float* part;        // [tiles][S][128][2r] (S > 1)
    uint64_t timeout_ns;
    int inject;
};

template <int BN>
struct GatedGradShape {
    static constexpr int TILE = 128 * 128;   // 128 rows x 64 bf16
    static constexpr int B_BYTES = BN * 128;  // 64 rows x BN columns
    static constexpr int B_OFF = 4 * TILE;    // behind dG, dU and their remainders
    static constexpr int STAGE = B_OFF + 2 * B_BYTES;
    static constexpr int STAGES = 2;
    static constexpr int SMEM = STAGE * STAGES + 1024 + 256;
    static constexpr int CWARPS = 16;                    // compute warps
    static constexpr int THREADS = 32 * (3 + CWARPS);    // producer, MMA, store, compute
    static constexpr int TMEM_COLS = 2 * BN;
};

template <int BN>
__global__ void __launch_bounds__(GatedGradShape<BN>::THREADS, 1)
    k_gated_grad_lora(const __grid_constant__ GatedGradParams p) {
    using S = GatedGradShape<BN>;
    constexpr int STAGES = S::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw_base);
    const uint32_t bar = base + S::STAGE * STAGES;
    auto full = [&](int s) { return bar + 8u * s; };
    auto ready = [&](int s) { return bar + 8u * (STAGES + s); };
    auto empty = [&](int s) { return bar + 8u * (2 * STAGES + s); };
    const uint32_t acc_full = bar + 8u * (3 * STAGES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(gbase + S::STAGE * STAGES + 8 * (3 * STAGES + 1));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCfg wc{p.timeout_ns};
    const int tile = blockIdx.x / p.S, z = blockIdx.x - tile * p.S;
    const int m0 = tile * 128;
    const int FS = p.F / 64;
    const int k0 = (int)((int64_t)FS * z / p.S), nk = (int)((int64_t)FS * (z + 1) / p.S) - k0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(ready(s), S::CWARPS);
            mbar_init(empty(s), 2);  // the products have read the stage, and the stores
        }
        mbar_init(acc_full, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&p.tmDGU);
        prefetch_tensormap(&p.tmB);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_holder), S::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // everything before this kernel is complete once the next one may start
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();

    if (warp == 0) {
        // ------------------------------------------------------------ producer of the B rows
        if (lane == 0 && !p.inject) {
            int last_use[STAGES];
            for (int s = 0; s < STAGES; ++s) last_use[s] = -1;
            for (int i = 0; i < nk; ++i) {
                const int s = i % STAGES, u = i / STAGES;
                if (!mbar_wait(empty(s), (u & 1) ^ 1, wc)) { *abort_flag = 1; break; }
                const int f = (k0 + i) * 64;
                const uint32_t st = base + s * S::STAGE;
                mbar_arrive_expect_tx(full(s), 2 * S::B_BYTES);
                for (int c = 0; c < BN / 64; ++c) {
                    tma_load_2d(st + S::B_OFF + 8192 * c, &p.tmB, full(s), 64 * c, f);
                    tma_load_2d(st + S::B_OFF + S::B_BYTES + 8192 * c, &p.tmB, full(s), 64 * c, p.F + f);
                }
                last_use[s] = u;
            }
            // every load has landed before the CTA exits
            for (int s = 0; s < STAGES; ++s)
                if (last_use[s] >= 0) mbar_wait(full(s), last_use[s] & 1, wc);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(128, BN, 0, 1);
            for (int i = 0; i < nk; ++i) {
                const int s = i % STAGES, u = i / STAGES;
                if (!mbar_wait(full(s), u & 1, wc) || !mbar_wait(ready(s), u & 1, wc)) { *abort_flag = 1; break; }
                tc_fence_after();
                const uint32_t st = base + s * S::STAGE;
                // tile t: dG, dU, then their remainders onto the same sums
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(tmem + (t & 1) * BN, smem_desc_sw128(st + t * S::TILE + kk * 32, 16, 1024),
                                  smem_desc_sw128(st + S::B_OFF + (t & 1) * S::B_BYTES + kk * 2048, 8192, 1024), idesc,
                                  (i > 0 || kk > 0 || t > 1) ? 1u : 0u);
                umma_commit(empty(s));
            }
            umma_commit(acc_full);
            mbar_wait(acc_full, 0, wc);  // nothing is in flight when the CTA exits
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ store issuer
        if (lane == 0) {
            for (int i = 0; i < nk; ++i) {
                const int s = i % STAGES, u = i / STAGES;
                if (!mbar_wait(ready(s), u & 1, wc)) { *abort_flag = 1; break; }
                const int f = (k0 + i) * 64;
                const uint32_t st = base + s * S::STAGE;
                tma_store_2d(&p.tmDGU, st, f, m0);
                tma_store_2d(&p.tmDGU, st + S::TILE, p.F + f, m0);
                bulk_commit_group();
                bulk_wait_group_read0();  // the step has been read out of its stage
                mbar_arrive(empty(s));
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
    } else {
        // ------------------------------------------------------------ compute
        // thread t: 16-byte chunk t % 8 of rows t / 8 and t / 8 + 64
        const int t = threadIdx.x - 96, c = t & 7, l = t >> 3;
        const bool live0 = m0 + l < p.M, live1 = m0 + l + 64 < p.M;
        const uint16_t* h0 = p.dH + (int64_t)(m0 + l) * p.F + (int64_t)k0 * 64 + c * 8;
        const uint16_t* g0 = p.GU + (int64_t)(m0 + l) * 2 * p.F + (int64_t)k0 * 64 + c * 8;
        const int64_t hs = (int64_t)64 * p.F, gs = (int64_t)128 * p.F;
        struct In {
            uint4 v[6];  // dH, g, u of the two rows
        };
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        auto fetch = [&](int i) {
            In x;
            const bool on = i < nk;
            x.v[0] = on && live0 ? __ldcg(reinterpret_cast<const uint4*>(h0 + i * 64)) : zero;
            x.v[1] = on && live0 ? __ldcg(reinterpret_cast<const uint4*>(g0 + i * 64)) : zero;
            x.v[2] = on && live0 ? __ldcg(reinterpret_cast<const uint4*>(g0 + p.F + i * 64)) : zero;
            x.v[3] = on && live1 ? __ldcg(reinterpret_cast<const uint4*>(h0 + hs + i * 64)) : zero;
            x.v[4] = on && live1 ? __ldcg(reinterpret_cast<const uint4*>(g0 + gs + i * 64)) : zero;
            x.v[5] = on && live1 ? __ldcg(reinterpret_cast<const uint4*>(g0 + gs + p.F + i * 64)) : zero;
            return x;
        };
        auto run = [&](auto act_tag) {
            constexpr int act = decltype(act_tag)::value;
            auto step = [&](int i, const In& x) {
                const int s = i % STAGES, u = i / STAGES;
                if (!__all_sync(0xffffffffu, mbar_wait(empty(s), (u & 1) ^ 1, wc))) {
                    *abort_flag = 1;
                    return false;
                }
                const uint32_t st = base + s * S::STAGE;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[4][4];  // [dG, dU and their remainders][column pair]
                    gated_grad8<act>(x.v[3 * h], x.v[3 * h + 1], x.v[3 * h + 2],
                                     [&](int q, float g0, float g1, float u0, float u1) {
                                         bf16_halves(g0, g1, &o[0][q], &o[2][q]);
                                         bf16_halves(u0, u1, &o[1][q], &o[3][q]);
                                     });
                    const uint32_t a = st + (uint32_t)(l + 64 * h) * 128u + (uint32_t)((c ^ (l & 7)) << 4);
#pragma unroll
                    for (int t = 0; t < 4; ++t) st_shared_v4(a + t * S::TILE, o[t][0], o[t][1], o[t][2], o[t][3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(ready(s));
                return true;
            };
            In a = fetch(0), b = fetch(1);
            for (int i = 0; i < nk; i += 2) {
                const In a2 = fetch(i + 2);
                if (!step(i, a)) break;
                a = a2;
                const In b2 = fetch(i + 3);
                if (i + 1 < nk && !step(i + 1, b)) break;
                b = b2;
            }
        };
        if (p.act == ACT_SILU)
            run(std::integral_constant<int, ACT_SILU>{});
        else
            run(std::integral_constant<int, ACT_GELU_TANH>{});

        // ------------------------------------------------------------ sG (the first four compute warps read TMEM)
        const int rt = 2 * p.r;
        const int cw = warp - 3;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const bool got = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, wc));
        if (!got) *abort_flag = 1;
        if (cw < 4 && got && !*abort_flag && nk > 0) {
            tc_fence_after();
            float* part = p.S > 1 ? p.part + ((int64_t)(tile * p.S + z) * 128 + row) * rt : nullptr;
            const bool live = m0 + row < p.M;
#pragma unroll 1
            for (int h = 0; h < 2; ++h)
#pragma unroll 1
                for (int c0 = 0; c0 < p.r; c0 += 32) {
                    uint32_t v[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(h * BN + c0), v);
                    tmem_ld_wait();
                    if (!live) continue;
                    if (p.S > 1) {
#pragma unroll
                        for (int q = 0; q < 32; q += 4)
                            if (c0 + q < p.r)
                                __stcg(reinterpret_cast<float4*>(part + h * p.r + c0 + q),
                                       make_float4(__uint_as_float(v[q]), __uint_as_float(v[q + 1]),
                                                   __uint_as_float(v[q + 2]), __uint_as_float(v[q + 3])));
                    } else {
                        uint16_t* o = p.sG + (int64_t)(m0 + row) * rt + h * p.r + c0;
#pragma unroll
                        for (int q = 0; q < 32; q += 4)
                            if (c0 + q < p.r)
                                *reinterpret_cast<uint2*>(o + q) = make_uint2(
                                    pack_bf16x2(__fmul_rn(__uint_as_float(v[q]), p.scale),
                                                __fmul_rn(__uint_as_float(v[q + 1]), p.scale)),
                                    pack_bf16x2(__fmul_rn(__uint_as_float(v[q + 2]), p.scale),
                                                __fmul_rn(__uint_as_float(v[q + 3]), p.scale)));
                    }
                }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, S::TMEM_COLS);
    }
}

// sG = bf16(scale * sum of the S partials), four columns a thread.
__global__ void __launch_bounds__(256) k_gated_sG(const float* part, uint16_t* sG, int64_t M, int rt, int S, float scale) {
    pdl_trigger();
    pdl_wait();
    const int r4 = rt / 4;
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= M * r4) return;
    const int64_t m = e / r4;
    const int j = (int)(e - m * r4) * 4;
    const float* src = part + ((m >> 7) * S * 128 + (m & 127)) * rt + j;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int z = 0; z < S; ++z) {
        const float4 b = __ldcg(reinterpret_cast<const float4*>(src + (int64_t)z * 128 * rt));
        a.x = __fadd_rn(a.x, b.x);
        a.y = __fadd_rn(a.y, b.y);
        a.z = __fadd_rn(a.z, b.z);
        a.w = __fadd_rn(a.w, b.w);
    }
    *reinterpret_cast<uint2*>(sG + m * rt + j) =
        make_uint2(pack_bf16x2(__fmul_rn(a.x, scale), __fmul_rn(a.y, scale)),
                   pack_bf16x2(__fmul_rn(a.z, scale), __fmul_rn(a.w, scale)));
}

}  // namespace qlora
