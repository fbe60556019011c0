// gated.cuh -- the gated feed-forward's elementwise mathematics.
//
// With g and u the gate and up projections of a token (each the frozen 4-bit
// linear with its adapter), the block's hidden value and its gradients are
//   H  = act(g) u
//   dG = dH u act'(g),   dU = dH act(g)
// act is SiLU, g sigma(g) with act' = sigma(g) (1 + g (1 - sigma(g))), or the
// tanh form of GELU, g/2 (1 + t) with t = tanh(c (g + 0.044715 g^3)),
// c = sqrt(2 / pi), act' = (1 + t) / 2 + g/2 (1 - t^2) c (1 + 3 * 0.044715 g^2).
// All of it is formed in fp32.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "dropout.cuh"

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

// act(g) and act'(g).
__device__ __forceinline__ float act_value(int act, float g) {
    if (act == ACT_SILU) return g * sigmoid_f(g);
    // (1 + tanh y) / 2 = sigma(2 y); at |g| = 32 it is 0 or 1 in fp32, and the
    // clamp keeps the cubic finite for every g
    const float x = fminf(fmaxf(g, -32.0f), 32.0f);
    return g * sigmoid_f(2.0f * 0.7978845608028654f * x * (1.0f + 0.044715f * x * x));
}
__device__ __forceinline__ void act_value_grad(int act, float g, float* v, float* dv) {
    if (act == ACT_SILU) {
        const float s = sigmoid_f(g);
        *v = g * s;
        *dv = s * (1.0f + g * (1.0f - s));
        return;
    }
    const float x = fminf(fmaxf(g, -32.0f), 32.0f), g2 = x * x;
    const float s = sigmoid_f(2.0f * 0.7978845608028654f * x * (1.0f + 0.044715f * g2));
    *v = g * s;
    // d/dg g sigma(2 y) = sigma + g 2 y' sigma (1 - sigma), y' = c (1 + 3 * 0.044715 g^2)
    *dv = s + x * (2.0f * 0.7978845608028654f) * (1.0f + 0.134145f * g2) * s * (1.0f - s);
}

// H[m][f] = act(GU[m][f]) GU[m][F + f]; eight columns a thread.
__global__ void __launch_bounds__(256) k_gated_act(const uint16_t* GU, uint16_t* H, int64_t M, int64_t F, int act) {
    pdl_trigger();
    pdl_wait();
    const int64_t f8 = F / 8;
    for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < M * f8;
         b += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = b / f8, c = b - m * f8;
        const uint4 gv = *reinterpret_cast<const uint4*>(GU + m * 2 * F + c * 8);
        const uint4 uv = *reinterpret_cast<const uint4*>(GU + m * 2 * F + F + c * 8);
        const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            o[q] = pack_bf16x2(act_value(act, bf16_lo(g[q])) * bf16_lo(u[q]), act_value(act, bf16_hi(g[q])) * bf16_hi(u[q]));
        *reinterpret_cast<uint4*>(H + m * F + c * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// dGU[m] = [dH u act'(g) | dH act(g)]; eight columns a thread.
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
        const uint32_t h[4] = {hv.x, hv.y, hv.z, hv.w}, g[4] = {gv.x, gv.y, gv.z, gv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w};
        uint32_t og[4], ou[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v0, d0, v1, d1;
            act_value_grad(act, bf16_lo(g[q]), &v0, &d0);
            act_value_grad(act, bf16_hi(g[q]), &v1, &d1);
            const float h0 = bf16_lo(h[q]), h1 = bf16_hi(h[q]);
            og[q] = pack_bf16x2(h0 * bf16_lo(u[q]) * d0, h1 * bf16_hi(u[q]) * d1);
            ou[q] = pack_bf16x2(h0 * v0, h1 * v1);
        }
        *reinterpret_cast<uint4*>(dGU + m * 2 * F + c * 8) = make_uint4(og[0], og[1], og[2], og[3]);
        *reinterpret_cast<uint4*>(dGU + m * 2 * F + F + c * 8) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    }
}

}  // namespace qlora
