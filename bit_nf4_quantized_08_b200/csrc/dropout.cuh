// dropout.cuh -- dropout from a counter-based generator, the keep mask
// recomputed wherever it is needed and never stored.
//
// Generator: Philox-4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit
// products, key = the 64-bit seed, counter = (64-bit block number, 64-bit
// offset).  One block gives the eight 15-bit numbers of eight consecutive
// elements: word j holds element 2j's number in bits 0..14 and element
// 2j + 1's in bits 16..30.  Element e = 8 block + i is kept if its number is
// at least T = round(2^15 p), that is with probability exactly 1 - T / 2^15,
// and kept elements are scaled by the exact inverse 2^15 / (2^15 - T).
// Fifteen bits, because the halfword compare is then one add (a carry into
// bit 15) and one byte permute for two elements; sixteen would take a compare
// and a select for each.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace qlora {

constexpr int kDropSteps = 32768;  // 2^15

// A dropout in launch form.  thr == 0: no dropout.
struct DropParams {
    uint32_t rk[20];    // round keys: key words of rounds 0..9
    uint32_t off_lo, off_hi;
    const unsigned long long* off_dev;  // added to the offset when the kernel runs, or nullptr
    uint32_t thr;       // T
    uint32_t add;       // (2^15 - T) in both halves
    float up;           // 2^15 / (2^15 - T)
};

inline void drop_params(DropParams* d, uint32_t thr, uint64_t seed, uint64_t offset, const uint64_t* offset_dev) {
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    for (int i = 0; i < 10; ++i) {
        d->rk[2 * i] = k0;
        d->rk[2 * i + 1] = k1;
        k0 += 0x9E3779B9u;  // Weyl constants of the paper
        k1 += 0xBB67AE85u;
    }
    d->off_lo = (uint32_t)offset;
    d->off_hi = (uint32_t)(offset >> 32);
    d->off_dev = reinterpret_cast<const unsigned long long*>(offset_dev);
    d->thr = thr;
    d->add = (uint32_t)(kDropSteps - thr) * 0x10001u;
    d->up = (float)((double)kDropSteps / (double)(kDropSteps - (int)thr));
}

// The offset words of a launch, with the device counter added.  The counter
// may be written by an earlier kernel of the stream: call after pdl_wait.
__device__ __forceinline__ uint2 drop_offset(const DropParams& d) {
    unsigned long long o = ((unsigned long long)d.off_hi << 32) | d.off_lo;
    if (d.off_dev) o += *d.off_dev;
    return make_uint2((uint32_t)o, (uint32_t)(o >> 32));
}

// What the first two rounds have in common for all blocks whose number has
// the same high word (the counter's other words are the launch's): one of the
// two products of each.  The products are the generator's cost: a 32 x 32 ->
// 64 bit multiplication issues once in 4 cycles a scheduler, so the 18 that
// are left take 72 cycles for a warp's 32 blocks (85 measured with all 20).
struct DropCtx {
    uint32_t k1, c1, a1, a0;
};
__device__ __forceinline__ DropCtx drop_ctx(const DropParams& d, uint2 off, uint32_t blk_hi) {
    const uint64_t p = (uint64_t)off.x * 0xCD9E8D57u;
    const uint64_t a = (uint64_t)((uint32_t)(p >> 32) ^ blk_hi ^ d.rk[0]) * 0xD2511F53u;
    DropCtx c;
    c.k1 = off.y ^ d.rk[1];
    c.c1 = (uint32_t)p ^ d.rk[2];
    c.a1 = (uint32_t)(a >> 32) ^ d.rk[3];
    c.a0 = (uint32_t)a;
    return c;
}

// Keep masks of the eight elements of the block with low word `blk`: m[j] has
// 0xFFFF in the low (high) half if element 2j (2j + 1) is kept, else 0.
__device__ __forceinline__ void drop_mask8(const DropParams& d, const DropCtx& x, uint32_t blk, uint32_t (&m)[4]) {
    const uint64_t p = (uint64_t)blk * 0xD2511F53u;
    const uint64_t q = (uint64_t)((uint32_t)(p >> 32) ^ x.k1) * 0xCD9E8D57u;
    uint32_t c0 = (uint32_t)(q >> 32) ^ x.c1, c1 = (uint32_t)q, c2 = (uint32_t)p ^ x.a1, c3 = x.a0;
#pragma unroll
    for (int i = 2; i < 10; ++i) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ d.rk[2 * i];
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ d.rk[2 * i + 1];
        c3 = (uint32_t)a;
    }
    const uint32_t w[4] = {c0, c1, c2, c3};
#pragma unroll
    for (int j = 0; j < 4; ++j)  // bit 15 of each half: number >= T; replicated over the half
        m[j] = prmt((w[j] & 0x7FFF7FFFu) + d.add, 0u, 0xBB99u);
}

// Keep bits of 32 consecutive elements from block `blk` (a multiple of 4):
// bit 4 b + j is element 8 b + 2 j, bit 16 + 4 b + j element 8 b + 2 j + 1.
__device__ __forceinline__ uint32_t drop_bits32(const DropParams& d, const DropCtx& x, uint32_t blk) {
    uint32_t bits = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        uint32_t m[4];
        drop_mask8(d, x, blk + b, m);
#pragma unroll
        for (int j = 0; j < 4; ++j) bits |= m[j] & (0x00010001u << (4 * b + j));
    }
    return bits;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// ---------------------------------------------------------------------------
// Y[e] = kept(e) ? X[e] * up : +0, elementwise (X and Y may be the same).
// A dropped element gives +0 whatever X holds there.  bf16 products are
// formed in fp32 and rounded once.
// Bound by HBM: each element is read and written once (2^27 bf16: 90 us, 5.96
// TB/s; the generator alone would take about 38 us).  A thread takes whole
// eight-element blocks: 16 bytes of bf16, 32 of fp32.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256, 8) k_dropout(const T* X, T* Y, int64_t n, const __grid_constant__ DropParams d) {
    constexpr bool F32 = sizeof(T) == 4;
    pdl_trigger();
    pdl_wait();
    const uint2 off = drop_offset(d);
    uint32_t hi = 0;
    DropCtx ctx = drop_ctx(d, off, 0u);
    auto mask = [&](int64_t b, uint32_t (&m)[4]) {
        if ((uint32_t)(b >> 32) != hi) {  // past 2^35 elements
            hi = (uint32_t)(b >> 32);
            ctx = drop_ctx(d, off, hi);
        }
        drop_mask8(d, ctx, (uint32_t)b, m);
    };
    const int64_t full = n >> 3;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    const int64_t t0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const uint4* xv = reinterpret_cast<const uint4*>(X);
    uint4* yv = reinterpret_cast<uint4*>(Y);
    for (int64_t b = t0; b < full; b += stride) {
        uint32_t m[4] = {~0u, ~0u, ~0u, ~0u};
        if (F32) {
            const uint4 v0 = xv[2 * b], v1 = xv[2 * b + 1];
            if (d.thr) mask(b, m);
            uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t keep = (i & 1) ? prmt(m[i >> 1], 0u, 0x3232u) : prmt(m[i >> 1], 0u, 0x1010u);
                w[i] = __float_as_uint(__fmul_rn(__uint_as_float(w[i]), d.up)) & keep;
            }
            yv[2 * b] = make_uint4(w[0], w[1], w[2], w[3]);
            yv[2 * b + 1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            const uint4 v = xv[b];
            if (d.thr) mask(b, m);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = pack_bf16x2(__fmul_rn(bf16_lo(w[j]), d.up), __fmul_rn(bf16_hi(w[j]), d.up)) & m[j];
            yv[b] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    // the last, partial block
    const int tail = (int)(n & 7);
    if (tail && t0 == 0) {
        uint32_t m[4] = {~0u, ~0u, ~0u, ~0u};
        if (d.thr) mask(full, m);
        for (int i = 0; i < tail; ++i) {
            const int64_t e = 8 * full + i;
            const bool keep = (m[i >> 1] >> (16 * (i & 1))) & 1u;
            if (F32) {
                const float x = reinterpret_cast<const float*>(X)[e];
                reinterpret_cast<float*>(Y)[e] = keep ? __fmul_rn(x, d.up) : 0.0f;
            } else {
                const float x = bf16_lo(reinterpret_cast<const uint16_t*>(X)[e]);
                reinterpret_cast<uint16_t*>(Y)[e] =
                    keep ? (uint16_t)(pack_bf16x2(__fmul_rn(x, d.up), 0.0f) & 0xFFFFu) : (uint16_t)0;
            }
        }
    }
}

}  // namespace qlora
