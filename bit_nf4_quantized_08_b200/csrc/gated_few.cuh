// gated_few.cuh -- the gated feed-forward's forward for up to 8 tokens
// (decoding), where a weight is used so seldom that expanding it into a
// tensor-core operand in shared memory costs more than the products.
//
//   H = act(g) u,   [g | u] = X W'^T + sU B^T
//
// The inner sums are warp MMAs (m16n8k16) whose weight operand is formed in
// registers: a table of code-byte pairs in shared memory gives the two fp32
// code values of a byte with one load, which are multiplied by the block
// constant and rounded to bf16.  That is qlora_nf4_dequantize's weight bit for
// bit, so that the block is the same function whatever the token count and its
// backward differentiates what its forward computed.  (With the code book
// itself rounded to bf16 and the constant applied to each block's sum, as in
// the plain linear for few tokens, H was 3.4e-3 off its definition instead of
// 1.7e-3, in 33 us instead of 39 us on LLaMA-7B and 84 instead of 102 us on
// LLaMA-65B.)  Sums, activation and product are fp32.  The weight is the
// 16-row operand: 8 gate rows and the 8 up rows of the same hidden columns, so
// that a thread ends with g and u of one column and forms H, and the tokens
// are the 8-column operand.
//
// A unit is (8 hidden columns, 256 elements of k): 16 lines of 128 bytes of
// codes.  A CTA owns a range of hidden columns and each of its 16 warps some
// unit columns (256 elements of k) of all of them, so that a warp's part of X
// stays in registers.  Every warp has a ring of its own, filled by TMA two
// units ahead (64 KB in flight an SM), and nothing in the loop waits for
// another warp.  The warps' fp32 sums of a chunk of hidden columns pass through
// shared memory and are added in warp order; then the adapters' products and
// the activation.
//
// Within a block, lane position t of a fragment's group of four holds bytes
// 4 t .. 4 t + 3 of both halves of a row's 32 code bytes (elements 8 t .. 8 t + 7
// and 32 + 8 t .. + 7): a load of one word a lane then covers a 16-byte chunk of
// eight rows, which the 128-byte swizzle spreads over all banks.
//
// Bound by shared memory: 51 wavefronts for a 64-element block of 16 rows, 32 of
// them table lookups (two for a warp's 64-bit loads), keep that pipe busy for
// 69 % of the time, and the latencies of 16 warps a SM take most of the rest;
// HBM (28 us on LLaMA-65B, 7 us on LLaMA-7B) does not.  One token, kernel
// alone: LLaMA-65B 97 us (1.9 TB/s), LLaMA-7B 32 us (1.5 TB/s; about 9 us of it
// are start, table, adapters and end).  k_gated_small takes 116 and 46 us
// there.  (Steps towards it, measured with the rounded code book: on LLaMA-65B
// 105 us with codes and constants loaded straight into registers, X read per
// block and a two-instruction table address, 92 us with X kept in registers, 78
// us with codes through TMA rings.)
#pragma once

#include "common.cuh"
#include "gated.cuh"
#include "nf4.cuh"
#include "smallm_mma.cuh"

namespace qlora {

struct GatedFewParams {
    CUtensorMap tmCodes;   // codes [2F][K/2] bytes, box {128 B, 8 rows}, 128-byte swizzle
    const uint8_t* codes;  // the same array
    const uint16_t* X;     // [M][K]
    const uint16_t* B;     // [2F][r]
    const uint16_t* sU;    // [M][2r]
    const uint8_t* q8;
    const float* c1;
    const float* offset;
    const float* absmax;   // without double quantization
    int dq;
    int F, M, K, kbs;      // kbs = K / 64
    int r, act;
    QFormat fmt;
    uint16_t* H;           // [M][F]
    uint16_t* GU;          // [M][2F] or nullptr
    int late, less;        // CTAs that start late, and the items that they have fewer
    uint64_t timeout_ns;
    int inject;
};

struct GatedFewShape {
    static constexpr int WARPS = 16;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int STAGES = 3;                 // of a warp's ring
    static constexpr int STAGE = 2048;               // 8 gate and 8 up rows of 128 bytes
    static constexpr int CHUNK = 7;                  // most items (8 hidden columns) between two reductions
    static constexpr int LUT_BYTES = 256 * 256;      // entry e of lane l at 256 e + 8 l
    static constexpr int RING_BYTES = WARPS * STAGES * STAGE;
    static constexpr int PART_BYTES = CHUNK * (WARPS + 1) * 32 * 16;  // [item of the chunk][warp or remainder][lane]
    // partial sums up to address 65536, the table, the rings (a window's first 1 KB is the system's)
    static constexpr int SMEM = 65536 + LUT_BYTES + RING_BYTES - 1024;
    static_assert(SMEM + 1536 <= 232448 && PART_BYTES + 4096 <= 65536, "shared memory per CTA");
};

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
// The two weights of code byte k of w, bf16(code * a) as qlora_nf4_dequantize
// rounds them; a2 holds the block constant a twice.  The table starts at a
// multiple of 64 KB, which tl (this lane's column of the first entry) holds in
// its upper half: one byte permute forms the address.
__device__ __forceinline__ uint32_t few_pair(uint32_t w, int k, uint32_t tl, uint64_t a2) {
    uint64_t v;
    asm("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(prmt(w, tl, 0x7604u | (uint32_t)(k << 4))));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(a2));
    return pack_bf16x2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

__device__ __forceinline__ uint64_t twice(float a) {
    return (uint64_t)__float_as_uint(a) << 32 | __float_as_uint(a);
}

__global__ void __launch_bounds__(GatedFewShape::THREADS, 1) k_gated_few(const __grid_constant__ GatedFewParams p) {
    using S = GatedFewShape;
    constexpr int W = S::WARPS;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const uint32_t dyn = smem_u32(smem_raw);
    const uint32_t lut = (dyn + (uint32_t)S::PART_BYTES + 65535u) & ~65535u, base = lut + (uint32_t)S::LUT_BYTES;
    float4* part = reinterpret_cast<float4*>(smem_raw);
    __shared__ float t8s[256];
    __shared__ __align__(8) uint64_t full_bar[W * S::STAGES];
    __shared__ volatile int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const uint32_t tl = lut + (uint32_t)lane * 8u;
    const int items = p.F / 8;
    // The last `late` CTAs find their SM when the kernel that forms sU has left
    // it, and take `less` items fewer than the others.
    const int G = gridDim.x, n_max = (items + G - 1) / G;
    const int less = min(p.less, n_max - 1), early = G - p.late;
    auto first_item = [&](int b) {
        const int64_t w = (int64_t)b * n_max - (int64_t)max(b - early, 0) * less;
        return (int)(items * w / ((int64_t)G * n_max - (int64_t)p.late * less));
    };
    const int i_begin = first_item(blockIdx.x), i_end = first_item(blockIdx.x + 1);
    const int chunks = (i_end - i_begin + S::CHUNK - 1) / S::CHUNK;
    const int chunk = chunks > 0 ? (i_end - i_begin + chunks - 1) / chunks : 1;  // even parts
    const int Q = p.kbs >> 2, rem = p.kbs & 3;  // whole units of an item, and the block columns after them
    const int NG = Q > 0 && Q < W ? W / Q : 1;  // warps on the same unit column take every NG-th item
    const int e0 = Q < W && Q > 0 ? warp / Q : 0, q0 = Q < W && Q > 0 ? warp % Q : warp;
    const bool busy = Q > 0 && e0 < NG;
    const int64_t ldc = p.K / 2, up_c = (int64_t)p.F * ldc;
    const int sh = p.fmt.bs_shift;
    const WaitCfg wc{p.timeout_ns};
    const uint32_t full0 = smem_u32(full_bar) + 8u * (uint32_t)(warp * S::STAGES);
    const uint32_t ring = base + (uint32_t)(warp * S::STAGES * S::STAGE);

    pdl_trigger();
    if (lane == 0) {  // (the warp's own barriers)
        for (int i = 0; i < S::STAGES; ++i) mbar_init(full0 + 8u * i, 1);
        fence_mbar_init();
        prefetch_tensormap(&p.tmCodes);
    }
    if (threadIdx.x == 0) abort_flag = 0;
    __syncwarp();
    // With adapters the kernel before is the one that forms sU, which waited
    // for its own predecessors before it let this one start.
    if (p.r == 0) pdl_wait();

    // Block constants: offsets from the group of 256 that holds the CTA's first
    // gate (up) row's first block.  (At most 2^40 elements over the CTAs: they
    // fit in 32 bits.)
    struct Blocks {
        const uint8_t* q8;
        const float* f;  // c1 or absmax
        uint32_t first;
    };
    auto blocks_at = [&](int64_t b) {
        const int64_t b0 = b & ~(int64_t)1023;
        return Blocks{p.dq ? p.q8 + (b0 >> sh) : nullptr, p.dq ? p.c1 + (b0 >> (sh + 8)) : p.absmax + (b0 >> sh),
                      (uint32_t)(b - b0)};
    };
    const Blocks bg = blocks_at((int64_t)i_begin * 8 * p.kbs), bu = blocks_at(((int64_t)p.F + i_begin * 8) * p.kbs);
    auto load_const = [&](const Blocks& t, uint32_t rel, float& sv, uint32_t& qv) {  // rel: blocks after the first
        const uint32_t b = (t.first + rel) >> sh;
        qv = p.dq ? (uint32_t)t.q8[b] : 0u;
        sv = p.dq ? t.f[b >> 8] : t.f[b];
    };
    // The warp's units of a chunk: for each of its unit columns q, its items.
    struct Pos {
        int e, q;
        uint32_t b;  // this lane's block of either row: column 4 q + tig
    };
    int item0 = i_begin, n_items = min(chunk, i_end - i_begin);
    auto place = [&](Pos& u) {
        u.b = (uint32_t)(((item0 - i_begin + u.e) * 8 + gid) * p.kbs + 4 * u.q + tig);
    };
    auto start = [&]() {
        Pos u;
        u.e = e0;
        u.q = q0;
        if (!busy || e0 >= n_items) u.q = Q;
        place(u);
        return u;
    };
    auto advance = [&](Pos& u) {
        u.e += NG;
        u.b += (uint32_t)(NG * 8 * p.kbs);
        if (u.e >= n_items) {
            u.e = e0;
            u.q += W;
            place(u);
        }
    };
    // A unit's codes into ring stage st and, in registers, the raw constants of
    // block column 4 q + tig of this lane's two rows.
    struct Raw {
        float s[2];
        uint32_t q[2];
    };
    auto fetch = [&](Raw& x, int st, Pos& u) {
        if (u.q >= Q) return;
        if (lane == 0 && !p.inject) {
            const uint32_t dst = ring + (uint32_t)(st * S::STAGE), bar = full0 + 8u * st;
            const int row = (item0 + u.e) * 8;
            mbar_arrive_expect_tx(bar, S::STAGE);
            tma_load_2d(dst, &p.tmCodes, bar, u.q * 128, row);
            tma_load_2d(dst + S::STAGE / 2, &p.tmCodes, bar, u.q * 128, p.F + row);
        }
        load_const(bg, u.b, x.s[0], x.q[0]);
        load_const(bu, u.b, x.s[1], x.q[1]);
        advance(u);
    };

    Raw raw[S::STAGES];
    uint32_t phases = 0;   // parity of each stage's next use
    bool dead = false;
    Pos next = start();  // the next unit to load
#pragma unroll
    for (int i = 0; i < S::STAGES - 1; ++i) fetch(raw[i], i, next);

    // (token rows past the last repeat it: nobody reads their sums)
    auto load_x = [&](uint4 (&x)[2], int kb) {
        const uint4* src =
            reinterpret_cast<const uint4*>(p.X + (int64_t)min(gid, p.M - 1) * p.K + kb * 64 + tig * 8);
        x[0] = src[0];
        x[1] = src[4];
    };
    uint4 x[4][2];
    int xq = -1;  // the unit column whose X the warp holds
    if (busy && i_end > i_begin) {
        xq = q0;
#pragma unroll
        for (int i = 0; i < 4; ++i) load_x(x[i], 4 * xq + i);
    }
    // the adapters' B rows of this CTA on their way to L2
    if (p.r > 0) {
        const int lines = (i_end - i_begin) * 8 * p.r * 2 / 128 + 1;
        for (int i = threadIdx.x; i < 2 * lines; i += S::THREADS) {
            const int64_t row = (int64_t)i_begin * 8 + (i >= lines ? p.F : 0);
            const int64_t at = min(row * p.r + (int64_t)(i >= lines ? i - lines : i) * 64, (int64_t)2 * p.F * p.r - 1);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.B + at));
        }
    }
    // the table and the 8-bit code book, while the first loads are on their way
    for (int e = warp; e < 256; e += W)
        *reinterpret_cast<float2*>(smem_raw + (tl - dyn) + 256 * e) =
            make_float2(code_value(p.fmt.code_type, e >> 4), code_value(p.fmt.code_type, e & 15));
    for (int i = threadIdx.x; i < 256; i += S::THREADS)
        t8s[i] = dq_value(p.fmt.dq_type, (p.fmt.dq_type == 0 || i < 253) ? i : 0);
    const float off = p.dq ? *p.offset : 0.0f;
    __syncthreads();

    auto block_const = [&](float s, uint32_t q) {
        return p.dq ? __fadd_rn(__fmul_rn(t8s[q], s), off) : s;
    };
    // acc += the products of one block column
    auto block = [&](float (&acc)[4], const uint2& cg, const uint2& cu, const uint4 (&x)[2], float sg, float su) {
        const uint64_t sg2 = twice(sg), su2 = twice(su);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t wg = j < 2 ? cg.x : cg.y, wu = j < 2 ? cu.x : cu.y;
            const int k = 2 * (j & 1);
            const uint32_t a0 = few_pair(wg, k, tl, sg2), a1 = few_pair(wu, k, tl, su2);
            const uint32_t a2 = few_pair(wg, k + 1, tl, sg2), a3 = few_pair(wu, k + 1, tl, su2);
            const uint4 v = x[j >> 1];
            mma_16816(acc, a0, a1, a2, a3, j & 1 ? v.z : v.x, j & 1 ? v.w : v.y);
        }
    };

    while (true) {
        Pos u = start();
        auto step = [&](const Raw& v, int st) {
            if (u.q != xq) {
                xq = u.q;
#pragma unroll
                for (int i = 0; i < 4; ++i) load_x(x[i], 4 * xq + i);
            }
            const float sc0 = block_const(v.s[0], v.q[0]), sc1 = block_const(v.s[1], v.q[1]);
            float4* slot = part + (u.e * (W + 1) + warp) * 32 + lane;
            const float4 o = u.q >= W ? *slot : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float acc[4] = {o.x, o.y, o.z, o.w};
            const uint32_t row = ring + (uint32_t)(st * S::STAGE) + (uint32_t)(gid * 128 + tig * 4) + ((uint32_t)gid << 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t c0 = row ^ (uint32_t)(i << 5), c1 = c0 ^ 16u;
                block(acc, make_uint2(ld_shared_u32(c0), ld_shared_u32(c1)),
                      make_uint2(ld_shared_u32(c0 + S::STAGE / 2), ld_shared_u32(c1 + S::STAGE / 2)), x[i],
                      __shfl_sync(0xffffffffu, sc0, (lane & 28) | i), __shfl_sync(0xffffffffu, sc1, (lane & 28) | i));
            }
            *slot = make_float4(acc[0], acc[1], acc[2], acc[3]);
            advance(u);
        };
        // (the stages take turns: the loop is unrolled by their number)
        while (u.q < Q) {
#pragma unroll
            for (int i = 0; i < S::STAGES; ++i) {
                if (u.q >= Q) break;
                // every lane is done with the unit before: its sums, which
                // depend on all that it read, are stored
                __syncwarp();
                if (!dead) fetch(raw[(i + S::STAGES - 1) % S::STAGES], (i + S::STAGES - 1) % S::STAGES, next);
                if (!dead && !__all_sync(0xffffffffu, mbar_wait(full0 + 8u * i, (phases >> i) & 1u, wc))) {
                    dead = true;
                    abort_flag = 1;
                }
                if (dead) {
                    advance(u);
                    continue;
                }
                phases ^= 1u << i;
                step(raw[i], i);
            }
        }
        // the block columns after the last whole unit
        if (rem)
            for (int e = warp; e < n_items; e += W) {
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                const int64_t row = (int64_t)(item0 + e) * 8 + gid;
#pragma unroll 1
                for (int kb = 4 * Q; kb < p.kbs; ++kb) {
                    const uint8_t* c = p.codes + row * ldc + (int64_t)kb * 32 + tig * 4;
                    float s0, s1;
                    uint32_t v0, v1;
                    const uint32_t b = (uint32_t)(((item0 - i_begin + e) * 8 + gid) * p.kbs + kb);
                    load_const(bg, b, s0, v0);
                    load_const(bu, b, s1, v1);
                    uint4 xr[2];
                    load_x(xr, kb);
                    auto word = [&](int64_t o) { return *reinterpret_cast<const uint32_t*>(c + o); };
                    block(acc, make_uint2(word(0), word(16)), make_uint2(word(up_c), word(up_c + 16)), xr,
                          block_const(s0, v0), block_const(s1, v1));
                }
                part[(e * (W + 1) + W) * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            }
        if (p.r > 0) pdl_wait();  // sU
        __syncthreads();

        // an item a warp: the warps' partial sums in order, then the adapters
        for (int e = warp; e < n_items; e += W) {
            const int w0 = Q < W ? (e % NG) * Q : 0, cnt = min(Q, W);
            const int f = (item0 + e) * 8 + gid;
            const int64_t fg = (int64_t)f * p.r, fu = ((int64_t)p.F + f) * p.r;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            auto add = [&](int w) {
                const float4 o = part[(e * (W + 1) + w) * 32 + lane];
                v[0] = __fadd_rn(v[0], o.x);
                v[1] = __fadd_rn(v[1], o.y);
                v[2] = __fadd_rn(v[2], o.z);
                v[3] = __fadd_rn(v[3], o.w);
            };
            for (int j = 0; j < cnt; ++j) add(w0 + j);
            if (rem) add(W);
            const int64_t tu = (int64_t)min(gid, p.M - 1) * 2 * p.r;
            for (int j0 = 0; j0 < p.r; j0 += 32) {
                const int j = j0 + 8 * tig;
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                const bool on = j < p.r;
                const uint4 b0 = on ? *reinterpret_cast<const uint4*>(p.B + fg + j) : z;
                const uint4 b1 = on ? *reinterpret_cast<const uint4*>(p.B + fu + j) : z;
                const uint4 u0 = on ? *reinterpret_cast<const uint4*>(p.sU + tu + j) : z;
                const uint4 u1 = on ? *reinterpret_cast<const uint4*>(p.sU + tu + p.r + j) : z;
                mma_16816(v, b0.x, 0u, b0.y, 0u, u0.x, u0.y);
                mma_16816(v, b0.z, 0u, b0.w, 0u, u0.z, u0.w);
                mma_16816(v, 0u, b1.x, 0u, b1.y, u1.x, u1.y);
                mma_16816(v, 0u, b1.z, 0u, b1.w, u1.z, u1.w);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = 2 * tig + h;
                if (m >= p.M || abort_flag || !QLORA_CHECK(f < p.F)) continue;
                const float g = v[h], u1 = v[2 + h];
                const float y = (p.act == ACT_SILU ? act_value(ACT_SILU, g) : act_value(ACT_GELU_TANH, g)) * u1;
                p.H[(int64_t)m * p.F + f] = (uint16_t)(pack_bf16x2(y, 0.0f) & 0xFFFFu);
                if (p.GU) {
                    p.GU[(int64_t)m * 2 * p.F + f] = (uint16_t)(pack_bf16x2(g, 0.0f) & 0xFFFFu);
                    p.GU[(int64_t)m * 2 * p.F + p.F + f] = (uint16_t)(pack_bf16x2(u1, 0.0f) & 0xFFFFu);
                }
            }
        }
        item0 += chunk;
        if (item0 >= i_end) break;
        n_items = min(chunk, i_end - item0);
        next = start();
        if (!dead) {
#pragma unroll
            for (int i = 0; i < S::STAGES - 1; ++i) fetch(raw[i], i, next);
        }
        __syncthreads();  // the partial sums are read
    }
    // (every load has landed: a unit that was fetched has been waited for,
    // unless a wait ran out)
    if (dead) {
        for (int i = 0; i < S::STAGES; ++i) mbar_wait(full0 + 8u * i, (phases >> i) & 1u, wc);
    }
}

}  // namespace qlora
