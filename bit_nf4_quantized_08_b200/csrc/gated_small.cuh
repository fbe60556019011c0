// gated_small.cuh -- the gated feed-forward's forward for 9 to 128 tokens
// (decoding in batches), where the frozen weight is streamed once and
// the NF4 expansion sets the pace.
//
//   H = act(g) u,   [g | u] = X W'^T + sU B^T  (adapters of the two halves)
//
// The weight rows are the MMA's N side: a unit of work is (128 hidden columns,
// one 64-element k-step), i.e. 128 gate rows and the 128 matching up rows as
// one 256-column operand against up to 128 tokens, so that one step of four
// 128 x 256 x 16 products (about 0.28 us) consumes 16384 weights.  (With the
// weight rows on the 128-row M side, as in the plain small-M linear, the same
// four issues and two commits consume 8192 in about 0.45 us, whatever the
// token count: the issue cost of small products bounds that form; projection
// and activation apart took 186 us on LLaMA-65B at 48 tokens, this 147 us.)
// The token tile's unused rows hold whatever follows it in shared memory; they
// only reach accumulator rows that nobody reads.
//
// The units, tiles x KS with KS = K/64 + ceil(2r/64), are split evenly over a
// persistent grid of one CTA per SM (stream-K).  A tile's g and u sit in one
// accumulator, so a CTA that holds a whole tile forms H from it; where a tile
// is cut between CTAs each publishes its fp32 partial sums and the one that
// arrives last (an integer counter with a launch epoch) adds them in CTA order
// (deterministic) and forms H.  Nothing waits on another CTA.
//
// Roles: warp 0 loads the codes and warp 6 the token tiles (X or sU) with TMA,
// warp 1 issues the MMAs, warps 2-5 drain the accumulators (double-buffered in
// TMEM), and three groups of eight dequant warps expand the units in turn, one
// thread per weight row, the block constants straight from the 8-bit codes.
// Warp 7 is idle: the groups start on a multiple of the four schedulers.
//
// Bound by the expansion (its integer pipe is busy for 64 % of the time) and
// the hand-overs between loads, expansion and products, not by HBM: codes and
// constants are 46 MB on LLaMA-7B (7 us) and 186 MB on LLaMA-65B (28 us).
// Measured with cold caches, kernel alone: LLaMA-65B 133 us at 48 tokens (1.4
// TB/s), LLaMA-7B 44 us at 16 or fewer (1.1 TB/s).  With two groups instead of three
// 65B took 151 us; two block columns a slot, 128-byte code lines, or a table of
// code pairs in shared memory instead of the byte permutes were no faster.
#pragma once

#include "common.cuh"
#include "dropout.cuh"
#include "gated.cuh"
#include "gemm.cuh"
#include "nf4.cuh"
#include "smallm_mma.cuh"

namespace qlora {

struct GatedSmallParams {
    CUtensorMap tmCodes;  // codes [2F][K/2] bytes, box {32 B, 128 rows}, 32-byte swizzle
    CUtensorMap tmX;      // X [M][K] bf16, box {64, TOK}, 128-byte swizzle
    CUtensorMap tmB;      // B [2F][r] bf16, box {64, 128}, 128-byte swizzle
    CUtensorMap tmU;      // sU [M][2r] bf16, box {64, TOK}, 128-byte swizzle
    const uint8_t* q8;
    const float* c1;
    const float* offset;
    const float* absmax;  // without double quantization
    int dq;
    int F, M, kbs;        // kbs = K / 64
    int ks_main, ks_lora, tiles, r, act;
    QFormat fmt;
    uint16_t* H;          // [M][F]
    uint16_t* GU;         // [M][2F] or nullptr
    float* part;          // [gridDim.x][2][M][256] fp32 partial tiles
    unsigned long long* counters;  // [tiles]: (epoch << 32) | arrivals
    int64_t part_cap;     // capacity of part (floats): bounds checks of the debug build
    uint32_t epoch;       // nonzero
    uint64_t timeout_ns;
    int inject;
};

// nf4_block_table with a code book known at compile time.
template <int CT>
__device__ constexpr uint32_t code_bits_of(int j) {
    constexpr uint32_t v[2][16] = {{QLORA_NF4_BITS}, {QLORA_FP4_BITS}};
    return v[CT][j];
}
template <int CT>
__device__ __forceinline__ Nf4BlockTable nf4_block_table_of(float a) {
    uint32_t P[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        P[i] = pack_bf16x2(__fmul_rn(__uint_as_float(code_bits_of<CT>(2 * i)), a),
                           __fmul_rn(__uint_as_float(code_bits_of<CT>(2 * i + 1)), a));
    Nf4BlockTable t;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        t.L[q] = prmt(P[2 * q], P[2 * q + 1], 0x6420u);
        t.H[q] = prmt(P[2 * q], P[2 * q + 1], 0x7531u);
    }
    return t;
}

template <int TOK>
struct GatedSmallShape {
    // Two rings: code stages (released by the dequant warps) and operand slots, the expanded rows or the adapters' B
    // rows and the token tile, released together by one tcgen05.commit.
    static constexpr int NG = 3;                     // dequant groups
    static constexpr int CODE_BYTES = 256 * 32;      // 256 weight rows x 64 codes
    static constexpr int C_STAGES = 6;
    static constexpr int B_BYTES = 256 * 128;        // 256 weight rows x 64 k bf16
    static constexpr int X_BYTES = TOK * 128;
    static constexpr int SLOT = B_BYTES + X_BYTES;
    static constexpr int SLOTS = TOK <= 64 ? 4 : 3;
    static constexpr int C_OFF = SLOT * SLOTS;       // (the last slot's products read up to 14 KB past it)
    static constexpr int T8_OFF = C_OFF + CODE_BYTES * C_STAGES;
    static constexpr int BAR_OFF = T8_OFF + 1024;
    static constexpr int SMEM = BAR_OFF + 512 + 1024;
    static constexpr int FIRST_DQ_WARP = 8;
    static constexpr int THREADS = 32 * (FIRST_DQ_WARP + 8 * NG);
    static_assert(SMEM <= 232448, "shared memory per CTA");
    static_assert(CODE_BYTES * C_STAGES >= (128 - TOK) * 128, "rows past the last token tile are readable");
    // A group's wait for a phase of a stage or slot must never find the phase
    // before it open: it meets the same stages every time, and the slot's use
    // before last lies behind products that it has waited for.
    static_assert(C_STAGES % NG == 0 && SLOTS >= NG, "phase parities");
};

template <int TOK>
__global__ void __launch_bounds__(GatedSmallShape<TOK>::THREADS, 1)
    k_gated_small(const __grid_constant__ GatedSmallParams p) {
    using S = GatedSmallShape<TOK>;
    constexpr int CS = S::C_STAGES, BS = S::SLOTS, NG = S::NG;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw_base);
    float* t8s = reinterpret_cast<float*>(gbase + S::T8_OFF);
    auto slotB = [&](int a) { return base + (uint32_t)(a * S::SLOT); };
    auto slotX = [&](int a) { return base + (uint32_t)(a * S::SLOT + S::B_BYTES); };
    auto stC = [&](int s) { return base + (uint32_t)(S::C_OFF + s * S::CODE_BYTES); };
    const uint32_t bar = base + S::BAR_OFF;
    auto c_full = [&](int s) { return bar + 8u * s; };
    auto c_empty = [&](int s) { return bar + 8u * (CS + s); };
    auto b_full = [&](int a) { return bar + 8u * (2 * CS + a); };
    auto b_empty = [&](int a) { return bar + 8u * (2 * CS + BS + a); };
    auto acc_full = [&](int b) { return bar + 8u * (2 * CS + 2 * BS + b); };
    auto acc_empty = [&](int b) { return bar + 8u * (2 * CS + 2 * BS + 2 + b); };
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(gbase + S::BAR_OFF + 8 * (2 * CS + 2 * BS + 4));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    volatile int* last_flag = reinterpret_cast<volatile int*>(tmem_holder + 2);
    static_assert(8 * (2 * CS + 2 * BS + 4) + 16 <= 512, "barriers");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCfg wc{p.timeout_ns};
    const int KS = p.ks_main + p.ks_lora;
    const int64_t I = (int64_t)p.tiles * KS;
    const int G = gridDim.x;
    const int64_t r_begin = I * blockIdx.x / G;
    const int64_t r_end = I * (blockIdx.x + 1) / G;
    const int nunits = (int)(r_end - r_begin);

    if (threadIdx.x == 0) {
        for (int s = 0; s < CS; ++s) {
            mbar_init(c_full(s), 1);
            mbar_init(c_empty(s), 8);  // the eight warps of the unit's dequant group
        }
        for (int a = 0; a < BS; ++a) {
            mbar_init(b_full(a), 9);  // those warps, and the loads of the token tile
            mbar_init(b_empty(a), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 4);  // the four epilogue warps
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 256; i += blockDim.x)
        t8s[i] = dq_value(p.fmt.dq_type, (p.fmt.dq_type == 0 || i < 253) ? i : 0);
    if (warp == 0 && lane == 0) {
        pdl_trigger();
        prefetch_tensormap(&p.tmCodes);
        prefetch_tensormap(&p.tmX);
        if (p.ks_lora) {
            prefetch_tensormap(&p.tmB);
            prefetch_tensormap(&p.tmU);
        }
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // Dependent launch: with adapters the kernel before is the sU GEMM, which
    // waited for its own predecessors before it let this one start, so only sU
    // needs the wait (the producer takes it before the first adapter step).
    // Without adapters every thread waits here.
    if (p.ks_lora == 0) pdl_wait();

    if (warp == 0) {
        // ------------------------------------------------------------ code producer
        if (lane == 0 && !p.inject) {
            int last_use[CS];
            for (int s = 0; s < CS; ++s) last_use[s] = -1;
            int tile = (int)(r_begin / KS), k = (int)(r_begin - (int64_t)tile * KS);
            for (int it = 0; it < nunits; ++it) {
                const int s = it % CS, u = it / CS;
                if (!mbar_wait_hint(c_empty(s), (u & 1) ^ 1, wc, 1000)) { *abort_flag = 1; break; }
                if (k < p.ks_main) {
                    mbar_arrive_expect_tx(c_full(s), S::CODE_BYTES);
                    tma_load_2d(stC(s), &p.tmCodes, c_full(s), k * 32, tile * 128);
                    tma_load_2d(stC(s) + S::CODE_BYTES / 2, &p.tmCodes, c_full(s), k * 32, p.F + tile * 128);
                } else {
                    mbar_arrive(c_full(s));  // an adapter step has no codes
                }
                last_use[s] = u;
                if (++k == KS) {
                    k = 0;
                    ++tile;
                }
            }
            for (int s = 0; s < CS; ++s)
                if (last_use[s] >= 0) mbar_wait(c_full(s), last_use[s] & 1, wc);
        }
    } else if (warp == 6) {
        // ------------------------------------------------------------ producer of the token tiles and B rows
        if (lane == 0 && !p.inject) {
            bool waited = false;
            int last_use[BS];
            for (int a = 0; a < BS; ++a) last_use[a] = -1;
            int tile = (int)(r_begin / KS), k = (int)(r_begin - (int64_t)tile * KS);
            for (int it = 0; it < nunits; ++it) {
                const int a = it % BS, u = it / BS;
                if (!mbar_wait_hint(b_empty(a), (u & 1) ^ 1, wc, 1000)) { *abort_flag = 1; break; }
                if (k < p.ks_main) {
                    mbar_arrive_expect_tx(b_full(a), S::X_BYTES);
                    tma_load_2d(slotX(a), &p.tmX, b_full(a), k * 64, 0);
                } else {
                    // adapter step: sU, from the kernel before this one, and
                    // the B rows in place of the expanded weight.  The up
                    // rows' columns are shifted by r, and the loads' zero fill
                    // makes the block-diagonal operand against [U_gate | U_up].
                    if (!waited) {
                        pdl_wait();
                        waited = true;
                    }
                    const int x = (k - p.ks_main) * 64;
                    mbar_arrive_expect_tx(b_full(a), S::X_BYTES + S::B_BYTES);
                    tma_load_2d(slotX(a), &p.tmU, b_full(a), x, 0);
                    tma_load_2d(slotB(a), &p.tmB, b_full(a), x, tile * 128);
                    tma_load_2d(slotB(a) + S::B_BYTES / 2, &p.tmB, b_full(a), x - p.r, p.F + tile * 128);
                }
                last_use[a] = u;
                if (++k == KS) {
                    k = 0;
                    ++tile;
                }
            }
            // every load has landed before the CTA exits (after an abort this
            // may run into its bound: the phase needs the dequant warps too)
            for (int a = 0; a < BS; ++a)
                if (last_use[a] >= 0) mbar_wait(b_full(a), last_use[a] & 1, wc);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(128, 256, 0, 0);
            const uint64_t xd0 = smem_desc_sw128(slotX(0), 16, 1024), bd0 = smem_desc_sw128(slotB(0), 16, 1024);
            bool ok = true;
            int seg = 0, it = 0;
            uint32_t a = 0, ph = 0;  // slot and phase of unit it
            while (ok && it < nunits) {
                const int64_t unit0 = r_begin + it;
                const int k0 = (int)(unit0 % KS);
                const int len = (int)min((int64_t)(KS - k0), (int64_t)(nunits - it));
                const int ab = seg & 1;
                if (seg >= 2 && !mbar_wait(acc_empty(ab), ((seg >> 1) - 1) & 1, wc)) {
                    ok = false;
                    *abort_flag = 1;
                }
                tc_fence_after();
                const uint32_t acc = tmem + (uint32_t)(ab * 256);
                for (int j = 0; ok && j < len; ++j, ++it) {
                    if (!mbar_wait(b_full((int)a), ph, wc)) { ok = false; *abort_flag = 1; break; }
                    tc_fence_after();
                    const uint64_t so = (uint64_t)(a * (uint32_t)(S::SLOT >> 4));
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk)
                        umma_bf16(acc, xd0 + so + 2 * kk, bd0 + so + 2 * kk, idesc, (j > 0 || kk > 0) ? 1u : 0u);
                    umma_commit(b_empty((int)a));
                    if (++a == (uint32_t)BS) {
                        a = 0;
                        ph ^= 1u;
                    }
                }
                umma_commit(acc_full(ab));  // one phase per segment, also when cut short
                ++seg;
            }
            if (!ok && seg > 0) mbar_wait(acc_full((seg - 1) & 1), ((seg - 1) >> 1) & 1, wc);
        }
    } else if (warp < 6) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;
        const int m = quarter * 32 + lane;  // TMEM lane = token
        const bool live = m < p.M;
        const bool warp_live = quarter * 32 < p.M;
        const int et = threadIdx.x - 64;    // 0..127
        const int F = p.F;
        auto store_h = [&](int tok, int f, const float (&g)[4], const float (&u)[4]) {  // four hidden columns
            float h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = (p.act == ACT_SILU ? act_value(ACT_SILU, g[i]) : act_value(ACT_GELU_TANH, g[i])) * u[i];
            if (!QLORA_CHECK(tok < p.M && f + 4 <= F)) return;
            *reinterpret_cast<uint2*>(p.H + (int64_t)tok * F + f) =
                make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
            if (p.GU) {
                uint16_t* o = p.GU + (int64_t)tok * 2 * F + f;
                *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]));
                *reinterpret_cast<uint2*>(o + F) = make_uint2(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]));
            }
        };
        bool dead = false;
        int seg = 0;
        for (int it = 0; it < nunits; ++seg) {
            const int64_t unit0 = r_begin + it;
            const int tile = (int)(unit0 / KS), k0 = (int)(unit0 - (int64_t)tile * KS);
            const int len = (int)min((int64_t)(KS - k0), (int64_t)(nunits - it));
            it += len;
            const int ab = seg & 1;
            const bool whole = k0 == 0 && len == KS;
            if (!dead && !__all_sync(0xffffffffu, mbar_wait_hint(acc_full(ab), (seg >> 1) & 1, wc, 4000))) {
                *abort_flag = 1;
                dead = true;
            }
            float* mine = p.part + ((int64_t)blockIdx.x * 2 + (k0 != 0 ? 0 : 1)) * p.M * 256;
            if (!dead && warp_live) {
                tc_fence_after();
                const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(ab * 256);
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    uint32_t g[32], u[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(ta + (uint32_t)c, g);
                    tmem_ld_32x32b_x32(ta + (uint32_t)(128 + c), u);
                    tmem_ld_wait();
                    if (!live) continue;
                    if (whole) {
#pragma unroll
                        for (int q = 0; q < 32; q += 4) {
                            const float gq[4] = {__uint_as_float(g[q]), __uint_as_float(g[q + 1]),
                                                 __uint_as_float(g[q + 2]), __uint_as_float(g[q + 3])};
                            const float uq[4] = {__uint_as_float(u[q]), __uint_as_float(u[q + 1]),
                                                 __uint_as_float(u[q + 2]), __uint_as_float(u[q + 3])};
                            store_h(m, tile * 128 + c + q, gq, uq);
                        }
                    } else {
                        uint4* o = reinterpret_cast<uint4*>(mine + (int64_t)m * 256 + c);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            if (!QLORA_CHECK((mine - p.part) + (int64_t)m * 256 + c + 128 + 4 * q + 4 <= p.part_cap)) continue;
                            __stcg(o + q, make_uint4(g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]));
                            __stcg(o + 32 + q, make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]));
                        }
                    }
                }
            }
            // the accumulator buffer is free for the segment after next
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && !dead) mbar_arrive(acc_empty(ab));
            if (whole) continue;
            // Part of a tile: the four warps meet whatever happened, so that
            // the named barriers are always met.
            const int64_t t0 = (int64_t)tile * KS;
            const int cf = owner_cta(t0, I, G), cl = owner_cta(t0 + KS - 1, I, G);  // (no share is empty)
            __threadfence();
            named_bar(1, 128);
            if (et == 0) {
                // (also after an abort, so that the count starts at 0 again
                // when a captured launch is replayed)
                int last = 0;
                unsigned long long* ctr = p.counters + tile;
                unsigned long long cv = *reinterpret_cast<volatile unsigned long long*>(ctr);
                const unsigned long long ep = (unsigned long long)p.epoch << 32;
                while (true) {
                    // a value of another epoch counts as no arrivals
                    const bool same = (cv & 0xFFFFFFFF00000000ull) == ep;
                    const unsigned long long want = same ? cv + 1ull : (ep | 1ull);
                    const unsigned long long prev = atomicCAS(ctr, cv, want);
                    if (prev == cv) {
                        last = (int)(want & 0xFFFFFFFFull) == cl - cf + 1;
                        break;
                    }
                    cv = prev;
                }
                if (last) *ctr = 0ull;  // for a replay of this launch
                *last_flag = last && !*abort_flag;
            }
            named_bar(1, 128);
            const bool last = *last_flag != 0;
            named_bar(1, 128);  // (the flag is read before the next segment writes it)
            if (!last) continue;
            __threadfence();
            for (int e = et; e < p.M * 32; e += 128) {
                const int tok = e >> 5, j = (e & 31) * 4;
                float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
                for (int c = cf; c <= cl; ++c) {
                    const int slot = I * c / G > t0 ? 0 : 1;
                    const float* src = p.part + (((int64_t)c * 2 + slot) * p.M + tok) * 256 + j;
                    const float4 a = __ldcg(reinterpret_cast<const float4*>(src));
                    const float4 b = __ldcg(reinterpret_cast<const float4*>(src + 128));
                    g[0] = __fadd_rn(g[0], a.x);
                    g[1] = __fadd_rn(g[1], a.y);
                    g[2] = __fadd_rn(g[2], a.z);
                    g[3] = __fadd_rn(g[3], a.w);
                    u[0] = __fadd_rn(u[0], b.x);
                    u[1] = __fadd_rn(u[1], b.y);
                    u[2] = __fadd_rn(u[2], b.z);
                    u[3] = __fadd_rn(u[3], b.w);
                }
                store_h(tok, tile * 128 + j, g, u);
            }
        }
    } else if (warp >= S::FIRST_DQ_WARP) {
        // ------------------------------------------------------------ dequant groups
        const int dw = warp - S::FIRST_DQ_WARP;
        const int g = dw >> 3;               // this warp's group: units it with it % NG == g
        const int t = (dw & 7) * 32 + lane;  // weight row of the unit: 0..127 gate, 128..255 up
        const int64_t row0 = (t < 128 ? 0 : (int64_t)p.F - 128) + t;
        const uint32_t code_off = sw32(t * 32), code_off2 = sw32(t * 32 + 16);
        const uint32_t row_x = (uint32_t)(t & 7) << 4, out_row = (uint32_t)t * 128u;
        const float off = p.dq ? *p.offset : 0.0f;
        const int sh = p.fmt.bs_shift, ct = p.fmt.code_type;
        // Block constants of this thread's row.  Blocks of 64: the 8-bit codes
        // by the aligned eight, the next eight loaded when these are taken up
        // (nothing touches a loaded value before that), and one c1 for 256
        // blocks; a new tile starts over.  Larger blocks, or fp32 constants:
        // loaded at their use.
        const int64_t nblocks = (int64_t)2 * p.F * p.kbs;  // (a multiple of 512)
        const bool fast = p.dq && sh == 0;
        int64_t wb = 0;  // first block of codes8
        int pos = 0;     // this visit's block - wb
        uint2 codes8 = make_uint2(0u, 0u), codes8_next = codes8;
        float c1 = 0.0f;
        auto load8 = [&](int64_t b) {
            return b < nblocks ? *reinterpret_cast<const uint2*>(p.q8 + b) : make_uint2(0u, 0u);
        };
        auto start_row = [&](int64_t b) {
            wb = b & ~(int64_t)7;
            pos = (int)(b & 7);
            codes8 = load8(wb);
            codes8_next = load8(wb + 8);
            c1 = p.c1[wb >> 8];
        };
        auto block_const = [&](int64_t blk64) -> float {
            if (!fast) {
                const int64_t b = blk64 >> sh;
                if (!p.dq) return __ldg(p.absmax + b);
                return __fadd_rn(__fmul_rn(t8s[__ldg(p.q8 + b)], __ldg(p.c1 + (b >> 8))), off);
            }
            if (pos >= 8) {
                pos -= 8;
                wb += 8;
                codes8 = codes8_next;
                codes8_next = load8(wb + 8);
                if ((wb & 255) == 0) c1 = p.c1[wb >> 8];
            }
            const uint32_t word = pos & 4 ? codes8.y : codes8.x;
            return __fadd_rn(__fmul_rn(t8s[(word >> (8 * (pos & 3))) & 255u], c1), off);
        };
        int tile = (int)((r_begin + g) / KS), k = (int)(r_begin + g - (int64_t)tile * KS);
        int64_t rb = (row0 + (int64_t)tile * 128) * p.kbs;  // the row's first 64-element block
        int s = g % CS, sph = 0, a = g % BS, aph = 1;       // code stage, operand slot, parities to wait for
        if (fast && g < nunits && k < p.ks_main) start_row(rb + k);
        bool dead = false;
        for (int it = g; it < nunits; it += NG) {
            const bool weight = k < p.ks_main;
            const float bc = weight ? block_const(rb + k) : 0.0f;
            if (!dead && (!__all_sync(0xffffffffu, mbar_wait_hint(c_full(s), (uint32_t)sph, wc, 1000)) ||
                          !__all_sync(0xffffffffu, mbar_wait_hint(b_empty(a), (uint32_t)aph, wc, 1000)))) {
                *abort_flag = 1;
                dead = true;
            }
            if (!dead) {
                if (weight) {
                    const uint32_t so = (slotB(a) + out_row) | row_x;  // (rows are 128-byte aligned)
                    const uint4 c0 = ld_shared_v4(stC(s) + code_off);
                    const uint4 c1v = ld_shared_v4(stC(s) + code_off2);
                    const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1v.x, c1v.y, c1v.z, c1v.w};
                    const Nf4BlockTable tb = ct == 0 ? nf4_block_table_of<0>(bc) : nf4_block_table_of<1>(bc);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        uint32_t o[4];
                        nf4_expand_word(words[q], tb, o);
                        st_shared_v4(so ^ (uint32_t)(q << 4), o[0], o[1], o[2], o[3]);
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                // (the code stage is released only here, after the stores that
                // depend on every read of it)
                if (lane == 0) {
                    mbar_arrive(b_full(a));
                    mbar_arrive(c_empty(s));
                }
            }
            k += NG;
            pos += NG;
            if (k >= KS) {
                do {
                    k -= KS;
                    rb += (int64_t)128 * p.kbs;
                } while (k >= KS);
                if (fast && it + NG < nunits && k < p.ks_main) start_row(rb + k);
            }
            s += NG;
            if (s >= CS) {
                s -= CS;
                sph ^= 1;
            }
            a += NG;
            if (a >= BS) {
                a -= BS;
                aph ^= 1;
            }
        }
    }

    // the kernel does not complete before the previous one
    if (threadIdx.x == 0) pdl_wait();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// sU = bf16(scale X A^T) for up to 16 tokens, ahead of the gated kernels and,
// under dropout, of the linear's (DROP: X masked in registers; every CTA forms
// the whole mask, some 2.6 us of generator for 16 tokens of 4096).  A CTA takes
// eight adapter rows, its 32 warps the 64-element block columns in turn; within
// a block thread t of a fragment's group of four holds elements 16 t .. 16 t +
// 15 of its rows for both operands, so that every load is 16 contiguous bytes
// (a sum over k does not depend on its order).  The warps' sums are added in
// warp order.
// Bound by latency: 1 to 2 MB of A through 2r / 8 CTAs, 4.6 us on LLaMA-7B
// against 11 us for the TMA-fed cluster kernel of larger batches, which also
// holds eight SMs' shared memory for that long.  (For more tokens its tiles
// are better: 27 us here against 14 us for 48 tokens, LLaMA-65B.)
// ---------------------------------------------------------------------------
template <bool DROP>
__global__ void __launch_bounds__(1024) k_small_u(const uint16_t* X, const uint16_t* A, uint16_t* U, int M, int K, int rt,
                                                  float scale, const __grid_constant__ DropParams d) {
    __shared__ float part[32][16][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    pdl_wait();
    pdl_trigger();
    const int j0 = blockIdx.x * 8;
    const uint4* av = reinterpret_cast<const uint4*>(A + (int64_t)(j0 + gid) * K + tig * 16);
    const uint4* x0 = reinterpret_cast<const uint4*>(X + (int64_t)gid * K + tig * 16);
    const uint4* x1 = reinterpret_cast<const uint4*>(X + (int64_t)(gid + 8) * K + tig * 16);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const DropCtx ctx = DROP ? drop_ctx(d, drop_offset(d), 0u) : DropCtx{};
    // the 16 elements of row m from column k (16 rows of less than 2^31: the
    // block number fits in 32 bits)
    auto mask = [&](uint4 (&x)[2], int m, int k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t b[4];
            drop_mask8(d, ctx, (uint32_t)(((int64_t)m * K + k) >> 3) + h, b);
            x[h].x &= b[0];
            x[h].y &= b[1];
            x[h].z &= b[2];
            x[h].w &= b[3];
        }
    };
#pragma unroll(DROP ? 1 : 2)
    for (int kb = warp; kb < K / 64; kb += 32) {
        const uint4 b[2] = {av[kb * 8], av[kb * 8 + 1]};
        uint4 lo[2] = {gid < M ? x0[kb * 8] : zero, gid < M ? x0[kb * 8 + 1] : zero};
        uint4 hi[2] = {gid + 8 < M ? x1[kb * 8] : zero, gid + 8 < M ? x1[kb * 8 + 1] : zero};
        if (DROP) {
            mask(lo, gid, kb * 64 + tig * 16);
            if (M > 8) mask(hi, gid + 8, kb * 64 + tig * 16);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            mma_16816(acc, lo[c].x, hi[c].x, lo[c].y, hi[c].y, b[c].x, b[c].y);
            mma_16816(acc, lo[c].z, hi[c].z, lo[c].w, hi[c].w, b[c].z, b[c].w);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][gid + 8 * (e >> 1)][2 * tig + (e & 1)] = acc[e];
    __syncthreads();
    const int m = threadIdx.x >> 3, j = threadIdx.x & 7;
    if (m < M) {
        float v = part[0][m][j];
#pragma unroll
        for (int w = 1; w < 32; ++w) v = __fadd_rn(v, part[w][m][j]);
        U[(int64_t)m * rt + j0 + j] = (uint16_t)(pack_bf16x2(__fmul_rn(v, scale), 0.0f) & 0xFFFFu);
    }
}

}  // namespace qlora
