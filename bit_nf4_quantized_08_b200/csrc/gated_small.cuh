// gated_small.cuh -- the gated feed-forward's forward for few tokens (M <= 128:
// decoding and small batches), where the frozen weight is streamed once and
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
// token count: the issue cost of small products bounds that form.)  The token
// tile's unused rows hold whatever follows it in shared memory; they only
// reach accumulator rows that nobody reads.
//
// The units, tiles x KS with KS = K/64 + ceil(2r/64), are split evenly over a
// persistent grid of one CTA per SM (stream-K).  A tile's g and u sit in one
// accumulator, so a CTA that holds a whole tile forms H from it; where a tile
// is cut between CTAs each publishes its fp32 partial sums and the one that
// arrives last (an integer counter with a launch epoch) adds them in CTA order
// (deterministic) and forms H.  Nothing waits on another CTA.
//
// Roles: warp 0 issues the TMA loads (codes, X or sU), warp 1 the MMAs, warps
// 2-5 drain the accumulators (double-buffered in TMEM), and two groups of
// eight dequant warps expand alternate units, one thread per weight row, the
// block constants straight from the 8-bit codes two visits ahead.
#pragma once

#include "common.cuh"
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

template <int TOK>
struct GatedSmallShape {
    static constexpr int NG = 2;                     // dequant groups
    static constexpr int B_BYTES = 256 * 128;        // 256 weight rows x 64 k bf16
    static constexpr int B_SLOTS = TOK <= 32 ? 4 : 3;
    static constexpr int CODE_BYTES = 256 * 32;
    static constexpr int X_BYTES = TOK * 128;
    static constexpr int T_BYTES = CODE_BYTES + X_BYTES;
    static constexpr int T_STAGES = TOK <= 16 ? 8 : TOK <= 32 ? 7 : TOK <= 64 ? 6 : 4;
    // A group's wait for a stage's phase must never find the phase before it
    // open: either the group meets the stage every time, or the stage's last
    // unit lies behind one whose products the group has waited for.
    static_assert(T_STAGES % NG == 0 || T_STAGES >= NG + B_SLOTS, "phase parities");
    static constexpr int T_OFF = B_BYTES * B_SLOTS;
    // the products read 128 token rows from the last stage's X tile on
    static constexpr int T_END = T_OFF + T_BYTES * T_STAGES + (128 - TOK) * 128;
    static constexpr int T8_OFF = T_END;
    static constexpr int BAR_OFF = T8_OFF + 1024;
    static constexpr int SMEM = BAR_OFF + 512 + 1024;
    static constexpr int FIRST_DQ_WARP = 6;
    static constexpr int THREADS = 32 * (FIRST_DQ_WARP + 8 * NG);
    static_assert(SMEM <= 232448, "shared memory per CTA");
};

template <int TOK>
__global__ void __launch_bounds__(GatedSmallShape<TOK>::THREADS, 1)
    k_gated_small(const __grid_constant__ GatedSmallParams p) {
    using S = GatedSmallShape<TOK>;
    constexpr int TS = S::T_STAGES, BS = S::B_SLOTS, NG = S::NG;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw_base);
    float* t8s = reinterpret_cast<float*>(gbase + S::T8_OFF);
    auto slotB = [&](int a) { return base + (uint32_t)(a * S::B_BYTES); };
    auto stC = [&](int s) { return base + (uint32_t)(S::T_OFF + s * S::T_BYTES); };
    auto stX = [&](int s) { return base + (uint32_t)(S::T_OFF + s * S::T_BYTES + S::CODE_BYTES); };
    const uint32_t bar = base + S::BAR_OFF;
    auto full_tma = [&](int s) { return bar + 8u * s; };
    auto empty_tma = [&](int s) { return bar + 8u * (TS + s); };
    auto b_full = [&](int a) { return bar + 8u * (2 * TS + a); };
    auto b_empty = [&](int a) { return bar + 8u * (2 * TS + BS + a); };
    auto acc_full = [&](int b) { return bar + 8u * (2 * TS + 2 * BS + b); };
    auto acc_empty = [&](int b) { return bar + 8u * (2 * TS + 2 * BS + 2 + b); };
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(gbase + S::BAR_OFF + 8 * (2 * TS + 2 * BS + 4));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    volatile int* last_flag = reinterpret_cast<volatile int*>(tmem_holder + 2);
    static_assert(8 * (2 * TS + 2 * BS + 4) + 16 <= 512, "barriers");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCfg wc{p.timeout_ns};
    const int KS = p.ks_main + p.ks_lora;
    const int64_t I = (int64_t)p.tiles * KS;
    const int G = gridDim.x;
    const int64_t r_begin = I * blockIdx.x / G;
    const int64_t r_end = I * (blockIdx.x + 1) / G;
    const int nunits = (int)(r_end - r_begin);

    if (threadIdx.x == 0) {
        for (int s = 0; s < TS; ++s) {
            mbar_init(full_tma(s), 1);
            mbar_init(empty_tma(s), 1);
        }
        for (int a = 0; a < BS; ++a) {
            mbar_init(b_full(a), 8);  // the eight warps of the unit's dequant group
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
        // ------------------------------------------------------------ producer
        if (lane == 0 && !p.inject) {
            bool waited = false;
            int last_use[TS];
            for (int s = 0; s < TS; ++s) last_use[s] = -1;
            int tile = (int)(r_begin / KS), k = (int)(r_begin - (int64_t)tile * KS);
            for (int it = 0; it < nunits; ++it) {
                const int s = it % TS, u = it / TS;
                if (!mbar_wait(empty_tma(s), (u & 1) ^ 1, wc)) { *abort_flag = 1; break; }
                if (k < p.ks_main) {
                    mbar_arrive_expect_tx(full_tma(s), S::CODE_BYTES + S::X_BYTES);
                    tma_load_2d(stC(s), &p.tmCodes, full_tma(s), k * 32, tile * 128);
                    tma_load_2d(stC(s) + S::CODE_BYTES / 2, &p.tmCodes, full_tma(s), k * 32, p.F + tile * 128);
                    tma_load_2d(stX(s), &p.tmX, full_tma(s), k * 64, 0);
                } else {
                    // adapter step: the sU tile here; the B rows are loaded
                    // into the unit's slot by its dequant group
                    if (!waited) {
                        pdl_wait();
                        waited = true;
                    }
                    mbar_arrive_expect_tx(full_tma(s), S::X_BYTES);
                    tma_load_2d(stX(s), &p.tmU, full_tma(s), (k - p.ks_main) * 64, 0);
                }
                last_use[s] = u;
                if (++k == KS) {
                    k = 0;
                    ++tile;
                }
            }
            for (int s = 0; s < TS; ++s)
                if (last_use[s] >= 0) mbar_wait(full_tma(s), last_use[s] & 1, wc);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(128, 256, 0, 0);
            bool ok = true;
            int seg = 0, it = 0;
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
                for (int j = 0; ok && j < len; ++j, ++it) {
                    const int s = it % TS, a = it % BS;
                    if (!mbar_wait(b_full(a), (it / BS) & 1, wc)) { ok = false; *abort_flag = 1; break; }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(tmem + (uint32_t)(ab * 256), smem_desc_sw128(stX(s) + kk * 32, 16, 1024),
                                  smem_desc_sw128(slotB(a) + kk * 32, 16, 1024), idesc, (j > 0 || kk > 0) ? 1u : 0u);
                    umma_commit(b_empty(a));
                    umma_commit(empty_tma(s));
                }
                umma_commit(acc_full(ab));  // one phase per segment, also when cut short
                ++seg;
            }
            if (!ok && seg > 0) mbar_wait(acc_full((seg - 1) & 1), ((seg - 1) >> 1) & 1, wc);
        }
    } else if (warp < S::FIRST_DQ_WARP) {
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
            if (!dead && !__all_sync(0xffffffffu, mbar_wait(acc_full(ab), (seg >> 1) & 1, wc))) {
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
                int last = 0;
                if (!*abort_flag) {
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
                }
                *last_flag = last;
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
    } else {
        // ------------------------------------------------------------ dequant groups
        const int dw = warp - S::FIRST_DQ_WARP;
        const int g = dw >> 3;               // this warp's group: units it with it % NG == g
        const int t = (dw & 7) * 32 + lane;  // weight row of the unit: 0..127 gate, 128..255 up
        const int64_t row0 = (t < 128 ? 0 : (int64_t)p.F - 128) + t;
        const uint32_t code_off = sw32(t * 32), code_off2 = sw32(t * 32 + 16);
        const uint32_t out_off = t * 128;
        const float off = p.dq ? *p.offset : 0.0f;
        struct Raw {
            int q;    // q8 code, or -1 for an adapter step
            float c;  // c1 (double quantization) or absmax
        };
        // raw block constant of the unit at (tile, k)
        auto fetch = [&](bool on, int tile, int k) -> Raw {
            Raw r{-1, 0.0f};
            if (!on || k >= p.ks_main) return r;
            const int64_t b = ((row0 + (int64_t)tile * 128) * p.kbs + k) >> p.fmt.bs_shift;
            if (!p.dq) {
                r.q = 0;
                r.c = __ldg(p.absmax + b);
            } else {
                r.q = __ldg(p.q8 + b);
                r.c = __ldg(p.c1 + (b >> 8));
            }
            return r;
        };
        struct Pos {
            int tile, k;
        };
        auto advance = [&](Pos x) {
            x.k += NG;
            while (x.k >= KS) {
                x.k -= KS;
                ++x.tile;
            }
            return x;
        };
        Pos p0;
        p0.tile = (int)((r_begin + g) / KS);
        p0.k = (int)(r_begin + g - (int64_t)p0.tile * KS);
        Pos p1 = advance(p0);
        Raw r0 = fetch(g < nunits, p0.tile, p0.k), r1 = fetch(g + NG < nunits, p1.tile, p1.k);
        bool dead = false;
        for (int it = g; it < nunits; it += NG) {
            const Raw rw = r0;
            const Pos at = p0;
            const Pos p2 = advance(p1);
            r0 = r1;
            r1 = fetch(it + 2 * NG < nunits, p2.tile, p2.k);
            p0 = p1;
            p1 = p2;
            if (dead) continue;
            const int s = it % TS, a = it % BS;
            if (!__all_sync(0xffffffffu, mbar_wait(full_tma(s), (it / TS) & 1, wc)) ||
                !__all_sync(0xffffffffu, mbar_wait(b_empty(a), ((it / BS) & 1) ^ 1, wc))) {
                *abort_flag = 1;
                dead = true;
                continue;
            }
            if (at.k >= p.ks_main) {
                // Adapter step: one thread loads the 256 B rows; its arrival
                // carries the transaction bytes, the other warps arrive below.
                // The up rows' columns are shifted by r, and the loads' zero
                // fill makes the block-diagonal operand against [U_gate | U_up].
                if ((dw & 7) == 0) {
                    if (lane == 0) {
                        const int x = (at.k - p.ks_main) * 64;
                        mbar_arrive_expect_tx(b_full(a), S::B_BYTES);
                        tma_load_2d(slotB(a), &p.tmB, b_full(a), x, at.tile * 128);
                        tma_load_2d(slotB(a) + S::B_BYTES / 2, &p.tmB, b_full(a), x - p.r, p.F + at.tile * 128);
                    }
                    continue;
                }
            } else {
                const uint32_t sB = slotB(a), sC = stC(s);
                const uint4 c0 = ld_shared_v4(sC + code_off);
                const uint4 c1 = ld_shared_v4(sC + code_off2);
                const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                const float bc = p.dq ? __fadd_rn(__fmul_rn(t8s[rw.q], rw.c), off) : rw.c;
                const Nf4BlockTable tb = nf4_block_table(bc, p.fmt.code_type);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint32_t o[4];
                    nf4_expand_word(words[q], tb, o);
                    st_shared_v4(sB + sw128(out_off + q * 16), o[0], o[1], o[2], o[3]);
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(b_full(a));
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

}  // namespace qlora
