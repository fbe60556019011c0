// gated_few.cuh -- the gated feed-forward's forward for the fewest tokens
// (decoding), where a weight is used so seldom that expanding it into a
// tensor-core operand in shared memory costs more than the products.
//
//   H = act(g) u,   [g | u] = X W'^T + sU B^T
//
// As in the plain linear for few tokens, the block constant is factored out of
// each 64-element block, so that the inner sums are warp MMAs (m16n8k16) whose
// weight operand comes from a table of code-byte pairs, one shared-memory load
// a register (smallm_mma.cuh has the table, its prescale and the permutation of
// k).  Here the weight is the 16-row operand: 8 gate rows and the 8 up rows of
// the same hidden columns, so that a thread ends with g and u of one column
// and forms H, and the tokens are the 8-column operand.
//
// A unit is (8 hidden columns, 256 elements of k): 16 lines of 128 bytes of
// codes, which every lane loads straight into registers, two units ahead (64
// KB in flight an SM); X comes through L1.  There is no ring, no barrier in the
// loop and no warp that only moves data.  A CTA owns a range of hidden columns; its 16 warps
// take the units in turn and leave fp32 partial sums in shared memory, which
// are added in k order; then the adapters' products and the activation.
#pragma once

#include "common.cuh"
#include "gated.cuh"
#include "nf4.cuh"
#include "smallm_mma.cuh"

namespace qlora {

struct GatedFewParams {
    const uint8_t* codes;  // [2F][K/2]
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
    float inv_scale;       // 1 / the table's prescale
    QFormat fmt;
    uint16_t* H;           // [M][F]
    uint16_t* GU;          // [M][2F] or nullptr
};

// NT: token tiles of 8.
template <int NT>
struct GatedFewShape {
    static constexpr int WARPS = 16;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int CHUNK = NT == 1 ? 10 : 6;             // items (8 hidden columns) between two reductions
    static constexpr int SMEM = CHUNK * WARPS * NT * 32 * 16;  // partial sums
};

template <int NT>
__global__ void __launch_bounds__(GatedFewShape<NT>::THREADS, 1) k_gated_few(const __grid_constant__ GatedFewParams p) {
    using S = GatedFewShape<NT>;
    constexpr int W = S::WARPS;
    extern __shared__ __align__(16) uint8_t few_smem[];
    float4* part = reinterpret_cast<float4*>(few_smem);  // [item of the chunk][warp][NT][lane]
    __shared__ float t8s[256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const uint32_t lane4 = (uint32_t)lane * 4u;
    const int items = p.F / 8;
    const int i_begin = (int)((int64_t)items * blockIdx.x / gridDim.x);
    const int i_end = (int)((int64_t)items * (blockIdx.x + 1) / gridDim.x);
    const int Q = (p.kbs + 3) >> 2;
    const int d_it = W / Q, d_q = W % Q;
    const int64_t ldc = p.K / 2;
    const int sh = p.fmt.bs_shift;

    pdl_trigger();
    // With adapters the kernel before is the one that forms sU, which waited
    // for its own predecessors before it let this one start.
    if (p.r == 0) pdl_wait();

    // A unit's codes (bytes 8 tig .. 8 tig + 7 of four 32-byte blocks, of a gate
    // and an up row) and, for block column 4 q + tig, the raw block constants.
    struct In {
        uint2 c[4][2];
        float s[2];
        uint32_t q[2];
    };
    auto fetch = [&](int it, int q, int n_items, int item0) {
        In x;
        const bool on = it < n_items;
        const int64_t row = (int64_t)(item0 + it) * 8 + gid;
        const uint8_t* cg = p.codes + row * ldc + q * 128 + tig * 8;
        const uint8_t* cu = cg + (int64_t)p.F * ldc;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool ok = on && 4 * q + i < p.kbs;
            x.c[i][0] = ok ? __ldcs(reinterpret_cast<const uint2*>(cg + 32 * i)) : make_uint2(0u, 0u);
            x.c[i][1] = ok ? __ldcs(reinterpret_cast<const uint2*>(cu + 32 * i)) : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t b = ((row + (int64_t)h * p.F) * p.kbs + 4 * q + tig) >> sh;
            const bool ok = on && 4 * q + tig < p.kbs;
            x.q[h] = ok && p.dq ? (uint32_t)p.q8[b] : 0u;
            x.s[h] = ok ? (p.dq ? p.c1[b >> 8] : p.absmax[b]) : 0.0f;
        }
        return x;
    };

    int item0 = i_begin, n_items = min(S::CHUNK, i_end - i_begin);
    const int it_w = warp / Q, q_w = warp - it_w * Q;  // the warp's first unit of a chunk
    In a = fetch(it_w, q_w, n_items, item0);

    // the table and the 8-bit code book, while the first loads are on their way
    {
        const float L = small_m_table_scale(p.fmt.code_type);
        for (int idx = threadIdx.x; idx < 256 * 32; idx += S::THREADS) {
            const int e = idx >> 5;
            g_small_m_lut[idx] = pack_bf16x2(__fmul_rn(code_value(p.fmt.code_type, e >> 4), L),
                                             __fmul_rn(code_value(p.fmt.code_type, e & 15), L));
        }
    }
    for (int i = threadIdx.x; i < 256; i += S::THREADS)
        t8s[i] = dq_value(p.fmt.dq_type, (p.fmt.dq_type == 0 || i < 253) ? i : 0);
    const float off = p.dq ? *p.offset : 0.0f;
    __syncthreads();

    for (; item0 < i_end; item0 += S::CHUNK) {
        n_items = min(S::CHUNK, i_end - item0);
        if (item0 != i_begin) a = fetch(it_w, q_w, n_items, item0);
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;

        auto consume = [&](const In& x, int q) {
            float sc[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                sc[h] = (p.dq ? __fadd_rn(__fmul_rn(t8s[x.q[h]], x.s[h]), off) : x.s[h]) * p.inv_scale;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * q + i >= p.kbs) break;
                float d[NT][4];
                const float sg = __shfl_sync(0xffffffffu, sc[0], (lane & 28) | i);
                const float su = __shfl_sync(0xffffffffu, sc[1], (lane & 28) | i);
                uint4 xv[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int tok = 8 * n + gid;
                    const uint4* src =
                        reinterpret_cast<const uint4*>(p.X + (int64_t)tok * p.K + (4 * q + i) * 64 + tig * 16);
                    xv[n][0] = tok < p.M ? src[0] : make_uint4(0u, 0u, 0u, 0u);
                    xv[n][1] = tok < p.M ? src[1] : make_uint4(0u, 0u, 0u, 0u);
                }
                const uint32_t wg[2] = {x.c[i][0].x, x.c[i][0].y}, wu[2] = {x.c[i][1].x, x.c[i][1].y};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = 2 * (j & 1);
                    const uint32_t a0 = lut_byte(wg[j >> 1], k, lane4), a1 = lut_byte(wu[j >> 1], k, lane4);
                    const uint32_t a2 = lut_byte(wg[j >> 1], k + 1, lane4), a3 = lut_byte(wu[j >> 1], k + 1, lane4);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 v = xv[n][j >> 1];
                        const uint32_t b0 = j & 1 ? v.z : v.x, b1 = j & 1 ? v.w : v.y;
                        if (j == 0)
                            mma_16816_z(d[n], a0, a1, a2, a3, b0, b1);
                        else
                            mma_16816(d[n], a0, a1, a2, a3, b0, b1);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] = __fmaf_rn(sg, d[n][0], acc[n][0]);
                    acc[n][1] = __fmaf_rn(sg, d[n][1], acc[n][1]);
                    acc[n][2] = __fmaf_rn(su, d[n][2], acc[n][2]);
                    acc[n][3] = __fmaf_rn(su, d[n][3], acc[n][3]);
                }
            }
        };

        int it = it_w, q = q_w;
        int itn = it + d_it, qn = q + d_q;  // the unit after it
        if (qn >= Q) { qn -= Q; ++itn; }
        In b = fetch(itn, qn, n_items, item0);
        while (it < n_items) {
            int it2 = itn + d_it, q2 = qn + d_q;
            if (q2 >= Q) { q2 -= Q; ++it2; }
            const In c = fetch(it2, q2, n_items, item0);
            consume(a, q);
            if (itn != it) {  // the warp's last unit of this item
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    part[((it * W + warp) * NT + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
                }
            }
            a = b;
            b = c;
            it = itn;
            q = qn;
            itn = it2;
            qn = q2;
        }
        if (p.r > 0) pdl_wait();  // sU
        __syncthreads();

        // an item a warp: the partial sums in the order of their first block
        // column, then the adapters
        for (int e = warp; e < n_items; e += W) {
            const int cnt = min(Q, W), w0 = (int)((int64_t)e * Q % W);
            const int f = (item0 + e) * 8 + gid;
            const int64_t fg = (int64_t)f * p.r, fu = (int64_t)(p.F + f) * p.r;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int j = 0; j < cnt; ++j) {
                    const float4 s = part[((e * W + (w0 + j) % W) * NT + n) * 32 + lane];
                    v[0] = __fadd_rn(v[0], s.x);
                    v[1] = __fadd_rn(v[1], s.y);
                    v[2] = __fadd_rn(v[2], s.z);
                    v[3] = __fadd_rn(v[3], s.w);
                }
                const int tok = 8 * n + gid;
                const int64_t tu = (int64_t)tok * 2 * p.r;
                for (int j0 = 0; j0 < p.r; j0 += 32) {
                    const int j = j0 + 8 * tig;
                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                    const bool on = j < p.r, ont = on && tok < p.M;
                    const uint4 bg = on ? *reinterpret_cast<const uint4*>(p.B + fg + j) : z;
                    const uint4 bu = on ? *reinterpret_cast<const uint4*>(p.B + fu + j) : z;
                    const uint4 ug = ont ? *reinterpret_cast<const uint4*>(p.sU + tu + j) : z;
                    const uint4 uu = ont ? *reinterpret_cast<const uint4*>(p.sU + tu + p.r + j) : z;
                    mma_16816(v, bg.x, 0u, bg.y, 0u, ug.x, ug.y);
                    mma_16816(v, bg.z, 0u, bg.w, 0u, ug.z, ug.w);
                    mma_16816(v, 0u, bu.x, 0u, bu.y, uu.x, uu.y);
                    mma_16816(v, 0u, bu.z, 0u, bu.w, uu.z, uu.w);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int m = 8 * n + 2 * tig + h;
                    if (m >= p.M || !QLORA_CHECK(f < p.F)) continue;
                    const float g = v[h], u = v[2 + h];
                    const float y = (p.act == ACT_SILU ? act_value(ACT_SILU, g) : act_value(ACT_GELU_TANH, g)) * u;
                    p.H[(int64_t)m * p.F + f] = (uint16_t)(pack_bf16x2(y, 0.0f) & 0xFFFFu);
                    if (p.GU) {
                        p.GU[(int64_t)m * 2 * p.F + f] = (uint16_t)(pack_bf16x2(g, 0.0f) & 0xFFFFu);
                        p.GU[(int64_t)m * 2 * p.F + p.F + f] = (uint16_t)(pack_bf16x2(u, 0.0f) & 0xFFFFu);
                    }
                }
            }
        }
        if (item0 + S::CHUNK < i_end) __syncthreads();  // the partial sums are read
    }
}

}  // namespace qlora
