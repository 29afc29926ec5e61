// epilogue.h -- the linear layer's epilogue: bias, activation, gating and
// residual on the fp32 accumulators, one rounding into Y, row-major or
// fragment-major.
//
//   Y = RN_t( act(acc + b) + r )                     EP_LIN
//   Y = RN_t( act(g + bg) * (u + bu) + r )           EP_GATED
//
// It runs once per output tile, on accumulators that are in registers
// anyway: what it saves is a launch and a full read and write of [M][N] per
// fused step.  Every step is binary32; the store is the only rounding to 16
// bits.
#pragma once

#include "common.h"

namespace qg {

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// v * sigmoid(z), the exponent x = -z log2 e given: SiLU with z = v; the tanh
// form of GELU with z = 2 sqrt(2/pi) (v + 0.044715 v^3), since (1 + tanh y) / 2
// = sigmoid(2y) -- no cancellation on the negative side.  Relative error 2^-21
// (v_exp_f32 and v_rcp_f32 are good to 1 ulp) and, where z is negative, what the
// roundings on the way to x make of it, up to 4 |x| 2^-24: 2^-19 for SiLU at v =
// -30, 2^-17 for GELU at v = -9, far below a rounding to 16 bits.  A result
// below |v| 2^-125, whose reciprocal has no normal binary32 value, may be 0.
// The two transcendentals are most of an activation's cost: about 6 us of the
// 189 that W4A16 2048x4096 -> 12288 takes with bias and GELU.
__device__ __forceinline__ float times_sigmoid(float v, float x) { return v * rcp_fast(1.0f + exp2_fast(x)); }

__device__ __forceinline__ float act_silu(float v) { return times_sigmoid(v, -1.4426950408889634f * v); }

__device__ __forceinline__ float act_gelu_tanh(float v)
{
    constexpr float a = -2.3022082f, b = -0.10294324f;  // -log2 e times 2 sqrt(2/pi) and that times 0.044715
    return times_sigmoid(v, v * __builtin_fmaf(b * v, v, a));
}

// v * Phi(v) = v erfc(-v/sqrt 2) / 2.  erfc(x) = exp(-x^2) erfcx(x) for x >=
// 0, and erfcx(x) = t P(t) with t = 1/(1 + 0.38 x), P of degree 8: a minimax
// fit of this file's own (relative error 2.5e-8 over x >= 0, 4e-7 with
// binary32 coefficients and arithmetic), so the tail does not cancel as 1 + erf
// would.  The roundings of the exponent x = v^2 log2(e) / 2 add up to 4 x 2^-24
// there: 2^-17 at v = -8, 2^-16 at -12.6; from about -13.2 on results are 0.
__device__ __forceinline__ float act_gelu(float v)
{
    constexpr float kLog2e = 1.4426950408889634f;
    const float x = __builtin_fabsf(v) * 0.70710678118654752f;
    const float t = rcp_fast(__builtin_fmaf(0.38f, x, 1.0f));
    float p = 0.05842172f;
    p = __builtin_fmaf(p, t, -0.25986003f);
    p = __builtin_fmaf(p, t, 0.35933812f);
    p = __builtin_fmaf(p, t, -0.15683829f);
    p = __builtin_fmaf(p, t, 0.2272183f);
    p = __builtin_fmaf(p, t, 0.13968066f);
    p = __builtin_fmaf(p, t, 0.20368521f);
    p = __builtin_fmaf(p, t, 0.21394446f);
    p = __builtin_fmaf(p, t, 0.21440983f);
    const float e = p * t * exp2_fast(-kLog2e * x * x);  // erfc(|v|/sqrt 2)
    return 0.5f * v * (v < 0.0f ? e : 2.0f - e);
}

// act on N consecutive values; `act` is the same for the whole launch, so the
// branch is uniform.
template <int N>
__device__ __forceinline__ void act_apply(int act, float (&v)[N])
{
    if (act == QGEMM_ACT_NONE) return;
    if (act == QGEMM_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; j++) v[j] = v[j] < 0.0f ? 0.0f : v[j];
    } else if (act == QGEMM_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; j++) v[j] = act_gelu(v[j]);
    } else if (act == QGEMM_ACT_GELU_TANH) {
#pragma unroll
        for (int j = 0; j < N; j++) v[j] = act_gelu_tanh(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) v[j] = act_silu(v[j]);
    }
}

template <int DT>
__device__ __forceinline__ float widen16(uint32_t bits16)
{
    if constexpr (DT == DT_F16) return f16_to_f32(bits16 & 0xFFFFu);
    else return __builtin_bit_cast(float, bits16 << 16);
}

// Four consecutive 16-bit elements at p (those below `left` of them), one
// 8-byte load when the rows are made of whole quads.
__device__ __forceinline__ u32x2 load_quad(const uint16_t *p, int left, bool quads)
{
    if (quads) return *(const u32x2 *)p;
    u32x2 r = {0u, 0u};
    r[0] = p[0];
    if (left > 1) r[0] |= (uint32_t)p[1] << 16;
    if (left > 2) r[1] = p[2];
    if (left > 3) r[1] |= (uint32_t)p[3] << 16;
    return r;
}

template <int DT>
__device__ __forceinline__ void add_quad(float (&v)[4], u32x2 q)
{
    v[0] += widen16<DT>(q[0]);
    v[1] += widen16<DT>(q[0] >> 16);
    v[2] += widen16<DT>(q[1]);
    v[3] += widen16<DT>(q[1] >> 16);
}

// Output quad (m, n0 .. n0+3) of Y: element offset in the layout of Y.
__device__ __forceinline__ long long y_offset(const Args &a, int m, int n0)
{
    if (a.y_frag)
        return (((long long)(m >> 5) * (a.N >> 7) + (n0 >> 7)) * 8 + ((n0 >> 4) & 7)) * 512 +
               (((n0 >> 3) & 1) * 32 + (m & 31)) * 8 + (n0 & 7);
    return (long long)m * a.N + n0;
}

// Rows past M that the fragment-major layout holds as zeros.
__device__ __forceinline__ int y_rows(const Args &a) { return a.y_frag ? (a.M + 31) & ~31 : a.M; }

template <int DT>
__device__ __forceinline__ void store_quad(const Args &a, int m, int n0, const float (&v)[4])
{
    uint16_t *y = a.Y + y_offset(a, m, n0);
    const uint32_t lo = pack_out<DT>(v[0], v[1]), hi = pack_out<DT>(v[2], v[3]);
    if ((a.N & 3) == 0) {
        *(u32x2 *)y = u32x2{lo, hi};
    } else {
        const uint16_t e[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
        for (int j = 0; j < 4 && n0 + j < a.N; j++) y[j] = e[j];
    }
}

// What the epilogue reads: the bias of an output quad's columns, and the
// residual of the quad.  Both are fetched ahead of the stores (Y may be the
// residual itself, so a load cannot move above a store by itself), the bias
// once for all of a wave's rows.
struct BiasQuad {
    u32x2 b, b2;
};

template <int EPI>
__device__ __forceinline__ BiasQuad bias_quad(const Args &a, int n0)
{
    BiasQuad q{{0u, 0u}, {0u, 0u}};
    if (!a.bias || n0 >= a.N) return q;
    const bool quads = (a.N & 3) == 0;
    q.b = load_quad(a.bias + n0, a.N - n0, quads);
    if constexpr (EPI == EP_GATED) q.b2 = load_quad(a.bias + a.N + n0, a.N - n0, quads);
    return q;
}

__device__ __forceinline__ u32x2 res_quad(const Args &a, int m, int n0)
{
    if (!a.res || n0 >= a.N || m >= a.M) return u32x2{0u, 0u};
    return load_quad(a.res + (long long)m * a.N + n0, a.N - n0, (a.N & 3) == 0);
}

// One output quad: v holds acc (EP_LIN) or the gate's acc with u the up
// projection's (EP_GATED).
template <int DT, int EPI>
__device__ __forceinline__ void finish_quad(const Args &a, int m, int n0, float (&v)[4], float (&u)[4], const BiasQuad &q,
                                            u32x2 res)
{
    if (n0 >= a.N || m >= y_rows(a)) return;
    if (m < a.M) {
        if (a.bias) add_quad<DT>(v, q.b);
        act_apply(a.act, v);
        if constexpr (EPI == EP_GATED) {
            if (a.bias) add_quad<DT>(u, q.b2);
#pragma unroll
            for (int j = 0; j < 4; j++) v[j] *= u[j];
        }
        if (a.res) add_quad<DT>(v, res);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = 0.0f;
    }
    store_quad<DT>(a, m, n0, v);
}

// Output column of accumulator columns n_base.. of a tile: tile panels pair up
// under EP_GATED.
template <int EPI>
__device__ __forceinline__ int out_col(int n_base)
{
    return EPI == EP_GATED ? n_base >> 1 : n_base;
}

// A 16x16 accumulator (store_block's layout) of tile panel n_base/16; under
// EP_GATED `v` is the gate panel's and `u` the next (up) panel's, n_base a
// multiple of 32.
template <int DT, int EPI>
__device__ __forceinline__ void store_block_ep(const Args &a, f32x4 v, f32x4 u, int m_base, int n_base, int lane)
{
    const int m = m_base + (lane & 15), n0 = out_col<EPI>(n_base) + 4 * (lane >> 4);
    const BiasQuad q = bias_quad<EPI>(a, n0);
    const u32x2 res = res_quad(a, m, n0);
    float g[4] = {v[0], v[1], v[2], v[3]}, w[4] = {u[0], u[1], u[2], u[3]};
    finish_quad<DT, EPI>(a, m, n0, g, w, q, res);
}

// A wave's PB x RB accumulators of 16x16, tile panels from column n_base,
// rows m_base + 16 rb.
template <int DT, int EPI, int PB, int RB>
__device__ __forceinline__ void store_wave16_ep(const Args &a, const f32x4 (&acc)[PB][RB], int m_base, int n_base,
                                                int lane)
{
    constexpr int PS = EPI == EP_GATED ? 2 : 1, O = PB / PS;  // output panels
    const int n = out_col<EPI>(n_base) + 4 * (lane >> 4);
    BiasQuad bias[O];
#pragma unroll
    for (int o = 0; o < O; o++) bias[o] = bias_quad<EPI>(a, n + 16 * o);
#pragma unroll
    for (int rb = 0; rb < RB; rb++) {
        const int m = m_base + 16 * rb + (lane & 15);
        u32x2 res[O];
#pragma unroll
        for (int o = 0; o < O; o++) res[o] = res_quad(a, m, n + 16 * o);
#pragma unroll
        for (int o = 0; o < O; o++) {
            const f32x4 g = acc[PS * o][rb], w = acc[PS * o + PS - 1][rb];
            float v[4] = {g[0], g[1], g[2], g[3]}, u[4] = {w[0], w[1], w[2], w[3]};
            finish_quad<DT, EPI>(a, m, n + 16 * o, v, u, bias[o], res[o]);
        }
    }
}

// A wave's CB x RB accumulators of 32x32 (store_block32's layout), rows m_base
// + 32 rb, tile columns n_base + 32 cb.  Under EP_GATED the first 16 columns
// of a block are a gate panel, the last 16 the up panel of the same outputs.
template <int DT, int EPI, int CB, int RB>
__device__ __forceinline__ void store_wave32_ep(const Args &a, const f32x16 (&acc)[CB][RB], int m_base, int n_base,
                                                int lane)
{
    constexpr int Q = EPI == EP_GATED ? 2 : 4;  // output quads per block and lane
    auto col = [&](int cb, int q) { return out_col<EPI>(n_base + 32 * cb) + 8 * q + 4 * (lane >> 5); };
    BiasQuad bias[CB][Q];
#pragma unroll
    for (int cb = 0; cb < CB; cb++)
#pragma unroll
        for (int q = 0; q < Q; q++) bias[cb][q] = bias_quad<EPI>(a, col(cb, q));
#pragma unroll
    for (int rb = 0; rb < RB; rb++) {
        const int m = m_base + 32 * rb + (lane & 31);
        u32x2 res[CB][Q];
#pragma unroll
        for (int cb = 0; cb < CB; cb++)
#pragma unroll
            for (int q = 0; q < Q; q++) res[cb][q] = res_quad(a, m, col(cb, q));
#pragma unroll
        for (int cb = 0; cb < CB; cb++)
#pragma unroll
            for (int q = 0; q < Q; q++) {
                float v[4], u[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    v[j] = acc[cb][rb][4 * q + j];
                    u[j] = EPI == EP_GATED ? acc[cb][rb][4 * (q + 4 - Q) + j] : 0.0f;
                }
                finish_quad<DT, EPI>(a, m, col(cb, q), v, u, bias[cb][q], res[cb][q]);
            }
    }
}

}  // namespace qg
