// kernels_moe.h -- a mixture-of-experts layer for a few tokens, two launches:
//
//   h[i]  = RN_t( act(x_t . Wg_e) * (x_t . Wu_e) )          k_moe_up
//   Y[t]  = RN_t( r[t] + sum_j w[t][j] * (h[i(t,j)] . Wd_e) ) k_moe_down
//
// for the pairs i of tokens t and experts e in the order of `rows` (grouped by
// expert, expert e's at offs[e] .. offs[e+1]-1; rows[i] = t * top_k + j).
//
// With a few rows per expert the layer is a stream of the active experts'
// packed weights: both kernels exist to keep that stream as deep as the
// memory's latency asks, and to read each weight once.
//   * k_moe_up: a workgroup owns one gate panel, the up panel of the same
//     outputs and one row tile of one expert; its waves split K.  It gathers
//     x by the pair's token, so no gathered copy is made.
//   * k_moe_down: a workgroup of 16 waves owns one 16-column panel of Y for
//     all tokens; its waves take the experts' row tiles in turn (and split K
//     when there are few), leave each pair's 16 outputs in LDS in fp32, and
//     the workgroup then adds them per token in slot order with the routing
//     weights: no atomics, no partial sums in memory, and a fixed order.
// h is rounded to the operand type because the second product's MFMA takes
// it so; the sum over a token's experts stays in fp32 until the one store.
#pragma once

#include <algorithm>

#include "epilogue.h"
#include "kernels_fp.h"

namespace qg {

constexpr int kMoeDownWaves = 16;

inline size_t moe_down_lds(long long pairs, long long E, int parts)
{
    const long long slots = std::min(pairs, (pairs + 15) / 16 + E);
    return (size_t)(parts * pairs * 64 + slots * 12 + pairs);
}

// acc[PN][RB] += X rows . panels over chunks [cb, ce), with up to D chunks of
// weights and activations in flight ahead of the one being multiplied.
template <int FMT, int DT, int RB, int PN, int D>
__device__ __forceinline__ void stream_chunks(const RunSrc<FMT> (&src)[PN], const uint16_t *const (&xrow)[RB], int cb,
                                              int ce, f32x4 (&acc)[PN][RB])
{
    RunRaw<FMT> raw[D][PN];
    u32x4 xf[D][RB][4];
    auto fetch = [&](int c, int d) {
#pragma unroll
        for (int pn = 0; pn < PN; pn++) src[pn].load(c, raw[d][pn]);
#pragma unroll
        for (int rb = 0; rb < RB; rb++)
#pragma unroll
            for (int i = 0; i < 4; i++) xf[d][rb][i] = *(const u32x4 *)(xrow[rb] + (long long)kChunk * c + 8 * i);
    };
#pragma unroll
    for (int d = 0; d < D; d++)
        if (cb + d < ce) fetch(cb + d, d);
    for (int c = cb; c < ce; c += D) {
#pragma unroll
        for (int d = 0; d < D; d++) {
            if (c + d >= ce) break;
            u32x4 wf[PN][4];
#pragma unroll
            for (int pn = 0; pn < PN; pn++) unpack_run<FMT, DT>(raw[d][pn], src[pn], c + d, wf[pn]);
            u32x4 xc[RB][4];
#pragma unroll
            for (int rb = 0; rb < RB; rb++)
#pragma unroll
                for (int i = 0; i < 4; i++) xc[rb][i] = xf[d][rb][i];
            if (c + d + D < ce) fetch(c + d + D, d);
#pragma unroll
            for (int rb = 0; rb < RB; rb++)
#pragma unroll
                for (int pn = 0; pn < PN; pn++)
#pragma unroll
                    for (int i = 0; i < 4; i++) acc[pn][rb] = mma<DT>(wf[pn][i], xc[rb][i], acc[pn][rb]);
        }
    }
}

// Pair index of sorted position i, clamped so that no contents of `rows`
// leave x, the weights or the LDS sums.
__device__ __forceinline__ int pair_at(const MoeArgs &m, int i)
{
    return (int)min((unsigned)m.rows[i], (unsigned)(m.g.M - 1));
}

// Grid: x = gate panels (inter/16), y = row-tile slots of 16*RB rows;
// 64*kw threads, kw waves splitting K.
template <int FMT, int DT, int RB, int D>
__global__ void __launch_bounds__(512) k_moe_up(MoeArgs m)
{
    extern __shared__ f32x4 red[];  // [kw][2*RB][64]
    const Args &a = m.g;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
    int e, lo, hi, t;
    // the same answer in every wave: the whole workgroup leaves together
    if (!find_group_tile(a, blockIdx.y, 16 * RB, lane, e, lo, hi, t)) return;
    Args b = a;
    b.W = a.W + (long long)e * a.wstride;
    const int m0 = lo + t * 16 * RB;
    RunSrc<FMT> src[2];
    src[0].init(b, blockIdx.x, g, col);
    src[1].init(b, (a.np >> 1) + blockIdx.x, g, col);
    const uint16_t *xrow[RB];
#pragma unroll
    for (int rb = 0; rb < RB; rb++) {
        const int tok = pair_at(m, min(m0 + 16 * rb + col, hi - 1)) / m.top_k;
        xrow[rb] = a.X + (long long)tok * a.K + 32 * g;
    }
    f32x4 acc[2][RB];
#pragma unroll
    for (int pn = 0; pn < 2; pn++)
#pragma unroll
        for (int rb = 0; rb < RB; rb++) acc[pn][rb] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int nch = a.K / kChunk;
    const int cb = (int)((long long)nch * w / a.kw), ce = (int)((long long)nch * (w + 1) / a.kw);
    stream_chunks<FMT, DT, RB, 2, D>(src, xrow, cb, ce, acc);
#pragma unroll
    for (int pn = 0; pn < 2; pn++)
#pragma unroll
        for (int rb = 0; rb < RB; rb++) red[(w * 2 * RB + pn * RB + rb) * 64 + lane] = acc[pn][rb];
    __syncthreads();
    for (int rb = w; rb < RB; rb += a.kw) {
        f32x4 vg = red[rb * 64 + lane], vu = red[(RB + rb) * 64 + lane];
        for (int ww = 1; ww < a.kw; ww++) {
            vg += red[(ww * 2 * RB + rb) * 64 + lane];
            vu += red[(ww * 2 * RB + RB + rb) * 64 + lane];
        }
        float v[4] = {vg[0], vg[1], vg[2], vg[3]};
        act_apply(a.act, v);
        const int i = m0 + 16 * rb + col;
        if (i < hi) {
            u32x2 o;
            o[0] = pack_out<DT>(v[0] * vu[0], v[1] * vu[1]);
            o[1] = pack_out<DT>(v[2] * vu[2], v[3] * vu[3]);
            *(u32x2 *)(m.H + (long long)i * m.inter + 16 * blockIdx.x + 4 * g) = o;
        }
    }
}

// Grid: x = panels of Y; 16 waves.  Dynamic LDS (moe_down_lds): parts * pairs
// * 16 floats, the row tiles (expert, first row, end of the expert's rows),
// and a flag per pair that some expert has computed it: a pair that no expert
// here serves adds nothing, whatever its weight holds.
template <int FMT, int DT, int D>
__global__ void __launch_bounds__(64 * kMoeDownWaves) k_moe_down(MoeArgs m)
{
    extern __shared__ float sums[];  // [parts][pairs][16]
    __shared__ int s_tiles;
    const Args &a = m.g;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, col = lane & 15, g = lane >> 4;
    const int P = a.M, span = P * 16;
    int *tile_e = (int *)(sums + (size_t)m.parts * span);
    const int slots = min(P, (P + 15) / 16 + a.E);  // a bound on the row tiles
    int *tile_lo = tile_e + slots, *tile_hi = tile_lo + slots;
    uint8_t *served = (uint8_t *)(tile_hi + slots);
    for (int i = tid; i < P; i += 64 * kMoeDownWaves) served[i] = 0;
    if (w == 0) {  // the row tiles, 64 experts at a time: a lane per expert, as find_group_tile clamps the offsets
        int qc = max(0, a.offs[0]), base = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            const int e = e0 + lane;
            const bool live = e < a.E;
            int q = live ? a.offs[e + 1] : INT_MIN;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int u = __shfl_up(q, d, 64);
                if (lane >= d) q = max(q, u);
            }
            q = max(q, qc);
            int qprev = __shfl_up(q, 1, 64);
            if (lane == 0) qprev = qc;
            const int lo = min(qprev, P), hi = min(q, P);
            const int nb = live ? (hi - lo + 15) / 16 : 0;
            int incl = nb;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int u = __shfl_up(incl, d, 64);
                if (lane >= d) incl += u;
            }
            for (int j = 0; j < nb; j++) {
                const int at = base + incl - nb + j;
                tile_e[at] = e;
                tile_lo[at] = lo + 16 * j;
                tile_hi[at] = hi;
            }
            base += __shfl(incl, 63, 64);
            qc = __shfl(q, 63, 64);
        }
        if (lane == 0) s_tiles = base;
    }
    __syncthreads();
    const int nch = a.K / kChunk, units = s_tiles * m.parts;
    for (int u = w; u < units; u += kMoeDownWaves) {
        const int tile = u / m.parts, part = u - tile * m.parts;
        const int lo = tile_lo[tile], hi = tile_hi[tile];
        Args b = a;
        b.W = a.W + (long long)tile_e[tile] * a.wstride;
        RunSrc<FMT> src[1];
        src[0].init(b, blockIdx.x, g, col);
        const int i = lo + col;
        const uint16_t *xrow[1] = {m.H + (long long)min(i, hi - 1) * a.K + 32 * g};
        const int pair = i < hi ? pair_at(m, i) : 0;
        f32x4 acc[1][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}};
        stream_chunks<FMT, DT, 1, 1, D>(src, xrow, (int)((long long)nch * part / m.parts),
                                        (int)((long long)nch * (part + 1) / m.parts), acc);
        if (i < hi) {
            *(f32x4 *)(sums + (size_t)part * span + pair * 16 + 4 * g) = acc[0][0];
            if (part == 0 && g == 0) served[pair] = 1;
        }
    }
    __syncthreads();
    for (int q = tid; q < m.T * 4; q += 64 * kMoeDownWaves) {
        const int t = q >> 2, n = 4 * (q & 3), n0 = 16 * blockIdx.x + n;
        if (n0 >= a.N) continue;
        float v[4] = {0.f, 0.f, 0.f, 0.f}, un[4];
        for (int j = 0; j < m.top_k; j++) {
            const int p = t * m.top_k + j;
            if (!served[p]) continue;
            f32x4 s = *(const f32x4 *)(sums + p * 16 + n);
            for (int k = 1; k < m.parts; k++) s += *(const f32x4 *)(sums + (size_t)k * span + p * 16 + n);
            const float wt = m.wts[p];
#pragma unroll
            for (int c = 0; c < 4; c++) v[c] = __builtin_fmaf(wt, s[c], v[c]);
        }
        Args y = a;  // the store sees T rows
        y.M = m.T;
        finish_quad<DT, EP_LIN>(y, t, n0, v, un, quad_in<EP_LIN>(y, t, n0));
    }
}

}  // namespace qg
