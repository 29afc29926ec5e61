// kernels_moe.h -- a mixture-of-experts layer for a few tokens, two launches:
//
//   h[i]  = act(x_t . Wg_e) * (x_t . Wu_e)                    k_moe_up
//   Y[t]  = RN_t( r[t] + sum_j w[t][j] * (h[i(t,j)] . Wd_e) ) k_moe_down
//
// for the pairs i of tokens t and experts e in the order of `rows` (grouped by
// expert, expert e's at offs[e] .. offs[e+1]-1; rows[i] = t * top_k + j).
//
// With a few rows per expert the layer is a stream of the active experts'
// packed weights: both kernels exist to keep that stream as deep as the
// memory's latency asks, and to read each weight once.
//   * k_moe_up: a wave owns one gate panel, the up panel of the same outputs,
//     one row tile of one expert and a share of K; the kw waves of a share
//     add up through LDS.  It gathers x by the pair's token, so no gathered
//     copy is made.
//   * k_moe_down: a workgroup owns one or two 16-column panels of Y for all
//     tokens and every split-th row tile of the experts; its waves take those
//     in turn (in parts of K when they are few), leave each pair's outputs in
//     LDS in fp32, and the workgroup adds them per token in slot order with
//     the routing weights.  With split > 1 the panels' workgroups leave those
//     sums in memory, and the last of them to arrive adds them in order: no
//     floating-point atomics, and a result that does not depend on timing.
// h goes to memory as its rounding to the operand type and what that rounding
// left, and the second product takes both, so h has twice the type's bits and
// the layer's error is that of Y's one rounding: with a few rows per expert in
// the MFMA columns that tiles of eight rows leave idle, with full tiles of
// sixteen as a second MFMA on the same unpacked weights.  (With a few rows per
// expert on average a popular one's weights are unpacked once per eight of its
// rows; against tiles of sixteen with the rounding alone, the whole layer: 64
// tokens, 8 of 128 experts, 97.0 against 96.4 us, every token with one expert in
// common 98.7 against 96.0; 32 tokens on one of eight experts 16.4 against 15.0.)
// The sum over a token's experts stays in fp32 until the one store.
#pragma once

#include <algorithm>

#include "epilogue.h"
#include "kernels_fp.h"

namespace qg {

inline size_t moe_down_lds(long long pairs, long long E, int parts, int pn, int rows)
{
    const long long slots = moe_tiles(pairs, E, rows);
    return (size_t)(parts * pairs * 64 * pn + slots * 12 + pairs * 5);
}

// Inclusive scans over the wave in DPP steps: row shifts inside rows of 16
// lanes, then the row broadcasts into the rows that lack them.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_from(int x, int identity)
{
    return __builtin_amdgcn_update_dpp(identity, x, CTRL, ROWS, 0xF, false);
}

__device__ __forceinline__ int wave_scan_add(int x)
{
    x += dpp_from<0x111, 0xF>(x, 0);  // row_shr:1
    x += dpp_from<0x112, 0xF>(x, 0);  // row_shr:2
    x += dpp_from<0x114, 0xF>(x, 0);  // row_shr:4
    x += dpp_from<0x118, 0xF>(x, 0);  // row_shr:8
    x += dpp_from<0x142, 0xA>(x, 0);  // row_bcast:15 into rows 1 and 3
    x += dpp_from<0x143, 0xC>(x, 0);  // row_bcast:31 into rows 2 and 3
    return x;
}

__device__ __forceinline__ int wave_scan_max(int x)
{
    x = max(x, dpp_from<0x111, 0xF>(x, INT_MIN));
    x = max(x, dpp_from<0x112, 0xF>(x, INT_MIN));
    x = max(x, dpp_from<0x114, 0xF>(x, INT_MIN));
    x = max(x, dpp_from<0x118, 0xF>(x, INT_MIN));
    x = max(x, dpp_from<0x142, 0xA>(x, INT_MIN));
    x = max(x, dpp_from<0x143, 0xC>(x, INT_MIN));
    return x;
}

// The experts' row tiles of ROWS rows, in expert order, 64 experts at a
// time, a lane per expert: visit(lane's expert, its first row, its end, its
// tile count, the tiles before it) until it returns true.  Offsets are
// clamped into [0, P] and made non-decreasing as the grouped GEMM does, so
// any contents stay inside the buffers.  Returns the tiles visited over.
template <int ROWS, class F>
__device__ __forceinline__ int visit_tiles(const Args &a, int lane, F visit)
{
    constexpr int G = 4;  // groups of 64 experts whose offsets are loaded together
    int qc = max(0, a.offs[0]), base = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64 * G) {
        int q[G];
#pragma unroll
        for (int i = 0; i < G; i++) {
            const int e = e0 + 64 * i + lane;
            q[i] = e < a.E ? a.offs[e + 1] : INT_MIN;
        }
#pragma unroll
        for (int i = 0; i < G; i++) {
            const int e = e0 + 64 * i + lane;
            if (e0 + 64 * i >= a.E) break;
            const int qi = max(wave_scan_max(q[i]), qc);                                 // max(0, offs[0..e+1])
            const int qp = __builtin_amdgcn_update_dpp(qc, qi, 0x138, 0xF, 0xF, false);  // wave_shr:1, lane 0 keeps qc
            const int lo = min(qp, a.M), hi = min(qi, a.M);
            const int nb = e < a.E ? (hi - lo + ROWS - 1) / ROWS : 0;
            const int incl = wave_scan_add(nb);
            if (visit(e, lo, hi, nb, base + incl - nb)) return base;
            base += __builtin_amdgcn_readlane(incl, 63);
            qc = __builtin_amdgcn_readlane(qi, 63);
        }
    }
    return base;
}

// Row tile j of 16 rows: expert e, rows [lo, hi) of the expert, tile t of it;
// false when j is past the last tile.  The same answer in every lane.
__device__ __forceinline__ bool find_moe_tile(const Args &a, int j, int lane, int &e_out, int &lo_out,
                                              int &hi_out, int &t_out)
{
    bool found = false;
    visit_tiles<16>(a, lane, [&](int e, int lo, int hi, int nb, int before) {
        const unsigned long long hit = __ballot(j >= before && j < before + nb);
        if (hit == 0ull) return false;
        const int l = __builtin_amdgcn_readfirstlane(__ffsll((long long)hit) - 1);
        e_out = __builtin_amdgcn_readlane(e, l);
        lo_out = __builtin_amdgcn_readlane(lo, l);
        hi_out = __builtin_amdgcn_readlane(hi, l);
        t_out = j - __builtin_amdgcn_readlane(before, l);
        found = true;
        return true;
    });
    return found;
}

// Four floats written to, or read from, the device's point of coherence (past
// the L2 of the XCD): how workgroups on different XCDs hand over sums inside
// one kernel.  Agent-scope atomics do that by themselves; a release fence
// would write back the XCD's whole L2, once per wave (measured: 105 instead
// of 10 us for the down product of one token).
__device__ __forceinline__ void store_agent(float *p, const float (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const unsigned long long x = (unsigned long long)__builtin_bit_cast(uint32_t, v[2 * i]) |
                                     (unsigned long long)__builtin_bit_cast(uint32_t, v[2 * i + 1]) << 32;
        __hip_atomic_store((unsigned long long *)p + i, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

__device__ __forceinline__ void load_agent(const float *p, float (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const unsigned long long x =
            __hip_atomic_load((const unsigned long long *)p + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        v[2 * i] = __builtin_bit_cast(float, (uint32_t)x);
        v[2 * i + 1] = __builtin_bit_cast(float, (uint32_t)(x >> 32));
    }
}

// Pair index of sorted position i, clamped so that no contents of `rows`
// leave x, the weights or the LDS sums.
__device__ __forceinline__ int pair_at(const MoeArgs &m, int i)
{
    return (int)min((unsigned)m.rows[i], (unsigned)(m.g.M - 1));
}

// h goes to memory as two numbers of the operand type: its rounding, and what
// the rounding left, scaled up so that fp16's subnormals do not cut it short
// (fp16's remainder is at most 2^-11 of h, bf16's 2^-8: scaled it is no larger
// than h).  Where h is beyond the type's range the rounding is infinite and
// nothing is left.
template <int DT> constexpr float kLowScale = DT == DT_F16 ? 2048.0f : 256.0f;

template <int DT>
__device__ __forceinline__ float low_part(float v, uint32_t bits16)
{
    const float hi = widen16<DT>(bits16);
    return fabsf(hi) < __builtin_inff() ? (v - hi) * kLowScale<DT> : 0.0f;
}

// A sum over RN(h) with the sum over what the rounding left, which is small
// beside it unless a weight or a product is infinite: there the two meet the
// same infinity with signs of their own (or 0), and the definition's answer is
// the rounding's.
template <int DT>
__device__ __forceinline__ float join_parts(float hi, float low)
{
    return fabsf(low) < __builtin_inff() ? __builtin_fmaf(low, 1.0f / kLowScale<DT>, hi) : hi;
}

// Element k (a multiple of 4) of sorted row i in a plane of the hidden matrix.
// Plain, for at most four pairs per expert: row-major.  BLOCKED, above: blocks
// of 16 rows, a chunk of 128 after the other, and inside a chunk the rows'
// 16-byte pieces (k = 32 g + 8 i .. + 8) ordered by i, g and row, so that the 16
// lanes of a k_moe_down load that hold one g read 256 consecutive bytes, not 16
// pieces of as many rows.  The down product of 256 tokens, 4 of 8 experts, 1024
// -> 1024, h rounded only: 22.4 against 28.9 us; with a few rows in a tile the
// blocks touch twice the cache lines and leave MFMA columns idle, and 64 tokens,
// 8 of 128 experts, take 105 against 97 for the whole layer, one token 18.9
// against 17.2.
template <bool BLOCKED>
__device__ __forceinline__ long long hidden_at(int inter, int i, int k)
{
    if (!BLOCKED) return (long long)i * inter + k;
    return ((long long)(i >> 4) * (inter >> 7) + (k >> 7)) * 2048 + ((k >> 3 & 3) * 4 + (k >> 5 & 3)) * 128 +
           (i & 15) * 8 + (k & 7);
}

// Raw bytes and activations of one chunk pair: PN panels, one row per column
// lane.  The k-quants' block header serves both chunks, so a pair costs one
// header load; second: the pair's second chunk exists (always for the
// k-quants; W4A16's K may end on a first one).
template <int FMT, int PN>
struct Pair {
    RunRaw<FMT> raw[PN][2];
    u32x4 x[2][4];

    __device__ __forceinline__ void load_w(const RunSrc<FMT> (&src)[PN], int p, int nch)
    {
        const bool second = FMT != FMT_W4 || 2 * p + 1 < nch;
#pragma unroll
        for (int pn = 0; pn < PN; pn++) load_pair<FMT>(src[pn], 2 * p, second, raw[pn]);
    }

    __device__ __forceinline__ void load_x(const uint16_t *xrow, int p, int nch)
    {
        const bool second = FMT != FMT_W4 || 2 * p + 1 < nch;
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                x[h][i] = *(const u32x4 *)(xrow + (long long)kChunk * (second ? 2 * p + h : 2 * p) + 8 * i);
    }
};

// acc[n] += the pair's product with the n-th of NX activation operands, one run
// unpacked at a time.  acts(h, x) gives the activations of chunk h; refill()
// issues the loads that take the pair's place.  Unpacking the whole pair first,
// so that those loads go out before the MFMAs, or holding two pairs, takes
// registers from the waves that hide the latency: 64 tokens of 8 of 128
// experts, Q4_K 2048 -> 768 pairs, weights rotating, 51.4 us so, 56 with two
// single chunks in flight, 64-66 with either of those.
template <int FMT, int DT, int PN, int NX, class X, class F>
__device__ __forceinline__ void multiply_pair(const Pair<FMT, PN> &q, const RunSrc<FMT> (&src)[PN], int p, int nch,
                                              f32x4 (&acc)[NX][PN], X acts, F refill)
{
#pragma unroll
    for (int h = 0; h < 2; h++) {
        if (FMT == FMT_W4 && h == 1 && 2 * p + 1 >= nch) continue;
        u32x4 x[NX][4];
        acts(h, x);
#pragma unroll
        for (int pn = 0; pn < PN; pn++) {
            u32x4 wf[4];
            unpack_run<FMT, DT>(q.raw[pn][h], src[pn], 2 * p + h, wf);
#pragma unroll
            for (int n = 0; n < NX; n++)
#pragma unroll
                for (int i = 0; i < 4; i++) acc[n][pn] = mma<DT>(wf[i], x[n][i], acc[n][pn]);
        }
    }
    refill();
    __builtin_amdgcn_sched_barrier(0);  // the loads go out here, not where they are next needed
}

// Grid: x = groups of kMoeUpWaves/kw gate panels (inter/16 in all), y =
// row-tile slots of 16 rows; kw waves split the K of one panel.  16-row tiles
// serve many rows per expert too: a tile's second reading of the weights comes
// from L2, and 32- and 64-row tiles, which unpack less, leave the chip emptier
// (64 tokens, both of 2 to 8 experts: 13.5-18.1 us against 13.0-17.0 and
// 17.5-24; 128 tokens, 8 of 16: 37.4 against 35.9 and 35.8, before the LDS
// tiles below, 36.0 with them).
//
// BLOCKED, where full tiles are likely (hidden_at): a load reads 256
// consecutive bytes of four rows of x, and a tile of the wave's own in LDS turns
// them into fragments, as the linear layer's row-major kernels do (128 tokens,
// 8 of 16 experts: 36.0 against 42.3 us; 128, 4 of 32, 4096 -> 1024: 66.4
// against 79.1).  With a few rows most lanes of a plain load read the same row, which
// costs little, and the LDS round trip does not pay (64 tokens, 8 of 128: 68.6
// against 65.2 us; one token 9.3 against 7.8).
template <int FMT, int DT, bool BLOCKED>
__global__ void __launch_bounds__(64 * kMoeUpWaves) k_moe_up(MoeArgs m)
{
    constexpr int kTile = BLOCKED ? 32 * kXStride : 2 * 64 * 16;  // a wave's 16 rows of two chunks, later its sums
    __shared__ __attribute__((aligned(16))) uint8_t lds[kMoeUpWaves * kTile];
    f32x4(*red)[2][64] = (f32x4(*)[2][64])lds;
    const Args &a = m.g;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    if (blockIdx.x == 0 && blockIdx.y == 0)  // the counters of k_moe_down, which runs after this launch
        for (int i = threadIdx.x; i < m.strips; i += 64 * kMoeUpWaves) m.arrived[i] = 0;
    int e, lo, hi, t;
    // the same answer in every wave: the whole workgroup leaves together
    if (!find_moe_tile(a, blockIdx.y, lane, e, lo, hi, t)) return;
    const int share = w % a.kw, pairs = a.np >> 1;
    const int own = (int)blockIdx.x * (kMoeUpWaves / a.kw) + w / a.kw;
    const int p = min(own, pairs - 1);  // past the end: computed and discarded
    Args b = a;
    b.W = a.W + (long long)e * a.wstride;
    RunSrc<FMT> src[2];
    src[0].init(b, p, g, col);
    src[1].init(b, pairs + p, g, col);
    const int i = lo + 16 * t + col;
    f32x4 acc[1][2] = {};
    const int nch = a.K / kChunk, np2 = (nch + 1) / 2;
    const int pe = np2 * (share + 1) / a.kw;
    int q = np2 * share / a.kw;
    if (q < pe) {
        Pair<FMT, 2> pr;
        pr.load_w(src, q, nch);
        __builtin_amdgcn_sched_barrier(0);  // the weights' loads go out before the token is known
        auto token_row = [&](int r) {  // row r of the tile, the last one for those past the expert's end
            return a.X + (long long)(pair_at(m, min(lo + 16 * t + r, hi - 1)) / m.top_k) * a.K;
        };
        const uint16_t *xrow[4];
#pragma unroll
        for (int j = 0; j < (BLOCKED ? 4 : 1); j++)
            xrow[j] = BLOCKED ? token_row(g + 4 * j) + 8 * col : token_row(col) + 32 * g;
        uint8_t *put = lds + w * kTile + g * kXStride + 16 * col;
        const uint8_t *get = lds + w * kTile + col * kXStride + 64 * g;
        auto load_x = [&](int q) {
            if constexpr (!BLOCKED) return pr.load_x(xrow[0], q, nch);
            const bool second = FMT != FMT_W4 || 2 * q + 1 < nch;
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    pr.x[h][j] = *(const u32x4 *)(xrow[j] + (long long)kChunk * (second ? 2 * q + h : 2 * q));
        };
        load_x(q);
        auto acts = [&](int h, u32x4(&x)[1][4]) {
            if constexpr (BLOCKED) {
#pragma unroll
                for (int j = 0; j < 4; j++) *(u32x4 *)(put + (16 * h + 4 * j) * kXStride) = pr.x[h][j];
                __builtin_amdgcn_wave_barrier();
            }
#pragma unroll
            for (int k = 0; k < 4; k++) x[0][k] = BLOCKED ? *(const u32x4 *)(get + 16 * h * kXStride + 16 * k) : pr.x[h][k];
            if constexpr (BLOCKED) __builtin_amdgcn_wave_barrier();
        };
        for (; q + 1 < pe; q++)
            multiply_pair<FMT, DT>(pr, src, q, nch, acc, acts, [&] {
                pr.load_w(src, q + 1, nch);
                load_x(q + 1);
            });
        multiply_pair<FMT, DT>(pr, src, q, nch, acc, acts, [] {});
    }
    if (a.kw > 1) {
        if (BLOCKED) __syncthreads();  // the sums take the tiles' place
        red[w][0][lane] = acc[0][0];
        red[w][1][lane] = acc[0][1];
        __syncthreads();
        if (share != 0) return;
        for (int ww = 1; ww < a.kw; ww++) {
            acc[0][0] += red[w + ww][0][lane];
            acc[0][1] += red[w + ww][1][lane];
        }
    }
    if (own >= pairs || i >= hi) return;
    const f32x4 gate = acc[0][0], up = acc[0][1];
    float v[4] = {gate[0], gate[1], gate[2], gate[3]};
    act_apply(a.act, v);
#pragma unroll
    for (int c = 0; c < 4; c++) v[c] *= up[c];
    const int k = 16 * p + 4 * g;
    uint16_t *h = m.H + hidden_at<BLOCKED>(m.inter, i, k);
    const u32x2 o = {pack_out<DT>(v[0], v[1]), pack_out<DT>(v[2], v[3])};
    *(u32x2 *)h = o;
#pragma unroll
    for (int c = 0; c < 4; c++) v[c] = low_part<DT>(v[c], o[c >> 1] >> (16 * (c & 1)));
    *(u32x2 *)(h + m.plane) = u32x2{pack_out<DT>(v[0], v[1]), pack_out<DT>(v[2], v[3])};
}

// Grid: x = strips of Y (PN panels each) times split.  Dynamic LDS
// (moe_down_lds): parts * pairs * 16 PN floats, the row tiles (expert, first
// row, end), the sorted pairs, and a flag per pair that
// some expert has computed it: a pair that no expert here serves adds nothing,
// whatever its weight holds.
//
// A wave's work is one sequence of chunk pairs over its units (row tile, part
// of K), the next pair's loads in flight across the units' borders: `front`
// walks the sequence where the loads are, `back` where the MFMAs are.
template <int FMT, int DT, int PN, bool BLOCKED>
__global__ void __launch_bounds__(64 * kMoeDownWaves, 4) k_moe_down(MoeArgs m)
{
    constexpr int NW = kMoeDownWaves, CW = 16 * PN, QW = 4 * PN;  // columns and quads of a strip's row
    constexpr int ROWS = moe_down_rows(BLOCKED);
    extern __shared__ float sums[];  // [parts][pairs][CW]
    __shared__ int s_tiles, s_last;
    const Args &a = m.g;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int P = a.M, span = P * CW;
    const int strip = blockIdx.x / m.split, slice = blockIdx.x - strip * m.split;
    int *tile_e = (int *)(sums + (size_t)m.parts * span);
    const int slots = (int)moe_tiles(P, a.E, ROWS);
    int *tile_lo = tile_e + slots, *tile_hi = tile_lo + slots;
    int *pair_of = tile_hi + slots;
    uint8_t *served = (uint8_t *)(pair_of + P);
    for (int i = tid; i < P; i += 64 * NW) {
        pair_of[i] = pair_at(m, i);
        served[i] = 0;
    }
    if (w == 0) {
        const int n = visit_tiles<ROWS>(a, lane, [&](int e, int lo, int hi, int nb, int before) {
            for (int j = 0; j < nb; j++) {
                tile_e[before + j] = e;
                tile_lo[before + j] = lo + ROWS * j;
                tile_hi[before + j] = min(lo + ROWS * (j + 1), hi);
            }
            return false;
        });
        if (lane == 0) s_tiles = n;
    }
    __syncthreads();
    const int nch = a.K / kChunk, np2 = (nch + 1) / 2, tiles = __builtin_amdgcn_readfirstlane(s_tiles);
    // this workgroup's units: tiles slice, slice + split, ..., each in `parts` parts of K
    const int units = (tiles > slice ? (tiles - slice + m.split - 1) / m.split : 0) * m.parts;

    struct Cursor {
        int u, c, ce;  // unit, next chunk pair, end of the unit's pairs
        int lo, hi;
    };
    auto open = [&](Cursor &q) {  // the unit's rows and pairs
        const int tile = slice + m.split * (q.u / m.parts), part = q.u % m.parts;
        q.lo = __builtin_amdgcn_readfirstlane(tile_lo[tile]);
        q.hi = __builtin_amdgcn_readfirstlane(tile_hi[tile]);
        q.c = np2 * part / m.parts;
        q.ce = np2 * (part + 1) / m.parts;
        return __builtin_amdgcn_readfirstlane(tile_e[tile]);
    };
    RunSrc<FMT> src[PN];   // at the front cursor's expert
    const uint16_t *xrow;  // at the front cursor's rows; BLOCKED: at the back cursor's
    auto rows_at = [&](const Cursor &q) {
        const int i = min(q.lo + (col & (ROWS - 1)), q.hi - 1);
        // plain: columns 8..15 take the low parts of the rows in 0..7
        xrow = m.H + (!BLOCKED && col > 7 ? m.plane : 0) + hidden_at<BLOCKED>(a.K, i, 32 * g);
    };
    auto aim = [&](Cursor &q) {
        const int e = open(q);
        Args b = a;
        b.W = a.W + (long long)e * a.wstride;
#pragma unroll
        for (int pn = 0; pn < PN; pn++) src[pn].init(b, PN * strip + pn, g, col);
        if (!BLOCKED) rows_at(q);
    };
    if (w < units) {
        Pair<FMT, PN> pr;
        Cursor front{w, 0, 0, 0, 0}, back{w, 0, 0, 0, 0};
        aim(front);
        open(back);
        if (BLOCKED) rows_at(back);
        int total = 0;  // pairs of this wave's sequence
        for (int u = w; u < units; u += NW) total += np2 * (u % m.parts + 1) / m.parts - np2 * (u % m.parts) / m.parts;
        auto fetch = [&] {
            pr.load_w(src, front.c, nch);
            if (!BLOCKED) pr.load_x(xrow, front.c, nch);
            if (++front.c == front.ce) {
                front.u += NW;
                if (front.u < units) aim(front);
            }
        };
        // BLOCKED: both parts of full rows are loaded when their chunk's turn
        // comes, under the unpack; ahead of it they would not fit the registers
        // (128 tokens, 8 of 16 experts: 27.8 us, 36.8 with the roundings ahead)
        constexpr int NX = BLOCKED ? 2 : 1;
        auto acts = [&](int h, u32x4(&x)[NX][4]) {
#pragma unroll
            for (int n = 0; n < NX; n++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    x[n][i] = BLOCKED ? *(const u32x4 *)(xrow + n * m.plane + 2048LL * (2 * back.c + h) + 512 * i)
                                      : pr.x[h][i];
        };
        f32x4 acc[NX][PN] = {};
        // the branches here touch LDS only: a load from memory in one would
        // make the next wait drain what is in flight
        auto close = [&] {  // the back cursor's pair is multiplied
            if (++back.c == back.ce) {
                const int i = back.lo + col;
                if constexpr (BLOCKED) {
#pragma unroll
                    for (int c = 0; c < QW; c++)
                        acc[0][c >> 2][c & 3] = join_parts<DT>(acc[0][c >> 2][c & 3], acc[1][c >> 2][c & 3]);
                } else {
#pragma unroll
                    for (int c = 0; c < QW; c++) {
                        const float y = acc[0][c >> 2][c & 3];
                        const int low = dpp_from<0x128, 0xF>(__builtin_bit_cast(int, y), 0);  // row_ror:8
                        acc[0][c >> 2][c & 3] = join_parts<DT>(y, __builtin_bit_cast(float, low));
                    }
                }
                if (i < back.hi) {
                    const int pair = pair_of[i], part = back.u % m.parts;
#pragma unroll
                    for (int pn = 0; pn < PN; pn++)
                        *(f32x4 *)(sums + (size_t)part * span + pair * CW + 16 * pn + 4 * g) = acc[0][pn];
                    if (part == 0 && g == 0) served[pair] = 1;
                }
#pragma unroll
                for (int n = 0; n < NX; n++)
#pragma unroll
                    for (int pn = 0; pn < PN; pn++) acc[n][pn] = f32x4{0.f, 0.f, 0.f, 0.f};
                back.u += NW;
                if (back.u < units) {
                    open(back);
                    if (BLOCKED) rows_at(back);
                }
            }
        };
        fetch();
        for (int s = 1; s < total; s++) {
            multiply_pair<FMT, DT>(pr, src, back.c, nch, acc, acts, fetch);
            close();
        }
        multiply_pair<FMT, DT>(pr, src, back.c, nch, acc, acts, [] {});
        close();
    }
    __syncthreads();

    // per token: its pairs in slot order, each the sum of its parts
    auto token_sum = [&](int t, int n, float (&v)[4]) {
        v[0] = v[1] = v[2] = v[3] = 0.0f;
        for (int j = 0; j < m.top_k; j++) {
            const int p = t * m.top_k + j;
            if (!served[p]) continue;
            f32x4 s = *(const f32x4 *)(sums + p * CW + n);
            for (int k = 1; k < m.parts; k++) s += *(const f32x4 *)(sums + (size_t)k * span + p * CW + n);
            const float wt = m.wts[p];
#pragma unroll
            for (int c = 0; c < 4; c++) v[c] = __builtin_fmaf(wt, s[c], v[c]);
        }
    };
    Args y = a;  // the store sees T rows
    y.M = m.T;
    float un[4];
    if (m.split == 1) {
        for (int q = tid; q < m.T * QW; q += 64 * NW) {
            const int t = q / QW, n = 4 * (q % QW), n0 = CW * strip + n;
            float v[4];
            token_sum(t, n, v);
            finish_quad<DT, EP_LIN>(y, t, n0, v, un, BiasQuad{}, res_quad(y, t, n0));
        }
        return;
    }
    float *mine = m.partial + ((long long)strip * m.split + slice) * m.T * CW;
    for (int q = tid; q < m.T * QW; q += 64 * NW) {
        float v[4];
        token_sum(q / QW, 4 * (q % QW), v);
        store_agent(mine + 4 * q, v);
    }
    // every wave's stores have reached the device's point of coherence before
    // the workgroup's arrival counts there, so the last one to arrive finds
    // all the others' sums
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0)
        s_last = __hip_atomic_fetch_add(m.arrived + strip, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == m.split - 1;
    __syncthreads();
    if (!s_last) return;
    const float *all = m.partial + (long long)strip * m.split * m.T * CW;
    for (int q = tid; q < m.T * QW; q += 64 * NW) {
        const int t = q / QW, n0 = CW * strip + 4 * (q % QW);
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < m.split; s += 4) {  // four in flight: each is a trip past the L2
            float x[4][4];
#pragma unroll
            for (int i = 0; i < 4; i++) load_agent(all + (long long)min(s + i, m.split - 1) * m.T * CW + 4 * q, x[i]);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int c = 0; c < 4; c++) v[c] = s + i < m.split ? v[c] + x[i][c] : v[c];
        }
        finish_quad<DT, EP_LIN>(y, t, n0, v, un, BiasQuad{}, res_quad(y, t, n0));
    }
}

}  // namespace qg
