// kv_cache.hip -- the passes around the 4-bit cache: norm and rotation of
// query and key heads, the append of new keys and values, and the read-back.
//
// D/8 lanes take a head, 8 neighbouring dims (16 bytes) each, so that its sum of squares is three
// or four steps inside a row of lanes and a cache group of 32 dims two; nothing is
// staged.  What a token's heads share (its place in the cache, the angles, the weights) is
// looked up once for HC heads, whose loads are in flight together.
#include "kv.h"

namespace qg {
namespace {

constexpr int E = 8;  // dims of a lane
template <int D>
constexpr int kItems = 256 * E / D;  // groups of D/E lanes in a workgroup

// x of another lane of the row of 16, by DPP (no trip through LDS).
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;  // lanes ^1, ^2, mirrored in 8, in 16

template <int CTRL>
__device__ __forceinline__ int dpp(int x) { return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xF, 0xF, false); }
template <int CTRL>
__device__ __forceinline__ float dpp(float x) { return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, x))); }
template <int CTRL>
__device__ __forceinline__ double dpp(double x)
{
    const u32x2 v = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{(uint32_t)dpp<CTRL>((int)v.x), (uint32_t)dpp<CTRL>((int)v.y)});
}

// Sums over 8 or 16 neighbours: each step joins blocks whose lanes already agree, so a mirror
// serves for a swap.
template <int LANES, typename F>
__device__ __forceinline__ F sum_of(F x)
{
    x += dpp<kSwap1>(x);
    x += dpp<kSwap2>(x);
    x += dpp<kHalfMirror>(x);
    if constexpr (LANES == 16) x += dpp<kMirror>(x);
    return x;
}

// E neighbouring elements as they lie in memory, and their values.
__device__ __forceinline__ void load_raw(const uint16_t *p, uint32_t (&w)[E / 2])
{
    __builtin_memcpy(w, __builtin_assume_aligned(p, 2 * E), 2 * E);
}

template <int DT, typename F>
__device__ __forceinline__ void values_of(const uint32_t (&w)[E / 2], F (&x)[E])
{
#pragma unroll
    for (int i = 0; i < E / 2; i++) {
        x[2 * i] = (F)of_bits<DT>(w[i] & 0xFFFFu);
        x[2 * i + 1] = (F)of_bits<DT>(w[i] >> 16);
    }
}

template <int N>
__device__ __forceinline__ void load_f32(const float *p, float (&x)[N])
{
    __builtin_memcpy(x, __builtin_assume_aligned(p, N * 4 < 16 ? N * 4 : 16), 4 * N);
}

// 1/sqrt(x) and 1/x to about a step of their type.
template <typename F>
__device__ __forceinline__ F reciprocal_root(F x)
{
    F r;
    if constexpr (sizeof(F) == 8) r = __builtin_amdgcn_rsq(x);
    else r = __builtin_amdgcn_rsqf(x);
    if (!(x < (F)INFINITY) || r == (F)INFINITY) return r;  // of 0, infinity and NaN as it is
#pragma unroll
    for (size_t i = 4; i <= sizeof(F); i += 4) r = fma(fma(-x * r, r, (F)1), (F)0.5 * r, r);
    return r;
}

__device__ __forceinline__ double reciprocal(double x)
{
    double r = __builtin_amdgcn_rcp(x);
    r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
}

// How a launch turns its heads, the same in all lanes.
enum : int { kPlain = 0, kHalves = 1, kPairs = 2 };  // no rotation; dims i and rot/2 + i; dims 2i and 2i + 1

template <int MODE, bool NORM>
struct TurnBy {
    static constexpr int mode = MODE;
    static constexpr bool norm = NORM;
};

// Calls f with the TurnBy of t: branches taken once, and none of them among the heads.
template <typename Fn>
__device__ __forceinline__ void turn_by(const TurnArgs &t, Fn f)
{
    const bool norm = t.eps >= 0.0f;
    if (!t.rope) norm ? f(TurnBy<kPlain, true>()) : f(TurnBy<kPlain, false>());
    else if (t.interleaved) norm ? f(TurnBy<kPairs, true>()) : f(TurnBy<kPairs, false>());
    else norm ? f(TurnBy<kHalves, true>()) : f(TurnBy<kHalves, false>());
}

// A lane's elements of HC heads from `head` on and, of the half-split form, those of their partner
// dims, from memory once more (the same cache lines) instead of across lanes.  Past the last
// head, those of the first again, which nobody uses.
template <typename By, int D, int HC>
__device__ __forceinline__ void load_heads(const TurnArgs &t, const Heads &h, int row, int head, int l,
                                           uint32_t (&own)[HC][E / 2], uint32_t (&part)[HC][E / 2])
{
    const uint16_t *x = h.x + (long long)row * h.stride + head * D;
    const int d0 = E * l, half = t.rot >> 1, dp = d0 >= t.rot ? d0 : d0 < half ? d0 + half : d0 - half;
#pragma unroll
    for (int i = 0; i < HC; i++) {
        const uint16_t *from = x + (head + i < h.heads ? i * D : 0);
        load_raw(from + d0, own[i]);
        if constexpr (By::mode == kHalves) load_raw(from + dp, part[i]);
    }
}

// What a lane's heads share: element i becomes inv * (x[i] * c[i] + p[i] * s[i]), p its partner,
// inv the norm's factor, and c and s the weights, also in the rotated part times the angles' cosine
// and sine.
template <typename F>
struct RowTurn {
    bool turned;
    F c[E], s[E];
};

template <typename By, typename F>
__device__ __forceinline__ void row_turn(const TurnArgs &t, const float *weight, int pos, int l, RowTurn<F> &r)
{
    const int d0 = E * l, half = t.rot >> 1;
    float w[E], wp[E];
    const bool low = d0 < half;
    r.turned = By::mode != kPlain && d0 < t.rot;
#pragma unroll
    for (int i = 0; i < E; i++) w[i] = wp[i] = 1.0f;
    if (By::norm && weight) {
        load_f32(weight + d0, w);
        if constexpr (By::mode == kHalves) load_f32(weight + (!r.turned ? d0 : low ? d0 + half : d0 - half), wp);
    }
#pragma unroll
    for (int i = 0; i < E; i++) r.c[i] = (F)w[i];
    if constexpr (By::mode == kPlain) return;
    const float *line = t.rope + (long long)pos * t.rot;
    if constexpr (By::mode == kHalves) {
        float c[E], s[E];
        line += !r.turned ? 0 : low ? d0 : d0 - half;
        load_f32(line, c);
        load_f32(line + half, s);
#pragma unroll
        for (int i = 0; i < E; i++) {
            if (r.turned) r.c[i] *= (F)c[i];
            r.s[i] = r.turned ? (F)wp[i] * (F)(low ? -s[i] : s[i]) : (F)0;
        }
    } else {
        float c[E / 2], s[E / 2];
        line += r.turned ? d0 / 2 : 0;
        load_f32(line, c);
        load_f32(line + half, s);
#pragma unroll
        for (int i = 0; i < E; i++) {
            if (r.turned) r.c[i] *= (F)c[i / 2];
            r.s[i] = r.turned ? (F)w[i ^ 1] * (F)(i & 1 ? s[i / 2] : -s[i / 2]) : (F)0;
        }
    }
}

// A lane's dims of one head, normed and rotated.
template <typename By, int DT, int D, typename F>
__device__ __forceinline__ void turn_head(const TurnArgs &t, const RowTurn<F> &r, const uint32_t (&own)[E / 2],
                                          const uint32_t (&part)[E / 2], F (&y)[E])
{
    F x[E], p[E];
    values_of<DT>(own, x);
    if constexpr (By::mode == kHalves) {
        uint32_t w[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; i++) w[i] = r.turned ? part[i] : 0u;  // no infinity times zero
        values_of<DT>(w, p);
    }
#pragma unroll
    for (int i = 0; i < E; i++) {
        y[i] = x[i] * r.c[i];
        if constexpr (By::mode == kHalves) y[i] = fma(p[i], r.s[i], y[i]);
        if constexpr (By::mode == kPairs) y[i] = r.turned ? fma(x[i ^ 1], r.s[i], y[i]) : y[i];
    }
    if constexpr (By::norm) {
        F ss = 0;
#pragma unroll
        for (int i = 0; i < E; i++) ss = fma(x[i], x[i], ss);
        const F inv = reciprocal_root<F>(sum_of<D / E>(ss) * (F)(1.0 / D) + (F)t.eps);
#pragma unroll
        for (int i = 0; i < E; i++) y[i] *= inv;
    }
}

// HC heads of one row from `head` on to y, in binary32 with one rounding at the end; zeros
// for a position outside the table.  pos_of: the row's position; false: it belongs to no sequence,
// and is left or, with zero_rest, zeros.
template <typename By, int DT, int D, int HC, typename PosOf>
__device__ __forceinline__ void turn_store(const TurnArgs &t, const Heads &h, int row, int head, int l, bool zero_rest, PosOf pos_of)
{
    uint32_t own[HC][E / 2], part[HC][E / 2];
    load_heads<By, D, HC>(t, h, row, head, l, own, part);
    int pos;
    const bool owned = pos_of(pos);
    if (!owned && !zero_rest) return;
    const bool inside = owned && (By::mode == kPlain || (unsigned)pos < (unsigned)t.rope_len);
    RowTurn<float> r;
    row_turn<By>(t, h.weight, inside ? pos : 0, l, r);
    uint16_t *o = h.y + (long long)row * h.y_stride + head * D + E * l;
#pragma unroll
    for (int i = 0; i < HC; i++) {
        float y[E];
        turn_head<By, DT, D>(t, r, own[i], part[i], y);
        if (head + i < h.heads && inside) store_out<DT, E>(o, i * D, y);
    }
    if (inside) return;
    const float zeros[E] = {};
    for (int i = 0; i < HC && head + i < h.heads; i++) store_out<DT, E>(o, i * D, zeros);
}

__host__ __device__ inline int chunks(int heads, int hc) { return (heads + hc - 1) / hc; }

// One read and one write of each head; bound by memory once the heads fill the CUs (4099 tokens of 36
// heads of 128 in 14.9 us, 75 MB at 5.0 TB/s out of and into the last-level cache) and by
// the launch and one chain of loads below (one token 2.5 us).
template <int DT, int D, int HC>
__global__ void __launch_bounds__(256) k_norm_rope(NormRopeArgs a)
{
    const int item = (int)(blockIdx.x * kItems<D> + threadIdx.x / (D / E)), l = threadIdx.x % (D / E);
    const int qc = chunks(a.q.heads, HC), all = qc + chunks(a.k.heads, HC), row = item / all, i = item - row * all;
    if (row >= a.T) return;
    const bool key = i >= qc;
    turn_by(a.t, [&](auto by) {
        turn_store<decltype(by), DT, D, HC>(a.t, key ? a.k : a.q, row, HC * (key ? i - qc : i), l, false, [&](int &p) {
            p = a.t.positions ? a.t.positions[row] : 0;
            return true;
        });
    });
}

// fp16 of a 64-bit value, rounded to binary32 on the way.  The compiler would
// merge the two conversions into one rounding (in software, and other bits
// where binary32 lands on a tie); the empty statement keeps them apart.
__device__ __forceinline__ _Float16 header_of(double x)
{
    float f = (float)x;
    asm("" : "+v"(f));
    return (_Float16)f;
}

// a/b with r about 1/b: a product and one correction, which makes a quotient that
// 64 bits hold (a tie between two codes) exact.
__device__ __forceinline__ double quotient(double a, double b, double r)
{
    const double q = a * r;
    return __builtin_fma(__builtin_fma(-q, b, a), r, q);
}

// The nearest whole number, ties to even, of |x| < 2^31: what a sum with 1.5 * 2^52 leaves in its
// low word.
__device__ __forceinline__ int nearest(double x)
{
    return (int)(uint32_t)__builtin_bit_cast(unsigned long long, x + 6755399441055744.0);
}

// The larger of two numbers, neither NaN: for 64 bits without the instructions that would quiet one.
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b)
{
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// The cache's codes of a lane's E dims and the header of their group of 32, which
// lies in 4 neighbouring lanes: minimum = fp16(min), scale = fp16((max -
// minimum)/15), both by way of binary32, code = the nearest of 0..15 to (x -
// minimum)/scale, ties to even.  In 64 bits, where vector arithmetic has the
// rate of 32 bits on this GPU: a code then is that of the definition and does
// not hang on the last bit of a binary32 norm or rotation.
template <typename F>
__device__ __forceinline__ uint32_t quantize(F (&x)[E], uint32_t (&code)[E])
{
    bool odd = false;
#pragma unroll
    for (int i = 0; i < E; i++) odd |= !(fabsf((float)x[i]) <= kKvMax);
    if (odd) {
#pragma unroll
        for (int i = 0; i < E; i++) x[i] = x[i] != x[i] ? (F)0 : fmin(fmax(x[i], -(F)kKvMax), (F)kKvMax);
    }
    float lo = (float)x[0];  // the rounding keeps the order
    F hi = x[0];
#pragma unroll
    for (int i = 1; i < E; i++) {
        lo = fminf(lo, (float)x[i]);
        hi = larger(hi, x[i]);
    }
    lo = fminf(lo, dpp<kSwap1>(lo));
    hi = larger(hi, dpp<kSwap1>(hi));
    lo = fminf(lo, dpp<kSwap2>(lo));
    hi = larger(hi, dpp<kSwap2>(hi));
    const _Float16 m = (_Float16)lo;
    const double md = (double)(float)m;
    const _Float16 s = header_of(quotient((double)hi - md, 15.0, 1.0 / 15.0));
    const double sd = (double)(float)s, inv = sd > 0.0 ? reciprocal(sd) : 0.0;
#pragma unroll
    for (int i = 0; i < E; i++) code[i] = (uint32_t)min(max(nearest(quotient((double)x[i] - md, sd, inv)), 0), 15);
    return (uint32_t)__builtin_bit_cast(uint16_t, s) | ((uint32_t)__builtin_bit_cast(uint16_t, m) << 16);
}

// Row t's sequence and place, for LANES lanes of equal t; INT_MIN for a row of no
// sequence.
template <int LANES>
__device__ __forceinline__ int place_of(const KvView &v, int t, int &s)
{
    s = v.offs ? find_seq<LANES>(v, t, 1, 0) : t;
    const Seq q = seq_of(v, s);
    return t >= q.row && t < q.row + q.n ? q.first + t - q.row : INT_MIN;
}

// HC key heads of one row into the cache.
template <typename By, int DT, int D, int HC>
__device__ __forceinline__ void append_keys(const AppendArgs &a, int row, int head, int l)
{
    using L = KvLay<D>;
    uint32_t own[HC][E / 2], part[HC][E / 2];
    load_heads<By, D, HC>(a.t, a.k, row, head, l, own, part);
    int s;
    const int at = place_of<D / E>(a.v, row, s);
    if (at == INT_MIN) return;
    const uint8_t *tile0 = tile_of<D>(a.v, s, at, head);
    const int pos = a.t.positions ? a.t.positions[row] : at;
    if (!tile0 || (By::mode != kPlain && (unsigned)pos >= (unsigned)a.t.rope_len)) return;
    RowTurn<double> t;
    row_turn<By>(a.t, a.k.weight, pos, l, t);
    const int r = at & 15, d0 = E * l, h = d0 / (D / 4), j = d0 % (D / 4) / 8;
    const long long region = (long long)L::kBytes << (a.v.page_shift - 4);  // of a head in a page
#pragma unroll
    for (int i = 0; i < HC; i++) {
        double y[E];
        uint32_t code[E], w = 0;
        turn_head<By, DT, D>(a.t, t, own[i], part[i], y);
        const uint32_t header = quantize(y, code);
#pragma unroll
        for (int e = 0; e < E; e++) {
            w |= code[e] << (4 * (e >> 1) + 16 * (e & 1));
        }
        if (head + i >= a.v.H) continue;
        uint8_t *tile = const_cast<uint8_t *>(tile0) + region * i;
        *(uint32_t *)(tile + (h * 16 + r) * L::kLane + 4 * j) = w;
        if (d0 % 32 == 0) *(uint32_t *)(tile + L::kKeyHead + (d0 / 32 * 16 + r) * 4) = header;
    }
}

// Values: D/8 lanes take a head of a quad of places, whose codes share words.  A quad whose
// tokens are not all new keeps the others' codes.
template <int DT, int D>
__device__ __forceinline__ void append_values(const AppendArgs &a, int slot, int head, int l)
{
    using L = KvLay<D>;
    const KvView &v = a.v;
    const int s = v.offs ? find_seq<D / E>(v, slot, kQuad, 2) : slot;
    const Seq q = seq_of(v, s);
    const int at0 = ((v.offs ? slot - (row_end(v, s) / kQuad + 2 * s) : 0) + (q.first >> 2)) * kQuad;
    if (at0 < 0 || at0 >= q.len) return;
    uint8_t *tile = tile_of<D>(v, s, at0, head);
    if (!tile) return;
    const int quad = (at0 >> 2) & 3, d0 = E * l, row0 = q.row + at0 - q.first;
    bool live[kQuad];
    uint32_t fresh = 0;
#pragma unroll
    for (int i = 0; i < kQuad; i++) {
        live[i] = at0 + i >= q.first && at0 + i < q.len;
        if (a.t.rope && live[i])  // else a padded row
            live[i] = (unsigned)(a.t.positions ? a.t.positions[row0 + i] : at0 + i) < (unsigned)a.t.rope_len;
        fresh |= live[i] ? 0x0F0Fu << (4 * (i >> 1) + 16 * (i & 1)) : 0u;
    }
    if (fresh == 0) return;
    const int some = fresh & 0x0F0Fu ? 0 : live[1] ? 1 : live[2] ? 2 : 3;
    uint32_t raw[kQuad][E / 2], words[E / 2], old[E / 2];
    uint32_t *out = (uint32_t *)(tile + L::kVal + quad * 16 * L::kLane + 2 * E * l);
#pragma unroll
    for (int i = 0; i < kQuad; i++)  // of rows that are not new, one that is, and not used
        load_raw(a.val + (long long)(row0 + (live[i] ? i : some)) * a.val_stride + head * D + d0, raw[i]);
    if (fresh != 0xFFFFFFFFu) __builtin_memcpy(old, __builtin_assume_aligned(out, 2 * E), 2 * E);
#pragma unroll
    for (int i = 0; i < E / 2; i++) words[i] = fresh != 0xFFFFFFFFu ? old[i] & ~fresh : 0u;
#pragma unroll
    for (int i = 0; i < kQuad; i++) {
        if (!live[i]) continue;
        float x[E];
        uint32_t code[E];
        values_of<DT>(raw[i], x);
        const uint32_t header = quantize(x, code);
#pragma unroll
        for (int j = 0; j < E; j++) words[j >> 1] |= code[j] << (4 * (2 * (j & 1) + (i >> 1)) + 16 * (i & 1));
        if (d0 % 32 == 0) *(uint32_t *)(tile + L::kValHead + (d0 / 32 * 16 + 4 * quad + i) * 4) = header;
    }
    __builtin_memcpy(__builtin_assume_aligned(out, 2 * E), words, 2 * E);
}

// Workgroups of values (quads, the longest chains, first), of keys and of queries.  Bound by the
// 64-bit arithmetic of the codes, about 30 instructions a dim, next to the loads: 4096 tokens of
// 32 query and 8 key heads of 128 take 24 us (89 MB, 3.7 TB/s), 8192 of 8 key heads of 64
// 14 us; one token takes 3.3 us, a chain of look-up, load and reduction.  A lane of 8 dims
// in place of 4 for heads of 64 took the 8192 tokens from 15.5 us to 14.
template <int DT, int D, int HC>
__global__ void __launch_bounds__(256) k_kv_append(AppendArgs a)
{
    const int l = threadIdx.x % (D / E), sub = threadIdx.x / (D / E), hc = chunks(a.v.H, HC);
    int b = blockIdx.x;
    if (b < a.value_blocks) {
        const int item = b * kItems<D> + sub, slot = item / a.v.H;
        const int slots = a.v.offs ? a.v.T / kQuad + 2 * a.v.S : a.v.S;
        if (slot < slots) append_values<DT, D>(a, slot, item - slot * a.v.H, l);
        return;
    }
    b -= a.value_blocks;
    if (b < a.key_blocks) {
        const int item = b * kItems<D> + sub, row = item / hc;
        if (row < a.v.T)
            turn_by(a.t, [&](auto by) { append_keys<decltype(by), DT, D, HC>(a, row, HC * (item - row * hc), l); });
        return;
    }
    const int qc = chunks(a.q.heads, HC), item = (b - a.key_blocks) * kItems<D> + sub, row = item / qc;
    if (row >= a.v.T) return;
    turn_by(a.t, [&](auto by) {
        turn_store<decltype(by), DT, D, HC>(a.t, a.q, row, HC * (item - row * qc), l, a.zero_rest, [&](int &p) {
            int s;
            const int at = place_of<D / E>(a.v, row, s);
            p = a.t.positions ? a.t.positions[row] : at;
            return at != INT_MIN;
        });
    });
}

// Bound by the writes: 8192 tokens of 8 heads of 128 in 10 us (44 MB, 4.4 TB/s).
template <int OT, int D, int HC>
__global__ void __launch_bounds__(256) k_kv_read(KvView v, void *ko, void *vo)
{
    using L = KvLay<D>;
    const int item = (int)(blockIdx.x * kItems<D> + threadIdx.x / (D / E)), l = threadIdx.x % (D / E), hc = chunks(v.H, HC);
    const int row = item / hc, head = HC * (item - row * hc);
    if (row >= v.T) return;
    int s;
    const int at = place_of<D / E>(v, row, s);  // no place at all is none of the table's
    const uint8_t *tile0 = tile_of<D>(v, s, at, head);
    const int r = at & 15, d0 = E * l, gr = d0 / 32, h = d0 / (D / 4), j = d0 % (D / 4) / 8, i = r & 3;
    const long long region = (long long)L::kBytes << (v.page_shift - 4);  // of a head in a page
    uint32_t kw[HC], kh[HC], vh[HC], vw[HC][E / 2];
    if (tile0) {
#pragma unroll
        for (int c = 0; c < HC; c++) {
            const uint8_t *tile = tile0 + (head + c < v.H ? region * c : 0);
            kw[c] = *(const uint32_t *)(tile + (h * 16 + r) * L::kLane + 4 * j);
            kh[c] = *(const uint32_t *)(tile + L::kKeyHead + (gr * 16 + r) * 4);
            vh[c] = *(const uint32_t *)(tile + L::kValHead + (gr * 16 + r) * 4);
            __builtin_memcpy(vw[c], __builtin_assume_aligned(tile + L::kVal + (r >> 2) * 16 * L::kLane + 2 * E * l, 2 * E), 2 * E);
        }
    }
#pragma unroll
    for (int c = 0; c < HC; c++) {
        float k[E], x[E];
#pragma unroll
        for (int e = 0; e < E; e++) {
            const uint32_t b = vw[c][e >> 1] >> (4 * (2 * (e & 1) + (i >> 1)) + 16 * (i & 1));
            k[e] = fmaf((float)((kw[c] >> (4 * (e >> 1) + 16 * (e & 1))) & 15u), f16_to_f32(kh[c] & 0xFFFFu), f16_to_f32(kh[c] >> 16));
            x[e] = fmaf((float)(b & 15u), f16_to_f32(vh[c] & 0xFFFFu), f16_to_f32(vh[c] >> 16));
            if (!tile0) k[e] = x[e] = 0.0f;
        }
        if (head + c >= v.H) continue;
        const long long o = ((long long)row * v.H + head + c) * D + d0;
        store_out<OT, E>(ko, o, k);
        store_out<OT, E>(vo, o, x);
    }
}

unsigned blocks(long long items, int per) { return (unsigned)((items + per - 1) / per); }

// Below this many heads D/8 lanes take one; from here on two.  One against two, heads of 128 in
// us: norm and rotation 3.6 and 3.5 at 10240 heads, 8.1 and 6.7 at 40960; append with the
// read-back 9.4 and 10.4 at 24576 of single tokens, 11.8 and 10.0 at 31584 of a prompt; read 4.0
// and 4.1 at 16384, 6.6 and 5.7 at 32768.  Four gained at most another 8% from 98304 on.
constexpr long long kManyHeads = 28672;

template <int DT, int D, int HC>
hipError_t start_norm_rope(const NormRopeArgs &a, hipStream_t s)
{
    const long long items = (long long)a.T * (chunks(a.q.heads, HC) + chunks(a.k.heads, HC));
    hipLaunchKernelGGL((k_norm_rope<DT, D, HC>), dim3(blocks(items, kItems<D>)), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t run_norm_rope(const NormRopeArgs &a, hipStream_t s)
{
    return (long long)a.T * (a.q.heads + a.k.heads) < kManyHeads ? start_norm_rope<DT, D, 1>(a, s) : start_norm_rope<DT, D, 2>(a, s);
}

template <int DT, int D, int HC>
hipError_t start_append(AppendArgs a, hipStream_t s)
{
    const long long slots = a.v.offs ? a.v.T / kQuad + 2LL * a.v.S : a.v.S;
    a.value_blocks = (int)blocks(slots * a.v.H, kItems<D>);
    a.key_blocks = (int)blocks((long long)a.v.T * chunks(a.v.H, HC), kItems<D>);
    const unsigned qb = a.q.x ? blocks((long long)a.v.T * chunks(a.q.heads, HC), kItems<D>) : 0;
    hipLaunchKernelGGL((k_kv_append<DT, D, HC>), dim3((unsigned)(a.value_blocks + a.key_blocks) + qb), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t run_append(const AppendArgs &a, hipStream_t s)
{
    return (long long)a.v.T * (2 * a.v.H + a.q.heads) < kManyHeads ? start_append<DT, D, 1>(a, s) : start_append<DT, D, 2>(a, s);
}

template <int OT, int D>
hipError_t run_read(const KvView &v, void *k, void *val, hipStream_t s)
{
    if ((long long)v.T * v.H < kManyHeads)
        hipLaunchKernelGGL((k_kv_read<OT, D, 1>), dim3(blocks((long long)v.T * v.H, kItems<D>)), dim3(256), 0, s, v, k, val);
    else
        hipLaunchKernelGGL((k_kv_read<OT, D, 2>), dim3(blocks((long long)v.T * chunks(v.H, 2), kItems<D>)), dim3(256), 0, s, v, k, val);
    return hipGetLastError();
}

}  // namespace

#define QG_BY_TYPE(fn, ...)                                                              \
    (dtype == DT_F16 ? (D == 64 ? fn<DT_F16, 64>(__VA_ARGS__) : fn<DT_F16, 128>(__VA_ARGS__)) \
                     : (D == 64 ? fn<DT_BF16, 64>(__VA_ARGS__) : fn<DT_BF16, 128>(__VA_ARGS__)))

hipError_t launch_norm_rope(int dtype, int D, const NormRopeArgs &a, hipStream_t s) { return QG_BY_TYPE(run_norm_rope, a, s); }
hipError_t launch_kv_append(int dtype, int D, const AppendArgs &a, hipStream_t s) { return QG_BY_TYPE(run_append, a, s); }

hipError_t launch_kv_read(int out_type, int D, const KvView &v, void *k, void *val, hipStream_t s)
{
    if (out_type == QGEMM_F32) return D == 64 ? run_read<QGEMM_F32, 64>(v, k, val, s) : run_read<QGEMM_F32, 128>(v, k, val, s);
    const int dtype = out_type;
    return QG_BY_TYPE(run_read, v, k, val, s);
}

}  // namespace qg
