// kv_cache.hip -- the passes around the 4-bit cache: norm and rotation of
// query and key heads, the append of new keys and values, and the read-back.
//
// Sixteen lanes take one head (of one token; in the append, of the four tokens
// that share value words), D/16 neighbouring dims each, so that a head is one
// contiguous load, its sum of squares four steps inside a row of lanes and
// a cache group of 32 dims two or three.  All of it is a stream of 16-byte
// loads and stores; nothing is staged.
#include "kv.h"

namespace qg {
namespace {

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

// Reductions over the first 4, 8 or 16 lanes' worth of neighbours: each step joins
// blocks whose lanes already agree, so a mirror serves for a swap.
template <typename F>
__device__ __forceinline__ F sum16(F x)
{
    x += dpp<kSwap1>(x);
    x += dpp<kSwap2>(x);
    x += dpp<kHalfMirror>(x);
    return x + dpp<kMirror>(x);
}

// E neighbouring elements.
template <int DT, int E, typename F>
__device__ __forceinline__ void load_row(const uint16_t *p, F (&x)[E])
{
    uint32_t w[E / 2];
    if constexpr (E == 8) __builtin_memcpy(w, __builtin_assume_aligned(p, 16), 16);
    else __builtin_memcpy(w, __builtin_assume_aligned(p, 8), 8);
#pragma unroll
    for (int i = 0; i < E / 2; i++) {
        x[2 * i] = (F)of_bits<DT>(w[i] & 0xFFFFu);
        x[2 * i + 1] = (F)of_bits<DT>(w[i] >> 16);
    }
}

template <int E>
__device__ __forceinline__ void load_f32(const float *p, float (&x)[E])
{
#pragma unroll
    for (int i = 0; i < E / 4; i++) {
        const f32x4 v = *(const f32x4 *)(p + 4 * i);
#pragma unroll
        for (int j = 0; j < 4; j++) x[4 * i + j] = v[j];
    }
}

// Dims E*l .. E*l+E-1 of one head, normed and rotated; false for a position
// outside the table.  The partner dims of a rotation come from memory once more
// (the same cache lines) instead of across lanes.
template <int DT, int D, typename F>
__device__ __forceinline__ bool turn_head(const TurnArgs &t, const uint16_t *x, const float *weight, int pos, int l,
                                          F (&y)[D / 16])
{
    constexpr int E = D / 16;
    const int d0 = E * l, half = t.rot >> 1;
    if (t.rope && (unsigned)pos >= (unsigned)t.rope_len) return false;
    const bool turned = t.rope && d0 < t.rot, low = d0 < half;
    const int dp = low ? d0 + half : d0 - half;  // the partners of the half-split form
    F p[E];
    load_row<DT, E>(x + d0, y);
    float c[E], s[E];
    if (turned) {
        const float *row = t.rope + (long long)pos * t.rot;
        if (t.interleaved) {
            __builtin_memcpy(c, __builtin_assume_aligned(row + d0 / 2, 2 * E), 2 * E);
            __builtin_memcpy(s, __builtin_assume_aligned(row + half + d0 / 2, 2 * E), 2 * E);
        } else {
            load_f32<E>(row + (low ? d0 : dp), c);
            load_f32<E>(row + half + (low ? d0 : dp), s);
            load_row<DT, E>(x + dp, p);
        }
    }
    if (t.eps >= 0.0f) {
        F ss = 0;
#pragma unroll
        for (int i = 0; i < E; i++) ss += y[i] * y[i];
        ss = sum16(ss);
        const F mean = ss * (F)(1.0 / D) + (F)t.eps;
        const F inv = (F)1 / (sizeof(F) == 8 ? (F)sqrt((double)mean) : (F)sqrtf((float)mean));
        if (weight) {
            float w[E];
            load_f32<E>(weight + d0, w);
#pragma unroll
            for (int i = 0; i < E; i++) y[i] *= inv * (F)w[i];
            if (turned && !t.interleaved) {
                load_f32<E>(weight + dp, w);
#pragma unroll
                for (int i = 0; i < E; i++) p[i] *= inv * (F)w[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) y[i] *= inv;
            if (turned && !t.interleaved) {
#pragma unroll
                for (int i = 0; i < E; i++) p[i] *= inv;
            }
        }
    }
    if (turned) {
        if (t.interleaved) {
#pragma unroll
            for (int i = 0; i < E / 2; i++) {
                const F a = y[2 * i], b = y[2 * i + 1], cc = (F)c[i], sn = (F)s[i];
                y[2 * i] = a * cc - b * sn;
                y[2 * i + 1] = b * cc + a * sn;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) {
                const F sn = low ? -(F)s[i] : (F)s[i];
                y[i] = y[i] * (F)c[i] + p[i] * sn;
            }
        }
    }
    return true;
}

// One head of one token to y, in binary32 with one rounding at the end; zeros
// for a position outside the table.
template <int DT, int D>
__device__ __forceinline__ void turn_store(const TurnArgs &t, const Heads &h, int row, int head, int pos, int l)
{
    constexpr int E = D / 16;
    float y[E];
    if (!turn_head<DT, D>(t, h.x + (long long)row * h.stride + head * D, h.weight, pos, l, y)) {
#pragma unroll
        for (int i = 0; i < E; i++) y[i] = 0.0f;
    }
    uint16_t *o = h.y + (long long)row * h.y_stride + head * D + E * l;
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; i++) w[i] = pack_out<DT>(y[2 * i], y[2 * i + 1]);
    __builtin_memcpy(__builtin_assume_aligned(o, 2 * E), w, 2 * E);
}

template <int DT, int D>
__global__ void __launch_bounds__(256) k_norm_rope(NormRopeArgs a)
{
    const int item = (int)(blockIdx.x * 16 + (threadIdx.x >> 4)), l = threadIdx.x & 15;
    const int all = a.q.heads + a.k.heads, row = item / all, head = item - row * all;
    if (row >= a.T) return;
    const int pos = a.t.positions ? a.t.positions[row] : 0;
    if (head < a.q.heads) turn_store<DT, D>(a.t, a.q, row, head, pos, l);
    else turn_store<DT, D>(a.t, a.k, row, head - a.q.heads, pos, l);
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

// 1/x to about a 64-bit step.
__device__ __forceinline__ double reciprocal(double x)
{
    double r = __builtin_amdgcn_rcp(x);
    r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
}

// a/b with r about 1/b: a product and one correction, which makes a quotient that
// 64 bits hold (a tie between two codes) exact.
__device__ __forceinline__ double quotient(double a, double b, double r)
{
    const double q = a * r;
    return __builtin_fma(__builtin_fma(-q, b, a), r, q);
}

// The cache's codes of a lane's E dims and the header of their group of 32, which
// lies in 32/E neighbouring lanes: minimum = fp16(min), scale = fp16((max -
// minimum)/15), both by way of binary32, code = the nearest of 0..15 to (x -
// minimum)/scale, ties to even.  In 64 bits, where vector arithmetic has the
// rate of 32 bits on this GPU: a code then is that of the definition and does
// not hang on the last bit of a binary32 norm or rotation.
template <int E>
__device__ __forceinline__ uint32_t quantize(double (&x)[E], uint32_t (&code)[E])
{
    bool odd = false;
#pragma unroll
    for (int i = 0; i < E; i++) odd |= !(fabsf((float)x[i]) <= kKvMax);
    if (odd) {
#pragma unroll
        for (int i = 0; i < E; i++) x[i] = x[i] != x[i] ? 0.0 : fmin(fmax(x[i], -(double)kKvMax), (double)kKvMax);
    }
    float lo = (float)x[0];  // the rounding keeps the order
    double hi = x[0];
#pragma unroll
    for (int i = 1; i < E; i++) {
        lo = fminf(lo, (float)x[i]);
        hi = fmax(hi, x[i]);
    }
    lo = fminf(lo, dpp<kSwap1>(lo));
    hi = fmax(hi, dpp<kSwap1>(hi));
    lo = fminf(lo, dpp<kSwap2>(lo));
    hi = fmax(hi, dpp<kSwap2>(hi));
    if constexpr (E == 4) {
        lo = fminf(lo, dpp<kHalfMirror>(lo));
        hi = fmax(hi, dpp<kHalfMirror>(hi));
    }
    const _Float16 m = (_Float16)lo;
    const double md = (double)(float)m;
    const _Float16 s = header_of(quotient(hi - md, 15.0, 1.0 / 15.0));
    const double sd = (double)(float)s, inv = sd > 0.0 ? reciprocal(sd) : 0.0;
#pragma unroll
    for (int i = 0; i < E; i++) code[i] = (uint32_t)(int)fminf(fmaxf((float)rint(quotient(x[i] - md, sd, inv)), 0.0f), 15.0f);
    return (uint32_t)__builtin_bit_cast(uint16_t, s) | ((uint32_t)__builtin_bit_cast(uint16_t, m) << 16);
}

// Row t's sequence and place, for 16 lanes of equal t; place -1 for a row of no
// sequence.
__device__ __forceinline__ int place_of(const KvView &v, int t, int &s)
{
    s = v.offs ? find_seq<16>(v, t, 1, 0) : t;
    const Seq q = seq_of(v, s);
    return t >= q.row && t < q.row + q.n ? q.first + t - q.row : INT_MIN;
}

// A row's key head into the cache.
template <int DT, int D>
__device__ __forceinline__ void append_key(const AppendArgs &a, int row, int head, int l)
{
    using L = KvLay<D>;
    constexpr int E = L::E;
    int s;
    const int at = place_of(a.v, row, s);
    if (at == INT_MIN) return;
    uint8_t *tile = tile_of<D>(a.v, s, at, head);
    double x[E];
    uint32_t code[E], w = 0;
    const int pos = a.t.positions ? a.t.positions[row] : at;
    if (!tile || !turn_head<DT, D>(a.t, a.k.x + (long long)row * a.k.stride + head * D, a.k.weight, pos, l, x)) return;
    const uint32_t header = quantize<E>(x, code);
    const int r = at & 15, d0 = E * l, h = d0 / (D / 4), j = d0 % (D / 4) / 8;
#pragma unroll
    for (int i = 0; i < E; i++) {
        const int c = (d0 & 4) + i;  // place in the word of 8 (E = 4: half a word)
        w |= code[i] << (4 * (c >> 1) + 16 * (c & 1));
    }
    if constexpr (E == 4) w |= (uint32_t)dpp<kSwap1>((int)w);
    if (E == 8 || (l & 1) == 0) *(uint32_t *)(tile + (h * 16 + r) * L::kLane + 4 * j) = w;
    if (d0 % 32 == 0) *(uint32_t *)(tile + L::kKeyHead + (d0 / 32 * 16 + r) * 4) = header;
}

// Values: 16 lanes take a quad of places, whose codes share words, and one head.
// A quad whose tokens are not all new keeps the others' codes.
template <int DT, int D>
__device__ __forceinline__ void append_values(const AppendArgs &a, int slot, int head, int l)
{
    using L = KvLay<D>;
    constexpr int E = L::E;
    const KvView &v = a.v;
    const int s = v.offs ? find_seq<16>(v, slot, kQuad, 2) : slot;
    const Seq q = seq_of(v, s);
    const int at0 = ((v.offs ? slot - (row_end(v, s) / kQuad + 2 * s) : 0) + (q.first >> 2)) * kQuad;
    if (at0 < 0 || at0 >= q.len) return;
    uint8_t *tile = tile_of<D>(v, s, at0, head);
    if (!tile) return;
    const int quad = (at0 >> 2) & 3, d0 = E * l;
    uint32_t *out = (uint32_t *)(tile + L::kVal + (quad * 16 + l) * L::kLane);
    uint32_t words[E / 2], fresh = 0;
#pragma unroll
    for (int i = 0; i < E / 2; i++) words[i] = 0;
#pragma unroll
    for (int i = 0; i < kQuad; i++) {
        const int at = at0 + i, row = q.row + at - q.first;
        if (at < q.first || at >= q.len) continue;
        if (a.t.rope && (unsigned)(a.t.positions ? a.t.positions[row] : at) >= (unsigned)a.t.rope_len) continue;  // a padded row
        double x[E];
        uint32_t code[E];
        load_row<DT, E>(a.val + (long long)row * a.val_stride + head * D + d0, x);
        const uint32_t header = quantize<E>(x, code);
#pragma unroll
        for (int j = 0; j < E; j++) words[j >> 1] |= code[j] << (4 * (2 * (j & 1) + (i >> 1)) + 16 * (i & 1));
        fresh |= 0x0F0Fu << (4 * (i >> 1) + 16 * (i & 1));
        if (d0 % 32 == 0) *(uint32_t *)(tile + L::kValHead + (d0 / 32 * 16 + 4 * quad + i) * 4) = header;
    }
    if (fresh == 0) return;
    if (fresh != 0xFFFFFFFFu) {
#pragma unroll
        for (int i = 0; i < E / 2; i++) words[i] |= out[i] & ~fresh;
    }
    __builtin_memcpy(__builtin_assume_aligned(out, 2 * E), words, 2 * E);
}

// Workgroups of values (quads, the longest chains, first), of keys and of queries.
template <int DT, int D>
__global__ void __launch_bounds__(256) k_kv_append(AppendArgs a)
{
    const int l = threadIdx.x & 15, sub = threadIdx.x >> 4;
    int b = blockIdx.x;
    if (b < a.value_blocks) {
        const int item = b * 16 + sub, slot = item / a.v.H;
        const int slots = a.v.offs ? a.v.T / kQuad + 2 * a.v.S : a.v.S;
        if (slot < slots) append_values<DT, D>(a, slot, item - slot * a.v.H, l);
        return;
    }
    b -= a.value_blocks;
    if (b < a.key_blocks) {
        const int item = b * 16 + sub, row = item / a.v.H;
        if (row < a.v.T) append_key<DT, D>(a, row, item - row * a.v.H, l);
        return;
    }
    const int item = (b - a.key_blocks) * 16 + sub, row = item / a.q.heads;
    if (row >= a.v.T) return;
    int s;
    const int at = place_of(a.v, row, s);
    if (at == INT_MIN) return;
    turn_store<DT, D>(a.t, a.q, row, item - row * a.q.heads, a.t.positions ? a.t.positions[row] : at, l);
}

// One token's head as the cache holds it: dims E*l .. of keys and values.
template <int D>
__device__ __forceinline__ void read_token(const uint8_t *tile, int r, int l, float (&k)[D / 16], float (&v)[D / 16])
{
    using L = KvLay<D>;
    constexpr int E = L::E;
    const int d0 = E * l, g = d0 / 32, h = d0 / (D / 4), j = d0 % (D / 4) / 8, i = r & 3;
    const uint32_t kw = *(const uint32_t *)(tile + (h * 16 + r) * L::kLane + 4 * j);
    const uint32_t kh = *(const uint32_t *)(tile + L::kKeyHead + (g * 16 + r) * 4);
    const uint32_t vh = *(const uint32_t *)(tile + L::kValHead + (g * 16 + r) * 4);
    const uint32_t *vw = (const uint32_t *)(tile + L::kVal + ((r >> 2) * 16 + l) * L::kLane);
#pragma unroll
    for (int e = 0; e < E; e++) {
        const int c = (d0 & 4) + e;
        k[e] = fmaf((float)((kw >> (4 * (c >> 1) + 16 * (c & 1))) & 15u), f16_to_f32(kh & 0xFFFFu), f16_to_f32(kh >> 16));
        const uint32_t b = vw[e >> 1] >> (4 * (2 * (e & 1) + (i >> 1)) + 16 * (i & 1));
        v[e] = fmaf((float)(b & 15u), f16_to_f32(vh & 0xFFFFu), f16_to_f32(vh >> 16));
    }
}

template <int OT, int D>
__global__ void __launch_bounds__(256) k_kv_read(KvView v, void *ko, void *vo)
{
    constexpr int E = D / 16;
    const int item = (int)(blockIdx.x * 16 + (threadIdx.x >> 4)), l = threadIdx.x & 15;
    const int row = item / v.H, head = item - row * v.H;
    if (row >= v.T) return;
    int s;
    const int at = place_of(v, row, s);  // no place at all is none of the table's
    float k[E], x[E];
#pragma unroll
    for (int i = 0; i < E; i++) k[i] = x[i] = 0.0f;
    if (const uint8_t *tile = tile_of<D>(v, s, at, head)) read_token<D>(tile, at & 15, l, k, x);
    const long long o = ((long long)row * v.H + head) * D + E * l;
    store_out<OT, E>(ko, o, k);
    store_out<OT, E>(vo, o, x);
}

unsigned blocks(long long items, int per) { return (unsigned)((items + per - 1) / per); }

template <int DT, int D>
hipError_t run_norm_rope(const NormRopeArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((k_norm_rope<DT, D>), dim3(blocks((long long)a.T * (a.q.heads + a.k.heads), 16)), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t run_append(AppendArgs a, hipStream_t s)
{
    const long long slots = a.v.offs ? a.v.T / kQuad + 2LL * a.v.S : a.v.S;
    a.value_blocks = (int)blocks(slots * a.v.H, 16);
    a.key_blocks = (int)blocks((long long)a.v.T * a.v.H, 16);
    const unsigned qb = a.q.x ? blocks((long long)a.v.T * a.q.heads, 16) : 0;
    hipLaunchKernelGGL((k_kv_append<DT, D>), dim3((unsigned)(a.value_blocks + a.key_blocks) + qb), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int OT, int D>
hipError_t run_read(const KvView &v, void *k, void *val, hipStream_t s)
{
    hipLaunchKernelGGL((k_kv_read<OT, D>), dim3(blocks((long long)v.T * v.H, 16)), dim3(256), 0, s, v, k, val);
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
