// kv_attention.hip -- attention over the 4-bit paged cache.
//
//   y_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(scale (q_i.k_t) - m_i)
//
// Both kernels compute the transposed products: S^T = K Q^T with the keys as
// the MFMA's A rows, then O^T = V^T P^T.  An accumulator column is then a query
// row: its running maximum and sum live in the lanes that hold the column, the
// rescaling of O is one factor per lane, and the registers that S^T leaves
// are, packed to fp16, the B operand of the second product as they stand (the
// order of the contraction is free as long as V's registers run over the same
// tokens, which the cache's layout does).  Nothing of P goes through LDS.
//
// Operands are fp16 for both activation types.  Queries in bfloat16 are scaled
// by a power of two per row, which fp16 then holds exactly but for elements 2^-22
// of the row's largest; keys and values are code*scale + minimum rounded once to
// fp16, probabilities likewise.
// Products, maxima, sums and O are binary32.
//
// Of an fp16 result, whose own rounding is no larger than these, the keys' is the one that
// shows: over few keys the errors of their products do not average out. Rows that see at most
// kFewKeys of them therefore take the keys in two fp16 parts, about 22 bits, and with them the
// other rows of their tile (few_keys). The error is then at most 1.4 times that of binary32
// arithmetic with the result rounded, where it was 1.8 over 20 keys, 1.65 over 100, 1.4 over 330 and 1.3
// over 658. In us, with one part and as it is: 658 tokens 22.2 and 23.7, 4096 165 and 170, 3000 with a
// window of 512, which all take two, 60 and 75. Two parts everywhere would cost 30% (4096 tokens 222, 64 single
// tokens over up to 8192 95 -> 121).
//
// With x the product and c the scale in log2 units, p = 2^(x*c - b): one FMA and one
// exponential.  b is an integer, so that a raised b rescales O by an exact power
// of two; it is raised only when some product passes it by more than kLift, to
// kRoom below the largest, which keeps the weights that matter far inside fp16's range on
// both sides.  Beyond |b| = 2^22 the product is rounded before b is taken off: one FMA
// would leave the rounding error of the largest itself, more than the exponential's range.
#include <algorithm>

#include "kv.h"

namespace qg {
namespace {

constexpr float kLift = 15.0f, kRoom = 7.0f;  // probabilities reach 2^15, and 2^-14, the least normal fp16, is 2^-21 of the largest at least
constexpr float kHuge = 4194304.0f;
constexpr float kLog2e = 1.44269504f;

template <int D>
struct Words {
    typedef uint32_t W __attribute__((ext_vector_type(D / 32)));  // a lane's codes of 16 tokens
};

// Two codes of a word, exactly: or'ed into the low bits of 1024 (four bits up, of 64), where a step is
// one, and the 1024 taken off.
template <uint32_t MASK, uint32_t BIAS>
__device__ __forceinline__ f16x2 biased_codes(uint32_t w)
{
    uint32_t mask = MASK, bias = BIAS;
    asm("" : "+s"(mask));  // constants in registers, for one v_and_or_b32, which takes no literals
    asm("" : "+v"(bias));
    return __builtin_bit_cast(f16x2, (w & mask) | bias) - __builtin_bit_cast(f16x2, BIAS);
}

__device__ __forceinline__ f16x2 low_codes(uint32_t w) { return biased_codes<0x000F000Fu, 0x64006400u>(w); }
__device__ __forceinline__ f16x2 high_codes(uint32_t w) { return biased_codes<0x00F000F0u, 0x54005400u>(w); }

// code * scale + minimum, all fp16, with one rounding: a packed FMA. (v_fma_mix, which the GEMMs' products of a
// code and a binary32 factor need, takes two issue slots for each value.)
__device__ __forceinline__ uint32_t values(f16x2 code, f16x2 scale, f16x2 min)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(code, scale, min));
}

// A key's header, both fields twice.
struct KeyHead {
    f16x2 s, m;
};

__device__ __forceinline__ KeyHead key_head(uint32_t h)
{
    return KeyHead{__builtin_bit_cast(f16x2, __builtin_amdgcn_perm(h, h, 0x01000100u)),
                   __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(h, h, 0x03020302u))};
}

// Eight codes of one key -> eight fp16 values.
struct Codes {
    f16x2 c[4];
};

__device__ __forceinline__ Codes codes_of(uint32_t w)
{
    return Codes{{low_codes(w), high_codes(w), low_codes(w >> 8), high_codes(w >> 8)}};
}

__device__ __forceinline__ u32x4 key_values(const Codes &c, const KeyHead &k)
{
    return u32x4{values(c.c[0], k.s, k.m), values(c.c[1], k.s, k.m), values(c.c[2], k.s, k.m), values(c.c[3], k.s, k.m)};
}

// What key_values' roundings left off, rounded in turn.
__device__ __forceinline__ u32x4 key_rests(const Codes &c, const KeyHead &k, u32x4 v)
{
    const float s = (float)k.s.x, m = (float)k.m.x;
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t rounded = v[i];  // by value: of a vector's element, the cast would read the first
        const f16x2 h = __builtin_bit_cast(f16x2, rounded);
        r[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)__builtin_fmaf((float)h.x, -1.0f, __builtin_fmaf((float)c.c[i].x, s, m)),
                                                  (_Float16)__builtin_fmaf((float)h.y, -1.0f, __builtin_fmaf((float)c.c[i].y, s, m))});
    }
    return r;
}

// A quad's headers, tokens 0 and 1, then 2 and 3; word w of a lane, dims 2w and 2w+1 of its four
// tokens, as two dims of two fp16 pairs.
struct QuadHead {
    f16x2 s[2], m[2];
};

__device__ __forceinline__ QuadHead quad_head(u32x4 h)
{
    QuadHead q;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        q.s[i] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(h[2 * i + 1], h[2 * i], 0x05040100u));
        q.m[i] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(h[2 * i + 1], h[2 * i], 0x07060302u));
    }
    return q;
}

__device__ __forceinline__ u32x2 quad_values(uint32_t w, const QuadHead &q)
{
    return u32x2{values(low_codes(w), q.s[0], q.m[0]), values(high_codes(w), q.s[1], q.m[1])};
}

// Keys that a range of rows sees.
struct Range {
    int lo, hi;
};

// Headers of four tokens, the first of them `from` places behind the first of the `n` that some row of a tile sees:
// those that none does (behind the last row's place, or in front of the first one's window) are cleared.  Their
// probability is 0, what lies there need not have been written, and 0 times it could be NaN.
__device__ __forceinline__ u32x4 live_heads(u32x4 h, int from, int n)
{
#pragma unroll
    for (int i = 0; i < 4; i++) h[i] = (unsigned)(from + i) < (unsigned)n ? h[i] : 0u;
    return h;
}

// What the table says of place t of sequence s (t and s the same in all lanes: a
// scalar load, from the constant address space, since nothing writes tables
// here; behind the table's end, its last entry again).  Not looked at here, so
// that a load ahead of its use is not waited for.
__device__ __forceinline__ int entry_of(const KvView &v, int s, int t)
{
    typedef const int __attribute__((address_space(4))) *Scalars;
    return ((Scalars)(uintptr_t)v.tables)[(long long)s * v.width + min(t >> v.page_shift, v.width - 1)];
}

__device__ __forceinline__ bool names_page(const KvView &v, int entry, int t)
{
    return (unsigned)entry < (unsigned)v.pages && (t >> v.page_shift) < v.width;
}

// The tile at place t for key head h, in the page of that entry (in the first page
// where it names none: the address is inside the cache either way).
template <int D>
__device__ __forceinline__ const uint8_t *tile_at(const KvView &v, int entry, int t, int h)
{
    const int id = (unsigned)entry < (unsigned)v.pages ? entry : 0;
    const int in = (t & ((1 << v.page_shift) - 1)) >> 4, tiles = 1 << (v.page_shift - 4);
    return v.cache + (long long)id * v.page_bytes + (long long)(h * tiles + in) * KvLay<D>::kBytes;
}

// One query row as P pieces of eight dims, `step` dims from one to the next, in
// fp16; returns log2 units per unit of the products.  The row's lanes are ACROSS
// lanes apart (a multiple of it up to 64).
template <int DT, int P, int ACROSS>
__device__ __forceinline__ float load_query(const uint16_t *x, bool live, int step, float scale, u32x4 (&f)[P])
{
    const uint32_t sign = scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int j = 0; j < P; j++) {
        f[j] = live ? *(const u32x4 *)(x + j * step) : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; i++) f[j][i] ^= sign;
    }
    float c = fabsf(scale) * kLog2e;
    if constexpr (DT == DT_BF16) {
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < P; j++)
#pragma unroll
            for (int i = 0; i < 4; i++) mx = max(mx, max(f[j][i] & 0x7FFFu, (f[j][i] >> 16) & 0x7FFFu));
#pragma unroll
        for (int d = ACROSS; d < 64; d <<= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, d, 64));
        int e = (int)(mx >> 7);                       // the largest magnitude's exponent
        e = e == 0xFF || mx == 0 ? 127 + 8 : max(e, 27);  // infinities and NaN as they are
        const float down = __builtin_bit_cast(float, (uint32_t)(127 + 8 + 127 - e) << 23);
        c *= __builtin_bit_cast(float, (uint32_t)(max(e - 8, 1)) << 23);
#pragma unroll
        for (int j = 0; j < P; j++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                f[j][i] = pack_out<DT_F16>(of_bits<DT_BF16>(f[j][i] & 0xFFFFu) * down, of_bits<DT_BF16>(f[j][i] >> 16) * down);
    }
    return fminf(fmaxf(c, 1.17549435e-38f), 1e37f);  // never 0 or infinite: an exponent's argument is 0 at the maximum, -inf where masked
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// 2^(x*c - b), and the argument for a wave that holds rows of huge products (see above).
__device__ __forceinline__ float weight_of(float x, float c, float b) { return exp2_of(__builtin_fmaf(x, c, -b)); }

__device__ __forceinline__ float argument_of_huge(float x, float c, float b)
{
    float xc = x * c;
    asm("" : "+v"(xc));  // not one FMA
    return fabsf(b) > kHuge ? xc - b : __builtin_fmaf(x, c, -b);
}

// The b of a row whose largest product is mx: by the row alone, whatever made its
// wave look.  -inf until the row has seen a key.
__device__ __forceinline__ float raised(float mx, float b, float c)
{
    const float v = mx * c;
    return v - b > kLift ? ceilf(v) - kRoom : b;
}

// b as a subtrahend: a row that has seen nothing takes 0, and its products are -inf.
__device__ __forceinline__ float shift_of(float b) { return b == -INFINITY ? 0.0f : b; }
__device__ __forceinline__ float rescale_of(float before, float after) { return before == -INFINITY ? 0.0f : exp2_of(before - after); }

// Adds the two probabilities as the second product sees them, rounded.
__device__ __forceinline__ float add_pair(uint32_t pair, float l)
{
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, pair), f16x2{(_Float16)1.0f, (_Float16)1.0f}, l, false);
}

// The part, of `splits` parts of `chunk` keys (the last one open), that holds all the
// keys of a range, or -1: rows of one part need no join, whatever the splits.
__device__ __forceinline__ int only_part(Range keys, int splits, int chunk)
{
    if (keys.hi <= keys.lo) return 0;
    const int first = min(keys.lo / chunk, splits - 1);
    return first == min((keys.hi - 1) / chunk, splits - 1) ? first : -1;
}

// The place in front of the window of a row at `place`; rows without a place, whose places are negative, count as at 0,
// so that no window takes it out of an int's range.
__device__ __forceinline__ int before_window(int place, int window) { return max(place, 0) - window; }

__device__ __forceinline__ Range seen(const AttnArgs &a, const Seq &q, int row0, int rows)
{
    const int cap = a.v.width << a.v.page_shift;
    const int pmin = q.first + row0 / a.group, pmax = q.first + (row0 + rows - 1) / a.group;
    return Range{a.window ? max(before_window(pmin, a.window) + 1, 0) : 0, min(pmax + 1, cap)};
}

// Whether some row of a tile sees at most kFewKeys keys, and the tile takes them in two parts.  With a row's place the number
// of its keys rises, stays (at the window) and falls (behind the table), so that it is least for the first row or the last.
constexpr int kFewKeys = 512;
template <int DT>
__device__ __forceinline__ bool few_keys(const AttnArgs &a, const Seq &q, int row0, int rows)
{
    if (DT != DT_F16) return false;
    const Range first = seen(a, q, row0, 1), last = seen(a, q, row0 + rows - 1, 1);
    return min(first.hi - first.lo, last.hi - last.lo) <= kFewKeys;
}

// Zeros to the rows of no sequence, in front of the first one and behind the last, by workgroups behind those of a launch
// that no join follows: beside the others' work, which they do not touch (658 tokens 23.6 us with and without them, 4096
// 159).  The join comes by every row anyway; workgroups behind those of a launch in parts, which are as many as the CUs hold,
// took 64 tokens behind 8000 from 49.9 us to 52.2.
__device__ __forceinline__ void zero_rest(const AttnArgs &a, int D)
{
    const long long per = (long long)a.heads * D / 8;  // pieces of 16 bytes in a row
    const long long front = row_end(a.v, 0) * per, back = row_end(a.v, a.v.S) * per, n = front + a.v.T * per - back;
    const long long step = (long long)a.rest_blocks * blockDim.x;
    for (long long i = (long long)(blockIdx.x - a.work_blocks) * blockDim.x + threadIdx.x; i < n; i += step)
        ((u32x4 *)a.y)[i < front ? i : i - front + back] = u32x4{0, 0, 0, 0};
}

// ---------------------------------------------------------------------------
// A few rows of each sequence (single tokens): a stream of the cache.  A
// workgroup takes one key head of one sequence, 16*RB rows and a chunk of the
// keys; its four or eight waves take steps of 32 keys in turn, straight from memory into
// MFMA registers, and add their results through LDS.
//
// Bound by the cache's bytes where it is long: 64 sequences of up to 8192 tokens,
// 432 MB of codes and headers, take 94 us with the join, 4.6 TB/s, where four instructions for two codes
// (and the arithmetic beside them) still fill half of the time.  The 16x16x32
// product leaves the fewest rows idle; 64 keys in flight a wave (two steps' registers in turn)
// and three workgroups a CU cover the loads: a third step in flight gained nothing, a fourth workgroup would
// spill (149 us).  Short ones are a
// chain of dependent loads (lengths, table, cache), a merge and a second launch to
// join: one sequence of 658 tokens 8.3 us, of 500 in one part 7.2 us.
// ---------------------------------------------------------------------------
constexpr int kStep = 32;

template <int D>
struct FewRaw {
    typename Words<D>::W k[2], v[2];
    uint32_t kh[2];
    u32x4 vh[2];
    int entry[2];
};

__device__ __forceinline__ void few_entries(const AttnArgs &a, int s, int t, int (&entry)[2])
{
#pragma unroll
    for (int i = 0; i < 2; i++) entry[i] = entry_of(a.v, s, t + 16 * i);
}

template <int D>
__device__ __forceinline__ void few_load(const AttnArgs &a, const int (&entry)[2], int h, int t, int lane, FewRaw<D> &r)
{
    using L = KvLay<D>;
    using W = typename Words<D>::W;
    const int n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        r.entry[i] = entry[i];
        const uint8_t *p = tile_at<D>(a.v, entry[i], t + 16 * i, h);
        r.k[i] = *(const W *)(p + lane * L::kLane);
        r.kh[i] = *(const uint32_t *)(p + L::kKeyHead + (g * (D / 4) / 32 * 16 + n) * 4);
        r.v[i] = *(const W *)(p + L::kVal + lane * L::kLane);
        r.vh[i] = *(const u32x4 *)(p + L::kValHead + (n * L::E / 32 * 16 + 4 * g) * 4);
    }
}

template <int DT, int D, int RB, int NW>
__global__ void __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW == 8 || RB == 2 ? 2 : D == 64 ? 4 : 3))) k_attn_few(AttnArgs a)
{
    using L = KvLay<D>;
    constexpr int E = L::E, J = D / 32, LD = D + 4;
    __shared__ __align__(16) float s_o[NW][16][LD];
    __shared__ float s_b[NW][16], s_l[NW][16];
    if ((int)blockIdx.x >= a.work_blocks) return zero_rest(a, D);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    // second blocks of rows last: those of a ragged batch mostly end at once, and spread over all XCDs
    const int pairs = a.v.S * a.v.H, rt = (int)blockIdx.x / pairs, sh = (int)blockIdx.x - rt * pairs, h = sh % a.v.H, s = sh / a.v.H, z = blockIdx.y;
    const Seq q = seq_of(a.v, s);
    const int all = q.n * a.group, row0 = rt * 16 * RB;
    if ((a.v.offs && all > a.few_rows) || row0 >= all) return;
    const int rows = min(all - row0, 16 * RB);
    const Range keys = seen(a, q, row0, rows);
    const bool rests = few_keys<DT>(a, q, row0, rows);
    const int only = only_part(keys, a.few_splits, a.few_chunk);
    if (only >= 0 && only != z) return;
    const int from = max(keys.lo & ~(kStep - 1), z * a.few_chunk), to = z + 1 < a.few_splits ? min(keys.hi, (z + 1) * a.few_chunk) : keys.hi;

    const int stride = kStep * NW, window = a.window ? a.window : INT_MAX;
    const int pmin = q.first + row0 / a.group, pmax_lo = a.window ? before_window(q.first + (row0 + rows - 1) / a.group, a.window) + 1 : 0;
    int t = from + wave * kStep, ahead[2];
    FewRaw<D> even, odd;  // this step's bytes and the next one's
    bool huge = false;
    if (t < to) {
        few_entries(a, s, t, ahead);
        few_load<D>(a, ahead, h, t, lane, even);
        few_entries(a, s, t + stride, ahead);
    }
    u32x4 qf[RB][J];
    float c[RB], b[RB], l[RB];
    int place[RB], low[RB];  // a row sees the places above low, up to its own
    f32x4 o[RB][E];
#pragma unroll
    for (int rb = 0; rb < RB; rb++) {
        const int r = row0 + 16 * rb + n, token = r / a.group;
        const bool live = r < all;
        place[rb] = live ? q.first + token : -1;
        low[rb] = before_window(place[rb], window);
        c[rb] = load_query<DT, J, 16>(a.q + (long long)(q.row + (live ? token : 0)) * a.q_stride +
                                          (h * a.group + r - token * a.group) * D + g * (D / 4),
                                      live, 8, a.scale, qf[rb]);
        b[rb] = -INFINITY;
        l[rb] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e++) o[rb][e] = f32x4{0, 0, 0, 0};
    }

    auto turn = [&](int t, FewRaw<D> &r, FewRaw<D> &next) {
        if (t + stride < to) {
            few_load<D>(a, ahead, h, t + stride, lane, next);
            few_entries(a, s, t + 2 * stride, ahead);
        }
        f32x4 x[RB][2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const KeyHead head = key_head(r.kh[i]);
#pragma unroll
            for (int rb = 0; rb < RB; rb++) x[rb][i] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < J; j++) {
                const Codes codes = codes_of(r.k[i][j]);
                const u32x4 kv = key_values(codes, head);
#pragma unroll
                for (int rb = 0; rb < RB; rb++) x[rb][i] = mma<DT_F16>(kv, qf[rb][j], x[rb][i]);
                if (!rests) continue;
                const u32x4 kr = key_rests(codes, head, kv);
#pragma unroll
                for (int rb = 0; rb < RB; rb++) x[rb][i] = mma<DT_F16>(kr, qf[rb][j], x[rb][i]);
            }
        }
        const bool there[2] = {names_page(a.v, r.entry[0], t), names_page(a.v, r.entry[1], t + 16)}, whole = there[0] && there[1];
        if (!(whole && t + kStep - 1 <= pmin && t >= pmax_lo)) {
#pragma unroll
            for (int rb = 0; rb < RB; rb++)
#pragma unroll
                for (int i = 0; i < 2; i++)
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const int at = t + 16 * i + 4 * g + u;
                        const bool ok = there[i] & (at <= place[rb]) & (at > low[rb]);
                        x[rb][i][u] = ok ? x[rb][i][u] : -INFINITY;
                    }
        }
        if (!(whole && t >= keys.lo && t + kStep <= keys.hi)) {
#pragma unroll
            for (int i = 0; i < 2; i++) r.vh[i] = live_heads(r.vh[i], t + 16 * i - keys.lo + 4 * g, there[i] ? keys.hi - keys.lo : 0);
        }
        u32x4 p[RB];
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            float mx = fmaxf(fmaxf(fmaxf(x[rb][0][0], x[rb][0][1]), fmaxf(x[rb][0][2], x[rb][0][3])),
                             fmaxf(fmaxf(x[rb][1][0], x[rb][1][1]), fmaxf(x[rb][1][2], x[rb][1][3])));
            if (__any(mx * c[rb] - b[rb] > kLift)) {
                mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                const float nb = raised(mx, b[rb], c[rb]), f = rescale_of(b[rb], nb);
                b[rb] = nb;
                huge = huge || __any(fabsf(nb) > kHuge && nb != -INFINITY);
                l[rb] *= f;
#pragma unroll
                for (int e = 0; e < E; e++) o[rb][e] *= f;
            }
            const float base = shift_of(b[rb]);
            float w[8];
            if (huge) {
#pragma unroll
                for (int u = 0; u < 8; u++) w[u] = exp2_of(argument_of_huge(x[rb][u >> 2][u & 3], c[rb], base));
            } else {
#pragma unroll
                for (int u = 0; u < 8; u++) w[u] = weight_of(x[rb][u >> 2][u & 3], c[rb], base);
            }
#pragma unroll
            for (int u = 0; u < 4; u++) {
                p[rb][u] = pack_out<DT_F16>(w[2 * u], w[2 * u + 1]);
                l[rb] = add_pair(p[rb][u], l[rb]);
            }
        }
        const QuadHead h0 = quad_head(r.vh[0]), h1 = quad_head(r.vh[1]);
#pragma unroll
        for (int e = 0; e < E; e++) {
            const u32x2 v0 = quad_values(r.v[0][e >> 1] >> (8 * (e & 1)), h0);
            const u32x2 v1 = quad_values(r.v[1][e >> 1] >> (8 * (e & 1)), h1);
            const u32x4 v = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
            for (int rb = 0; rb < RB; rb++) o[rb][e] = mma<DT_F16>(v, p[rb], o[rb][e]);
        }
    };
    for (; t < to; t += 2 * stride) {
        turn(t, even, odd);
        if (t + stride < to) turn(t + stride, odd, even);
    }

#pragma unroll
    for (int rb = 0; rb < RB; rb++) {
        if (RB > 1 && 16 * rb >= rows) break;
        l[rb] += __shfl_xor(l[rb], 16, 64);
        l[rb] += __shfl_xor(l[rb], 32, 64);
        if (rb) __syncthreads();
        // lane: row n, dims E*(4g + i) + e
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < E; e += 4)
                *(f32x4 *)&s_o[wave][n][E * (4 * g + i) + e] =
                    f32x4{o[rb][e][i], o[rb][e + 1][i], o[rb][e + 2][i], o[rb][e + 3][i]};
        if (g == 0) {
            s_b[wave][n] = b[rb];
            s_l[wave][n] = l[rb];
        }
        __syncthreads();
        const int rr = threadIdx.x >> 4, dl = threadIdx.x & 15, r = 16 * rb + rr;
        if (rr >= 16 || r >= rows) continue;
        float top = s_b[0][rr], sum = 0.0f, y[E];
#pragma unroll
        for (int w = 1; w < NW; w++) top = fmaxf(top, s_b[w][rr]);
#pragma unroll
        for (int e = 0; e < E; e++) y[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const float f = rescale_of(s_b[w][rr], top);
            sum += s_l[w][rr] * f;
#pragma unroll
            for (int e = 0; e < E; e++) y[e] += s_o[w][rr][E * dl + e] * f;
        }
        const int ra = row0 + r, token = ra / a.group;
        if (only >= 0) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int e = 0; e < E; e++) y[e] *= inv;
            store_out<DT, E>(a.y, ((long long)(q.row + token) * a.heads + h * a.group + ra - token * a.group) * D + E * dl, y);
        } else {
            const long long entry = ((long long)(s * a.v.H + h) * a.few_rows + ra) * a.few_splits + z;
            if (sum != 0.0f) store_out<QGEMM_F32, E>(a.few_sum, entry * D + E * dl, y);
            if (dl == 0) a.few_stat[entry] = f32x2{top, sum};
        }
    }
}

// ---------------------------------------------------------------------------
// Many rows (prompts): a workgroup takes one key head and 32 rows per wave,
// row r being token r/group, head r%group of the key head's; tiles of 64 keys are
// unpacked once into LDS, in fragment order, for all its waves.
//
// Bound by the exponentials and the unpacking beside the products, and by the power
// limit: 4096 tokens of 32 query heads of 128 (137 GFLOP under the mask) take 156 to 163 us, 0.84 to 0.88
// PFLOP/s, where the matrix units alone, on random operands, sustain 1.35.  The 32x32x16
// product reads the fewest LDS bytes a flop; a 64-key tile takes a CU's 8 waves 4160 cycles,
// half of them products.  Eight waves share a tile's unpacking (179 us with four) where that
// still fills the CUs; short prompts are a chain of one tile after the other (658 tokens
// of fp16 23.7 us), which two waves to 32 rows shorten.
// ---------------------------------------------------------------------------
constexpr int kKeys = 64;

// A wave's share of a tile's raw bytes: N words a lane of 16 tokens' keys and values,
// all of them where four waves share a tile, half where eight do.
template <int D, int PARTS>
struct ManyRaw {
    static constexpr int N = D / 32 / PARTS;
    typedef uint32_t W __attribute__((ext_vector_type(N)));
    W k, v;
    uint32_t kh;
    u32x4 vh;
    int entry;  // of the table
};

template <int D, int PARTS>
__device__ __forceinline__ void many_load(const AttnArgs &a, int entry, int h, int at, int part, int lane, ManyRaw<D, PARTS> &r)
{
    using L = KvLay<D>;
    using W = typename ManyRaw<D, PARTS>::W;
    const int n = lane & 15, g = lane >> 4;
    const uint8_t *p = tile_at<D>(a.v, entry, at, h);
    const int mine = lane * L::kLane + part * (L::kLane / PARTS);
    r.entry = entry;
    r.k = *(const W *)(p + mine);
    r.v = *(const W *)(p + L::kVal + mine);
    r.kh = *(const uint32_t *)(p + L::kKeyHead + (g * (D / 4) / 32 * 16 + n) * 4);
    r.vh = *(const u32x4 *)(p + L::kValHead + (n * L::E / 32 * 16 + 4 * g) * 4);
}

// LDS of a tile: keys as [32-key half][8-dim piece][key] of 16 bytes; values as
// [16 tokens][32-dim block][quad parity][dim row] of 16 bytes, two quads of four
// tokens.  Row d of block b is dim E*(d%16) + 2b + d/16: a wave's stores are then
// contiguous, and a lane ends with E neighbouring dims.
template <int D>
struct ManyTile {
    uint4 k[2][D / 8][32];
    uint2 v[4][D / 32][2][32][2];
};

// i: which 16 tokens of the tile, from place `at` behind the first of the n_seen keys that the row tile sees (0 where the
// table names no page); rests: where the keys' second parts go, or null.
template <int D, int PARTS>
__device__ __forceinline__ void many_store(ManyTile<D> &t, ManyTile<D> *rests, const ManyRaw<D, PARTS> &r, int i, int part, int at, int n_seen, int lane)
{
    constexpr int N = ManyRaw<D, PARTS>::N;
    const int n = lane & 15, g = lane >> 4;
    const KeyHead head = key_head(r.kh);
#pragma unroll
    for (int j = 0; j < N; j++) {
        const Codes codes = codes_of(r.k[j]);
        const u32x4 v = key_values(codes, head);
        *(u32x4 *)&t.k[i >> 1][(D / 32) * g + N * part + j][16 * (i & 1) + n] = v;
        if (rests) *(u32x4 *)&rests->k[i >> 1][(D / 32) * g + N * part + j][16 * (i & 1) + n] = key_rests(codes, head, v);
    }
    const QuadHead q = quad_head(live_heads(r.vh, at + 4 * g, n_seen));
#pragma unroll
    for (int j = 0; j < N; j++)
#pragma unroll
        for (int e = 0; e < 2; e++)
            *(u32x2 *)&t.v[i][N * part + j][g & 1][n + 16 * e][g >> 1] = quad_values(r.v[j] >> (8 * e), q);
}

// While a tile is multiplied, the next one is unpacked into the other LDS buffer
// and the two after it are on their way from memory; one barrier per tile (two where the
// keys have second parts).
// KS = 2: two waves share 32 rows, each with half of every tile's keys, and are joined at the end.
template <int DT, int D, int NW, int KS>
__global__ void __launch_bounds__(64 * NW * KS) __attribute__((amdgpu_waves_per_eu(2, 2))) k_attn_many(AttnArgs a)
{
    constexpr int E = D / 16, B = D / 32, P = D / 16, PARTS = NW * KS / 4, HALVES = 2 / KS;
    __shared__ __align__(16) ManyTile<D> s_tile[2];
    if ((int)blockIdx.x >= a.work_blocks) return zero_rest(a, D);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = KS == 2 ? wave / NW : 0;  // the first of the tile's halves of 32 keys that it takes
    const int n = lane & 31, g = lane >> 5;
    // key heads side by side, so that with a multiple of eight of them each XCD's
    // L2 holds its own; later row tiles, which see more keys, first
    const int h = blockIdx.x % a.v.H, slot = a.slots - 1 - (int)(blockIdx.x / a.v.H), z = blockIdx.y;
    const int s = __builtin_amdgcn_readfirstlane(find_seq<64>(a.v, slot, a.tile_tokens, 1));
    const Seq q = seq_of(a.v, s);
    const int all = q.n * a.group;
    const int tile = slot - (row_end(a.v, s) / a.tile_tokens + s), row0 = tile * a.tile_tokens * a.group;
    if (tile < 0 || row0 >= all || all <= a.few_rows) return;
    const int rows = min(all - row0, a.tile_tokens * a.group);
    const Range keys = seen(a, q, row0, rows);
    const bool rests = few_keys<DT>(a, q, row0, rows);  // then one tile at a time, its second parts in the other's place
    const int only = only_part(keys, a.many_splits, a.many_chunk);
    if (only >= 0 && only != z) return;
    const int from = max(keys.lo, z * a.many_chunk), to = z + 1 < a.many_splits ? min(keys.hi, (z + 1) * a.many_chunk) : keys.hi;
    const int kt0 = from / kKeys, kt1 = to > from ? (to + kKeys - 1) / kKeys : kt0;

    const int w0 = 32 * (wave % NW), r = row0 + w0 + n, token = r / a.group;
    const bool live = w0 + n < rows;
    const int place = live ? q.first + token : -1, low = before_window(place, a.window ? a.window : INT_MAX);
    // tiles in which some row of the wave sees a key, and keys that all its rows see
    const Range mine = w0 < rows ? seen(a, q, row0 + w0, min(rows - w0, 32)) : Range{0, 0};
    const int mt0 = mine.lo / kKeys, mt1 = (mine.hi + kKeys - 1) / kKeys;
    // places from `cap` on lie behind the table, also those of a last tile that it ends inside of (capacities that are
    // no multiple of 64), whatever the length
    const int cap = a.v.width << a.v.page_shift, last = min(place, cap - 1);
    const int clear_hi = min(q.first + (row0 + w0) / a.group, cap - 1);
    const int clear_lo = a.window ? before_window(q.first + (row0 + min(rows, w0 + 32) - 1) / a.group, a.window) + 1 : 0;

    // this wave's 16 tokens of a tile; past the last tile, of the last once more
    auto place_in = [&](int kt) { return min(kt, kt1 - 1) * kKeys + 16 * (wave & 3); };
    auto load = [&](int kt, int entry, ManyRaw<D, PARTS> &to_raw) {
        many_load<D, PARTS>(a, entry, h, place_in(kt), wave >> 2, lane, to_raw);
    };
    auto store = [&](int kt, const ManyRaw<D, PARTS> &of_raw) {
        many_store<D, PARTS>(s_tile[rests ? 0 : (kt - kt0) & 1], rests ? &s_tile[1] : nullptr, of_raw, wave & 3, wave >> 2,
                             place_in(kt) - keys.lo, names_page(a.v, of_raw.entry, place_in(kt)) ? keys.hi - keys.lo : 0, lane);
    };
    ManyRaw<D, PARTS> raw, later;  // the next tile's bytes, and those of the one after it
    int ahead = 0;                 // the table's entry for the one after that
    auto next = [&](int kt) {
        store(kt + 1, raw);
        raw = later;
        load(kt + 3, ahead, later);
        ahead = entry_of(a.v, s, place_in(kt + 4));
    };
    // The next tile is unpacked between this one's products, beside the first ones, by waves that have the keys to
    // themselves (2048 tokens behind 6000 282 -> 276 us); by those that halve them, after (658 tokens of 64 dims 16.1, else
    // 16.9).
    const bool early = KS == 1 && !rests;
    u32x4 qf[P];
    float c = 0.0f, b = -INFINITY, l = 0.0f;
    bool gaps = false, huge = false;  // gaps: pages that the table does not name, looked for once
    f32x16 o[B];
#pragma unroll
    for (int d = 0; d < B; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) o[d][i] = 0.0f;
    if (kt0 < kt1) {  // everything that the first products wait for at once
        const int e0 = entry_of(a.v, s, place_in(kt0)), e1 = entry_of(a.v, s, place_in(kt0 + 1)), e2 = entry_of(a.v, s, place_in(kt0 + 2));
        ahead = entry_of(a.v, s, place_in(kt0 + 3));
        ManyRaw<D, PARTS> first;
        load(kt0, e0, first);
        c = load_query<DT, P, 32>(a.q + (long long)(q.row + (live ? token : 0)) * a.q_stride +
                                      (h * a.group + r - token * a.group) * D + 8 * g,
                                  live, 16, a.scale, qf);
        for (int i = (kt0 * kKeys >> a.v.page_shift) + lane; i <= (to - 1) >> a.v.page_shift; i += 64)
            gaps |= (unsigned)a.v.tables[(long long)s * a.v.width + i] >= (unsigned)a.v.pages;
        load(kt0 + 1, e1, raw);
        load(kt0 + 2, e2, later);
        store(kt0, first);
        gaps = __any(gaps);
    }
    for (int kt = kt0; kt < kt1; kt++) {
        __syncthreads();  // this tile is whole, and the other buffer's readers are done
        const int k0 = kt * kKeys;
        const ManyTile<D> &t = s_tile[rests ? 0 : (kt - kt0) & 1];
        if (kt >= mt0 && kt < mt1) {
            f32x16 x[HALVES];
#pragma unroll
            for (int i = 0; i < HALVES; i++) {
#pragma unroll
                for (int j = 0; j < 16; j++) x[i][j] = 0.0f;
#pragma unroll
                for (int p = 0; p < P; p++) x[i] = mma32<DT_F16>(*(const u32x4 *)&t.k[half + i][2 * p + g][n], qf[p], x[i]);
                if (!rests) continue;
#pragma unroll
                for (int p = 0; p < P; p++) x[i] = mma32<DT_F16>(*(const u32x4 *)&s_tile[1].k[half + i][2 * p + g][n], qf[p], x[i]);
            }
            if (early) next(kt);
            if (gaps || k0 + kKeys - 1 > clear_hi || k0 < clear_lo) {
#pragma unroll
                for (int u = 0; u < 2 * HALVES; u++) {
                    const int k = k0 + 32 * half + 16 * u;
                    const bool there = !gaps || names_page(a.v, entry_of(a.v, s, k), k);
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const int at = k + 8 * (i >> 2) + 4 * g + (i & 3);
                        const bool ok = there & (at <= last) & (at > low);
                        x[u >> 1][8 * (u & 1) + i] = ok ? x[u >> 1][8 * (u & 1) + i] : -INFINITY;
                    }
                }
            }
            float mx = x[0][0];
#pragma unroll
            for (int i = 0; i < 16; i++) mx = fmaxf(fmaxf(mx, x[0][i]), x[HALVES - 1][i]);
            if (__any(mx * c - b > kLift)) {
                const float nb = raised(fmaxf(mx, __shfl_xor(mx, 32, 64)), b, c), f = rescale_of(b, nb);
                b = nb;
                huge = huge || __any(fabsf(nb) > kHuge && nb != -INFINITY);
                l *= f;
#pragma unroll
                for (int d = 0; d < B; d++) o[d] *= f;
            }
            const float base = shift_of(b);
            if (huge) {  // the arguments as they are to be: what follows then adds and multiplies nothing
#pragma unroll
                for (int u = 0; u < HALVES; u++)
#pragma unroll
                    for (int i = 0; i < 16; i++) x[u][i] = argument_of_huge(x[u][i], c, base);
            }
            const float cc = huge ? 1.0f : c, bb = huge ? 0.0f : base;
#pragma unroll
            for (int u = 0; u < 2 * HALVES; u++) {  // 16 tokens: registers 8*(u%2) .. +7 of half u/2
                u32x4 p;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int k = 8 * (u & 1) + 2 * i;
                    p[i] = pack_out<DT_F16>(weight_of(x[u >> 1][k], cc, bb), weight_of(x[u >> 1][k + 1], cc, bb));
                    l = add_pair(p[i], l);
                }
#pragma unroll
                for (int d = 0; d < B; d++) o[d] = mma32<DT_F16>(*(const u32x4 *)&t.v[2 * half + u][d][g][n][0], p, o[d]);
            }
        }
        if (!early || !(kt >= mt0 && kt < mt1)) {
            if (rests) __syncthreads();  // all have read this one
            next(kt);
        }
    }
    l += __shfl_xor(l, 32, 64);
    if constexpr (KS == 2) {  // through the LDS of the tiles
        __shared__ f32x2 s_stat[NW][64];
        static_assert(sizeof(s_tile) == sizeof(float) * NW * B * 16 * 64, "the tiles' LDS holds half of the waves' sums");
        float *sums = (float *)s_tile + (wave % NW) * B * 16 * 64 + lane;
        __syncthreads();
        if (half == 1) {
#pragma unroll
            for (int d = 0; d < B; d++)
#pragma unroll
                for (int i = 0; i < 16; i++) sums[(d * 16 + i) * 64] = o[d][i];
            s_stat[wave % NW][lane] = f32x2{b, l};
        }
        __syncthreads();
        if (half == 1) return;
        const f32x2 st = s_stat[wave][lane];
        const float top = fmaxf(b, st.x), f = l == 0.0f ? 0.0f : rescale_of(b, top), f1 = st.y == 0.0f ? 0.0f : rescale_of(st.x, top);
        b = top;
        l = l * f + st.y * f1;
#pragma unroll
        for (int d = 0; d < B; d++)
#pragma unroll
            for (int i = 0; i < 16; i++) o[d][i] = o[d][i] * f + sums[(d * 16 + i) * 64] * f1;
    }
    if (!live) return;
    const long long row = (long long)(q.row + token) * a.heads + h * a.group + r - token * a.group;
    const long long part = row * a.many_splits + z;
    const float inv = only < 0 ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float v[E];
#pragma unroll
        for (int d = 0; d < B; d++) {
            v[2 * d] = o[d][i] * inv;
            v[2 * d + 1] = o[d][i + 8] * inv;
        }
        const int d = E * (8 * (i >> 2) + 4 * g + (i & 3));
        if (only >= 0) store_out<DT, E>(a.y, row * D + d, v);
        else if (l != 0.0f) store_out<QGEMM_F32, E>(a.many_sum, part * D + d, v);
    }
    if (only < 0 && g == 0) a.many_stat[part] = f32x2{b, l};
}

// The parts of a row's keys joined, a row and query head at a time by G groups of
// 16 lanes: group i takes every G-th part, and the groups' results meet in LDS.  Its time is a
// launch and a chain of loads (4.3 us for one token in six parts, 4.9 for 64 in two) until rows
// are many (1100 rows of 32 heads in three parts: 16 us, 3.4 TB/s).
template <int DT, int D, int G>
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs a)
{
    constexpr int E = D / 16;
    __shared__ __align__(16) float s_y[G > 1 ? G : 1][D + 4];
    const int item = (int)(blockIdx.x * (16 / G) + (threadIdx.x >> 4) / G), dl = threadIdx.x & 15, gi = (threadIdx.x >> 4) % G;
    const int row = item / a.heads, head = item - row * a.heads;
    if (row >= a.v.T) return;
    const int s = a.v.offs ? find_seq<16>(a.v, row, 1, 0) : row;
    const Seq q = seq_of(a.v, s);
    if (row < q.row || row >= q.row + q.n) {
        const float zeros[E] = {};
        if (a.zero_rest && gi == 0) store_out<DT, E>(a.y, ((long long)row * a.heads + head) * D + E * dl, zeros);
        return;
    }
    const bool few = !a.v.offs || q.n * a.group <= a.few_rows;
    const int splits = few ? a.few_splits : a.many_splits, chunk = few ? a.few_chunk : a.many_chunk;
    const int h = head / a.group, ra = (row - q.row) * a.group + head - h * a.group;
    // the row tile it was computed in: rows of one part are written already
    const int tile_rows = few ? a.few_tile_rows : a.tile_tokens * a.group, row0 = ra / tile_rows * tile_rows;
    const Range keys = seen(a, q, row0, min(q.n * a.group - row0, tile_rows));
    if (only_part(keys, splits, chunk) >= 0) return;
    const int z0 = min(keys.lo / chunk, splits - 1), z1 = min((keys.hi - 1) / chunk, splits - 1);
    const long long entry = few ? ((long long)(s * a.v.H + h) * a.few_rows + ra) * splits
                                : ((long long)row * a.heads + head) * splits;
    const f32x2 *stat = (few ? a.few_stat : a.many_stat) + entry;
    const float *sums = (few ? a.few_sum : a.many_sum) + entry * D + E * dl;
    float top = -INFINITY;
    for (int z = z0 + dl; z <= z1; z += 16) top = fmaxf(top, stat[z].x);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 16));
    float y[E], sum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; e++) y[e] = 0.0f;
    for (int z = z0 + gi; z <= z1; z += G) {
        const f32x2 st = stat[z];
        if (st.y == 0.0f) continue;  // it saw no key, and wrote no sums
        const float f = rescale_of(st.x, top);
        sum += st.y * f;
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const f32x4 v = *(const f32x4 *)(sums + (long long)z * D + e);
#pragma unroll
            for (int i = 0; i < 4; i++) y[e + i] += v[i] * f;
        }
    }
    if constexpr (G > 1) {
        static_assert(G == 16, "one row and head to a workgroup");
#pragma unroll
        for (int e = 0; e < E; e++) s_y[gi][E * dl + e] = y[e];
        if (dl == 0) s_y[gi][D] = sum;
        __syncthreads();
        if (gi) return;
        sum = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e++) y[e] = 0.0f;
        for (int i = 0; i < G; i++) {
            sum += s_y[i][D];
#pragma unroll
            for (int e = 0; e < E; e++) y[e] += s_y[i][E * dl + e];
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < E; e++) y[e] *= inv;
    store_out<DT, E>(a.y, ((long long)row * a.heads + head) * D + E * dl, y);
}

long long ceil_of(long long a, long long b) { return (a + b - 1) / b; }

template <int DT, int D, int RB, int NW>
void run_few(AttnArgs a, hipStream_t s)
{
    a.work_blocks = a.v.S * a.v.H * a.few_tiles;
    hipLaunchKernelGGL((k_attn_few<DT, D, RB, NW>), dim3((unsigned)(a.work_blocks + a.rest_blocks), (unsigned)a.few_splits),
                       dim3(64 * NW), 0, s, a);
}

template <int DT, int D, int NW, int KS>
hipError_t run_many(AttnArgs a, hipStream_t s)
{
    a.work_blocks = a.slots * a.v.H;
    hipLaunchKernelGGL((k_attn_many<DT, D, NW, KS>), dim3((unsigned)(a.work_blocks + a.rest_blocks), (unsigned)a.many_splits), dim3(64 * NW * KS), 0, s, a);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t run_attention(const AttnPlan &pl, AttnArgs a, hipStream_t s)
{
    const int splits = pl.few && pl.few_splits > 1 ? pl.few_splits : pl.many ? pl.many_splits : 1;
    // a workgroup for every 32 KB of results, up to one to a CU
    const int rest = !a.zero_rest || splits > 1 ? 0 : (int)std::min(ceil_of((long long)a.v.T * a.heads * D, 16384), 256LL);
    if (pl.few) {
        a.rest_blocks = pl.many ? 0 : rest;
        if (pl.few_rb == 2) run_few<DT, D, 2, 4>(a, s);
        else if (pl.few_waves == 8) run_few<DT, D, 1, 8>(a, s);
        else run_few<DT, D, 1, 4>(a, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (pl.many) {
        a.rest_blocks = rest;
        const hipError_t e = pl.many_waves == 8 ? run_many<DT, D, 8, 1>(a, s)
                             : pl.many_halves ? run_many<DT, D, 4, 2>(a, s)
                                              : run_many<DT, D, 4, 1>(a, s);
        if (e != hipSuccess) return e;
    }
    if (splits > 1) {
        const long long items = (long long)a.v.T * a.heads;
        // a workgroup to a row and head where 16 lanes would walk through many parts and there are few of
        // them: one token over 8192 in 64 parts 42 us by 16 lanes, 14 by 256
        if (splits > 4 && items <= 4096) hipLaunchKernelGGL((k_attn_join<DT, D, 16>), dim3((unsigned)items), dim3(256), 0, s, a);
        else hipLaunchKernelGGL((k_attn_join<DT, D, 1>), dim3((unsigned)ceil_of(items, 16)), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

AttnPlan plan_attention(long long T, long long S, int heads, int kv_heads, int D, long long max_len, bool ragged)
{
    AttnPlan p{};
    const int group = heads / kv_heads;
    // ragged: k_attn_few takes the sequences of at most 32 rows, if there can be any beside one long one
    p.few = !ragged || S > 1 || T * group <= 32;
    p.many = ragged && T * group > 32;
    p.few_rows = !p.few ? 0 : ragged ? 32 : group;
    // Blocks of 16 rows that share the unpacked keys and values: two where rows, evenly shared out, would need them. A
    // ragged batch of single tokens (or of those and prompts) takes one, and a second workgroup for what has more: 64
    // single tokens over up to 1000 24.8 us against 30.4, 64 sequences of 3 over up to 4000 54 against 68; 5 and 8 of each are the same.
    const bool two = ragged ? T * group > 16 * S && T * group <= 32 * S : p.few_rows > 16;
    p.few_rb = two ? 2 : 1;
    p.few_tiles = (int)ceil_of(p.few_rows > 0 ? p.few_rows : 1, 16 * p.few_rb);
    if (max_len < 1) max_len = 1;
    // chunks of whole steps for every wave; as many workgroups as the CUs hold at once: three or four
    const long long step = kStep * 4, units = S * kv_heads * (ragged ? 1 : p.few_tiles);
    long long chunk = ceil_of(ceil_of(units * max_len, D == 64 ? 1024 : 768), step) * step;
    // One part where a second launch costs more than it gains.  Of eight waves up to 1024 keys, while a workgroup (or, with
    // heads of 64, two) to a CU holds them: always up to 512 (768), above where parts would be more workgroups than
    // CUs.  In us, 32 query and 8 key heads of 128, parts and one part: one sequence of 500 9.4 and 7.2, of 658 8.4 and
    // 8.6, 8 of 658 9.7 and 7.6, 16 of 1000 12.3 and 10.3, 4 of 1000 8.7 and 10.0, 64 of 1000 20.1 and 20.5.  Of four
    // waves up to 384 keys else: one of 200 5.6 (eight waves 6.0), 128 of 300 15.7 (21.8).
    const bool one = p.few_rb == 1 && max_len > 256 && max_len <= 1024 && units <= (D == 64 ? 512 : 256) &&
                     (max_len <= (D == 64 ? 768 : 512) || units * ceil_of(max_len, step) > 256);
    p.few_waves = one ? 8 : 4;
    // Parts of 128 up to 4096 keys (one sequence of 2000: 8.6, and 9.7 in parts of 256) and of 256 at least from
    // there on (of 8192: 13.5 and 11.5).
    const long long least_few = one ? 1024 : max_len <= 384 ? 384 : max_len <= 4096 ? step : 256;
    if (chunk < least_few) chunk = least_few;
    if (ceil_of(max_len, chunk) > 128) chunk = ceil_of(ceil_of(max_len, 128), step) * step;  // what the workspace holds
    p.few_chunk = (int)(chunk < INT32_MAX / 2 ? chunk : INT32_MAX / 2);
    p.few_splits = (int)ceil_of(max_len, p.few_chunk);
    p.few_entries = p.few && p.few_splits > 1 ? S * kv_heads * (long long)p.few_rows * p.few_splits : 0;
    // row tiles of 128 rows until tiles of 256 more than fill the CUs; a sequence's last one counts half, of
    // sequences that have 128 at least (the others may be single tokens)
    const long long each = (T + S - 1) / S, wide = 256 / group, full = T * group / 128, long_ones = S < full ? S : full > 1 ? full : 1;
    auto count = [&](long long tokens) { return ceil_of(T + (long_ones - 1) * tokens / 2, tokens) * kv_heads; };
    p.many_waves = count(wide) > 256 ? 8 : 4;
    p.tile_tokens = 32 * p.many_waves / group;
    p.slots = T / p.tile_tokens + S;
    // Keys are split where tiles of 128 rows do not fill the CUs, of a prompt's own triangle only where they leave
    // half of them idle: joining costs more than it gains else.  Eight waves of two halves make a workgroup
    // to a CU; where whole parts leave too many idle that way, two workgroups of four waves.
    // In us, 32 query and 8 key heads of 128.  One wave and two to 32 rows: 1300 tokens 42 and 35, 658 tokens
    // of fp16 26.8 and 23.7, 256 tokens behind 4000 60 and 45; but 2000 tokens of heads of 64 (500 tiles) 44 and 47.
    // Whole and in parts: 64 tokens behind 8000 162 and 50, 512 behind 7600 166 and 102, 1100 of three sequences
    // behind up to 8000 (288 tiles) 185 and 132; 1024 behind 7000 (256 tiles) 182 and 179.
    // max_len is what the caller bounds the lengths by: where it is many times the lengths (the default, in tables of
    // 32768), parts are too long and prompts are taken for chunks behind a context: 16 single tokens over 4096 36 us for
    // 21, 8 over 2000 20.3 for 11.4, 658 tokens 28.8 for 23.7, 512 behind 7600 168 for 102, 4096 tokens the same.
    const long long tiles = count(p.tile_tokens);
    const bool behind = max_len > 2 * each;
    long long least = 512;
    chunk = max_len;
    p.many_halves = p.many_waves == 4 && max_len > 256 && tiles <= (behind ? 256 : 384);
    if (p.many_waves == 4 && tiles <= (behind ? 256 : 128)) {
        const bool pairs = behind && 256 / tiles * tiles < 176;
        if (pairs) p.many_halves = false;
        if (!behind) least = 1024;
        chunk = ceil_of(max_len, (pairs ? 512 : 256) / tiles);
    } else if (p.many_waves == 4 && behind && tiles < 512) {
        chunk = ceil_of(tiles * max_len, 640);
        least = 2048;
    }
    chunk = chunk < least ? least : ceil_of(chunk, kKeys) * kKeys;
    if (ceil_of(max_len, chunk) > 64) chunk = ceil_of(ceil_of(max_len, 64), kKeys) * kKeys;
    p.many_chunk = (int)(chunk < INT32_MAX / 2 ? chunk : INT32_MAX / 2);
    p.many_splits = (int)ceil_of(max_len, p.many_chunk);
    p.many_entries = p.many && p.many_splits > 1 ? T * heads * (long long)p.many_splits : 0;
    p.few_entries += p.few_entries & 1;  // the sums behind the statistics stay 16-byte aligned
    p.many_entries += p.many_entries & 1;
    p.bytes = (size_t)(p.few_entries + p.many_entries) * (size_t)(D + 2) * 4;
    return p;
}

hipError_t launch_kv_attention(int dtype, int D, const AttnPlan &pl, AttnArgs a, bool zero_rest, void *workspace, hipStream_t s)
{
    a.few_rows = pl.few_rows;
    a.few_tiles = pl.few_tiles;
    a.few_tile_rows = 16 * pl.few_rb;
    a.few_splits = pl.few_splits;
    a.few_chunk = pl.few_chunk;
    a.many_splits = pl.many_splits;
    a.many_chunk = pl.many_chunk;
    a.tile_tokens = pl.tile_tokens;
    a.slots = (int)pl.slots;
    float *w = (float *)workspace;
    a.few_stat = (f32x2 *)w;
    a.many_stat = a.few_stat + pl.few_entries;
    a.few_sum = (float *)(a.many_stat + pl.many_entries);
    a.many_sum = a.few_sum + pl.few_entries * D;
    a.zero_rest = zero_rest && a.v.offs;  // without offsets every row is a sequence's
    if (dtype == DT_F16) return D == 64 ? run_attention<DT_F16, 64>(pl, a, s) : run_attention<DT_F16, 128>(pl, a, s);
    return D == 64 ? run_attention<DT_BF16, 64>(pl, a, s) : run_attention<DT_BF16, 128>(pl, a, s);
}

}  // namespace qg
