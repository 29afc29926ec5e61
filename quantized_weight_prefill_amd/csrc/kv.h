// kv.h -- what the attention layer's kernels share: the 4-bit paged cache of
// keys and values, its sequences, and the launch arguments.
//
// A cache is a pool of pages; a sequence's tokens lie in the pages that its
// row of `tables` names.  A page holds one region per key head, each of tiles
// of 16 tokens, 20*D bytes a tile:
//   key codes      8*D  lane (h, r), h = 0..3, r = token: dims D/4*h .. +D/4-1
//   key headers    2*D  [D/32 groups][16 tokens] (scale, minimum), two fp16
//   value codes    8*D  lane (h, n), n = 0..15: dims E*n .. E*n+E-1 (E = D/16)
//                       of tokens 4h .. 4h+3
//   value headers  2*D  as the keys'
// Both code regions are the 16x16x32 MFMA's A operand as a wave loads it, D/8
// bytes per lane and all of them contiguous: for keys the rows are tokens and the
// lane's registers run over dims (the contraction of q.k), for values the rows
// are dims and the registers run over tokens (the contraction of p.v), so
// neither product needs a transposition.  A lane's keys share one header (two
// where D/4 > 32), its values one per token.
// Key words hold 8 codes in the packed weights' pair order; a value word holds
// two dims of four tokens, dim parity b and token i at bits 4*(2b + i/2) +
// 16*(i%2): one AND leaves two neighbouring codes 16 bits apart in both.
#pragma once

#include "common.h"

namespace qg {

constexpr int kTile = 16;          // tokens of a tile
constexpr int kQuad = 4;           // tokens whose value codes share a word
constexpr float kKvMax = 32768.0f;  // magnitudes are held to this: code*scale + minimum then stays in fp16's range

template <int D>
struct KvLay {
    static constexpr int E = D / 16;            // dims of a lane's values
    static constexpr int kLane = D / 8;         // code bytes of a lane
    static constexpr int kKeyHead = 8 * D, kVal = 10 * D, kValHead = 18 * D, kBytes = 20 * D;
    static constexpr int kGroups = D / 32;
};

struct KvView {
    uint8_t *cache;
    long long page_bytes;
    int pages, page_shift;
    const int *tables;      // [S][width]
    int width;
    const int *lens;        // [S], new tokens included
    const int *offs;        // [S+1] rows of the new tokens, or null: one each
    int S, T, H;            // sequences, rows, key heads
};

// A sequence's rows [row, row + n) and the place of the first of them.  Any
// contents of offs and lens give rows inside [0, T); places outside the
// table are for tile_of and the callers' range checks.
struct Seq {
    int row, n, first, len;
};

constexpr int kMaxLen = 0x7FFFFF00;  // lengths are clamped to it, so that a few tokens more stay in range

__device__ __forceinline__ int row_end(const KvView &v, int s)
{
    return min(max(v.offs[s], 0), v.T);
}

__device__ __forceinline__ Seq seq_of(const KvView &v, int s)
{
    Seq q;
    q.len = min(max(v.lens[s], 0), kMaxLen);
    if (v.offs) {
        q.row = row_end(v, s);
        q.n = max(row_end(v, s + 1) - q.row, 0);
    } else {
        q.row = s;
        q.n = 1;
    }
    q.first = q.len - q.n;
    return q;
}

// Slots: work is handed out in units of `per` rows, and sequence s starts at
// slot row/per + extra*s, so that `extra` units more than row/per counts are left for
// what its ends cut off; slots past a sequence's need find nothing to do.
// The sequence that owns slot x: the last one starting at or before x, found by W
// lanes that probe W places at a time (x is the same in all of them).
template <int W>
__device__ __forceinline__ int find_seq(const KvView &v, int x, int per, int extra)
{
    const int lane = threadIdx.x & (W - 1), shift = (threadIdx.x & 63) & ~(W - 1);
    int lo = 0, span = v.S;
    while (span > 1) {
        const int step = (span + W - 1) / W, s = lo + lane * step;
        const bool before = s < min(lo + span, v.S) && row_end(v, s) / per + extra * s <= x;
        const unsigned long long b = (__ballot(before) >> shift) & (~0ull >> (64 - W));
        lo += max(__popcll(b) - 1, 0) * step;
        span = step;
    }
    return min(lo, v.S - 1);
}

// Bytes of the tile that holds place `at` of sequence s for key head h, or
// null where its table names no page.
template <int D>
__device__ __forceinline__ uint8_t *tile_of(const KvView &v, int s, int at, int h)
{
    const int i = at >> v.page_shift;
    if (at < 0 || i >= v.width) return nullptr;
    const int id = v.tables[(long long)s * v.width + i];
    if ((unsigned)id >= (unsigned)v.pages) return nullptr;
    const int in = (at & ((1 << v.page_shift) - 1)) >> 4, tiles = 1 << (v.page_shift - 4);
    return v.cache + (long long)id * v.page_bytes + (long long)(h * tiles + in) * KvLay<D>::kBytes;
}

template <int DT>
__device__ __forceinline__ float of_bits(uint32_t bits16)
{
    if constexpr (DT == DT_F16) return f16_to_f32(bits16);
    else return __builtin_bit_cast(float, bits16 << 16);
}

// E neighbouring values as 16-bit ones or floats.
template <int OT, int E>
__device__ __forceinline__ void store_out(void *base, long long i, const float (&x)[E])
{
    if constexpr (OT == QGEMM_F32) {
#pragma unroll
        for (int j = 0; j < E / 4; j++)
            *(f32x4 *)((float *)base + i + 4 * j) = f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
    } else {
        uint32_t w[E / 2];
#pragma unroll
        for (int j = 0; j < E / 2; j++) w[j] = pack_out<OT>(x[2 * j], x[2 * j + 1]);
        __builtin_memcpy(__builtin_assume_aligned((uint16_t *)base + i, 2 * E), w, 2 * E);
    }
}

// Norm and rotation of heads: what qk_norm_rope and kv_append share.
struct TurnArgs {
    const float *rope;      // [rope_len][rot]: cosines, then sines; null: none
    const int *positions;   // [T]; null: the token's place in its sequence
    int rope_len, rot, interleaved;
    float eps;              // negative: no norm
};

struct Heads {
    const uint16_t *x;      // [T] rows of `stride` elements, heads of D side by side
    long long stride;
    const float *weight;    // [D] or null
    uint16_t *y;
    long long y_stride;
    int heads;
};

struct NormRopeArgs {
    TurnArgs t;
    Heads q, k;
    int T;
};

struct AppendArgs {
    KvView v;
    TurnArgs t;
    Heads k, q;             // q.x null: no queries
    const uint16_t *val;
    long long val_stride;
    int value_blocks, key_blocks;  // workgroups of values and of keys; the rest are the queries'
    bool zero_rest;         // zeros to the queries of no sequence
};

// Partial results of the attention, of one row and query head from one part of
// the keys: the sums of p*v [D], and (b, sum of p) with p relative to 2^b.
typedef float f32x2 __attribute__((ext_vector_type(2)));

struct AttnArgs {
    KvView v;
    const uint16_t *q;
    long long q_stride;
    uint16_t *y;            // [T][heads][D]
    int heads, group;       // query heads, and of them to a key head
    int window;             // 0: none
    float scale;
    int few_rows;           // sequences of at most so many rows (tokens * group) are k_attn_few's
    int few_tiles, few_tile_rows;  // k_attn_few: row tiles of a sequence, rows of each
    int few_splits, few_chunk;    // k_attn_few: workgroups along the keys, keys of each
    int many_splits, many_chunk;  // k_attn_many's
    int tile_tokens, slots;       // k_attn_many: tokens of a row tile, row tiles of all sequences (a bound)
    bool zero_rest;               // zeros to the rows of no sequence: by k_attn_join or, without it, by
    int work_blocks, rest_blocks;  // rest_blocks workgroups behind the work_blocks of the last launch
    float *few_sum, *many_sum;    // partial results (null: one split)
    f32x2 *few_stat, *many_stat;
};

// The parts of a call's workspace and its launches (kv_attention.hip).
struct AttnPlan {
    bool few, many, many_halves;  // halves: two waves to 32 rows, each with half of the keys
    int few_rows, few_tiles, few_rb, few_waves;
    int few_splits, few_chunk, many_splits, many_chunk, tile_tokens, many_waves;
    long long slots, few_entries, many_entries;  // entries: rows * heads * splits kept
    size_t bytes;
};
AttnPlan plan_attention(long long T, long long S, int heads, int kv_heads, int D, long long max_len, bool ragged);

hipError_t launch_norm_rope(int dtype, int D, const NormRopeArgs &a, hipStream_t s);
hipError_t launch_kv_append(int dtype, int D, const AppendArgs &a, hipStream_t s);
// out_type: QGEMM_F16, QGEMM_BF16 or QGEMM_F32
hipError_t launch_kv_read(int out_type, int D, const KvView &v, void *k, void *val, hipStream_t s);
// zero_rest: zeros to the rows of no sequence
hipError_t launch_kv_attention(int dtype, int D, const AttnPlan &pl, AttnArgs a, bool zero_rest, void *workspace, hipStream_t s);

}  // namespace qg
