// kv_api.hip -- host side of the attention layer's operators: argument checks
// and the C ABI of include/qgemm.h.  No kernels live here; the launch functions
// of kv.h do.
#include <cmath>
#include <cstdio>

#include "kv.h"

namespace qg {
namespace {

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

int status_of(hipError_t e, const char *what)
{
    if (e == hipSuccess) return QGEMM_OK;
    fprintf(stderr, "qgemm: %s launch failed: %s (%d)\n", what, hipGetErrorString(e), (int)e);
    return QGEMM_ERR_HIP;
}

// Items of at most 16 lanes in one launch, whose lanes, those of a last workgroup that is not full among them, stay below
// 2^32; a kernel's item index is an int.
bool items_fit(long long n) { return n >= 0 && n <= (1LL << 28) - 16; }

int page_shift(long long page)
{
    for (int s = 4; s <= 8; s++)
        if (page == (1LL << s)) return s;
    return -1;
}

int head_shape(long long heads, long long kv_heads, long long D)
{
    if (D != 64 && D != 128) return QGEMM_ERR_SHAPE;
    if (kv_heads < 1 || heads < 0 || kv_heads > 65536 || heads > 65536) return QGEMM_ERR_SHAPE;
    return QGEMM_OK;
}

// Rows of heads: 16-byte pieces, rows that hold all heads.
int rows_of(const void *x, long long stride, long long heads, long long D, bool written)
{
    if (!x) return QGEMM_ERR_NULL;
    if (!aligned(x, 16)) return QGEMM_ERR_ALIGN;
    if (stride < (written ? heads * D : 0) || stride % 8 != 0 || stride > INT32_MAX) return QGEMM_ERR_SHAPE;
    return QGEMM_OK;
}

int turn_of(const float *rope, long long rope_len, long long rot, int interleaved, const int32_t *positions, float eps,
            long long D, TurnArgs &t)
{
    if (rope && (rot < 16 || rot > D || rot % 16 != 0 || rope_len < 1 || rope_len > INT32_MAX)) return QGEMM_ERR_SHAPE;
    if (!aligned(rope, 16) || !aligned(positions, 4)) return QGEMM_ERR_ALIGN;
    if (eps != eps) return QGEMM_ERR_SHAPE;
    t = TurnArgs{rope, positions, rope ? (int)rope_len : 0, rope ? (int)rot : 0, interleaved != 0, eps};
    return QGEMM_OK;
}

// The cache, its tables and its sequences.
int view_of(const void *cache, long long pages, long long page, const int32_t *tables, long long width,
            const int32_t *lens, const int32_t *offsets, long long S, long long T, long long kv_heads, long long D,
            KvView &v)
{
    const int shift = page_shift(page);
    if (shift < 0) return QGEMM_ERR_FORMAT;
    if (S < 0 || T < 0 || T > INT32_MAX / 2 || S > INT32_MAX / 8 || (!offsets && S != T)) return QGEMM_ERR_SHAPE;
    if (pages < 1 || pages > INT32_MAX || width < 1 || width > ((1 << 30) >> shift)) return QGEMM_ERR_SHAPE;
    if (T == 0 || S == 0) return QGEMM_OK;
    if (!cache || !tables || !lens) return QGEMM_ERR_NULL;
    if (!aligned(cache, 16) || !aligned(tables, 4) || !aligned(lens, 4) || !aligned(offsets, 4)) return QGEMM_ERR_ALIGN;
    v = KvView{(uint8_t *)cache, kv_heads * page / kTile * 20 * D, (int)pages, shift, tables, (int)width, lens, offsets,
               (int)S, (int)T, (int)kv_heads};
    return QGEMM_OK;
}

// Sizes of an attention call, S and T checked before; max_len is the bound on the lengths that counts.
int attention_shape(long long T, long long S, long long heads, long long kv_heads, long long D, long long max_len)
{
    int st = head_shape(heads, kv_heads, D);
    if (st != QGEMM_OK) return st;
    if (heads < 1 || heads % kv_heads != 0 || heads / kv_heads > 128 || T > INT32_MAX / 2 || S > INT32_MAX / 8 ||
        max_len < 0 || max_len > INT32_MAX)
        return QGEMM_ERR_SHAPE;
    // every launch's work-items along x below 2^32: 16 lanes a row and head, 512 threads for each sequence's key head
    // and for each 128 of its rows
    return items_fit(T * heads) && items_fit(64 * S * heads) ? QGEMM_OK : QGEMM_ERR_SHAPE;
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" {

int qgemm_rope_table(int64_t positions, int64_t rot, double base, double scale, float *table)
{
    if (positions < 1 || positions > INT32_MAX || rot < 2 || rot > 65536 || rot % 2 != 0 || !(base > 0.0) ||
        !std::isfinite(base) || !std::isfinite(scale))
        return QGEMM_ERR_SHAPE;
    if (!table) return QGEMM_ERR_NULL;
    const int64_t half = rot / 2;
    for (int64_t i = 0; i < half; i++) {
        const double f = scale * std::pow(base, -2.0 * (double)i / (double)rot);
        for (int64_t p = 0; p < positions; p++) {
            table[p * rot + i] = (float)std::cos((double)p * f);
            table[p * rot + half + i] = (float)std::sin((double)p * f);
        }
    }
    return QGEMM_OK;
}

size_t qgemm_kv_page_bytes(int64_t kv_heads, int64_t head_dim, int64_t page)
{
    if (head_shape(1, kv_heads, head_dim) != QGEMM_OK || page_shift(page) < 0) return 0;
    return (size_t)(kv_heads * page / kTile * 20 * head_dim);
}

int qgemm_qk_norm_rope(const void *Q, int64_t q_stride, const void *K, int64_t k_stride, const float *q_weight,
                       const float *k_weight, const float *rope, int64_t rope_len, int64_t rot, int interleaved,
                       const int32_t *positions, float eps, void *Qout, int64_t qout_stride, void *Kout,
                       int64_t kout_stride, int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim, int dtype,
                       void *stream)
{
    NormRopeArgs a{};
    if (dtype != DT_F16 && dtype != DT_BF16) return QGEMM_ERR_DTYPE;
    if (head_dim != 64 && head_dim != 128) return QGEMM_ERR_SHAPE;
    if (heads < 0 || kv_heads < 0 || heads > 65536 || kv_heads > 65536 || heads + kv_heads < 1 || T < 0 || T > INT32_MAX / 2 ||
        !items_fit(T * (heads + kv_heads)))
        return QGEMM_ERR_SHAPE;
    int st = turn_of(rope, rope_len, rot, interleaved, positions, eps, head_dim, a.t);
    if (st != QGEMM_OK) return st;
    if (T == 0) return QGEMM_OK;
    if (rope && !positions) return QGEMM_ERR_NULL;
    if (heads) {
        if ((st = rows_of(Q, q_stride, heads, head_dim, false)) != QGEMM_OK) return st;
        if ((st = rows_of(Qout, qout_stride, heads, head_dim, true)) != QGEMM_OK) return st;
    }
    if (kv_heads) {
        if ((st = rows_of(K, k_stride, kv_heads, head_dim, false)) != QGEMM_OK) return st;
        if ((st = rows_of(Kout, kout_stride, kv_heads, head_dim, true)) != QGEMM_OK) return st;
    }
    if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return QGEMM_ERR_ALIGN;
    a.q = Heads{(const uint16_t *)Q, q_stride, q_weight, (uint16_t *)Qout, qout_stride, (int)heads};
    a.k = Heads{(const uint16_t *)K, k_stride, k_weight, (uint16_t *)Kout, kout_stride, (int)kv_heads};
    a.T = (int)T;
    return status_of(launch_norm_rope(dtype, (int)head_dim, a, (hipStream_t)stream), "head norm and rotation");
}

int qgemm_kv_append(void *cache, int64_t pages, int64_t page, const int32_t *tables, int64_t table_width,
                    const int32_t *lens, const int32_t *offsets, int64_t S, const void *K, int64_t k_stride,
                    const void *V, int64_t v_stride, const float *k_weight, const float *rope, int64_t rope_len,
                    int64_t rot, int interleaved, const int32_t *positions, float eps, const void *Q, int64_t q_stride,
                    const float *q_weight, void *Qout, int64_t qout_stride, int64_t T, int64_t heads, int64_t kv_heads,
                    int64_t head_dim, int dtype, void *stream)
{
    AppendArgs a{};
    a.zero_rest = (dtype & QGEMM_ZERO_REST) != 0;
    dtype &= ~QGEMM_ZERO_REST;
    if (dtype != DT_F16 && dtype != DT_BF16) return QGEMM_ERR_DTYPE;
    int st = head_shape(heads, kv_heads, head_dim);
    if (st != QGEMM_OK) return st;
    if ((st = view_of(cache, pages, page, tables, table_width, lens, offsets, S, T, kv_heads, head_dim, a.v)) != QGEMM_OK)
        return st;
    if (!items_fit((2 * T + 8 * S) * (heads + kv_heads))) return QGEMM_ERR_SHAPE;
    if ((st = turn_of(rope, rope_len, rot, interleaved, positions, eps, head_dim, a.t)) != QGEMM_OK) return st;
    if (T == 0 || S == 0) return QGEMM_OK;
    if ((st = rows_of(K, k_stride, kv_heads, head_dim, false)) != QGEMM_OK) return st;
    if ((st = rows_of(V, v_stride, kv_heads, head_dim, false)) != QGEMM_OK) return st;
    if (Q) {
        if (heads < 1) return QGEMM_ERR_SHAPE;
        if ((st = rows_of(Q, q_stride, heads, head_dim, false)) != QGEMM_OK) return st;
        if ((st = rows_of(Qout, qout_stride, heads, head_dim, true)) != QGEMM_OK) return st;
    }
    if (!aligned(k_weight, 16) || !aligned(q_weight, 16)) return QGEMM_ERR_ALIGN;
    a.k = Heads{(const uint16_t *)K, k_stride, k_weight, nullptr, 0, (int)kv_heads};
    a.q = Heads{(const uint16_t *)Q, q_stride, q_weight, (uint16_t *)Qout, qout_stride, Q ? (int)heads : 0};
    a.val = (const uint16_t *)V;
    a.val_stride = v_stride;
    return status_of(launch_kv_append(dtype, (int)head_dim, a, (hipStream_t)stream), "cache append");
}

int qgemm_kv_read(const void *cache, int64_t pages, int64_t page, const int32_t *tables, int64_t table_width,
                  const int32_t *lens, const int32_t *offsets, int64_t S, void *K, void *V, int64_t T, int64_t kv_heads,
                  int64_t head_dim, int out_type, void *stream)
{
    KvView v{};
    if (out_type != QGEMM_F16 && out_type != QGEMM_BF16 && out_type != QGEMM_F32) return QGEMM_ERR_DTYPE;
    int st = head_shape(1, kv_heads, head_dim);
    if (st != QGEMM_OK) return st;
    if ((st = view_of(cache, pages, page, tables, table_width, lens, offsets, S, T, kv_heads, head_dim, v)) != QGEMM_OK) return st;
    if (!items_fit(T * kv_heads)) return QGEMM_ERR_SHAPE;
    if (T == 0 || S == 0) return QGEMM_OK;
    if (!K || !V) return QGEMM_ERR_NULL;
    if (!aligned(K, 16) || !aligned(V, 16)) return QGEMM_ERR_ALIGN;
    return status_of(launch_kv_read(out_type, (int)head_dim, v, K, V, (hipStream_t)stream), "cache read");
}

size_t qgemm_kv_attention_workspace_bytes(int64_t T, int64_t S, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                          int64_t max_len, int ragged)
{
    if (T < 1 || S < 1 || T > INT32_MAX / 2 || S > INT32_MAX / 8 || attention_shape(T, S, heads, kv_heads, head_dim, max_len) != QGEMM_OK) return 0;
    return plan_attention(T, S, (int)heads, (int)kv_heads, (int)head_dim, max_len, ragged != 0).bytes;
}

int qgemm_kv_attention(const void *Q, int64_t q_stride, const void *cache, int64_t pages, int64_t page,
                       const int32_t *tables, int64_t table_width, const int32_t *lens, const int32_t *offsets, int64_t S,
                       void *Y, int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t window, float scale,
                       int64_t max_len, int dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    AttnArgs a{};
    const bool zero_rest = (dtype & QGEMM_ZERO_REST) != 0;
    dtype &= ~QGEMM_ZERO_REST;
    if (dtype != DT_F16 && dtype != DT_BF16) return QGEMM_ERR_DTYPE;
    int st = head_shape(heads, kv_heads, head_dim);
    if (st != QGEMM_OK) return st;
    if (window < 0 || max_len < 0 || !std::isfinite(scale)) return QGEMM_ERR_SHAPE;
    if ((st = view_of(cache, pages, page, tables, table_width, lens, offsets, S, T, kv_heads, head_dim, a.v)) != QGEMM_OK)
        return st;
    const long long capacity = table_width * page, bound = max_len == 0 || max_len > capacity ? capacity : max_len;
    if ((st = attention_shape(T, S, heads, kv_heads, head_dim, bound)) != QGEMM_OK) return st;
    if (T == 0 || S == 0) return QGEMM_OK;
    if ((st = rows_of(Q, q_stride, heads, head_dim, false)) != QGEMM_OK) return st;
    if (!Y) return QGEMM_ERR_NULL;
    if (!aligned(Y, 16)) return QGEMM_ERR_ALIGN;
    const AttnPlan pl = plan_attention(T, S, (int)heads, (int)kv_heads, (int)head_dim, bound, offsets != nullptr);
    if (pl.bytes && (!workspace || workspace_bytes < pl.bytes)) return QGEMM_ERR_SIZE;
    if (!aligned(workspace, 16)) return QGEMM_ERR_ALIGN;
    a.q = (const uint16_t *)Q;
    a.q_stride = q_stride;
    a.y = (uint16_t *)Y;
    a.heads = (int)heads;
    a.group = (int)(heads / kv_heads);
    a.window = (int)(window > INT32_MAX ? 0 : window);
    a.scale = scale;
    return status_of(launch_kv_attention(dtype, (int)head_dim, pl, a, zero_rest, workspace, (hipStream_t)stream), "cache attention");
}

}  // extern "C"
