// moe_route.hip -- routing of a mixture-of-experts layer: each token's top_k
// experts and their weights from its logits, and the token-expert pairs
// grouped by expert (offsets and the stable order the grouped GEMM and the
// few-token layer read).
//
// One wave per token: lane l holds logits l, l+64, ... as order-preserving
// 32-bit keys, so that each of the top_k rounds is a wave maximum (six DPP
// steps) and a ballot for the lowest index that holds it.  The keys order the
// logits themselves, not rounded scores, so the choice is exact and ties go
// to the lowest index.  Up to kFusedTokens tokens and kFusedPairs pairs, one
// workgroup routes all tokens and groups the pairs in LDS (one launch); above
// that the tokens spread over the CUs and a second launch groups.  Both are latency: a
// routing reads and writes at most a few hundred KB.
#include <cfloat>

#include "common.h"
#include "plan.h"

namespace qg {
namespace {

struct RouteArgs {
    const void *logits;
    int T, E, k;
    int score;   // QGEMM_SCORE_*
    int renorm;
    float scale;
    int *ids;    // [T][k]
    float *weights;
    int *offsets, *rows;
};

// Pairs that one workgroup of 1024 threads groups, one per thread.
constexpr int kFusedPairs = 1024;
// Tokens that the same workgroup routes first, four per wave.
constexpr int kFusedTokens = 64;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x)
{
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, false));
}

// Maximum over the wave, the same in every lane: row shifts inside rows of 16
// lanes, then the two row broadcasts; lane 63 ends with the whole maximum.
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    x = dpp_max<0x111>(x);  // row_shr:1
    x = dpp_max<0x112>(x);  // row_shr:2
    x = dpp_max<0x114>(x);  // row_shr:4
    x = dpp_max<0x118>(x);  // row_shr:8
    x = dpp_max<0x142>(x);  // row_bcast:15
    x = dpp_max<0x143>(x);  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
    return x;
}

// Order-preserving key of a logit: larger logit, larger key; NaN as -inf,
// +inf as the largest finite value, -0 as +0.  Never 0, the key of a taken
// or absent expert.
__device__ __forceinline__ uint32_t key_of(float v)
{
    v = v != v ? -INFINITY : fminf(v, FLT_MAX) + 0.0f;
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float of_key(uint32_t k)
{
    return __builtin_bit_cast(float, k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

enum { LOGIT_F16 = QGEMM_F16, LOGIT_BF16 = QGEMM_BF16, LOGIT_F32 = QGEMM_F32 };

template <int LT>
__device__ __forceinline__ float load_logit(const void *p, long long i)
{
    if constexpr (LT == LOGIT_F32) return ((const float *)p)[i];
    else if constexpr (LT == LOGIT_F16) return f16_to_f32(((const uint16_t *)p)[i]);
    else return __builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16);
}

// One token by one wave; lane j < k returns its j-th expert and weight.
template <int LT, int R>
__device__ __forceinline__ void route_token(const RouteArgs &a, int t, int lane, int &id, float &w)
{
    uint32_t key[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int e = 64 * r + lane;
        key[r] = e < a.E ? key_of(load_logit<LT>(a.logits, (long long)t * a.E + e)) : 0u;
    }
    uint32_t own = 0;
#pragma unroll
    for (int r = 0; r < R; r++) own = max(own, key[r]);
    const uint32_t top = wave_max(own);
    const float mx = of_key(top);
    float denom = 1.0f;
    if (a.score == QGEMM_SCORE_SOFTMAX && !a.renorm) {  // renormalised weights need the chosen ones only
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < R; r++)
            if (key[r] != 0u) s += expf(of_key(key[r]) - mx);
        denom = wave_sum(s);
    }
    id = 0;
    uint32_t mine = 0;
    for (int j = 0; j < a.k; j++) {
        const uint32_t m = j == 0 ? top : wave_max(own);
        int e = 0;
        bool found = false;
#pragma unroll
        for (int r = 0; r < R; r++) {
            const unsigned long long b = __ballot(key[r] == m);
            if (!found && b != 0ull) {
                found = true;
                const int l = __ffsll((long long)b) - 1;
                e = 64 * r + l;
                if (lane == l) key[r] = 0u;
            }
        }
        own = 0;
#pragma unroll
        for (int r = 0; r < R; r++) own = max(own, key[r]);
        if (lane == j) {
            id = e;
            mine = m;
        }
    }
    w = 0.0f;
    if (lane < a.k) {
        const float v = of_key(mine);
        if (a.score == QGEMM_SCORE_SIGMOID) w = 1.0f / (1.0f + expf(-v));
        else if (mx > -INFINITY) w = expf(v - mx) / denom;  // a row of -inf has no weights
    }
    if (a.renorm) {
        const float s = wave_sum(w);
        w = s > 0.0f ? w / s : 0.0f;
    }
    w *= a.scale;
}

template <int LT, int R>
__device__ __forceinline__ void route_store(const RouteArgs &a, int t, int lane, int *lds_ids)
{
    int id;
    float w;
    route_token<LT, R>(a, t, lane, id, w);
    if (lane < a.k) {
        const long long p = (long long)t * a.k + lane;
        a.ids[p] = id;
        a.weights[p] = w;
        if (lds_ids) lds_ids[p] = id;
    }
}

template <int LT>
__device__ __forceinline__ void route_any(const RouteArgs &a, int t, int lane, int *lds_ids)
{
    if (a.E <= 64) route_store<LT, 1>(a, t, lane, lds_ids);
    else if (a.E <= 128) route_store<LT, 2>(a, t, lane, lds_ids);
    else if (a.E <= 256) route_store<LT, 4>(a, t, lane, lds_ids);
    else if (a.E <= 512) route_store<LT, 8>(a, t, lane, lds_ids);
    else route_store<LT, 16>(a, t, lane, lds_ids);
}

// Pairs grouped by expert inside one workgroup of 1024 threads, pair p on
// thread p (P <= 1024), ids read from LDS: the lanes of a wave with equal ids
// find one another by one ballot per id bit; the first of them leaves the
// wave's count in `count` [16 waves][E]; a prefix over the waves and then over
// the experts turns the counts into positions.  `base` has E+1 entries.
__device__ __forceinline__ void group_block(const int *ids, int P, int E, int *offsets, int *rows, uint16_t *count,
                                            int *base)
{
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int nw = (P + 63) >> 6;
    for (int i = tid; i < nw * E; i += 1024) count[i] = 0;
    __syncthreads();
    int e = E;
    if (tid < P) {
        e = ids[tid];
        if (e < 0 || e > E) e = E;  // a dropped pair
    }
    unsigned long long same = ~0ull;
    for (int b = 0; (E >> b) != 0; b++) {
        const unsigned long long bal = __ballot((e >> b) & 1);
        same &= ((e >> b) & 1) ? bal : ~bal;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1ull));
    if (e < E && rank == 0) count[wv * E + e] = (uint16_t)__popcll(same);
    __syncthreads();
    // per expert: exclusive prefix over the waves, total in base[e]
    for (int x = tid; x < E; x += 1024) {
        int run = 0;
        for (int v = 0; v < nw; v++) {
            const int c = count[v * E + x];
            count[v * E + x] = (uint16_t)run;
            run += c;
        }
        base[x] = run;
    }
    __syncthreads();
    if (wv == 0) {  // exclusive prefix over the experts, 64 at a time
        int carry = 0;
        for (int x0 = 0; x0 < E; x0 += 64) {
            const int x = x0 + lane, c = x < E ? base[x] : 0;
            int incl = c;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int u = __shfl_up(incl, d, 64);
                if (lane >= d) incl += u;
            }
            if (x < E) {
                base[x] = carry + incl - c;
                offsets[x] = carry + incl - c;
            }
            carry += __shfl(incl, 63, 64);
        }
        if (lane == 0) {
            base[E] = carry;
            offsets[E] = carry;
        }
    }
    __syncthreads();
    if (e < E) rows[base[e] + count[wv * E + e] + rank] = tid;
    if (tid < P && tid >= base[E]) rows[tid] = -1;
}

// Dynamic LDS of group_block for P pairs and E experts: ids, base, counts.
size_t group_lds(int P, int E) { return 4 * (size_t)P + 4 * (size_t)(E + 1) + 2 * (size_t)((P + 63) / 64) * E; }

template <int LT>
__global__ void __launch_bounds__(1024) k_route_group(RouteArgs a)
{
    extern __shared__ int sh[];
    const int P = a.T * a.k;
    int *ids = sh, *base = sh + P;
    uint16_t *count = (uint16_t *)(base + a.E + 1);
    for (int t = threadIdx.x >> 6; t < a.T; t += 16) route_any<LT>(a, t, threadIdx.x & 63, ids);
    __syncthreads();
    group_block(ids, P, a.E, a.offsets, a.rows, count, base);
}

__global__ void __launch_bounds__(1024) k_group_small(const int *ids_in, int P, int E, int *offsets, int *rows)
{
    extern __shared__ int sh[];
    int *ids = sh, *base = sh + P;
    uint16_t *count = (uint16_t *)(base + E + 1);
    if ((int)threadIdx.x < P) ids[threadIdx.x] = ids_in[threadIdx.x];
    group_block(ids, P, E, offsets, rows, count, base);  // its first barrier orders the ids
}

template <int LT>
__global__ void __launch_bounds__(256) k_route(RouteArgs a)
{
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t < a.T) route_any<LT>(a, t, threadIdx.x & 63, nullptr);
}

// Many pairs: workgroup x owns expert x (x = E: the dropped pairs).  Its waves
// split the pairs into 16 contiguous ranges; pass one counts, per wave, the
// pairs of earlier experts and of its own; pass two writes its own pairs in
// order behind them.  Every workgroup reads all ids twice (from L2): no
// atomics, no second launch, and the order does not depend on timing.  The
// reads' latency and two comparisons per pair bound it, so the bulk of a range
// goes in blocks of kBlock pairs, four per lane and eight loads in flight, and
// what is left in rows of 64, one pair per lane and eight rows in flight
// (65536 pairs over 128 experts 11.2 us a call in blocks, 13.1 in rows; the
// 5264 pairs of 658 tokens, routed first, 12.7 in guarded blocks, 9.6 in
// rows).
constexpr int kBlock = 2048;

__global__ void __launch_bounds__(1024) k_group_large(const int *ids, int P, int E, int *offsets, int *rows)
{
    __shared__ int s_less[16], s_own[16];
    const int x = blockIdx.x, lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long n = ((long long)P + 63) / 64;
    // a multiple of 64 pairs, so a block's 16-byte loads are aligned
    const int lo = (int)(n * wv / 16) * 64, hi = (int)min((long long)P, n * (wv + 1) / 16 * 64);
    const int bulk = lo + (hi - lo) / kBlock * kBlock;
    // as unsigned, dropped ids are at least E
    const unsigned first = (unsigned)x, span = x < E ? 0u : 0xFFFFFFFFu - (unsigned)E;
    auto mine = [&](int v) { return (unsigned)v - first <= span; };
    auto block = [&](int p0, int4 (&q)[8]) {
#pragma unroll
        for (int u = 0; u < 8; u++) q[u] = *(const int4 *)(ids + p0 + 256 * u + 4 * lane);
    };
    auto rows8 = [&](int p0, int (&v)[8]) {  // rows past the end repeat the last pair
#pragma unroll
        for (int u = 0; u < 8; u++) v[u] = ids[min(p0 + 64 * u + lane, hi - 1)];
    };

    int less = 0, own = 0;
    for (int p0 = lo; p0 < bulk; p0 += kBlock) {
        int4 q[8];
        block(p0, q);
#pragma unroll
        for (int u = 0; u < 8; u++) {
            const int v[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                less += (unsigned)v[j] < first;
                own += mine(v[j]);
            }
        }
    }
    for (int p0 = bulk; p0 < hi; p0 += 512) {
        int v[8];
        rows8(p0, v);
#pragma unroll
        for (int u = 0; u < 8; u++) {
            const bool live = lane < hi - p0 - 64 * u;
            less += live && (unsigned)v[u] < first;
            own += live && mine(v[u]);
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        less += __shfl_xor(less, d, 64);
        own += __shfl_xor(own, d, 64);
    }
    if (lane == 0) {
        s_less[wv] = less;
        s_own[wv] = own;
    }
    __syncthreads();
    int pos = 0;
    for (int v = 0; v < 16; v++) pos += s_less[v];
    if (threadIdx.x == 0) offsets[x] = pos;
    for (int v = 0; v < wv; v++) pos += s_own[v];
    if (own == 0) return;
    const unsigned long long before = (1ull << lane) - 1ull;
    for (int p0 = lo; p0 < bulk; p0 += kBlock) {
        int4 q[8];
        block(p0, q);
#pragma unroll
        for (int u = 0; u < 8; u++) {  // 256 pairs in pair order: lanes first, then their four
            const int v[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
            unsigned long long b[4];
#pragma unroll
            for (int j = 0; j < 4; j++) b[j] = __ballot(mine(v[j]));
            if ((b[0] | b[1] | b[2] | b[3]) == 0ull) continue;
            int at = pos;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                at += __popcll(b[j] & before);
                pos += __popcll(b[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (mine(v[j])) rows[at++] = x < E ? p0 + 256 * u + 4 * lane + j : -1;
        }
    }
    for (int p0 = bulk; p0 < hi; p0 += 512) {
        int v[8];
        rows8(p0, v);
#pragma unroll
        for (int u = 0; u < 8; u++) {
            const int p = p0 + 64 * u + lane;
            const bool hit = lane < hi - p0 - 64 * u && mine(v[u]);
            const unsigned long long b = __ballot(hit);
            if (hit) rows[pos + __popcll(b & before)] = x < E ? p : -1;
            pos += __popcll(b);
        }
    }
}

hipError_t launch_group(const int *ids, int P, int E, int *offsets, int *rows, hipStream_t s)
{
    if (P <= kFusedPairs) {
        hipLaunchKernelGGL(k_group_small, dim3(1), dim3(1024), group_lds(P, E), s, ids, P, E, offsets, rows);
    } else {
        hipLaunchKernelGGL(k_group_large, dim3((unsigned)E + 1), dim3(1024), 0, s, ids, P, E, offsets, rows);
    }
    return hipGetLastError();
}

template <int LT>
hipError_t launch_route(const RouteArgs &a, hipStream_t s)
{
    const long long P = (long long)a.T * a.k;
    if (P <= kFusedPairs && a.T <= kFusedTokens) {
        hipLaunchKernelGGL((k_route_group<LT>), dim3(1), dim3(1024), group_lds((int)P, a.E), s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((k_route<LT>), dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_group(a.ids, (int)P, a.E, a.offsets, a.rows, s);
}

}  // namespace

hipError_t launch_moe_route(int logit_type, const void *logits, int T, int E, int k, int score, int renorm, float scale,
                            int *ids, float *weights, int *offsets, int *rows, hipStream_t s)
{
    const RouteArgs a{logits, T, E, k, score, renorm, scale, ids, weights, offsets, rows};
    if (logit_type == LOGIT_F32) return launch_route<LOGIT_F32>(a, s);
    return logit_type == LOGIT_F16 ? launch_route<LOGIT_F16>(a, s) : launch_route<LOGIT_BF16>(a, s);
}

hipError_t launch_moe_group(const int *ids, int P, int E, int *offsets, int *rows, hipStream_t s)
{
    return launch_group(ids, P, E, offsets, rows, s);
}

}  // namespace qg
