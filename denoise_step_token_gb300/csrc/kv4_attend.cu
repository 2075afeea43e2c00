// dllm_kv4_attend: attention of a block's queries over the paged 4-bit cache,
// and the weight every cached token receives.
//
// Mathematics, per row (one query position and head) over tokens j, in base 2:
// a_j = (scale log2 e) q . k_j.  A running offset m follows the largest a_j seen;
// l = sum 2^(a_j - m) and O = sum 2^(a_j - m) v_j are held in 32 bits and scaled by
// 2^(m - m') when the offset moves to m'.  out = O / l, lse = (m + log2 l) ln 2.
// The offset sits 7 below the maximum it was set from and moves only when a
// score passes it by more than 15: 2^(a_j - m) stays below 2^15, inside fp16's
// range, moves are rare, and weights down to 2^-31 of a row's largest keep
// their place in fp16.  The weights are rounded to fp16 for the product with the
// values, as the tensor cores take them: within 2^-11 of each, an eighth of what
// rounding the output to bf16 costs it.  (Outputs are 0.0017 of their norm from 64
// bits, as those of a 32-bit softmax rounded to bf16 are; the weights' other bits
// would be a second product with the values.)  The normaliser l sums them before
// that rounding.  Keys and values are exact in fp16 (see kv4.cuh), queries down to
// 2^-16 of their row's largest (see kv4_mma.cuh), so a score's only other roundings
// are the tensor cores' 32-bit sums.
//
// The weights of the tokens need every row's lse first, so a second kernel forms
// the scores again and adds 2^(a_j - lse) over the rows, one warp owning a token.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kv4_attend.cuh"

namespace dllm {
namespace {

// ---------------------------------------------------------------------------
// Few rows: 16 rows per CTA, four warps with 16 tokens at a time
// ---------------------------------------------------------------------------
// A thread loads the codes that it feeds to the tensor cores and widens them in
// registers.  Bound by each warp's dependent chain (load, widen, score products,
// vote, exponentials, widen, value products) with three warps per scheduler, not by
// memory: 64 blocks of 32 rows over caches of 96 to 1280 tokens take 177 us (1.26
// TB/s), 16 single tokens over caches of 8 to 33 K 109 us (1.47 TB/s).  The same
// chain fed from rings of bulk copies, 166 KB in flight per SM, took 189 and 108 us.
constexpr int kRowWarps = 4;

// V codes of 16 tokens: tokens 2t, 2t+1, 2t+8, 2t+9; channels [g D/8, (g+1) D/8).
template <int D>
struct ValueTile {
    static constexpr int kWords = D / 64;
    uint32_t w[4][kWords];
    uint32_t par[4];
    __device__ __forceinline__ void load(const uint8_t* half, int shift, int slot0, int g, int t) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int slot = slot0 + 2 * t + (k & 1) + (k >> 1) * 8;
            const uint8_t* c = half + slot * (D / 2) + g * (D / 16);
            if constexpr (D == 128) {
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(c));
                w[k][0] = q.x; w[k][1] = q.y;
            } else {
                w[k][0] = __ldg(reinterpret_cast<const uint32_t*>(c));
            }
            par[k] = __ldg(reinterpret_cast<const uint16_t*>(half + ((D / 2) << shift) + slot * (D / 16)) + g * (D / 8) / 32);
        }
    }
};

// grid: (splits, key/value heads * tiles, requests)
template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_attend_rows_kernel(const __grid_constant__ AttendParams P) {
    constexpr int kNt = D / 8;    // n8 tiles of the output
    constexpr int kKs = D / 16;   // products along the channels
    __shared__ float s_o[kRowWarps][16][D + 4];
    __shared__ float s_m[kRowWarps][16], s_l[kRowWarps][16];
    __shared__ int s_last;
    pdl_wait();
    pdl_release();
    const int b = blockIdx.z, head = blockIdx.y / P.tiles, tile = blockIdx.y - head * P.tiles, split = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int n = kv4_len(P.C, P.lens, b);
    const int blocks = (n + 15) >> 4;
    const int lo = (int)((long long)blocks * split / P.splits), hi = (int)((long long)blocks * (split + 1) / P.splits);

    // queries: rows g and g + 8 of the tile
    uint32_t qa[kKs][4];
    float rs[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = tile * 16 + g + 8 * h;
        uint32_t w[D / 8];
        if (r < P.Q.rows) {
            const uint4* src = reinterpret_cast<const uint4*>(P.Q.at(b, head, r) + t * (D / 4));
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const uint4 q = __ldg(src + k);
                w[4 * k] = q.x; w[4 * k + 1] = q.y; w[4 * k + 2] = q.z; w[4 * k + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < D / 8; ++k) w[k] = 0;
        }
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float down, up;
        row_power(amax, down, up);
        rs[h] = P.scale2 * up;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
            const uint32_t v = pack_h2(bf16_lo(w[k]) * down, bf16_hi(w[k]) * down);
            qa[k >> 1][h + 2 * (k & 1)] = v;
        }
    }

    float o[kNt][4];
#pragma unroll
    for (int k = 0; k < kNt; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int slot_mask = (1 << P.C.page_shift) - 1;
    for (int blk = lo + warp; blk < hi; blk += kRowWarps) {
        const int j0 = blk * 16;
        const uint8_t* page = kv4_page(P.C, P.C.table, b, j0 >> P.C.page_shift, P.C.max_pages, head);
        if (!page) page = P.C.pages;   // the error is recorded; results unspecified
        const int slot0 = j0 & slot_mask;
        KeyTile<D> kt[2];
        ValueTile<D> vt;
        kt[0].load(page, P.C.page_shift, slot0 + g, t);
        kt[1].load(page, P.C.page_shift, slot0 + 8 + g, t);
        vt.load(page + P.C.head_bytes / 2, P.C.page_shift, slot0, g, t);
        float s[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t bb[kKs][2];
            kt[u].widen(bb);
            s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < kKs; ++k) mma16816(s[u], qa[k], bb[k][0], bb[k][1]);
        }
        float top[2] = {-INFINITY, -INFINITY};
        const bool ragged = j0 + 16 > n;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[u][e] *= rs[e >> 1];
                if (ragged && j0 + u * 8 + 2 * t + (e & 1) >= n) s[u][e] = -INFINITY;
                top[e >> 1] = fmaxf(top[e >> 1], s[u][e]);
            }
        if (__any_sync(0xffffffffu, top[0] > m[0] + kAbove || top[1] > m[1] + kAbove)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = top[h];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                const float mn = fmaxf(m[h], x - kBelow);
                const float f = m[h] == -INFINITY ? 0.0f : ex2_approx(m[h] - mn);
                m[h] = mn;
                l[h] *= f;
#pragma unroll
                for (int k = 0; k < kNt; ++k) {
                    o[k][2 * h] *= f;
                    o[k][2 * h + 1] *= f;
                }
            }
        }
        uint32_t pa[4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float p0 = ex2_approx(s[u][2 * h] - m[h]), p1 = ex2_approx(s[u][2 * h + 1] - m[h]);
                l[h] += p0 + p1;
                pa[h + 2 * u] = pack_h2(p0, p1);
            }
        // values: parameters of tokens (2t, 2t+1) and (2t+8, 2t+9) side by side; past the end they make zeros
        Kv4Scale vs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            vs[u] = kv4_scale(vt.par[2 * u] | (vt.par[2 * u + 1] << 16));
            if (ragged) {
                const int j = j0 + u * 8 + 2 * t;
                const uint32_t keep = (j < n ? 0xffffu : 0u) | (j + 1 < n ? 0xffff0000u : 0u);
                vs[u].s &= keep;
                vs[u].c &= keep;
            }
        }
#pragma unroll
        for (int k = 0; k < ValueTile<D>::kWords; ++k) {
            uint32_t bv[2][8];   // [token pair][channel of the word]
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t a = vt.w[2 * u][k], c = vt.w[2 * u + 1][k];
                kv4_widen(__byte_perm(a, c, 0x5410), vs[u], bv[u][0], bv[u][2], bv[u][4], bv[u][6]);
                kv4_widen(__byte_perm(a, c, 0x7632), vs[u], bv[u][1], bv[u][3], bv[u][5], bv[u][7]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) mma16816(o[8 * k + e], pa, bv[0][e], bv[1][e]);
        }
    }

    // the warps' results, then the CTA's
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (t == 0) {
            s_m[warp][g + 8 * h] = m[h];
            s_l[warp][g + 8 * h] = l[h];
        }
#pragma unroll
        for (int k = 0; k < kNt; ++k) {
            s_o[warp][g + 8 * h][2 * t * kNt + k] = o[k][2 * h];
            s_o[warp][g + 8 * h][(2 * t + 1) * kNt + k] = o[k][2 * h + 1];
        }
    }
    __syncthreads();
    const int row = tid >> 3, part = tid & 7;   // 8 threads per row, D/8 channels each
    float acc[kNt], mm = -INFINITY, ll = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) mm = fmaxf(mm, s_m[w][row]);
#pragma unroll
    for (int k = 0; k < kNt; ++k) acc[k] = 0.0f;
    for (int w = 0; w < kRowWarps; ++w) {
        const float mw = s_m[w][row];
        const float f = mw == -INFINITY ? 0.0f : ex2_approx(mw - mm);
        ll += f * s_l[w][row];
#pragma unroll
        for (int k = 0; k < kNt; ++k) acc[k] += f * s_o[w][row][part * kNt + k];
    }
    if (P.splits > 1) {
        const long long unit = ((long long)b * gridDim.y + blockIdx.y);
        constexpr int kSlot = 16 * (D + 2);
        float* mine = P.partial + (unit * P.splits + split) * kSlot;
#pragma unroll
        for (int k = 0; k < kNt; ++k) mine[row * D + part * kNt + k] = acc[k];
        if (part == 0) {
            mine[16 * D + row] = mm;
            mine[16 * D + 16 + row] = ll;
        }
        __threadfence();
        __syncthreads();
        if (tid == 0) s_last = atom_add_acqrel_gpu(P.counters + unit, 1) == P.splits - 1;
        __syncthreads();
        if (!s_last) return;
        __threadfence();
        if (tid == 0) P.counters[unit] = 0;
        const float* all = P.partial + unit * P.splits * kSlot;
        mm = -INFINITY;
        for (int k = 0; k < P.splits; ++k) mm = fmaxf(mm, __ldcg(all + (size_t)k * kSlot + 16 * D + row));
        ll = 0.0f;
#pragma unroll
        for (int k = 0; k < kNt; ++k) acc[k] = 0.0f;
        for (int s = 0; s < P.splits; ++s) {   // in split order: equal calls give equal bits
            const float* from = all + (size_t)s * kSlot;
            const float mw = __ldcg(from + 16 * D + row);
            const float f = mw == -INFINITY ? 0.0f : ex2_approx(mw - mm);
            ll += f * __ldcg(from + 16 * D + 16 + row);
#pragma unroll
            for (int k = 0; k < kNt; k += 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(from + row * D + part * kNt + k));
                acc[k] += f * v.x;
                acc[k + 1] += f * v.y;
                acc[k + 2] += f * v.z;
                acc[k + 3] += f * v.w;
            }
        }
    }
    const int r = tile * 16 + row;
    if (r >= P.Q.rows) return;
    const long long at = P.row_at(b, head, r);
    if (part == 0 && P.lse) P.lse[at] = n > 0 ? (mm + log2f(ll)) * kLn2 : -INFINITY;
    const float inv = n > 0 ? 1.0f / ll : 0.0f;
    uint4* dst = reinterpret_cast<uint4*>(P.out + at * D + part * kNt);
#pragma unroll
    for (int k = 0; k < kNt; k += 8) {
        dst[k / 8] = make_uint4(pack_bf2(acc[k] * inv, acc[k + 1] * inv), pack_bf2(acc[k + 2] * inv, acc[k + 3] * inv),
                                pack_bf2(acc[k + 4] * inv, acc[k + 5] * inv), pack_bf2(acc[k + 6] * inv, acc[k + 7] * inv));
    }
}

// ---------------------------------------------------------------------------
// The tokens' weights: a warp owns 32 tokens and runs over all rows
// ---------------------------------------------------------------------------
constexpr int kWeightWarps = 8;
constexpr int kWeightTiles = 8;   // 16-row tiles staged at a time

// grid: (token tiles of 256, key/value heads, requests)
template <int D>
__global__ void __launch_bounds__(kWeightWarps * 32) kv4_weights_kernel(const __grid_constant__ AttendParams P) {
    constexpr int kKs = D / 16;
    __shared__ uint32_t s_q[kWeightTiles][kKs][32][4];   // queries in the product's order
    __shared__ float2 s_row[kWeightTiles * 16];          // (row scale, lse in base 2)
    pdl_wait();
    pdl_release();
    const int b = blockIdx.z, head = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int n = kv4_len(P.C, P.lens, b);
    const int base = blockIdx.x * (kWeightWarps * 32);
    if (base >= n) return;
    const int j0 = base + warp * 32;
    const int slot_mask = (1 << P.C.page_shift) - 1;
    uint32_t kb[4][kKs][2];
    int where[4];   // page of each 8 tokens, -1: none
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int j = j0 + u * 8;
        where[u] = -1;
        KeyTile<D> kt;
        kt.par = 0;
#pragma unroll
        for (int k = 0; k < KeyTile<D>::kWords; ++k) kt.w[k] = 0;
        if (j < n) {
            const uint8_t* page = kv4_page(P.C, P.C.table, b, j >> P.C.page_shift, P.C.max_pages, head, &where[u]);
            if (page) kt.load(page, P.C.page_shift, (j & slot_mask) + g, t);
        }
        kt.widen(kb[u]);
    }
    float sum[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) sum[u][0] = sum[u][1] = 0.0f;
    for (int r0 = 0; r0 < P.Q.rows; r0 += kWeightTiles * 16) {
        const int rows = min(kWeightTiles * 16, (P.Q.rows - r0 + 15) & ~15);
        __syncthreads();
        for (int rr = warp; rr < rows; rr += kWeightWarps) {   // a warp stages a row: D/32 channels per lane
            const int r = r0 + rr;
            constexpr int kPer = D / 32;   // 4 or 2
            uint32_t w[kPer / 2];
#pragma unroll
            for (int k = 0; k < kPer / 2; ++k) w[k] = 0;
            if (r < P.Q.rows) {
                const uint16_t* src = P.Q.at(b, head, r) + lane * kPer;
#pragma unroll
                for (int k = 0; k < kPer / 2; ++k) w[k] = __ldg(reinterpret_cast<const uint32_t*>(src) + k);
            }
            float amax = 0.0f;
#pragma unroll
            for (int k = 0; k < kPer / 2; ++k) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            float down, up;
            row_power(amax, down, up);
#pragma unroll
            for (int k = 0; k < kPer / 2; ++k) {
                const int c = lane * kPer + 2 * k;              // first channel of the pair
                const int ct = c / (D / 4), in = c % (D / 4);   // its thread of the quad, its place there
                s_q[rr >> 4][in / 4][(rr & 7) * 4 + ct][((rr >> 3) & 1) + 2 * ((in & 3) >> 1)] =
                    pack_h2(bf16_lo(w[k]) * down, bf16_hi(w[k]) * down);
            }
            if (lane == 0) {
                float2 v = make_float2(0.0f, INFINITY);   // a row past the end gives 2^(0 - inf) = 0
                if (r < P.Q.rows) {
                    v = make_float2(P.scale2 * up, P.lse[P.row_at(b, head, r)] * kLog2e);
                }
                s_row[rr] = v;
            }
        }
        __syncthreads();
        for (int mt = 0; mt < rows / 16; ++mt) {
            float s[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < kKs; ++k) {
                const uint4 q = *reinterpret_cast<const uint4*>(s_q[mt][k][lane]);
                const uint32_t a[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) mma16816(s[u], a, kb[u][k][0], kb[u][k][1]);
            }
            const float2 r0v = s_row[mt * 16 + g], r1v = s_row[mt * 16 + g + 8];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    sum[u][e] += ex2_approx(fmaf(s[u][e], r0v.x, -r0v.y)) + ex2_approx(fmaf(s[u][2 + e], r1v.x, -r1v.y));
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float v = sum[u][e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            const int j = j0 + u * 8 + 2 * t + e;
            if (g == 0 && j < n && where[u] >= 0) {
                const long long at = (((long long)where[u] * P.C.heads + head) << P.C.page_shift) + (j & slot_mask);
                P.weights[at] = (P.prior ? P.prior[at] : 0.0f) + v;
            }
        }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
constexpr int kMaxSlots = 4096;   // splits of all units (request, head, tile) in a call
constexpr int kMaxSplits = 64;    // of one unit
// Up to this many rows per key/value head: kv4_attend_rows_kernel, then the tile
// kernels.  64 requests of 8 heads and 96 to 1280 tokens: 16 rows 51 us (tiles 61),
// 32 rows 60 (61), 40 rows 79 (63).  With weights the tiles are ahead from 24 rows
// on (94 against 110), and over 4 requests of 20 to 33 K tokens and 4 heads at any
// number (8 rows: 61 against 69).
constexpr int kFewRows = 32;

// Splits of a unit's tokens: enough that every SM has its three resident CTAs
// twice over, none under 256 tokens.  One row of seven heads a key/value head, us:
//   six CTAs an SM (three, twelve): 32 requests of 4 heads and 8 to 33 K tokens 166
//   (192, 168), 8 such requests 65 (61, 87), 64 of 8 heads and up to 400 tokens 32
//   (16, 32);
//   256 tokens (128, 512): one request of 4 heads and up to 1280 tokens 11.0 (11.3,
//   12.2), 8 of them 14 (17, 13), 32 of up to 400 tokens 15 (18, 8).
inline int pick_splits(long long units, int max_tokens, int sms) {
    if (units > kJoinCounters) return 1;
    long long s = ((long long)sms * 6 + units - 1) / units;
    s = std::min<long long>(s, (max_tokens + 255) / 256);
    s = std::min<long long>(s, kMaxSlots / units);
    return (int)std::max<long long>(std::min<long long>(s, kMaxSplits), 1);
}

// Blocks of rows of a key/value head, and the items a plan may hold: every unit
// once, and a piece more for every CTA.
inline int row_blocks(int rows) { return (rows + kTileRows - 1) / kTileRows; }
inline size_t max_items(const dllm_kv4_cache& c, int rows) {
    return (size_t(std::max(c.B, 1)) * c.heads * row_blocks(rows) + kMaxCtas + 7) & ~size_t(7);
}

inline int check_rows(const dllm_kv4_cache& c, int L, int q_heads) {
    if (L < 1 || L > DLLM_MAX_L || q_heads < 1 || q_heads % c.heads) return DLLM_ERR_INVAL;
    if ((long long)L * q_heads > (1 << 20)) return DLLM_ERR_UNSUPPORTED;
    return DLLM_OK;
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_kv4_attend_workspace_size(const dllm_kv4_cache* c, int32_t L, int32_t q_heads) {
    if (!c || c->heads < 1 || dllm_kv4_page_bytes(c->page_size, c->head_dim) == 0) return 0;
    if (check_rows(*c, L, q_heads) != DLLM_OK) return 0;
    const int rows = L * (q_heads / c->heads);
    size_t n = size_t(kJoinCounters) * 4;
    if (rows <= kFewRows) {   // no more for fewer units, or a shorter table: one workspace serves a shrinking batch
        const size_t units = size_t(std::max(c->B, 1)) * c->heads * ((rows + 15) / 16);
        return n + std::min(units * kMaxSplits, size_t(kMaxSlots)) * 16 * (c->head_dim + 2) * 4;
    }
    n += sizeof(TilePlan) + max_items(*c, rows) * sizeof(TileItem);
    return n + size_t(2 * kMaxCtas) * kTileRows * (c->head_dim + 2) * 4;
}

extern "C" int dllm_kv4_attend(const dllm_kv4_attend_args* a, void* stream) {
    if (!a) return DLLM_ERR_INVAL;
    AttendParams P;
    int rc = kv4_check(a->cache, &P.C);
    if (rc != DLLM_OK) return rc;
    const int H = a->cache.heads, D = a->cache.head_dim, B = a->cache.B;
    rc = check_rows(a->cache, a->L, a->q_heads);
    if (rc != DLLM_OK) return rc;
    if (!isfinite(a->scale)) return DLLM_ERR_INVAL;
    if (B == 0) return DLLM_OK;
    if (!a->q || !a->lens || !a->out || (a->weights && !a->lse) || (a->prior && !a->weights)) return DLLM_ERR_INVAL;
    if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out)) & 15) return DLLM_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if (a->q_stride[i] % 8) return DLLM_ERR_ALIGN;
    if (!a->workspace || (reinterpret_cast<uintptr_t>(a->workspace) & 255) ||
        a->workspace_bytes < dllm_kv4_attend_workspace_size(&a->cache, a->L, a->q_heads))
        return DLLM_ERR_WORKSPACE;
    const int group = a->q_heads / H;
    if ((long long)H * ((a->L * group + 15) / 16) > 65535) return DLLM_ERR_UNSUPPORTED;
    int sms = 0;
    rc = kv4_device(&P.C, &sms);
    if (rc != DLLM_OK) return rc;
    P.Q = QueryRows{a->q, a->q_stride[0], a->q_stride[1], a->q_stride[2], a->L, group, a->L * group};
    P.q_heads = a->q_heads;
    P.scale2 = a->scale * kLog2e;
    P.lens = a->lens;
    P.out = a->out;
    P.lse = a->lse;
    P.prior = a->prior;
    P.weights = a->weights;
    P.tiles = (P.Q.rows + 15) / 16;
    P.splits = pick_splits((long long)B * H * P.tiles, P.C.max_tokens, sms);
    unsigned char* ws = static_cast<unsigned char*>(a->workspace);
    P.counters = reinterpret_cast<int*>(ws);
    ws += size_t(kJoinCounters) * 4;
    P.row_blocks = row_blocks(P.Q.rows);
    P.block_rows = (P.Q.rows + P.row_blocks - 1) / P.row_blocks;
    P.ctas = std::min(sms, kMaxCtas);
    P.plan = reinterpret_cast<TilePlan*>(ws);
    P.items = reinterpret_cast<TileItem*>(ws + sizeof(TilePlan));
    cudaStream_t s = as_stream(stream);
    if (P.Q.rows <= kFewRows) {
        P.partial = reinterpret_cast<float*>(ws);
        DLLM_CUDA_TRY(launch_dependent(D == 128 ? kv4_attend_rows_kernel<128> : kv4_attend_rows_kernel<64>,
                                       dim3(P.splits, H * P.tiles, B), dim3(kRowWarps * 32), 0, s, P));
    } else {
        P.partial = reinterpret_cast<float*>(ws + sizeof(TilePlan) + max_items(a->cache, P.Q.rows) * sizeof(TileItem));
        rc = launch_attend_tiles(P, D, s);
        if (rc != DLLM_OK) return rc;
    }
    if (a->weights && P.Q.rows > kFewRows) return launch_weight_tiles(P, D, s);
    if (a->weights) {
        const unsigned gx = (P.C.max_tokens + kWeightWarps * 32 - 1) / (kWeightWarps * 32);
        DLLM_CUDA_TRY(launch_dependent(D == 128 ? kv4_weights_kernel<128> : kv4_weights_kernel<64>, dim3(gx, H, B),
                                       dim3(kWeightWarps * 32), 0, s, P));
    }
    return DLLM_OK;
}
