// dllm_kv4_attend for many query rows: 128-token tiles through the tensor cores.
//
// Three launches: kv4_plan_kernel lays out the work, kv4_tile_kernel does it,
// kv4_join_kernel joins what was cut.
//
// Plan.  A unit is (request, key/value head, block of up to 256 query rows) and
// has ceil(len / 128) tiles.  Units are cut into pieces of at most C tiles, the
// smallest C that leaves no more pieces than CTAs when units are few, an even
// share of all tiles otherwise (so only units longer than that are cut), never
// under 8 tiles.  Items go out longest first, forwards and backwards over the
// CTAs in turn, so that every CTA gets about the same number of tiles.
//
// Tile kernel: one CTA per SM, warps with roles, all running through the CTA's
// items without a common barrier:
//   warps 0-7   two streams of four softmax warps, a thread per row;
//   warps 8-11  widen codes to fp16 tiles in shared memory, and the queries;
//   warp 12     issues the tensor-core products.
// A stream holds 128 rows' scores S (128 columns of TMEM) and output O (D
// columns).  With more than 128 rows the streams hold different rows of the same
// tiles; with fewer they take the tiles in turn, each with sums of its own, and
// are joined at the end.  While one stream's softmax runs the tensor cores serve
// the other.  Softmax weights go back to TMEM over the scores they came from, in
// fp16, as the A operand of the product with the values.  The two products of a
// tile and stream cost 4 x 128 x 128 x D operations whatever the rows, so the
// kernel is bound by the tensor cores (2 x 512 cycles per tile and stream at
// D = 128) when the rows fill the streams.
//
// Codes go from global memory to registers (one half-tile ahead) to the fp16
// tile: 16 bytes of codes make 64 bytes of tile, so shared memory is crossed
// once.  Tiles are 128-byte-swizzled; eight lanes that store together take 4
// tokens x 2 groups, which the swizzle spreads over all banks.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kv4_attend.cuh"
#include "tcgen05.cuh"

namespace dllm {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;   // any single wait gives up after 2 s
constexpr int kSoftWarps = 8, kWidenWarps = 4;
constexpr int kTileThreads = (kSoftWarps + kWidenWarps + 1) * 32;
constexpr int kMinPiece = 8;   // tiles; shorter pieces cost more to join than they save

// ---------------------------------------------------------------------------
// Plan: one CTA
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 1024;   // piece lengths, longer ones together

__device__ __forceinline__ long long block_sum(long long v, long long* s_red) {
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    long long t = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) t += s_red[w];
    return t;
}

__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const __grid_constant__ AttendParams P) {
    __shared__ long long s_red[kPlanThreads / 32];
    __shared__ int s_bin[kPlanBins];
    __shared__ int s_split, s_slot;
    pdl_wait();
    pdl_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = P.C.heads * P.row_blocks;   // units of a request
    const int B = P.C.B;
    long long mine = 0;
    for (int b = tid; b < B; b += kPlanThreads) mine += (kv4_len(P.C, P.lens, b) + kTileTokens - 1) / kTileTokens;
    const long long total = block_sum(mine, s_red) * per;
    long long C = max((total + P.ctas - 1) / P.ctas, (long long)kMinPiece);
    if ((long long)B * per <= P.ctas && total > 0) {
        // smallest C with no more pieces than CTAs: any C of at least the longest unit will do
        long long lo = C, hi = max(C, (long long)(P.C.max_tokens / kTileTokens + 1));
        while (lo < hi) {
            const long long mid = (lo + hi) / 2;
            long long p = 0;
            for (int b = tid; b < B; b += kPlanThreads) {
                const long long n = (kv4_len(P.C, P.lens, b) + kTileTokens - 1) / kTileTokens;
                p += max((n + mid - 1) / mid, 1ll);
            }
            if (block_sum(p, s_red) * per <= P.ctas) hi = mid;
            else lo = mid + 1;
        }
        C = lo;
    }
    // items per piece length, longest first
    for (int i = tid; i < kPlanBins; i += kPlanThreads) s_bin[i] = 0;
    if (tid == 0) s_split = s_slot = 0;
    __syncthreads();
    for (int b = tid; b < B; b += kPlanThreads) {
        const int n = (kv4_len(P.C, P.lens, b) + kTileTokens - 1) / kTileTokens;
        const int pieces = max((int)((n + C - 1) / C), 1);
        const int size = (n + pieces - 1) / pieces;
        atomicAdd(&s_bin[kPlanBins - 1 - min(size, kPlanBins - 1)], pieces * per);
    }
    __syncthreads();
    {   // exclusive scan, one bin per thread
        const int v = s_bin[tid];
        int x = v;
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) s_red[warp] = x;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < warp; ++w) before += (int)s_red[w];
        s_bin[tid] = before + x - v;
        if (tid == kPlanThreads - 1) P.plan->items = before + x;
    }
    __syncthreads();
    for (int b = warp; b < B; b += kPlanThreads / 32) {   // a warp per request
        const int n = (kv4_len(P.C, P.lens, b) + kTileTokens - 1) / kTileTokens;
        const int pieces = max((int)((n + C - 1) / C), 1);
        const int size = (n + pieces - 1) / pieces;
        int at = 0, split = 0, slot = 0;
        if (lane == 0) {
            at = atomicAdd(&s_bin[kPlanBins - 1 - min(size, kPlanBins - 1)], pieces * per);
            if (pieces > 1) {
                split = atomicAdd(&s_split, per);
                slot = atomicAdd(&s_slot, pieces * per);
            }
        }
        at = __shfl_sync(0xffffffffu, at, 0);
        split = __shfl_sync(0xffffffffu, split, 0);
        slot = __shfl_sync(0xffffffffu, slot, 0);
        for (int i = lane; i < pieces * per; i += 32) {
            const int unit = i / pieces, piece = i - unit * pieces;
            TileItem t;
            t.b = b;
            t.head = unit / P.row_blocks;
            t.rb = unit - t.head * P.row_blocks;
            t.t0 = (int)((long long)n * piece / pieces);
            t.t1 = (int)((long long)n * (piece + 1) / pieces);
            t.slot = pieces > 1 ? slot + i : -1;
            t.pad[0] = t.pad[1] = 0;
            P.items[at + i] = t;
            if (pieces > 1 && piece == 0) {
                TileSplit s;
                s.b = b;
                s.head = t.head;
                s.rb = t.rb;
                s.slot0 = slot + i;
                s.pieces = pieces;
                s.pad[0] = s.pad[1] = s.pad[2] = 0;
                P.plan->split[split + unit] = s;
            }
        }
    }
    __syncthreads();
    if (tid == 0) P.plan->splits = s_split;
}

// The k-th item of CTA c: forwards over the CTAs, then backwards, in turn.
__device__ __forceinline__ int item_index(int k, int c, int ctas) { return k * ctas + ((k & 1) ? ctas - 1 - c : c); }

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
constexpr uint32_t kBlockBytes = kTileTokens * 128;   // 128 rows of 64 channels

template <bool kRows2>
struct TileShared {
    uint64_t full[8], empty[8];       // ring of widened half-tiles
    uint64_t q_full[2], q_empty;      // by item parity: staging may run two items ahead of the softmax
    uint64_t s_full[2], p_ready[2], o_done[2];
    uint64_t pair[4];                 // the two warps of the same rows, where the streams share them
    uint32_t tmem;
    int abort;
    float row_scale[2][kRows2 ? 256 : 128];   // by item parity
    float m[2][kRows2 ? 1 : 128], l[2][kRows2 ? 1 : 128];   // the streams' sums, where they are joined
};

template <int D, bool kRows2>   // kRows2: the streams hold different rows
struct TileShape {
    static constexpr int kBlocks = D / 64;                      // 64-channel blocks of a tile
    static constexpr uint32_t kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kQueryTiles = kRows2 ? 2 : 1;
    static constexpr int kSlots = 5;   // half-tiles of the ring
    static constexpr uint32_t kTiles = (kQueryTiles + kSlots) * kTileBytes;
    static constexpr size_t kSmem = kTiles + sizeof(TileShared<kRows2>);
    static_assert(kSmem <= 232448, "227 KB per CTA");
};

// What a widening thread does: 16 bytes of codes (a token's group of 32 channels)
// of D/32 tokens of a half-tile.  Eight lanes that store together take 4 tokens
// x 2 groups.
template <int D>
struct Widen {
    static constexpr int kEach = D / 32;
    static constexpr int kStep = D == 128 ? 32 : 64;   // tokens between a thread's pieces
    int group, token0;
    uint32_t block_off;
    const uint8_t* page[kEach];
    uint4 w[kEach];          // of the half-tile fetched last
    uint16_t par[kEach];

    __device__ __forceinline__ Widen(int warp, int lane) {
        const int q4 = lane >> 3, tk = (lane & 7) >> 1, gg = lane & 1;
        group = D == 128 ? (q4 & 1) * 2 + gg : gg;
        token0 = D == 128 ? warp * 8 + (q4 >> 1) * 4 + tk : warp * 16 + q4 * 4 + tk;
        block_off = (uint32_t)(group >> 1) * kBlockBytes;
    }
    // The pages of tile t of (b, head), n tokens long.
    __device__ __forceinline__ void find(const Kv4& C, int b, int head, int n, int t) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int j = t * kTileTokens + token0 + i * kStep;
            page[i] = nullptr;
            if (j < n) page[i] = kv4_page(C, C.table, b, j >> C.page_shift, C.max_pages, head);
        }
    }
    // Start loading the tile's keys (which 0) or values (1).
    __device__ __forceinline__ void fetch(const Kv4& C, int t, int which) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int slot = (t * kTileTokens + token0 + i * kStep) & ((1 << C.page_shift) - 1);
            w[i] = make_uint4(0, 0, 0, 0);
            par[i] = 0;
            if (page[i]) {
                const uint8_t* p = page[i] + (which ? C.head_bytes / 2 : 0);
                w[i] = __ldcs(reinterpret_cast<const uint4*>(p + slot * (D / 2)) + group);
                par[i] = __ldcs(reinterpret_cast<const uint16_t*>(p + ((D / 2) << C.page_shift) + slot * (D / 16)) + group);
            }
        }
    }
    // Widen what was fetched into `tile`; tokens past the end become zeros.
    __device__ __forceinline__ void store(unsigned char* tile, int valid) const {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int token = token0 + i * kStep;
            Kv4Scale sc = kv4_scale(kv4_splat(par[i]));
            if (token >= valid) sc.s = sc.c = 0;
            const uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            unsigned char* row = tile + block_off + token * 128;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint4 o;
                kv4_widen(words[e], sc, o.x, o.y, o.z, o.w);
                *reinterpret_cast<uint4*>(row + ((((group & 1) * 4 + e) ^ (token & 7)) << 4)) = o;
            }
        }
    }
};

// Queries row0 .. row0 + rows of (b, head) as fp16 rows of `tiles` (128 rows to
// a tile, zeros past `rows` up to `padded`): each row's largest brought into
// [1, 2) by a power of two, negated when the scale is negative.  Four warps call;
// 8 lanes hold a row.  done(r, up) receives the row's inverse power.
template <int D, typename Done>
__device__ __forceinline__ void stage_queries(const AttendParams& P, unsigned char* tiles, int b, int head, int row0,
                                              int rows, int padded, int warp, int lane, Done done) {
    const float sign = P.scale2 < 0.0f ? -1.0f : 1.0f;
    constexpr int kCh = D / 8;   // channels per lane: 16 or 8
    for (int r0 = warp * 4; r0 < padded; r0 += kWidenWarps * 4) {
        const int r = r0 + (lane >> 3), part = lane & 7;
        uint32_t v[kCh / 2];
#pragma unroll
        for (int i = 0; i < kCh / 2; ++i) v[i] = 0;
        if (r < rows) {
            const uint4* src = reinterpret_cast<const uint4*>(P.Q.at(b, head, row0 + r) + part * kCh);
#pragma unroll
            for (int i = 0; i < kCh / 8; ++i) {
                const uint4 x = __ldg(src + i);
                v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
            }
        }
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kCh / 2; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(v[i])), fabsf(bf16_hi(v[i]))));
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        float down, up;
        row_power(amax, down, up);
        if (part == 0) done(r, up);
        down *= sign;
#pragma unroll
        for (int i = 0; i < kCh / 2; ++i) v[i] = pack_h2(bf16_lo(v[i]) * down, bf16_hi(v[i]) * down);
        unsigned char* row = tiles + (r >> 7) * (D / 64 * kBlockBytes) + (r & 127) * 128;
#pragma unroll
        for (int i = 0; i < kCh / 8; ++i) {
            const int piece = part * (kCh / 8) + i;   // 16-byte piece of the row, over all blocks
            *reinterpret_cast<uint4*>(row + (piece >> 3) * kBlockBytes + (((piece & 7) ^ (r & 7)) << 4)) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
    }
}

// One bounded wait; false once any wait of the CTA has given up.
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, int* abort_flag, int* err) {
    if (!mbar_wait_bounded(bar, parity, kWaitNs)) {
        set_error(err, DLLM_DEVERR_TIMEOUT);
        *(volatile int*)abort_flag = 1;
    }
    return *(volatile int*)abort_flag == 0;
}
// Leave the enclosing loop when a wait has given up: a whole warp at once, or one thread.
#define TILE_WAIT(bar, parity) \
    if (!__all_sync(0xffffffffu, tile_wait((bar), (parity), &sh.abort, P.C.err))) break;
#define TILE_WAIT_ONE(bar, parity) \
    if (!tile_wait((bar), (parity), &sh.abort, P.C.err)) break;

template <int D, bool kRows2>
__global__ void __launch_bounds__(kTileThreads, 1) kv4_tile_kernel(const __grid_constant__ AttendParams P) {
    using T = TileShape<D, kRows2>;
    extern __shared__ __align__(1024) unsigned char tiles[];   // swizzle atoms are 1024 bytes
    TileShared<kRows2>& sh = *reinterpret_cast<TileShared<kRows2>*>(tiles + T::kTiles);
    const uint32_t base = smem_addr(tiles);
    const uint32_t ring = base + T::kQueryTiles * T::kTileBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        sh.abort = 0;
        for (int i = 0; i < T::kSlots; ++i) {
            mbar_init(smem_addr(&sh.full[i]), kWidenWarps);
            mbar_init(smem_addr(&sh.empty[i]), 1);
        }
        mbar_init(smem_addr(&sh.q_empty), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&sh.q_full[s]), kWidenWarps);
            mbar_init(smem_addr(&sh.s_full[s]), 1);
            mbar_init(smem_addr(&sh.p_ready[s]), kSoftWarps / 2);
            mbar_init(smem_addr(&sh.o_done[s]), 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(smem_addr(&sh.pair[i]), 2);
        mbar_fence_init();
    }
    if (warp == kSoftWarps + kWidenWarps) tmem_alloc(smem_addr(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // TMEM columns: S0, S1 (128 each), O0, O1 (D each)
    pdl_wait();
    pdl_release();
    const int n_items = P.plan->items;

    if (warp < kSoftWarps) {
        // ------------------------------------------------------------ softmax
        const int st = warp >> 2, quad = warp & 3;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lanes + st * 128, tO = tmem + lanes + 256 + st * D;
        const uint32_t bar_s = smem_addr(&sh.s_full[st]), bar_p = smem_addr(&sh.p_ready[st]);
        uint32_t count = 0;       // tiles of this stream so far
        uint32_t outs = 0;        // items with tiles of this stream so far
        uint32_t outs_other = 0;
        uint32_t used = 0;        // items with tiles so far
        for (int k = 0, idx; (idx = item_index(k, blockIdx.x, P.ctas)) < n_items; ++k) {
            const TileItem it = P.items[idx];
            const int n = kv4_len(P.C, P.lens, it.b);
            const int row0 = it.rb * P.block_rows;
            const int rows = min(P.block_rows, P.Q.rows - row0);
            const int row = (kRows2 ? st * 128 : 0) + quad * 32 + lane;   // of the item
            const bool live = (kRows2 ? st * 128 : 0) + quad * 32 < rows;   // the warp has rows
            float rs = 0.0f;
            if (it.t0 + (kRows2 ? 0 : st) < it.t1) {   // a stream without tiles may be items behind: it does not look
                TILE_WAIT(smem_addr(&sh.q_full[used & 1]), used >> 1 & 1)
                rs = sh.row_scale[used & 1][row];
            }
            float m = -INFINITY, l = 0.0f;
            bool stop = false;
            int done = 0;
            for (int t = it.t0 + (kRows2 ? 0 : st); t < it.t1; t += kRows2 ? 1 : 2, ++done, ++count) {
                stop = true;
                TILE_WAIT(bar_s, count & 1)
                stop = false;
                tc_fence_after();
                if (live) {
                    const int left = n - t * kTileTokens;   // valid columns
                    float mx = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tc_ld32(r, tS + c * 32);
                        tc_wait_ld();
                        if (left >= kTileTokens) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(r[i]));
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c * 32 + i < left) mx = fmaxf(mx, __uint_as_float(r[i]));
                        }
                    }
                    mx *= rs;
                    if (__any_sync(0xffffffffu, mx > m + kAbove)) {
                        const float mn = fmaxf(m, mx - kBelow);
                        const float f = m == -INFINITY ? 0.0f : ex2_approx(m - mn);
                        m = mn;
                        l *= f;
                        if (done > 0) {   // the product that last wrote O came before this tile's scores
#pragma unroll
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t r[32];
                                tc_ld32(r, tO + c * 32);
                                tc_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                                tc_st32(tO + c * 32, r);
                            }
                            tc_wait_st();
                        }
                    }
                    float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32], p[16];
                        tc_ld32(r, tS + c * 32);
                        tc_wait_ld();
                        if (left < kTileTokens) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c * 32 + i >= left) r[i] = 0xff800000u;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                // rs is not negative: -inf stays -inf (or, times 0, becomes NaN: kept out)
                                const float a = c * 32 + 2 * i < left ? ex2_approx(fmaf(__uint_as_float(r[2 * i]), rs, -m)) : 0.0f;
                                const float b = c * 32 + 2 * i + 1 < left ? ex2_approx(fmaf(__uint_as_float(r[2 * i + 1]), rs, -m)) : 0.0f;
                                l0 += a;
                                l1 += b;
                                p[i] = pack_h2(a, b);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float a = ex2_approx(fmaf(__uint_as_float(r[2 * i]), rs, -m));
                                const float b = ex2_approx(fmaf(__uint_as_float(r[2 * i + 1]), rs, -m));
                                l0 += a;
                                l1 += b;
                                p[i] = pack_h2(a, b);
                            }
                        }
                        tc_st16(tS + c * 16, p);   // over scores already read
                    }
                    l += l0 + l1;
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p);
            }
            if (stop) break;
            // the item's end
            const int tiles_all = it.t1 - it.t0;
            if (done > 0) {
                TILE_WAIT(smem_addr(&sh.o_done[st]), outs & 1)
                ++outs;
            }
            const long long at = live && row < rows ? P.row_at(it.b, it.head, row0 + row) : 0;
            float* const slot = it.slot < 0 ? nullptr : P.partial + (size_t)it.slot * (kTileRows * (D + 2));
            float f0 = 1.0f, f1 = 0.0f;
            int c0 = 0, c1 = D / 32;
            if (!kRows2 && tiles_all > 0) {
                // both streams hold sums of the same rows: exchange them, each then writes half the channels
                const int other_tiles = tiles_all - done;
                if (other_tiles > 0) {
                    TILE_WAIT(smem_addr(&sh.o_done[st ^ 1]), outs_other & 1)
                    ++outs_other;
                }
                sh.m[st][quad * 32 + lane] = m;
                sh.l[st][quad * 32 + lane] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.pair[quad]));
                TILE_WAIT(smem_addr(&sh.pair[quad]), 0)   // two phases an item
                const float m0 = sh.m[0][quad * 32 + lane], m1 = sh.m[1][quad * 32 + lane];
                const float l0 = sh.l[0][quad * 32 + lane], l1 = sh.l[1][quad * 32 + lane];
                m = fmaxf(m0, m1);
                f0 = m0 == -INFINITY ? (l0 == 0.0f ? 0.0f : 1.0f) : ex2_approx(m0 - m);
                f1 = m1 == -INFINITY ? (l1 == 0.0f ? 0.0f : 1.0f) : ex2_approx(m1 - m);
                l = f0 * l0 + f1 * l1;
            }
            if constexpr (!kRows2) {
                c0 = st * (D / 64);
                c1 = c0 + D / 64;
            }
            tc_fence_after();
            if (live) {
                const bool has = tiles_all > 0;
                const float inv = !has ? 0.0f : slot ? 1.0f : 1.0f / l;
                for (int c = c0; c < c1; ++c) {
                    uint32_t r[32];
                    if constexpr (kRows2) {
                        if (has) {
                            tc_ld32(r, tO + c * 32);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * inv);
                        }
                    } else {
                        if (has) {
                            // O0 holds something whenever there are tiles; O1 when there are two
                            tc_ld32(r, tmem + lanes + 256 + c * 32);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f0);
                            if (tiles_all > 1) {
                                uint32_t q[32];
                                tc_ld32(q, tmem + lanes + 256 + D + c * 32);
                                tc_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    r[i] = __float_as_uint(fmaf(__uint_as_float(q[i]), f1, __uint_as_float(r[i])));
                            }
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * inv);
                        }
                    }
                    if (!has) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = 0;
                    }
                    if (row < rows) {
                        if (slot) {
                            float4* dst = reinterpret_cast<float4*>(slot + row * D + c * 32);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                dst[i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                                     __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
                        } else {
                            uint4* dst = reinterpret_cast<uint4*>(P.out + at * D + c * 32);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    w[e] = pack_bf2(__uint_as_float(r[8 * i + 2 * e]), __uint_as_float(r[8 * i + 2 * e + 1]));
                                dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                }
                if (row < rows && (kRows2 || st == 0)) {
                    if (slot) {
                        slot[kTileRows * D + row] = m;
                        slot[kTileRows * (D + 1) + row] = l;
                    } else if (P.lse) {
                        P.lse[at] = has ? (m + log2f(l)) * kLn2 : -INFINITY;
                    }
                }
            }
            tc_fence_before();
            if (!kRows2 && tiles_all > 0) {   // O0, O1 and the sums are free
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.pair[quad]));
                TILE_WAIT(smem_addr(&sh.pair[quad]), 1)
            }
            used += tiles_all > 0;
        }
    } else if (warp < kSoftWarps + kWidenWarps) {
        // ------------------------------------------------------------ widening
        const int w = warp - kSoftWarps;
        Widen<D> wd(w, lane);
        uint32_t half = 0;   // half-tiles so far
        uint32_t used = 0;   // items with tiles so far
        for (int k = 0, idx; (idx = item_index(k, blockIdx.x, P.ctas)) < n_items; ++k) {
            const TileItem it = P.items[idx];
            if (it.t0 == it.t1) continue;
            const int n = kv4_len(P.C, P.lens, it.b);
            const int row0 = it.rb * P.block_rows;
            const int rows = min(P.block_rows, P.Q.rows - row0);
            wd.find(P.C, it.b, it.head, n, it.t0);
            wd.fetch(P.C, it.t0, 0);
            if (used > 0) {
                TILE_WAIT(smem_addr(&sh.q_empty), (used - 1) & 1)
            }
            float* scale = sh.row_scale[used & 1];
            const float s2 = fabsf(P.scale2);
            stage_queries<D>(P, tiles, it.b, it.head, row0, rows, T::kQueryTiles * 128, w, lane,
                             [&](int r, float up) { scale[r] = s2 * up; });
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[used & 1]));
            bool stop = false;
            for (int t = it.t0; t < it.t1 && !stop; ++t) {
#pragma unroll 1
                for (int which = 0; which < 2; ++which, ++half) {
                    const Widen<D> cur = wd;
                    if (which == 0) {
                        wd.fetch(P.C, t, 1);
                    } else if (t + 1 < it.t1) {
                        wd.find(P.C, it.b, it.head, n, t + 1);
                        wd.fetch(P.C, t + 1, 0);
                    }
                    const uint32_t s = half % T::kSlots;
                    stop = true;
                    TILE_WAIT(smem_addr(&sh.empty[s]), (half / T::kSlots & 1) ^ 1)
                    stop = false;
                    cur.store(tiles + (T::kQueryTiles + s) * T::kTileBytes, n - t * kTileTokens);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.full[s]));
                }
            }
            if (stop) break;
            ++used;
        }
    } else if (lane == 0) {
        // ------------------------------------------------------------ products
        constexpr uint32_t kScoreDesc = tc_idesc(128, kTileTokens, false);
        constexpr uint32_t kValueDesc = tc_idesc(128, D, true);
        uint32_t half = 0;            // half-tiles consumed before this item
        uint32_t p_count[2] = {0, 0};
        uint32_t used = 0;            // items with tiles so far
        for (int k = 0, idx; (idx = item_index(k, blockIdx.x, P.ctas)) < n_items; ++k) {
            const TileItem it = P.items[idx];
            const int nt = it.t1 - it.t0;
            if (nt == 0) continue;
            TILE_WAIT_ONE(smem_addr(&sh.q_full[used & 1]), used >> 1 & 1)
            ++used;
            // half-tile 2 t holds tile t's keys, 2 t + 1 its values
            auto slot_of = [&](int h) { return (half + h) % T::kSlots; };
            auto phase_of = [&](int h) { return ((half + h) / T::kSlots) & 1; };
            auto scores = [&](int st, int t) {
                const uint32_t a = base + (kRows2 ? st : 0) * T::kTileBytes, b = ring + slot_of(2 * t) * T::kTileBytes;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const uint32_t off = (c >> 2) * kBlockBytes + (c & 3) * 32;
                    tc_mma_ss(tmem + st * 128, tc_desc(a + off, 16, 1024), tc_desc(b + off, 16, 1024), kScoreDesc, c > 0);
                }
                tc_commit(smem_addr(&sh.s_full[st]));
            };
            auto values = [&](int st, int t, bool acc) {
                const uint32_t b = ring + slot_of(2 * t + 1) * T::kTileBytes;
#pragma unroll
                for (int c = 0; c < kTileTokens / 16; ++c)
                    tc_mma_ts(tmem + 256 + st * D, tmem + st * 128 + c * 8, tc_desc(b + c * 2048, kBlockBytes, 1024),
                              kValueDesc, acc || c > 0);
            };
            bool stop = false;
            do {
                stop = true;
                TILE_WAIT_ONE(smem_addr(&sh.full[slot_of(0)]), phase_of(0))
                tc_fence_after();
                scores(0, 0);
                if (kRows2) scores(1, 0);
                tc_commit(smem_addr(&sh.empty[slot_of(0)]));
                if (!kRows2 && nt > 1) {
                    TILE_WAIT_ONE(smem_addr(&sh.full[slot_of(2)]), phase_of(2))
                    tc_fence_after();
                    scores(1, 1);
                    tc_commit(smem_addr(&sh.empty[slot_of(2)]));
                }
                if (nt <= (kRows2 ? 1 : 2)) tc_commit(smem_addr(&sh.q_empty));
                stop = false;
            } while (false);
            for (int t = 0; t < nt && !stop; ++t) {
#pragma unroll 1
                for (int u = 0; u < (kRows2 ? 2 : 1); ++u) {
                    const int st = kRows2 ? u : t & 1;
                    const int ahead = t + (kRows2 ? 1 : 2);   // the stream's next tile
                    stop = true;
                    if (u == 0) {
                        TILE_WAIT_ONE(smem_addr(&sh.full[slot_of(2 * t + 1)]), phase_of(2 * t + 1))
                    }
                    TILE_WAIT_ONE(smem_addr(&sh.p_ready[st]), p_count[st] & 1)
                    ++p_count[st];
                    tc_fence_after();
                    values(st, t, t >= (kRows2 ? 1 : 2));
                    if (!kRows2 || u == 1) tc_commit(smem_addr(&sh.empty[slot_of(2 * t + 1)]));
                    if (ahead < nt) {
                        if (u == 0) {
                            TILE_WAIT_ONE(smem_addr(&sh.full[slot_of(2 * ahead)]), phase_of(2 * ahead))
                            tc_fence_after();
                        }
                        scores(st, ahead);
                        if (!kRows2 || u == 1) {
                            tc_commit(smem_addr(&sh.empty[slot_of(2 * ahead)]));
                            if (ahead == nt - 1) tc_commit(smem_addr(&sh.q_empty));   // the item's last scores
                        }
                    } else {
                        tc_commit(smem_addr(&sh.o_done[st]));
                    }
                    stop = false;
                }
            }
            if (stop) break;
            half += 2 * nt;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps + kWidenWarps) {
        tc_fence_after();
        if (sh.abort) __nanosleep(1000000);   // products still in flight end before their TMEM goes
        tmem_free(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// The tokens' weights, many rows: the scores again, tokens down the lanes
// ---------------------------------------------------------------------------
// S^T = K Q^T: a tile's 128 tokens are the rows of the product and all of up to
// 256 query rows its columns, so a thread owns a token and adds 2^(s - lse) over
// the columns by itself: no maximum, no exchange, no atomics.  Two tiles' scores
// (256 columns each) fill TMEM; four warps work on one while the tensor cores
// write the other.  Column (row of queries) facts come from shared memory, two
// columns to a 16-byte broadcast: scales and negated lse, for packed f32 fmas.
struct WeightShared {
    uint64_t full[4], empty[4];
    uint64_t q_full[2], q_empty, cols_empty[2];   // by use parity
    uint64_t s_full[2], s_empty[2];
    uint32_t tmem;
    int abort;
    float4 cols[2][kTileRows / 2];   // by use parity: (scale, scale, -lse, -lse) of two rows
};
template <int D>
struct WeightShape {
    static constexpr uint32_t kTileBytes = D / 64 * kBlockBytes;
    static constexpr int kSlots = 4;
    static constexpr uint32_t kTiles = (2 + kSlots) * kTileBytes;
    static constexpr size_t kSmem = kTiles + sizeof(WeightShared);
};

__device__ __forceinline__ unsigned long long pack_f2(float lo, float hi) {
    return ((unsigned long long)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}

template <int D>
__global__ void __launch_bounds__(kTileThreads, 1) kv4_weight_tile_kernel(const __grid_constant__ AttendParams P) {
    using T = WeightShape<D>;
    extern __shared__ __align__(1024) unsigned char tiles[];
    WeightShared& sh = *reinterpret_cast<WeightShared*>(tiles + T::kTiles);
    const uint32_t base = smem_addr(tiles), ring = base + 2 * T::kTileBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        sh.abort = 0;
        for (int i = 0; i < T::kSlots; ++i) {
            mbar_init(smem_addr(&sh.full[i]), kWidenWarps);
            mbar_init(smem_addr(&sh.empty[i]), 1);
        }
        mbar_init(smem_addr(&sh.q_empty), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&sh.q_full[s]), kWidenWarps);
            mbar_init(smem_addr(&sh.cols_empty[s]), kSoftWarps);
            mbar_init(smem_addr(&sh.s_full[s]), 1);
            mbar_init(smem_addr(&sh.s_empty[s]), kSoftWarps / 2);
        }
        mbar_fence_init();
    }
    if (warp == kSoftWarps + kWidenWarps) tmem_alloc(smem_addr(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    pdl_wait();
    pdl_release();
    const int n_items = P.plan->items;
    const int blocks = (P.Q.rows + kTileRows - 1) / kTileRows;
    const int block_rows = (P.Q.rows + blocks - 1) / blocks;
    const int cols = (block_rows + 31) & ~31;   // columns of the product; queries past the rows are zeros

    if (warp < kSoftWarps) {
        const int buf = warp >> 2, quad = warp & 3;
        const uint32_t tS = tmem + ((uint32_t)(quad * 32) << 16) + buf * 256;
        uint32_t tile = 0, used = 0;   // this buffer's tiles and uses of the queries so far
        bool stop = false;
        for (int k = 0, idx; !stop && (idx = item_index(k, blockIdx.x, P.ctas)) < n_items; ++k) {
            const TileItem it = P.items[idx];
            if (it.t0 == it.t1) continue;
            const int n = kv4_len(P.C, P.lens, it.b);
            for (int rb = 0; rb < blocks && !stop; ++rb, ++used) {
                stop = true;
                TILE_WAIT(smem_addr(&sh.q_full[used & 1]), used >> 1 & 1)
                stop = false;
                const float4* col = sh.cols[used & 1];
                // a token's tile takes the same buffer for every block of rows: its thread adds to its own sums
                for (int t = it.t0 + ((k ^ buf) & 1); t < it.t1; t += 2, ++tile) {
                    stop = true;
                    TILE_WAIT(smem_addr(&sh.s_full[buf]), tile & 1)
                    stop = false;
                    tc_fence_after();
                    unsigned long long acc[4] = {0, 0, 0, 0};
                    for (int c = 0; c < cols; c += 32) {
                        uint32_t r[32];
                        tc_ld32(r, tS + c);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float4 f = col[c / 2 + i];
                            unsigned long long x = pack_f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                            asm("{\n\t.reg .b32 l, h;\n\t"
                                "fma.rn.f32x2 %0, %0, %2, %3;\n\t"
                                "mov.b64 {l, h}, %0;\n\t"
                                "ex2.approx.ftz.f32 l, l;\n\t"
                                "ex2.approx.ftz.f32 h, h;\n\t"
                                "mov.b64 %0, {l, h};\n\t"
                                "add.rn.f32x2 %1, %1, %0;\n\t}"
                                : "+l"(x), "+l"(acc[i & 3])
                                : "l"(pack_f2(f.x, f.y)), "l"(pack_f2(f.z, f.w)));
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.s_empty[buf]));
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sum += __uint_as_float((uint32_t)acc[i]) + __uint_as_float((uint32_t)(acc[i] >> 32));
                    const int j = t * kTileTokens + quad * 32 + lane;
                    int page;
                    if (j < n && kv4_page(P.C, P.C.table, it.b, j >> P.C.page_shift, P.C.max_pages, it.head, &page)) {
                        const long long at = (((long long)page * P.C.heads + it.head) << P.C.page_shift) +
                                             (j & ((1 << P.C.page_shift) - 1));
                        const float* from = rb == 0 ? P.prior : P.weights;
                        P.weights[at] = (from ? __ldcg(from + at) : 0.0f) + sum;
                    }
                }
                if (stop) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.cols_empty[used & 1]));
            }
        }
    } else if (warp < kSoftWarps + kWidenWarps) {
        const int w = warp - kSoftWarps;
        Widen<D> wd(w, lane);
        uint32_t tile = 0, used = 0;
        bool stop = false;
        for (int k = 0, idx; !stop && (idx = item_index(k, blockIdx.x, P.ctas)) < n_items; ++k) {
            const TileItem it = P.items[idx];
            if (it.t0 == it.t1) continue;
            const int n = kv4_len(P.C, P.lens, it.b);
            for (int rb = 0; rb < blocks && !stop; ++rb, ++used) {
                wd.find(P.C, it.b, it.head, n, it.t0);
                wd.fetch(P.C, it.t0, 0);
                stop = true;
                if (used > 0) {
                    TILE_WAIT(smem_addr(&sh.q_empty), (used - 1) & 1)
                }
                if (used > 1) {
                    TILE_WAIT(smem_addr(&sh.cols_empty[used & 1]), (used >> 1 & 1) ^ 1)
                }
                stop = false;
                const int row0 = rb * block_rows, rows = min(block_rows, P.Q.rows - row0);
                float* col = reinterpret_cast<float*>(sh.cols[used & 1]);
                const float s2 = fabsf(P.scale2);
                stage_queries<D>(P, tiles, it.b, it.head, row0, rows, cols, w, lane, [&](int r, float up) {
                    float* f = col + (r >> 1) * 4 + (r & 1);
                    f[0] = r < rows ? s2 * up : 0.0f;
                    f[2] = r < rows ? -P.lse[P.row_at(it.b, it.head, row0 + r)] * kLog2e : -INFINITY;
                });
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[used & 1]));
                for (int t = it.t0; t < it.t1; ++t, ++tile) {
                    const Widen<D> cur = wd;
                    if (t + 1 < it.t1) {
                        wd.find(P.C, it.b, it.head, n, t + 1);
                        wd.fetch(P.C, t + 1, 0);
                    }
                    const uint32_t s = tile % T::kSlots;
                    stop = true;
                    TILE_WAIT(smem_addr(&sh.empty[s]), (tile / T::kSlots & 1) ^ 1)
                    stop = false;
                    cur.store(tiles + (2 + s) * T::kTileBytes, n - t * kTileTokens);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.full[s]));
                }
            }
        }
    } else if (lane == 0) {
        const uint32_t idesc = tc_idesc(128, cols, false);
        uint32_t tile = 0, used = 0, bufs[2] = {0, 0};
        bool stop = false;
        for (int k = 0, idx; !stop && (idx = item_index(k, blockIdx.x, P.ctas)) < n_items; ++k) {
            const TileItem it = P.items[idx];
            if (it.t0 == it.t1) continue;
            for (int rb = 0; rb < blocks && !stop; ++rb, ++used) {
                stop = true;
                TILE_WAIT_ONE(smem_addr(&sh.q_full[used & 1]), used >> 1 & 1)
                stop = false;
                for (int t = it.t0; t < it.t1; ++t, ++tile) {
                    const uint32_t s = tile % T::kSlots, buf = (t - it.t0 + k) & 1;
                    stop = true;
                    TILE_WAIT_ONE(smem_addr(&sh.full[s]), tile / T::kSlots & 1)
                    TILE_WAIT_ONE(smem_addr(&sh.s_empty[buf]), (bufs[buf]++ & 1) ^ 1)
                    stop = false;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const uint32_t off = (c >> 2) * kBlockBytes + (c & 3) * 32;
                        const uint64_t a = tc_desc(ring + s * T::kTileBytes + off, 16, 1024);
                        // rows 128.. of the queries are a tile further on: two products when there are any
                        tc_mma_ss(tmem + buf * 256, a, tc_desc(base + off, 16, 1024), cols > 128 ? tc_idesc(128, 128, false) : idesc, c > 0);
                        if (cols > 128)
                            tc_mma_ss(tmem + buf * 256 + 128, a, tc_desc(base + T::kTileBytes + off, 16, 1024),
                                      tc_idesc(128, cols - 128, false), c > 0);
                    }
                    tc_commit(smem_addr(&sh.empty[s]));
                    tc_commit(smem_addr(&sh.s_full[buf]));
                }
                if (!stop) tc_commit(smem_addr(&sh.q_empty));
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps + kWidenWarps) {
        tc_fence_after();
        if (sh.abort) __nanosleep(1000000);
        tmem_free(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Join: a warp per row of a cut unit
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) kv4_join_kernel(const __grid_constant__ AttendParams P) {
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31;
    const int splits = P.plan->splits;
    constexpr int kPer = D / 32;
    constexpr size_t kSlot = (size_t)kTileRows * (D + 2);
    const long long total = (long long)splits * P.block_rows;
    for (long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += (long long)gridDim.x * 8) {
        const int s = (int)(w / P.block_rows), row = (int)(w - (long long)s * P.block_rows);
        const TileSplit sp = P.plan->split[s];
        const int r = sp.rb * P.block_rows + row;
        if (r >= P.Q.rows) continue;
        const float* base = P.partial + sp.slot0 * kSlot;
        float m = -INFINITY;
        for (int p = lane; p < sp.pieces; p += 32) m = fmaxf(m, __ldcg(base + p * kSlot + kTileRows * D + row));
#pragma unroll
        for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        float l = 0.0f, acc[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
        for (int p0 = 0; p0 < sp.pieces; p0 += 32) {
            float f = 0.0f, lp = 0.0f;
            if (p0 + lane < sp.pieces) {
                const float* at = base + (p0 + lane) * kSlot + kTileRows * D + row;
                const float mp = __ldcg(at);
                lp = __ldcg(at + kTileRows);
                f = mp == -INFINITY ? 1.0f : ex2_approx(mp - m);   // only NaN sums come with no offset
            }
            const int here = min(32, sp.pieces - p0);
#pragma unroll 8
            for (int p = 0; p < here; ++p) {   // in piece order: equal calls give equal bits
                const float fp = __shfl_sync(0xffffffffu, f, p);
                l += fp * __shfl_sync(0xffffffffu, lp, p);
                const float* at = base + (p0 + p) * kSlot + row * D + lane * kPer;
                if constexpr (kPer == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(at));
                    acc[0] += fp * v.x; acc[1] += fp * v.y; acc[2] += fp * v.z; acc[3] += fp * v.w;
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(at));
                    acc[0] += fp * v.x; acc[1] += fp * v.y;
                }
            }
        }
        const float inv = 1.0f / l;
        const long long at = P.row_at(sp.b, sp.head, r);
        uint32_t* dst = reinterpret_cast<uint32_t*>(P.out + at * D + lane * kPer);
#pragma unroll
        for (int i = 0; i < kPer / 2; ++i) dst[i] = pack_bf2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
        if (lane == 0 && P.lse) P.lse[at] = (m + log2f(l)) * kLn2;
    }
}

template <int D, bool kRows2>
int launch_tile(const AttendParams& P, cudaStream_t s) {
    using T = TileShape<D, kRows2>;
    auto kernel = kv4_tile_kernel<D, kRows2>;
    static SmemOnce done;
    DLLM_CUDA_TRY(allow_smem(kernel, T::kSmem, done));
    DLLM_CUDA_TRY(launch_dependent(kernel, dim3(P.ctas), dim3(kTileThreads), T::kSmem, s, P));
    return DLLM_OK;
}

}  // namespace

int launch_attend_tiles(const AttendParams& P, int D, cudaStream_t s) {
    DLLM_CUDA_TRY(launch_dependent(kv4_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, P));
    int rc;
    if (P.block_rows > 128) rc = D == 128 ? launch_tile<128, true>(P, s) : launch_tile<64, true>(P, s);
    else rc = D == 128 ? launch_tile<128, false>(P, s) : launch_tile<64, false>(P, s);
    if (rc != DLLM_OK) return rc;
    if (P.C.max_tokens > kMinPiece * kTileTokens)   // else nothing is ever cut
        DLLM_CUDA_TRY(launch_dependent(D == 128 ? kv4_join_kernel<128> : kv4_join_kernel<64>, dim3(2 * P.ctas), dim3(256),
                                       0, s, P));
    return DLLM_OK;
}

template <int D>
int launch_weights(const AttendParams& P, cudaStream_t s) {
    auto kernel = kv4_weight_tile_kernel<D>;
    static SmemOnce done;
    DLLM_CUDA_TRY(allow_smem(kernel, WeightShape<D>::kSmem, done));
    DLLM_CUDA_TRY(launch_dependent(kernel, dim3(P.ctas), dim3(kTileThreads), WeightShape<D>::kSmem, s, P));
    return DLLM_OK;
}

int launch_weight_tiles(const AttendParams& P, int D, cudaStream_t s) {
    if (P.row_blocks == 1) return D == 128 ? launch_weights<128>(P, s) : launch_weights<64>(P, s);
    // the weights run over all blocks of rows at once: their items are whole heads
    AttendParams W = P;
    W.row_blocks = 1;
    DLLM_CUDA_TRY(launch_dependent(kv4_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, W));
    return D == 128 ? launch_weights<128>(W, s) : launch_weights<64>(W, s);
}

}  // namespace dllm
