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
//   warps 8-11  widen codes to fp16 tiles in shared memory;
//   warp 12     issues the tensor-core products;
//   warp 13     walks the list of tiles, looks their pages up and copies their
//               codes to shared memory, six half-tiles ahead (bulk copies).
// A softmax thread also brings its row of queries to fp16 in shared memory: it
// loads the next item's row when it has handed over its last weights of this one,
// so that the next item's scores are formed while the output is written.
// A stream holds 128 rows' scores S (128 columns of TMEM) and output O (D
// columns).  With more than 128 rows the streams hold different rows of the same
// tiles; with fewer they take the tiles in turn, each with sums of its own, and
// are joined at the end.  While one stream's softmax runs the tensor cores serve
// the other.  Softmax weights go back to TMEM over the scores they came from, in
// fp16, as the A operand of the product with the values.  The two products of a
// tile and stream cost 4 x 128 x 128 x D operations whatever the rows: 2 x 512
// cycles of the tensor cores per tile and stream at D = 128.
//
// Codes are copied to shared memory by the TMA engine, read from there and
// widened: 16 bytes of codes make 64 bytes of tile.  Six half-tiles of codes, 55
// KB, are in flight per SM.  The issuing thread orders the tiles' generic writes
// before its products' reads (one proxy fence after each wait).  Tiles are
// 128-byte-swizzled; eight lanes that store together take 4 tokens x 2 groups,
// which the swizzle spreads over all banks.
//
// Measured over contexts of 104 and 110 K tokens, 4 heads, 224 rows each (44 tiles a
// CTA): this kernel 121 us, 5.4 thousand cycles a tile, tensor pipes 38 % active,
// issue slots 36 %; the weights' kernel 82 us, 3.6 thousand, 25 % and 37 %.  Neither
// pipe is what they wait for: the roles wait for one another, a tile's widening,
// products and softmax being one chain that the streams and the ring overlap in part.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kv4_attend.cuh"
#include "tcgen05.cuh"

namespace dllm {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;   // any single wait gives up after 2 s
constexpr int kSoftWarps = 8, kWidenWarps = 4;
constexpr int kIssueWarp = kSoftWarps + kWidenWarps, kCopyWarp = kIssueWarp + 1;
constexpr int kTileThreads = (kSoftWarps + kWidenWarps + 4) * 32;   // the last two warps only fill the warpgroup
// Registers per thread: 128 at launch (512 threads); two warpgroups give 32 each to the softmax's two, whose threads
// hold a whole row of scores: 2 x 128 (128 - 96) >= 256 (160 - 128).
constexpr int kLaunchRegs = 128, kSoftRegs = 160, kOtherRegs = 96;
static_assert(256 * (kLaunchRegs - kOtherRegs) >= 256 * (kSoftRegs - kLaunchRegs), "registers given cover those taken");
// The weights' kernel: eight warps add, four widen, one issues, one copies, six bring the queries.
constexpr int kQueryWarps = 6;
constexpr int kWeightThreads = (kSoftWarps + kWidenWarps + 2 + kQueryWarps) * 32;
// Tiles of the shortest piece (4, 16 in brackets), 224 rows a key/value head: one
// request of 4 heads and up to 1600 tokens 33 us (29, 41), of up to 5000 40 (33, 50);
// 2 requests of 32 heads and up to 1600 tokens 50 (49, 41); with more pieces than
// CTAs either way no difference.
constexpr int kMinPiece = 8;

// ---------------------------------------------------------------------------
// Plan: one CTA
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 1024;   // piece lengths, longer ones together

__device__ __forceinline__ long long warp_sum(long long v) {
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const __grid_constant__ AttendParams P) {
    __shared__ long long s_red[kPlanThreads / 32];
    __shared__ int s_bin[kPlanBins];
    __shared__ int4 s_req[kPlanThreads];   // of a chunk of requests: first item, first split, first slot, pieces
    __shared__ int s_split, s_slot;
    pdl_wait();
    pdl_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = P.C.heads * P.row_blocks;   // units of a request
    const int B = P.C.B;
    auto tiles_of = [&](int b) { return (min(max(__ldg(P.lens + b), 0), P.C.max_tokens) + kTileTokens - 1) / kTileTokens; };
    s_bin[tid] = 0;
    if (tid == 0) s_split = s_slot = 0;
    long long mine = 0;
    for (int b = tid; b < B; b += kPlanThreads) mine += tiles_of(b);
    mine = warp_sum(mine);
    if (lane == 0) s_red[warp] = mine;
    __syncthreads();
    const long long total = warp_sum(s_red[lane]) * per;
    long long C = max((total + P.ctas - 1) / P.ctas, (long long)kMinPiece);
    if ((long long)B * per <= P.ctas && total > 0) {
        // smallest C with no more pieces than CTAs (any C of at least the longest unit will do): every warp tries
        // one of 32 lengths between the bounds, until they meet
        long long lo = C, hi = max(C, (long long)(P.C.max_tokens / kTileTokens + 1));
        while (lo < hi) {
            const long long step = (hi - lo + 31) / 32, c = min(lo + warp * step, hi);
            long long p = 0;
            for (int b = lane; b < B; b += 32) p += max((tiles_of(b) + c - 1) / c, 1ll);
            p = warp_sum(p) * per;
            __syncthreads();
            if (lane == 0) s_red[warp] = p <= P.ctas ? c : hi;
            __syncthreads();
            long long best = s_red[lane];   // the smallest length that will do
            for (int off = 16; off; off >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, off));
            lo = max(lo, best - step + 1);  // the one tried before it would not
            hi = best;
            if (best == lo) break;
        }
        C = hi;
    }
    // items per piece length, longest first
    auto pieces_of = [&](int n) { return max((int)((n + C - 1) / C), 1); };
    auto bin_of = [&](int n) { return kPlanBins - 1 - min((n + pieces_of(n) - 1) / pieces_of(n), kPlanBins - 1); };
    __syncthreads();
    for (int b = tid; b < B; b += kPlanThreads) {
        const int n = tiles_of(b);
        atomicAdd(&s_bin[bin_of(n)], pieces_of(n) * per);
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
        long long before = lane < warp ? s_red[lane] : 0;
        before = warp_sum(before);
        s_bin[tid] = (int)before + x - v;
        if (tid == kPlanThreads - 1) P.plan->items = (int)before + x;
    }
    __syncthreads();
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
        if (b0 + tid < B) {   // places, a thread per request
            const int n = tiles_of(b0 + tid), pieces = pieces_of(n);
            int4 r = make_int4(atomicAdd(&s_bin[bin_of(n)], pieces * per), 0, 0, pieces);
            if (pieces > 1) {
                r.y = atomicAdd(&s_split, per);
                r.z = atomicAdd(&s_slot, pieces * per);
            }
            s_req[tid] = r;
        }
        __syncthreads();
        for (int q = warp; q < min(B - b0, kPlanThreads); q += kPlanThreads / 32) {   // items, a warp per request
            const int b = b0 + q, n = tiles_of(b);
            const int4 r = s_req[q];
            const int pieces = r.w;
            for (int i = lane; i < pieces * per; i += 32) {
                const int unit = i / pieces, piece = i - unit * pieces;
                TileItem t;
                t.b = b;
                t.head = unit / P.row_blocks;
                t.rb = unit - t.head * P.row_blocks;
                t.t0 = (int)((long long)n * piece / pieces);
                t.t1 = (int)((long long)n * (piece + 1) / pieces);
                t.slot = pieces > 1 ? r.z + i : -1;
                t.n = kv4_len(P.C, P.lens, b);
                t.pad = 0;
                P.items[r.x + i] = t;
                if (pieces > 1 && piece == 0) {
                    TileSplit s;
                    s.b = b;
                    s.head = t.head;
                    s.rb = t.rb;
                    s.slot0 = r.z + i;
                    s.pieces = pieces;
                    s.pad[0] = s.pad[1] = s.pad[2] = 0;
                    P.plan->split[r.y + unit] = s;
                }
            }
        }
        __syncthreads();
    }
    if (tid == 0) P.plan->splits = s_split;
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
// The ring of half-tiles of codes as they lie in the cache: codes [128][D/2], then
// parameters [128][D/32].
constexpr int kRaw = 6;
struct RawRing {
    uint64_t full[kRaw], empty[kRaw];
    int valid[kRaw];   // tokens up to the request's end, -1: no more tiles
};

constexpr uint32_t kBlockBytes = kTileTokens * 128;   // 128 rows of 64 channels

template <bool kRows2>
struct TileShared {
    uint64_t full[8], empty[8];       // ring of widened half-tiles
    uint64_t q_full[2][2], q_empty;   // by item parity and stream
    uint64_t s_full[2], p_ready[2], o_done[2];
    uint64_t pair[4];                 // the two warps of the same rows, where the streams share them
    RawRing raw;
    uint32_t tmem;
    int abort;
    float row_scale[2][kRows2 ? 1 : 128];     // of rows the streams share, by item parity
    float m[2][kRows2 ? 1 : 128], l[2][kRows2 ? 1 : 128];   // the streams' sums, where they are joined
};

template <int D, bool kRows2>   // kRows2: the streams hold different rows
struct TileShape {
    static constexpr int kBlocks = D / 64;                      // 64-channel blocks of a tile
    static constexpr uint32_t kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kQueryTiles = kRows2 ? 2 : 1;
    static constexpr int kSlots = kRows2 ? 3 : 4;   // half-tiles of the ring
    static constexpr uint32_t kRawBytes = kTileTokens * (D / 2 + D / 16);
    static constexpr uint32_t kRawAt = (kQueryTiles + kSlots) * kTileBytes;
    static constexpr uint32_t kTiles = kRawAt + kRaw * kRawBytes;
    static constexpr size_t kSmem = kTiles + sizeof(TileShared<kRows2>);
    static_assert(kSmem <= 232448, "227 KB per CTA");
};

// The k-th item of CTA c: forwards over the CTAs, then backwards, in turn.
__device__ __forceinline__ int item_index(int k, int c, int ctas) { return k * ctas + ((k & 1) ? ctas - 1 - c : c); }

// The tiles of a CTA's items, one after the other; each item `times` times over.
struct TileCursor {
    int k, n_items, left, times;   // the item after the next; rounds of the current one still to come
    int b, head, n, t, t0, t1;     // the current item and tile; t1 -1: none
    int4 a1, a2;                   // the next item (b, head, rb, t0), (t1, slot, n, -)

    __device__ __forceinline__ void load(const AttendParams& P) {
        const int idx = item_index(k++, blockIdx.x, P.ctas);
        a2.x = -1;
        if (idx < n_items) {
            a1 = *reinterpret_cast<const int4*>(P.items + idx);
            a2 = *(reinterpret_cast<const int4*>(P.items + idx) + 1);
        }
    }
    __device__ __forceinline__ void take(const AttendParams& P) {   // the next item that has tiles
        do {
            b = a1.x; head = a1.y; t0 = a1.w; t1 = a2.x; n = a2.z;
            if (t1 >= 0) load(P);
        } while (t1 >= 0 && t0 == t1);
        t = t0;
        left = times - 1;
    }
    __device__ __forceinline__ TileCursor(const AttendParams& P, int items, int rounds) : k(0), n_items(items), times(rounds) {
        load(P);
        take(P);
    }
    __device__ __forceinline__ void advance(const AttendParams& P) {
        if (t1 >= 0 && ++t == t1) {
            if (left-- > 0) t = t0;
            else take(P);
        }
    }
};

// Widen a half-tile of codes into `tile`; tokens from `valid` on become zeros.  A
// thread takes 16 bytes of codes (a token's group of 32 channels) of D/32 tokens;
// eight lanes that store together take 4 tokens x 2 groups.  kWidenWarps call.
template <int D>
__device__ __forceinline__ void widen_half(unsigned char* tile, const unsigned char* raw, int valid, int warp, int lane) {
    constexpr int kEach = D / 32, kStep = kTileTokens / kEach;
    const int g = D == 128 ? ((lane >> 3) & 1) * 2 + (lane & 1) : lane & 1;
    const int token0 = D == 128 ? warp * 8 + (lane >> 4) * 4 + ((lane & 7) >> 1) : warp * 16 + (lane >> 3) * 4 + ((lane & 7) >> 1);
    uint4 w[kEach];
    uint32_t par[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int token = token0 + i * kStep;
        w[i] = reinterpret_cast<const uint4*>(raw + token * (D / 2))[g];
        par[i] = reinterpret_cast<const uint16_t*>(raw + kTileTokens * (D / 2) + token * (D / 16))[g];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int token = token0 + i * kStep;
        Kv4Scale sc = kv4_scale(kv4_splat(par[i]));
        if (token >= valid) sc.s = sc.c = 0;
        const uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        unsigned char* row = tile + (g >> 1) * kBlockBytes + token * 128;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint4 o;
            kv4_widen(words[e], sc, o.x, o.y, o.z, o.w);
            *reinterpret_cast<uint4*>(row + ((((g & 1) * 4 + e) ^ (token & 7)) << 4)) = o;
        }
    }
}

// Queries row0 .. row0 + rows of (b, head) as fp16 rows of `tiles` (128 rows to
// a tile, zeros past `rows` up to `padded`): each row's largest brought into
// [1, 2) by a power of two, negated when the scale is negative.  kWarps warps call;
// 8 lanes hold a row.  done(r, up) receives the row's inverse power.
template <int D, int kWarps, typename Done>
__device__ __forceinline__ void stage_queries(const AttendParams& P, unsigned char* tiles, int b, int head, int row0,
                                              int rows, int padded, int warp, int lane, Done done) {
    const float sign = P.scale2 < 0.0f ? -1.0f : 1.0f;
    constexpr int kCh = D / 8;                 // channels per lane: 16 or 8
    constexpr int kAtOnce = 4;                 // rows in flight per lane
    constexpr int kRows = kWarps * 4;          // rows per pass of the warps
    const int part = lane & 7;
    for (int r0 = warp * 4 + (lane >> 3); r0 < padded; r0 += kAtOnce * kRows) {
        uint32_t v[kAtOnce][kCh / 2];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int r = r0 + u * kRows;
#pragma unroll
            for (int i = 0; i < kCh / 2; ++i) v[u][i] = 0;
            if (r < rows) {
                const uint4* src = reinterpret_cast<const uint4*>(P.Q.at(b, head, row0 + r) + part * kCh);
#pragma unroll
                for (int i = 0; i < kCh / 8; ++i) {
                    const uint4 x = __ldg(src + i);
                    v[u][4 * i] = x.x; v[u][4 * i + 1] = x.y; v[u][4 * i + 2] = x.z; v[u][4 * i + 3] = x.w;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int r = r0 + u * kRows;
            if (r >= padded) break;   // padded is a multiple of the 4 rows of a warp
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < kCh / 2; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(v[u][i])), fabsf(bf16_hi(v[u][i]))));
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            float down, up;
            row_power(amax, down, up);
            if (part == 0) done(r, up);
            down *= sign;
            unsigned char* row = tiles + (r >> 7) * (D / 64 * kBlockBytes) + (r & 127) * 128;
#pragma unroll
            for (int i = 0; i < kCh / 8; ++i) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = pack_h2(bf16_lo(v[u][4 * i + e]) * down, bf16_hi(v[u][4 * i + e]) * down);
                const int piece = part * (kCh / 8) + i;   // 16-byte piece of the row, over all blocks
                *reinterpret_cast<uint4*>(row + (piece >> 3) * kBlockBytes + (((piece & 7) ^ (r & 7)) << 4)) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

// One bounded wait; false once any wait of the CTA has given up.  A patient one
// sleeps between looks: its warp's work is not the next thing anyone needs, and
// looking takes issue slots from those whose is.
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, int* abort_flag, int* err, bool patient = false) {
    if (patient) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_test_wait(bar, parity)) {
            __nanosleep(200);
            if (*(volatile int*)abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitNs) {
                set_error(err, DLLM_DEVERR_TIMEOUT);
                *(volatile int*)abort_flag = 1;
            }
        }
        return *(volatile int*)abort_flag == 0;
    }
    if (!mbar_wait_bounded(bar, parity, kWaitNs)) {
        set_error(err, DLLM_DEVERR_TIMEOUT);
        *(volatile int*)abort_flag = 1;
    }
    return *(volatile int*)abort_flag == 0;
}
// Leave the enclosing loop when a wait has given up: a whole warp at once, or one thread.
#define TILE_WAIT(bar, parity) \
    if (!__all_sync(0xffffffffu, tile_wait((bar), (parity), &sh.abort, P.C.err))) break;
#define TILE_WAIT_PATIENT(bar, parity) \
    if (!__all_sync(0xffffffffu, tile_wait((bar), (parity), &sh.abort, P.C.err, true))) break;
#define TILE_WAIT_ONE(bar, parity) \
    if (!tile_wait((bar), (parity), &sh.abort, P.C.err)) break;

// The copying warp: the codes of every tile of the CTA's items (each item `times`
// times over), keys then values where asked, then the end.
template <int D, int kHalves>
__device__ __forceinline__ void copy_tiles(const AttendParams& P, RawRing& ring, uint32_t raw, int n_items, int times,
                                           int lane, int* abort_flag) {
    constexpr uint32_t kRawBytes = kTileTokens * (D / 2 + D / 16);
    TileCursor cur(P, n_items, times);
    const int shift = P.C.page_shift, piece = min(1 << shift, kTileTokens);   // tokens of a page in a tile
    const uint64_t policy = l2_policy_evict_first();
    uint32_t e = 0, phase = 1;
    for (;;) {
        const bool more = cur.t1 >= 0;
        const int j0 = cur.t * kTileTokens, left = more ? cur.n - j0 : -1;
        // lane i copies the tile's i-th page
        int page = -1;
        if (lane * piece < min(left, kTileTokens)) {
            page = __ldg(P.C.table + (long long)cur.b * P.C.max_pages + ((j0 + lane * piece) >> shift));
            if ((unsigned)page >= (unsigned)P.C.n_pages) {   // what the ring held stands in
                set_error(P.C.err, DLLM_DEVERR_PAGE);
                page = -1;
            }
        }
        const uint32_t pages = __popc(__ballot_sync(0xffffffffu, page >= 0));
        const uint8_t* src = P.C.pages + ((page < 0 ? 0 : page) * P.C.page_bytes + (uint32_t)cur.head * P.C.head_bytes);
        const int slot = j0 & ((1 << shift) - 1);   // in a page larger than a tile
#pragma unroll
        for (int which = 0; which < kHalves; ++which) {
            if (!__all_sync(0xffffffffu, tile_wait(smem_addr(&ring.empty[e]), phase, abort_flag, P.C.err))) return;
            if (lane == 0) {
                ring.valid[e] = left;
                mbar_arrive_expect_tx(smem_addr(&ring.full[e]), pages * (uint32_t)piece * (D / 2 + D / 16));
            }
            __syncwarp();
            if (page >= 0) {
                const uint32_t dst = raw + e * kRawBytes, bar = smem_addr(&ring.full[e]);
                const uint8_t* from = src + (which ? P.C.head_bytes / 2 : 0u);
                bulk_g2s(dst + lane * piece * (D / 2), from + slot * (D / 2), piece * (D / 2), bar, policy);
                bulk_g2s(dst + kTileTokens * (D / 2) + lane * piece * (D / 16), from + ((D / 2) << shift) + slot * (D / 16),
                         piece * (D / 16), bar, policy);
            }
            if (++e == kRaw) {
                e = 0;
                phase ^= 1;
            }
            if (!more) return;
        }
        cur.advance(P);
    }
}

// The widening warps: every half-tile of codes through the ring of `slots` at `tiles`.
template <int D>
__device__ __forceinline__ void widen_tiles(const AttendParams& P, RawRing& ring, const unsigned char* raw, uint64_t* full,
                                            uint64_t* empty, int slots, unsigned char* tiles, int w, int lane,
                                            int* abort_flag) {
    constexpr uint32_t kBytes = D / 64 * kBlockBytes, kRawBytes = kTileTokens * (D / 2 + D / 16);
    uint32_t e = 0, e_phase = 0, slot = 0, phase = 1;
    for (;;) {
        if (!__all_sync(0xffffffffu, tile_wait(smem_addr(&ring.full[e]), e_phase, abort_flag, P.C.err))) return;
        const int valid = ring.valid[e];
        if (valid < 0) return;
        if (!__all_sync(0xffffffffu, tile_wait(smem_addr(&empty[slot]), phase, abort_flag, P.C.err))) return;
        widen_half<D>(tiles + slot * kBytes, raw + e * kRawBytes, valid, w, lane);
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_addr(&full[slot]));
            mbar_arrive(smem_addr(&ring.empty[e]));
        }
        if (++slot == (uint32_t)slots) {
            slot = 0;
            phase ^= 1;
        }
        if (++e == kRaw) {
            e = 0;
            e_phase ^= 1;
        }
    }
}

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
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(smem_addr(&sh.raw.full[i]), 1);
            mbar_init(smem_addr(&sh.raw.empty[i]), kWidenWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&sh.q_full[0][s]), kSoftWarps / 2);
            mbar_init(smem_addr(&sh.q_full[1][s]), kSoftWarps / 2);
            mbar_init(smem_addr(&sh.s_full[s]), 1);
            mbar_init(smem_addr(&sh.p_ready[s]), kSoftWarps / 2);
            mbar_init(smem_addr(&sh.o_done[s]), 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(smem_addr(&sh.pair[i]), 2);
        mbar_fence_init();
    }
    if (warp == kIssueWarp) tmem_alloc(smem_addr(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // TMEM columns: S0, S1 (128 each), O0, O1 (D each)
    pdl_wait();
    pdl_release();
    if (warp >= kSoftWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    const int n_items = P.plan->items;

    if (warp < kSoftWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ------------------------------------------------------------ softmax
        const int st = warp >> 2, quad = warp & 3;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lanes + st * 128, tO = tmem + lanes + 256 + st * D;
        const uint32_t bar_s = smem_addr(&sh.s_full[st]), bar_p = smem_addr(&sh.p_ready[st]);
        uint32_t count = 0;       // tiles of this stream so far
        uint32_t outs = 0;        // items with tiles of this stream so far
        uint32_t outs_other = 0;
        uint32_t used = 0;        // items with tiles so far
        const int mine = (kRows2 ? st * 128 : 0) + quad * 32 + lane;   // the thread's row of an item
        const bool stages = kRows2 || st == 0;                         // shared rows are the first stream's to bring
        float rs = 0.0f, rs_next = 0.0f;
        // The next item with tiles, from the k-th on: its queries into shared memory.
        auto stage = [&](int k, uint32_t use) -> bool {
            TileItem it;
            int idx;
            do {
                idx = item_index(k++, blockIdx.x, P.ctas);
                if (idx >= n_items) return true;
                it = P.items[idx];
            } while (it.t0 == it.t1);
            if (!stages) return true;
            const int row0 = it.rb * P.block_rows, rows = min(P.block_rows, P.Q.rows - row0);
            uint4 v[D / 8];
            if (mine < rows) {
                const uint4* src = reinterpret_cast<const uint4*>(P.Q.at(it.b, it.head, row0 + mine));
#pragma unroll
                for (int i = 0; i < D / 8; ++i) v[i] = __ldg(src + i);
            }
            if (!kRows2 && use > 0) {   // the other stream's products read these rows too
                if (!__all_sync(0xffffffffu, tile_wait(smem_addr(&sh.q_empty), (use - 1) & 1, &sh.abort, P.C.err))) return false;
            }
            if (mine < rows) {
                uint32_t big = 0;   // magnitudes order like their bits
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) big = __vmaxu2(big, w[e] & 0x7fff7fffu);
                }
                float down, up;
                row_power(__uint_as_float(max(big << 16, big & 0xffff0000u)), down, up);
                rs_next = fmaxf(fabsf(P.scale2) * up, 1.2e-38f);
                if (P.scale2 < 0.0f) down = -down;
                if (!kRows2) sh.row_scale[use & 1][mine] = rs_next;
                unsigned char* row = tiles + (mine >> 7) * T::kTileBytes + (mine & 127) * 128;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = pack_h2(bf16_lo(w[e]) * down, bf16_hi(w[e]) * down);
                    *reinterpret_cast<uint4*>(row + (i >> 3) * kBlockBytes + (((i & 7) ^ (mine & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            // rows past the item's are left as they are: what they give goes nowhere
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[use & 1][kRows2 ? st : 0]));
            return true;
        };
        bool alive = stage(0, 0);
        for (int k = 0, idx; alive && (idx = item_index(k, blockIdx.x, P.ctas)) < n_items; ++k) {
            const TileItem it = P.items[idx];
            const int n = it.n;
            const int row0 = it.rb * P.block_rows;
            const int rows = min(P.block_rows, P.Q.rows - row0);
            const int row = (kRows2 ? st * 128 : 0) + quad * 32 + lane;   // of the item
            const bool live = (kRows2 ? st * 128 : 0) + quad * 32 < rows;   // the warp has rows
            rs = rs_next;
            if (!kRows2 && st == 1 && it.t0 + 1 < it.t1) {
                TILE_WAIT(smem_addr(&sh.q_full[used & 1][0]), used >> 1 & 1)
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
                    if (left < kTileTokens) {   // the last tile: -inf over what lies past the end
#pragma unroll 1
                        for (int c = left >> 4; c < 8; ++c) {
                            uint32_t x[16];
                            tc_ld16(x, tS + c * 16);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (c * 16 + i >= left) x[i] = 0xff800000u;
                            tc_st16(tS + c * 16, x);
                        }
                        tc_wait_st();
                    }
                    uint32_t x[4][32];   // the row's scores
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc_ld32(x[c], tS + c * 32);
                    tc_wait_ld();
                    float top[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        top[c] = __uint_as_float(x[c][0]);
#pragma unroll
                        for (int i = 1; i < 32; ++i) top[c] = fmaxf(top[c], __uint_as_float(x[c][i]));
                    }
                    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * rs;
                    // lanes past the item's rows hold whatever was there: a move they asked for would change how
                    // the rows beside them are rounded
                    if (__any_sync(0xffffffffu, row < rows && mx > m + kAbove)) {
                        const float mn = fmaxf(m, mx - kBelow);
                        const float f = m == -INFINITY ? 0.0f : ex2_approx(m - mn);
                        m = mn;
                        l *= f;
                        if (done > 0) {   // the product that last wrote O came before this tile's scores
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t o[16];
                                tc_ld16(o, tO + c * 16);
                                tc_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tc_st16(tO + c * 16, o);
                            }
                            tc_wait_st();
                        }
                    }
                    const unsigned long long rs2 = f32x2_splat(rs), m2 = f32x2_splat(-m);
                    unsigned long long l2[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const unsigned long long y = f32x2_fma(
                                f32x2_pack(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])), rs2, m2);
                            const float a = ex2_approx(f32x2_lo(y)), b = ex2_approx(f32x2_hi(y));
                            l2[i & 1] = f32x2_add(l2[i & 1], f32x2_pack(a, b));
                            p[i] = pack_h2(a, b);
                        }
                        tc_st16(tS + c * 16, p);   // over scores already read
                    }
                    l += (f32x2_lo(l2[0]) + f32x2_hi(l2[0])) + (f32x2_lo(l2[1]) + f32x2_hi(l2[1]));
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p);
            }
            if (stop) break;
            // the item's end: the next one's queries first
            const int tiles_all = it.t1 - it.t0;
            if (tiles_all > 0 && !(alive = stage(k + 1, used + 1))) break;
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
        widen_tiles<D>(P, sh.raw, tiles + T::kRawAt, sh.full, sh.empty, T::kSlots, tiles + T::kQueryTiles * T::kTileBytes,
                       warp - kSoftWarps, lane, &sh.abort);
    } else if (warp == kCopyWarp) {
        copy_tiles<D, 2>(P, sh.raw, base + T::kRawAt, n_items, 1, lane, &sh.abort);
    } else if (warp == kIssueWarp && lane == 0) {
        // ------------------------------------------------------------ products
        constexpr uint32_t kScoreDesc = tc_idesc(128, kTileTokens, false);
        constexpr uint32_t kValueDesc = tc_idesc(128, D, true);
        uint32_t half = 0;            // half-tiles consumed before this item
        uint32_t p_count[2] = {0, 0};
        uint32_t used = 0;            // items with tiles so far
        TileItem nx;
        nx.t1 = -1;
        if (item_index(0, blockIdx.x, P.ctas) < n_items) nx = P.items[item_index(0, blockIdx.x, P.ctas)];
        for (int k = 0, idx; (idx = item_index(k, blockIdx.x, P.ctas)) < n_items; ++k) {
            const TileItem it = nx;
            idx = item_index(k + 1, blockIdx.x, P.ctas);
            if (idx < n_items) nx = P.items[idx];   // ahead of its use
            const int nt = it.t1 - it.t0;
            if (nt == 0) continue;
            const uint32_t use = used++;
            TILE_WAIT_ONE(smem_addr(&sh.q_full[use & 1][0]), use >> 1 & 1)   // a fence follows before its use
            // half-tile 2 t holds tile t's keys, 2 t + 1 its values
            auto slot_of = [&](int h) { return (half + h) % T::kSlots; };
            auto phase_of = [&](int h) { return ((half + h) / T::kSlots) & 1; };
            auto scores = [&](int st, int t) {
                const uint32_t a = tc_desc_low(base + (kRows2 ? st : 0) * T::kTileBytes, 16);
                const uint32_t b = tc_desc_low(ring + slot_of(2 * t) * T::kTileBytes, 16);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const uint32_t off = ((c >> 2) * kBlockBytes + (c & 3) * 32) >> 4;
                    tc_mma_ss(tmem + st * 128, a + off, b + off, kScoreDesc, c > 0);
                }
                tc_commit(smem_addr(&sh.s_full[st]));
            };
            auto values = [&](int st, int t, bool acc) {
                const uint32_t b = tc_desc_low(ring + slot_of(2 * t + 1) * T::kTileBytes, kBlockBytes);
#pragma unroll
                for (int c = 0; c < kTileTokens / 16; ++c)
                    tc_mma_ts(tmem + 256 + st * D, tmem + st * 128 + c * 8, b + c * (2048 >> 4), kValueDesc, acc || c > 0);
            };
            bool stop = false;
            do {
                stop = true;
                TILE_WAIT_ONE(smem_addr(&sh.full[slot_of(0)]), phase_of(0))
                fence_async_shared();
                tc_fence_after();
                scores(0, 0);
                if (kRows2) {
                    TILE_WAIT_ONE(smem_addr(&sh.q_full[use & 1][1]), use >> 1 & 1)
                    fence_async_shared();
                    scores(1, 0);
                }
                tc_commit(smem_addr(&sh.empty[slot_of(0)]));
                if (!kRows2 && nt > 1) {
                    TILE_WAIT_ONE(smem_addr(&sh.full[slot_of(2)]), phase_of(2))
                    fence_async_shared();
                    tc_fence_after();
                    scores(1, 1);
                    tc_commit(smem_addr(&sh.empty[slot_of(2)]));
                }
                if (!kRows2 && nt <= 2) tc_commit(smem_addr(&sh.q_empty));
                stop = false;
            } while (false);
            for (int t = 0; t < nt && !stop; ++t) {
#pragma unroll 1
                for (int u = 0; u < (kRows2 ? 2 : 1); ++u) {
                    const int st = kRows2 ? u : t & 1;
                    const int ahead = t + (kRows2 ? 1 : 2);   // the stream's next tile
                    stop = true;
                    if (u == 0) {   // both tiles that this turn needs, while the softmax is still at work
                        TILE_WAIT_ONE(smem_addr(&sh.full[slot_of(2 * t + 1)]), phase_of(2 * t + 1))
                        if (ahead < nt) {
                            TILE_WAIT_ONE(smem_addr(&sh.full[slot_of(2 * ahead)]), phase_of(2 * ahead))
                        }
                        fence_async_shared();
                    }
                    TILE_WAIT_ONE(smem_addr(&sh.p_ready[st]), p_count[st] & 1)
                    ++p_count[st];
                    tc_fence_after();
                    values(st, t, t >= (kRows2 ? 1 : 2));
                    if (!kRows2 || u == 1) tc_commit(smem_addr(&sh.empty[slot_of(2 * t + 1)]));
                    if (ahead < nt) {
                        scores(st, ahead);
                        if (!kRows2 || u == 1) {
                            tc_commit(smem_addr(&sh.empty[slot_of(2 * ahead)]));
                            if (!kRows2 && ahead == nt - 1) tc_commit(smem_addr(&sh.q_empty));   // the item's last scores
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
    if (warp == kIssueWarp) {
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
    RawRing raw;
    uint32_t tmem;
    int abort;
    float4 cols[2][kTileRows / 2];   // by use parity: (scale, scale, -lse, -lse) of two rows
};
template <int D>
struct WeightShape {
    static constexpr uint32_t kTileBytes = D / 64 * kBlockBytes;
    static constexpr int kSlots = 3;
    static constexpr uint32_t kRawBytes = kTileTokens * (D / 2 + D / 16);
    static constexpr uint32_t kRawAt = (2 + kSlots) * kTileBytes;
    static constexpr uint32_t kTiles = kRawAt + kRaw * kRawBytes;
    static constexpr size_t kSmem = kTiles + sizeof(WeightShared);
};

template <int D>
__global__ void __launch_bounds__(kWeightThreads, 1) kv4_weight_tile_kernel(const __grid_constant__ AttendParams P) {
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
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(smem_addr(&sh.raw.full[i]), 1);
            mbar_init(smem_addr(&sh.raw.empty[i]), kWidenWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&sh.q_full[s]), kQueryWarps);
            mbar_init(smem_addr(&sh.cols_empty[s]), kSoftWarps);
            mbar_init(smem_addr(&sh.s_full[s]), 1);
            mbar_init(smem_addr(&sh.s_empty[s]), kSoftWarps / 2);
        }
        mbar_fence_init();
    }
    if (warp == kIssueWarp) tmem_alloc(smem_addr(&sh.tmem), 512);
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
            const int n = it.n;
            for (int rb = 0; rb < blocks && !stop; ++rb, ++used) {
                stop = true;
                TILE_WAIT(smem_addr(&sh.q_full[used & 1]), used >> 1 & 1)
                stop = false;
                const float4* col = sh.cols[used & 1];
                // a token's tile takes the same buffer for every block of rows: its thread adds to its own sums
                for (int t = it.t0 + ((k ^ buf) & 1); t < it.t1; t += 2, ++tile) {
                    // the token's place and what it had, while its scores are on their way; later blocks of rows
                    // add to what this thread itself wrote
                    const int j = t * kTileTokens + quad * 32 + lane;
                    long long at = -1;
                    float had = 0.0f;
                    int page;
                    if (j < n && kv4_page(P.C, P.C.table, it.b, j >> P.C.page_shift, P.C.max_pages, it.head, &page)) {
                        at = (((long long)page * P.C.heads + it.head) << P.C.page_shift) + (j & ((1 << P.C.page_shift) - 1));
                        const float* from = rb == 0 ? P.prior : P.weights;
                        if (from) had = __ldcg(from + at);
                    }
                    stop = true;
                    TILE_WAIT(smem_addr(&sh.s_full[buf]), tile & 1)
                    stop = false;
                    tc_fence_after();
                    unsigned long long acc[4] = {0, 0, 0, 0};
                    uint32_t r[2][16];   // the next columns arrive while these are worked on
                    auto add = [&](const uint32_t(&x)[16], int c) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 f = col[c / 2 + i];
                            const unsigned long long y =
                                f32x2_fma(f32x2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                                          f32x2_pack(f.x, f.y), f32x2_pack(f.z, f.w));
                            acc[i & 3] = f32x2_add(acc[i & 3], f32x2_pack(ex2_approx(f32x2_lo(y)), ex2_approx(f32x2_hi(y))));
                        }
                    };
                    tc_ld16(r[0], tS);
                    for (int c = 0; c < cols; c += 32) {
                        tc_wait_ld();
                        tc_ld16(r[1], tS + c + 16);
                        add(r[0], c);
                        tc_wait_ld();
                        if (c + 32 < cols) tc_ld16(r[0], tS + c + 32);
                        add(r[1], c + 16);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.s_empty[buf]));
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sum += f32x2_lo(acc[i]) + f32x2_hi(acc[i]);
                    if (at >= 0) P.weights[at] = had + sum;
                }
                if (stop) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.cols_empty[used & 1]));
            }
        }
    } else if (warp < kSoftWarps + kWidenWarps) {
        widen_tiles<D>(P, sh.raw, tiles + T::kRawAt, sh.full, sh.empty, T::kSlots, tiles + 2 * T::kTileBytes,
                       warp - kSoftWarps, lane, &sh.abort);
    } else if (warp == kCopyWarp) {
        copy_tiles<D, 1>(P, sh.raw, base + T::kRawAt, n_items, blocks, lane, &sh.abort);   // again for each block of rows
    } else if (warp > kCopyWarp) {
        uint32_t used = 0;
        bool stop = false;
        for (int k = 0, idx; !stop && (idx = item_index(k, blockIdx.x, P.ctas)) < n_items; ++k) {
            const TileItem it = P.items[idx];
            if (it.t0 == it.t1) continue;
            for (int rb = 0; rb < blocks && !stop; ++rb, ++used) {
                stop = true;
                if (used > 0) {
                    TILE_WAIT_PATIENT(smem_addr(&sh.q_empty), (used - 1) & 1)
                }
                if (used > 1) {
                    TILE_WAIT_PATIENT(smem_addr(&sh.cols_empty[used & 1]), (used >> 1 & 1) ^ 1)
                }
                stop = false;
                const int row0 = rb * block_rows, rows = min(block_rows, P.Q.rows - row0);
                float* col = reinterpret_cast<float*>(sh.cols[used & 1]);
                const float s2 = fabsf(P.scale2);
                stage_queries<D, kQueryWarps>(P, tiles, it.b, it.head, row0, rows, cols, warp - kCopyWarp - 1, lane,
                                              [&](int r, float up) {
                    float* f = col + (r >> 1) * 4 + (r & 1);
                    f[0] = r < rows ? s2 * up : 0.0f;
                    f[2] = r < rows ? -P.lse[P.row_at(it.b, it.head, row0 + r)] * kLog2e : -INFINITY;
                });
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[used & 1]));
            }
        }
    } else if (lane == 0) {
        const uint32_t first_desc = tc_idesc(128, min(cols, 128), false), second_desc = tc_idesc(128, max(cols - 128, 32), false);
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
                    fence_async_shared();
                    tc_fence_after();
                    const uint32_t a = tc_desc_low(ring + s * T::kTileBytes, 16);
                    const uint32_t q0 = tc_desc_low(base, 16), q1 = tc_desc_low(base + T::kTileBytes, 16);
                    const uint32_t d = tmem + buf * 256;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const uint32_t off = ((c >> 2) * kBlockBytes + (c & 3) * 32) >> 4;
                        // rows 128.. of the queries are a tile further on: two products when there are any
                        tc_mma_ss(d, a + off, q0 + off, first_desc, c > 0);
                        if (cols > 128) tc_mma_ss(d + 128, a + off, q1 + off, second_desc, c > 0);
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
    if (warp == kIssueWarp) {
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
    static std::atomic<int> regs{0};
    DLLM_CUDA_TRY(allow_smem(kernel, T::kSmem, done));
    if (regs.load(std::memory_order_acquire) == 0) {
        cudaFuncAttributes attr;
        DLLM_CUDA_TRY(cudaFuncGetAttributes(&attr, kernel));
        regs.store(attr.numRegs, std::memory_order_release);
    }
    // the split of registers above is of kLaunchRegs: with fewer at launch the softmax would wait for ever
    if (regs.load(std::memory_order_acquire) != kLaunchRegs) return DLLM_ERR_UNSUPPORTED;
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
    DLLM_CUDA_TRY(launch_dependent(kernel, dim3(P.ctas), dim3(kWeightThreads), WeightShape<D>::kSmem, s, P));
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
