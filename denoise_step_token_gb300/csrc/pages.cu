// dllm_pages_*: who holds which pages of a cache's pools: forks, growth, release,
// copies between pools, and the closing of a pool's gaps.
//
// A page is in use while its count of holders (refs) is above zero.  Pages are
// handed out lowest first, entries in their order, so equal calls give equal
// tables.  What has to be decided over the whole pool is one block's: sums over
// refs, 8192 pages a round (a round is about 1.5 us; pools of a server have some
// ten thousand pages).  What moves pages or goes through tables is a launch over
// all SMs behind it, bound by memory: a page's bytes are read and written once.
#include <stdint.h>

#include <algorithm>

#include "common.cuh"

namespace dllm {
namespace {

constexpr int kMaxArrays = DLLM_PAGES_MAX_ARRAYS;
constexpr int kThreads = 1024;   // of the deciding block
constexpr int kMoveThreads = 256;

struct Batch {
    int B, max_pages, page_size, n_pages;
    int* table;
    int* held;
    int* refs;
    int* err;

    __device__ __forceinline__ bool ok(bool v) const {
        if (!v) set_error(err, DLLM_DEVERR_PAGE);
        return v;
    }
    __device__ __forceinline__ bool row_ok(int b) const { return ok((unsigned)b < (unsigned)B); }
    __device__ __forceinline__ bool page_ok(int page) const { return ok((unsigned)page < (unsigned)n_pages); }
    // Pages held, within the table.
    __device__ __forceinline__ int within(int n) const { return ok(n >= 0 && n <= max_pages) ? n : min(max(n, 0), max_pages); }
};

// ---------------------------------------------------------------------------
// Moving pages.
// ---------------------------------------------------------------------------
constexpr int kDeep = 8;                       // 16-byte pieces a thread has in flight
constexpr int kTile = 32 * kDeep * 16;         // bytes a warp moves at a time

struct Moves {
    int n_from, n_to, n_arrays, tiles;         // pages of the pools; tiles of a page over all arrays
    int n_most;                                // pairs
    const int* n;                              // their number on the device, or NULL
    const int* src;                            // pages, -1: skip
    const int* dst;
    int* err;
    const void* from[kMaxArrays];
    void* to[kMaxArrays];
    long long bytes[kMaxArrays];               // of a page
    int tile0[kMaxArrays + 1];                 // first tile of each array
};

// A warp an item: a tile of a pair's page.  What the tiles belong to is looked up by the warp's lanes in shared memory.
__device__ __forceinline__ void move_pages(const Moves& P) {
    __shared__ const char* s_from[kMaxArrays];
    __shared__ char* s_to[kMaxArrays];
    __shared__ long long s_bytes[kMaxArrays];
    __shared__ int s_tile0[kMaxArrays];
    for (int k = threadIdx.x; k < kMaxArrays; k += blockDim.x) {
        s_from[k] = static_cast<const char*>(P.from[k]);
        s_to[k] = static_cast<char*>(P.to[k]);
        s_bytes[k] = P.bytes[k];
        s_tile0[k] = k < P.n_arrays ? P.tile0[k] : 0x7fffffff;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const long long n = P.n ? min(__ldg(P.n), P.n_most) : P.n_most;
    for (long long w = (long long)blockIdx.x * warps + (threadIdx.x >> 5); w < n * P.tiles; w += (long long)gridDim.x * warps) {
        const int i = (int)(w / P.tiles), t = (int)(w - (long long)i * P.tiles);
        const int a = __ldg(P.src + i), b = __ldg(P.dst + i);
        if (a == -1 || b == -1) continue;
        if ((unsigned)a >= (unsigned)P.n_from || (unsigned)b >= (unsigned)P.n_to) {
            if (lane == 0) set_error(P.err, DLLM_DEVERR_PAGE);
            continue;
        }
        static_assert(kMaxArrays == 64, "two arrays a lane");
        const int k = __popc(__ballot_sync(0xffffffffu, s_tile0[lane] <= t)) +
                      __popc(__ballot_sync(0xffffffffu, s_tile0[lane + 32] <= t)) - 1;
        const long long bytes = s_bytes[k], at = (long long)(t - s_tile0[k]) * kTile;
        const uint4* const from = reinterpret_cast<const uint4*>(s_from[k] + a * bytes + at);
        uint4* const to = reinterpret_cast<uint4*>(s_to[k] + b * bytes + at);
        const int left = (int)min((long long)kTile, bytes - at) / 16;
        uint4 q[kDeep];
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
            if (d * 32 + lane < left) q[d] = __ldcs(from + d * 32 + lane);
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
            if (d * 32 + lane < left) __stcs(to + d * 32 + lane, q[d]);
    }
}

__global__ void __launch_bounds__(kMoveThreads) copy_kernel(const __grid_constant__ Moves P) {
    pdl_wait();
    pdl_release();
    move_pages(P);
}

// ---------------------------------------------------------------------------
// Deciding, one block of kThreads.
// ---------------------------------------------------------------------------
// Sum over the block's threads before this one; `total` of all.  Every thread calls.
__device__ __forceinline__ int block_before(int v, int* total) {
    __shared__ int sums[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();   // the last call's sums are read
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int s = sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    const int before = __shfl_sync(0xffffffffu, s, warp ? warp - 1 : 0);
    return x - v + (warp ? before : 0);
}

constexpr int kEach = 8;   // pages of a thread and round
// Which of pages [p, p + 8) are in use, a bit each; pages past the pool: `past`.
__device__ __forceinline__ uint32_t used_bits(const int* refs, int p, int n_pages, uint32_t past) {
    uint32_t u = 0;
    if (p + kEach <= n_pages) {
        const int4 a = *reinterpret_cast<const int4*>(refs + p), b = *reinterpret_cast<const int4*>(refs + p + 4);
        u = (a.x > 0) | (a.y > 0) << 1 | (a.z > 0) << 2 | (a.w > 0) << 3;
        return u | (b.x > 0) << 4 | (b.y > 0) << 5 | (b.z > 0) << 6 | (b.w > 0) << 7;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) u |= (p + k < n_pages ? refs[p + k] > 0 : past) << k;
    return u;
}

// The first `count` free pages into list, lowest first; how many there were.
__device__ __forceinline__ int list_free(const int* refs, int n_pages, int count, int* list) {
    int have = 0;
#pragma unroll 1
    for (int p0 = 0; p0 < n_pages && have < count; p0 += kThreads * kEach) {
        const int p = p0 + threadIdx.x * kEach;
        uint32_t open = ~used_bits(refs, p, n_pages, 1) & 0xffu;
        int total;
        int rank = have + block_before(__popc(open), &total);
        for (; open && rank < count; open &= open - 1) list[rank++] = p + __ffs(open) - 1;
        have += total;
    }
    __syncthreads();
    return min(have, count);
}

struct ForkParams {
    Batch T;
    int* lens;
    int F;
    const int* src;
    const int* dst;
    int* fresh;   // [F] the page that each fork took, -1 none, -2 not served
    int* from;    // [F] what is to be copied there, -1 nothing
    int* list;    // [F]
    Moves moves;  // from -> fresh
};

// Tokens of a fork's source, as far as its pages reach.
__device__ __forceinline__ int fork_tokens(const ForkParams& P, int s) {
    const int n = P.lens[s];
    const long long most = min((long long)P.T.within(P.T.held[s]) * P.T.page_size, 0x7fffffffll);
    return P.T.ok(n >= 0 && n <= most) ? n : (int)min(max((long long)n, 0ll), most);
}

// Forks that end inside a page take a free one, in their order; from the first that finds none on they are not served.
// Nor is one whose rows or pages are outside: its tables' entries are looked through first, a warp's lanes over each of its
// forks in turn (neighbouring forks in different warps), so that it takes no page.
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ ForkParams P) {
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int f0 = 0; f0 < P.F; f0 += kThreads) {
        const int f = f0 + lane * (kThreads / 32) + warp;
        int s = 0, pages = 0;   // the fork's source and the pages that it takes over
        bool ok = false;
        if (f < P.F) {
            s = __ldg(P.src + f);
            ok = P.T.row_ok(s) && P.T.row_ok(__ldg(P.dst + f));
            if (ok) {
                const int n = fork_tokens(P, s);
                pages = n / P.T.page_size + (n % P.T.page_size != 0);
            }
        }
        uint32_t bad = 0;   // a bit for each of the warp's forks
        const uint32_t some = __ballot_sync(0xffffffffu, pages > 0);
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += 4) {   // four forks' loads at once
            if ((some >> i0 & 15) == 0) continue;
            const int* row[4];
            int most[4], page[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                most[k] = __shfl_sync(0xffffffffu, pages, i0 + k);
                row[k] = P.T.table + (long long)__shfl_sync(0xffffffffu, s, i0 + k) * P.T.max_pages;
                page[k] = lane < most[k] ? row[k][lane] : 0;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bool out = (unsigned)page[k] >= (unsigned)P.T.n_pages;
#pragma unroll 4
                for (int j = lane + 32; j < most[k]; j += 32) out |= (unsigned)row[k][j] >= (unsigned)P.T.n_pages;
                if (out) bad |= 1u << (i0 + k);
            }
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (f < P.F) P.fresh[f] = P.T.ok(!(bad >> lane & 1)) && ok ? 0 : -2;
    }
    __syncthreads();
    int need = 0;
    for (int f0 = 0; f0 < P.F; f0 += kThreads) {
        const int f = f0 + threadIdx.x;
        int from = -1;
        bool ok = false;
        if (f < P.F && P.fresh[f] == 0) {
            ok = true;
            const int s = __ldg(P.src + f), n = fork_tokens(P, s);
            if (n % P.T.page_size) from = P.T.table[(long long)s * P.T.max_pages + n / P.T.page_size];
        }
        int total;
        const int rank = need + block_before(from >= 0, &total);
        if (f < P.F) {
            P.from[f] = from;
            P.fresh[f] = from >= 0 ? rank : ok ? -1 : -2;
        }
        need += total;
    }
    const int have = list_free(P.T.refs, P.T.n_pages, need, P.list);
    if (have < need && threadIdx.x == 0) set_error(P.T.err, DLLM_DEVERR_PAGE);
    for (int f = threadIdx.x; f < P.F; f += kThreads) {
        if (P.from[f] < 0) continue;
        const int rank = P.fresh[f];
        if (rank < have) {
            P.fresh[f] = P.list[rank];
            P.T.refs[P.list[rank]] = 1;
        } else {
            P.fresh[f] = -2;
            P.from[f] = -1;
        }
    }
}

// The tables (a warp a fork) and the last pages' contents.
__global__ void __launch_bounds__(kMoveThreads) fork_spread_kernel(const __grid_constant__ ForkParams P) {
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31, warps = kMoveThreads / 32;
    for (int f = blockIdx.x * warps + (threadIdx.x >> 5); f < P.F; f += gridDim.x * warps) {
        const int s = __ldg(P.src + f), d = __ldg(P.dst + f), fresh = P.fresh[f];
        if ((unsigned)d >= (unsigned)P.T.B) continue;
        if (fresh == -2) {
            if (lane == 0) P.lens[d] = P.T.held[d] = 0;
            continue;
        }
        const int n = fork_tokens(P, s), full = n / P.T.page_size, tail = n % P.T.page_size != 0;
        const int* const from = P.T.table + (long long)s * P.T.max_pages;
        int* const to = P.T.table + (long long)d * P.T.max_pages;
        for (int j = lane; j < full; j += 32) {
            const int page = from[j];
            to[j] = page;
            if (P.T.page_ok(page)) atomicAdd(P.T.refs + page, 1);
        }
        if (lane == 0) {
            if (tail) to[full] = fresh;
            P.T.held[d] = full + tail;
            P.lens[d] = n;
        }
    }
    move_pages(P.moves);
}

struct GrowParams {
    Batch T;
    const int* lens;
    int R, extra;
    const int* rows;
    int* taken;   // [R] pages taken, -1 not served
    int* start;   // [R] rank of the first
    int* list;    // [n_pages]
};

__global__ void __launch_bounds__(kThreads) grow_kernel(const __grid_constant__ GrowParams P) {
    pdl_wait();
    pdl_release();
    int need = 0;   // saturates behind the pool's pages: what passes them is not served
    for (int r0 = 0; r0 < P.R; r0 += kThreads) {
        const int r = r0 + threadIdx.x;
        int more = -1;
        if (r < P.R) {
            const int b = __ldg(P.rows + r);
            if (P.T.row_ok(b)) {
                const long long pages = (max((long long)P.lens[b] + P.extra, 0ll) + P.T.page_size - 1) / P.T.page_size;
                if (P.T.ok(pages <= P.T.max_pages)) more = max((int)pages - P.T.within(P.T.held[b]), 0);
            }
        }
        int total;
        const int rank = need + block_before(max(more, 0), &total);   // 2^30 at most
        if (r < P.R) {
            P.taken[r] = more;
            P.start[r] = rank;
        }
        need = (int)min((long long)need + total, P.T.n_pages + 1ll);   // 2^30 and 2^30 may meet
    }
    const int have = list_free(P.T.refs, P.T.n_pages, min(need, P.T.n_pages), P.list);
    if (have < need && threadIdx.x == 0) set_error(P.T.err, DLLM_DEVERR_PAGE);
    const int lane = threadIdx.x & 31;
    for (int r = threadIdx.x >> 5; r < P.R; r += kThreads / 32) {
        const int more = P.taken[r], start = P.start[r];
        __syncwarp();
        if (more <= 0) continue;
        if ((long long)start + more > have) {
            if (lane == 0) P.taken[r] = -1;
            continue;
        }
        const int b = __ldg(P.rows + r), held = P.T.within(P.T.held[b]);
        for (int k = lane; k < more; k += 32) {
            const int page = P.list[start + k];
            P.T.refs[page] = 1;
            if (held + k < P.T.max_pages) P.T.table[(long long)b * P.T.max_pages + held + k] = page;
        }
        __syncwarp();
        if (lane == 0) P.T.held[b] = min(held + more, P.T.max_pages);
    }
}

// A warp a request.  held is taken at once, so that a row given twice gives its pages back once.
__global__ void __launch_bounds__(kMoveThreads) free_kernel(const __grid_constant__ Batch T, const int* rows, int R) {
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31, r = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
    if (r >= R) return;
    const int b = __ldg(rows + r);
    if (!T.row_ok(b)) return;
    int held = 0;
    if (lane == 0) held = T.within(atomicExch(T.held + b, 0));
    held = __shfl_sync(0xffffffffu, held, 0);
    for (int j = lane; j < held; j += 32) {
        const int page = T.table[(long long)b * T.max_pages + j];
        if (!T.page_ok(page)) continue;
        if (!T.ok(atomicSub(T.refs + page, 1) > 0)) atomicAdd(T.refs + page, 1);
    }
}

struct CompactParams {
    Batch T;
    int* used;      // [1]
    int* map;       // [n_pages]
    int* n_moves;   // [1]
    int* movers;    // [n_pages]
    int* holes;     // [n_pages]
    Moves moves;    // movers -> holes
};

// With U pages in use, those from U on move into the free ones below U, both in their order.
__global__ void __launch_bounds__(kThreads) compact_plan_kernel(const __grid_constant__ CompactParams P) {
    pdl_wait();
    pdl_release();
    const int n = P.T.n_pages, tid = threadIdx.x;
    int mine = 0, U;
    for (int p = tid * kEach; p < n; p += kThreads * kEach) mine += __popc(used_bits(P.T.refs, p, n, 0));
    block_before(mine, &U);
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < n; p0 += kThreads * kEach) {
        const int p = p0 + tid * kEach;
        const uint32_t used = used_bits(P.T.refs, p, n, 0), in = n - p >= kEach ? 0xffu : n > p ? (1u << (n - p)) - 1u : 0;
        const uint32_t low = U - p >= kEach ? 0xffu : U > p ? (1u << (U - p)) - 1u : 0;   // pages below U
        uint32_t hole = ~used & in & low, mover = used & ~low;
        int total;   // both counts in one sum: under 2^13 each
        const int rank = block_before(__popc(hole) | __popc(mover) << 16, &total);
        int h = holes + (rank & 0xffff), m = movers + (rank >> 16);
        for (int k = 0; k < kEach; ++k) {
            if (!(in >> k & 1)) continue;
            P.map[p + k] = used >> k & 1 ? p + k : -1;
            if (hole >> k & 1) P.holes[h++] = p + k;
            if (mover >> k & 1) P.movers[m++] = p + k;
        }
        holes += total & 0xffff;
        movers += total >> 16;
    }
    __syncthreads();
    for (int i = tid; i < movers; i += kThreads) {
        const int a = P.movers[i], b = P.holes[i];
        P.map[a] = b;
        P.T.refs[b] = P.T.refs[a];
        P.T.refs[a] = 0;
    }
    if (tid == 0) {
        *P.used = U;
        *P.n_moves = movers;
    }
}

__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const __grid_constant__ CompactParams P) {
    pdl_wait();
    pdl_release();
    const int lane = threadIdx.x & 31, warps = kMoveThreads / 32;
    for (int b = blockIdx.x * warps + (threadIdx.x >> 5); b < P.T.B; b += gridDim.x * warps) {
        const int held = P.T.within(P.T.held[b]);
        int* const row = P.T.table + (long long)b * P.T.max_pages;
        for (int j = lane; j < held; j += 32) {
            const int page = row[j];
            if (!P.T.page_ok(page)) continue;
            const int to = __ldcg(P.map + page);
            if (P.T.ok(to >= 0)) row[j] = to;   // a page that nobody counts stays as it is
        }
    }
    move_pages(P.moves);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
int check_batch(const dllm_pages_batch& a, Batch* T) {
    if (a.n_pages < 1 || a.B < 0 || a.max_pages < 1 || a.page_size < 1) return DLLM_ERR_INVAL;
    if (!a.refs || (a.B > 0 && (!a.table || !a.held))) return DLLM_ERR_INVAL;
    if (reinterpret_cast<uintptr_t>(a.refs) & 15) return DLLM_ERR_ALIGN;
    if (a.n_pages > 0x3fffffff || a.max_pages > 1 << 20) return DLLM_ERR_UNSUPPORTED;
    *T = Batch{a.B, a.max_pages, a.page_size, a.n_pages, a.table, a.held, a.refs, nullptr};
    return DLLM_OK;
}

int check_pool(const dllm_pages_pool& a) {
    if (a.n_pages < 1 || a.n_arrays < 0 || a.n_arrays > kMaxArrays) return DLLM_ERR_INVAL;
    for (int k = 0; k < a.n_arrays; ++k) {
        if (!a.arrays[k] || a.page_bytes[k] < 1) return DLLM_ERR_INVAL;
        if ((reinterpret_cast<uintptr_t>(a.arrays[k]) & 15) || a.page_bytes[k] % 16) return DLLM_ERR_ALIGN;
        if (a.page_bytes[k] > (1ll << 32)) return DLLM_ERR_UNSUPPORTED;
    }
    return DLLM_OK;
}

void set_moves(Moves* M, const dllm_pages_pool& from, const dllm_pages_pool& to, const int* src, const int* dst, int n_most,
               const int* n, int* err) {
    M->n_from = from.n_pages;
    M->n_to = to.n_pages;
    M->n_arrays = from.n_arrays;
    M->src = src;
    M->dst = dst;
    M->n_most = n_most;
    M->n = n;
    M->err = err;
    int tiles = 0;
    for (int k = 0; k < kMaxArrays; ++k) {
        const bool have = k < from.n_arrays;
        M->from[k] = have ? from.arrays[k] : nullptr;
        M->to[k] = have ? to.arrays[k] : nullptr;
        M->bytes[k] = have ? from.page_bytes[k] : 0;
        M->tile0[k] = tiles;
        if (have) tiles += (int)((from.page_bytes[k] + kTile - 1) / kTile);
    }
    M->tile0[kMaxArrays] = M->tiles = tiles;
}

// CTAs for `items` warps' work: no more than fill the SMs.
unsigned move_grid(long long items, int sms) {
    return (unsigned)std::max(1ll, std::min((items + kMoveThreads / 32 - 1) / (kMoveThreads / 32), (long long)sms * 6));
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_pages_workspace_size(int32_t n_pages, int32_t entries) {
    if (n_pages < 1 || entries < 0) return 0;
    return (size_t(n_pages) * 2 + size_t(entries) * 2 + 64) * sizeof(int);
}

namespace {
int check_workspace(const void* ws, size_t bytes, int n_pages, int entries) {
    return ws && bytes >= dllm_pages_workspace_size(n_pages, entries) && (reinterpret_cast<uintptr_t>(ws) & 15) == 0
               ? DLLM_OK : DLLM_ERR_WORKSPACE;
}
}  // namespace

extern "C" int dllm_pages_copy(const dllm_pages_pool* from, const dllm_pages_pool* to, int32_t n, const int32_t* src,
                               const int32_t* dst, void* stream) {
    if (!from || !to || n < 0) return DLLM_ERR_INVAL;
    int rc = check_pool(*from);
    if (rc == DLLM_OK) rc = check_pool(*to);
    if (rc != DLLM_OK) return rc;
    if (from->n_arrays != to->n_arrays) return DLLM_ERR_INVAL;
    for (int k = 0; k < from->n_arrays; ++k)
        if (from->page_bytes[k] != to->page_bytes[k]) return DLLM_ERR_INVAL;
    if (n == 0 || from->n_arrays == 0) return DLLM_OK;
    if (!src || !dst) return DLLM_ERR_INVAL;
    const int sms = sm_count();
    int* const err = error_word_ptr();
    if (sms <= 0 || !err) return DLLM_ERR_CUDA;
    Moves M;
    set_moves(&M, *from, *to, src, dst, n, nullptr, err);
    DLLM_CUDA_TRY(launch_dependent(copy_kernel, dim3(move_grid((long long)n * M.tiles, sms)), dim3(kMoveThreads), 0,
                                   as_stream(stream), M));
    return DLLM_OK;
}

extern "C" int dllm_pages_fork(const dllm_pages_batch* batch, const dllm_pages_pool* pool, int32_t* lens, int32_t F,
                               const int32_t* src, const int32_t* dst, int32_t* fresh, void* workspace,
                               size_t workspace_bytes, void* stream) {
    if (!batch || !pool || F < 0) return DLLM_ERR_INVAL;
    ForkParams P;
    int rc = check_batch(*batch, &P.T);
    if (rc == DLLM_OK) rc = check_pool(*pool);
    if (rc != DLLM_OK) return rc;
    if (pool->n_pages != batch->n_pages) return DLLM_ERR_INVAL;
    if (F == 0) return DLLM_OK;
    if (!src || !dst || !fresh || !lens) return DLLM_ERR_INVAL;
    rc = check_workspace(workspace, workspace_bytes, batch->n_pages, F);
    if (rc != DLLM_OK) return rc;
    const int sms = sm_count();
    P.T.err = error_word_ptr();
    if (sms <= 0 || !P.T.err) return DLLM_ERR_CUDA;
    P.lens = lens;
    P.F = F;
    P.src = src;
    P.dst = dst;
    P.fresh = fresh;
    P.from = static_cast<int*>(workspace);
    P.list = P.from + F;
    set_moves(&P.moves, *pool, *pool, P.from, fresh, F, nullptr, P.T.err);
    cudaStream_t s = as_stream(stream);
    DLLM_CUDA_TRY(launch_dependent(fork_kernel, dim3(1), dim3(kThreads), 0, s, P));
    const long long items = std::max<long long>((long long)F * P.moves.tiles, F);
    DLLM_CUDA_TRY(launch_dependent(fork_spread_kernel, dim3(move_grid(items, sms)), dim3(kMoveThreads), 0, s, P));
    return DLLM_OK;
}

extern "C" int dllm_pages_grow(const dllm_pages_batch* batch, const int32_t* lens, int32_t R, const int32_t* rows,
                               int32_t extra, int32_t* taken, void* workspace, size_t workspace_bytes, void* stream) {
    if (!batch || R < 0 || extra < 0) return DLLM_ERR_INVAL;
    GrowParams P;
    int rc = check_batch(*batch, &P.T);
    if (rc != DLLM_OK) return rc;
    if (R == 0) return DLLM_OK;
    if (!rows || !taken || !lens) return DLLM_ERR_INVAL;
    rc = check_workspace(workspace, workspace_bytes, batch->n_pages, R);
    if (rc != DLLM_OK) return rc;
    P.T.err = error_word_ptr();
    if (!P.T.err) return DLLM_ERR_CUDA;
    P.lens = lens;
    P.R = R;
    P.extra = extra;
    P.rows = rows;
    P.taken = taken;
    P.start = static_cast<int*>(workspace);
    P.list = P.start + R;
    DLLM_CUDA_TRY(launch_dependent(grow_kernel, dim3(1), dim3(kThreads), 0, as_stream(stream), P));
    return DLLM_OK;
}

extern "C" int dllm_pages_free(const dllm_pages_batch* batch, int32_t R, const int32_t* rows, void* stream) {
    if (!batch || R < 0) return DLLM_ERR_INVAL;
    Batch T;
    const int rc = check_batch(*batch, &T);
    if (rc != DLLM_OK) return rc;
    if (R == 0) return DLLM_OK;
    if (!rows) return DLLM_ERR_INVAL;
    T.err = error_word_ptr();
    if (!T.err) return DLLM_ERR_CUDA;
    const unsigned grid = (unsigned)(((long long)R + kMoveThreads / 32 - 1) / (kMoveThreads / 32));
    DLLM_CUDA_TRY(launch_dependent(free_kernel, dim3(grid), dim3(kMoveThreads), 0, as_stream(stream), T, rows, R));
    return DLLM_OK;
}

extern "C" int dllm_pages_compact(const dllm_pages_batch* batch, const dllm_pages_pool* pool, int32_t* used, int32_t* map,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    if (!batch || !pool) return DLLM_ERR_INVAL;
    CompactParams P;
    int rc = check_batch(*batch, &P.T);
    if (rc == DLLM_OK) rc = check_pool(*pool);
    if (rc != DLLM_OK) return rc;
    if (pool->n_pages != batch->n_pages || !used || !map) return DLLM_ERR_INVAL;
    rc = check_workspace(workspace, workspace_bytes, batch->n_pages, 0);
    if (rc != DLLM_OK) return rc;
    const int sms = sm_count();
    P.T.err = error_word_ptr();
    if (sms <= 0 || !P.T.err) return DLLM_ERR_CUDA;
    P.used = used;
    P.map = map;
    P.n_moves = static_cast<int*>(workspace);
    P.movers = P.n_moves + 16;
    P.holes = P.movers + batch->n_pages;
    set_moves(&P.moves, *pool, *pool, P.movers, P.holes, batch->n_pages, P.n_moves, P.T.err);
    cudaStream_t s = as_stream(stream);
    DLLM_CUDA_TRY(launch_dependent(compact_plan_kernel, dim3(1), dim3(kThreads), 0, s, P));
    // at most half of the pages move
    const long long items = std::max<long long>((long long)(batch->n_pages / 2) * P.moves.tiles, batch->B);
    DLLM_CUDA_TRY(launch_dependent(compact_move_kernel, dim3(move_grid(items, sms)), dim3(kMoveThreads), 0, s, P));
    return DLLM_OK;
}
