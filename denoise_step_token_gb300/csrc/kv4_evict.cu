// dllm_kv4_evict: a cache's least attended tokens leave, the others move in
// their order to new pages.
//
// Per request and head, over n tokens of which k stay, r of them the last ones:
// the k - r largest of the first n - r weights, ties to the lowest token.  The
// weights' order-preserving bits make the choice exact: a radix selection finds
// the (k - r)-th largest key T, byte by byte from the top; with g keys above T,
// the first (k - r) - g tokens of key T stay too.  A token's new place is the
// number of kept tokens before it: (keys above T before it) + min(keys equal to
// T before it, (k - r) - g).
//
// Two launches.  kv4_select_kernel: a cluster of 1 to 8 CTAs per request and head,
// each keeping the keys of its share of the tokens in shared memory; four digits
// of 8 bits, counted per CTA and added up over the cluster through distributed
// shared memory, then one pass that places the kept tokens in `src`.
// What bounds it: the latency of its rounds (about 10 us), not its bytes.
// kv4_move_kernel copies the listed tokens, 16-byte pieces of codes, two runs of
// parameters and a weight for each: 1.125 D + 4 bytes read and written per kept
// token, bound by memory.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kv4.cuh"

namespace dllm {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 256;
constexpr int kKeys = 12288;   // keys a CTA holds; further ones are read again in each pass

struct EvictParams {
    Kv4 C;
    int recent, dst_max_pages, cap, D;   // cap = dst_max_pages * page_size
    const int* lens;
    const int* keep;
    float* weights;
    const int* dst_table;
    int* dst_lens;
    int* src;
};

// Order-preserving bits (-0 as +0); NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    if (x != x) return 0;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Tokens that stay, of request b (the same in both kernels).
__device__ __forceinline__ int kept_tokens(const EvictParams& P, int b, int n) {
    int k = min(max(P.keep[b], 0), n);
    if (k > P.cap) {
        set_error(P.C.err, DLLM_DEVERR_PAGE);
        k = P.cap;
    }
    return k;
}

// The page that holds token j, -1 when the table's entry is not in the pool.
__device__ __forceinline__ int token_page(const EvictParams& P, int b, int j) {
    const int page = __ldg(P.C.table + (long long)b * P.C.max_pages + (j >> P.C.page_shift));
    return (unsigned)page < (unsigned)P.C.n_pages ? page : -1;
}
// Its weight (this kernel writes none); 0 without a page.
__device__ __forceinline__ float token_weight(const EvictParams& P, int page, int head, int j) {
    const int slot = j & ((1 << P.C.page_shift) - 1);
    return page < 0 ? 0.0f : __ldg(P.weights + ((((long long)page * P.C.heads + head) << P.C.page_shift) + slot));
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// A word of CTA `cta`'s shared memory, at the place `p` has in this one.
__device__ __forceinline__ int peer_word(const int* p, int cta) {
    uint32_t at;
    int v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(cta));
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

struct SelectShared {
    int hist[2][kBins];   // digits 0 and 2, 1 and 3
    int warp_sum[kSelWarps];
    int warp_gt[kSelWarps], warp_eq[kSelWarps];
    int total[2];   // of the CTA: keys above T, keys equal to T
    uint32_t prefix;
    int need;
    uint32_t keys[kKeys];
};

// grid: (cluster, heads, requests)
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const __grid_constant__ EvictParams P) {
    extern __shared__ __align__(16) unsigned char select_smem[];
    SelectShared& sh = *reinterpret_cast<SelectShared*>(select_smem);
    pdl_wait();
    pdl_release();
    const int head = blockIdx.y, b = blockIdx.z, ctas = gridDim.x, rank = ctas > 1 ? (int)cluster_rank() : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = kv4_len(P.C, P.lens, b);
    const int k = kept_tokens(P, b, n);
    const int r = min(P.recent, k);
    const int m = n - r, kk = k - r;   // kk of the first m stay
    int* src = P.src + ((long long)b * P.C.heads + head) * P.cap;
    const int gt_id = rank * kSelThreads + tid, step = ctas * kSelThreads;
    if (head == 0 && gt_id == 0) P.dst_lens[b] = k;
    for (int i = k + gt_id; i < P.cap; i += step) src[i] = -1;
    for (int i = gt_id; i < r; i += step) src[kk + i] = m + i;
    if (kk == 0) return;   // the whole cluster agrees
    if (kk == m) {
        for (int i = gt_id; i < m; i += step) src[i] = i;
        return;
    }
    const int j0 = (int)((long long)m * rank / ctas), j1 = (int)((long long)m * (rank + 1) / ctas), count = j1 - j0;
    for (int i = tid; i < 2 * kBins; i += kSelThreads) sh.hist[0][i] = 0;
    constexpr int kAtOnce = 8;   // weights in flight per thread
    for (int i0 = tid; i0 < min(count, kKeys); i0 += kAtOnce * kSelThreads) {
        int page[kAtOnce];
        float w[kAtOnce];
        bool lost = false;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = i0 + u * kSelThreads;
            page[u] = i < count ? token_page(P, b, j0 + i) : 0;
            lost = lost || page[u] < 0;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = i0 + u * kSelThreads;
            w[u] = i < count ? token_weight(P, page[u], head, j0 + i) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = i0 + u * kSelThreads;
            if (i < min(count, kKeys)) sh.keys[i] = weight_key(w[u]);
        }
        if (lost) set_error(P.C.err, DLLM_DEVERR_PAGE);
    }
    for (int i = kKeys + tid; i < count; i += kSelThreads)   // the keys not held: their pages, once
        if (token_page(P, b, j0 + i) < 0) set_error(P.C.err, DLLM_DEVERR_PAGE);
    __syncthreads();
    auto key_at = [&](int i) {
        return i < kKeys ? sh.keys[i] : weight_key(token_weight(P, token_page(P, b, j0 + i), head, j0 + i));
    };
    uint32_t prefix = 0;
    int need = kk;   // of the keys that share the prefix, the need-th largest is T
#pragma unroll 1
    for (int digit = 0; digit < 4; ++digit) {
        const int shift = 24 - 8 * digit;
        int* const hist = sh.hist[digit & 1];
        for (int i = tid; i < count; i += kSelThreads) {
            const uint32_t key = key_at(i);
            if (digit == 0 || ((key ^ prefix) >> (shift + 8)) == 0) atomicAdd(&hist[(key >> shift) & (kBins - 1)], 1);
        }
        if (ctas > 1) cluster_sync();
        else __syncthreads();
        // a bin per thread of the first half, the highest first
        const int bin = kBins - 1 - tid;
        int c = 0;
        if (tid < kBins) {
            c = ctas > 1 ? 0 : hist[bin];
            if (ctas > 1) {
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)
                    if (q < ctas) c += peer_word(hist + bin, q);
            }
        }
        int x = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) sh.warp_sum[warp] = x;
        // the next digit but one counts here: its peers' reads of this one come before the next barrier
        if (tid < kBins && digit > 0) sh.hist[(digit & 1) ^ 1][tid] = 0;
        __syncthreads();
        int above = x - c;
        for (int w = 0; w < min(warp, kBins / 32); ++w) above += sh.warp_sum[w];
        if (tid < kBins && above < need && above + c >= need) {   // one bin
            sh.prefix = prefix | ((uint32_t)bin << shift);
            sh.need = need - above;
        }
        __syncthreads();
        prefix = sh.prefix;
        need = sh.need;
    }
    // T = prefix; `need` of the keys equal to T stay, the lowest tokens first.
    // Each warp places the kept tokens of a run of the CTA's share.
    const int w0 = (int)((long long)count * warp / kSelWarps), w1 = (int)((long long)count * (warp + 1) / kSelWarps);
    int gt = 0, eq = 0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < w1 ? key_at(i) : 0;
        gt += __popc(__ballot_sync(0xffffffffu, i < w1 && key > prefix));
        eq += __popc(__ballot_sync(0xffffffffu, i < w1 && key == prefix));
    }
    if (lane == 0) {
        sh.warp_gt[warp] = gt;
        sh.warp_eq[warp] = eq;
    }
    __syncthreads();
    int g = 0, e = 0;   // before this warp
    for (int w = 0; w < kSelWarps; ++w) {
        if (w == warp) {
            gt = g;
            eq = e;
        }
        g += sh.warp_gt[w];
        e += sh.warp_eq[w];
    }
    if (tid == 0) {
        sh.total[0] = g;
        sh.total[1] = e;
    }
    g = gt;
    e = eq;
    if (ctas > 1) {
        cluster_sync();
        for (int q = 0; q < rank; ++q) {
            g += peer_word(&sh.total[0], q);
            e += peer_word(&sh.total[1], q);
        }
    }
    const unsigned below = (1u << lane) - 1u;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < w1 ? key_at(i) : 0;
        const unsigned bg = __ballot_sync(0xffffffffu, i < w1 && key > prefix);
        const unsigned be = __ballot_sync(0xffffffffu, i < w1 && key == prefix);
        const int mg = g + __popc(bg & below), me = e + __popc(be & below);
        if ((bg >> lane & 1) || ((be >> lane & 1) && me < need)) src[mg + min(me, need)] = j0 + i;
        g += __popc(bg);
        e += __popc(be);
    }
    if (ctas > 1) cluster_sync();   // no CTA leaves while another reads its totals
}

constexpr int kMoveTokens = 128;   // tokens per CTA and pass

// grid: (token tiles, heads, requests)
__global__ void __launch_bounds__(256) kv4_move_kernel(const __grid_constant__ EvictParams P) {
    __shared__ const uint8_t* s_from[kMoveTokens];
    __shared__ uint8_t* s_to[kMoveTokens];
    __shared__ int s_slots[kMoveTokens][2];
    pdl_wait();
    pdl_release();
    const int head = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int n = kv4_len(P.C, P.lens, b);
    const int k = kept_tokens(P, b, n);
    const int* src = P.src + ((long long)b * P.C.heads + head) * P.cap;
    const int shift = P.C.page_shift, slot_mask = (1 << shift) - 1;
    const int code = P.D / 2, par = P.D / 16;   // bytes per token
    const uint32_t half = P.C.head_bytes / 2;
    for (int i0 = blockIdx.x * kMoveTokens; i0 < k; i0 += gridDim.x * kMoveTokens) {
        const int tokens = min(kMoveTokens, k - i0);
        __syncthreads();
        if (tid < tokens) {
            const int j = src[i0 + tid], i = i0 + tid;
            const uint8_t* from = nullptr;
            uint8_t* to = nullptr;
            int fp = 0, tp = 0;
            if (j >= 0 && j < n) {
                from = kv4_page(P.C, P.C.table, b, j >> shift, P.C.max_pages, head, &fp);
                to = kv4_page(P.C, P.dst_table, b, i >> shift, P.dst_max_pages, head, &tp);
            }
            s_from[tid] = to ? from : nullptr;
            s_to[tid] = to;
            s_slots[tid][0] = j & slot_mask;
            s_slots[tid][1] = i & slot_mask;
            if (from && to)
                P.weights[(((long long)tp * P.C.heads + head) << shift) + (i & slot_mask)] =
                    P.weights[(((long long)fp * P.C.heads + head) << shift) + (j & slot_mask)];
        }
        __syncthreads();
        // codes: 16-byte pieces, code/16 of them for keys and as many for values
        const int pieces = code / 8;
        for (int u = tid; u < tokens * pieces; u += 256) {
            const int t = u / pieces, p = u - t * pieces;
            const int which = p >= pieces / 2, q = p - (which ? pieces / 2 : 0);
            if (!s_from[t]) continue;
            const uint32_t base = which ? half : 0;
            *reinterpret_cast<uint4*>(s_to[t] + base + s_slots[t][1] * code + q * 16) =
                __ldcs(reinterpret_cast<const uint4*>(s_from[t] + base + s_slots[t][0] * code + q * 16));
        }
        // parameters: 4-byte pieces
        const int words = par / 2;   // par/4 for keys and as many for values
        for (int u = tid; u < tokens * words; u += 256) {
            const int t = u / words, p = u - t * words;
            const int which = p >= words / 2, q = p - (which ? words / 2 : 0);
            if (!s_from[t]) continue;
            const uint32_t base = (which ? half : 0) + ((uint32_t)code << shift);
            *reinterpret_cast<uint32_t*>(s_to[t] + base + s_slots[t][1] * par + q * 4) =
                *reinterpret_cast<const uint32_t*>(s_from[t] + base + s_slots[t][0] * par + q * 4);
        }
    }
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" int dllm_kv4_evict(const dllm_kv4_evict_args* a, void* stream) {
    if (!a) return DLLM_ERR_INVAL;
    EvictParams P;
    int rc = kv4_check(a->cache, &P.C);
    if (rc != DLLM_OK) return rc;
    if (a->recent < 0 || a->dst_max_pages < 1) return DLLM_ERR_INVAL;
    if ((long long)a->dst_max_pages * a->cache.page_size > 0x3fffffffll) return DLLM_ERR_UNSUPPORTED;
    if (a->cache.B == 0) return DLLM_OK;
    if (!a->lens || !a->keep || !a->weights || !a->dst_table || !a->dst_lens || !a->src) return DLLM_ERR_INVAL;
    int sms = 0;
    rc = kv4_device(&P.C, &sms);
    if (rc != DLLM_OK) return rc;
    P.recent = a->recent;
    P.dst_max_pages = a->dst_max_pages;
    P.cap = a->dst_max_pages * a->cache.page_size;
    P.D = a->cache.head_dim;
    P.lens = a->lens;
    P.keep = a->keep;
    P.weights = a->weights;
    P.dst_table = a->dst_table;
    P.dst_lens = a->dst_lens;
    P.src = a->src;
    const int B = a->cache.B, H = a->cache.heads;
    cudaStream_t s = as_stream(stream);
    // CTAs per request and head: as many as fill the SMs, none with under 2048 tokens (a cluster's rounds cost
    // about 1 us each: at 1024 tokens two CTAs are no faster than one)
    int ctas = 1;
    while (ctas < kMaxCluster && (long long)B * H * ctas < sms && P.C.max_tokens / (2 * ctas) >= 2048) ctas *= 2;
    static SmemOnce done;
    DLLM_CUDA_TRY(allow_smem(kv4_select_kernel, sizeof(SelectShared), done));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, H, B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = sizeof(SelectShared);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    DLLM_CUDA_TRY(cudaLaunchKernelEx(&cfg, kv4_select_kernel, P));
    const int most = std::max(1, sms * 32 / (B * H));
    const unsigned gx = std::min((P.cap + kMoveTokens - 1) / kMoveTokens, most);
    DLLM_CUDA_TRY(launch_dependent(kv4_move_kernel, dim3(gx, H, B), dim3(256), 0, s, P));
    return DLLM_OK;
}
