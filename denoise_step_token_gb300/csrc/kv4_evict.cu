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
// Two launches: kv4_select_kernel (one CTA per request and head) writes the
// list `src`; kv4_move_kernel copies the listed tokens, eight 16-byte pieces of
// codes, two runs of parameters and a weight for each.  What bounds it: the
// move reads and writes 1.125 D + 4 bytes a kept token (memory); the selection
// reads the weights from L2 and is bound by its passes' latency.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kv4.cuh"

namespace dllm {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

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

__device__ __forceinline__ float token_weight(const EvictParams& P, int b, int head, int j) {
    const int page = __ldg(P.C.table + (long long)b * P.C.max_pages + (j >> P.C.page_shift));
    if ((unsigned)page >= (unsigned)P.C.n_pages) {
        set_error(P.C.err, DLLM_DEVERR_PAGE);
        return 0.0f;
    }
    const int slot = j & ((1 << P.C.page_shift) - 1);
    return P.weights[(((long long)page * P.C.heads + head) << P.C.page_shift) + slot];
}

// grid: (heads, requests)
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const __grid_constant__ EvictParams P) {
    __shared__ int s_hist[256];
    __shared__ unsigned long long s_warp[kSelWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    pdl_wait();
    pdl_release();
    const int head = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = kv4_len(P.C, P.lens, b);
    const int k = kept_tokens(P, b, n);
    const int r = min(P.recent, k);
    const int m = n - r, kk = k - r;   // kk of the first m stay
    int* src = P.src + ((long long)b * P.C.heads + head) * P.cap;
    if (head == 0 && tid == 0) P.dst_lens[b] = k;
    for (int i = k + tid; i < P.cap; i += kSelThreads) src[i] = -1;
    for (int i = tid; i < r; i += kSelThreads) src[kk + i] = m + i;
    if (kk == 0) return;
    if (kk == m) {
        for (int i = tid; i < m; i += kSelThreads) src[i] = i;
        return;
    }
    uint32_t prefix = 0;
    int need = kk;   // of the keys that share the prefix, the need-th largest is T
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) s_hist[i] = 0;
        __syncthreads();
        for (int j = tid; j < m; j += kSelThreads) {
            const uint32_t key = weight_key(token_weight(P, b, head, j));
            if (shift == 24 || ((key ^ prefix) >> (shift + 8)) == 0) atomicAdd(&s_hist[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, bin = 255;
            while (bin > 0 && s_hist[bin] < left) left -= s_hist[bin--];
            s_prefix = prefix | ((uint32_t)bin << shift);
            s_need = left;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        __syncthreads();
    }
    // T = prefix; `need` of the keys equal to T stay, the lowest tokens first
    int gt0 = 0, eq0 = 0;   // before this tile
    for (int j0 = 0; j0 < m; j0 += kSelThreads) {
        const int j = j0 + tid;
        const uint32_t key = j < m ? weight_key(token_weight(P, b, head, j)) : 0;
        const bool gt = j < m && key > prefix, eq = j < m && key == prefix;
        const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) s_warp[warp] = ((unsigned long long)__popc(bg) << 32) | __popc(be);
        __syncthreads();
        unsigned long long before = 0, all = 0;
        for (int w = 0; w < kSelWarps; ++w) {
            const unsigned long long v = s_warp[w];
            before += w < warp ? v : 0ull;
            all += v;
        }
        const unsigned below = (1u << lane) - 1u;
        const int g = gt0 + (int)(before >> 32) + __popc(bg & below);
        const int e = eq0 + (int)(uint32_t)before + __popc(be & below);
        if (gt || (eq && e < need)) src[g + min(e, need)] = j;
        gt0 += (int)(all >> 32);
        eq0 += (int)(uint32_t)all;
        __syncthreads();
    }
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
    DLLM_CUDA_TRY(launch_dependent(kv4_select_kernel, dim3(H, B), dim3(kSelThreads), 0, as_stream(stream), P));
    const int most = std::max(1, sms * 32 / (B * H));
    const unsigned gx = std::min((P.cap + kMoveTokens - 1) / kMoveTokens, most);
    DLLM_CUDA_TRY(launch_dependent(kv4_move_kernel, dim3(gx, H, B), dim3(256), 0, as_stream(stream), P));
    return DLLM_OK;
}
