// The 4-bit cache's layout and arithmetic, shared by its kernels.
//
// A group of 32 channels: step s, zero point z, codes u in [0, 15], values
// s (u - z).  The parameter holds 16 s as an fp16 pattern, whose low 7 bits are
// zero, with z in the low 4 bits.
//
// Widening.  A nibble at bits [7:4] of a half with exponent bits 0x5400 is the
// fp16 number 64 + u; then (64 + u) s - (64 + z) s is one fma with an exact
// result: s has 4 significant bits, so (64 + z) s has at most 11 and
// s (u - z) at most 8, and s <= 768 keeps (64 + z) s below fp16's largest.
// With channels 2i and 2i + 1 sixteen bits apart, one 32-bit word widens to
// its 8 channels with 3 shifts, 4 lop3 and 4 packed fmas.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dllm {

constexpr int kKv4Group = DLLM_KV4_GROUP;
constexpr float kKv4MinStep = 3.814697265625e-06f;   // 2^-18: 16 s is fp16's smallest normal number
constexpr float kKv4MaxStep = 768.0f;                // (64 + 15) * 768 < 65504
constexpr uint16_t kKv4NanParam = 0x7e00u;

// The cache as kernels take it.
struct Kv4 {
    int n_pages, heads, page_shift, B, max_pages, max_tokens;   // max_tokens = max_pages * page_size
    uint32_t head_bytes;      // one head's part of a page
    long long page_bytes;     // heads * head_bytes: page * page_bytes passes 32 bits in a large pool
    uint8_t* pages;
    const int* table;
    int* err;
};

// One head's part of page `n` of request b; nullptr and the device error when
// the table's entry is not in the pool.
__device__ __forceinline__ uint8_t* kv4_page(const Kv4& C, const int* table, int b, int n, int max_pages, int head,
                                             int* page_out = nullptr) {
    const int page = __ldg(table + (long long)b * max_pages + n);
    if ((unsigned)page >= (unsigned)C.n_pages) {
        set_error(C.err, DLLM_DEVERR_PAGE);
        return nullptr;
    }
    if (page_out) *page_out = page;
    return C.pages + page * C.page_bytes + (size_t)head * C.head_bytes;
}

// lens[b] as the kernels use it: within [0, max_tokens].
__device__ __forceinline__ int kv4_len(const Kv4& C, const int* lens, int b) {
    const int n = __ldg(lens + b);
    if (n > C.max_tokens) {
        set_error(C.err, DLLM_DEVERR_PAGE);
        return C.max_tokens;
    }
    return max(n, 0);
}

__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// (s, -(64 + z) s) for two parameters, one in each half.
struct Kv4Scale {
    uint32_t s, c;
};
__device__ __forceinline__ Kv4Scale kv4_scale(uint32_t par2) {
    Kv4Scale r;
    r.s = h2_mul(par2 & 0x7f807f80u, 0x2c002c00u);                        // 16 s / 16
    r.c = h2_mul(((par2 & 0x000f000fu) << 4) | 0xd400d400u, r.s);         // -(64 + z) s; NaN stays NaN
    return r;
}
__device__ __forceinline__ uint32_t kv4_splat(uint32_t par) { return __byte_perm(par, par, 0x1010); }

// The 8 channels of a word, in order, as four packed pairs.
__device__ __forceinline__ void kv4_widen(uint32_t w, const Kv4Scale& p, uint32_t& a, uint32_t& b, uint32_t& c,
                                          uint32_t& d) {
    a = h2_fma(((w << 4) & 0x00f000f0u) | 0x54005400u, p.s, p.c);
    b = h2_fma((w & 0x00f000f0u) | 0x54005400u, p.s, p.c);
    c = h2_fma(((w >> 4) & 0x00f000f0u) | 0x54005400u, p.s, p.c);
    d = h2_fma(((w >> 8) & 0x00f000f0u) | 0x54005400u, p.s, p.c);
}

// Host: fill C from the caller's description; a DLLM_ERR_* code.
inline int kv4_check(const dllm_kv4_cache& a, Kv4* C) {
    if (a.n_pages < 1 || a.heads < 1 || a.B < 0 || a.max_pages < 1) return DLLM_ERR_INVAL;
    const size_t bytes = dllm_kv4_page_bytes(a.page_size, a.head_dim);
    if (bytes == 0) return DLLM_ERR_UNSUPPORTED;
    if ((long long)a.max_pages * a.page_size > 0x3fffffffll || a.heads > 4096 || a.B > 65535)
        return DLLM_ERR_UNSUPPORTED;
    if (!a.pages || (a.B > 0 && !a.table)) return DLLM_ERR_INVAL;
    if (reinterpret_cast<uintptr_t>(a.pages) & 15) return DLLM_ERR_ALIGN;
    C->n_pages = a.n_pages;
    C->heads = a.heads;
    C->page_shift = 0;
    while ((1 << C->page_shift) < a.page_size) ++C->page_shift;
    C->B = a.B;
    C->max_pages = a.max_pages;
    C->max_tokens = a.max_pages * a.page_size;
    C->head_bytes = (uint32_t)bytes;
    C->page_bytes = (long long)bytes * a.heads;
    C->pages = a.pages;
    C->table = a.table;
    C->err = nullptr;
    return DLLM_OK;
}

// Host, once every argument is known to be good: the device's facts.
inline int kv4_device(Kv4* C, int* sms) {
    *sms = sm_count();
    C->err = error_word_ptr();
    return *sms > 0 && C->err ? DLLM_OK : DLLM_ERR_CUDA;
}

}  // namespace dllm
