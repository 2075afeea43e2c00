// dllm_kv4_write: keys and values into the paged 4-bit cache.
//
// Mathematics, per group of 32 channels with its range widened to hold 0:
// s = (max - min) / 15 rounded up to 4 significant bits, z = rint(-min / s),
// u = clamp(rint(x / s) + z, 0, 15), with s cut to its upper bound after z is
// chosen (what is too large for it saturates on both sides).  The divisions are IEEE ones: for bf16
// inputs x / s is a ratio of an 8-bit and a 4-bit integer, which a correctly
// rounded 32-bit quotient never moves across a half, so the codes are those of
// the definition in exact arithmetic.
//
// What bounds it: memory (4 D bytes read per token and head, 1.125 D written,
// 4 D more with the values out); a block's write is launch latency.
//
// Layout.  Four lanes hold a group, 8 channels (one 16-byte load) each: a warp
// reads 512 contiguous bytes, finds the range with two shuffles, and each lane
// writes one word of codes, so that codes leave in 128-byte runs.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kv4.cuh"

namespace dllm {
namespace {

struct WriteParams {
    Kv4 C;
    int W, D;
    const uint16_t* x[2];
    long long stride[2][3];
    uint16_t* out[2];
    const int* pos;
    const int* first;
    const int* count;
};

__device__ __forceinline__ int nibble(float x, float s, float z) {
    return (int)fminf(fmaxf(rintf(__fdiv_rn(x, s)) + z, 0.0f), 15.0f);
}

// grid: (token tiles, 1, requests); a thread's item: 8 channels of one (column, k or v, head).
__global__ void __launch_bounds__(256) kv4_write_kernel(const __grid_constant__ WriteParams P) {
    pdl_wait();
    pdl_release();
    const int b = blockIdx.z;
    const int first = P.first ? P.first[b] : 0;
    const int count = P.count ? P.count[b] : P.W - first;
    const int pos = P.pos[b];
    const int lo = max(first, 0), hi = min((long long)P.W, (long long)first + count);
    if (pos < 0 || (long long)pos + count > P.C.max_tokens || first < 0 || (long long)first + count > P.W) {
        if (count > 0) {
            if (threadIdx.x == 0) set_error(P.C.err, DLLM_DEVERR_PAGE);
            return;
        }
    }
    const int lanes = P.D >> 3;                      // threads per head row
    const int per_token = lanes * P.C.heads * 2;     // a multiple of 16
    const long long total = (long long)max(hi - lo, 0) * per_token;
    const int page_mask = (1 << P.C.page_shift) - 1;
    for (long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x; at < total;
         at += (long long)gridDim.x * blockDim.x) {
        // total is a multiple of 16, so the four lanes of a group are here together
        const unsigned mask = 0xfu << (threadIdx.x & 28);
        const int c = lo + (int)(at / per_token);
        int rest = (int)(at - (long long)(c - lo) * per_token);
        const int which = rest >= per_token / 2;
        rest -= which ? per_token / 2 : 0;
        const int head = rest / lanes, l = rest - head * lanes;
        const uint16_t* src = P.x[which] + b * P.stride[which][0] + c * P.stride[which][1] + head * P.stride[which][2];
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(src) + l);
        float x[8];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = bf16_lo(w[k]);
            x[2 * k + 1] = bf16_hi(w[k]);
        }
        float low = 0.0f, high = 0.0f;
        bool finite = true;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            low = fminf(low, x[k]);
            high = fmaxf(high, x[k]);
            finite = finite && isfinite(x[k]);
        }
        int bad = !finite;
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            low = fminf(low, __shfl_xor_sync(mask, low, off));
            high = fmaxf(high, __shfl_xor_sync(mask, high, off));
            bad |= __shfl_xor_sync(mask, bad, off);
        }
        float s = __fdiv_rn(__fsub_rn(high, low), 15.0f);
        s = __uint_as_float((__float_as_uint(s) + 0xfffffu) & ~0xfffffu);   // up to 4 significant bits
        s = fmaxf(s, kKv4MinStep);
        const float z = fminf(rintf(__fdiv_rn(-low, s)), 15.0f);
        s = fminf(s, kKv4MaxStep);
        uint32_t word = 0;
        uint32_t val[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int u0 = nibble(x[2 * k], s, z), u1 = nibble(x[2 * k + 1], s, z);
            word |= (uint32_t)u0 << (4 * k) | (uint32_t)u1 << (16 + 4 * k);
            // 8 significant bits: the upper half of the float is the bf16 value
            const float y0 = bad ? NAN : s * ((float)u0 - z), y1 = bad ? NAN : s * ((float)u1 - z);
            val[k] = __byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x7632);
        }
        const uint16_t par = bad ? kKv4NanParam
                                 : (uint16_t)(__half_as_ushort(__float2half_rn(16.0f * s)) | (unsigned)z);
        const int j = pos + (c - first);
        uint8_t* page = kv4_page(P.C, P.C.table, b, j >> P.C.page_shift, P.C.max_pages, head);
        if (page) {
            const int slot = j & page_mask;
            page += which ? P.C.head_bytes / 2 : 0;
            reinterpret_cast<uint32_t*>(page + (size_t)slot * (P.D / 2))[l] = bad ? 0u : word;
            uint8_t* pars = page + ((size_t)(P.D / 2) << P.C.page_shift);
            if ((l & 3) == 0) reinterpret_cast<uint16_t*>(pars + (size_t)slot * (P.D / 16))[l >> 2] = par;
        }
        if (P.out[which]) {
            uint16_t* o = P.out[which] + (((long long)b * P.W + c) * P.C.heads + head) * P.D;
            reinterpret_cast<uint4*>(o)[l] = make_uint4(val[0], val[1], val[2], val[3]);
        }
    }
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_kv4_page_bytes(int32_t page_size, int32_t head_dim) {
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return 0;
    if (head_dim != 64 && head_dim != 128) return 0;
    return (size_t)page_size * (head_dim + head_dim / 8);
}

extern "C" int dllm_kv4_write(const dllm_kv4_write_args* a, void* stream) {
    if (!a) return DLLM_ERR_INVAL;
    WriteParams P;
    int rc = kv4_check(a->cache, &P.C);
    if (rc != DLLM_OK) return rc;
    if (a->W < 0) return DLLM_ERR_INVAL;
    if (a->W == 0 || a->cache.B == 0) return DLLM_OK;
    if (!a->k || !a->v || !a->pos) return DLLM_ERR_INVAL;
    const uintptr_t bases = reinterpret_cast<uintptr_t>(a->k) | reinterpret_cast<uintptr_t>(a->v) |
                            reinterpret_cast<uintptr_t>(a->k_out) | reinterpret_cast<uintptr_t>(a->v_out);
    if (bases & 15) return DLLM_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if (a->k_stride[i] % 8 || a->v_stride[i] % 8) return DLLM_ERR_ALIGN;
    int sms = 0;
    rc = kv4_device(&P.C, &sms);
    if (rc != DLLM_OK) return rc;
    P.W = a->W;
    P.D = a->cache.head_dim;
    P.x[0] = a->k;
    P.x[1] = a->v;
    for (int i = 0; i < 3; ++i) {
        P.stride[0][i] = a->k_stride[i];
        P.stride[1][i] = a->v_stride[i];
    }
    P.out[0] = a->k_out;
    P.out[1] = a->v_out;
    P.pos = a->pos;
    P.first = a->first;
    P.count = a->count;
    const long long items = (long long)a->W * a->cache.heads * (P.D / 8) * 2;
    const long long most = std::max<long long>(1, (long long)sms * 64 / a->cache.B);
    const unsigned gx = (unsigned)std::min<long long>((items + 255) / 256, most);
    DLLM_CUDA_TRY(launch_dependent(kv4_write_kernel, dim3(gx, 1, a->cache.B), dim3(256), 0, as_stream(stream), P));
    return DLLM_OK;
}
