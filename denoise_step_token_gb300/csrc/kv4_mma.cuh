// 16-row score tiles of mma.m16n8k16 over the 4-bit cache: fragments straight
// from the codes, shared by the attention of few rows and by the weights.
//
// The products' k index runs over channels in an order of our choosing, the
// same for both operands: thread t of a quad owns channels [t D/4, (t+1) D/4),
// so one load brings a thread all the codes of a key that it feeds to the
// tensor cores, and they never pass through shared memory.
#pragma once

#include "kv4.cuh"

namespace dllm {

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Query rows of one key/value head: row r is position r / group, head
// head * group + r % group.
struct QueryRows {
    const uint16_t* q;
    long long sb, sl, sh;   // strides: request, position, head
    int L, group, rows;     // rows = L * group
    __device__ __forceinline__ const uint16_t* at(int b, int head, int r) const {
        const int i = r / group;
        return q + b * sb + i * sl + (long long)(head * group + (r - i * group)) * sh;
    }
};

// The power of two that brings a row of largest magnitude `amax` into [1, 2)
// (fp16 then holds every bf16 within 2^-16 of the largest exactly and the
// others to 2^-25 of it), and its inverse.
__device__ __forceinline__ void row_power(float amax, float& down, float& up) {
    const int e = (int)(__float_as_uint(amax) >> 23) & 255;
    if (e == 255) {   // infinite: the row's results are NaN whatever the scale
        down = up = 1.0f;
        return;
    }
    const int d = min(254 - e, 252);
    down = __uint_as_float((uint32_t)max(d, 1) << 23);
    up = __uint_as_float((uint32_t)(254 - max(d, 1)) << 23);
}

// Codes and parameters of 8 keys (one n8 tile) for the score product.
template <int D>
struct KeyTile {
    static constexpr int kWords = D / 32;   // words of codes per thread
    uint32_t w[kWords];
    uint32_t par;
    // key `lane / 4` at `slot`, channels of thread lane % 4
    __device__ __forceinline__ void load(const uint8_t* page, int shift, int slot, int t) {
        const uint8_t* c = page + slot * (D / 2) + t * (D / 8);
        if constexpr (D == 128) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(c));
            w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
        } else {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(c));
            w[0] = q.x; w[1] = q.y;
        }
        par = __ldg(reinterpret_cast<const uint16_t*>(page + ((D / 2) << shift) + slot * (D / 16)) + t * (D / 4) / 32);
    }
    // b0, b1 of the D/16 products along the channels
    __device__ __forceinline__ void widen(uint32_t (&b)[D / 16][2]) const {
        const Kv4Scale p = kv4_scale(kv4_splat(par));
#pragma unroll
        for (int i = 0; i < kWords; ++i) kv4_widen(w[i], p, b[2 * i][0], b[2 * i][1], b[2 * i + 1][0], b[2 * i + 1][1]);
    }
};

}  // namespace dllm
