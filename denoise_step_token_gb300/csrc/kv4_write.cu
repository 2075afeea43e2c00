// dllm_kv4_write: keys and values into the paged 4-bit cache.
//
// Mathematics, per group of 32 channels with its range widened to hold 0:
// s = (max - min) / 15 rounded up to 4 significant bits, z = rint(-min / s),
// u = clamp(rint(x / s) + z, 0, 15), with s cut to its upper bound after z is
// chosen (what is too large for it saturates on both sides).  For bf16 inputs
// x / s is a ratio of an 8-bit and a 4-bit integer, which a correctly rounded
// 32-bit quotient never moves across a half, so the codes are those of the
// definition in exact arithmetic: a quotient within the codes' range is either a
// half or at least 1/510 away from one.  So x (1/s), one fma, is first rounded to
// multiples of 2^-10 by adding 1.5 * 2^13 (halves stay halves, nothing else
// becomes one), clamped to [-z, 15 - z], and then to integers by adding
// 1.5 * 2^23 - 1.5 * 2^13.
//
// What bounds it: memory (4 D bytes read per token and head, 1.125 D written,
// 4 D more with the values out); a block's write is launch latency.
//
// Layout.  Four lanes hold a group, 8 channels (one 16-byte load) each: a warp
// reads 512 contiguous bytes, finds the range in packed bf16 with two shuffles
// (the maximum and the negated minimum in one register), and each lane writes
// one word of codes.  A head's row is D/8 lanes, so codes leave in runs of D/2
// bytes (64 at D = 128: half a cache line, two heads to a warp) and parameters of
// D/16, which keeps large writes from the memory's rate: 64 prompts of up to 1024
// tokens and 32 heads move 4.9 TB/s.  A thread keeps its place within a column
// (head, channels) and steps through columns, with four loads in flight.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kv4.cuh"

namespace dllm {
namespace {

struct WriteParams {
    Kv4 C;
    int W, lane_shift, per_token;   // 8-channel items per head row (their log2) and per column
    const uint16_t* x[2];
    long long stride[2][3];
    uint16_t* out[2];
    const int* pos;
    const int* first;
    const int* count;
};

constexpr int kAtOnce = 4;   // loads in flight per thread

__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// grid: (column tiles, 1, requests), gridDim.x * 256 a multiple of per_token.  An
// item: 8 channels of one (column, k or v, head).
__global__ void __launch_bounds__(256) kv4_write_kernel(const __grid_constant__ WriteParams P) {
    pdl_wait();
    pdl_release();
    const int b = blockIdx.z;
    const int first = P.first ? P.first[b] : 0;
    const int count = P.count ? P.count[b] : P.W - max(first, 0);   // a negative first is refused below
    const int pos = P.pos[b];
    if (count <= 0) return;
    if (pos < 0 || (long long)pos + count > P.C.max_tokens || first < 0 || (long long)first + count > P.W) {
        if (threadIdx.x == 0) set_error(P.C.err, DLLM_DEVERR_PAGE);
        return;
    }
    // the thread's place within a column, and its first column; per_token is a multiple of 16, so the four lanes
    // of a group have the same columns
    const int at = blockIdx.x * 256 + threadIdx.x;
    const int dcol = (int)(gridDim.x * 256) / P.per_token;
    const int col0 = at / P.per_token, rest = at - col0 * P.per_token;
    const int which = rest >= P.per_token / 2;
    const int in = rest - (which ? P.per_token / 2 : 0);
    const int head = in >> P.lane_shift, l = in & ((1 << P.lane_shift) - 1);
    const int D = 8 << P.lane_shift, shift = P.C.page_shift;
    const unsigned quad = 0xfu << (threadIdx.x & 28);
    const long long sc = P.stride[which][1];
    const uint16_t* src = P.x[which] + b * P.stride[which][0] + (first + col0) * sc + head * P.stride[which][2] + l * 8;
    uint16_t* dst = P.out[which];
    const long long dst_step = (long long)P.C.heads * D;
    if (dst) dst += (((long long)b * P.W + first + col0) * P.C.heads + head) * D + l * 8;
    const uint32_t in_page = (uint32_t)head * P.C.head_bytes + (which ? P.C.head_bytes / 2 : 0);
    const uint32_t par_at = (uint32_t)(D / 2) << shift;
    const int* table = P.C.table + (long long)b * P.C.max_pages;
    for (int c0 = col0; c0 < count; c0 += kAtOnce * dcol) {
        uint4 q[kAtOnce];
        int page[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int c = c0 + u * dcol;
            if (c < count) {
                q[u] = __ldcs(reinterpret_cast<const uint4*>(src + (long long)(u * dcol) * sc));
                page[u] = __ldg(table + ((pos + c) >> shift));
            }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int c = c0 + u * dcol;
            if (c >= count) break;
            const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
            const uint32_t hi2 = bf16x2_max_nan(bf16x2_max_nan(w[0], w[1]), bf16x2_max_nan(w[2], w[3]));
            const uint32_t lo2 = bf16x2_max_nan(bf16x2_max_nan(w[0] ^ 0x80008000u, w[1] ^ 0x80008000u),
                                                bf16x2_max_nan(w[2] ^ 0x80008000u, w[3] ^ 0x80008000u));
            // (max, -min), at least 0: the range holds 0
            uint32_t range = bf16x2_max_nan(__byte_perm(hi2, lo2, 0x5410), __byte_perm(hi2, lo2, 0x7632));
            range = bf16x2_max_nan(range, __shfl_xor_sync(quad, range, 1));
            range = bf16x2_max_nan(range, __shfl_xor_sync(quad, range, 2));
            range = bf16x2_max_nan(range, 0u);
            const bool bad = (range & 0x7f80u) == 0x7f80u || (range & 0x7f800000u) == 0x7f800000u;
            // halves: the whole range, up to twice bf16's largest, may pass 32 bits (what halving loses of subnormal
            // numbers is far under the least step)
            const float low = bf16_hi(range), wide = fmaf(bf16_lo(range), 0.5f, 0.5f * low);   // low: negated
            // wide / 15 correctly rounded (P. Markstein, "Computation of elementary functions on the IBM RISC
            // System/6000 processor", 1990), then up to 4 significant bits
            constexpr float k15 = 1.0f / 15.0f;
            float s = __fmul_rn(wide, k15);
            s = fmaf(fmaf(-s, 15.0f, wide), k15, s);
            s = __uint_as_float((__float_as_uint(s) + 0xfffffu) & ~0xfffffu);
            s = fmaxf(2.0f * s, kKv4MinStep);
            constexpr float kGrid = 12288.0f, kInt = 12582912.0f;   // 1.5 * 2^13, 1.5 * 2^23
            float r = __frcp_rn(s);
            const float z = fminf((fmaf(low, r, kGrid) + (kInt - kGrid)) - kInt, 15.0f);
            if (s > kKv4MaxStep) {
                s = kKv4MaxStep;
                r = __frcp_rn(s);
            }
            const float least = kGrid - z, most = kGrid + (15.0f - z), sk = -s * kInt;   // all exact
            // the integer n of kInt + n is its lowest bits: words add up modulo 2^32, the constants taken off once
            uint32_t word = 0;
            uint32_t val[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float n0 = fminf(fmaxf(fmaf(bf16_lo(w[k]), r, kGrid), least), most) + (kInt - kGrid);
                const float n1 = fminf(fmaxf(fmaf(bf16_hi(w[k]), r, kGrid), least), most) + (kInt - kGrid);
                word += __float_as_uint(n0) * (1u << (4 * k)) + __float_as_uint(n1) * (1u << (16 + 4 * k));
                // s n has 8 significant bits: the upper half of the float is the bf16 value
                val[k] = __byte_perm(__float_as_uint(fmaf(s, n0, sk)), __float_as_uint(fmaf(s, n1, sk)), 0x7632);
            }
            const uint32_t zi = (uint32_t)(int)z;
            word += (zi - 0x4b400000u) * 0x11111111u;
            uint32_t par = (uint32_t)__half_as_ushort(__float2half_rn(16.0f * s)) | zi;
            if (bad) {
                word = 0;
                par = kKv4NanParam;
#pragma unroll
                for (int k = 0; k < 4; ++k) val[k] = 0x7fff7fffu;
            }
            if ((unsigned)page[u] < (unsigned)P.C.n_pages) {
                const uint32_t slot = (uint32_t)(pos + c) & ((1u << shift) - 1);
                uint8_t* p = P.C.pages + (page[u] * P.C.page_bytes + in_page);
                reinterpret_cast<uint32_t*>(p + slot * (D / 2))[l] = word;
                if ((l & 3) == 0) reinterpret_cast<uint16_t*>(p + par_at + slot * (D / 16))[l >> 2] = (uint16_t)par;
            } else {
                set_error(P.C.err, DLLM_DEVERR_PAGE);
            }
            if (dst) __stcs(reinterpret_cast<uint4*>(dst + (long long)(u * dcol) * dst_step), make_uint4(val[0], val[1], val[2], val[3]));
        }
        src += (long long)(kAtOnce * dcol) * sc;
        if (dst) dst += (long long)(kAtOnce * dcol) * dst_step;
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
    if ((long long)a->W * a->cache.heads * a->cache.head_dim / 4 > (1 << 30)) return DLLM_ERR_UNSUPPORTED;
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
    P.lane_shift = a->cache.head_dim == 128 ? 4 : 3;
    P.per_token = (a->cache.heads << P.lane_shift) * 2;
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
    // whole columns per step of the grid: its threads a multiple of per_token (16 times an integer).  One item
    // per thread for a block's write, up to 32 CTAs per SM for larger ones (8, 16, 64 in brackets): 64 prompts of
    // 1024 tokens and 32 heads 455 us (506, 464, 457), 16 of 512 and 8 heads 26 (19, 21, 34).
    int unit = P.per_token / 16;
    for (int two = 0; two < 4 && unit % 2 == 0; ++two) unit /= 2;   // per_token / gcd(per_token, 256)
    const long long items = (long long)a->W * P.per_token;
    const long long most = std::max<long long>(1, (long long)sms * 32 / a->cache.B);
    long long gx = std::min<long long>((items + 255) / 256, most);
    gx = (gx + unit - 1) / unit * unit;
    if (gx > (1 << 22)) return DLLM_ERR_UNSUPPORTED;
    DLLM_CUDA_TRY(launch_dependent(kv4_write_kernel, dim3((unsigned)gx, 1, a->cache.B), dim3(256), 0, as_stream(stream), P));
    return DLLM_OK;
}
