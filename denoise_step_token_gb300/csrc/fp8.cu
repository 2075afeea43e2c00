// dllm_fp8_quantize and dllm_fp8_matmul: a product in 8-bit floating point (e4m3)
// with a 32-bit scale for each row and 128 columns of A and for each 128 x 128
// block of B:
//   out[m][n] = sum_b sa[m][b] sb[n / 128][b] sum_{k in block b} A[m][k] B[n][k].
//
// The inner sums are the tensor cores' (kind::f8f6f4, 32-bit accumulators), a
// block of 128 at a time; the scales differ from block to block, so each inner sum
// is read back from TMEM and added, scaled, to 32-bit registers.
//
// Tile: 256 x 256 by a pair of CTAs (cta_group::2): each holds 128 rows of A and
// 128 of B, and the 128 x 256 sums of its own rows.  A block of 128 is 4 products
// of 512 cycles together; meanwhile 16 warps a CTA read 128 x 256 sums (a thread a
// row and 64 columns) and add them with 32 packed operations a thread.  What the
// pair saves is L2 traffic: 32 KB a CTA and block; single CTAs with 128 x 256 tiles
// would need 48.
// What bounds it: those sums, about 1000 cycles a block with the barriers on both
// sides (tensor pipes 53 % active).  1851 x 151936 x 3584: 870 us over the same operands again and
// again, 900 in a graph with others, 960 over changing ones (2320 to 2100 TFLOP/s: the card's power); 21 x
// 126464 x 4096: 120 to 150 us, 4.3 to 3.5 TB/s of weights.  With 8 warps of sums and 128 columns a
// thread 1037 and 187 us, where this form then took 996 and 143.
// Two TMEM buffers of 256 columns: a block's sums are read while the next block's
// are formed.  Six stages of 32 KB in shared memory.
// Tiles run along the rows of A first: the CTAs in flight share few tiles of B, which
// comes from DRAM once, and A stays in L2.  For few rows the tile is the same, though its
// sums, of rows that are not there for the most part, then take longer than reading the
// weights (77 us); no other tile has been measured.
#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "tcgen05.cuh"

namespace dllm {
namespace {

constexpr int kBlock = DLLM_FP8_BLOCK;
static_assert(kBlock == 128, "a row of a tile is one swizzle span");

// ---------------------------------------------------------------------------
// Quantising.
// ---------------------------------------------------------------------------
struct QuantizeParams {
    int M, K, blocks;
    long long x_rows, ldx;
    const uint16_t* x;
    const int* rows;
    uint8_t* codes;
    float* scale;
};

// Four packed bf16 pairs: the largest magnitude's bits (an infinity or NaN: 0x7f80 or more).
__device__ __forceinline__ uint32_t top_bits(const uint4& q) {
    const uint32_t w[4] = {q.x & 0x7fff7fffu, q.y & 0x7fff7fffu, q.z & 0x7fff7fffu, q.w & 0x7fff7fffu};
    uint32_t t = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) t = max(t, max(w[k] & 0xffffu, w[k] >> 16));
    return t;
}
constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126
__device__ __forceinline__ float scale_of(uint32_t top) {
    return top >= 0x7f80u ? __int_as_float(0x7fc00000) : fmaxf(__fdiv_rn(__uint_as_float(top << 16), 448.0f), kLeastScale);
}
// x / scale to the nearest code, for 8 values.  The quotient is the correctly rounded one, as the definition has it.
__device__ __forceinline__ uint2 codes_of(const uint4& q, float scale) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float lo = __fdiv_rn(bf16_lo(w[k]), scale), hi = __fdiv_rn(bf16_hi(w[k]), scale);
        uint16_t pair;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(hi), "f"(lo));
        c[k] = pair;
    }
    return scale == scale ? make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16) : make_uint2(0, 0);
}

constexpr int kQuantThreads = 256;
// 16 lanes a block of 128 values of one row.
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const __grid_constant__ QuantizeParams P) {
    pdl_wait();
    pdl_release();
    const int part = threadIdx.x & 15;
    const long long items = (long long)P.M * P.blocks, step = (long long)gridDim.x * (kQuantThreads / 16);
    // whole warps stay in the loop: their lanes exchange maxima
    for (long long i0 = (long long)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 5) * 2; i0 < items; i0 += step) {
        const long long i = i0 + (threadIdx.x >> 4 & 1);
        const long long m = i / P.blocks;
        const int b = (int)(i - m * P.blocks), k = b * kBlock + part * 8;
        const bool have = i < items && k < P.K;
        uint4 q = make_uint4(0, 0, 0, 0);
        if (have) {
            const long long r = P.rows ? (long long)__ldg(P.rows + m) : m;
            if (r >= 0 && r < P.x_rows) q = __ldg(reinterpret_cast<const uint4*>(P.x + r * P.ldx + k));
        }
        uint32_t top = top_bits(q);
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float s = scale_of(top);
        if (have) *reinterpret_cast<uint2*>(P.codes + m * P.K + k) = codes_of(q, s);
        if (i < items && part == 0) P.scale[i] = s;
    }
}

// A CTA a block of 128 x 128: a thread holds 8 columns of 8 rows.
__global__ void __launch_bounds__(kQuantThreads) quantize_blocks_kernel(const __grid_constant__ QuantizeParams P) {
    __shared__ uint32_t s_top[kQuantThreads / 32];
    pdl_wait();
    pdl_release();
    const int tid = threadIdx.x, k = blockIdx.x * kBlock + (tid & 15) * 8;
    const long long m0 = (long long)blockIdx.y * kBlock + (tid >> 4);
    uint4 q[8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long m = m0 + j * 16;
        q[j] = make_uint4(0, 0, 0, 0);
        if (m < P.M && k < P.K) {
            const long long r = P.rows ? (long long)__ldg(P.rows + m) : m;
            if (r >= 0 && r < P.x_rows) q[j] = __ldg(reinterpret_cast<const uint4*>(P.x + r * P.ldx + k));
        }
        top = max(top, top_bits(q[j]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) top = max(top, s_top[w]);
    const float s = scale_of(top);
    if (tid == 0) P.scale[(long long)blockIdx.y * P.blocks + blockIdx.x] = s;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long m = m0 + j * 16;
        if (m < P.M && k < P.K) *reinterpret_cast<uint2*>(P.codes + m * P.K + k) = codes_of(q[j], s);
    }
}

// ---------------------------------------------------------------------------
// The product.
// ---------------------------------------------------------------------------
constexpr int kRows = 128;                      // of A, and of B, that a CTA holds
constexpr int kTile = 2 * kRows;                // the pair's tile is kTile x kTile
constexpr int kStages = 6;
constexpr uint32_t kOperand = kRows * kBlock;   // bytes of one operand's part of a stage
constexpr int kSumWarps = 16, kCopyWarp = kSumWarps, kIssueWarp = kSumWarps + 1;
constexpr int kCols = kTile / (kSumWarps / 4);   // columns of a thread
constexpr int kThreads = (kSumWarps + 4) * 32;   // the last two warps only fill the warpgroup
// Registers per thread: 96 at launch (640 threads); the last warpgroup gives 32 each to the four that hold sums:
// 128 (96 - 64) >= 512 (104 - 96).  With 96 for all, the sums spill (1117 us for 996, 1851 x 151936 x 3584).
constexpr int kLaunchRegs = 96, kSumRegs = 104, kOtherRegs = 64;
static_assert(128 * (kLaunchRegs - kOtherRegs) >= kSumWarps * 32 * (kSumRegs - kLaunchRegs), "registers given cover those taken");
constexpr uint64_t kWaitNs = 2000000000ull;

struct MatmulParams {
    CUtensorMap a, b;
    int M, N, blocks, m_tiles;
    int wide;   // rows of out lie on 32-byte boundaries
    long long tiles;
    long long ldo;
    const float* a_scale;
    const float* b_scale;
    uint16_t* out;
    int* err;
};

struct Shared {
    uint64_t full[kStages], empty[kStages], ready[2], read[2];   // ready, read: of the TMEM buffers
    uint32_t tmem;
    int abort;
};
constexpr size_t kSmem = kStages * 2 * kOperand + 1024 + sizeof(Shared);

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t of_leader(uint32_t at) {
    uint32_t p;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(p) : "r"(at));
    return p;
}
// A box of 128 columns x 128 rows, at (column, row); its bytes count on the leader's barrier.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int col, int row, uint32_t leader_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(col), "r"(row), "r"(leader_bar)
        : "memory");
}
__device__ __forceinline__ void pair_commit(uint32_t bar) {   // arrives at both CTAs' barrier
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// e4m3 x e4m3 -> f32, kTile x kTile.
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
__device__ __forceinline__ void pair_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kIdesc), "r"(acc), "r"(kTcDescHigh)
        : "memory");
}

// A wait that gives up (and with it every later one of the CTA).
__device__ __forceinline__ void wait_for(uint32_t bar, uint32_t parity, Shared& sh, int* err) {
    if (mbar_test_wait(bar, parity) || *(volatile int*)&sh.abort) return;
    if (mbar_wait_bounded(bar, parity, kWaitNs)) return;
    set_error(err, DLLM_DEVERR_TIMEOUT);
    *(volatile int*)&sh.abort = 1;
}

__global__ void __launch_bounds__(kThreads, 1) fp8_matmul_kernel(const __grid_constant__ MatmulParams P) {
    extern __shared__ __align__(16) unsigned char raw[];
    // tiles on a 1024-byte boundary (the swizzle's atoms), at the same place in both CTAs
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    Shared& sh = *reinterpret_cast<Shared*>(raw + (base - smem_addr(raw)) + kStages * 2 * kOperand);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_rank();
    if (tid == 0) {
        sh.abort = 0;
        for (int k = 0; k < kStages; ++k) {
            mbar_init(smem_addr(&sh.full[k]), 1);
            mbar_init(smem_addr(&sh.empty[k]), 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(smem_addr(&sh.ready[k]), 1);
            mbar_init(smem_addr(&sh.read[k]), 2 * kSumWarps);
        }
        mbar_fence_init();
    }
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    pdl_wait();
    pdl_release();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (warp >= kSumWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kSumWarps) {
        // ---------------------------------------------------------- sums: a thread a row and kCols columns
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        const int part = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // the warp's quarter of TMEM's lanes
        uint32_t n = 0;
        for (long long t = pair; t < P.tiles; t += pairs) {
            const int m = (int)(t % P.m_tiles) * kTile + rank * kRows + (warp & 3) * 32 + lane;
            const int n0 = (int)(t / P.m_tiles) * kTile + part * kCols;
            const float* const sa = P.a_scale + (long long)min(m, P.M - 1) * P.blocks;
            const float* const sb = P.b_scale + (long long)min(n0 / kBlock, (P.N - 1) / kBlock) * P.blocks;
            unsigned long long acc[kCols / 2];
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) acc[c] = 0;
            float sa_next = __ldg(sa), sb_next = __ldg(sb);
            for (int b = 0; b < P.blocks; ++b, ++n) {
                const uint32_t buf = n & 1;
                // The scales' product, where it is a normal number.  Where it is not, the sum is multiplied by one after the
                // other: above 2^128 by the smaller (>= 1) first, below 2^-126 by the larger (< 2^23) first, so that nothing
                // passes the range on the way unless the result does.  Scales of 2^-126 (kLeastScale) are left with the
                // product: they belong to groups of zeros, and the multiplications cost 1030 us for 880 where a warp
                // has such a row (1851 x 151936 x 3584).
                const float both = sa_next * sb_next, lo = fminf(sa_next, sb_next), hi = fmaxf(sa_next, sb_next);
                const bool small = fabsf(both) < kLeastScale;
                const bool alone = (small && lo > 0.0f && lo != kLeastScale) || fabsf(both) == INFINITY;   // (0: the product is 0)
                const bool apart = __any_sync(0xffffffffu, alone);
                const unsigned long long s2 = f32x2_splat(alone ? small ? lo : hi : both);
                const unsigned long long first = f32x2_splat(alone ? small ? hi : lo : 1.0f);
                if (b + 1 < P.blocks) {
                    sa_next = __ldg(sa + b + 1);
                    sb_next = __ldg(sb + b + 1);
                }
                wait_for(smem_addr(&sh.ready[buf]), n >> 1 & 1, sh, P.err);
                __syncwarp();
                tc_fence_after();
                const uint32_t from = tmem + lanes + buf * kTile + part * kCols;
#pragma unroll
                for (int c0 = 0; c0 < kCols; c0 += 16) {
                    uint32_t v[16];
                    tc_ld16(v, from + c0);
                    tc_wait_ld();
                    if (c0 + 16 == kCols) {   // all read: the next block but one may be formed
                        tc_fence_before();
                        __syncwarp();
                        // (released at CTA scope: no memory but TMEM is handed over, and a cluster-wide release costs
                        // 1500 cycles)
                        if (lane == 0)
                            asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(of_leader(smem_addr(&sh.read[buf])))
                                         : "memory");
                    }
                    if (apart) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const unsigned long long y =
                                f32x2_mul(f32x2_pack(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), first);
                            v[2 * c] = __float_as_uint(f32x2_lo(y));
                            v[2 * c + 1] = __float_as_uint(f32x2_hi(y));
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        acc[c0 / 2 + c] = f32x2_fma(f32x2_pack(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), s2,
                                                    acc[c0 / 2 + c]);
                }
            }
            if (m < P.M) {
                uint16_t* const row = P.out + (long long)m * P.ldo + n0;
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    if (n0 + c >= P.N) break;
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float lo = n0 + c + 2 * k < P.N ? f32x2_lo(acc[c / 2 + k]) : 0.0f;
                        const float hi = n0 + c + 2 * k + 1 < P.N ? f32x2_hi(acc[c / 2 + k]) : 0.0f;
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(hi), "f"(lo));
                    }
                    if (P.wide && n0 + c + 8 < P.N) {   // whole 32-byte sectors (halves of them: 1010 us for 887)
                        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(row + c), "r"(w[0]), "r"(w[1]),
                                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                                     : "memory");
                    } else {
                        *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
                        if (n0 + c + 8 < P.N) *reinterpret_cast<uint4*>(row + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
            }
        }
    } else if (warp == kCopyWarp) {
        if (lane == 0) {
            uint32_t n = 0;
            for (long long t = pair; t < P.tiles; t += pairs) {
                const int m0 = (int)(t % P.m_tiles) * kTile + rank * kRows, n0 = (int)(t / P.m_tiles) * kTile + rank * kRows;
                for (int b = 0; b < P.blocks; ++b, ++n) {
                    const uint32_t s = n % kStages;
                    wait_for(smem_addr(&sh.empty[s]), (n / kStages & 1) ^ 1, sh, P.err);
                    if (*(volatile int*)&sh.abort) break;
                    const uint32_t bar = of_leader(smem_addr(&sh.full[s])), at = base + s * 2 * kOperand;
                    if (rank == 0) mbar_arrive_expect_tx(smem_addr(&sh.full[s]), 4 * kOperand);
                    load_box(at, &P.a, b * kBlock, m0, bar);
                    load_box(at + kOperand, &P.b, b * kBlock, n0, bar);
                }
                if (*(volatile int*)&sh.abort) break;
            }
            // the stages' last releases land in this CTA's memory: it is left after them
            for (uint32_t k = n > kStages ? n - kStages : 0; k < n; ++k)
                wait_for(smem_addr(&sh.empty[k % kStages]), k / kStages & 1, sh, P.err);
        }
    } else if (warp == kIssueWarp) {
        if (lane == 0 && rank == 0) {
            uint32_t n = 0;
            for (long long t = pair; t < P.tiles; t += pairs)
                for (int b = 0; b < P.blocks; ++b, ++n) {
                    const uint32_t s = n % kStages, buf = n & 1;
                    wait_for(smem_addr(&sh.read[buf]), (n >> 1 & 1) ^ 1, sh, P.err);
                    wait_for(smem_addr(&sh.full[s]), n / kStages & 1, sh, P.err);
                    if (*(volatile int*)&sh.abort) break;
                    tc_fence_after();
                    const uint32_t at = base + s * 2 * kOperand;
                    const uint32_t da = tc_desc_low(at, 0), db = tc_desc_low(at + kOperand, 0);
#pragma unroll
                    for (int k = 0; k < kBlock / 32; ++k) pair_mma(tmem + buf * kTile, da + k * 2, db + k * 2, k > 0);
                    pair_commit(smem_addr(&sh.empty[s]));
                    pair_commit(smem_addr(&sh.ready[buf]));
                }
        }
    }
    // after a wait that gave up: copies still in flight land before the CTA's memory is another's
    if (*(volatile int*)&sh.abort) __nanosleep(1000000);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == kIssueWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int encoder(EncodeTiled* out) {
    static std::atomic<void*> known{nullptr};
    void* fn = known.load(std::memory_order_acquire);
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        DLLM_CUDA_TRY(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found));
        if (found != cudaDriverEntryPointSuccess || !fn) {
            note_cuda_error(cudaErrorNotSupported);
            return DLLM_ERR_CUDA;
        }
        known.store(fn, std::memory_order_release);
    }
    *out = reinterpret_cast<EncodeTiled>(fn);
    return DLLM_OK;
}

// Rows of K bytes, `ld` apart; boxes of 128 x 128 bytes, zeros outside.
int make_map(EncodeTiled encode, CUtensorMap* map, const void* p, int K, int rows, long long ld) {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {kBlock, kRows}, steps[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, steps,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return DLLM_OK;
    note_cuda_error(cudaErrorInvalidValue);
    return DLLM_ERR_CUDA;
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" int dllm_fp8_quantize(const dllm_fp8_quantize_args* a, void* stream) {
    if (!a || a->M < 0 || a->K < 1 || a->x_rows < 0 || a->ldx < a->K) return DLLM_ERR_INVAL;
    if (a->block_rows != 1 && a->block_rows != kBlock) return DLLM_ERR_INVAL;
    if (a->M > 0 && ((a->x_rows > 0 && !a->x) || !a->codes || !a->scale)) return DLLM_ERR_INVAL;
    if (a->K % 16 || a->ldx % 8 || (reinterpret_cast<uintptr_t>(a->x) & 15) || (reinterpret_cast<uintptr_t>(a->codes) & 15))
        return DLLM_ERR_ALIGN;
    if (a->K > 1 << 24 || a->M > 65535 * kBlock) return DLLM_ERR_UNSUPPORTED;
    if (a->M == 0) return DLLM_OK;
    const int sms = sm_count();
    if (sms <= 0) return DLLM_ERR_CUDA;
    QuantizeParams P{a->M, a->K, (a->K + kBlock - 1) / kBlock, a->x_rows, a->ldx, a->x, a->rows, a->codes, a->scale};
    cudaStream_t s = as_stream(stream);
    if (a->block_rows == 1) {
        const long long ctas = ((long long)P.M * P.blocks + kQuantThreads / 16 - 1) / (kQuantThreads / 16);
        DLLM_CUDA_TRY(launch_dependent(quantize_rows_kernel, dim3((unsigned)std::min<long long>(ctas, sms * 8ll)),
                                       dim3(kQuantThreads), 0, s, P));
    } else {
        DLLM_CUDA_TRY(launch_dependent(quantize_blocks_kernel, dim3(P.blocks, (P.M + kBlock - 1) / kBlock),
                                       dim3(kQuantThreads), 0, s, P));
    }
    return DLLM_OK;
}

extern "C" int dllm_fp8_matmul(const dllm_fp8_matmul_args* a, void* stream) {
    if (!a || a->M < 0 || a->N < 1 || a->K < 1 || a->lda < a->K || a->ldb < a->K || a->ldo < ((long long)a->N + 7) / 8 * 8)
        return DLLM_ERR_INVAL;
    if (a->M > 0 && (!a->a || !a->b || !a->a_scale || !a->b_scale || !a->out)) return DLLM_ERR_INVAL;
    const uintptr_t all = reinterpret_cast<uintptr_t>(a->a) | reinterpret_cast<uintptr_t>(a->b) | reinterpret_cast<uintptr_t>(a->out);
    if ((all & 15) || a->K % 16 || a->lda % 16 || a->ldb % 16 || a->ldo % 8) return DLLM_ERR_ALIGN;
    if (a->K > 1 << 24 || a->M > 1 << 28 || a->N > 1 << 28 || a->lda > 1ll << 38 || a->ldb > 1ll << 38)
        return DLLM_ERR_UNSUPPORTED;
    if (a->M == 0) return DLLM_OK;
    const int sms = sm_count();
    MatmulParams P;
    P.err = error_word_ptr();
    if (sms < 2 || !P.err) return DLLM_ERR_CUDA;
    EncodeTiled encode = nullptr;
    int rc = encoder(&encode);
    if (rc == DLLM_OK) rc = make_map(encode, &P.a, a->a, a->K, a->M, a->lda);
    if (rc == DLLM_OK) rc = make_map(encode, &P.b, a->b, a->K, a->N, a->ldb);
    if (rc != DLLM_OK) return rc;
    P.M = a->M;
    P.N = a->N;
    P.blocks = (a->K + kBlock - 1) / kBlock;
    P.m_tiles = (a->M + kTile - 1) / kTile;
    P.tiles = (long long)P.m_tiles * ((a->N + kTile - 1) / kTile);
    P.ldo = a->ldo;
    P.wide = a->ldo % 16 == 0 && (reinterpret_cast<uintptr_t>(a->out) & 31) == 0;
    P.a_scale = a->a_scale;
    P.b_scale = a->b_scale;
    P.out = a->out;
    static SmemOnce done;
    DLLM_CUDA_TRY(allow_smem(fp8_matmul_kernel, kSmem, done));
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_acquire) == 0) {
        cudaFuncAttributes attr;
        DLLM_CUDA_TRY(cudaFuncGetAttributes(&attr, fp8_matmul_kernel));
        regs.store(attr.numRegs, std::memory_order_release);
    }
    // the split of registers above is of kLaunchRegs: with fewer at launch the sums' warps would wait for ever
    if (regs.load(std::memory_order_acquire) != kLaunchRegs) return DLLM_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long long>(P.tiles, sms / 2) * 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    DLLM_CUDA_TRY(cudaLaunchKernelEx(&cfg, fp8_matmul_kernel, P));
    return DLLM_OK;
}
