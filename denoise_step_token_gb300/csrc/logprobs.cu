// dllm_logprobs: log probabilities of given tokens, entropy and the best
// alternatives of logits rows, in one pass over each row.
//
// Mathematics, in base 2 (c = log2 e).  With m = max x, y_v = c x_v - c m,
// z = sum 2^y and t = sum 2^y y:
//   log p_v = ln 2 (y_v - log2 z),   entropy = ln 2 (log2 z - t / z).
// m, z and t are kept running: moving from m to m' >= m with d = c m - c m'
// scales z by f = 2^d and takes t to f (t + z d).
//
// What bounds it: reading the rows (about 4.5 instructions a value, under half
// of what an SM can issue while its share of memory arrives), or, for a row or
// two, the launch and the joins.
//
// Split.  All entries' rounds (a round: 128 threads x 64 bytes of a row) are one
// stream, cut evenly over the CTAs, six per SM.  A fifth warp keeps up to four
// rounds of its CTA in flight as bulk copies (8 KB each, 190 KB per SM: under
// load a copy lands about 2.8 us after its issue, and with the next round's loads
// in registers, 64 KB per SM, the stream ran at 4.4 TB/s).  A CTA writes the
// entries that lie wholly in its share; what it has of the two others it
// publishes (sums and best keys), and whichever CTA arrives last at an entry
// joins the parts in stream order.
//
// Best alternatives.  A value and its token make one 64-bit key (the value's
// order-preserving bits above the inverted token), so all keys differ and
// larger keys come first.  The streaming threads only compare their round's
// maximum with a floor; a warp looks through the 32 values of a thread whose
// maximum passes, one value per lane, while the round is in shared memory, and
// appends the keys above the floor to a list.  After rounds 1, 4, 16, ... the list
// is sorted by counting down to the best `top`, and the floor rises to the last
// of them: about 3 `top` keys come while what was seen grows fourfold.  The
// first floor: in each full warp the q-th largest of its lanes' maxima, q warps
// >= top, and the least of those over the warps; at least `top` values of the
// round reach it.  Rows that overfill the list (sorted ones, many equal values)
// take a radix selection over the CTA's part of the row instead.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"

namespace dllm {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 128;         // streaming threads of a CTA
constexpr int kWarps = kThreads / 32;
constexpr int kVec = 4;              // 16-byte loads per thread and round
constexpr int kStages = 4;
constexpr uint32_t kRoundBytes = kThreads * kVec * 16;
constexpr int kPerSm = 6;            // CTAs: what the rings leave room for
constexpr int kMaxCtas = 1024;
constexpr uint64_t kWaitNs = 2000000000ull;   // any single wait gives up after 2 s
constexpr int kCap = 256;            // candidate keys of a stage, the best so far among them
constexpr float kPlain = 16384.0f;   // maxima up to this size take the packed loop
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct LogprobParams {
    int N, V, top, rounds, ctas;     // rounds per row
    long long total;                 // rounds of all entries
    long long ldv, logits_rows;
    const void* logits;
    const int* rows;
    const int* tokens;
    float* logprob;
    float* entropy;
    int* top_ids;
    float* top_logprobs;
    int* counters;    // [ctas], zero between calls: of the entry that ends the CTA's share
    float4* partial;  // [ctas][2] (m, z, t, -): of the entry that begins the share, and the one that ends it
    u64* keys;        // [ctas][2][top]
    int* err;

    __device__ __forceinline__ long long share(int c) const { return total * c / ctas; }
    // the CTA whose share holds round g
    __device__ __forceinline__ int owner(long long g) const {
        int c = (int)(g * ctas / total);
        while (c + 1 < ctas && share(c + 1) <= g) ++c;
        while (c > 0 && share(c) > g) --c;
        return c;
    }
    __device__ __forceinline__ long long row_of(int i) const {
        const long long r = rows ? (long long)__ldg(rows + i) : i;
        return r >= 0 && r < logits_rows ? r : -1;
    }
};

// The streaming warps' own barrier (the copying warp runs ahead of it).
__device__ __forceinline__ void sync_streams() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Bits in the order of the values (-0 as +0), 0 < key for every float.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ u64 make_key(float x, int v) {
    return ((u64)ordered(x) << 32) | (uint32_t)~v;
}
// The value a key >= k must reach (k below every key: -inf).
__device__ __forceinline__ float key_floor(u64 k) {
    return (uint32_t)(k >> 32) < 0x007fffffu ? -INFINITY : unordered((uint32_t)(k >> 32));
}
__device__ __forceinline__ int key_token(u64 k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float key_value(u64 k) { return unordered((uint32_t)(k >> 32)); }

struct Sums {
    float m, z, t;
};

// Sums under a maximum within kPlain are formed with c m rounded once, the same
// everywhere: their y are c (x - m) + offset2(m).  Beyond it they are c (x - m).
__device__ __forceinline__ float offset2(float m) {
    return fabsf(m) <= kPlain ? fmaf(m, kLog2e, -__fmul_rn(m, kLog2e)) : 0.0f;
}
// What takes sums under a to sums under b: c a - c b as they hold it.
__device__ __forceinline__ float diff2(float a, float b) {
    return fabsf(b) <= kPlain && fabsf(a) <= kPlain ? __fsub_rn(__fmul_rn(a, kLog2e), __fmul_rn(b, kLog2e))
                                                    : fmaf(a - b, kLog2e, offset2(b) - offset2(a));
}
// ln p of one value, lz = log2 z: by the y the sums were formed with where c x
// is sure to be finite.
__device__ __forceinline__ float log_prob(float x, float m, float lz) {
    if (fabsf(m) <= kPlain && fabsf(x) <= kPlain) return (fmaf(x, kLog2e, -__fmul_rn(m, kLog2e)) - lz) * kLn2;
    return (x - m) - (lz - offset2(m)) * kLn2;
}

// (a, then b): sums over both ranges.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
    Sums r;
    r.m = max_nan(a.m, b.m);
    if (r.m == -INFINITY) return Sums{-INFINITY, 0.0f, 0.0f};
    // a side without a finite value has z = 0 and drops out
    const float da = fmaxf(diff2(a.m, r.m), -1e4f), db = fmaxf(diff2(b.m, r.m), -1e4f);
    const float fa = exp2f(da), fb = exp2f(db);
    r.z = a.z * fa + b.z * fb;
    r.t = fa * (a.t + a.z * da) + fb * (b.t + b.z * db);
    return r;
}

template <typename T>
struct Round;   // one thread's values of a round

template <>
struct Round<uint16_t> {
    static constexpr int kPer = 8;   // values per 16-byte load
    static __device__ __forceinline__ float get(const uint4& q, int k) {
        const uint32_t w = k < 2 ? q.x : k < 4 ? q.y : k < 6 ? q.z : q.w;
        return (k & 1) ? bf16_hi(w) : bf16_lo(w);
    }
    static constexpr uint32_t kNegInfWord = 0xff80ff80u;
};
template <>
struct Round<float> {
    static constexpr int kPer = 4;
    static __device__ __forceinline__ float get(const uint4& q, int k) {
        return __uint_as_float(k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w);
    }
    static constexpr uint32_t kNegInfWord = 0xff800000u;
};

// This thread's values of a round in shared memory; pieces past V: -inf.
template <typename T>
__device__ __forceinline__ void load_round(uint4 (&q)[kVec], const unsigned char* stage, int v0, int V) {
    constexpr int per = Round<T>::kPer;
#pragma unroll
    for (int i = 0; i < kVec; ++i) q[i] = reinterpret_cast<const uint4*>(stage)[i * kThreads + (int)threadIdx.x];
    if (V - v0 < kThreads * kVec * per) {
        const uint32_t ninf = Round<T>::kNegInfWord;
#pragma unroll
        for (int i = 0; i < kVec; ++i)   // not copied: whatever the ring held
            if ((i * kThreads + (int)threadIdx.x) * per >= V - v0) q[i] = make_uint4(ninf, ninf, ninf, ninf);
    }
}

// -inf into the values past V (only the round that holds V needs it).
template <typename T>
__device__ __forceinline__ void mask_round(uint4 (&q)[kVec], int v0, int V) {
    constexpr int per = Round<T>::kPer;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int n = V - v0 - (i * kThreads + (int)threadIdx.x) * per;   // valid values of this load
        if (n >= per) continue;
        uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (per == 4) {
                if (k >= n) w[k] = 0xff800000u;
            } else {
                if (2 * k >= n) w[k] = 0xff80ff80u;
                else if (2 * k + 1 >= n) w[k] = (w[k] & 0xffffu) | 0xff800000u;
            }
        }
        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <typename T>
__device__ __forceinline__ float round_max(const uint4 (&q)[kVec]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t a = 0xff80ff80u;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            uint32_t b, c;
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(q[i].x), "r"(q[i].y));
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(q[i].z), "r"(q[i].w));
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(b), "r"(c));
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        }
        return max_nan(bf16_lo(a), bf16_hi(a));
    } else {
        float a = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) a = max_nan(a, Round<T>::get(q[i], k));
        return a;
    }
}

// Sort `n` keys of `from` (n <= kCap, every thread calls, a barrier before) by
// counting; the largest min(n, top) go to `to`, largest first.  The caller
// places a barrier before either list is used again.  Returns that count.
__device__ __forceinline__ int keep_best(const u64* from, u64* to, int n, int top) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const u64 mine = from[i];
        int r = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) r += from[j] > mine;
        if (r < top) to[r] = mine;
    }
    return min(n, top);
}

struct Shared {
    uint64_t full[kStages], empty[kStages];
    int abort;
    u64 lists[2][kCap];   // the one in use, and the other to sort into
    float part[3][kWarps];
    uint32_t floors[kWarps];   // of the first round
    uint32_t prefix;
    int count, over, need, last;
};

template <typename T>
__device__ __forceinline__ float load_value(const T* row, int v) {
    if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)__ldg(row + v) << 16);
    else return __ldg(row + v);
}

// Append the keys above `above` of one round's values of the lanes in `who`, from
// shared memory.  A whole warp calls.
template <typename T>
__device__ __forceinline__ void append(Shared& sh, u64* list, const unsigned char* stage, unsigned who, int v0, int V, u64 above) {
    constexpr int per = Round<T>::kPer, values = kVec * per;
    const int lane = threadIdx.x & 31;
    const float low = key_floor(above);
    while (who) {
        const int thread = (int)(threadIdx.x & ~31u) + __ffs(who) - 1;
        who &= who - 1;
        if (lane < values) {
            const int at = ((lane / per) * kThreads + thread) * per + lane % per;
            float x;
            if constexpr (sizeof(T) == 2) x = __uint_as_float((uint32_t)reinterpret_cast<const T*>(stage)[at] << 16);
            else x = reinterpret_cast<const T*>(stage)[at];
            if (at < V - v0 && x >= low) {
                const u64 key = make_key(x, v0 + at);
                if (key > above) {
                    const int slot = atomicAdd(&sh.count, 1);
                    if (slot < kCap) list[slot] = key;
                }
            }
        }
    }
}

// The best `top` of values [v0, v1) by radix selection, into `to`, sorted; `list` is
// used on the way.  Every thread calls; a barrier before and after is the caller's.
template <typename T>
__device__ __noinline__ int select_slow(Shared& sh, u64* list, u64* to, const T* row, int v0, int v1, int top) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = v1 - v0;
    int* const hist = reinterpret_cast<int*>(to);   // 256 counts, until the sort
    if (tid == 0) sh.count = 0;
    if (n <= top) {
        for (int i = tid; i < n; i += kThreads) list[i] = make_key(load_value(row, v0 + i), v0 + i);
        sync_streams();
        return keep_best(list, to, n, top);
    }
    uint32_t prefix = 0;
    int need = top;
    for (int shift = 24; shift >= (sizeof(T) == 2 ? 16 : 0); shift -= 8) {
        for (int k = tid; k < 256; k += kThreads) hist[k] = 0;
        sync_streams();
        for (uint32_t i = tid; i < (uint32_t)n; i += kThreads) {
            const uint32_t k = ordered(load_value(row, v0 + i));
            if (shift == 24 || ((k ^ prefix) >> (shift + 8)) == 0) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        sync_streams();
        if (tid == 0) {
            int left = need, bin = 255;
            while (bin > 0 && hist[bin] < left) left -= hist[bin--];
            sh.prefix = prefix | ((uint32_t)bin << shift);
            sh.need = left;
        }
        sync_streams();
        prefix = sh.prefix;
        need = sh.need;
        sync_streams();
    }
    // of the values with this prefix (bf16: equal ones) the first `need` tokens
    constexpr uint32_t kBits = sizeof(T) == 2 ? 0xffff0000u : 0xffffffffu;
    int before = 0;
    for (uint32_t w0 = 0; w0 < (uint32_t)n; w0 += kThreads) {
        const uint32_t i = w0 + tid;
        const int v = v0 + (int)i;
        const float x = i < (uint32_t)n ? load_value(row, v) : 0.0f;
        const uint32_t k = ordered(x) & kBits;
        const bool eq = i < (uint32_t)n && k == prefix;
        const unsigned bal = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) hist[warp] = __popc(bal);
        sync_streams();
        int here = before;
        for (int w = 0; w < kWarps; ++w) {
            here += w < warp ? hist[w] : 0;
            before += hist[w];
        }
        if (i < (uint32_t)n && (k > prefix || (eq && here + __popc(bal & ((1u << lane) - 1u)) < need)))
            list[atomicAdd(&sh.count, 1)] = make_key(x, v);   // `top` in all
        sync_streams();
    }
    return keep_best(list, to, sh.count, top);
}

// z and t of a round's values above the running m (m is at least their maximum),
// as packed pairs.
template <typename T>
__device__ __forceinline__ void round_sums(const uint4 (&q)[kVec], float m, u64& z, u64& t) {
    if (m == -INFINITY) return;   // nothing yet
    if (fabsf(m) <= kPlain) {
        // values under -2 kPlain are 2^(-20000) = 0 all the same: held there, -inf adds 0 to both sums
        const u64 c2 = f32x2_splat(kLog2e), cm = f32x2_splat(-__fmul_rn(m, kLog2e));
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int k = 0; k < 4; k += sizeof(T) == 2 ? 1 : 2) {
                float lo, hi;
                if constexpr (sizeof(T) == 2) {
                    const uint32_t x = bf16x2_max(w[k], 0xc700c700u);
                    lo = bf16_lo(x);
                    hi = bf16_hi(x);
                } else {
                    lo = fmaxf(__uint_as_float(w[k]), -2 * kPlain);
                    hi = fmaxf(__uint_as_float(w[k + 1]), -2 * kPlain);
                }
                const u64 y = f32x2_fma(f32x2_pack(lo, hi), c2, cm);
                const u64 p = f32x2_pack(ex2_approx(f32x2_lo(y)), ex2_approx(f32x2_hi(y)));
                z = f32x2_add(z, p);
                t = f32x2_fma(p, y, t);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int k = 0; k < Round<T>::kPer; k += 2) {
            const float ya = fmaxf((Round<T>::get(q[i], k) - m) * kLog2e, -1e4f);
            const float yb = fmaxf((Round<T>::get(q[i], k + 1) - m) * kLog2e, -1e4f);
            const u64 p = f32x2_pack(ex2_approx(ya), ex2_approx(yb));
            z = f32x2_add(z, p);
            t = f32x2_fma(p, f32x2_pack(ya, yb), t);
        }
}

// Results of entry i from its row's sums and its sorted keys.
template <typename T>
__device__ __forceinline__ void write_entry(const LogprobParams& P, int i, const T* row, const Sums& s,
                                            const u64* list, int kept) {
    const float nan = __int_as_float(0x7fc00000);
    const bool ok = row && isfinite(s.m);   // z >= 1 then
    const float lz = ok ? log2f(s.z) : nan;
    if (threadIdx.x == 0) {
        if (P.entropy) P.entropy[i] = ok ? (lz - s.t / s.z) * kLn2 : nan;
        if (P.logprob) {
            const int t = P.tokens[i];
            P.logprob[i] = ok && t >= 0 && t < P.V ? log_prob(load_value(row, t), s.m, lz) : nan;
        }
    }
    for (int k = threadIdx.x; k < P.top; k += kThreads) {
        const bool have = ok && k < kept;
        P.top_ids[(long long)i * P.top + k] = have ? key_token(list[k]) : -1;
        P.top_logprobs[(long long)i * P.top + k] = have ? log_prob(key_value(list[k]), s.m, lz) : nan;
    }
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads + 32, kPerSm) logprob_kernel(const __grid_constant__ LogprobParams P) {
    extern __shared__ __align__(128) unsigned char ring[];
    Shared& sh = *reinterpret_cast<Shared*>(ring + kStages * kRoundBytes);
    constexpr int per = Round<T>::kPer;
    constexpr int kRound = kThreads * kVec * per;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        sh.abort = 0;
        sh.count = sh.over = 0;
        for (int k = 0; k < kStages; ++k) {
            mbar_init(smem_addr(&sh.full[k]), 1);
            mbar_init(smem_addr(&sh.empty[k]), kWarps);
        }
        mbar_fence_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_release();
    const long long g0 = P.share(blockIdx.x), g1 = P.share(blockIdx.x + 1);
    if (warp == kWarps) {
        // ---------------------------------------------------------- copies
        if (lane == 0) {
            const uint64_t once = l2_policy_evict_first();
            int i = (int)(g0 / P.rounds), rd = (int)(g0 - (long long)i * P.rounds);
            long long r = P.row_of(i);
            for (long long g = g0; g < g1; ++g) {
                const uint32_t n = (uint32_t)(g - g0), k = n % kStages;
                if (!mbar_wait_bounded(smem_addr(&sh.empty[k]), (n / kStages & 1) ^ 1, kWaitNs) ||
                    *(volatile int*)&sh.abort) {
                    set_error(P.err, DLLM_DEVERR_TIMEOUT);
                    *(volatile int*)&sh.abort = 1;
                    break;
                }
                const int v0 = rd * kRound;
                const uint32_t bytes = r < 0 ? 0u : min(kRoundBytes / 16, (uint32_t)((P.V - v0 - 1) / per + 1)) * 16u;
                mbar_arrive_expect_tx(smem_addr(&sh.full[k]), bytes);
                if (bytes)
                    bulk_g2s(smem_addr(ring + k * kRoundBytes), static_cast<const T*>(P.logits) + r * P.ldv + v0, bytes,
                             smem_addr(&sh.full[k]), once);
                if (++rd == P.rounds && g + 1 < g1) {
                    rd = 0;
                    r = P.row_of(++i);
                }
            }
        }
        return;
    }
    // -------------------------------------------------------------- streams
    int i = (int)(g0 / P.rounds);
    for (long long g = g0; g < g1; ++i) {
        // entry i from round rd0 of its row to `rounds`, as far as the share goes
        const long long begin = (long long)i * P.rounds;
        const int rd0 = (int)(g - begin), rd1 = (int)min((long long)P.rounds, g1 - begin);
        const long long r = P.row_of(i);
        const T* row = r >= 0 ? static_cast<const T*>(P.logits) + r * P.ldv : nullptr;
        float m = -INFINITY;
        u64 z = 0, t = 0;
        u64 above = 0;        // keys at or under it are not among the best
        float low = INFINITY; // what a round's maximum must pass to be noted
        int kept = 0, stage = 1, in_use = 0;
        for (int rd = rd0; rd < rd1; ++rd, ++g) {
            const uint32_t n = (uint32_t)(g - g0), k = n % kStages;
            // once a wait has given up the rest runs through without waiting, every barrier met
            if (*(volatile int*)&sh.abort == 0 &&
                !mbar_wait_bounded(smem_addr(&sh.full[k]), n / kStages & 1, kWaitNs)) {
                set_error(P.err, DLLM_DEVERR_TIMEOUT);
                *(volatile int*)&sh.abort = 1;
            }
            const int v0 = rd * kRound;
            uint4 q[kVec];
            const unsigned char* const in = ring + k * kRoundBytes;
            load_round<T>(q, in, v0, P.V);
            if (!row) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.empty[k]));
                continue;
            }
            if (P.V - v0 < kRound) mask_round<T>(q, v0, P.V);
            const float bm = round_max<T>(q);
            uint32_t fl = 0;
            if constexpr (kTop) {
                if (rd == rd0) {
                    // the first floor, by bits of the order-preserving key from the top (16 of them)
                    const int full = min((P.V - v0) / (32 * per), kWarps);   // warps whose lanes all have values
                    const uint32_t key = ordered(bm);
                    if (warp < full) {
                        const int want = (P.top + full - 1) / full;
#pragma unroll 1
                        for (uint32_t bit = 0x80000000u; bit >= 0x10000u; bit >>= 1) {
                            const unsigned at = __ballot_sync(0xffffffffu, key >= (fl | bit));
                            if (__popc(at) >= want) fl |= bit;
                        }
                    } else if (full > 0) {
                        fl = 0xffffffffu;
                    }
                    if (lane == 0) sh.floors[warp] = fl;
                } else {
                    const unsigned who = __ballot_sync(0xffffffffu, bm > low || above == 0);
                    if (who) append<T>(sh, sh.lists[in_use], in, who, v0, P.V, above);
                }
            }
            if (!kTop || rd != rd0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.empty[k]));
            }
            if (!(bm <= m)) {
                const float mn = max_nan(m, bm);
                const float d = fmaxf(diff2(m, mn), -1e4f), f = ex2_approx(d);
                const u64 f2 = f32x2_splat(f);
                t = f32x2_mul(f2, f32x2_fma(z, f32x2_splat(d), t));
                z = f32x2_mul(z, f2);
                m = mn;
            }
            round_sums<T>(q, m, z, t);
            if constexpr (kTop) {
                if (rd == rd0) {
                    sync_streams();
                    fl = sh.floors[0];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) fl = min(fl, sh.floors[w]);
                    above = fl ? ((u64)fl << 32) - 1 : 0;   // every key of a value at the floor passes
                    low = key_floor(above + 1);
                    append<T>(sh, sh.lists[0], in, __ballot_sync(0xffffffffu, bm >= low), v0, P.V, above);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.empty[k]));
                }
                if (rd - rd0 + 1 == stage || rd + 1 == rd1) {
                    stage *= 4;
                    sync_streams();
                    const int n = sh.count;
                    if (n <= kCap) {
                        kept = keep_best(sh.lists[in_use], sh.lists[in_use ^ 1], n, P.top);
                        in_use ^= 1;
                    }
                    sync_streams();
                    // a list that ran over starts again; the part is selected anew at its end
                    if (n > kCap) kept = 0;
                    if (tid == 0) {
                        if (n > kCap) sh.over = 1;
                        sh.count = kept;
                    }
                    if (kept == P.top) {
                        above = max(above, sh.lists[in_use][kept - 1]);
                        low = key_value(above);
                    }
                    if (rd + 1 < rd1) sync_streams();   // the count is set before later rounds append
                }
            }
        }
        if (kTop && row) {
            sync_streams();
            if (sh.over) {
                kept = select_slow<T>(sh, sh.lists[in_use], sh.lists[in_use ^ 1], row, rd0 * kRound, rd1 < P.rounds ? rd1 * kRound : P.V, P.top);
                in_use ^= 1;
                sync_streams();
            }
        }
        // the CTA's sums: the maximum first, then every thread moves its sums to it once
        Sums s;
        s.m = m;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) s.m = max_nan(s.m, __shfl_xor_sync(0xffffffffu, s.m, off));
        if (lane == 0) sh.part[0][warp] = s.m;
        sync_streams();
        if (kTop && tid == 0) sh.count = sh.over = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s.m = max_nan(s.m, sh.part[0][w]);
        {
            const float d = fmaxf(diff2(m, s.m), -1e4f), f = ex2_approx(d);   // m -inf: z is 0
            const float zz = f32x2_lo(z) + f32x2_hi(z);
            s.z = f * zz;
            s.t = f * (f32x2_lo(t) + f32x2_hi(t) + zz * d);
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            s.z += __shfl_xor_sync(0xffffffffu, s.z, off);
            s.t += __shfl_xor_sync(0xffffffffu, s.t, off);
        }
        if (lane == 0) {
            sh.part[1][warp] = s.z;
            sh.part[2][warp] = s.t;
        }
        sync_streams();
        s.z = s.t = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s.z += sh.part[1][w];
            s.t += sh.part[2][w];
        }
        if (rd0 == 0 && rd1 == P.rounds) {
            write_entry<T>(P, i, row, s, sh.lists[in_use], kept);
        } else if (!row) {
            if (rd0 == 0) write_entry<T>(P, i, nullptr, s, nullptr, 0);   // all parts agree: none counts itself
        } else {
            // the parts of an entry: the last of CTA c0's share, then the first of c0 + 1 .. c1
            const int c0 = P.owner(begin), c1 = P.owner(begin + P.rounds - 1);
            const int mine = blockIdx.x == c0 && begin > g0 ? 1 : 0;
            const long long slot = (long long)blockIdx.x * 2 + mine;
            if (tid == 0) __stcg(P.partial + slot, make_float4(s.m, s.z, s.t, 0.0f));
            if constexpr (kTop) {
                for (int k = tid; k < P.top; k += kThreads) __stcg(P.keys + slot * P.top + k, k < kept ? sh.lists[in_use][k] : 0ull);
            }
            __threadfence();
            sync_streams();
            if (tid == 0) sh.last = atom_add_acqrel_gpu(P.counters + c0, 1) == c1 - c0;
            sync_streams();
            if (sh.last) {
                __threadfence();
                if (tid == 0) P.counters[c0] = 0;
                auto slot_of = [&](int c) { return (long long)c * 2 + (c == c0 && begin > P.share(c0) ? 1 : 0); };
                s = Sums{-INFINITY, 0.0f, 0.0f};
                if (tid == 0) sh.count = 0;
                sync_streams();
                for (int c = c0; c <= c1; ++c) {
                    const float4 p = __ldcg(P.partial + slot_of(c));
                    s = join(s, Sums{p.x, p.y, p.z});
                }
                int n = 0;
                if constexpr (kTop) {
                    // batches that fit the list beside the best so far
                    const int batch = (kCap - P.top) / P.top;
                    for (int c = c0; c <= c1; c += batch) {
                        u64* const list = sh.lists[in_use];
                        const int here = min(batch, c1 - c + 1);
                        for (int k = tid; k < here * P.top; k += kThreads) {
                            const u64 key = __ldcg(P.keys + slot_of(c + k / P.top) * P.top + k % P.top);
                            if (key) list[n + atomicAdd(&sh.count, 1)] = key;
                        }
                        sync_streams();
                        const int all = n + sh.count;
                        n = keep_best(list, sh.lists[in_use ^ 1], all, P.top);
                        in_use ^= 1;
                        sync_streams();
                        if (tid == 0) sh.count = 0;
                        sync_streams();
                    }
                }
                write_entry<T>(P, i, row, s, sh.lists[in_use], n);
            }
        }
        sync_streams();   // the list and the parts are free
    }
    // after a wait that gave up: copies still in flight land in this CTA's memory, not in its successor's
    if (*(volatile int*)&sh.abort) __nanosleep(1000000);
}

inline int round_values(int dtype) { return kThreads * kVec * (dtype == DLLM_DTYPE_F32 ? 4 : 8); }

constexpr size_t kSmem = kStages * kRoundBytes + sizeof(Shared);
static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "the CTAs share an SM's shared memory");

template <typename T, bool kTop>
int launch(const LogprobParams& P, cudaStream_t s) {
    auto kernel = logprob_kernel<T, kTop>;
    static SmemOnce done;
    DLLM_CUDA_TRY(allow_smem(kernel, kSmem, done));
    DLLM_CUDA_TRY(launch_dependent(kernel, dim3(P.ctas), dim3(kThreads + 32), kSmem, s, P));
    return DLLM_OK;
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_logprobs_workspace_size(int32_t N, int32_t V, int32_t top) {
    if (N < 0 || V < 1 || top < 0 || top > DLLM_MAX_TOP) return 0;
    return size_t(kJoinCounters) * 4 + size_t(kMaxCtas) * 2 * (sizeof(float4) + size_t(top) * 8);
}

extern "C" int dllm_logprobs(const dllm_logprobs_args* a, void* stream) {
    if (!a || a->N < 0 || a->V < 1 || a->top < 0 || a->top > DLLM_MAX_TOP || a->logits_rows < 0) return DLLM_ERR_INVAL;
    if (a->dtype != DLLM_DTYPE_BF16 && a->dtype != DLLM_DTYPE_F32) return DLLM_ERR_INVAL;
    if (a->ldv < a->V) return DLLM_ERR_INVAL;
    if (a->N > 0 && a->logits_rows > 0 && !a->logits) return DLLM_ERR_INVAL;
    if ((a->tokens == nullptr) != (a->logprob == nullptr)) return DLLM_ERR_INVAL;
    if (a->top > 0 && a->N > 0 && (!a->top_ids || !a->top_logprobs)) return DLLM_ERR_INVAL;
    const int vec = a->dtype == DLLM_DTYPE_F32 ? 4 : 8;
    if ((reinterpret_cast<uintptr_t>(a->logits) & 15) || a->ldv % vec) return DLLM_ERR_ALIGN;
    if (a->N == 0) return DLLM_OK;
    const size_t need = dllm_logprobs_workspace_size(a->N, a->V, a->top);
    if (!a->workspace || a->workspace_bytes < need || (reinterpret_cast<uintptr_t>(a->workspace) & 255))
        return DLLM_ERR_WORKSPACE;
    const int sms = sm_count();
    if (sms <= 0) return DLLM_ERR_CUDA;
    LogprobParams P;
    P.N = a->N;
    P.V = a->V;
    P.top = a->top;
    P.rounds = (a->V - 1) / round_values(a->dtype) + 1;
    P.total = (long long)a->N * P.rounds;
    P.ctas = (int)std::min<long long>(P.total, std::min(sms * kPerSm, kMaxCtas));
    P.ldv = a->ldv;
    P.logits_rows = a->logits_rows;
    P.logits = a->logits;
    P.rows = a->rows;
    P.tokens = a->tokens;
    P.logprob = a->logprob;
    P.entropy = a->entropy;
    P.top_ids = a->top_ids;
    P.top_logprobs = a->top_logprobs;
    unsigned char* ws = static_cast<unsigned char*>(a->workspace);
    P.counters = reinterpret_cast<int*>(ws);
    ws += size_t(kJoinCounters) * 4;
    P.partial = reinterpret_cast<float4*>(ws);
    ws += size_t(kMaxCtas) * 2 * sizeof(float4);
    P.keys = reinterpret_cast<u64*>(ws);
    P.err = error_word_ptr();
    if (!P.err) return DLLM_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    if (a->dtype == DLLM_DTYPE_F32) return a->top ? launch<float, true>(P, s) : launch<float, false>(P, s);
    return a->top ? launch<uint16_t, true>(P, s) : launch<uint16_t, false>(P, s);
}
