// dllm_logprobs: log probabilities of given tokens, entropy and the best
// alternatives of logits rows, in one pass over each row.
//
// Mathematics, in base 2 (c = log2 e).  With m = max x, y_v = c x_v - c m,
// z = sum 2^y and t = sum 2^y y:
//   log p_v = ln 2 (y_v - log2 z),   entropy = ln 2 (log2 z - t / z).
// m, z and t are kept running: moving from m to m' >= m with d = c m - c m'
// scales z by f = 2^d and takes t to f (t + z d).
//
// What bounds it: reading the rows (4 instructions a value at 2 bytes a value,
// about half of what an SM can issue while its share of memory arrives), or,
// for a row or two, the launch and the joins.
//
// Split.  A row is cut into `pieces` runs of whole rounds (a round: 256
// threads x 64 bytes); one CTA reduces one piece with 16-byte loads straight
// to registers, the next round's in flight, several CTAs per SM.  With one
// piece per row it writes the results itself; otherwise it publishes its
// triple and its best `top` keys, and the piece that arrives last joins them
// in piece order.
//
// Best alternatives.  A value and its token make one 64-bit key (the value's
// order-preserving bits above the inverted token), so all keys differ and
// larger keys come first.  The streaming threads only compare their round's
// maximum with a floor and note (round, thread) in a list when it passes.  After
// rounds 1, 2, 4, 8, ... the noted values are read again (from L2), those above
// the floor sorted among the best so far by counting, and the floor rises to
// the top-th of them; each stage notes about `top` threads.  The first floor: in
// each full warp the q-th largest of its lanes' maxima, q warps >= top, and the
// least of those over the warps; at least `top` values of the round reach it.
// Rows that overfill the lists (sorted ones, many equal values) take a radix
// selection over the piece instead.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"

namespace dllm {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVec = 4;              // 16-byte loads per thread and round
constexpr int kMaxPieces = 32;
constexpr int kMaxSlots = 4096;      // pieces of cut rows in all
constexpr int kCap = 1024;           // candidate keys of a stage, the best so far among them
constexpr int kHits = 512;           // noted threads of a stage
constexpr float kPlain = 16384.0f;   // maxima up to this size take the packed loop
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct LogprobParams {
    int N, V, top, pieces, rounds;   // rounds per row
    long long ldv, logits_rows;
    const void* logits;
    const int* rows;
    const int* tokens;
    float* logprob;
    float* entropy;
    int* top_ids;
    float* top_logprobs;
    int* counters;    // [kJoinCounters], zero between calls
    float4* partial;  // [N][pieces] (m, z, t, -)
    u64* keys;        // [N][pieces][top]
};

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

// c a - c b as the sums hold it (c m is rounded once, the same everywhere).
__device__ __forceinline__ float diff2(float a, float b) {
    return fabsf(b) <= kPlain && fabsf(a) <= kPlain ? __fsub_rn(__fmul_rn(a, kLog2e), __fmul_rn(b, kLog2e))
                                                    : (a - b) * kLog2e;
}
// ln p of one value, lz = log2 z: by the y the sums were formed with where c x
// is sure to be finite.
__device__ __forceinline__ float log_prob(float x, float m, float lz) {
    if (fabsf(m) <= kPlain && fabsf(x) <= kPlain) return (fmaf(x, kLog2e, -__fmul_rn(m, kLog2e)) - lz) * kLn2;
    return (x - m) - lz * kLn2;
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

// Values v0 .. v0 + 4 * 256 * kPer of the row, this thread's share; past V: -inf.
template <typename T>
__device__ __forceinline__ void load_round(uint4 (&q)[kVec], const T* row, int v0, int V) {
    constexpr int per = Round<T>::kPer;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = v0 + (i * kThreads + (int)threadIdx.x) * per;
        const uint32_t ninf = Round<T>::kNegInfWord;
        q[i] = make_uint4(ninf, ninf, ninf, ninf);
        if (v < V) q[i] = __ldcs(reinterpret_cast<const uint4*>(row + v));
    }
}

// -inf into the values past V (only the round that holds V needs it).
template <typename T>
__device__ __forceinline__ void mask_round(uint4 (&q)[kVec], int v0, int V) {
    constexpr int per = Round<T>::kPer;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int n = V - (v0 + (i * kThreads + (int)threadIdx.x) * per);   // valid values of this load
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

// Sort `n` keys of `list` (n <= kCap, every thread calls) by counting; the
// largest min(n, top) end up first, largest first.  Returns that count.
__device__ __forceinline__ int keep_best(u64* list, int n, int top) {
    constexpr int kEach = kCap / kThreads;
    u64 mine[kEach];
    int rank[kEach];
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
        const int i = c * kThreads + (int)threadIdx.x;
        rank[c] = kCap;
        if (i < n) {
            mine[c] = list[i];
            int r = 0;
            for (int j = 0; j < n; ++j) r += list[j] > mine[c];
            rank[c] = r;
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kEach; ++c)
        if (rank[c] < top) list[rank[c]] = mine[c];
    __syncthreads();
    return min(n, top);
}

struct Shared {
    u64 list[kCap];
    int hits[kHits];
    int hist[256];
    Sums part[kWarps];
    uint32_t floor;   // of the first round
    uint32_t prefix;
    int count, n_hits, over, need, last;
};

template <typename T>
__device__ __forceinline__ float load_value(const T* row, int v) {
    if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)__ldg(row + v) << 16);
    else return __ldg(row + v);
}

// Read the noted threads' values again and append the keys above `above`; then
// keep the best.  Every thread calls; returns how many are kept, sorted.
template <typename T>
__device__ __forceinline__ int take_hits(Shared& sh, const T* row, int V, int top, int kept, u64 above) {
    constexpr int per = Round<T>::kPer, values = kVec * per;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hits = min(sh.n_hits, kHits);
    if (threadIdx.x == 0) sh.count = kept;
    __syncthreads();
    const float low = key_floor(above);
    constexpr int kAtOnce = 4;
    for (int h0 = warp * kAtOnce; h0 < hits; h0 += kWarps * kAtOnce) {
        float x[kAtOnce];
        int v[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int h = h0 + u < hits ? sh.hits[h0 + u] : -1;
            v[u] = (h / kThreads) * (kThreads * values) + ((lane / per) * kThreads + h % kThreads) * per + lane % per;
            x[u] = -INFINITY;
            if (h >= 0 && lane < values && v[u] < V) x[u] = load_value(row, v[u]);
            else v[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (v[u] < 0 || !(x[u] >= low)) continue;
            const u64 key = make_key(x[u], v[u]);
            if (key > above) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kCap) sh.list[at] = key;
            }
        }
    }
    __syncthreads();
    const int n = sh.count;
    if (n > kCap || sh.n_hits > kHits) {   // too many to sort: the piece is selected anew at its end
        __syncthreads();
        if (threadIdx.x == 0) {
            sh.over = 1;
            sh.n_hits = 0;
        }
        __syncthreads();
        return kept;
    }
    const int k = keep_best(sh.list, n, top);
    if (threadIdx.x == 0) sh.n_hits = 0;
    __syncthreads();
    return k;
}

// The best `top` of values [v0, v1) by radix selection, into the list, sorted.
template <typename T>
__device__ __noinline__ int select_slow(Shared& sh, const T* row, int v0, int v1, int top) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = v1 - v0;
    if (tid == 0) sh.count = 0;
    if (n <= top) {
        __syncthreads();
        for (int v = v0 + tid; v < v1; v += kThreads) sh.list[v - v0] = make_key(load_value(row, v), v);
        __syncthreads();
        return keep_best(sh.list, n, top);
    }
    uint32_t prefix = 0;
    int need = top;
    for (int shift = 24; shift >= (sizeof(T) == 2 ? 16 : 0); shift -= 8) {
        sh.hist[tid] = 0;
        __syncthreads();
        for (int v = v0 + tid; v < v1; v += kThreads) {
            const uint32_t k = ordered(load_value(row, v));
            if (shift == 24 || ((k ^ prefix) >> (shift + 8)) == 0) atomicAdd(&sh.hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, bin = 255;
            while (bin > 0 && sh.hist[bin] < left) left -= sh.hist[bin--];
            sh.prefix = prefix | ((uint32_t)bin << shift);
            sh.need = left;
        }
        __syncthreads();
        prefix = sh.prefix;
        need = sh.need;
        __syncthreads();
    }
    // of the values with this prefix (bf16: equal ones) the first `need` tokens
    constexpr uint32_t kBits = sizeof(T) == 2 ? 0xffff0000u : 0xffffffffu;
    int before = 0;
    for (int w0 = v0; w0 < v1; w0 += kThreads) {
        const int v = w0 + tid;
        const float x = v < v1 ? load_value(row, v) : 0.0f;
        const uint32_t k = ordered(x) & kBits;
        const bool eq = v < v1 && k == prefix;
        const unsigned bal = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) sh.hist[warp] = __popc(bal);
        __syncthreads();
        int here = before;
        for (int w = 0; w < kWarps; ++w) {
            here += w < warp ? sh.hist[w] : 0;
            before += sh.hist[w];
        }
        if (v < v1 && (k > prefix || (eq && here + __popc(bal & ((1u << lane) - 1u)) < need)))
            sh.list[atomicAdd(&sh.count, 1)] = make_key(x, v);   // `top` in all
        __syncthreads();
    }
    return keep_best(sh.list, sh.count, top);
}

// z and t of a round's values above the running m (m is at least their maximum).
template <typename T>
__device__ __forceinline__ void round_sums(const uint4 (&q)[kVec], float m, u64& z2, u64& t2) {
    if (fabsf(m) <= kPlain) {
        // values under -2 kPlain are 2^(-20000) = 0 all the same: held there, -inf adds 0 to both sums
        const u64 c2 = f32x2_splat(kLog2e), n2 = f32x2_splat(-__fmul_rn(m, kLog2e));
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t x = bf16x2_max(w[k], 0xc700c700u);
                    asm("{\n\t.reg .b32 l, h;\n\t.reg .b64 y, p;\n\t"
                        "prmt.b32 l, %2, 0, 0x1044;\n\t"
                        "and.b32 h, %2, 0xffff0000;\n\t"
                        "mov.b64 y, {l, h};\n\t"
                        "fma.rn.f32x2 y, y, %3, %4;\n\t"
                        "mov.b64 {l, h}, y;\n\t"
                        "ex2.approx.ftz.f32 l, l;\n\t"
                        "ex2.approx.ftz.f32 h, h;\n\t"
                        "mov.b64 p, {l, h};\n\t"
                        "add.rn.f32x2 %0, %0, p;\n\t"
                        "fma.rn.f32x2 %1, p, y, %1;\n\t}"
                        : "+l"(z2), "+l"(t2)
                        : "r"(x), "l"(c2), "l"(n2));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const float l = fmaxf(__uint_as_float(w[k]), -2 * kPlain), h = fmaxf(__uint_as_float(w[k + 1]), -2 * kPlain);
                    asm("{\n\t.reg .b32 l, h;\n\t.reg .b64 y, p;\n\t"
                        "mov.b64 y, {%2, %3};\n\t"
                        "fma.rn.f32x2 y, y, %4, %5;\n\t"
                        "mov.b64 {l, h}, y;\n\t"
                        "ex2.approx.ftz.f32 l, l;\n\t"
                        "ex2.approx.ftz.f32 h, h;\n\t"
                        "mov.b64 p, {l, h};\n\t"
                        "add.rn.f32x2 %0, %0, p;\n\t"
                        "fma.rn.f32x2 %1, p, y, %1;\n\t}"
                        : "+l"(z2), "+l"(t2)
                        : "f"(l), "f"(h), "l"(c2), "l"(n2));
                }
            }
        }
        return;
    }
    if (m == -INFINITY) return;   // nothing yet
    float z = 0.0f, t = 0.0f;
#pragma unroll 1
    for (int i = 0; i < kVec * Round<T>::kPer; ++i) {
        uint4 v = q[0];
#pragma unroll
        for (int k = 1; k < kVec; ++k)
            if (i / Round<T>::kPer == k) v = q[k];
        const int e = i % Round<T>::kPer;
        float x = Round<T>::get(v, 0);
#pragma unroll
        for (int k = 1; k < Round<T>::kPer; ++k)
            if (e == k) x = Round<T>::get(v, k);
        const float y = fmaxf((x - m) * kLog2e, -1e4f), p = ex2_approx(y);
        z += p;
        t = fmaf(p, y, t);
    }
    z2 = f32x2_add(z2, (u64)__float_as_uint(z));
    t2 = f32x2_add(t2, (u64)__float_as_uint(t));
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
__global__ void __launch_bounds__(kThreads, 4) logprob_kernel(const __grid_constant__ LogprobParams P) {
    __shared__ Shared sh;
    constexpr int per = Round<T>::kPer;
    constexpr int kRound = kThreads * kVec * per;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i = blockIdx.x / P.pieces, piece = blockIdx.x - i * P.pieces;
    pdl_wait();
    pdl_release();
    const long long r = P.rows ? (long long)P.rows[i] : i;
    const T* row = r >= 0 && r < P.logits_rows ? static_cast<const T*>(P.logits) + r * P.ldv : nullptr;
    if (!row) {   // the whole row agrees: no piece counts itself
        if (piece == 0) write_entry<T>(P, i, nullptr, Sums{}, sh.list, 0);
        return;
    }
    const int first = (int)((long long)P.rounds * piece / P.pieces);
    const int end = (int)((long long)P.rounds * (piece + 1) / P.pieces);
    float m = -INFINITY;
    u64 z2 = 0, t2 = 0;
    u64 above = 0;        // keys at or under it are not among the best
    float low = INFINITY; // what a round's maximum must pass to be noted
    int kept = 0, stage = 1;
    if (kTop) {
        if (tid == 0) {
            sh.n_hits = sh.over = 0;
            sh.floor = 0xffffffffu;
        }
        __syncthreads();
    }
    uint4 q[kVec], nx[kVec];
    load_round<T>(nx, row, first * kRound, P.V);
    for (int rd = first; rd < end; ++rd) {
        const int v0 = rd * kRound;
#pragma unroll
        for (int k = 0; k < kVec; ++k) q[k] = nx[k];
        if (rd + 1 < end) load_round<T>(nx, row, v0 + kRound, P.V);
        if (v0 + kRound > P.V) mask_round<T>(q, v0, P.V);
        const float bm = round_max<T>(q);
        if (!(bm <= m)) {
            const float mn = max_nan(m, bm);
            const float d = fmaxf(diff2(m, mn), -1e4f), f = ex2_approx(d);
            const u64 f2 = f32x2_splat(f);
            t2 = f32x2_mul(f2, f32x2_fma(z2, f32x2_splat(d), t2));
            z2 = f32x2_mul(z2, f2);
            m = mn;
        }
        round_sums<T>(q, m, z2, t2);
        if constexpr (kTop) {
            if (rd == first) {
                // the first floor, by bits of the order-preserving key from the top (16 of them)
                const int full = min(max(P.V - v0, 0) / (32 * per), kWarps);   // warps whose lanes all have values
                const uint32_t key = ordered(bm);
                uint32_t fl = 0;
                if (warp < full) {
                    const int want = (P.top + full - 1) / full;
#pragma unroll 1
                    for (uint32_t bit = 0x80000000u; bit >= 0x10000u; bit >>= 1) {
                        const unsigned at = __ballot_sync(0xffffffffu, key >= (fl | bit));
                        if (__popc(at) >= want) fl |= bit;
                    }
                    if (lane == 0) atomicMin(&sh.floor, fl);
                }
                __syncthreads();
                fl = full > 0 ? sh.floor : 0;
                above = fl ? ((u64)fl << 32) - 1 : 0;   // every key of a value at the floor passes
                low = key_floor(above + 1);
                if (bm >= low) {
                    const int at = atomicAdd(&sh.n_hits, 1);
                    if (at < kHits) sh.hits[at] = rd * kThreads + tid;
                }
            } else if (bm > low || above == 0) {
                const int at = atomicAdd(&sh.n_hits, 1);
                if (at < kHits) sh.hits[at] = rd * kThreads + tid;
            }
            if (rd - first + 1 == stage || rd + 1 == end) {
                stage *= 2;
                __syncthreads();
                if (!sh.over) {
                    kept = take_hits<T>(sh, row, P.V, P.top, kept, above);
                    if (kept == P.top && !sh.over) {
                        above = max(above, sh.list[kept - 1]);
                        low = key_value(above);
                    }
                    __syncthreads();   // the list is read before a later stage appends
                }
            }
        }
    }
    if constexpr (kTop) {
        if (sh.over) kept = select_slow<T>(sh, row, first * kRound, min(end * kRound, P.V), P.top);
    }
    const float z = __uint_as_float((uint32_t)z2) + __uint_as_float((uint32_t)(z2 >> 32));
    const float t = __uint_as_float((uint32_t)t2) + __uint_as_float((uint32_t)(t2 >> 32));
    Sums s{m, z, t};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        Sums o;
        o.m = __shfl_xor_sync(0xffffffffu, s.m, off);
        o.z = __shfl_xor_sync(0xffffffffu, s.z, off);
        o.t = __shfl_xor_sync(0xffffffffu, s.t, off);
        s = (lane & off) ? join(o, s) : join(s, o);
    }
    if (lane == 0) sh.part[warp] = s;
    __syncthreads();
    s = sh.part[0];
    for (int w = 1; w < kWarps; ++w) s = join(s, sh.part[w]);
    if (P.pieces == 1) {
        write_entry<T>(P, i, row, s, sh.list, kept);
        return;
    }
    const long long slot = (long long)i * P.pieces;
    if (tid == 0) P.partial[slot + piece] = make_float4(s.m, s.z, s.t, 0.0f);
    if constexpr (kTop) {
        for (int k = tid; k < P.top; k += kThreads)
            P.keys[(slot + piece) * P.top + k] = k < kept ? sh.list[k] : 0ull;
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) sh.last = atom_add_acqrel_gpu(P.counters + i, 1) == P.pieces - 1;
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
    if (tid == 0) P.counters[i] = 0;
    const float4 p0 = __ldcg(P.partial + slot);
    s = Sums{p0.x, p0.y, p0.z};
    for (int k = 1; k < P.pieces; ++k) {
        const float4 p = __ldcg(P.partial + slot + k);
        s = join(s, Sums{p.x, p.y, p.z});
    }
    int n = 0;
    if constexpr (kTop) {
        if (tid == 0) sh.count = 0;
        __syncthreads();
        for (int k = tid; k < P.pieces * P.top; k += kThreads) {
            const u64 key = __ldcg(P.keys + slot * P.top + k);
            if (key) sh.list[atomicAdd(&sh.count, 1)] = key;   // pieces * top <= kCap
        }
        __syncthreads();
        n = keep_best(sh.list, sh.count, P.top);
    }
    write_entry<T>(P, i, row, s, sh.list, n);
}

inline int round_values(int dtype) { return kThreads * kVec * (dtype == DLLM_DTYPE_F32 ? 4 : 8); }

// Pieces per row.  One CTA per row leaves SMs idle until there are a few rows
// per resident CTA (3 per SM); below that rows are cut, at most to single
// rounds, so that about 4 waves of CTAs are there to balance.
inline int pick_pieces(int N, int V, int top, int dtype, int sms) {
    const int rounds = (V + round_values(dtype) - 1) / round_values(dtype);
    const long long want = ((long long)sms * 12 + N - 1) / std::max(N, 1);
    if (N > kJoinCounters) return 1;
    long long p = std::min<long long>({(long long)rounds, want, (long long)kMaxPieces, (long long)kMaxSlots / N});
    if (top > 0) p = std::min<long long>(p, kCap / top);
    return (int)std::max<long long>(p, 1);
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_logprobs_workspace_size(int32_t N, int32_t V, int32_t top) {
    if (N < 0 || V < 1 || top < 0 || top > DLLM_MAX_TOP) return 0;
    return size_t(kJoinCounters) * 4 + size_t(kMaxSlots) * (sizeof(float4) + size_t(top) * 8);
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
    P.pieces = pick_pieces(a->N, a->V, a->top, a->dtype, sms);
    P.rounds = (a->V + round_values(a->dtype) - 1) / round_values(a->dtype);
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
    ws += size_t(kMaxSlots) * sizeof(float4);
    P.keys = reinterpret_cast<u64*>(ws);
    const long long grid = (long long)a->N * P.pieces;
    if (grid > 0x7fffffffll) return DLLM_ERR_UNSUPPORTED;
    auto kernel = a->dtype == DLLM_DTYPE_F32 ? (a->top ? logprob_kernel<float, true> : logprob_kernel<float, false>)
                                             : (a->top ? logprob_kernel<uint16_t, true> : logprob_kernel<uint16_t, false>);
    DLLM_CUDA_TRY(launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), 0, as_stream(stream), P));
    return DLLM_OK;
}
