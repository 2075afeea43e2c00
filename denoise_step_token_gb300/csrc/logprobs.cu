// dllm_logprobs: log probabilities of given tokens, entropy and the best
// alternatives of logits rows, in one pass over each row.
//
// Mathematics.  With m = max x, z = sum exp(x - m) and t = sum exp(x - m)(x - m):
//   log p_v = x_v - m - ln z,   entropy = ln z - t / z.
// m, z and t are kept running: moving from m to m' >= m scales z by
// f = exp(m - m') and takes t to f (t + z (m - m')).
//
// What bounds it: reading the rows (one FMA-class operation or so per value
// and 1 exp, well under the issue rate at 2 bytes a value), or, for a row or
// two, the launch and the joins.
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
// larger keys come first.  Each piece keeps a candidate list in shared memory
// and a threshold below which nothing can be among its best `top`: the first
// round takes the top-th largest of the threads' own maxima (at least `top`
// values reach it, and only `top` threads can hold such values, so the list
// cannot overflow); later rounds append what exceeds the threshold and sort
// the list down to `top` by counting when it fills.

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
constexpr int kCap = 1024 + 64;      // candidates: at most 32 values of each of DLLM_MAX_TOP threads, and the kept
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

// (a, then b): sums over both ranges.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
    Sums r;
    r.m = max_nan(a.m, b.m);
    if (r.m == -INFINITY) return Sums{-INFINITY, 0.0f, 0.0f};
    // a side without a finite value has z = 0 and drops out
    const float da = fmaxf(a.m - r.m, -1e4f), db = fmaxf(b.m - r.m, -1e4f);
    const float fa = exp2f(da * kLog2e), fb = exp2f(db * kLog2e);
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
    constexpr int kEach = (kCap + kThreads - 1) / kThreads;
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
    u64 maxes[kThreads];
    Sums part[kWarps];
    u64 bound;
    int count, last;
};

// Append this thread's values of the round that have keys >= bound.
template <typename T>
__device__ __forceinline__ void append(Shared& sh, const uint4 (&q)[kVec], int v0, int V, u64 bound) {
    constexpr int per = Round<T>::kPer;
    const float low = key_floor(bound);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int k = 0; k < per; ++k) {
            const float x = Round<T>::get(q[i], k);
            if (x >= low) {
                const int v = v0 + (i * kThreads + (int)threadIdx.x) * per + k;
                const u64 key = make_key(x, v);
                if (v < V && key >= bound) {
                    const int at = atomicAdd(&sh.count, 1);
                    if (at < kCap) sh.list[at] = key;
                }
            }
        }
}

// The top-th largest of the threads' largest keys of the round (0 when fewer
// threads have one): at least `top` keys of the round reach it.
template <typename T>
__device__ __forceinline__ u64 round_bound(Shared& sh, const uint4 (&q)[kVec], int v0, int V, int top) {
    constexpr int per = Round<T>::kPer;
    u64 best = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int k = 0; k < per; ++k) {
            const int v = v0 + (i * kThreads + (int)threadIdx.x) * per + k;
            const u64 key = make_key(Round<T>::get(q[i], k), v);
            if (v < V && key > best) best = key;
        }
    sh.maxes[threadIdx.x] = best;
    if (threadIdx.x == 0) sh.bound = 0;
    __syncthreads();
    int r = 0;
    for (int j = 0; j < kThreads; ++j) r += sh.maxes[j] > best;
    if (best && r == top - 1) sh.bound = best;   // keys differ: one thread at most
    __syncthreads();
    return sh.bound;
}

// Results of entry i from its row's sums and its sorted keys.
template <typename T>
__device__ __forceinline__ void write_entry(const LogprobParams& P, int i, const T* row, const Sums& s,
                                            const u64* list, int kept) {
    const float nan = __int_as_float(0x7fc00000);
    const bool ok = row && isfinite(s.m);   // z >= 1 then
    const float lnz = ok ? logf(s.z) : nan;
    if (threadIdx.x == 0) {
        if (P.entropy) P.entropy[i] = ok ? lnz - s.t / s.z : nan;
        if (P.logprob) {
            const int t = P.tokens[i];
            float lp = nan;
            if (ok && t >= 0 && t < P.V) {
                float x;
                if constexpr (sizeof(T) == 2) x = __uint_as_float((uint32_t)row[t] << 16);
                else x = row[t];
                lp = (x - s.m) - lnz;
            }
            P.logprob[i] = lp;
        }
    }
    for (int k = threadIdx.x; k < P.top; k += kThreads) {
        const bool have = ok && k < kept;
        P.top_ids[(long long)i * P.top + k] = have ? key_token(list[k]) : -1;
        P.top_logprobs[(long long)i * P.top + k] = have ? (key_value(list[k]) - s.m) - lnz : nan;
    }
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 3) logprob_kernel(const __grid_constant__ LogprobParams P) {
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
    float m = -INFINITY, z = 0.0f, t = 0.0f;
    u64 bound = 0;
    int kept = 0;
    if (tid == 0) sh.count = 0;
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
            const float d = fmaxf(m - mn, -1e4f), f = ex2_approx(d * kLog2e);
            t = f * (t + z * d);
            z *= f;
            m = mn;
        }
        // x - m is held above -1e4 (its exp is 0 there): -inf contributes 0 to both sums
#pragma unroll
        for (int k = 0; k < kVec; ++k)
#pragma unroll
            for (int e = 0; e < per; ++e) {
                const float d = fmaxf(Round<T>::get(q[k], e) - m, -1e4f);
                const float p = ex2_approx(d * kLog2e);
                z += p;
                t = fmaf(p, d, t);
            }
        if constexpr (kTop) {
            if (rd == first) {
                bound = round_bound<T>(sh, q, v0, P.V, P.top);
                append<T>(sh, q, v0, P.V, bound);
                __syncthreads();
            } else {
                const int before = sh.count;   // the same in every thread: the barrier below orders it
                __syncthreads();
                if (bm >= key_floor(bound)) append<T>(sh, q, v0, P.V, bound + 1);
                __syncthreads();
                if (sh.count > kCap) {
                    // more than the list holds: drop this round's, raise the threshold, take the round again
                    const int n = keep_best(sh.list, before, P.top);
                    if (n == P.top) bound = max(bound, sh.list[n - 1]);
                    if (tid == 0) sh.count = n;
                    const u64 rb = round_bound<T>(sh, q, v0, P.V, P.top);
                    append<T>(sh, q, v0, P.V, max(rb, bound + 1));
                    __syncthreads();
                }
            }
            const int n = sh.count;
            if (n > 128 || rd + 1 == end) {
                kept = keep_best(sh.list, n, P.top);
                if (kept == P.top) bound = max(bound, sh.list[kept - 1]);
                if (tid == 0) sh.count = kept;
                __syncthreads();
            }
        }
    }
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
