// dllm_sample: one token per logits row, drawn with temperature, top-k, min-p and
// top-p by a given number u in [0, 1); dllm_sample_conf: also the token's softmax
// probability, the step's confidence, from the same counts (its weights are a
// second sum over the row's different values).
//
// Mathematics.  In the order of falling values (ties: lowest token first) with
// w = exp((x - m) / T), every filter keeps a prefix, and the draw is the first
// token whose cumulative w passes u times the kept mass.  u lies next to one of
// up to V borders, so an error eps of the cumulative masses draws another token
// about (mean rank of the draw) * eps times: 32-bit sums (1e-7) would err once in
// some hundred rows of a flat distribution.  A bf16 row holds few different
// values, though: a histogram of its values is exact, each value's weight is
// computed once, to 2^-44 in its exponent and 2^-62 in itself, and masses are
// sums of count * weight in 64-bit fixed point, in units that leave room for V
// tokens of the largest weight (2^-45 of it at 126464, 2^-33 at 2^28).  The rest works on the histogram:
// what the filters leave, the mass, the value that the draw falls on, and which
// of the tokens with that value, counted from the lowest, it is.
//
// Split.  A cluster of 1 to 8 CTAs takes a row, each CTA a slice: a copying warp
// keeps the ring of bulk copies full (also with the next rows' pieces), sixteen
// warps count values with shared-memory atomics.  Segments of 32 values are
// summed by all warps of the cluster (counts of the others by distributed shared
// memory), one warp walks the segments' sums, and the CTA whose slice holds the
// token reads its slice again, from its end, to find it.
// What bounds it: the phases of a row follow one another, two CTAs an SM overlap; issue
// slots are 57 % used, much of it the counters' shared-memory atomics.  1851 rows of
// 151936 values: 270 us (2.1 TB/s; on the way there, at 292: without the search 238, without the
// counters' atomics too 123).
// CTAs a row: as many as fill the SMs, none with under 4096 values.  More than
// needed cost: 353 us for clusters of two in that batch, the only one where the
// rule's other side was measured.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"

namespace dllm {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;   // counting threads of a CTA (256: 320 us instead of 292 on the way, 1851 rows of 151936)
constexpr int kWarps = kThreads / 32;
// The ring: fewer, larger copies leave fewer barriers a value (7 stages of 4096 values: 285 us instead of 270).
constexpr int kStages = 3;
constexpr int kChunk = 8192;    // values of a stage
constexpr int kLeast = 4096;    // values of the smallest slice worth a CTA
constexpr int kPerSm = 2;
constexpr int kMaxCluster = 8;
constexpr uint64_t kWaitNs = 2000000000ull;

// Values 2^-28 < |x| < 2^8 have a counter each, per sign; smaller ones share the
// first counter, larger ones the last.
constexpr uint32_t kLow = 0x3180, kHigh = 0x4380;
constexpr int kValues = kHigh - kLow;                  // index of the last counter
constexpr uint32_t kNegative = 0x8000;                 // byte offset of the negative values' counters
constexpr int kHalfBins = (kValues + 32) / 32 * 32;    // bins of a sign, whole segments
constexpr int kSegments = 2 * kHalfBins / 32;
// Rows that this does not hold go by all 65536 keys, a window at a time.
constexpr int kWindow = 4096;
constexpr int kWideSegment = 64;
constexpr int kWideSegments = 65536 / kWideSegment;

// 2^(i / 256) in units of 2^-63, i in [0, 256), from square roots of 2 in whole numbers.
constexpr int kPowers = 256;
struct PowerTable {
    u64 t[kPowers];
};
constexpr u64 root_of(unsigned __int128 v) {   // floor of the square root
    u64 r = 0;
    for (int b = 63; b >= 0; --b) {
        const u64 c = r | (1ull << b);
        if ((unsigned __int128)c * c <= v) r = c;
    }
    return r;
}
constexpr PowerTable make_powers() {
    u64 root[8] = {};                                    // 2^(2^-(k+1))
    unsigned __int128 v = (unsigned __int128)1 << 127;   // 2, in units of 2^-126
    for (int k = 0; k < 8; ++k) {
        root[k] = root_of(v);
        v = (unsigned __int128)root[k] << 63;
    }
    PowerTable p = {};
    for (int i = 0; i < kPowers; ++i) {
        unsigned __int128 x = (unsigned __int128)1 << 63;
        for (int b = 0; b < 8; ++b)
            if (i >> b & 1) x = x * root[7 - b] >> 63;
        p.t[i] = (u64)x;
    }
    return p;
}
__constant__ PowerTable c_powers = make_powers();
static_assert(make_powers().t[128] == 13043817825332782212ull, "sqrt(2) * 2^63");

struct SampleParams {
    int N, V;
    long long ldv, logits_rows;
    const uint16_t* logits;
    const int* rows;
    const float* u;
    const float* temperature;
    const int* top_k;
    const float* top_p;
    const float* min_p;
    int* tokens;
    float* prob;
    float* conf;          // (kConf)
    int* err;
    int cluster, slice;   // values of a CTA's slice
    int shift;            // masses are in units of 2^(shift - 62)
};

// The weights of one row's values, by pairs of 32-bit floats and whole numbers (64-bit floating point runs at 2 operations
// an SM and cycle here).
struct Weights {
    float m;           // the maximum
    float scale;       // 1, or 2^-64 for temperatures where log2(e) / T would lose bits
    float s, s_low;    // log2(e) / T in two parts, over `scale`
    u64 least;         // min-p in units of 2^-62: smaller weights are left out
    int shift;

    __device__ __forceinline__ void set(float top, float T, float min_p) {
        m = top;
        T = fmaxf(T, 1.17549435e-38f);
        scale = T > 1.8446744e19f ? 5.4210109e-20f : 1.0f;
        const float t = T * scale;   // inf stays
        constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f;
        s = kLog2e / t;
        s_low = isinf(t) ? 0.0f : (fmaf(-s, t, kLog2e) + kLog2eLow) / t;
        least = min_p > 0.0f ? __float2ull_ru(fminf(min_p, 1.0f) * 4.611686e18f) : 0;
    }
    // (x - m) s to 32 bits.
    __device__ __forceinline__ float rough(float x) const { return (x * scale - m * scale) * s; }
    // w in units of 2^-62; 0 below that and where min-p leaves the value out.  No branches: callers have several under way.
    __device__ __forceinline__ u64 of(float x, const u64* powers) const {
        // x - m = d + e without error, its product with s = p + rest
        const float xs = x * scale, ms = -m * scale;
        const float d = xs + ms, v = d - xs, e = (xs - (d - v)) + (ms - v);
        const float p = d * s;
        const bool live = p > -62.0f;   // p <= 0
        const float rest = fmaf(e, s, fmaf(d, s_low, fmaf(d, s, -p)));
        // p = j / 256 + h, |h| <= 2^-9
        const float at = fmaf(fmaxf(p, -64.0f), 256.0f, 12582912.0f);
        const int j = __float_as_int(at) - 0x4b400000;
        const float h = fmaf(at - 12582912.0f, -0.00390625f, fmaxf(p, -64.0f));
        // 2^(h + rest) - 1: the leading product h ln 2 in two parts, the other powers behind it
        constexpr float kLn2 = 0.693147182f, kLn2Low = -1.90465421e-9f;
        const float g = h * kLn2;
        float more = fmaf(h, 9.61812911e-3f, 5.55041087e-2f);
        more = fmaf(h, more, 2.40226507e-1f);
        more = fmaf(h * h, more, fmaf(rest, kLn2, fmaf(h, kLn2Low, fmaf(h, kLn2, -g))));
        // in units of 2^-40: g to 31 bits, the rest by its place behind 1.5 * 2^23
        const int part = __float2int_rn(g * 1.09951163e12f) + (__float_as_int(fmaf(more, 1.09951163e12f, 12582912.0f)) - 0x4b400000);
        const u64 t = powers[j & 255];
        // t (1 + part 2^-40), the product with t's upper 32 bits
        const long long add = ((long long)part << 31) + (long long)part * (int)((t >> 32) - 0x80000000u);
        const u64 w = (u64)((long long)(t >> 1) + (add >> 9)) >> (-(j >> 8) & 63);
        return live && w >= least ? w : 0;
    }
    // Mass of `count` tokens of weight w.
    __device__ __forceinline__ u64 mass(uint32_t count, u64 w) const {
        const u64 lo = (u64)count * (uint32_t)w, hi = (u64)count * (uint32_t)(w >> 32);
        return (hi << (32 - shift)) + ((lo + (1ull << (shift - 1))) >> shift);
    }
};

// What a CTA tells the others of its slice.
struct SliceFacts {
    float max;    // NaN if the slice holds one
    int other;    // values that only the wide path tells apart
    int low;      // values at or under -2^8
};

struct Found {
    u64 mass;        // of the tokens up to and with the one found
    uint32_t bits;   // its value; 0 stands for both zeros
    uint32_t r, n;   // which of the value's n tokens, from 0
    u64 w;
};

// What the functions behind the counting need of the row, in shared memory: they run once a row, and parameters behind
// a pointer or on the stack are fetched from L2 each time (sums of a row: 32,000 cycles so).
struct RowFacts {
    Weights W;
    const uint16_t* x;
    int V, cluster;
};

struct Shared {
    uint64_t full[kStages], empty[kStages], meet[2];
    u64 powers[kPowers];
    u64 seg_mass[kSegments];
    uint32_t seg_count[kSegments];
    u64 warp_mass[kWarps];
    uint32_t warp_count[kWarps];
    uint32_t groups[64], counts[3];
    float part[kWarps];
    u64 plain[kMaxCluster * kWarps];   // the first CTA's: sums of weights at temperature 1, a warp of the cluster each
    SliceFacts facts;
    Found found;
    u64 kept;
    RowFacts row;
    int abort, segment, flag;
};
constexpr uint32_t kGap = (kValues + 1) * 4 + 15 & ~15u;   // the struct lies between the counters of both signs
static_assert(kGap + sizeof(Shared) <= kNegative, "fits between the counters");
constexpr uint32_t kRing = (kNegative + (kValues + 1) * 4 + 127) & ~127u;
constexpr size_t kSmem = kRing + kStages * kChunk * 2;
static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
// the wide path's: window counters where the negatives' are, segment sums where the positives' are
static_assert(kWindow * 4 <= (kValues + 1) * 4 && kWideSegments * 12 <= kGap, "the wide path's arrays");

__device__ __forceinline__ void sync_warps() { asm volatile("bar.sync 1, 512;" ::: "memory"); }
// All threads of the cluster, before their roles part.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t at, int cta) {
    uint32_t p;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(at), "r"(cta));
    return p;
}
__device__ __forceinline__ uint32_t cluster_load(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t peer_load(uint32_t at, int cta) { return cluster_load(peer_addr(at, cta)); }
__device__ __forceinline__ void peer_store(uint32_t at, int cta, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(peer_addr(at, cta)), "r"(v) : "memory");
}
__device__ __forceinline__ void peer_store64(uint32_t at, int cta, u64 v) {
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(peer_addr(at, cta)), "l"(v) : "memory");
}

// Meetings of the cluster's counting warps (the copying warps run ahead of them, so the hardware's cluster barrier will
// not do): every CTA arrives at every CTA's barrier.  Two barriers in turn: a CTA that has left one meeting may arrive
// at the next before all arrivals of the last have landed everywhere.
__device__ __forceinline__ bool meet_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 1000000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
struct Meeting {
    uint32_t bars;   // two barriers
    uint32_t n;
    int ctas;
    __device__ __forceinline__ void arrive() const {
        sync_warps();
        if ((int)threadIdx.x < ctas)
            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                             peer_addr(bars + (n & 1) * 8, threadIdx.x))
                         : "memory");
    }
    __device__ __noinline__ void wait(int* abort, int* err) {
        const uint32_t bar = bars + (n & 1) * 8, parity = n >> 1 & 1;
        ++n;
        if (*(volatile int*)abort || meet_try(bar, parity)) return;
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            if (meet_try(bar, parity)) return;
            if ((it & 255u) == 0 && globaltimer_ns() - t0 > kWaitNs) break;
        }
        set_error(err, DLLM_DEVERR_TIMEOUT);
        *(volatile int*)abort = 1;
    }
};

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void count_at(uint32_t addr) {
    asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(addr));
}

__device__ __forceinline__ u64 warp_sum64(u64 v) {   // the sum below 2^64
    const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x7ffffffu);
    const uint32_t mid = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 27) & 0x7ffffffu);
    const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 54));
    return (u64)lo + ((u64)mid << 27) + ((u64)hi << 54);
}

extern __shared__ __align__(128) unsigned char smem[];

__device__ __forceinline__ Shared& shared() { return *reinterpret_cast<Shared*>(smem + kGap); }
__device__ __forceinline__ uint32_t word_at(uint32_t at) { return *reinterpret_cast<const uint32_t*>(smem + at); }

// The bins of a row, in falling order of their values: kSegments * 32 of the counters, or (kWide) all keys.
template <bool kWide>
struct Bins {
    static constexpr int kCount = kWide ? kWideSegments : kSegments;   // of segments
    static constexpr int kSize = kWide ? kWideSegment : 32;            // of one

    static __device__ __forceinline__ uint32_t bits(int o) {
        if (kWide) {
            const uint32_t key = 0xffffu - o;
            return key & 0x8000u ? key ^ 0x8000u : ~key & 0xffffu;
        }
        if (o < kHalfBins) {
            const int c = kHalfBins - 1 - o;
            return c == 0 ? 0 : kLow + c;
        }
        return 0x8000u | (kLow + (o - kHalfBins));
    }
    static __device__ __forceinline__ float value(int o) { return __uint_as_float(bits(o) << 16); }
    static __device__ __forceinline__ uint32_t* seg_count() {
        return kWide ? reinterpret_cast<uint32_t*>(smem + kWideSegments * 8) : shared().seg_count;
    }
    static __device__ __forceinline__ u64* seg_mass() { return kWide ? reinterpret_cast<u64*>(smem) : shared().seg_mass; }
};

// The counts of kN bins, over the cluster.
template <int kN>
__device__ __forceinline__ void counts_of(const int (&o)[kN], uint32_t (&n)[kN], int cluster) {
    uint32_t at[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        const bool neg = o[j] >= kHalfBins;
        const int c = neg ? o[j] - kHalfBins : kHalfBins - 1 - o[j];
        at[j] = (neg ? kNegative : 0u) + min(c, kValues) * 4;
        n[j] = word_at(at[j]);
    }
    if (cluster > 1) {
        const uint32_t base = smem_addr(smem);
        const int self = (int)cluster_rank();
#pragma unroll 1
        for (int q = 1; q < cluster; ++q) {   // its size is a power of two
            const uint32_t from = peer_addr(base, self ^ q);
#pragma unroll
            for (int j = 0; j < kN; ++j) n[j] += cluster_load(from + at[j]);
        }
    }
    // bins without a value of their own took the last counter, which is left out
#pragma unroll
    for (int j = 0; j < kN; ++j) n[j] = (at[j] & ~kNegative) == kValues * 4 ? 0 : n[j];
}

// The segments' sums become sums up to and with each segment (every thread).
template <bool kWide>
__device__ __noinline__ void add_up() {
    Shared& sh = shared();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int n = Bins<kWide>::kCount, per = (n + kThreads - 1) / kThreads;
    uint32_t* const counts = Bins<kWide>::seg_count();
    u64* const masses = Bins<kWide>::seg_mass();
    uint32_t cs[per], c = 0;
    u64 ms[per], m = 0;
#pragma unroll
    for (int k = 0; k < per; ++k) {
        const int s = tid * per + k;
        c += cs[k] = s < n ? counts[s] : 0;
        m += ms[k] = s < n ? masses[s] : 0;
    }
    const uint32_t c1 = c;
    const u64 m1 = m;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t cy = __shfl_up_sync(0xffffffffu, c, off);
        const u64 my = __shfl_up_sync(0xffffffffu, m, off);
        if (lane >= off) {
            c += cy;
            m += my;
        }
    }
    if (lane == 31) {
        sh.warp_count[warp] = c;
        sh.warp_mass[warp] = m;
    }
    sync_warps();
    c -= c1;
    m -= m1;
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w) {
        c += w < warp ? sh.warp_count[w] : 0;
        m += w < warp ? sh.warp_mass[w] : 0;
    }
#pragma unroll
    for (int k = 0; k < per; ++k) {
        const int s = tid * per + k;
        c += cs[k];
        m += ms[k];
        if (s < n) {
            counts[s] = c;
            masses[s] = m;
        }
    }
    sync_warps();
}

// Counts the row's values with keys 0xffff - o for o in [o0, o0 + n) (wide path; every thread).
__device__ __noinline__ void count_keys(int o0, int n) {
    uint32_t* const counts = reinterpret_cast<uint32_t*>(smem + kNegative);
    const uint16_t* const x = shared().row.x;
    const int V = shared().row.V;
    for (int i = threadIdx.x; i < n; i += kThreads) counts[i] = 0;
    sync_warps();
#pragma unroll 1
    for (int e = threadIdx.x * 8; e < V; e += kThreads * 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(x + e);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t b = w[k / 2] >> (k & 1 ? 16 : 0) & 0xffffu;
            if (b == 0x8000u) b = 0;
            const uint32_t o = 0xffffu - (b & 0x8000u ? ~b & 0xffffu : b | 0x8000u);
            if (o - o0 < (uint32_t)n && b != 0xff80u && e + k < V) atomicAdd(&counts[o - o0], 1u);
        }
    }
    sync_warps();
}

// The first token whose count reaches `target` (by_count), or whose cumulative mass does; a target within the totals.
// The first warp calls; in the wide path every thread.  The answer is in shared memory.
template <bool kWide>
__device__ __noinline__ void find(bool by_count, u64 target) {
    using B = Bins<kWide>;
    Shared& sh = shared();
    const int lane = threadIdx.x & 31;
    uint32_t c0 = 0;
    u64 m0 = 0;
    int seg = 0;
    if (threadIdx.x < 32) {
        // the first segment that reaches the target: among every per-th one, then among the per before it
        constexpr int last = B::kCount - 1, per = (B::kCount + 31) / 32;
        auto reaches = [&](int s) { return (by_count ? (u64)B::seg_count()[s] : B::seg_mass()[s]) >= target; };
        unsigned who = __ballot_sync(0xffffffffu, reaches(min(lane * per + per - 1, last)));
        const int run = who ? (__ffs(who) - 1) * per : last;
        who = __ballot_sync(0xffffffffu, reaches(min(run + min(lane, per - 1), last)));
        seg = who ? min(run + __ffs(who) - 1, last) : last;
        if (seg > 0) {
            c0 = B::seg_count()[seg - 1];
            m0 = B::seg_mass()[seg - 1];
        }
        if (kWide && lane == 0) sh.segment = seg;
    }
    if (kWide) {
        sync_warps();
        count_keys(sh.segment * B::kSize, B::kSize);
    }
    if (threadIdx.x < 32) {
        const Weights W = sh.row.W;
#pragma unroll 1
        for (int b0 = 0; b0 < B::kSize; b0 += 32) {
            const int o[1] = {seg * B::kSize + b0 + lane};
            uint32_t count[1];
            if (kWide) count[0] = word_at(kNegative + (b0 + lane) * 4);
            else counts_of(o, count, sh.row.cluster);
            uint32_t n = count[0];
            const u64 w = W.of(B::value(o[0]), sh.powers);
            if (w == 0) n = 0;
            uint32_t ci = n;
            const u64 mine = W.mass(n, w);
            u64 mi = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t cy = __shfl_up_sync(0xffffffffu, ci, off);
                const u64 my = __shfl_up_sync(0xffffffffu, mi, off);
                if (lane >= off) {
                    ci += cy;
                    mi += my;
                }
            }
            const unsigned who = __ballot_sync(0xffffffffu, n && (by_count ? (u64)(c0 + ci) : m0 + mi) >= target);
            if (who) {
                if (lane == __ffs(who) - 1) {
                    // tokens of the bin that are needed, 1 to n
                    uint32_t j;
                    const u64 before = m0 + mi - mine;
                    if (by_count) {
                        j = (uint32_t)(target - (c0 + ci - n));
                    } else {
                        // a quotient in 32 bits, twice made good, then to the token
                        const u64 rem = target > before ? target - before : 1;
                        const float ones = __frcp_rn((float)w * __uint_as_float((uint32_t)(127 - W.shift) << 23));
                        j = (uint32_t)fminf(fmaxf((float)rem * ones, 1.0f), (float)n);
#pragma unroll 1
                        for (int k = 0; k < 2 && n > 1; ++k) {
                            const float off = rintf((float)(long long)(rem - W.mass(j, w)) * ones);
                            j = (uint32_t)min(max((long long)j + (long long)off, 1ll), (long long)n);
                        }
#pragma unroll 1
                        for (int k = 0; k < 4 && j > 1 && W.mass(j - 1, w) >= rem; ++k) --j;
#pragma unroll 1
                        for (int k = 0; k < 4 && j < n && W.mass(j, w) < rem; ++k) ++j;
                    }
                    sh.found = Found{before + W.mass(j, w), B::bits(o[0]), j - 1, n, w};
                }
                break;
            }
            c0 += __shfl_sync(0xffffffffu, ci, 31);
            m0 += __shfl_sync(0xffffffffu, mi, 31);
        }
        __syncwarp();
    }
    if (kWide) sync_warps();
}

// x times v for 0 <= x < 1, rounded up or down; x < 0: 0.
__device__ __forceinline__ u64 part_of(float x, u64 v, bool up) {
    if (!(x > 0.0f)) return 0;
    // x = c 2^-k, c < 2^24
    const uint32_t b = __float_as_uint(x), e = b >> 23;
    const u64 c = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int k = 150 - (int)max(e, 1u);                   // >= 24
    const u64 hi = __umul64hi(c, v), lo = c * v;           // hi < 2^24
    if (k >= 88) return up ? 1 : 0;                        // c v < 2^88
    const u64 q = k >= 64 ? hi >> (k - 64) : hi << (64 - k) | lo >> k;
    const u64 left = k >= 64 ? (hi & ((1ull << (k - 64)) - 1)) | lo : lo & ((1ull << k) - 1);
    return q + (up && left);
}

// Filters and draw, from the segments' sums.  As find() is called.
template <bool kWide>
__device__ __noinline__ void choose(float u, int k, float p) {
    using B = Bins<kWide>;
    Shared& sh = shared();
    u64 kept = B::seg_mass()[B::kCount - 1];
    const uint32_t count = B::seg_count()[B::kCount - 1];
    bool last = false;   // what was found last is the last kept token
    if (k > 0 && (uint32_t)k < count) {
        find<kWide>(true, (uint32_t)k);
        kept = sh.found.mass;
        last = true;
        __syncwarp();
    }
    if (p < 1.0f) {
        find<kWide>(false, max(part_of(p, kept, true), 1ull));
        kept = min(kept, sh.found.mass);
        last = true;
        __syncwarp();
    }
    if (!(u >= 1.0f)) find<kWide>(false, u >= 0.0f ? min(part_of(u, kept, false) + 1, kept) : 1);
    else if (!last) find<kWide>(true, count);   // by count: a last token's mass may round to nothing
    if (threadIdx.x == 0) sh.kept = kept;
}

// The drawn token's w over the kept mass: the quotient of the leading 24 bits, made good by what they leave out.
__device__ __forceinline__ float probability(u64 w, u64 kept, int shift) {
    const float unit = __uint_as_float((uint32_t)(127 - shift) << 23);
    const float a1 = (float)w * unit, a0 = (float)(long long)(w - (u64)((float)w)) * unit;
    const float b1 = (float)kept, b0 = (float)(long long)(kept - (u64)b1);
    const float q = a1 / b1;
    return q + (fmaf(-q, b1, a1) + a0 - q * b0) / b1;
}

// The wide path's segment sums: windows of keys from the maximum's down, as far as weights reach (every thread).
__device__ __noinline__ void sum_wide() {
    using B = Bins<true>;
    Shared& sh = shared();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Weights W = sh.row.W;
    for (int s = threadIdx.x; s < B::kCount; s += kThreads) {
        B::seg_mass()[s] = 0;
        B::seg_count()[s] = 0;
    }
#pragma unroll 1
    for (int o0 = 0; o0 < 65536; o0 += kWindow) {
        // the window's first finite value is its largest, its last one the smallest
        const float last = B::value(o0 + kWindow - 1), first = B::value(o0);
        if (last > W.m) continue;                                           // all above the maximum
        if (!isnan(first) && first < W.m && W.of(first, sh.powers) == 0) break;
        count_keys(o0, kWindow);
#pragma unroll 1
        for (int s = warp; s < kWindow / B::kSize; s += kWarps) {
            uint32_t c = 0;
            u64 m = 0;
#pragma unroll 1
            for (int o = s * B::kSize + lane; o < (s + 1) * B::kSize; o += 32) {
                const uint32_t n = word_at(kNegative + o * 4);
                const u64 w = n ? W.of(B::value(o0 + o), sh.powers) : 0;
                if (w) c += n;
                m += W.mass(n, w);
            }
            c = __reduce_add_sync(0xffffffffu, c);
            m = warp_sum64(m);
            if (lane == 0) {
                B::seg_mass()[o0 / B::kSize + s] = m;
                B::seg_count()[o0 / B::kSize + s] = c;
            }
        }
        sync_warps();
    }
    sync_warps();
}

// The row's mass at temperature 1 without filters, each warp's part into `plain` (the cluster's counting threads).
__device__ __noinline__ void sum_plain(float top, int shift, int rank, int ctas) {
    Shared& sh = shared();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Weights W;
    W.shift = shift;
    W.set(top, 1.0f, 0.0f);
    u64 m = 0;
#pragma unroll 1
    for (int s = rank * kWarps + warp; s < kSegments; s += ctas * kWarps) {
        const int o[1] = {s * 32 + lane};
        uint32_t c[1];
        counts_of(o, c, ctas);
        if (__any_sync(0xffffffffu, c[0])) m += W.mass(c[0], W.of(Bins<false>::value(o[0]), sh.powers));
    }
    m = warp_sum64(m);
    if (lane) return;
    if (ctas > 1) peer_store64(smem_addr(&sh.plain[rank * kWarps + warp]), 0, m);
    else sh.plain[warp] = m;
}
// The same on the wide path (every thread of the first CTA).
__device__ __noinline__ void sum_plain_wide() {
    using B = Bins<true>;
    Shared& sh = shared();
    Weights W = sh.row.W;
    W.set(W.m, 1.0f, 0.0f);
    u64 m = 0;
#pragma unroll 1
    for (int o0 = 0; o0 < 65536; o0 += kWindow) {
        const float last = B::value(o0 + kWindow - 1), first = B::value(o0);
        if (last > W.m) continue;
        if (!isnan(first) && first < W.m && W.of(first, sh.powers) == 0) break;
        count_keys(o0, kWindow);
#pragma unroll 1
        for (int o = threadIdx.x; o < kWindow; o += kThreads) {
            const uint32_t n = word_at(kNegative + o * 4);
            if (n) m += W.mass(n, W.of(B::value(o0 + o), sh.powers));
        }
        sync_warps();
    }
    m = warp_sum64(m);
    if ((threadIdx.x & 31) == 0) sh.plain[threadIdx.x >> 5] = m;
}
// The found token's softmax probability, of the first `n` parts (one thread).
__device__ __noinline__ float softmax_of(float top, int shift, int n) {
    Shared& sh = shared();
    Weights W;
    W.set(top, 1.0f, 0.0f);
    u64 all = 0;
#pragma unroll 8
    for (int k = 0; k < n; ++k) all += sh.plain[k];
    return probability(W.of(__uint_as_float(sh.found.bits << 16), sh.powers), all, shift);
}

// Which of the first `have` halves of four words are 0, a bit each.
__device__ __noinline__ uint32_t zero_halves(uint32_t a, uint32_t b, uint32_t c, uint32_t d, int have) {
    uint32_t h = (a & 0xffffu) == 0 | (a >> 16 == 0) << 1 | ((b & 0xffffu) == 0) << 2 | (b >> 16 == 0) << 3;
    h |= ((c & 0xffffu) == 0) << 4 | (c >> 16 == 0) << 5 | ((d & 0xffffu) == 0) << 6 | (d >> 16 == 0) << 7;
    return have < 8 ? h & ((1u << have) - 1u) : h;
}

// Token number r (from the lowest) of the n with value `bits` in values [e0, e1) of x; `token` is where it goes.  Every
// thread calls.  A pass takes 16384 values in their order (piece d of 4, thread, value) and counts the matches; the pass
// that reaches r is resolved.  From the slice's end, whose values came last: what L2 holds of the rows in flight (304 of
// 300 KB) is their later part.
__device__ __noinline__ void locate(const uint16_t* x, int* token, uint32_t bits, uint32_t r, uint32_t n, int e0, int e1) {
    Shared& sh = shared();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t both = bits | bits << 16, care = bits == 0 ? 0x7fff7fffu : 0xffffffffu;
    constexpr int kDeep = 4, kPass = kThreads * 8 * kDeep;   // 32 KB of the CTA's in flight
    uint32_t behind = n - 1 - r;                             // matches behind the wanted one
    if (tid < 3) sh.counts[tid] = 0;
    sync_warps();
#pragma unroll 1
    for (int e = e0 + (e1 - e0 - 1) / kPass * kPass, pass = 0; e >= e0; e -= kPass, pass = pass == 2 ? 0 : pass + 1) {
        uint4 q[kDeep];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int at = e + (d * kThreads + tid) * 8;
            q[d] = at < e1 ? __ldg(reinterpret_cast<const uint4*>(x + at)) : make_uint4(~both, ~both, ~both, ~both);
        }
        uint32_t hit = 0;   // 8 bits of a piece each
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            // a half that is 0 after the xor is one whose borrow sets its top bit; the halves are looked at only then
            const uint32_t t[4] = {(q[d].x ^ both) & care, (q[d].y ^ both) & care, (q[d].z ^ both) & care,
                                   (q[d].w ^ both) & care};
            const uint32_t any = (((t[0] - 0x00010001u) & ~t[0]) | ((t[1] - 0x00010001u) & ~t[1]) |
                                  ((t[2] - 0x00010001u) & ~t[2]) | ((t[3] - 0x00010001u) & ~t[3])) & 0x80008000u;
            if (any) hit |= zero_halves(t[0], t[1], t[2], t[3], e1 - (e + (d * kThreads + tid) * 8)) << (d * 8);
        }
        if (hit) atomicAdd(&sh.counts[pass], __popc(hit));
        if (tid == 0) sh.counts[pass == 2 ? 0 : pass + 1] = 0;
        sync_warps();
        const uint32_t all = sh.counts[pass];
        if (behind >= all) {
            behind -= all;
            continue;
        }
        r = all - 1 - behind;
        // 64 groups in order: piece d, warp
        static_assert(kDeep * kWarps == 64, "two groups a lane");
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const uint32_t c = __reduce_add_sync(0xffffffffu, __popc(hit >> (d * 8) & 0xffu));
            if (lane == 0) sh.groups[d * kWarps + warp] = c;
        }
        sync_warps();
        auto before_of = [&](uint32_t c) {   // sum over the lanes before this one
            uint32_t s = c;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, s, off);
                if (lane >= off) s += y;
            }
            return s - c;
        };
        const uint32_t g0 = sh.groups[2 * lane], g1 = sh.groups[2 * lane + 1];
        const uint32_t start = before_of(g0 + g1);
        const int src = 31 - __clz(__ballot_sync(0xffffffffu, start <= r && g0 + g1 > 0));   // its pair of groups
        const uint32_t left = r - __shfl_sync(0xffffffffu, start, src), of0 = __shfl_sync(0xffffffffu, g0, src);
        const int g = 2 * src + (left >= of0);
        const uint32_t want = left >= of0 ? left - of0 : left;   // within the group
        if (g % kWarps == warp) {
            const int d = g / kWarps;
            uint32_t h = hit >> (d * 8) & 0xffu;
            const uint32_t before = before_of(__popc(h));
            if (want >= before && want < before + __popc(h)) {
#pragma unroll 1
                for (uint32_t k = before; k < want; ++k) h &= h - 1;
                *token = e + (d * kThreads + tid) * 8 + __ffs(h) - 1;
            }
        }
        break;
    }
    sync_warps();
}

// One 16-byte piece: its values into the counters, its maximum into `top`.
__device__ __forceinline__ void count_word(uint32_t w, uint32_t base, uint32_t& top) {
    top = max_nan_bf16x2(top, w);
    uint32_t a = w & 0x7fff7fffu;
    a = min_bf16x2(bf16x2_max(a, kLow | kLow << 16), kHigh | kHigh << 16);
    // 4 (a - low) of both halves, the sign above it
    const uint32_t at = (a * 4 - (kLow | kLow << 16) * 4) | (w & 0x80008000u);
    count_at(base + (at & 0xffffu));
    count_at(base + (at >> 16));
}

// kConf: with the softmax probability (in the same kernel, unused, it cost the plain draw 2 %: code to fetch).
template <bool kConf>
__global__ void __launch_bounds__(kThreads + 32, kPerSm) sample_kernel(const __grid_constant__ SampleParams P) {
    Shared& sh = shared();
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        sh.abort = 0;
        for (int k = 0; k < kStages; ++k) {
            mbar_init(smem_addr(&sh.full[k]), 1);
            mbar_init(smem_addr(&sh.empty[k]), kWarps);
        }
        for (int k = 0; k < 2; ++k) mbar_init(smem_addr(&sh.meet[k]), P.cluster);
        mbar_fence_init();
    }
    if (tid < kPowers) sh.powers[tid] = c_powers.t[tid];
    __syncthreads();
    const int ctas = P.cluster;
    if (ctas > 1) cluster_sync();
    pdl_wait();
    pdl_release();
    const int rank = ctas > 1 ? (int)cluster_rank() : 0;
    const int first = blockIdx.x / ctas, step = gridDim.x / ctas;
    const int e0 = min(rank * P.slice, P.V), e1 = min(e0 + P.slice, P.V);
    const int chunks = (e1 - e0 + kChunk - 1) / kChunk;
    auto row_of = [&](int i) -> const uint16_t* {
        const long long r = P.rows ? (long long)__ldg(P.rows + i) : i;
        return r >= 0 && r < P.logits_rows ? P.logits + r * P.ldv : nullptr;
    };
    if (warp == kWarps) {
        // -------------------------------------------------------------- copies
        if (lane == 0) {
            uint32_t n = 0;
            uint64_t keep;
            asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
            bool lost = false;
            for (int i = first; i < P.N && !lost; i += step) {
                const uint16_t* const x = row_of(i);
                if (!x) continue;
#pragma unroll 1
                for (int c = 0; c < chunks; ++c, ++n) {
                    const uint32_t k = n % kStages;
                    if (!mbar_wait_bounded(smem_addr(&sh.empty[k]), (n / kStages & 1) ^ 1, kWaitNs) ||
                        *(volatile int*)&sh.abort) {
                        set_error(P.err, DLLM_DEVERR_TIMEOUT);
                        *(volatile int*)&sh.abort = 1;
                        lost = true;
                        break;
                    }
                    const int v0 = e0 + c * kChunk;
                    const uint32_t bytes = min(kChunk / 8, (e1 - v0 + 7) / 8) * 16;
                    mbar_arrive_expect_tx(smem_addr(&sh.full[k]), bytes);
                    bulk_g2s(base + kRing + k * kChunk * 2, x + v0, bytes, smem_addr(&sh.full[k]), keep);
                }
            }
        }
        __syncwarp();
        if (ctas > 1) cluster_sync();
        return;
    }
    // ------------------------------------------------------------------ counts
    uint32_t n = 0;
    Meeting meeting{smem_addr(&sh.meet[0]), 0, ctas};
    for (int i = first; i < P.N; i += step) {
        const uint16_t* const x = row_of(i);
        if (!x) {
            if (rank == 0 && tid == 0) {
                P.tokens[i] = -1;
                P.prob[i] = __int_as_float(0x7fc00000);
                if constexpr (kConf) P.conf[i] = __int_as_float(0x7fc00000);
            }
            continue;
        }
        const float T = P.temperature ? __ldg(P.temperature + i) : 1.0f, u = __ldg(P.u + i);
        const float p = P.top_p ? __ldg(P.top_p + i) : 1.0f, min_p = P.min_p ? __ldg(P.min_p + i) : 0.0f;
        const int k = P.top_k ? __ldg(P.top_k + i) : 0;
#pragma unroll 1
        for (uint32_t at = tid * 16; at < (kValues + 1) * 4; at += kThreads * 16) {
            // the last piece may reach into the word behind, which is padding on both sides
            *reinterpret_cast<uint4*>(smem + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(smem + kNegative + at) = make_uint4(0, 0, 0, 0);
        }
        sync_warps();
        uint32_t top = 0xff80ff80u;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c, ++n) {
            const uint32_t stage = n % kStages;
            if (*(volatile int*)&sh.abort == 0 &&
                !mbar_wait_bounded(smem_addr(&sh.full[stage]), n / kStages & 1, kWaitNs)) {
                set_error(P.err, DLLM_DEVERR_TIMEOUT);
                *(volatile int*)&sh.abort = 1;
            }
            const int left = e1 - (e0 + c * kChunk);
            const uint4* const in = reinterpret_cast<const uint4*>(smem + kRing + stage * kChunk * 2);
            constexpr int kPieces = kChunk / 8 / kThreads;
            uint4 q[kPieces];
#pragma unroll
            for (int d = 0; d < kPieces; ++d) q[d] = in[d * kThreads + tid];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.empty[stage]));
            if (left < kChunk) {   // -inf behind the slice's end
#pragma unroll
                for (int d = 0; d < kPieces; ++d) {
                    const int have = left - (d * kThreads + tid) * 8;   // values of this piece
                    q[d].x = have > 1 ? q[d].x : (q[d].x & 0xffffu) | 0xff800000u;
                    q[d].y = have > 3 ? q[d].y : have > 2 ? (q[d].y & 0xffffu) | 0xff800000u : 0xff80ff80u;
                    q[d].z = have > 5 ? q[d].z : have > 4 ? (q[d].z & 0xffffu) | 0xff800000u : 0xff80ff80u;
                    q[d].w = have > 7 ? q[d].w : have > 6 ? (q[d].w & 0xffffu) | 0xff800000u : 0xff80ff80u;
                }
            }
#pragma unroll
            for (int d = 0; d < kPieces; ++d) {
                if ((d * kThreads + tid) * 8 >= left) break;
                count_word(q[d].x, base, top);
                count_word(q[d].y, base, top);
                count_word(q[d].z, base, top);
                count_word(q[d].w, base, top);
            }
        }
        // what the slice holds besides the counted values
        float m = max_nan(bf16_lo(top), bf16_hi(top));
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane == 0) sh.part[warp] = m;
        if (tid == 0) sh.flag = 0;
        sync_warps();
        uint32_t* const pos = reinterpret_cast<uint32_t*>(smem);
        uint32_t* const neg = reinterpret_cast<uint32_t*>(smem + kNegative);
        const bool zeros = pos[0] + neg[0] > 0;
        if (zeros) {   // exact zeros, or small values that only the wide path tells apart
            bool small = false;
#pragma unroll 1
            for (int e = e0 + tid * 8; e < e1; e += kThreads * 8) {
                const uint4 q = *reinterpret_cast<const uint4*>(x + e);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t a = w[k / 2] >> (k & 1 ? 16 : 0) & 0x7fffu;
                    small = small || (a != 0 && a <= kLow && e + k < e1);
                }
            }
            if (__any_sync(0xffffffffu, small) && lane == 0) sh.flag = 1;
            sync_warps();
        }
        if (tid == 0) {
            SliceFacts f;
            f.max = sh.part[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) f.max = max_nan(f.max, sh.part[w]);
            f.other = sh.flag | (pos[kValues] > 0);
            f.low = (int)neg[kValues] - ((e0 - e1) & 7);   // without what fills the last piece
            sh.facts = f;
            pos[0] += neg[0];   // -0 is 0
            neg[0] = 0;
        }
        if (ctas > 1) {
            meeting.arrive();
            meeting.wait(&sh.abort, P.err);
        } else {
            sync_warps();
        }
        SliceFacts all = sh.facts;
        if (ctas > 1) {
            const uint32_t at = smem_addr(&sh.facts);
            all = SliceFacts{-INFINITY, 0, 0};
#pragma unroll 1
            for (int q = 0; q < ctas; ++q) {
                all.max = max_nan(all.max, __uint_as_float(peer_load(at, q)));
                all.other |= (int)peer_load(at + 4, q);
                all.low += (int)peer_load(at + 8, q);
            }
        }
        const bool ok = isfinite(all.max) && T >= 0.0f;
        Weights W;
        W.shift = P.shift;
        W.set(all.max, T == 0.0f ? 1.0f : T, T == 0.0f ? 0.0f : min_p);
        // low values count where their weights may: -256 is the largest (-inf is counted with them, so from a temperature of
        // (256 + maximum) / 55 on a row with masked tokens goes the wide path too)
        const bool wide = all.other || (all.low > 0 && W.rough(-256.0f) > -80.0f);
        if (tid == 0) sh.row = RowFacts{W, x, P.V, ctas};
        if (ok && !wide) {
            // Sums of the segments, a warp 2 neighbouring ones at a time: the weights' chains of operations run side by side
            constexpr int kGroup = 2;
            static_assert(kSegments % kGroup == 0, "whole groups");
#pragma unroll 1
            for (int g = rank * kWarps + warp; g * kGroup < kSegments; g += ctas * kWarps) {
                int o[kGroup];
                uint32_t c[kGroup], any = 0;
                u64 mass[kGroup] = {};
#pragma unroll
                for (int j = 0; j < kGroup; ++j) o[j] = (g * kGroup + j) * 32 + lane;
                counts_of(o, c, ctas);
#pragma unroll
                for (int j = 0; j < kGroup; ++j) any |= c[j];
                if (__any_sync(0xffffffffu, any)) {
#pragma unroll
                    for (int j = 0; j < kGroup; ++j) {
                        const u64 w = W.of(Bins<false>::value(o[j]), sh.powers);
                        if (w == 0) c[j] = 0;
                        mass[j] = W.mass(c[j], w);
                    }
#pragma unroll
                    for (int j = 0; j < kGroup; ++j) {
                        c[j] = __reduce_add_sync(0xffffffffu, c[j]);
                        mass[j] = warp_sum64(mass[j]);
                    }
                }
                if (lane < kGroup) {
                    const uint32_t count = lane ? c[1] : c[0];
                    const u64 m = lane ? mass[1] : mass[0];
                    const int seg = g * kGroup + lane;
                    if (ctas > 1) {
                        peer_store(smem_addr(&sh.seg_count[seg]), 0, count);
                        peer_store64(smem_addr(&sh.seg_mass[seg]), 0, m);
                    } else {
                        sh.seg_count[seg] = count;
                        sh.seg_mass[seg] = m;
                    }
                }
            }
            if constexpr (kConf) sum_plain(all.max, P.shift, rank, ctas);
        }
        if (ctas > 1) {
            meeting.arrive();
            meeting.wait(&sh.abort, P.err);
        } else {
            sync_warps();
        }
        if (rank == 0 && ok) {
            if (!wide) {
                add_up<false>();
                if (warp == 0) choose<false>(u, T == 0.0f ? 1 : k, p);
            } else {
                sum_wide();
                add_up<true>();
                choose<true>(u, T == 0.0f ? 1 : k, p);
                if constexpr (kConf) sum_plain_wide();
            }
        }
        if (ctas > 1) {
            meeting.arrive();
            meeting.wait(&sh.abort, P.err);
        } else {
            sync_warps();
        }
        uint32_t bits = sh.found.bits, r = sh.found.r, count = sh.found.n;
        int l0 = e0, l1 = e1;
        bool mine = ok && (rank == 0 || !wide);
        if (wide) {
            l0 = 0;
            l1 = P.V;
        } else if (ctas > 1 && ok) {
            // the slice that holds the token
            const uint32_t at = smem_addr(&sh.found);
            bits = peer_load(at + offsetof(Found, bits), 0);
            r = peer_load(at + offsetof(Found, r), 0);
            mine = false;
            const uint32_t c0 = (bits & 0x7fffu) == 0 ? 0 : min((bits & 0x7fffu) - kLow, (uint32_t)kValues);
            const uint32_t counter = (bits & 0x8000u ? kNegative : 0u) + c0 * 4;
#pragma unroll 1
            for (int q = 0; q <= rank; ++q) {
                const uint32_t c = peer_load(base + counter, q);
                if (q == rank) mine = r < (count = c);
                else if (r >= c) r -= c;
                else break;   // a slice before this one
            }
        }
        if (ctas > 1) meeting.arrive();   // this CTA has read the others' counters
        if (rank == 0 && tid == kThreads - 32) {
            P.prob[i] = ok ? probability(sh.found.w, sh.kept, P.shift) : __int_as_float(0x7fc00000);
            if (!ok) P.tokens[i] = -1;
            if constexpr (kConf)
                P.conf[i] = ok ? softmax_of(all.max, P.shift, wide ? kWarps : ctas * kWarps) : __int_as_float(0x7fc00000);
        }
        if (mine) locate(x, P.tokens + i, bits, r, count, l0, l1);
        if (ctas > 1) meeting.wait(&sh.abort, P.err);
        else sync_warps();
    }
    // after a wait that gave up: copies still in flight land in this CTA's memory, not in its successor's
    if (*(volatile int*)&sh.abort) __nanosleep(1000000);
    // no CTA leaves while another may arrive at its barriers, even where waits gave up
    __syncwarp();
    if (ctas > 1) cluster_sync();
}

}  // namespace
}  // namespace dllm

using namespace dllm;

namespace {
int launch_sample(const dllm_sample_args* a, float* conf, void* stream) {
    if (!a || a->N < 0 || a->V < 1 || a->logits_rows < 0 || a->ldv < a->V) return DLLM_ERR_INVAL;
    if (a->N > 0 && ((a->logits_rows > 0 && !a->logits) || !a->u || !a->tokens || !a->prob)) return DLLM_ERR_INVAL;
    if ((reinterpret_cast<uintptr_t>(a->logits) & 15) || a->ldv % 8) return DLLM_ERR_ALIGN;
    if (a->V > 1 << 28) return DLLM_ERR_UNSUPPORTED;
    if (a->N == 0) return DLLM_OK;
    const int sms = sm_count();
    if (sms <= 0) return DLLM_ERR_CUDA;
    SampleParams P;
    P.N = a->N;
    P.V = a->V;
    P.ldv = a->ldv;
    P.logits_rows = a->logits_rows;
    P.logits = a->logits;
    P.rows = a->rows;
    P.u = a->u;
    P.temperature = a->temperature;
    P.top_k = a->top_k;
    P.top_p = a->top_p;
    P.min_p = a->min_p;
    P.tokens = a->tokens;
    P.prob = a->prob;
    P.conf = conf;
    P.err = error_word_ptr();
    if (!P.err) return DLLM_ERR_CUDA;
    int c = 1;
    while (c < kMaxCluster && (long long)a->N * c < sms && a->V / (2 * c) >= kLeast) c *= 2;
    P.cluster = c;
    P.slice = ((a->V + c - 1) / c + 7) / 8 * 8;
    int bits = 0;   // V tokens of mass 2^(62 - shift) stay below 2^62
    while ((1ll << bits) <= a->V) ++bits;
    P.shift = std::max(16, bits);
    const auto kernel = conf ? sample_kernel<true> : sample_kernel<false>;
    static SmemOnce done[2];
    DLLM_CUDA_TRY(allow_smem(kernel, kSmem, done[conf ? 1 : 0]));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(a->N, sms * kPerSm / c) * c);
    cfg.blockDim = dim3(kThreads + 32);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c > 1 ? 2 : 1;
    DLLM_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, P));
    return DLLM_OK;
}
}  // namespace

extern "C" int dllm_sample(const dllm_sample_args* a, void* stream) { return launch_sample(a, nullptr, stream); }

extern "C" int dllm_sample_conf(const dllm_sample_args* a, float* conf, void* stream) {
    if (a && a->N > 0 && !conf) return DLLM_ERR_INVAL;
    return launch_sample(a, conf, stream);
}
