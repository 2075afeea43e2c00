// dllm_sample: one token per logits row, drawn with temperature, top-k, min-p and
// top-p by a given number u in [0, 1).
//
// Mathematics.  In the order of falling values (ties: lowest token first) with
// w = exp((x - m) / T), every filter keeps a prefix, and the draw is the first
// token whose cumulative w passes u times the kept mass.  u lies next to one of
// up to V borders, so an error eps of the cumulative masses draws another token
// about (mean rank of the draw) * eps times: 32-bit sums (1e-7) would err once in
// some hundred rows of a flat distribution.  A bf16 row holds few different
// values, though: a histogram of its values is exact, each value's weight is
// computed once, to 2^-44 in its exponent and 2^-62 in itself, and masses are
// sums of count * weight in 64-bit fixed point.  The rest works on the histogram:
// what the filters leave, the mass, the value that the draw falls on, and which
// of the tokens with that value, counted from the lowest, it is.
//
// Split.  A cluster of 1 to 8 CTAs takes a row, each CTA a slice: a copying warp
// keeps the ring of bulk copies full (also with the next rows' pieces), eight
// warps count values with shared-memory atomics.  Segments of 32 values are
// summed by all warps of the cluster (counts of the others by distributed shared
// memory), one warp walks the segments' sums, and the CTA whose slice holds the
// token reads its slice again (from L2) to find it.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"

namespace dllm {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;   // counting threads of a CTA
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 7;
constexpr int kChunk = 4096;    // values of a stage
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
constexpr int kList = 1024;     // tokens of the drawn value held at once
constexpr int kBuckets = 256;

// Tables of 2^(i / 16^(l+1)): level 0 in units of 2^-62, the others less 1 in
// units of 2^-64, from square roots of 2 in whole numbers.
struct PowerTable {
    u64 t[4][16];
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
    u64 root[16] = {};                         // 2^(2^-(k+1)) in units of 2^-63
    unsigned __int128 v = (unsigned __int128)1 << 127;   // 2 * 2^126
    for (int k = 0; k < 16; ++k) {
        root[k] = root_of(v);
        v = (unsigned __int128)root[k] << 63;
    }
    PowerTable p = {};
    for (int l = 0; l < 4; ++l)
        for (int i = 0; i < 16; ++i) {
            unsigned __int128 x = (unsigned __int128)1 << 63;
            for (int b = 0; b < 4; ++b)
                if (i >> b & 1) x = x * root[4 * l + 3 - b] >> 63;
            p.t[l][i] = l == 0 ? (u64)(x >> 1) : (u64)((x - ((unsigned __int128)1 << 63)) << 1);
        }
    return p;
}
__constant__ PowerTable c_powers = make_powers();
static_assert(make_powers().t[0][8] == 6521908912666391106ull, "sqrt(2) * 2^62");

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
    int* err;
    int cluster, slice;   // values of a CTA's slice
    int shift;            // masses are in units of 2^(shift - 62)
};

// What a CTA tells the others of its slice.
struct SliceFacts {
    float max;    // NaN if the slice holds one
    int other;    // values that only the wide path tells apart
    int low;      // values at or under -2^8
};

struct Draw {
    uint32_t bits;  // the value; zero stands for both zeros
    long long r;    // which of its tokens
    float prob;
};

struct Shared {
    uint64_t full[kStages], empty[kStages], meet[2];
    u64 powers[4][16];
    u64 seg_mass[kSegments];
    uint32_t seg_count[kSegments];
    int list[kList];
    int buckets[kBuckets];
    float part[kWarps];
    SliceFacts facts;
    Draw draw;
    u64 found_mass;
    int abort, count, segment, flag;
};
constexpr uint32_t kGap = (kValues + 1) * 4 + 15 & ~15u;   // the struct lies between the counters of both signs
static_assert(kGap + sizeof(Shared) <= kNegative, "fits between the counters");
constexpr uint32_t kRing = (kNegative + (kValues + 1) * 4 + 127) & ~127u;
constexpr size_t kSmem = kRing + kStages * kChunk * 2;
static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
// the wide path's: window counters where the negatives' are, segment sums where the positives' are
static_assert(kWindow * 4 <= (kValues + 1) * 4 && kWideSegments * 12 <= kGap, "the wide path's arrays");

__device__ __forceinline__ void sync_warps() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
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
__device__ __forceinline__ uint32_t peer_load(uint32_t at, int cta) {
    uint32_t v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(peer_addr(at, cta)) : "memory");
    return v;
}
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
    __device__ __forceinline__ void wait(int* abort, int* err) {
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

// The weights of one row's values.
struct Weights {
    double m, s;      // the maximum; log2(e) / T
    float m32, s32;
    u64 least;        // min-p in units of 2^-62: smaller weights are left out
    int shift;

    // w in units of 2^-62; 0 below 2^-75 and where min-p leaves the value out.
    __device__ __forceinline__ u64 of(float x, const u64 (*pw)[16]) const {
        if (x == m32) return 1ull << 62;
        if (!((x - m32) * s32 > -75.0f)) return 0;
        // y = (x - m) s, rounded to 2^-44: 384 + y stays in [256, 512)
        const double r = fma((double)x - m, s, 384.0);
        const long long y = __double_as_longlong(r) - __double_as_longlong(384.0);
        const int n = (int)(y >> 44);                       // <= -1, or 0 with no fraction
        const uint32_t hi = (uint32_t)(y >> 28);            // the 16 upper bits of the fraction
        const u64 rest = (u64)(y & 0xfffffffll);            // < 2^-16
        // 2^rest - 1 = a + a^2 / 2, a = rest ln 2 (what follows is under 2^-51), in units of 2^-64
        const u64 a = rest * 0xb17217f8ull >> 12;
        const u64 a24 = a >> 24;
        u64 w = pw[0][hi >> 12 & 15];
        w += __umul64hi(w, pw[1][hi >> 8 & 15]);
        w += __umul64hi(w, pw[2][hi >> 4 & 15]);
        w += __umul64hi(w, pw[3][hi & 15]);
        w += __umul64hi(w, a + (a24 * a24 >> 17));
        w >>= min(-n, 63);
        return w >= least ? w : 0;
    }
    __device__ __forceinline__ double unit() const { return __longlong_as_double((long long)(1023 - shift) << 52); }
    // Mass of `count` tokens of weight w.
    __device__ __forceinline__ u64 mass(uint32_t count, u64 w) const {
        const u64 lo = (u64)count * (uint32_t)w, hi = (u64)count * (uint32_t)(w >> 32);
        return (hi << (32 - shift)) + ((lo + (1ull << (shift - 1))) >> shift);
    }
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {   // v < 2^59
    const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x7ffffffu);
    const uint32_t mid = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 27) & 0x7ffffffu);
    const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 54));
    return (u64)lo + ((u64)mid << 27) + ((u64)hi << 54);
}

// One row as a cluster (rank 0 to `cluster` - 1) or, in the wide path, rank 0 alone
// sees it.
struct Row {
    const SampleParams& P;
    Shared& sh;
    unsigned char* smem;
    uint32_t base;           // of the dynamic shared memory
    const uint16_t* x;
    Weights W;
    bool wide;

    // The value of bin o, in falling order.
    __device__ __forceinline__ uint32_t bits_of(int o) const {
        if (wide) {
            const uint32_t key = 0xffffu - o;
            return key & 0x8000u ? key ^ 0x8000u : ~key & 0xffffu;
        }
        if (o < kHalfBins) {
            const int c = kHalfBins - 1 - o;
            return c == 0 ? 0 : kLow + c;
        }
        return 0x8000u | (kLow + (o - kHalfBins));
    }
    // Its counters, over the cluster.  Bins without a value of their own: 0.
    __device__ __forceinline__ uint32_t count_of(int o) const {
        if (wide) return reinterpret_cast<const uint32_t*>(smem + kNegative)[o];
        const bool neg = o >= kHalfBins;
        const int c = neg ? o - kHalfBins : kHalfBins - 1 - o;
        if (c >= kValues || (neg && c == 0)) return 0;
        const uint32_t at = (neg ? kNegative : 0u) + c * 4;
        uint32_t n = 0;
        if (P.cluster == 1) {
            n = *reinterpret_cast<const uint32_t*>(smem + at);
            if (c == 0) n += *reinterpret_cast<const uint32_t*>(smem + kNegative);   // -0 is 0
            return n;
        }
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q)
            if (q < P.cluster) {
                n += peer_load(base + at, q);
                if (c == 0) n += peer_load(base + kNegative, q);
            }
        return n;
    }
    __device__ __forceinline__ int segments() const { return wide ? kWideSegments : kSegments; }
    __device__ __forceinline__ int segment_bins() const { return wide ? kWideSegment : 32; }
    __device__ __forceinline__ uint32_t seg_count(int s) const {
        return wide ? reinterpret_cast<const uint32_t*>(smem + kWideSegments * 8)[s] : sh.seg_count[s];
    }
    __device__ __forceinline__ u64 seg_mass(int s) const {
        return wide ? reinterpret_cast<const u64*>(smem)[s] : sh.seg_mass[s];
    }

    // Counts the row's values with keys 0xffff - o for o in [o0, o0 + n), n a power of two (wide path; every thread).
    __device__ void count_keys(int o0, int n) const {
        uint32_t* const counts = reinterpret_cast<uint32_t*>(smem + kNegative);
        for (int i = threadIdx.x; i < n; i += kThreads) counts[i] = 0;
        sync_warps();
        for (int e = threadIdx.x * 8; e < P.V; e += kThreads * 8) {
            const uint4 q = *reinterpret_cast<const uint4*>(x + e);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t b = w[k / 2] >> (k & 1 ? 16 : 0) & 0xffffu;
                if (b == 0x8000u) b = 0;
                const uint32_t o = 0xffffu - (b & 0x8000u ? ~b & 0xffffu : b | 0x8000u);
                if (o - o0 < (uint32_t)n && b != 0xff80u && e + k < P.V) atomicAdd(&counts[o - o0], 1u);
            }
        }
        sync_warps();
    }

    struct Lane {      // sums before this lane's segments, and of them
        uint32_t count0;
        u64 mass0;
        uint32_t total_count;
        u64 total_mass;
        int s0, s1;
    };
    // One warp: every lane's run of segments.
    __device__ Lane walk() const {
        const int lane = threadIdx.x & 31, n = segments(), per = (n + 31) / 32;
        Lane L;
        L.s0 = min(lane * per, n);
        L.s1 = min(L.s0 + per, n);
        uint32_t c = 0;
        u64 m = 0;
        for (int s = L.s0; s < L.s1; ++s) {
            c += seg_count(s);
            m += seg_mass(s);
        }
        uint32_t ci = c;
        u64 mi = m;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t cy = __shfl_up_sync(0xffffffffu, ci, off);
            const u64 my = __shfl_up_sync(0xffffffffu, mi, off);
            if (lane >= off) {
                ci += cy;
                mi += my;
            }
        }
        L.count0 = ci - c;
        L.mass0 = mi - m;
        L.total_count = __shfl_sync(0xffffffffu, ci, 31);
        L.total_mass = __shfl_sync(0xffffffffu, mi, 31);
        return L;
    }

    struct Found {
        u64 mass;        // of the tokens up to and with the one found
        uint32_t bits;   // its value
        uint32_t r;      // which of the value's tokens, from 0
        u64 w;
    };
    // The first token whose count reaches `target` (by_count), or whose cumulative mass does; a target within the
    // totals.  The warp that walks calls with its lanes' sums; in the wide path every thread calls.
    __device__ Found find(const Lane& L, bool by_count, u64 target) const {
        const int lane = threadIdx.x & 31;
        Found f = {};
        uint32_t c0 = 0;
        u64 m0 = 0;
        int seg = 0;
        if (threadIdx.x < 32) {
            // the lane whose run holds the target, then its segment
            uint32_t c = L.count0;
            u64 m = L.mass0;
            int mine = -1;
            for (int s = L.s0; s < L.s1 && mine < 0; ++s) {
                const uint32_t cn = c + seg_count(s);
                const u64 mn = m + seg_mass(s);
                if ((by_count ? (u64)cn : mn) >= target) {
                    mine = s;
                } else {
                    c = cn;
                    m = mn;
                }
            }
            const unsigned who = __ballot_sync(0xffffffffu, mine >= 0);
            const int src = who ? __ffs(who) - 1 : 31;
            seg = max(0, __shfl_sync(0xffffffffu, mine, src));
            c0 = __shfl_sync(0xffffffffu, c, src);
            m0 = __shfl_sync(0xffffffffu, m, src);
            if (wide && lane == 0) sh.segment = seg;
        }
        if (wide) {
            sync_warps();
            count_keys(sh.segment * kWideSegment, kWideSegment);
        }
        if (threadIdx.x < 32) {
            for (int b0 = 0; b0 < segment_bins(); b0 += 32) {
                const int o = seg * segment_bins() + b0 + lane;
                uint32_t n = count_of(wide ? b0 + lane : o);
                const uint32_t bits = bits_of(o);
                const u64 w = n ? W.of(__uint_as_float(bits << 16), sh.powers) : 0;
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
                const u64 have = by_count ? (u64)(c0 + ci) : m0 + mi;
                const unsigned who = __ballot_sync(0xffffffffu, n && have >= target);
                if (who) {
                    // tokens of the bin that are needed, 1 to n
                    uint32_t j;
                    const u64 before = m0 + mi - mine;
                    if (by_count) {
                        j = (uint32_t)(target - (c0 + ci - n));
                    } else {
                        const u64 rem = target > before ? target - before : 1;
                        const double one = (double)w * W.unit();
                        j = (uint32_t)min(max(ceil(((double)rem - 0.5) / one), 1.0), (double)n);
                        for (int k = 0; k < 4 && j > 1 && W.mass(j - 1, w) >= rem; ++k) --j;
                        for (int k = 0; k < 4 && j < n && W.mass(j, w) < rem; ++k) ++j;
                    }
                    const int src = __ffs(who) - 1;
                    f.mass = __shfl_sync(0xffffffffu, before + W.mass(j, w), src);
                    f.bits = __shfl_sync(0xffffffffu, bits, src);
                    f.r = __shfl_sync(0xffffffffu, j - 1, src);
                    f.w = __shfl_sync(0xffffffffu, w, src);
                    break;
                }
                c0 += __shfl_sync(0xffffffffu, ci, 31);
                m0 += __shfl_sync(0xffffffffu, mi, 31);
            }
        }
        if (wide) sync_warps();
        return f;
    }

    // Filters and draw, from the segments' sums.  As find() is called.
    __device__ void choose(int i, float T) const {
        Lane L = {};
        if (threadIdx.x < 32) L = walk();
        const float u = __ldg(P.u + i);
        const float p = P.top_p ? __ldg(P.top_p + i) : 1.0f;
        int k = P.top_k ? __ldg(P.top_k + i) : 0;
        if (T == 0.0f) k = 1;
        // the other warps (wide path) follow the walking one's branches
        u64 kept = L.total_mass;
        bool cut = k > 0 && (uint32_t)k < L.total_count;
        if (wide) cut = share(cut);
        if (cut) kept = find(L, true, (uint32_t)k).mass;
        if (p < 1.0f) {
            const double t = ceil((double)p * (double)kept);
            const u64 target = t >= 1.0 ? min((u64)t, kept) : 1;
            kept = min(kept, find(L, false, target).mass);
        }
        const double t = (double)u * (double)kept;
        const u64 target = t >= 0.0 ? (t < (double)kept ? min((u64)t + 1, kept) : kept) : 1;
        const Found f = find(L, false, target);
        if (threadIdx.x == 0) {
            sh.draw.bits = f.bits;
            sh.draw.r = f.r;
            sh.draw.prob = (float)((double)f.w * W.unit() / (double)kept);
        }
    }
    __device__ bool share(bool v) const {
        if (threadIdx.x == 0) sh.flag = v;
        sync_warps();
        v = sh.flag;
        sync_warps();
        return v;
    }

    // The wide path's segment sums: windows of keys from the maximum's down, as far as weights reach (every thread).
    __device__ void sum_wide() const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        u64* const mass = reinterpret_cast<u64*>(smem);
        uint32_t* const count = reinterpret_cast<uint32_t*>(smem + kWideSegments * 8);
        for (int s = threadIdx.x; s < kWideSegments; s += kThreads) {
            mass[s] = 0;
            count[s] = 0;
        }
        for (int o0 = 0; o0 < 65536; o0 += kWindow) {
            // the window's first finite value is its largest: its last one is the smallest
            const float last = __uint_as_float(bits_of(o0 + kWindow - 1) << 16), first = __uint_as_float(bits_of(o0) << 16);
            if (last > W.m32) continue;                                        // all above the maximum
            if (!isnan(first) && first < W.m32 && W.of(first, sh.powers) == 0) break;
            count_keys(o0, kWindow);
            for (int s = warp; s < kWindow / kWideSegment; s += kWarps) {
                uint32_t c = 0;
                u64 m = 0;
                for (int b = lane; b < kWideSegment; b += 32) {
                    const int o = s * kWideSegment + b;
                    const uint32_t n = count_of(o);
                    const u64 w = n ? W.of(__uint_as_float(bits_of(o0 + o) << 16), sh.powers) : 0;
                    if (w) c += n;
                    m += W.mass(n, w);
                }
                c = __reduce_add_sync(0xffffffffu, c);
                m = warp_sum64(m);
                if (lane == 0) {
                    mass[o0 / kWideSegment + s] = m;
                    count[o0 / kWideSegment + s] = c;
                }
            }
            sync_warps();
        }
        sync_warps();
    }

    // Token number r (from the lowest) of those with value `bits` in [e0, e1), into P.tokens[i].  Every thread calls.
    __device__ void locate(int i, uint32_t bits, long long r, int e0, int e1) const {
        const uint32_t care = bits == 0 ? 0x7fffu : 0xffffu;
        int span = e1 - e0;
        for (;;) {
            // gather the matches; too many for the list: a bucket of the range that holds the wanted one
            const int per = max(8, ((span + kBuckets - 1) / kBuckets + 7) / 8 * 8);
            for (int b = threadIdx.x; b < kBuckets; b += kThreads) sh.buckets[b] = 0;
            if (threadIdx.x == 0) sh.count = 0;
            sync_warps();
            constexpr int kDeep = 8;   // 32 KB of the CTA's in flight
            for (int e = e0 + (int)threadIdx.x * 8; e < e0 + span; e += kThreads * 8 * kDeep) {
                uint4 q[kDeep];
#pragma unroll
                for (int d = 0; d < kDeep; ++d) {
                    const int at = e + d * kThreads * 8;
                    q[d] = at < e0 + span ? *reinterpret_cast<const uint4*>(x + at) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int d = 0; d < kDeep; ++d) {
                    const int at = e + d * kThreads * 8;
                    const uint32_t w[4] = {q[d].x, q[d].y, q[d].z, q[d].w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t b = w[k / 2] >> (k & 1 ? 16 : 0);
                        if (((b ^ bits) & care) == 0 && at + k < e0 + span) {
                            const int slot = atomicAdd(&sh.count, 1);
                            if (slot < kList) sh.list[slot] = at + k;
                            atomicAdd(&sh.buckets[(at + k - e0) / per], 1);
                        }
                    }
                }
            }
            sync_warps();
            const int n = sh.count;
            if (n <= kList || per == 8) break;
            if (threadIdx.x == 0) {
                int b = 0;
                while (b + 1 < kBuckets && r >= sh.buckets[b]) r -= sh.buckets[b++];
                sh.segment = b;
                sh.draw.r = r;
            }
            sync_warps();
            e0 += sh.segment * per;
            span = min(per, e1 - e0);
            r = sh.draw.r;
            sync_warps();
        }
        const int n = min(sh.count, kList);
        for (int a = threadIdx.x; a < n; a += kThreads) {
            const int mine = sh.list[a];
            int before = 0;
            for (int b = 0; b < n; ++b) before += sh.list[b] < mine;
            if (before == r) P.tokens[i] = mine;
        }
        sync_warps();
    }
};

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

__global__ void __launch_bounds__(kThreads + 32, kPerSm) sample_kernel(const __grid_constant__ SampleParams P) {
    extern __shared__ __align__(128) unsigned char smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + kGap);
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
    if (tid < 64) sh.powers[tid >> 4][tid & 15] = c_powers.t[tid >> 4][tid & 15];
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
            }
            continue;
        }
        for (uint32_t at = tid * 16; at < (kValues + 1) * 4; at += kThreads * 16) {
            // the last piece may reach into the word behind, which is padding on both sides
            *reinterpret_cast<uint4*>(smem + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(smem + kNegative + at) = make_uint4(0, 0, 0, 0);
        }
        sync_warps();
        uint32_t top = 0xff80ff80u;
        for (int c = 0; c < chunks; ++c, ++n) {
            const uint32_t k = n % kStages;
            if (*(volatile int*)&sh.abort == 0 &&
                !mbar_wait_bounded(smem_addr(&sh.full[k]), n / kStages & 1, kWaitNs)) {
                set_error(P.err, DLLM_DEVERR_TIMEOUT);
                *(volatile int*)&sh.abort = 1;
            }
            const int left = e1 - (e0 + c * kChunk);
            const uint4* const in = reinterpret_cast<const uint4*>(smem + kRing + k * kChunk * 2);
            constexpr int kPieces = kChunk / 8 / kThreads;
            uint4 q[kPieces];
#pragma unroll
            for (int d = 0; d < kPieces; ++d) q[d] = in[d * kThreads + tid];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.empty[k]));
            if (left >= kChunk) {
#pragma unroll
                for (int d = 0; d < kPieces; ++d) {
                    count_word(q[d].x, base, top);
                    count_word(q[d].y, base, top);
                    count_word(q[d].z, base, top);
                    count_word(q[d].w, base, top);
                }
            } else {
#pragma unroll
                for (int d = 0; d < kPieces; ++d) {
                    const int have = left - (d * kThreads + tid) * 8;   // values of this piece
                    const uint32_t w[4] = {q[d].x, q[d].y, q[d].z, q[d].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (2 * j + 1 < have) count_word(w[j], base, top);
                        else if (2 * j < have) count_word((w[j] & 0xffffu) | 0xff800000u, base, top);   // counted as low
                    }
                }
            }
        }
        // what the slice holds besides the counted values
        float m = max_nan(bf16_lo(top), bf16_hi(top));
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane == 0) sh.part[warp] = m;
        if (tid == 0) sh.flag = 0;
        sync_warps();
        const uint32_t* const pos = reinterpret_cast<const uint32_t*>(smem);
        const uint32_t* const neg = reinterpret_cast<const uint32_t*>(smem + kNegative);
        const bool zeros = pos[0] + neg[0] > 0;
        if (zeros) {   // exact zeros, or small values that only the wide path tells apart
            bool small = false;
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
            f.low = (int)neg[kValues] - (e1 == P.V && e1 > e0 ? P.V & 1 : 0);   // the odd last value's partner
            sh.facts = f;
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
            for (int q = 0; q < ctas; ++q) {
                all.max = max_nan(all.max, __uint_as_float(peer_load(at, q)));
                all.other |= (int)peer_load(at + 4, q);
                all.low += (int)peer_load(at + 8, q);
            }
        }
        const float T = P.temperature ? __ldg(P.temperature + i) : 1.0f;
        const bool ok = isfinite(all.max) && T >= 0.0f;
        Row R{P, sh, smem, base, x, Weights{}, false};
        R.W.m32 = all.max;
        R.W.m = all.max;
        R.W.s = T > 0.0f ? 1.4426950408889634 / (double)T : 1.0;
        R.W.s32 = (float)fmin(R.W.s, 3e38);
        R.W.shift = P.shift;
        R.W.least = 0;
        if (P.min_p && T > 0.0f) {
            const float least = __ldg(P.min_p + i);
            if (least > 0.0f) R.W.least = (u64)ceil(fmin((double)least, 1.0) * 4611686018427387904.0);
        }
        // low values count where their weights do: -256 is the largest
        R.wide = all.other || (all.low > 0 && (-256.0f - all.max) * R.W.s32 > -80.0f);
        if (ok && !R.wide) {
            for (int s = rank * kWarps + warp; s < kSegments; s += ctas * kWarps) {
                const int o = s * 32 + lane;
                uint32_t c = R.count_of(o);
                u64 mass = 0;
                if (__any_sync(0xffffffffu, c > 0)) {
                    const u64 w = c ? R.W.of(__uint_as_float(R.bits_of(o) << 16), sh.powers) : 0;
                    if (w == 0) c = 0;
                    mass = warp_sum64(R.W.mass(c, w));
                    c = __reduce_add_sync(0xffffffffu, c);
                }
                if (lane == 0) {
                    if (ctas > 1) {
                        peer_store(smem_addr(&sh.seg_count[s]), 0, c);
                        peer_store64(smem_addr(&sh.seg_mass[s]), 0, mass);
                    } else {
                        sh.seg_count[s] = c;
                        sh.seg_mass[s] = mass;
                    }
                }
            }
        }
        if (ctas > 1) {
            meeting.arrive();
            meeting.wait(&sh.abort, P.err);
        } else {
            sync_warps();
        }
        if (rank == 0) {
            if (ok && !R.wide && warp == 0) R.choose(i, T);
            if (ok && R.wide) {
                R.sum_wide();
                R.choose(i, T);
            }
        }
        if (ctas > 1) {
            meeting.arrive();
            meeting.wait(&sh.abort, P.err);
        } else {
            sync_warps();
        }
        Draw d = sh.draw;
        int l0 = e0, l1 = e1;
        bool mine = ok && (rank == 0 || !R.wide);
        if (ctas > 1 && !(ok && R.wide)) {
            if (ok) {
                const uint32_t at = smem_addr(&sh.draw);
                d.bits = peer_load(at + offsetof(Draw, bits), 0);
                d.r = peer_load(at + offsetof(Draw, r), 0);
                const uint32_t c4 = (d.bits & 0x7fffu) == 0 ? 0 : ((d.bits & 0x7fffu) - kLow) * 4;
                for (int q = 0; q <= rank; ++q) {
                    uint32_t c = peer_load(base + (d.bits & 0x8000u ? kNegative : 0u) + c4, q);
                    if (c4 == 0) c += peer_load(base + kNegative, q);
                    if (q < rank) d.r -= c;
                    else mine = d.r >= 0 && d.r < (long long)c;
                }
            }
        } else if (ok && R.wide) {
            l0 = 0;
            l1 = P.V;
        }
        if (ctas > 1) meeting.arrive();   // this CTA has read the others' counters
        if (rank == 0 && tid == 0) {
            P.prob[i] = ok ? sh.draw.prob : __int_as_float(0x7fc00000);
            if (!ok) P.tokens[i] = -1;
        }
        if (mine) R.locate(i, d.bits, d.r, l0, l1);
        if (ctas > 1) meeting.wait(&sh.abort, P.err);
        else sync_warps();
    }
    // after a wait that gave up: copies still in flight land in this CTA's memory, not in its successor's
    if (*(volatile int*)&sh.abort) __nanosleep(1000000);
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" int dllm_sample(const dllm_sample_args* a, void* stream) {
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
    P.err = error_word_ptr();
    if (!P.err) return DLLM_ERR_CUDA;
    int c = 1;
    while (c < kMaxCluster && (long long)a->N * c < sms && a->V / (2 * c) >= kChunk) c *= 2;
    P.cluster = c;
    P.slice = ((a->V + c - 1) / c + 7) / 8 * 8;
    int bits = 0;   // V tokens of mass 2^(62 - shift) stay below 2^62
    while ((1ll << bits) <= a->V) ++bits;
    P.shift = std::max(16, bits);
    static SmemOnce done;
    DLLM_CUDA_TRY(allow_smem(sample_kernel, kSmem, done));
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
    DLLM_CUDA_TRY(cudaLaunchKernelEx(&cfg, sample_kernel, P));
    return DLLM_OK;
}
