// Shared by the kernels of dllm_kv4_attend: its parameters, the softmax's
// constants and packing.
#pragma once

#include "kv4_mma.cuh"

namespace dllm {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kBelow = 7.0f;    // the offset sits this far below the maximum it was set from
constexpr float kAbove = 15.0f;   // and moves when a score passes it by more than this

constexpr int kTileTokens = 128;   // tokens of a tile of the many-row kernels
constexpr int kTileRows = 256;     // query rows of one of their items, at most
constexpr int kMaxCtas = 160;      // one per SM

// A run of tiles of one (request, key/value head, block of rows).
struct alignas(16) TileItem {
    int b, head, rb;
    int t0, t1;    // tiles; both 0: a request without tokens
    int slot;      // where its partial result goes, -1: it is whole
    int n;         // the request's tokens
    int pad;
};
// The partial results to join.
struct alignas(16) TileSplit {
    int b, head, rb, slot0, pieces;
    int pad[3];
};
struct TilePlan {
    int items, splits;
    int pad[62];
    TileSplit split[kMaxCtas];
};

struct AttendParams {
    Kv4 C;
    QueryRows Q;
    int q_heads;
    float scale2;                 // scale * log2 e
    const int* lens;
    uint16_t* out;
    float* lse;
    const float* prior;
    float* weights;
    // few rows
    int tiles, splits;            // 16-row tiles per key/value head; splits of a unit's tokens
    int* counters;                // zero between calls
    float* partial;               // few rows: [unit][split][16 (D + 2)]; many: [slot][kTileRows (D + 2)]
    // many rows
    int row_blocks, block_rows;   // blocks of rows per key/value head, rows of each (the last may have fewer)
    int ctas;
    TilePlan* plan;
    TileItem* items;

    // (request, position, head) of row r, in the order of out and lse
    __device__ __forceinline__ long long row_at(int b, int head, int r) const {
        const int i = r / Q.group;
        return ((long long)b * Q.L + i) * q_heads + head * Q.group + (r - i * Q.group);
    }
};

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// kv4_tile.cu: the attention of many rows (plan, tiles, join).  P.row_blocks,
// block_rows, ctas, plan, items and partial are set.
int launch_attend_tiles(const AttendParams& P, int D, cudaStream_t stream);
// The tokens' weights of many rows, after launch_attend_tiles on the same P.
int launch_weight_tiles(const AttendParams& P, int D, cudaStream_t stream);

}  // namespace dllm
