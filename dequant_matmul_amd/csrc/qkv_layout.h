// qkv_layout.h -- where the paged cache keeps a value (the layout stated in
// include/qkv.h), shared by the kernels that write, read and attend to it.
//
// A tile is 64 tokens of one kv head: codes, then scales.  The codes stand in
// fragment order of v_mfma_f32_16x16x32_f16, so that a wave's 64 lanes load 64
// consecutive 16-byte (8-byte, 12-byte) pieces:
//   K, as operand A (rows = tokens, contraction = dims): row tile c of the four
//     takes tokens 16 q + 4 c + r, row m = 4 q + r.  The accumulator then holds,
//     in lane group h, tokens 16 h + 4 c + i: over the four row tiles each lane
//     owns 16 consecutive tokens of one query row, which is exactly operand B of
//     the second product.  No value moves between lanes from the scores to the
//     output.
//   V, as operand A (rows = dims, contraction = tokens): lane (m, h) holds dim
//     16 t + m of tokens 16 h + 8 s + j for contraction step s.
#pragma once

#include "qmm_device.h"

namespace qmm {

enum : int { KV_F16 = 0, KV_Q8 = 1, KV_Q4 = 2 };   // cache types as template arguments

constexpr int KV_TILE = 64;

template <int NB, int KT>
struct KvLay {
    static constexpr int DP = 32 * NB;                      // stored dims of a row
    static constexpr int CODE_BYTES = KT == KV_F16 ? KV_TILE * DP * 2 : KT == KV_Q8 ? KV_TILE * DP : KV_TILE * DP / 2;
    static constexpr int TILE_BYTES = CODE_BYTES + (KT == KV_F16 ? 0 : KV_TILE * NB * 2);
    // K: blocks of a lane's piece, bytes of one 8-dim unit
    static constexpr int G = KT == KV_F16 ? 1 : KT == KV_Q8 ? (NB % 2 == 0 ? 2 : 1) : (NB < 4 ? NB : 4);
    static constexpr int UNIT = KT == KV_F16 ? 16 : KT == KV_Q8 ? 8 : 4;
    static constexpr int ROW_BYTES = KT == KV_F16 ? 64 * NB : KT == KV_Q8 ? 34 * NB : 18 * NB;

    // byte offset of the 8 dims 32 b + 8 h .. of token key (0..63) of a K tile
    static __device__ __forceinline__ int k_unit(int key, int b, int h)
    {
        const int c = (key >> 2) & 3, lane = h * 16 + (key >> 4) * 4 + (key & 3);
        return (((c * (NB / G) + b / G) * 64 + lane) * G + b % G) * UNIT;
    }
    static __device__ __forceinline__ int k_scale(int key, int b) { return CODE_BYTES + (key * NB + b) * 2; }
    // byte offset of dim 16 t + m of token key of a V tile (Q4: the byte that
    // also holds dim 16 (t ^ 1) + m)
    static __device__ __forceinline__ int v_code(int key, int t, int m)
    {
        const int lane = (key >> 4) * 16 + m, i = key & 15;
        if constexpr (KT == KV_F16)
            return (((t * 2 + (i >> 3)) * 64 + lane) * 8 + (i & 7)) * 2;
        else if constexpr (KT == KV_Q8)
            return (t * 64 + lane) * 16 + i;
        else
            return ((t >> 1) * 64 + lane) * 16 + i;
    }
    static __device__ __forceinline__ int v_scale(int key, int b) { return CODE_BYTES + (b * KV_TILE + key) * 2; }
};

// One of the two buffers of a cache as the kernels take it.
struct KvView {
    uint8_t *k, *v;
    int64_t pages;
    int32_t kv_heads, head_dim, page_shift, nb;
};

// First byte of the tile of head `head` holding offset `off` of page `page`.
template <class L>
__device__ __forceinline__ int64_t tile_at(const KvView &c, int64_t page, int head, int off)
{
    return (((page * c.kv_heads + head) << (c.page_shift - 6)) + (off >> 6)) * (int64_t)L::TILE_BYTES;
}

// Whether a slot lies in the cache; its tile and its place in the tile.
template <class L>
__device__ __forceinline__ bool slot_at(const KvView &c, int32_t slot, int head, int64_t &tile, int &key)
{
    const int64_t page = (int64_t)slot >> c.page_shift;
    if (slot < 0 || page >= c.pages)
        return false;
    const int off = slot & ((1 << c.page_shift) - 1);
    tile = tile_at<L>(c, page, head, off);
    key = off & (KV_TILE - 1);
    return true;
}

}  // namespace qmm
