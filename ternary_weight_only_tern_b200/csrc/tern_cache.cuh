// The 4-bit KV cache's places and host checks, shared by append, read and attention.
#pragma once

#include "tern_nib.cuh"

namespace tern {
namespace kv {

using namespace nib;

constexpr int kTok = 16;                   // tokens per block
constexpr int kGrp = 64;                   // entries of a head that share a step and a zero

constexpr int unit_bytes(int D) { return 18 * D; }
constexpr int v_codes(int D) { return 8 * D; }      // byte offsets within a block
constexpr int k_scales(int D) { return 16 * D; }
constexpr int v_scales(int D) { return 17 * D; }

// The pool and the tables that say where a sequence's tokens lie.
struct Pool {
    uint8_t* pool;
    int64_t pages;
    const int32_t* table;
    int64_t width;
    int per_page;       // blocks per page
    int heads;

    // Place in the pool of block `blk` (tokens 16 blk ..) of sequence b and kv head h, counted in blocks, or -1 where there
    // is no page (check_cache keeps the count below 2^31).
    __device__ __forceinline__ int place(int64_t b, int h, int64_t blk) const {
        const int64_t col = blk < 0x7fffffff ? int64_t(uint32_t(blk) / uint32_t(per_page)) : blk / per_page;
        if (blk < 0 || col >= width) return -1;
        const int page = __ldg(table + b * width + col);
        if (page < 0 || page >= pages) return -1;
        return (page * heads + h) * per_page + int(blk - col * per_page);
    }

    template <int D>
    __device__ __forceinline__ uint8_t* block(int64_t b, int h, int64_t blk) const {
        const int at = place(b, h, blk);
        return at < 0 ? nullptr : pool + int64_t(at) * unit_bytes(D);
    }
};

inline tern_status check_cache(const tern_cache* c) {
    if (!c) return TERN_ERR_NULL;
    if (c->pages <= 0 || c->pages > 0x7fffffff || c->page <= 0 || c->page % kTok || c->page > 65536 ||
        c->kv_heads <= 0 || c->kv_heads > 65535 || (c->head_dim != 64 && c->head_dim != 128))
        return TERN_ERR_SHAPE;
    if (c->pages > 0x7fffffff / (int64_t(c->kv_heads) * (c->page / kTok))) return TERN_ERR_SHAPE;   // blocks are counted in int32
    if (!c->pool) return TERN_ERR_NULL;
    return aligned16(c->pool) ? TERN_OK : TERN_ERR_ALIGN;
}

// Limits of a call's batch: every product of the sizes stays well inside 63 bits.
inline bool batch_ok(int64_t B, int64_t T, int64_t width) {
    return B >= 0 && B <= 65535 && T >= 0 && T <= (int64_t(1) << 24) && width >= 0 && width <= (int64_t(1) << 24);
}

inline Pool pool_of(const tern_cache* c, const int32_t* table, int64_t width) {
    return Pool{c->pool, c->pages, table, width, c->page / kTok, c->kv_heads};
}

}  // namespace kv
}  // namespace tern
