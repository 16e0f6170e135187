// attention.cuh -- what the attention kernels share: the split of a batch's
// work over the CTAs, the partial results of work that was cut, and the
// masks.
//
// Work.  An item is (sequence, row tile, key/value head): the rows are the
// sequence's new tokens times the query heads that share the key/value head
// (row r: token r / group, query head head * group + r % group), in the
// form's row tiles; its keys come in the form's key tiles.  Items lie on a
// line in order, each with as many places as it may be cut into, and every
// CTA takes the same number of places:
//
//   cut = 0          a place is a key tile: every CTA gets the same number of
//                    tiles, whatever the lengths, and may cut two items
//   cut = L          an item is L tiles at most a place, and there are no
//                    more places than CTAs: a CTA has one part of one item
//   cut = kWhole     items are not cut (short contexts), or by a cluster of
//                    CTAs that join their parts themselves
//
// An item that is cut is joined afterwards: a CTA leaves at most two partial
// results, slot 2 g for a part that does not begin its item, 2 g + 1 for one
// that does, and the CTA with the item's last part says where the item's
// others are (CutItem).  Lengths live on the device, so the split is worked
// out there, by every CTA from the same numbers.
#pragma once

#include <cuda.h>

#include "cache.cuh"

namespace iq4xs {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kWhole = INT32_MAX;
constexpr int kMaxCluster = 8;

struct AttnParams {
    const uint16_t* q;
    float* out;
    const uint64_t* mask;
    struct CutItem* cuts;  // [G]
    float* part_o;     // [2 G slots][slot_rows][D]
    float2* part_ml;   // [2 G slots][slot_rows] {max (log2 units), sum}
    int64_t q_row_stride, out_row_stride, rows;
    int64_t layer_offset;  // elements of K and V
    float scale_log2;  // |scale| log2(e): scores are kept in log2 units
    uint32_t q_and, q_xor;  // the scale's sign (or zero), put on q: scores may be masked with -inf before scaling
    int group, kv_heads, mask_words, head_dim;
    uint64_t group_magic;  // ceil(2^38 / group): row / group by one multiplication
    int wide_out;      // out and its rows are 32-byte aligned
    int ctas;          // CTAs the work is split over, at most
    int whole_items;   // 1: cut = kWhole
    int cluster;       // CTAs that share an item, meeting in shared memory (1: none); then p.ctas counts clusters
    int part_tiles;    // what starting and ending a part costs, in key tiles
    int slot_rows;     // rows of a partial result: the row tile, or all rows if fewer
    int box_slots, box_chunks;  // of a copy: slots of a page, 64-channel chunks
    int skip_stage;    // test hook: this stage of every CTA is left unissued
};

// Row r's token and query head of the group (r < 2^25, group <= 2^10: the
// magic's excess, below 2^10 / 2^38 of a row, never reaches the next token).
__device__ __forceinline__ int token_of(const AttnParams& p, int r) {
    return (int)(((uint64_t)(uint32_t)r * p.group_magic) >> 38);
}

// One sequence as the split sees it.
struct SeqWork {
    int row0, tokens, len, row_tiles, key_tiles;
    __device__ __forceinline__ int unit(int cut) const {  // places of an item
        return cut == 0 ? key_tiles : cut == kWhole ? 1 : (key_tiles + cut - 1) / cut;
    }
    __device__ __forceinline__ int64_t items(const AttnParams& p) const {
        return tokens > 0 ? (int64_t)row_tiles * p.kv_heads : 0;
    }
    __device__ __forceinline__ int64_t places(const AttnParams& p, int cut) const { return items(p) * unit(cut); }
};

// F: kRows and kKeys of the form's tiles.  From the sequence's row offsets
// and length as they were read.
template <class F>
__device__ __forceinline__ SeqWork seq_of(const AttnParams& p, int first, int last, int len, int* err) {
    SeqWork w;
    w.row0 = first;
    w.tokens = last - first;
    w.len = len;
    if (first < 0 || last < first || last > p.rows) {
        data_error(err, kDataOffsets);
        w.tokens = 0;
    }
    if (len < 0 || len > (INT32_MAX >> 1)) {
        data_error(err, kDataLens);
        w.tokens = w.len = 0;
    }
    w.row_tiles = (w.tokens * p.group + F::kRows - 1) / F::kRows;
    w.key_tiles = (w.len + w.tokens + F::kKeys - 1) / F::kKeys;
    return w;
}
// Sequence s (none behind the last: no tokens).
template <class F>
__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, const BatchView& b, int s, int* err) {
    if (s < b.sequences) return seq_of<F>(p, b.row_offsets[s], b.row_offsets[s + 1], b.lens[s], err);
    return seq_of<F>(p, 0, 0, 0, err);
}
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
    if (__all_sync(0xffffffffu, v < (int64_t(1) << 26)))  // (one instruction where 32 of them fit 31 bits)
        return (int64_t)__reduce_add_sync(0xffffffffu, (unsigned)v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// a / b, both mostly of 32 bits (a 64-bit division costs ten times one of 32).
__device__ __forceinline__ int64_t div_long(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ int64_t div_small(int64_t a, int b) { return div_long(a, b); }

// The split: `cut` as above, W places over `ctas` CTAs (no more than places,
// so that none is empty): each W / ctas of them, the first `more` one more.
struct Split {
    int64_t each, more;
    int cut, ctas;
    __device__ __forceinline__ int64_t start(int g) const { return each * g + min((int64_t)g, more); }
    __device__ __forceinline__ int owner(int64_t x) const {
        const int64_t in_more = more * (each + 1);
        return (int)(x < in_more ? div_long(x, each + 1) : more + div_long(x - in_more, each));
    }
    // By a whole warp, 32 sequences a step, one a lane (`mine`: the lane's
    // among the first 32, read by the caller).
    template <class F>
    __device__ __forceinline__ void plan(const AttnParams& p, const BatchView& b, const SeqWork& mine, int* err) {
        const int lane = threadIdx.x & 31;
        int64_t tiles = mine.places(p, 0), items = mine.items(p);
        for (int s0 = 32; s0 < b.sequences; s0 += 32) {
            const SeqWork w = seq_work<F>(p, b, s0 + lane, err);
            tiles += w.places(p, 0);
            items += w.items(p);
        }
        tiles = warp_sum(tiles);
        items = warp_sum(items);
        cut = p.whole_items ? kWhole : 0;
        int64_t places = p.whole_items ? items : tiles;
        // Parts of one item each, if the longest is not behind an even share
        // by more than the second part costs that a CTA has without them.
        if (!p.whole_items && items <= p.ctas && items > 0) {
            const int share = (int)div_small(tiles + p.ctas - 1, p.ctas);
            const int step = max(1, p.part_tiles / 4);
            for (int len = share; len <= share + p.part_tiles; len += step) {
                int64_t n = mine.places(p, len);
                for (int s0 = 32; s0 < b.sequences; s0 += 32)
                    n += seq_work<F>(p, b, s0 + lane, err).places(p, len);
                n = warp_sum(n);
                if (n <= p.ctas) {
                    cut = len;
                    places = n;
                    break;
                }
            }
        }
        ctas = (int)min((int64_t)p.ctas, places);
        each = ctas > 0 ? div_small(places, ctas) : 0;
        more = places - each * ctas;
    }
};

// The cut item whose last part is CTA g's (entry g): its first part's CTA and
// its rows.  first < 0: CTA g ends none.
struct CutItem {
    int first, rows, row0, head, first_row;
    int pad[3];
};

// A CTA's walk over its range, item by item.
template <class F>
struct WorkWalk {
    Split split;
    int64_t left;        // places of the range from the current part on
    SeqWork w;
    int s;
    int row_end, next_end, next_len;  // offsets and length behind the sequence, read ahead
    // the current item's part
    int head, row_tile, tile0, tile1;
    bool whole;          // this CTA has all of the item's key tiles
    int slot;            // of its partial result, if not
    static constexpr int kRows = F::kRows;

    __device__ __forceinline__ void start(const AttnParams& p, const BatchView& b, int g, int* err) {
        const int lane = threadIdx.x & 31;
        const SeqWork mine = seq_work<F>(p, b, lane, err);
        split.plan<F>(p, b, mine, err);
        left = 0;
        if (g >= split.ctas) return;
        const int64_t x = split.start(g);
        left = split.start(g + 1) - x;
        // the sequence that holds x: the first whose end lies behind it
        int64_t before = 0, seq_x = 0;
        s = 0;
        for (int s0 = 0; s0 < b.sequences; s0 += 32) {
            int64_t sums = (s0 == 0 ? mine : seq_work<F>(p, b, s0 + lane, err)).places(p, split.cut);
            if (__all_sync(0xffffffffu, sums < (int64_t(1) << 26))) {
                int v = (int)sums;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += y;
                }
                sums = v;
            } else {
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, sums, o);
                    if (lane >= o) sums += y;
                }
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + sums > x);
            if (past != 0) {
                const int k = __ffs(past) - 1;
                const int64_t up = __shfl_sync(0xffffffffu, sums, k > 0 ? k - 1 : 0);
                s = s0 + k;
                seq_x = before + (k > 0 ? up : 0);
                break;
            }
            before += __shfl_sync(0xffffffffu, sums, 31);
        }
        if (s < 32) {  // (one of those that the lanes hold)
            const int first = __shfl_sync(0xffffffffu, mine.row0, s), n = __shfl_sync(0xffffffffu, mine.tokens, s);
            w = seq_of<F>(p, first, first + n, __shfl_sync(0xffffffffu, mine.len, s), err);
            row_end = first + n;
        } else {
            row_end = b.row_offsets[s + 1];
            w = seq_of<F>(p, b.row_offsets[s], row_end, b.lens[s], err);
        }
        read_ahead(b);
        const int unit = w.unit(split.cut);
        const int item = (int)div_small(x - seq_x, unit);
        head = item / w.row_tiles;
        row_tile = item - head * w.row_tiles;
        set((int)(x - seq_x - (int64_t)item * unit), unit, g);
    }
    __device__ __forceinline__ void read_ahead(const BatchView& b) {
        if (s + 1 < b.sequences) {
            next_end = b.row_offsets[s + 2];
            next_len = b.lens[s + 1];
        }
    }
    // Entry g of the cut items, before the first next().
    __device__ __forceinline__ void tell_cut(const AttnParams& p, int g) const {
        CutItem t = {};
        t.first = -1;
        if (valid() && tile0 > 0 && tile1 == w.key_tiles) {
            t.first = split.cut == 0 ? split.owner(split.start(g) - tile0) : g - (w.unit(split.cut) - 1);
            t.rows = min(F::kRows, w.tokens * p.group - row_tile * F::kRows);
            t.row0 = w.row0;
            t.head = head;
            t.first_row = row_tile * F::kRows;
        }
        p.cuts[g] = t;
    }
    // The part that begins at the item's place `at` of `unit`.
    __device__ __forceinline__ void set(int at, int unit, int g) {
        if (split.cut == 0) {
            tile0 = at;
            tile1 = (int)min((int64_t)w.key_tiles, at + left);
        } else {
            tile0 = (int)div_small((int64_t)at * w.key_tiles, unit);
            tile1 = (int)div_small((int64_t)(at + 1) * w.key_tiles, unit);
        }
        whole = tile0 == 0 && tile1 == w.key_tiles;
        slot = 2 * g + (tile0 == 0 ? 1 : 0);
    }
    __device__ __forceinline__ bool valid() const { return left > 0; }
    __device__ __forceinline__ bool last() const { return left <= (split.cut == 0 ? tile1 - tile0 : 1); }
    __device__ __forceinline__ void next(const AttnParams& p, const BatchView& b, int g, int* err) {
        left -= split.cut == 0 ? tile1 - tile0 : 1;
        if (left <= 0) return;
        if (++row_tile == w.row_tiles) {
            row_tile = 0;
            if (++head == p.kv_heads) {
                head = 0;
                do {  // (sequences without work are passed over)
                    ++s;
                    w = seq_of<F>(p, row_end, next_end, next_len, err);
                    row_end = next_end;
                    read_ahead(b);
                } while (w.tokens == 0);
            }
        }
        set(0, split.cut == 0 ? w.key_tiles : 1, g);
    }
    // Key tiles that a row of this item can see: without a mask (a chain) the
    // row tile's last token ends them.
    __device__ __forceinline__ int seen_tiles(const AttnParams& p) const {
        int keys = w.len + w.tokens;
        if (p.mask == nullptr) {
            const int last = min(w.tokens - 1, token_of(p, (row_tile + 1) * F::kRows - 1));
            keys = w.len + last + 1;
        }
        return min(tile1, (keys + F::kKeys - 1) / F::kKeys);
    }
};

// Whether token t (row `row` of the batch) sees its sequence's new token j >= 0.
__device__ __forceinline__ bool sees_new(const AttnParams& p, int row, int t, int j, const Bc& bc) {
    if (p.mask == nullptr) return j <= t;
    const int word = j >> 6;
    const uint64_t* m = p.mask + (int64_t)row * p.mask_words + word;
    return word < p.mask_words && bc_global(bc, m, 8, p.mask, 8 * p.rows * p.mask_words, kBcAttnMask) &&
           (*m >> (j & 63) & 1) != 0;
}

// Row r of a cut item's slot in the workspace: its {max, sum} and, at a
// channel, its unjoined outputs; nullptr if the bounds-checked build finds
// them outside (n channels).
__device__ __forceinline__ float2* part_sum(const AttnParams& p, int64_t slot, int r, const Bc& bc) {
    float2* at = p.part_ml + slot * p.slot_rows + r;
    return bc_global(bc, at, 8, p.part_ml, 16 * (int64_t)p.ctas * p.slot_rows, kBcAttnWork) ? at : nullptr;
}
__device__ __forceinline__ float* part_row(const AttnParams& p, int64_t slot, int r, int channel, int n, const Bc& bc) {
    float* at = p.part_o + (slot * p.slot_rows + r) * p.head_dim + channel;
    return bc_global(bc, at, 4 * n, p.part_o, 8 * (int64_t)p.ctas * p.slot_rows * p.head_dim, kBcAttnWork) ? at : nullptr;
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
// A row's view of its sequence's new tokens: the mask's first word, read when
// the row's item starts, and the row, for masks of more words.
struct RowSight {
    uint64_t word;
    int row, token;
    __device__ __forceinline__ void open(const AttnParams& p, int row0, int t, const Bc& bc) {
        row = row0 + t;
        token = t;
        word = 0;
        if (p.mask == nullptr) return;
        const uint64_t* m = p.mask + (int64_t)row * p.mask_words;
        if (!bc_global(bc, m, 8 * (int64_t)p.mask_words, p.mask, 8 * p.rows * p.mask_words, kBcAttnMask)) row = 0;
        else word = *m;
    }
    // Bit k: the row sees the position k behind one whose place among the new
    // tokens is j0 (negative: context); `have` positions lie before the end.
    __device__ __forceinline__ uint32_t bits(const AttnParams& p, int j0, int have) const {
        uint32_t fresh;
        if (p.mask == nullptr) {
            fresh = low_bits(token - j0 + 1);
        } else {
            const int lo = max(j0, 0), at = lo >> 6, sh = lo & 63;
            const uint64_t* m = p.mask + (int64_t)row * p.mask_words;
            uint64_t v = 0;
            if (at < p.mask_words) v = (at == 0 ? word : m[at]) >> sh;
            if (sh > 32 && at + 1 < p.mask_words) v |= m[at + 1] << (64 - sh);
            fresh = lo - j0 >= 32 ? 0u : (uint32_t)v << (lo - j0);
        }
        return (low_bits(-j0) | fresh) & low_bits(have);
    }
};

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Softmax weights are exp2(score - m + kWeightBits) with m the running
// maximum, or up to kLazy below it: O and the sum are rescaled only when a
// maximum rises by more than kLazy.  kWeightBits uses fp16's range: weights
// go up to 2^(6 + 8), and the largest of a row is 2^6 at least.
constexpr float kWeightBits = 6.0f;
constexpr float kLazy = 8.0f;

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t x, y, z;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(y), "l"(z));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t x, y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ float2 mask2(float2 a, uint32_t mask) {
    return make_float2(__uint_as_float(__float_as_uint(a.x) & mask), __uint_as_float(__float_as_uint(a.y) & mask));
}
// Two weights as the sum of kN packed 16-bit parts, largest first; the last
// one is kept times 2^kLastShift, and so is what it makes of V until it meets
// the others.  fp16: 11 bits cut off, down to the subnormals' 2^-24, and what
// is left of the stored value (exact in fp32) times 2^12: 22 bits of every
// weight from 2^-14 on and 2^-36 of smaller ones, 2^-42 of the row's largest.
// (Without the factor what is left of a weight below 2^-14 falls under half of
// 2^-24 and is lost: beside one key that outweighs the others by 2^20 the
// result was off by 2e-5, by 2^24 by 7e-4.)  bf16: 8 + 8 + 8 bits cut off, the
// whole value.  No part is negative: an infinity among the V that a row sees
// times a negative part would meet itself with the other sign.
template <class T>
struct Parts;
template <>
struct Parts<KvF16> {
    static constexpr int kN = 2, kLastShift = 12;
    static __device__ __forceinline__ void split(float2 a, uint32_t* out) {
        constexpr float kUp = 1 << kLastShift;
        out[0] = KvF16::pack_rz(a.x, a.y);
        const float2 r = fma2(KvF16::unpack(out[0]), make_float2(-1.f, -1.f), a);
        out[1] = KvF16::pack(r.x * kUp, r.y * kUp);
    }
};
template <>
struct Parts<KvBf16> {
    static constexpr int kN = 3, kLastShift = 0;
    static __device__ __forceinline__ void split(float2 a, uint32_t* out) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            out[i] = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x7632u);
            if (i < 2) a = fma2(mask2(a, 0xffff0000u), make_float2(-1.f, -1.f), a);
        }
    }
};

// Eight values of q, with the scale's sign.
__device__ __forceinline__ uint4 sign_q(const AttnParams& p, uint4 v) {
    return make_uint4((v.x & p.q_and) ^ p.q_xor, (v.y & p.q_and) ^ p.q_xor, (v.z & p.q_and) ^ p.q_xor,
                      (v.w & p.q_and) ^ p.q_xor);
}

// Tiles of 16-bit rows in shared memory: [64-channel chunk][row][128 bytes],
// 16-byte units swizzled within each 8-row atom as TMA's 128-byte swizzle
// does.  Offset of unit u (8 channels) of row r.
constexpr int kChunkBytes = 128;
__device__ __forceinline__ uint32_t unit_at(int r, int u, int rows) {
    return (uint32_t)((u >> 3) * rows * kChunkBytes + r * kChunkBytes + (((u & 7) ^ (r & 7)) << 4));
}
// Shared-memory matrix descriptor, 128-byte swizzle.  K-major: sbo between
// 8-row groups.  MN-major: lbo between 64-element chunks of the M/N axis, sbo
// between 8-row groups of the K axis.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor, kind::f16, D fp32, M = 128; type 0 fp16, 1 bf16;
// b_mn: B is N-major.
constexpr uint32_t idesc_kv(int n, uint32_t type, bool b_mn) {
    return (1u << 4) | (type << 7) | (type << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           (8u << 24);
}
// A box of K or V: from (chunk, slot) of a page and head on.
__device__ __forceinline__ void tma_load_kv(uint32_t dst, const void* map, int slot, int chunk, int head, int page,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(0), "r"(slot), "r"(chunk), "r"(head), "r"(page), "r"(smem_u32(bar))
        : "memory");
}
// mbar_wait whose first probe does not suspend (most phases are complete when
// they are asked for).
__device__ __forceinline__ bool kv_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0 || mbar_wait(bar, parity, abort_flag, err, code);
}
// kv_wait by a whole warp, with one answer for all of its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err,
                                          int code) {
    return __all_sync(0xffffffffu, kv_wait(bar, parity, abort_flag, err, code)) != 0;
}

// Page ids of 32 pages of a sequence, one a lane, and the 32 behind them on their way.
struct PageWindow {
    const int32_t* table;
    int held, first, ids, ids2;
    __device__ __forceinline__ int read(int page) const { return page < held ? table[page] : -1; }
    __device__ __forceinline__ void open(const BatchView& b, int s) {
        table = b.page_table + s * b.table_stride;
        held = min(b.held[s], b.table_width);
        first = -64;
        ids2 = -1;
    }
    // Brings the window over `page`, a tile's first; by a whole warp.
    __device__ __forceinline__ void move(int page, int lane) {
        if (page >= first && page < first + 32) return;
        ids = page == first + 32 ? ids2 : read(page + lane);
        first = page;
        ids2 = read(page + 32 + lane);
    }
    __device__ __forceinline__ int id(int page) const { return __shfl_sync(0xffffffffu, ids, (page - first) & 31); }
};

// The forms' tiles: row tiles of 8 or 16 on the warp-level form, of 128 on
// tcgen05; there 128 keys a tile where two tiles of K, of V and of scores fit
// the SM, 64 at 256 channels.
template <int NT>
struct MmaForm {
    static constexpr int kRows = 8 * NT, kKeys = 64;
};
template <int D>
struct TcForm {
    static constexpr int kRows = 128, kKeys = D == 256 ? 64 : 128;
};

// Launchers of the two forms (csrc/attention_mma.cu, csrc/attention_tc.cu).
cudaError_t launch_attention_mma(int row_tile, const AttnParams& p, const void* tk, const void* tv, const CacheView& c,
                                 const BatchView& b, bool bf16, int* err, cudaStream_t stream);
cudaError_t launch_attention_tc(const AttnParams& p, const void* tk, const void* tv, const CacheView& c,
                                const BatchView& b, bool bf16, int* err, cudaStream_t stream);

}  // namespace iq4xs
