// attention_tc.cu -- tree attention for many rows a key/value head (drafted
// trees, prompt chunks): tcgen05 on tiles of 128 rows x 128 keys (64 at 256 channels).
//
// One pass, as in the warp-level form; here a row is a lane of tensor memory:
//
//   S = Q K^T      Q from tensor memory (shared where that is full), K from shared
//   P = exp2(S - m) split into 16-bit parts, back into tensor memory over S
//   T = P V        P from tensor memory, V from shared memory (as it
//                  lies: channels contiguous)
//   O = O f + T    in fp32 registers of the threads that own the row
//
// T starts from zero for every key tile and is added to O by rounded fp32
// arithmetic: the tensor core cuts its sums off, and thousands of tiles on
// one accumulator would add those cuts up.
//
// Roles: two producer warps, one thread that issues the MMAs, and eight
// softmax warps, two per 32-lane quadrant, each with half of a tile's keys and
// of O's channels; they share a row's maximum through shared memory.  The MMAs of tile j + 1's scores are issued
// before tile j's output product, so the tensor core works while the softmax
// runs.  K and V tiles go through one ring in the order the MMAs take them,
// K0 K1 V0 K2 V1 ... V(n-1), K by one warp and V by another (TMA).
//
// Up to about 48 rows HBM bounds it (4 D bytes a key), above that the tensor
// core (1 + parts products of 128 x tile x D) and the softmax.
//
// Measured: a tree of 64 tokens over 131,071, 24 heads over 4 of 256, fp16:
// 238 us a call in a hundred from idle, 257-268 in long runs, where the power
// cap lowers the clock (206 GFLOP counting the output product once, 0.8-0.87
// PFLOP/s); prompt chunks of 2 x 512 over 8,000, 32 heads over 8 of 128, bf16:
// 182 us.  The tensor pipe is 60 % and 52 % busy; a 64-key tile of the former
// takes about 2,100 cycles of the softmax warps (scores and maximum 250, the
// exchange 200, weights 600: exponentials at 16 a cycle and SM and the parts'
// shuffles; O 600, where tensor memory is read at about 220 bytes a cycle), 1,536 of them
// under products.  Measured as well: 16 softmax warps, no faster (tree 250,
// chunk 188 us, 20 rows over 20k 61 against 54); T over four tiles before O
// takes it, 224 against 230 us for the tree, 134 against 122 for 64 rows over
// 9k in bf16; O's reads of 32 channels at a time spill (245 us).
#include "attention.cuh"

namespace iq4xs {
namespace {

constexpr int kRowTile = TcForm<64>::kRows;
constexpr int kShares = 2;     // softmax warps of a quadrant: each has that part of the keys and of the channels
constexpr int kSoftWarps = 4 * kShares;
constexpr int kFirstSoft = 4;  // warps 4-11: two whole warpgroups
constexpr int kThreads = 32 * (kFirstSoft + kSoftWarps);
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kTmemCols = 512;
constexpr int kItems = 4;     // item descriptors in flight
constexpr int kAccCols = 16;  // channels of T read at a time

// One item's part as the producer hands it to the other warps.
struct Item {
    int row0, tokens, len;  // the sequence's first row, new tokens and length
    int seq, head, first;   // first: the row tile's first row (token and query head of the group)
    int tile0, n, turn;     // key tiles tile0 .. + n - 1, starting at tile0 + turn; n < 0: no more items
    int tile1;              // end of the part (rows may see fewer tiles)
    int slot;               // of the partial result; -1: the item is whole
    int pad;
    __device__ __forceinline__ int tile(int j) const { return tile0 + (j + turn >= n ? j + turn - n : j + turn); }
};
static_assert(sizeof(Item) % 16 == 0, "descriptors stay aligned");

template <int D, class T>
struct TcAttn {
    static constexpr int kTile = TcForm<D>::kKeys;           // keys a tile
    static constexpr int kParts = Parts<T>::kN;
    static constexpr int kChunks = D / 64;
    static constexpr int kChunkStride = kTile * kChunkBytes;
    static constexpr int kTileBytes = kTile * D * 2;
    // Tensor memory: T (two of them where 512 columns hold them); Q in 16-bit
    // pairs, if they hold it; two score buffers: S, overlaid in place by P:
    // the first two parts of 16 keys take the keys' own 16 columns, a third 8
    // more behind S.
    static constexpr int kScoreCols = kParts == 3 ? kTile * 3 / 2 : kTile;
    static constexpr int kTBufs = 2 * D + 2 * kScoreCols <= kTmemCols ? 2 : 1;
    static constexpr bool kQInTmem = kTBufs * D + D / 2 + 2 * kScoreCols <= kTmemCols;
    static constexpr int kQCol = kTBufs * D;
    static constexpr int kScores = kQCol + (kQInTmem ? D / 2 : 0);
    static_assert(kScores + 2 * kScoreCols <= kTmemCols, "tensor memory");
    // shared memory
    static constexpr int kQBytes = kQInTmem ? 0 : kRowTile * D * 2;
    static constexpr int kStageCols = kQInTmem ? 16 : 8;     // channels of a row on its way out, and their pitch
    static constexpr int kStageRow = kStageCols + 4;
    static constexpr int kStageBytes = kSoftThreads * kStageRow * 4;
    static constexpr int kSlots = (224 * 1024 - kQBytes - kStageBytes) / kTileBytes;
    static constexpr int kQ = kSlots * kTileBytes;
    static constexpr int kOut = kQ + kQBytes;                // rows on their way out (and Q's into tensor memory)
    static constexpr int kMax = kOut + kStageBytes;          // [2][shares][128] row maxima of a tile
    static constexpr int kEnd = kMax + 2 * kShares * kRowTile * 4;  // [1 + shares][128] an item's maxima and sums
    static constexpr int kDesc = kEnd + (1 + kShares) * kRowTile * 4;
    static constexpr int kBars = kDesc + kItems * (int)sizeof(Item);
    static constexpr int kNumBars = 2 * kSlots + 2 * kItems + 2 + 2 + 2 + 2 + 1 + 1;
    static constexpr int kMisc = kBars + kNumBars * 8;       // tensor memory address, abort, odd values
    static constexpr int kLast = kMisc + 16;                 // the last place loaded into each slot
    static constexpr int kSmem = kLast + kSlots * 4;
    static_assert(kSlots >= 4, "K and V of two tiles");
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static constexpr int kShareD = D / kShares;
    static constexpr int kHold = D == 256 ? 16 : 32;                         // scores a thread holds at a time
    static constexpr int kStep = 16;                         // and weights
    // Column of a part of the weights of keys 16 key16 .. + 15, from the buffer's first.
    static __device__ __forceinline__ uint32_t p_col(int key16, int part) {
        return part < 2 ? 16 * key16 + 8 * part : kTile + 8 * key16;
    }
};
// The softmax warps keep up to 128 output channels a thread: the producers' and
// the issuer's warpgroup gives up registers (80 + 2 * 208 <= 3 * 168, the launch's).
constexpr int kSoftRegs = 208, kOtherRegs = 80;
static_assert(kOtherRegs + kShares * kSoftRegs <= (1 + kShares) * 168, "register split within the launch's");

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
           ((uint32_t)(kRowTile >> 4) << 24);
}
__device__ __forceinline__ void quad_sync(int quadrant) {
    asm volatile("bar.sync %0, %1;" ::"r"(quadrant + 1), "n"(32 * kShares) : "memory");
}
__device__ __forceinline__ void soft_sync() {
    asm volatile("bar.sync 5, %0;" ::"n"(kSoftThreads) : "memory");
}
// Whether x holds for any softmax thread: one answer for all of them.
__device__ __forceinline__ bool soft_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 5, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(kSoftThreads)
        : "memory");
    return r != 0;
}
// NaN or infinities among two 16-bit values (exponent bits all set).
template <class T>
__device__ __forceinline__ bool any_odd(uint32_t w) {
    constexpr uint32_t kExp = Parts<T>::kN == 3 ? 0x7f807f80u : 0x7c007c00u;
    const uint32_t t = (w & kExp) ^ kExp;  // a zero half: odd
    return ((t - 0x00010001u) & ~t & 0x80008000u) != 0;
}
// Largest of n values.
template <int n>
__device__ __forceinline__ float max_of(const uint32_t* x, float top) {
#pragma unroll
    for (int k = 0; k < n; k += 2)
        asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(__uint_as_float(x[k])), "f"(__uint_as_float(x[k + 1])));
    return top;
}
template <int n>
__device__ __forceinline__ void tmem_ld_wait(uint32_t at, uint32_t* x) {
    if constexpr (n == 4)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
            : "r"(at)
            : "memory");
    else if constexpr (n == 8)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
            : "r"(at)
            : "memory");
    else if constexpr (n == 16) tmem_ld16_wait(at, x);
    else tmem_ld32_wait(at, x);
}
template <int n>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t* v) {
    if constexpr (n == 2)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(at), "r"(v[0]), "r"(v[1]) : "memory");
    else if constexpr (n == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3])
                     : "memory");
    else if constexpr (n == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]),
                     "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else tmem_st16(at, v);
}

// The thread's kKeys scores of a tile -> weights, written over them as parts.
//   s_at   the score buffer's first column in the thread's lane
//   key    the thread's first key in the tile
//   masked some row of the tile sees less than all of it; then the first
//          key's place among the new tokens is j0, and `have` keys lie
//          before the end
//   maxima where the row's shares leave theirs, kRowTile apart; the thread's is `share`
// m, l: running maximum (log2 units) and sum.  Returns the factor for what O holds.
template <int D, class T, int kKeys>
__device__ __forceinline__ float weigh(const AttnParams& p, const RowSight& sight, bool masked, int j0, int have,
                                       uint32_t s_at, int key, volatile float* maxima, int share, int quad,
                                       float& m, float& l) {
    using C = TcAttn<D, T>;
    constexpr int kHold = kKeys < C::kHold ? kKeys : C::kHold;  // scores held at a time
    constexpr int kStep = kHold < C::kStep ? kHold : C::kStep;
    uint32_t x[kHold];
    auto read = [&](int h) {
        tmem_ld_wait<kHold>(s_at + key + h, x);
        if (masked) {
            const uint32_t seen = sight.bits(p, j0 + h, have - h);
#pragma unroll
            for (int k = 0; k < kHold; ++k)
                if (!(seen >> k & 1)) x[k] = 0xff800000u;  // -inf
        }
    };
    float mx = -INFINITY;
#pragma unroll
    for (int h = 0; h < kKeys; h += kHold) {
        read(h);
        mx = max_of<kHold>(x, mx);
    }
    maxima[share * kRowTile] = mx;
    quad_sync(quad);  // (also: all have read what the weights overwrite)
#pragma unroll
    for (int i = 0; i < kShares; ++i) mx = fmaxf(mx, maxima[i * kRowTile]);
    mx *= p.scale_log2;  // (the scale is positive)
    float f = 1.f;
    if (mx > m + kLazy) {
        f = fast_exp2(m - mx);
        m = mx;
        l *= f;
    }
    const float shift = m == -INFINITY ? 0.f : kWeightBits - m;
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), shift2 = make_float2(shift, shift);
    float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int h = kKeys - kHold; h >= 0; h -= kHold) {  // (the last ones are still here)
        if (h < kKeys - kHold) read(h);                // (a thread's weights lie over its own scores only)
#pragma unroll
        for (int h2 = 0; h2 < kHold; h2 += kStep) {
            uint32_t part[C::kParts][kStep / 2];
#pragma unroll
            for (int k = 0; k < kStep / 2; ++k) {
                const uint32_t* xk = x + h2 + 2 * k;
                float2 a = fma2(make_float2(__uint_as_float(xk[0]), __uint_as_float(xk[1])), scale2, shift2);
                a = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                l2 = add2(l2, a);
                uint32_t out[C::kParts];
                Parts<T>::split(a, out);
#pragma unroll
                for (int i = 0; i < C::kParts; ++i) part[i][k] = out[i];
            }
            const int at = key + h + h2;
#pragma unroll
            for (int i = 0; i < C::kParts; ++i)
                tmem_st<kStep / 2>(s_at + C::p_col(at / 16, i) + at % 16 / 2, part[i]);
        }
    }
    l += l2.x + l2.y;
    return f;
}
// Takes NaN and infinities out of a V tile's keys first .. have - 1, and
// everything out of those behind; all softmax threads.  True where a thread
// found some among the former.
template <int D, class T>
__device__ __noinline__ bool scrub_tile(uint32_t tile, int first, int have, int thread) {
    using C = TcAttn<D, T>;
    constexpr int kTile = C::kTile;
    bool odd = false;
    for (int u = first * (D / 8) + thread; u < kTile * (D / 8); u += kSoftThreads) {
        const int key = u / (D / 8);
        const uint32_t at = tile + unit_at(key, u % (D / 8), kTile);
        if (key >= have) {
            sts_u128(at, make_uint4(0, 0, 0, 0));
            continue;
        }
        uint32_t v[4];
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at));
        if (any_odd<T>(v[0]) || any_odd<T>(v[1]) || any_odd<T>(v[2]) || any_odd<T>(v[3])) {
            odd = true;
            for (int k = 0; k < 8; ++k) {
                const float2 t = T::unpack(k & 1 ? v[k >> 1] >> 16 : v[k >> 1] & 0xffffu);
                if (!isfinite(t.x))
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(at + 2 * k), "h"((unsigned short)0) : "memory");
            }
        }
    }
    return odd;
}
// Adds to n channels of a row's output the NaN and infinities of the new
// tokens in tiles tile0 .. tile1 - 1 that it sees (their finite values are in
// it already).
template <int D, class T>
__device__ __noinline__ void add_odd(const AttnParams& p, const CacheView& c, const BatchView& b, const Item& d,
                                     int row, int token, float* out, int channel, int n, int* err) {
    const Bc bc = bc_open(err);
    for (int t = 0; t < d.tokens; ++t) {
        const int pos = d.len + t;
        if (pos < d.tile0 * TcForm<D>::kKeys || pos >= d.tile1 * TcForm<D>::kKeys ||
            !sees_new(p, row, token, t, bc))
            continue;
        const int page = page_of(c, b, d.seq, pos, err);
        if (page < 0) continue;
        const uint16_t* src = c.v + p.layer_offset + page * c.page_stride + d.head * c.head_stride +
                              (pos & (c.page_size - 1)) * c.slot_stride + channel;
        if (!bc_global(bc, src, 2 * n, c.v, c.extent, kBcAttnKv)) continue;
        for (int i = 0; i < n; ++i) {
            const float2 v = T::unpack(src[i]);
            if (!isfinite(v.x)) out[i] += v.x;
        }
    }
}
// Places in the ring of tile j's K and V, an item of n tiles starting at place 0.
__device__ __forceinline__ int place_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int place_v(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

template <int D, class T>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ AttnParams p, const __grid_constant__ CacheView c,
                        const __grid_constant__ BatchView b, int* err) {
    using C = TcAttn<D, T>;
    constexpr int kParts = C::kParts;
    constexpr uint32_t kType = kParts == 3 ? 1u : 0u;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    if ((base & 1023) != 0) {  // (no static shared memory: the swizzle atoms' alignment)
        if (threadIdx.x == 0) atomicCAS(err, 0, kDevErrLayout);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
    uint64_t* slot_free = full + C::kSlots;
    uint64_t* item_full = slot_free + C::kSlots;
    uint64_t* item_free = item_full + kItems;
    uint64_t* s_full = item_free + kItems;
    uint64_t* p_full = s_full + 2;
    uint64_t* t_full = p_full + 2;
    uint64_t* t_free = t_full + 2;
    uint64_t* q_full = t_free + 2;
    uint64_t* drained = q_full + 1;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_at + 1);
    volatile int* odd_flag = abort_flag + 1;  // [2]: an item met NaN or infinities among the new tokens' values
    volatile int* last_place = reinterpret_cast<volatile int*>(smem + C::kLast);
    Item* items = reinterpret_cast<Item*>(smem + C::kDesc);
    float* maxima = reinterpret_cast<float*>(smem + C::kMax);
    float* ends = reinterpret_cast<float*>(smem + C::kEnd);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = blockIdx.x;
    const Bc bc = bc_open(err);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(full + i, 1);
            mbar_init(slot_free + i, 1);
            last_place[i] = -1;
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(item_full + i, 1);
            mbar_init(item_free + i, kSoftWarps + 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, kSoftWarps);
            mbar_init(t_full + i, 1);
            mbar_init(t_free + i, kSoftWarps);
            odd_flag[i] = 0;
        }
        mbar_init(q_full, kSoftWarps);
        mbar_init(drained, 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    if (warp == 1) tmem_alloc(tmem_at, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_at);
    griddep_wait();
    griddep_launch_dependents();

    if (warp < kFirstSoft) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // One tile of K or V into its place of the ring, by a whole warp, a
        // box a lane.  False: a wait ran out.
        const int boxes_down = C::kTile / p.box_slots, boxes_across = C::kChunks / p.box_chunks;  // together <= 16
        const int sub = lane / boxes_across, chunk = lane % boxes_across;
        const uint32_t box_bytes = p.box_slots * p.box_chunks * kChunkBytes;
        const uint32_t dst0 = base + chunk * C::kChunkStride + sub * p.box_slots * kChunkBytes;
        auto load = [&](const void* map, const Item& d, int tile, int place, PageWindow& pages) {
            const int st = place % C::kSlots, pos0 = tile * C::kTile, pos = pos0 + sub * p.box_slots;
            pages.move(pos0 >> c.page_shift, lane);
            int page = pages.id(pos >> c.page_shift);
            // boxes that hold a key: those of slots at or behind the end stay out
            const int used = boxes_across * min(boxes_down, (d.len + d.tokens - pos0 + p.box_slots - 1) / p.box_slots);
            if (place >= C::kSlots &&
                !warp_wait(slot_free + st, ((place / C::kSlots) - 1) & 1, abort_flag, err, kDevErrTimeoutKvSlot))
                return false;
            if (place == p.skip_stage) return true;
            if (lane == 0) {
                mbar_arrive_expect_tx(full + st, used * box_bytes);
                last_place[st] = place;
            }
            __syncwarp();
            if (lane < used) {
                if (page < 0 || page >= c.pages) {
                    data_error(err, kDataPage);
                    page = c.pages;  // outside the map: zeros
                }
                const int slot = pos & (c.page_size - 1);
                bc_tma(bc, 0, 2, 64, 64, slot, c.page_size, kBcAttnKv, kBcAttnKv);
                tma_load_kv(dst0 + st * C::kTileBytes, map, slot, chunk, d.head, page, full + st);
            }
            __syncwarp();
            return true;
        };
        if (warp == 0) {
            // ------------------------------------------ producer: items and K
            WorkWalk<TcForm<D>> w;
            w.start(p, b, g, err);
            if (lane == 0 && !p.whole_items) w.tell_cut(p, g);
            int place0 = 0, count = 0;  // ring place at the item's start, items so far
            bool live = true;
            PageWindow pages;
            // The next item's descriptor, when a place for it is free.
            auto publish = [&](const Item& d) {
                const int at = count % kItems;
                if (count >= kItems && !warp_wait(item_free + at, (count / kItems - 1) & 1, abort_flag, err,
                                                  kDevErrTimeoutKvSlot)) {
                    live = false;
                    return;
                }
                if (lane == 0) {
                    items[at] = d;
                    mbar_arrive(item_full + at);
                }
                __syncwarp();
                ++count;
            };
            for (; live && w.valid(); w.next(p, b, g, err)) {
                Item d;
                d.row0 = w.w.row0;
                d.tokens = w.w.tokens;
                d.len = w.w.len;
                d.seq = w.s;
                d.head = w.head;
                d.first = w.row_tile * kRowTile;
                d.tile0 = w.tile0;
                d.tile1 = w.tile1;
                d.n = max(0, w.seen_tiles(p) - w.tile0);
                // Row tiles of one head read the same keys: each CTA starts
                // where the tile number is a multiple of a CTA's share, so
                // that they read a key at about the same time and HBM gives
                // it once (three row tiles over 131k tokens: 1.6 GB of reads
                // become 0.5).
                d.turn = 0;
                if (w.w.row_tiles > 1 && w.split.cut == 0) {
                    const int each = (int)min(w.split.each, (int64_t)INT32_MAX), past = w.tile0 % each;
                    if (past != 0 && each - past < d.n) d.turn = each - past;
                }
                d.slot = w.whole ? -1 : w.slot;
                d.pad = 0;
                publish(d);
                pages.open(b, d.seq);
                for (int j = 0; live && j < d.n; ++j) live = load(&tk, d, d.tile(j), place0 + place_k(j), pages);
                place0 += 2 * d.n;
            }
            if (live) {
                Item d = {};
                d.n = -1;
                publish(d);
            }
        } else if (warp == 2) {
            // ---------------------------------------------------- producer: V
            int place0 = 0;
            bool live = true;
            PageWindow pages;
            for (int count = 0; live; ++count) {
                const int at = count % kItems;
                if (!warp_wait(item_full + at, (count / kItems) & 1, abort_flag, err, kDevErrTimeoutScore)) break;
                const Item d = items[at];
                __syncwarp();
                if (lane == 0) mbar_arrive(item_free + at);
                if (d.n < 0) break;
                pages.open(b, d.seq);
                for (int j = 0; live && j < d.n; ++j) live = load(&tv, d, d.tile(j), place0 + place_v(j, d.n), pages);
                place0 += 2 * d.n;
            }
        } else if (warp == 1 && elect_one()) {
            // -------------------------------------------- issuer: one thread
            constexpr uint32_t kIdS = idesc_kv(C::kTile, kType, false), kIdT = idesc_kv(D, kType, true);
            int place0 = 0, it = 0, with_keys = 0;  // ring place and tile number at the item's start
            bool live = true;
            auto scores = [&](int j) {
                const int place = place0 + place_k(j), st = place % C::kSlots, buf = (it + j) & 1;
                live = live && kv_wait(full + st, (place / C::kSlots) & 1, abort_flag, err, kDevErrTimeoutKv);
                if (!live) return;
                tc_fence_after();
                const uint64_t k_desc = desc_sw128(base + st * C::kTileBytes, 16, 1024);
                const uint32_t s_at = tmem + C::kScores + buf * C::kScoreCols;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t kd = k_desc + (((k / 4) * C::kChunkStride + (k % 4) * 32) >> 4);
                    if constexpr (C::kQInTmem)
                        tc_mma_f16_ta(s_at, tmem + C::kQCol + 8 * k, kd, kIdS, k > 0);
                    else
                        tc_mma_f16(s_at,
                                   desc_sw128(base + C::kQ, 16, 1024) +
                                       (((k / 4) * kRowTile * kChunkBytes + (k % 4) * 32) >> 4),
                                   kd, kIdS, k > 0);
                }
                tc_commit(s_full + buf);
                tc_commit(slot_free + st);
            };
            for (int count = 0; live; ++count) {
                const int at = count % kItems;
                live = kv_wait(item_full + at, (count / kItems) & 1, abort_flag, err, kDevErrTimeoutScore);
                if (!live) break;
                const int n = *const_cast<volatile int*>(&items[at].n);
                if (n < 0) break;
                mbar_arrive(item_free + at);
                if (n == 0) continue;
                live = kv_wait(q_full, with_keys & 1, abort_flag, err, kDevErrTimeoutScore);
                scores(0);
                for (int j = 0; live && j < n; ++j) {
                    if (j + 1 < n) scores(j + 1);
                    const int place = place0 + place_v(j, n), st = place % C::kSlots;
                    const int i = it + j, buf = i & 1, tb = i % C::kTBufs;
                    live = live && kv_wait(full + st, (place / C::kSlots) & 1, abort_flag, err, kDevErrTimeoutKv);
                    if (i >= C::kTBufs)
                        live = live && kv_wait(t_free + tb, (i / C::kTBufs - 1) & 1, abort_flag, err,
                                                 kDevErrTimeoutScore);
                    live = live && kv_wait(p_full + buf, (i >> 1) & 1, abort_flag, err, kDevErrTimeoutScore);
                    if (!live) break;
                    tc_fence_after();
                    const uint64_t v_desc = desc_sw128(base + st * C::kTileBytes, C::kChunkStride, 1024);
                    const uint32_t p_at = tmem + C::kScores + buf * C::kScoreCols, t_at = tmem + tb * D;
#pragma unroll
                    for (int part = kParts - 1; part >= 0; --part)  // the smallest parts first
#pragma unroll
                        for (int k = 0; k < C::kTile / 16; ++k) {
                            const uint64_t vd = v_desc + ((k * 16 * kChunkBytes) >> 4);
                            // (the product that joins the smallest parts brings their sum down to scale)
                            if (Parts<T>::kLastShift > 0 && part == kParts - 2 && k == 0)
                                tc_mma_f16_ta_down<Parts<T>::kLastShift>(t_at, p_at + C::p_col(k, part), vd, kIdT);
                            else
                                tc_mma_f16_ta(t_at, p_at + C::p_col(k, part), vd, kIdT, part < kParts - 1 || k > 0);
                        }
                    tc_commit(t_full + tb);
                    tc_commit(slot_free + st);
                }
                place0 += 2 * n;
                it += n;
                ++with_keys;
            }
            // Tensor memory is given back only when every product is done.
            if (*abort_flag) {
                tc_commit(drained);
                int no_abort = 0;
                kv_wait(drained, 0, &no_abort, err, kDevErrTimeoutScore);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int quad = warp & 3, share = (warp - kFirstSoft) >> 2;
        const int st_id = threadIdx.x - 32 * kFirstSoft;
        const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
        int place0 = 0, it = 0;
        for (int count = 0;; ++count) {
            const int at = count % kItems;
            const bool got = kv_wait(item_full + at, (count / kItems) & 1, abort_flag, err, kDevErrTimeoutScore);
            if (soft_any(!got)) break;  // (all softmax threads leave together)
            const Item& d = items[at];
            const int n = d.n;
            if (n < 0) break;
            const int len = d.len, keys = len + d.tokens;
            const int rows = min(kRowTile, d.tokens * p.group - d.first);
            // Up to 32 (64) rows stand in all four quadrants (in two pairs of
            // them), each with a quarter (a half) of every tile's keys: all the
            // SM's schedulers work on the softmax, and the copies' results
            // are joined at the item's end.
            const int copies = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
            const int spread = 4 / copies;            // quadrants of a copy
            const int copy = quad / spread;
            const int r = quad % spread * 32 + lane;  // the thread's row of the tile
            const bool busy = quad % spread * 32 < rows;  // the warp has rows
            const int my_keys = C::kTile / kShares / copies, my_key = (kShares * copy + share) * my_keys;
            RowSight sight;
            float2 o[C::kShareD / 2];
#pragma unroll
            for (int i = 0; i < C::kShareD / 2; ++i) o[i] = make_float2(0.f, 0.f);
            float m = -INFINITY, l = 0.f, f_last = 1.f;
            {
                // Q of the item's rows: each thread its share of its row's
                // channels.  Rows behind the last are zero.
                const int row = d.first + min(r, rows - 1), tok = token_of(p, row);
                sight.open(p, d.row0, tok, bc);
                // Warps take rows, lanes neighbouring 16 bytes of them (256 /
                // D * 2 rows at a time).  Rows behind the last keep what is
                // there: a row's products reach its own lane only.
                if (n > 0) {
                    constexpr int kAcross = D / 8, kDown = 32 / kAcross;
                    constexpr int kPitch = C::kStageRow * 4, kPiece = C::kShareD < 32 ? C::kShareD : 32;
                    uint8_t* const stage = smem + C::kOut;
                    const int soft = warp - kFirstSoft, col = lane % kAcross * 8;
                    const uint16_t* src = p.q + d.row0 * p.q_row_stride + (int64_t)d.head * p.group * D + col;
                    constexpr int kMost = kRowTile / (kSoftWarps * kDown);
                    uint4 v[kMost];
#pragma unroll
                    for (int i = 0; i < kMost; ++i) {
                        // (the last row again instead of a branch: all loads are in flight together)
                        const int from = min((i * kSoftWarps + soft) * kDown + lane / kAcross, rows - 1);
                        const int t = token_of(p, d.first + from);
                        const uint16_t* at_q = src + t * p.q_row_stride + (d.first + from - t * p.group) * D;
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (bc_global(bc, at_q, 16, p.q,
                                      2 * ((p.rows - 1) * p.q_row_stride + (int64_t)p.group * p.kv_heads * D), kBcAttnQ))
                            v[i] = *reinterpret_cast<const uint4*>(at_q);
                    }
#pragma unroll
                    for (int i = 0; i < kMost; ++i) v[i] = sign_q(p, v[i]);
                    if constexpr (C::kQInTmem) {
                        // through the staging rows, 32 channels of each share (or all) at a time
#pragma unroll
                        for (int c0 = 0; c0 < C::kShareD; c0 += kPiece) {
                            if (c0 > 0) soft_sync();
                            const int in_share = col % C::kShareD - c0;
#pragma unroll
                            for (int i = 0; i < kMost; ++i) {
                                const int from = (i * kSoftWarps + soft) * kDown + lane / kAcross;
                                if (from < rows && in_share >= 0 && in_share < kPiece)
                                    *reinterpret_cast<uint4*>(stage + (col / C::kShareD * kRowTile + from) * kPitch +
                                                              in_share * 2) = v[i];
                            }
                            soft_sync();
                            if (busy) {
                                uint4 mine[kPiece / 8];
#pragma unroll
                                for (int i = 0; i < kPiece / 8; ++i)
                                    mine[i] = *reinterpret_cast<const uint4*>(stage + (share * kRowTile + r) * kPitch +
                                                                              16 * i);
                                tmem_st<kPiece / 2>(tmem + lane_at + C::kQCol + (share * C::kShareD + c0) / 2,
                                                    reinterpret_cast<const uint32_t*>(mine));
                            }
                        }
                        if (busy) tmem_wait_st();
                        tc_fence_before();
                    } else {
#pragma unroll
                        for (int i = 0; i < kMost; ++i) {
                            const int from = (i * kSoftWarps + soft) * kDown + lane / kAcross;
                            if (from < rows)  // (row `from` of every copy)
                                for (int k = 0; k < copies; ++k)
                                    sts_u128(base + C::kQ + unit_at(k * spread * 32 + from, col / 8, kRowTile), v[i]);
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_full);
                }
            }
            // O takes tile j's product while tile j + 1's is under way
            auto accumulate = [&](int i, float f) {
                const int tb = i % C::kTBufs;
                kv_wait(t_full + tb, (i / C::kTBufs) & 1, abort_flag, err, kDevErrTimeoutScore);
                if (busy) {
                    tc_fence_after();
                    const float2 f2 = make_float2(f, f);
#pragma unroll
                    for (int k = 0; k < C::kShareD; k += kAccCols) {
                        uint32_t t[kAccCols];
                        tmem_ld_wait<kAccCols>(tmem + lane_at + tb * D + share * C::kShareD + k, t);
#pragma unroll
                        for (int x = 0; x < kAccCols / 2; ++x)
                            o[k / 2 + x] = fma2(o[k / 2 + x], f2,
                                                make_float2(__uint_as_float(t[2 * x]), __uint_as_float(t[2 * x + 1])));
                    }
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(t_free + tb);
            };
            for (int j = 0; j < n; ++j) {
                const int i = it + j, buf = i & 1;
                const int pos0 = d.tile(j) * C::kTile, key0 = pos0 + my_key;
                kv_wait(s_full + buf, (i >> 1) & 1, abort_flag, err, kDevErrTimeoutScore);
                float f = 1.f;
                if (busy) {
                    tc_fence_after();
                    const uint32_t s_at = tmem + lane_at + C::kScores + buf * C::kScoreCols;
                    const bool masked = pos0 + C::kTile > len;
                    volatile float* most = maxima + buf * kShares * kRowTile + quad * 32 + lane;
                    const int j0 = key0 - len, have = keys - key0;
                    constexpr int kK = C::kTile / kShares;
                    if (copies == 1) {
                        f = weigh<D, T, kK>(p, sight, masked, j0, have, s_at, my_key, most, share, quad, m, l);
                    } else {
                        f = copies == 2
                                ? weigh<D, T, kK / 2>(p, sight, masked, j0, have, s_at, my_key, most, share, quad, m, l)
                                : weigh<D, T, kK / 4>(p, sight, masked, j0, have, s_at, my_key, most, share, quad, m, l);
                        // the other copies' keys weigh nothing in these lanes
                        const uint32_t zero[16] = {};
                        const int own = C::kTile / 16 / copies;  // 16-key groups of a copy
#pragma unroll
                        for (int k = 0; k < C::kTile / 16; ++k)
                            if (k / own != copy && k % kShares == share) {
                                tmem_st<16>(s_at + 16 * k, zero);
                                if constexpr (kParts == 3) tmem_st<8>(s_at + C::p_col(k, 2), zero);
                            }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                if (pos0 + C::kTile > len && (keys - pos0 < C::kTile || keys - len > 1 || p.mask != nullptr)) {
                    // Slots behind the end may hold anything, and so may tokens
                    // that some row does not see (without a mask a single new
                    // token sees itself): a zero weight would carry their NaN
                    // and infinities into its sum.  Such values leave the tile;
                    // rows that do see them get them at the item's end.
                    const int place = place0 + place_v(j, n), st = place % C::kSlots;
                    kv_wait(full + st, (place / C::kSlots) & 1, abort_flag, err, kDevErrTimeoutKv);
                    if (scrub_tile<D, T>(base + st * C::kTileBytes, max(0, len - pos0), min(C::kTile, keys - pos0), st_id))
                        odd_flag[count & 1] = 1;
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + buf);
                if (j > 0) accumulate(i - 1, f_last);
                f_last = f;
            }
            if (n > 0) accumulate(it + n - 1, f_last);
            place0 += 2 * n;
            it += n;
            // (Every thread is past the previous item: its flag serves the next.)
            if (n > 0 && st_id == 0) odd_flag[(count & 1) ^ 1] = 0;

            // The row's maximum over its copies and sum over copies and
            // shares (all threads have read the last item's by now).
            const int lane_row = quad * 32 + lane;
            float top = m, fix = 1.f, sum = 0.f;
            if (copies > 1) {
                if (busy && share == 0) ends[lane_row] = m;
                soft_sync();
                for (int i = 0; i < copies; ++i) top = fmaxf(top, ends[(i * spread + quad % spread) * 32 + lane]);
                fix = m == -INFINITY ? 0.f : fast_exp2(m - top);
                if (m != -INFINITY) l *= fix;  // (else nothing was seen: 0, or NaN)
            }
            if (busy) ends[(1 + share) * kRowTile + lane_row] = l;
            if (copies > 1) soft_sync();
            else if (busy) quad_sync(quad);
            for (int i = 0; i < copies; ++i)
#pragma unroll
                for (int k = 0; k < kShares; ++k)
                    sum += ends[(1 + k) * kRowTile + (i * spread + quad % spread) * 32 + lane];
            const bool whole = d.slot < 0;
            if (!whole && share == 0 && copy == 0 && r < rows)
                if (float2* to = part_sum(p, d.slot, r, bc)) *to = make_float2(top, sum);
            if (copies > 1) {
                // The other copies hand their outputs to the first, kStageCols
                // channels at a time through shared memory.
                constexpr int kCols = C::kStageCols, kPitch = C::kStageRow;
                float* const stage = reinterpret_cast<float*>(smem + C::kOut) + share * kRowTile * kPitch;
#pragma unroll
                for (int ch = 0; ch < C::kShareD / kCols; ++ch) {
                    if (ch > 0) soft_sync();
                    if (busy && copy > 0) {
#pragma unroll
                        for (int i = 0; i < kCols / 4; ++i) {
                            const float2 x = o[ch * (kCols / 2) + 2 * i], y = o[ch * (kCols / 2) + 2 * i + 1];
                            *reinterpret_cast<float4*>(stage + lane_row * kPitch + 4 * i) =
                                make_float4(x.x * fix, x.y * fix, y.x * fix, y.y * fix);
                        }
                    }
                    soft_sync();
                    if (busy && copy == 0) {
#pragma unroll
                        for (int i = 0; i < kCols / 2; ++i) {
                            float2& x = o[ch * (kCols / 2) + i];
                            x = make_float2(x.x * fix, x.y * fix);
                        }
                        for (int k = 1; k < copies; ++k) {
                            const float* from = stage + (k * spread * 32 + r) * kPitch;
#pragma unroll
                            for (int i = 0; i < kCols / 4; ++i) {
                                const float4 t = *reinterpret_cast<const float4*>(from + 4 * i);
                                float2 &x = o[ch * (kCols / 2) + 2 * i], &y = o[ch * (kCols / 2) + 2 * i + 1];
                                x = make_float2(x.x + t.x, x.y + t.y);
                                y = make_float2(y.x + t.z, y.y + t.w);
                            }
                        }
                    }
                }
            }
            if (copy == 0 && r < rows) {
                const float scale = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;  // a row that sees nothing: zeros
                const int row = d.first + r, tok = sight.token;
                float* const dst = (whole ? p.out + (d.row0 + tok) * p.out_row_stride +
                                                ((int64_t)d.head * p.group + row - tok * p.group) * D
                                          : part_row(p, d.slot, r, 0, D, bc)) + share * C::kShareD;
                if (!whole ? part_row(p, d.slot, r, 0, D, bc) != nullptr : bc_global(bc, dst, 4 * C::kShareD, p.out,
                                        4 * ((p.rows - 1) * p.out_row_stride + (int64_t)p.group * p.kv_heads * D),
                                        kBcAttnOut)) {
                    if (!whole || p.wide_out) {
#pragma unroll
                        for (int i = 0; i < C::kShareD / 8; ++i) {
                            const float2* x = o + 4 * i;
                            asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 8 * i),
                                         "f"(x[0].x * scale), "f"(x[0].y * scale), "f"(x[1].x * scale),
                                         "f"(x[1].y * scale), "f"(x[2].x * scale), "f"(x[2].y * scale),
                                         "f"(x[3].x * scale), "f"(x[3].y * scale)
                                         : "memory");
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < C::kShareD / 4; ++i)
                            *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(
                                o[2 * i].x * scale, o[2 * i].y * scale, o[2 * i + 1].x * scale, o[2 * i + 1].y * scale);
                    }
                    if (odd_flag[count & 1] != 0)
                        add_odd<D, T>(p, c, b, d, sight.row, tok, dst, share * C::kShareD, C::kShareD, err);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(item_free + at);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // No copy may be in flight when the CTA ends; all were waited for, unless
    // a wait ran out.
    if (*abort_flag && warp == 0)
        for (int i = 0; i < C::kSlots; ++i)
            if (last_place[i] >= 0) {
                int no_abort = 0;
                kv_wait(full + i, (last_place[i] / C::kSlots) & 1, &no_abort, err, kDevErrTimeoutKv);
            }
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <int D, class T>
cudaError_t launch_one(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, const CacheView& c,
                       const BatchView& b, int* err, cudaStream_t stream) {
    const cudaError_t e = allow_smem<attention_tc_kernel<D, T>>(TcAttn<D, T>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_chained(attention_tc_kernel<D, T>, dim3((unsigned)p.ctas), dim3(kThreads), TcAttn<D, T>::kSmem, stream, 1,
                          tk, tv, p, c, b, err);
}

template <class T>
cudaError_t launch_type(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, const CacheView& c,
                        const BatchView& b, int* err, cudaStream_t stream) {
    switch (c.head_dim) {
        case 64: return launch_one<64, T>(p, tk, tv, c, b, err, stream);
        case 128: return launch_one<128, T>(p, tk, tv, c, b, err, stream);
        case 256: return launch_one<256, T>(p, tk, tv, c, b, err, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_attention_tc(const AttnParams& p, const void* tk, const void* tv, const CacheView& c,
                                const BatchView& b, bool bf16, int* err, cudaStream_t stream) {
    const CUtensorMap& mk = *static_cast<const CUtensorMap*>(tk);
    const CUtensorMap& mv = *static_cast<const CUtensorMap*>(tv);
    return bf16 ? launch_type<KvBf16>(p, mk, mv, c, b, err, stream) : launch_type<KvF16>(p, mk, mv, c, b, err, stream);
}

}  // namespace iq4xs
