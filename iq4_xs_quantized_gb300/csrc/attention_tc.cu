// attention_tc.cu -- tree attention for many rows a key/value head (drafted
// trees, prompt chunks): tcgen05 on tiles of 128 rows x 64 keys.
//
// One pass, as in the warp-level form; here a row is a lane of tensor memory:
//
//   S = Q K^T      128 x 64, Q from tensor memory, K from shared memory
//   P = exp2(S - m) split into 16-bit parts, back into tensor memory over S
//   T = P V        128 x D, P from tensor memory, V from shared memory (as it
//                  lies: channels contiguous)
//   O = O f + T    in fp32 registers of the threads that own the row
//
// T starts from zero for every key tile and is added to O by rounded fp32
// arithmetic: the tensor core cuts its sums off, and thousands of tiles on
// one accumulator would add those cuts up.
//
// Roles: a producer warp (TMA), a warp whose first lane issues the MMAs, and
// eight softmax warps, two per 32-lane quadrant: one takes keys 0-31 of a
// tile and channels 0..D/2-1 of O, the other the rest; they share a row's
// maximum through shared memory.  The MMAs of tile j + 1's scores are issued
// before tile j's output product, so the tensor core works while the softmax
// runs.  K and V tiles go through one ring in the order the MMAs take them:
// K0 K1 V0 K2 V1 ... V(n-1).
//
// Up to about 48 rows HBM bounds it (4 D bytes a key), above that the tensor
// core (1 + parts products of 128 x 64 x D a tile).
#include "attention.cuh"

namespace iq4xs {
namespace {

constexpr int kRowTile = 128;
constexpr int kSoftWarps = 8;
constexpr int kFirstSoft = 4;  // warps 4-11: two whole warpgroups
constexpr int kThreads = 32 * (kFirstSoft + kSoftWarps);
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kHalfKeys = kKeyTile / 2;
constexpr int kTmemCols = 512;
constexpr int kStageCols = 16, kStageRow = kStageCols + 4;  // floats of a row on its way out, and its pitch

template <int D, class T>
struct TcAttn {
    static constexpr int kParts = Parts<T>::kN;
    static constexpr int kChunks = D / 64;
    static constexpr int kTileBytes = kKeyTile * D * 2;
    static constexpr int kTBufs = D == 256 ? 1 : 2;          // output products in flight
    // Tensor memory: T; Q (16-bit pairs), except where 512 columns do not
    // hold it; two score buffers: S (64 columns), overlaid in place by P: the
    // first two parts of 16 keys take the keys' own 16 columns, a third 8 more.
    static constexpr int kScoreCols = kParts == 3 ? 96 : 64;
    static constexpr bool kQInTmem = kTBufs * D + D / 2 + 2 * kScoreCols <= kTmemCols;
    static constexpr int kQCol = kTBufs * D;
    static constexpr int kScores = kQCol + (kQInTmem ? D / 2 : 0);
    static_assert(kScores + 2 * kScoreCols <= kTmemCols, "tensor memory");
    // shared memory
    static constexpr int kQBytes = kQInTmem ? 0 : kRowTile * D * 2;
    static constexpr int kStageBytes = kSoftWarps * 32 * kStageRow * 4;
    static constexpr int kSlots = (224 * 1024 - kQBytes - kStageBytes) / kTileBytes;  // 6 (4 with Q), 12, 25
    static constexpr int kQ = kSlots * kTileBytes;
    static constexpr int kOut = kQ + kQBytes;                // the warps' outputs on their way out
    static constexpr int kMax = kOut + kStageBytes;          // [2][2 halves][128] row maxima
    static constexpr int kBars = kMax + 2 * 2 * kRowTile * 4;
    static constexpr int kNumBars = 2 * kSlots + 2 + 2 + 2 + 2 + 1 + 1;
    static constexpr int kMisc = kBars + kNumBars * 8;       // tensor memory address, abort, odd values
    static constexpr int kSmem = kMisc + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static constexpr int kHalfD = D / 2;
    static constexpr int kHold = D == 256 ? 16 : 32;         // scores a thread holds at a time
    // Column of a part of the weights of keys 16 key16 .. + 15, from the buffer's first.
    static __device__ __forceinline__ uint32_t p_col(int key16, int part) {
        return part < 2 ? 16 * key16 + 8 * part : kKeyTile + 8 * key16;
    }
};
// D = 256 keeps 128 output channels a softmax thread: the producer's and the
// issuer's warpgroup gives up registers (80 + 2 * 208 <= 3 * 168, the launch's).
constexpr int kSoftRegs = 208, kOtherRegs = 80;
static_assert(kOtherRegs + 2 * kSoftRegs <= 3 * 168, "register split within the launch's");

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
__device__ __forceinline__ void pair_sync(int quadrant) {
    asm volatile("bar.sync %0, 64;" ::"r"(quadrant + 1) : "memory");
}
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 5, 256;" ::: "memory"); }
static_assert(kSoftThreads == 256, "the softmax warps' barrier");
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
    if constexpr (n == 8)
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
    if constexpr (n == 4)
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
//   seen   bit k: the row sees key + k
//   mine, theirs  where the thread and the one that has the row's other half leave their maxima
// m, l: running maximum (log2 units) and sum.  Returns the factor for what O holds.
template <int D, class T, int kKeys>
__device__ __forceinline__ float weigh(const AttnParams& p, uint32_t s_at, int key, uint32_t seen,
                                       volatile float* mine, volatile float* theirs, int quad, float& m, float& l) {
    using C = TcAttn<D, T>;
    constexpr int kHold = kKeys == 32 ? C::kHold : kKeys;  // scores held at a time
    constexpr int kStep = kKeys < 16 ? kKeys : 16;
    uint32_t x[kHold];
    float mx = -INFINITY;
#pragma unroll
    for (int h = 0; h < kKeys; h += kHold) {
        tmem_ld_wait<kHold>(s_at + key + h, x);
        if (seen != 0xffffffffu) {
#pragma unroll
            for (int k = 0; k < kHold; ++k)
                if (!(seen >> (h + k) & 1)) x[k] = 0xff800000u;  // -inf
        }
        mx = max_of<kHold>(x, mx);
    }
    *mine = mx;
    pair_sync(quad);  // (also: both have read what the weights overwrite)
    mx = fmaxf(mx, *theirs) * p.scale_log2;  // (the scale is positive)
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
    for (int h = 0; h < kKeys; h += kStep) {
        if constexpr (kHold < kKeys) {  // (read again: a thread's weights lie over its own scores only)
            tmem_ld_wait<kStep>(s_at + key + h, x);
            if (seen != 0xffffffffu) {
#pragma unroll
                for (int k = 0; k < kStep; ++k)
                    if (!(seen >> (h + k) & 1)) x[k] = 0xff800000u;
            }
        }
        uint32_t part[C::kParts][kStep / 2];
#pragma unroll
        for (int k = 0; k < kStep / 2; ++k) {
            const uint32_t* xk = x + (kHold < kKeys ? 0 : h) + 2 * k;
            float2 a = fma2(make_float2(__uint_as_float(xk[0]), __uint_as_float(xk[1])), scale2, shift2);
            a = make_float2(fast_exp2(a.x), fast_exp2(a.y));
            l2 = add2(l2, a);
            uint32_t out[C::kParts];
            Parts<T>::split(a, out);
#pragma unroll
            for (int i = 0; i < C::kParts; ++i) part[i][k] = out[i];
        }
#pragma unroll
        for (int i = 0; i < C::kParts; ++i)
            tmem_st<kStep / 2>(s_at + C::p_col((key + h) / 16, i) + (key + h) % 16 / 2, part[i]);
    }
    l += l2.x + l2.y;
    return f;
}
// Places in the ring of tile j's K and V, an item of n tiles starting at place 0.
__device__ __forceinline__ int place_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int place_v(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

template <int D, class T>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const AttnParams p, const CacheView c, const BatchView b, int* err) {
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
    uint64_t* s_full = slot_free + C::kSlots;
    uint64_t* p_full = s_full + 2;
    uint64_t* t_full = p_full + 2;
    uint64_t* t_free = t_full + 2;
    uint64_t* q_full = t_free + 2;
    uint64_t* drained = q_full + 1;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_at + 1);
    volatile int* odd_flag = abort_flag + 1;  // this item met NaN or infinities among the new tokens' values
    float* maxima = reinterpret_cast<float*>(smem + C::kMax);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = blockIdx.x;
    const Bc bc = bc_open(err);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(full + i, 1);
            mbar_init(slot_free + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, kSoftWarps);
            mbar_init(t_full + i, 1);
            mbar_init(t_free + i, kSoftWarps);
        }
        mbar_init(q_full, kSoftWarps);
        mbar_init(drained, 1);
        *abort_flag = 0;
        *odd_flag = 0;
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
    WorkWalk<kRowTile> w;
    w.start(p, b, g, err);

    if (warp < kFirstSoft) {
        if constexpr (D == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 0) {
            // ------------------------------------------------------ producer
            const int box_slots = min(c.page_size, kKeyTile);
            const int boxes = kKeyTile / box_slots * C::kChunks;  // at most 16: one a lane
            const uint32_t box_bytes = box_slots * kChunkBytes;
            const int sub = lane / C::kChunks, chunk = lane % C::kChunks;
            const uint32_t dst0 = base + chunk * kKeyTile * kChunkBytes + sub * box_bytes;
            int place = 0;  // in the ring, over all items
            bool live = true;
            auto load = [&](const void* map, int page, int slot, int used) {
                const int st = place % C::kSlots;
                if (place >= C::kSlots && !warp_wait(slot_free + st, ((place / C::kSlots) - 1) & 1, abort_flag, err,
                                                     kDevErrTimeoutKvSlot)) {
                    live = false;
                    return;
                }
                const bool skip = place == p.skip_stage;
                if (lane == 0 && !skip) mbar_arrive_expect_tx(full + st, used * box_bytes);
                __syncwarp();
                if (lane < used && !skip) {
                    const int y = p.slot_axis == 1 ? slot : w.head, z = p.slot_axis == 1 ? w.head : slot;
                    bc_tma(bc, chunk * 64, 2, 64, D, slot, c.page_size, kBcAttnKv, kBcAttnKv);
                    tma_load_4d(dst0 + st * C::kTileBytes, map, chunk * 64, y, z, page, full + st);
                }
                __syncwarp();
                ++place;
            };
            for (; live && w.valid(); w.next(p, b, g, err)) {
                const int end = w.seen_tiles(p);
                const int keys = w.w.len + w.w.tokens;
                const int held = min(b.held[w.s], b.table_width);
                const int32_t* table = b.page_table + w.s * b.table_stride;
                int page0 = (w.tile0 * kKeyTile) >> c.page_shift;
                int ids = page0 + lane < held ? table[page0 + lane] : -1;
                int ids2 = page0 + 32 + lane < held ? table[page0 + 32 + lane] : -1;
                int page_v = 0, slot_v = 0, used_v = 0;  // the previous tile's boxes, for its V
                for (int tile = w.tile0; live && tile < end; ++tile) {
                    const int pos0 = tile * kKeyTile, pos = pos0 + sub * box_slots;
                    while ((pos0 >> c.page_shift) >= page0 + 32) {
                        page0 += 32;
                        ids = ids2;
                        ids2 = page0 + 32 + lane < held ? table[page0 + 32 + lane] : -1;
                    }
                    const int used =
                        min(boxes, (min(kKeyTile, keys - pos0) + box_slots - 1) / box_slots * C::kChunks);
                    int page = __shfl_sync(0xffffffffu, ids, ((pos >> c.page_shift) - page0) & 31);
                    if (lane < used && (page < 0 || page >= c.pages)) {
                        data_error(err, kDataPage);
                        page = c.pages;  // outside the map: zeros
                    }
                    const int slot = pos & (c.page_size - 1);
                    load(&tk, page, slot, used);
                    if (live && tile > w.tile0) load(&tv, page_v, slot_v, used_v);
                    page_v = page;
                    slot_v = slot;
                    used_v = used;
                }
                if (live && end > w.tile0) load(&tv, page_v, slot_v, used_v);
            }
            // No copy may be in flight when the CTA ends.
            if (*abort_flag)
                for (int i = max(0, place - C::kSlots); i < place; ++i)
                    if (i != p.skip_stage) {
                        int no_abort = 0;
                        mbar_wait(full + i % C::kSlots, (i / C::kSlots) & 1, &no_abort, err, kDevErrTimeoutKv);
                    }
        } else if (warp == 1 && elect_one()) {
            // -------------------------------------------- issuer: one thread
            constexpr uint32_t kIdS = idesc_kv(kKeyTile, kType, false), kIdT = idesc_kv(D, kType, true);
            int place0 = 0, it = 0, items = 0;  // ring place and tile number at the item's start
            bool live = true;
            auto scores = [&](int j) {
                const int place = place0 + place_k(j), st = place % C::kSlots, buf = (it + j) & 1;
                live = live && mbar_wait(full + st, (place / C::kSlots) & 1, abort_flag, err, kDevErrTimeoutKv);
                if (!live) return;
                tc_fence_after();
                const uint64_t k_desc = desc_sw128(base + st * C::kTileBytes, 16, 1024);
                const uint32_t s_at = tmem + C::kScores + buf * C::kScoreCols;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t kd = k_desc + (((k / 4) * kKeyTile * kChunkBytes + (k % 4) * 32) >> 4);
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
            for (; live && w.valid(); w.next(p, b, g, err)) {
                const int n = w.seen_tiles(p) - w.tile0;
                if (n <= 0) continue;
                live = mbar_wait(q_full, items & 1, abort_flag, err, kDevErrTimeoutScore);
                scores(0);
                for (int j = 0; live && j < n; ++j) {
                    if (j + 1 < n) scores(j + 1);
                    const int place = place0 + place_v(j, n), st = place % C::kSlots;
                    const int i = it + j, buf = i & 1, tb = i % C::kTBufs;
                    live = live && mbar_wait(full + st, (place / C::kSlots) & 1, abort_flag, err, kDevErrTimeoutKv);
                    if (i >= C::kTBufs)
                        live = live && mbar_wait(t_free + tb, (i / C::kTBufs - 1) & 1, abort_flag, err,
                                                 kDevErrTimeoutScore);
                    live = live && mbar_wait(p_full + buf, (i >> 1) & 1, abort_flag, err, kDevErrTimeoutScore);
                    if (!live) break;
                    tc_fence_after();
                    const uint64_t v_desc = desc_sw128(base + st * C::kTileBytes, kKeyTile * kChunkBytes, 1024);
                    const uint32_t p_at = tmem + C::kScores + buf * C::kScoreCols, t_at = tmem + tb * D;
#pragma unroll
                    for (int part = kParts - 1; part >= 0; --part)  // the smallest parts first
#pragma unroll
                        for (int k = 0; k < kKeyTile / 16; ++k)
                            tc_mma_f16_ta(t_at, p_at + C::p_col(k, part), v_desc + ((k * 16 * kChunkBytes) >> 4), kIdT,
                                          part < kParts - 1 || k > 0);
                    tc_commit(t_full + tb);
                    tc_commit(slot_free + st);
                }
                place0 += 2 * n;
                it += n;
                ++items;
            }
            // Tensor memory is given back only when every product is done.
            if (*abort_flag) {
                tc_commit(drained);
                int no_abort = 0;
                mbar_wait(drained, 0, &no_abort, err, kDevErrTimeoutScore);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        if constexpr (D == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int quad = warp & 3, half = (warp - kFirstSoft) >> 2;
        const int st_id = threadIdx.x - 32 * kFirstSoft;
        const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
        int place0 = 0, it = 0;
        for (; w.valid(); w.next(p, b, g, err)) {
            const int n = max(0, w.seen_tiles(p) - w.tile0);
            const int rows = min(kRowTile, w.w.tokens * p.group - w.row_tile * kRowTile);
            const int keys = w.w.len + w.w.tokens;
            // Up to 32 (64) rows stand in all four quadrants (in two pairs of
            // them), each with a quarter (half) of every tile's keys: all the
            // SM's schedulers work on the softmax, and the copies' results
            // are joined at the item's end.
            const int copies = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
            const int spread = 4 / copies;            // quadrants of a copy
            const int copy = quad / spread;
            const int r = quad % spread * 32 + lane;  // the thread's row of the tile
            const bool busy = quad % spread * 32 < rows;  // the warp has rows
            const int my_row = w.row_tile * kRowTile + min(r, rows - 1);
            const int tok = my_row / p.group;
            const int my_keys = kHalfKeys / copies, my_key = (2 * copy + half) * my_keys;
            float2 o[C::kHalfD / 2];
#pragma unroll
            for (int i = 0; i < C::kHalfD / 2; ++i) o[i] = make_float2(0.f, 0.f);
            float m = -INFINITY, l = 0.f, f_last = 1.f;
            if (n > 0) {
                // Q of the item's rows: each thread its row's half of the
                // channels.  Rows behind the last are zero.
                const uint16_t* src = p.q + (w.w.row0 + tok) * p.q_row_stride +
                                      ((int64_t)w.head * p.group + my_row % p.group) * D + half * C::kHalfD;
                const bool ok = r < rows &&
                                bc_global(bc, src, 2 * C::kHalfD, p.q,
                                          2 * ((p.rows - 1) * p.q_row_stride + (int64_t)p.group * p.kv_heads * D),
                                          kBcAttnQ);
                uint4 v[C::kHalfD / 8];
#pragma unroll
                for (int i = 0; i < C::kHalfD / 8; ++i)
                    v[i] = ok ? load_q(p, src + 8 * i) : make_uint4(0, 0, 0, 0);
                if constexpr (C::kQInTmem) {
                    if (busy) {
#pragma unroll
                        for (int i = 0; i < C::kHalfD / 32; ++i)
                            tmem_st16(tmem + lane_at + C::kQCol + half * (C::kHalfD / 2) + 16 * i,
                                      reinterpret_cast<const uint32_t*>(v + 4 * i));
                        tmem_wait_st();
                        tc_fence_before();
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < C::kHalfD / 8; ++i)
                        sts_u128(base + C::kQ + unit_at(quad * 32 + lane, half * (C::kHalfD / 8) + i, kRowTile), v[i]);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            // O takes tile j's product while tile j + 1's is under way
            auto accumulate = [&](int i, float f) {
                const int tb = i % C::kTBufs;
                mbar_wait(t_full + tb, (i / C::kTBufs) & 1, abort_flag, err, kDevErrTimeoutScore);
                if (busy) {
                    tc_fence_after();
                    const float2 f2 = make_float2(f, f);
#pragma unroll
                    for (int k = 0; k < C::kHalfD / 32; ++k) {
                        uint32_t t[32];
                        tmem_ld32_wait(tmem + lane_at + tb * D + half * C::kHalfD + 32 * k, t);
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            o[16 * k + x] = fma2(o[16 * k + x], f2,
                                                 make_float2(__uint_as_float(t[2 * x]), __uint_as_float(t[2 * x + 1])));
                    }
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(t_free + tb);
            };
            for (int j = 0; j < n; ++j) {
                const int i = it + j, buf = i & 1;
                const int pos0 = (w.tile0 + j) * kKeyTile, key0 = pos0 + my_key;
                mbar_wait(s_full + buf, (i >> 1) & 1, abort_flag, err, kDevErrTimeoutScore);
                float f = 1.f;
                if (busy) {
                    tc_fence_after();
                    const uint32_t s_at = tmem + lane_at + C::kScores + buf * C::kScoreCols;
                    uint32_t seen = 0xffffffffu;
                    if (key0 + my_keys > w.w.len || key0 + my_keys > keys)
                        seen = seen_bits(p, w.w.row0 + tok, tok, key0 - w.w.len, keys - key0);
                    volatile float* mine = maxima + (buf * 2 + half) * kRowTile + quad * 32 + lane;
                    volatile float* theirs = maxima + (buf * 2 + (half ^ 1)) * kRowTile + quad * 32 + lane;
                    if (copies == 1) {
                        f = weigh<D, T, 32>(p, s_at, my_key, seen, mine, theirs, quad, m, l);
                    } else {
                        f = copies == 2 ? weigh<D, T, 16>(p, s_at, my_key, seen, mine, theirs, quad, m, l)
                                        : weigh<D, T, 8>(p, s_at, my_key, seen, mine, theirs, quad, m, l);
                        // the other copies' keys weigh nothing in these lanes
                        const uint32_t zero[16] = {};
                        const int own = 4 / copies;  // 16-key groups of a copy
#pragma unroll
                        for (int k = 0; k < kKeyTile / 16; ++k)
                            if (k / own != copy && (k & 1) == half) {
                                tmem_st<16>(s_at + 16 * k, zero);
                                if constexpr (kParts == 3) tmem_st<8>(s_at + C::p_col(k, 2), zero);
                            }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                if (pos0 + kKeyTile > w.w.len && (keys - pos0 < kKeyTile || w.w.tokens > 1)) {
                    // Slots behind the end may hold anything, and so may tokens
                    // that some row does not see: a zero weight would carry their
                    // NaN and infinities into its sum.  Such values leave the
                    // tile; rows that do see them get them at the item's end.
                    const int place = place0 + place_v(j, n), st = place % C::kSlots;
                    mbar_wait(full + st, (place / C::kSlots) & 1, abort_flag, err, kDevErrTimeoutKv);
                    const int first_new = max(0, w.w.len - pos0), have = min(kKeyTile, keys - pos0);
                    bool odd = false;
                    for (int u = first_new * (D / 8) + st_id; u < kKeyTile * (D / 8); u += kSoftThreads) {
                        const int key = u / (D / 8);
                        const uint32_t at = base + st * C::kTileBytes + unit_at(key, u % (D / 8), kKeyTile);
                        uint32_t v[4] = {0, 0, 0, 0};
                        bool bad = key >= have;
                        if (!bad) {
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                         : "r"(at));
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 t = T::unpack(v[k]);
                                const bool b0 = !isfinite(t.x), b1 = !isfinite(t.y);
                                v[k] &= (b0 ? 0u : 0xffffu) | (b1 ? 0u : 0xffff0000u);
                                bad |= b0 || b1;
                            }
                            odd |= bad;
                        }
                        if (bad) sts_u128(at, make_uint4(v[0], v[1], v[2], v[3]));
                    }
                    if (odd) *odd_flag = 1;
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

            // The row's maximum over its copies and sum over copies and
            // halves.  Buffer it & 1 is the one that the last tile did not
            // use; the other is free once all threads are past that tile.
            float* all_m = maxima + (it & 1) * 2 * kRowTile;
            float* all_l = half == 0 ? all_m + kRowTile : maxima + ((it & 1) ^ 1) * 2 * kRowTile;
            const int at = quad * 32 + lane;
            if (busy && half == 0) all_m[at] = m;
            soft_sync();
            const bool odd_values = *odd_flag != 0;
            float top = m, fix = 1.f;
            if (copies > 1) {
                for (int i = 0; i < copies; ++i) top = fmaxf(top, all_m[(i * spread + quad % spread) * 32 + lane]);
                fix = m == -INFINITY ? 0.f : fast_exp2(m - top);
                if (m != -INFINITY) l *= fix;  // (else nothing was seen: 0, or NaN)
            }
            if (busy) all_l[at] = l;
            soft_sync();
            if (st_id == 0) *odd_flag = 0;
            float sum = 0.f;
            for (int i = 0; i < copies; ++i) {
                const int from = (i * spread + quad % spread) * 32 + lane;
                sum += all_m[kRowTile + from] + maxima[((it & 1) ^ 1) * 2 * kRowTile + from];
            }
            if (odd_values && busy && r < rows) {
#pragma unroll
                for (int i = 0; i < C::kHalfD / 2; ++i) o[i] = make_float2(o[i].x * fix, o[i].y * fix);
                fix = 1.f;
                for (int t = 0; copy == 0 && t < w.w.tokens; ++t) {
                    const int pos = w.w.len + t;
                    if (pos < w.tile0 * kKeyTile || pos >= w.tile1 * kKeyTile ||
                        !sees_new(p, w.w.row0 + tok, tok, t))
                        continue;
                    const int page = page_of(c, b, w.s, pos, err);
                    if (page < 0) continue;
                    const uint16_t* src = c.v + p.layer_offset + page * c.page_stride + w.head * c.head_stride +
                                          (pos & (c.page_size - 1)) * c.slot_stride + half * C::kHalfD;
#pragma unroll
                    for (int i = 0; i < C::kHalfD / 2; ++i) {
                        const float2 v = T::unpack(*reinterpret_cast<const uint32_t*>(src + 2 * i));
                        if (!isfinite(v.x)) o[i].x += v.x;
                        if (!isfinite(v.y)) o[i].y += v.y;
                    }
                }
            }
            if (!w.whole && half == 0 && copy == 0 && r < rows)
                p.part_ml[(int64_t)w.slot * p.slot_rows + r] = make_float2(top, sum);
            // Out through shared memory, 16 channels at a time, so that four
            // lanes write 64 bytes of a row; the copies' warps share the rows
            // and add up the copies.
            const float scale = !w.whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;  // a row that sees nothing: zeros
            const int64_t row_at = w.whole ? (w.w.row0 + tok) * p.out_row_stride +
                                                 ((int64_t)w.head * p.group + my_row % p.group) * D
                                           : ((int64_t)w.slot * p.slot_rows + r) * D;
            float* const out = w.whole ? p.out : p.part_o;
            float* const stage = reinterpret_cast<float*>(smem + C::kOut) + half * 4 * 32 * kStageRow;
#pragma unroll
            for (int ch = 0; ch < C::kHalfD / kStageCols; ++ch) {
                if (busy) {
#pragma unroll
                    for (int i = 0; i < kStageCols / 4; ++i) {
                        const float2 a = o[ch * (kStageCols / 2) + 2 * i], z = o[ch * (kStageCols / 2) + 2 * i + 1];
                        *reinterpret_cast<float4*>(stage + at * kStageRow + 4 * i) =
                            make_float4(a.x * fix, a.y * fix, z.x * fix, z.y * fix);
                    }
                }
                if (copies == 1) __syncwarp();
                else soft_sync();
                if (busy) {
                    const int col = (lane & 3) * 4;
                    for (int i = copy * spread; i < (copy + 1) * spread; ++i) {
                        const int rr = i * 8 + (lane >> 2);  // row of the quadrant
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int k = 0; k < copies; ++k) {
                            const float4 t = *reinterpret_cast<const float4*>(
                                stage + ((k * spread + quad % spread) * 32 + rr) * kStageRow + col);
                            v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
                        }
                        const float f = __shfl_sync(0xffffffffu, scale, rr);
                        float* dst = out + __shfl_sync(0xffffffffu, row_at, rr) + half * C::kHalfD + ch * kStageCols + col;
                        if (quad % spread * 32 + rr < rows &&
                            (!w.whole || bc_global(bc, dst, 16, p.out,
                                                   4 * ((p.rows - 1) * p.out_row_stride +
                                                        (int64_t)p.group * p.kv_heads * D), kBcAttnOut)))
                            *reinterpret_cast<float4*>(dst) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
                    }
                }
                if (copies == 1) __syncwarp();
                else soft_sync();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <int D, class T>
cudaError_t launch_one(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, const CacheView& c,
                       const BatchView& b, int* err, cudaStream_t stream) {
    const cudaError_t e = allow_smem<attention_tc_kernel<D, T>>(TcAttn<D, T>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_chained(attention_tc_kernel<D, T>, dim3((unsigned)p.ctas), dim3(kThreads), TcAttn<D, T>::kSmem, stream,
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
