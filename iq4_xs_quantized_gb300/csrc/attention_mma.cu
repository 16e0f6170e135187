// attention_mma.cu -- tree attention for few rows a key/value head (single
// tokens, short drafts): warp-level MMA (m16n8k16) with the keys on the
// 16-wide side and the rows on the 8-wide one.
//
//   S^T = K Q^T      16 keys x 8 rows a product
//   O^T += V^T P^T   16 channels x 8 rows
//
// Few rows make the cache the whole cost: 4 D bytes a key against 4 D flops
// a row and key, so HBM bounds it and the rest has to stay out of the way.
// That way round a tile of 8 rows costs 8 rows' work (the other way round
// 16), and its output takes D / 4 registers a thread.
//
// Two producer warps stream 64-key tiles of K and of V into shared memory by
// TMA (up to 64 slots of a page a copy, 128-byte swizzle).  Two sets of four
// consumer warps (one where the outputs take more registers) take the tiles
// in turn, each from a ring of its own, K0 V0 K1 V1 ..., and each warp 16
// keys of the tile, with a running maximum, sum and output of its own: no
// warp waits for another until the item ends.  (A ring of its own, because a
// parity wait cannot tell a phase from the next but one: a set must see every
// phase of the barriers that it waits on.)  The weights go from the first
// product's accumulators to the second one's B operand by 8 x 8 transposes in
// registers, as the sum of 16-bit parts (two for fp16, three for bf16), so
// that rounding them costs less than fp32 accumulation does.
//
// Measured: one new token of 24 sequences of 8,191, 32 heads over 8 of 128,
// bf16: 605 MB in 100 us, 6.0 TB/s, 89 % of a copy's rate (tensor pipe 14 %
// busy, the warps wait for K and V).  64 channels and pages of 16 slots stop at
// about 4.2 TB/s: a copy is 2 KB there, and the copy unit's rate binds.  One
// token over 517 cached, 24 heads over 4 of 256: 9.0 us by clusters, latency.
// 16 rows at 128 channels, in two sets, do not fit the registers: ptxas spills
// up to 174 bytes a thread there (the other forms at most 42).
#include "attention.cuh"

namespace iq4xs {
namespace {

constexpr int kKeyTile = MmaForm<1>::kKeys;
constexpr int kSetWarps = 4;
constexpr int kWarpKeys = kKeyTile / kSetWarps;
static_assert(kWarpKeys == 16, "a warp's keys are one k16 step of the second product");

template <int D, int NT>
struct MmaAttn {
    static constexpr int kRows = MmaForm<NT>::kRows;
    static constexpr int kTileBytes = kKeyTile * D * 2;      // K or V of a tile
    static constexpr int kSets = NT * D <= 256 ? 2 : 1;
    static constexpr int kConsumers = kSetWarps * kSets;
    static constexpr int kThreads = 32 * (kConsumers + 2);
    static constexpr int kSlots = 192 * 1024 / kSets / kTileBytes;  // of a set's ring: 3 (6 in one set), 6, 12
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kJoinCols = NT == 1 ? 64 : 32;      // channels of the warps' outputs joined at a time
    static constexpr int kJoinPitch = kJoinCols + 4;         // (conflict-free for the fragments' rows and channels)
    static constexpr int kJoinBytes = kConsumers * kRows * kJoinPitch * 4;
    // a CTA's last item joins whole rows in the ring, which nothing fills any
    // more, and a cluster's parts meet behind them
    static constexpr int kLastPitch = D + 4;
    static constexpr int kPart = kConsumers * kRows * kLastPitch * 4;
    static_assert(kPart + kRows * D * 4 <= kSets * kSlots * kTileBytes, "last join in the ring");
    static constexpr int kQ = kSets * kSlots * kTileBytes;
    static constexpr int kJoin = kQ + kQBytes;
    static constexpr int kMl = kJoin + kJoinBytes;           // per warp and row: max, sum; then joined
    static constexpr int kBars = kMl + (kConsumers + 1) * kRows * 8;
    static constexpr int kSmem = kBars + 2 * kSets * kSlots * 8 + 16;
    static constexpr bool kQInRegs = NT == 1;
    static_assert(kSets * kSlots <= 32, "a lane keeps a slot's last place");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 8 x 8 transpose of 16-bit values held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <class T>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<KvF16>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<KvBf16>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int kConsumers>
__device__ __forceinline__ void consumers_meet() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
}

// Offset of unit u (8 channels) of row r of a strip (which starts at a
// multiple of 8 rows of its box, so that r alone gives the swizzle).
__device__ __forceinline__ uint32_t strip_unit(int r, int u, uint32_t chunk_stride) {
    return (uint32_t)(u >> 3) * chunk_stride + r * kChunkBytes + (((u & 7) ^ (r & 7)) << 4);
}
// All threads of the cluster; what they wrote before is seen after.
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    cluster_arrive_release();
    cluster_wait();
}
// What CTA `rank` of the cluster has at the place of `at` in this one.
__device__ __forceinline__ float2 cluster_read(const float2* at, int rank) {
    uint32_t a;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_read(const float4* at, int rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
// Four channels of an item's row r: the joined sums over the row's total.
template <class Walk>
__device__ __forceinline__ void put_row(const AttnParams& p, const CacheView& c, const Walk& w, int r, int channel,
                                        float4 v, float sum, const Bc& bc) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that sees nothing: zeros
    const int row = w.row_tile * Walk::kRows + r, t = token_of(p, row), D = c.head_dim;
    float* dst = p.out + (w.w.row0 + t) * p.out_row_stride + ((int64_t)w.head * p.group + row - t * p.group) * D +
                 channel;
    if (bc_global(bc, dst, 16, p.out, 4 * ((p.rows - 1) * p.out_row_stride + (int64_t)p.group * p.kv_heads * D),
                  kBcAttnOut))
        *reinterpret_cast<float4*>(dst) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
}

// Keys `have` .. 15 of a warp's V strip become zero, and so does every key
// that holds NaN or infinities when `hidden` (some row does not see all of the
// strip): a zero weight would carry such values into rows that do not see
// them.  Rows that do see such a key get its share here, from e, the weights
// (x = -inf: not seen).  A lane has channels ch, ch + 8 and rows 2 ct, 2 ct +
// 1 of every 16 x 8 output tile.
template <int D, class T, int NT>
__device__ __forceinline__ void scrub_strip(uint32_t v_s, uint32_t chunk_stride, int have, bool hidden, const float (*x)[4],
                                            const float (*e)[4], float (*o)[NT][4]) {
    const int lane = threadIdx.x & 31, rg = lane >> 2, ct = lane & 3;
    for (int key = 0; key < kWarpKeys; ++key) {
        bool odd = key >= have;
        if (!odd && hidden) {
            for (int u = lane; u < D / 8; u += 32) {
                uint32_t v[4];
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                             : "r"(v_s + strip_unit(key, u, chunk_stride)));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = T::unpack(v[i]);
                    odd |= !isfinite(f.x) || !isfinite(f.y);
                }
            }
            odd = __any_sync(0xffffffffu, odd);
            if (odd) {
                const int src = (key & 7) * 4 + ct;
                float pk[NT][2], xk[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        pk[n][r] = __shfl_sync(0xffffffffu, key < 8 ? e[n][r] : e[n][2 + r], src);
                        xk[n][r] = __shfl_sync(0xffffffffu, key < 8 ? x[n][r] : x[n][2 + r], src);
                    }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    float v[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t w = lds_u32_ordered(v_s + strip_unit(key, 2 * i + k, chunk_stride) + (rg >> 1) * 4);
                        v[k] = T::unpack(rg & 1 ? w >> 16 : w & 0xffffu).x;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            if (xk[n][r] != -INFINITY) {
                                o[i][n][r] = fmaf(pk[n][r], v[0], o[i][n][r]);
                                o[i][n][2 + r] = fmaf(pk[n][r], v[1], o[i][n][2 + r]);
                            }
                }
            }
        }
        __syncwarp();
        if (odd)
            for (int u = lane; u < D / 8; u += 32) sts_u128(v_s + strip_unit(key, u, chunk_stride), make_uint4(0, 0, 0, 0));
    }
    __syncwarp();
    fence_proxy_async_smem();  // these writes come before the slot's next copy
}

template <int D, class T, int NT>
__global__ void __launch_bounds__(MmaAttn<D, NT>::kThreads, 1)
    attention_mma_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                         const __grid_constant__ AttnParams p, const __grid_constant__ CacheView c,
                         const __grid_constant__ BatchView b, int* err) {
    using C = MmaAttn<D, NT>;
    using F = MmaForm<NT>;
    constexpr int kConsumers = C::kConsumers;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    if ((base & 1023) != 0) {  // (no static shared memory: the swizzle atoms' alignment)
        if (threadIdx.x == 0) atomicCAS(err, 0, kDevErrLayout);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);  // [set][slot]
    uint64_t* slot_free = full + C::kSets * C::kSlots;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(slot_free + C::kSets * C::kSlots);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = blockIdx.x / p.cluster;
    const Bc bc = bc_open(err);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSets * C::kSlots; ++i) {
            mbar_init(full + i, 1);
            mbar_init(slot_free + i, kSetWarps);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kConsumers && lane == 0) {
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    __syncthreads();
    griddep_wait();  // lengths, tables, q and the cache's newest rows come from earlier launches
    griddep_launch_dependents();
    WorkWalk<F> w;
    w.start(p, b, g, err);
    // A cluster shares one item, an eighth of its key tiles a CTA.  It takes
    // one alone, and there are as many clusters as items, unless row offsets
    // fall (recorded), so that sequences overlap: items past the clusters are
    // left out, for the ring of the first one is where its parts meet.
    const int rank = p.cluster > 1 ? (int)cluster_ctarank() : 0;
    if (threadIdx.x == 0 && !p.whole_items) w.tell_cut(p, g);
    if (p.cluster > 1 && w.valid()) {
        const int tiles = w.w.key_tiles;
        w.tile0 = rank * tiles / p.cluster;
        w.tile1 = (rank + 1) * tiles / p.cluster;
        w.whole = false;
        w.left = 1;
    }

    if (warp >= kConsumers) {
        // ----------------------------------------------- producers: K, then V
        const int kv = warp - kConsumers;
        const void* map = kv ? &tv : &tk;
        const int boxes = kKeyTile / p.box_slots;  // a lane copies one
        const uint32_t box_bytes = p.box_slots * D * 2;
        const uint32_t dst0 = base + lane * box_bytes;
        PageWindow pages;
        int it = 0, last = -1;  // tiles so far; the last place loaded into slot `lane`
        bool live = true;
        const bool in_cluster = p.cluster > 1 && w.valid();
        for (; live && w.valid(); w.next(p, b, g, err)) {
            const int end = w.seen_tiles(p);
            const int keys = w.w.len + w.w.tokens;
            pages.open(b, w.s);
            for (int tile = w.tile0; live && tile < end; ++tile, ++it) {
                const int pos0 = tile * kKeyTile, pos = pos0 + lane * p.box_slots;
                pages.move(pos0 >> c.page_shift, lane);
                int page = pages.id(pos >> c.page_shift);
                // boxes that hold a key: those of slots at or behind the end stay out
                const int used = min(boxes, (keys - pos0 + p.box_slots - 1) / p.box_slots);
                if (lane < used && (page < 0 || page >= c.pages)) {
                    data_error(err, kDataPage);
                    page = c.pages;  // outside the map: zeros
                }
                const int slot = pos & (c.page_size - 1);
                bc_tma(bc, 0, 2, 64, 64, slot, c.page_size, kBcAttnKv, kBcAttnKv);
                const int place = it / C::kSets * 2 + kv, st = it % C::kSets * C::kSlots + place % C::kSlots;
                live = place < C::kSlots || warp_wait(slot_free + st, (place / C::kSlots - 1) & 1, abort_flag, err,
                                                      kDevErrTimeoutKvSlot);
                if (!live || it == p.skip_stage) continue;
                if (lane == 0) mbar_arrive_expect_tx(full + st, used * box_bytes);
                if (lane == st) last = place;
                __syncwarp();
                if (lane < used) tma_load_kv(dst0 + st * C::kTileBytes, map, slot, 0, w.head, page, full + st);
                __syncwarp();
            }
        }
        // No copy may be in flight when the CTA ends; the consumers wait for
        // every one, unless a wait ran out.
        if (*abort_flag)
            for (int i = 0; i < C::kSets * C::kSlots; ++i) {
                const int place = __shfl_sync(0xffffffffu, last, i);
                int no_abort = 0;
                if (place >= 0)
                    mbar_wait(full + i, (place / C::kSlots) & 1, &no_abort, err, kDevErrTimeoutKv);
            }
        if (in_cluster) {  // (the consumers' two meetings count every thread)
            cluster_meet();
            cluster_meet();
        }
        return;
    }

    // ------------------------------------------------------------ consumers
    constexpr int kRows = C::kRows;
    const uint32_t q_s = base + C::kQ;
    float* join = reinterpret_cast<float*>(smem + C::kJoin);
    float2* ml = reinterpret_cast<float2*>(smem + C::kMl);
    const int rg = lane >> 2, ct = lane & 3;           // fragment row (key or channel) and column pair (rows)
    const int set = warp / kSetWarps, strip = warp % kSetWarps * kWarpKeys;
    // the strip's rows in a tile of [box][chunk][slot][128 bytes]
    const uint32_t chunk_stride = p.box_slots * kChunkBytes;
    const uint32_t strip_at = strip / p.box_slots * p.box_slots * D * 2 + strip % p.box_slots * kChunkBytes;
    const auto consumer_sync = [] { consumers_meet<kConsumers>(); };
    int it = 0;
    bool live = true;  // no wait has run out: after that a warp waits for nothing and arrives nowhere
    for (; w.valid(); w.next(p, b, g, err)) {
        const int end = w.seen_tiles(p);
        const int rows = min(kRows, w.w.tokens * p.group - w.row_tile * kRows);
        const int keys = w.w.len + w.w.tokens;
        // q of the item's rows (behind the last row the last one again,
        // instead of a branch: all loads are in flight together)
        constexpr int kQUnits = (kRows * (D / 8) + 32 * kConsumers - 1) / (32 * kConsumers);
        uint4 qv[kQUnits];
#pragma unroll
        for (int i = 0; i < kQUnits; ++i) {
            const int u = threadIdx.x + i * 32 * kConsumers, col = u % (D / 8);
            const int row = w.row_tile * kRows + min(u / (D / 8), rows - 1), t = token_of(p, row);
            const uint16_t* src = p.q + (w.w.row0 + t) * p.q_row_stride +
                                  ((int64_t)w.head * p.group + row - t * p.group) * D + col * 8;
            qv[i] = make_uint4(0, 0, 0, 0);
            if (bc_global(bc, src, 16, p.q,
                          2 * ((p.rows - 1) * p.q_row_stride + (int64_t)p.group * p.kv_heads * D), kBcAttnQ))
                qv[i] = *reinterpret_cast<const uint4*>(src);
        }
        int tok[NT][2];  // the tokens of the lane's rows 8 n + 2 ct + r (behind the last: the last)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                tok[n][r] = min(w.w.tokens - 1, token_of(p, w.row_tile * kRows + 8 * n + 2 * ct + r));
#pragma unroll
        for (int i = 0; i < kQUnits; ++i) {
            const int u = threadIdx.x + i * 32 * kConsumers;
            if (u < kRows * (D / 8)) sts_u128(q_s + unit_at(u / (D / 8), u % (D / 8), kRows), sign_q(p, qv[i]));
        }
        consumer_sync();
        // B operand of k16 steps 2 k, 2 k + 1 and rows 8 n ..: four 8 x 8 blocks
        auto q_frag = [&](int k, int n, uint32_t* f) {
            ldsm4(q_s + unit_at(8 * n + (lane & 7), 4 * k + (lane >> 3), kRows), f);
        };
        uint32_t qf[C::kQInRegs ? D / 32 : 1][C::kQInRegs ? NT : 1][4];
        if constexpr (C::kQInRegs) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n) q_frag(k, n, qf[k][n]);
        }

        float o[D / 16][NT][4];  // channels 16 i + rg, + 8; rows 8 n + 2 ct, + 1
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }

        for (int tile = w.tile0; tile < end; ++tile, ++it) {
            if (it % C::kSets != set || !live) continue;
            const int k_place = it / C::kSets * 2, v_place = k_place + 1;
            const int k_st = set * C::kSlots + k_place % C::kSlots, v_st = set * C::kSlots + v_place % C::kSlots;
            const uint32_t k_s = base + k_st * C::kTileBytes + strip_at, v_s = base + v_st * C::kTileBytes + strip_at;
            const auto k_done = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(slot_free + k_st);
            };
            const auto v_wait = [&] {
                live = warp_wait(full + v_st, (v_place / C::kSlots) & 1, abort_flag, err, kDevErrTimeoutKv);
                return live;
            };
            const int key0 = tile * kKeyTile + strip;       // the warp's first position
            const int have = min(kWarpKeys, keys - key0);   // its positions before the end
            live = warp_wait(full + k_st, (k_place / C::kSlots) & 1, abort_flag, err, kDevErrTimeoutKv);
            if (!live) continue;
            if (have > 0) {
                float s[2][NT][4];  // [even, odd k step]
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[i][n][0] = s[i][n][1] = s[i][n][2] = s[i][n][3] = 0.f;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t kf[2][4];
                    ldsm4(k_s + strip_unit(lane & 15, 4 * k + (lane >> 4), chunk_stride), kf[0]);
                    ldsm4(k_s + strip_unit(lane & 15, 4 * k + 2 + (lane >> 4), chunk_stride), kf[1]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t qt[4];
                        const uint32_t* f = qt;
                        if constexpr (C::kQInRegs) f = qf[k][n];
                        else q_frag(k, n, qt);
                        mma16816<T>(s[0][n], kf[0], f[0], f[1]);
                        mma16816<T>(s[1][n], kf[1], f[2], f[3]);
                    }
                }
                k_done();
                float x[NT][4];  // keys rg (rows 2 ct, 2 ct + 1), rg + 8 (the same rows)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[n][i] = (s[0][n][i] + s[1][n][i]) * p.scale_log2;
                bool hidden = false;  // a new token of this strip that some row does not see
                if (key0 + kWarpKeys > w.w.len) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = rg + (i >> 1) * 8, j = key0 + key - w.w.len, t = tok[n][i & 1];
                            const bool inside = key < have;
                            const bool see = inside && (j < 0 || sees_new(p, w.w.row0 + t, t, j, bc));
                            hidden |= inside && !see;
                            if (!see) x[n][i] = -INFINITY;
                        }
                    hidden = __any_sync(0xffffffffu, hidden);
                }
                // running maximum (lazily) and weights
                float mx[NT][2];
                bool rise = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float t = fmaxf(x[n][r], x[n][2 + r]);
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                        mx[n][r] = t;
                        rise |= t > m[n][r] + kLazy;
                    }
                if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const bool up = mx[n][r] > m[n][r] + kLazy;
                            const float f = up ? fast_exp2(m[n][r] - mx[n][r]) : 1.f;
                            m[n][r] = up ? mx[n][r] : m[n][r];
                            l[n][r] *= f;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                o[i][n][r] *= f;
                                o[i][n][2 + r] *= f;
                            }
                        }
                }
                float e[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float shift = m[n][r] == -INFINITY ? 0.f : kWeightBits - m[n][r];
                        e[n][r] = fast_exp2(x[n][r] + shift);
                        e[n][2 + r] = fast_exp2(x[n][2 + r] + shift);
                        l[n][r] += e[n][r] + e[n][2 + r];
                    }

                if (!v_wait()) continue;
                if (hidden || have < kWarpKeys) scrub_strip<D, T, NT>(v_s, chunk_stride, have, hidden, x, e, o);
                uint32_t pf[Parts<T>::kN][NT][2];  // B operand: keys 2 ct, 2 ct + 1 (+ 8), row rg
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t part[Parts<T>::kN];
                        Parts<T>::split(make_float2(e[n][2 * h], e[n][2 * h + 1]), part);
#pragma unroll
                        for (int i = 0; i < Parts<T>::kN; ++i) pf[i][n][h] = transpose8(part[i]);
                    }
                const int vr = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t vf[4];
                    ldsm4_t(v_s + strip_unit(vr, 2 * i + ((lane >> 3) & 1), chunk_stride), vf);
                    // A product of its own, smallest parts first, added to o by
                    // rounded fp32 adds: the MMA cuts its sums off instead of
                    // rounding them, which over thousands of tiles would lean
                    // all to one side (4e-5 of the result at 131k tokens).
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = Parts<T>::kN - 1; k >= 0; --k) {
                            mma16816<T>(t, vf, pf[k][n][0], pf[k][n][1]);
                            if (Parts<T>::kLastShift > 0 && k == Parts<T>::kN - 1) {
                                constexpr float kDown = 1.0f / (1 << Parts<T>::kLastShift);
                                t[0] *= kDown; t[1] *= kDown; t[2] *= kDown; t[3] *= kDown;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[i][n][k] += t[k];
                    }
                }
            } else {
                k_done();
                if (!v_wait()) continue;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(slot_free + v_st);
        }

        // Join the warps' results.
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float t = l[n][r];
                t += __shfl_xor_sync(0xffffffffu, t, 4);
                t += __shfl_xor_sync(0xffffffffu, t, 8);
                t += __shfl_xor_sync(0xffffffffu, t, 16);
                if (rg == 0) ml[warp * kRows + 8 * n + 2 * ct + r] = make_float2(m[n][r], t);
            }
        consumer_sync();
        float f[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 8 * n + 2 * ct + r;
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int i = 0; i < kConsumers; ++i) top = fmaxf(top, ml[i * kRows + row].x);
#pragma unroll
                for (int i = 0; i < kConsumers; ++i) {
                    const float2 t = ml[i * kRows + row];
                    // (a maximum of -inf: the warp saw nothing, sum 0, or only NaN)
                    sum += t.x == -INFINITY ? t.y : t.y * fast_exp2(t.x - top);
                }
                f[n][r] = m[n][r] == -INFINITY ? 0.f : fast_exp2(m[n][r] - top);
                if (warp == 0 && rg == 0) {
                    ml[kConsumers * kRows + row] = make_float2(top, sum);
                    if (!w.whole && p.cluster == 1 && row < rows)
                        if (float2* to = part_sum(p, w.slot, row, bc)) *to = make_float2(top, sum);
                }
            }
        const bool last = w.last();
        constexpr int kCols = C::kJoinCols;
        float* const buf = last ? reinterpret_cast<float*>(smem) : join;
        const int pitch = last ? C::kLastPitch : C::kJoinPitch;
        float* const part = reinterpret_cast<float*>(smem + C::kPart);  // this CTA's part of a cluster's item
        // Adds up `cols` joined channels from channel c0 on and puts them where they belong.
        const auto put = [&](int c0, int cols) {
            for (int u = threadIdx.x; u < rows * (cols / 4); u += 32 * kConsumers) {
                const int r = u / (cols / 4), col = u % (cols / 4) * 4;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kConsumers; ++i) {
                    const float4 t = *reinterpret_cast<const float4*>(buf + (i * kRows + r) * pitch + col);
                    v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
                }
                if (p.cluster > 1) {
                    *reinterpret_cast<float4*>(part + r * D + col) = v;
                } else if (w.whole) {
                    put_row(p, c, w, r, c0 + col, v, ml[kConsumers * kRows + r].y, bc);
                } else {
                    if (float* to = part_row(p, w.slot, r, c0 + col, 4, bc)) *reinterpret_cast<float4*>(to) = v;
                }
            }
        };
#pragma unroll
        for (int ch = 0; ch < D / kCols; ++ch) {
            if (ch > 0 && !last) consumer_sync();
#pragma unroll
            for (int i = 0; i < kCols / 16; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        buf[(warp * kRows + 8 * n + 2 * ct + (k & 1)) * pitch + (last ? ch * kCols : 0) + 16 * i + rg +
                            (k >> 1) * 8] = o[ch * (kCols / 16) + i][n][k] * f[n][k & 1];
            if (!last) {
                consumer_sync();
                put(ch * kCols, kCols);
            }
        }
        consumer_sync();
        if (last) put(0, D);
        if (p.cluster > 1) {
            cluster_meet();
            // every CTA joins its share of the item's values from all parts
            const float2* const my_ml = ml + kConsumers * kRows;
            for (int u = rank * 32 * kConsumers + threadIdx.x; u < rows * (D / 4); u += p.cluster * 32 * kConsumers) {
                const int r = u / (D / 4), col = u % (D / 4) * 4;
                float2 t[kMaxCluster];
                float4 v[kMaxCluster];
#pragma unroll
                for (int i = 0; i < kMaxCluster; ++i) {
                    t[i] = make_float2(-INFINITY, 0.f);
                    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < p.cluster) {
                        t[i] = cluster_read(my_ml + r, i);
                        v[i] = cluster_read(reinterpret_cast<const float4*>(part + r * D + col), i);
                    }
                }
                float top = -INFINITY, sum = 0.f;
                float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kMaxCluster; ++i) top = fmaxf(top, t[i].x);
#pragma unroll
                for (int i = 0; i < kMaxCluster; ++i) {
                    const float a = t[i].x == -INFINITY ? t[i].y : fast_exp2(t[i].x - top);  // (nothing seen: 0, or NaN)
                    sum += t[i].x == -INFINITY ? t[i].y : t[i].y * a;
                    all.x = fmaf(v[i].x, a, all.x);
                    all.y = fmaf(v[i].y, a, all.y);
                    all.z = fmaf(v[i].z, a, all.z);
                    all.w = fmaf(v[i].w, a, all.w);
                }
                put_row(p, c, w, r, col, all, sum, bc);
            }
            cluster_meet();  // no CTA ends while another reads its part
            return;
        }
    }
}

template <int D, class T, int NT>
cudaError_t launch_one(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, const CacheView& c,
                       const BatchView& b, int* err, cudaStream_t stream) {
    const cudaError_t e = allow_smem<attention_mma_kernel<D, T, NT>>(MmaAttn<D, NT>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_chained(attention_mma_kernel<D, T, NT>, dim3((unsigned)(p.ctas * p.cluster)),
                          dim3(MmaAttn<D, NT>::kThreads), MmaAttn<D, NT>::kSmem, stream, p.cluster, tk, tv, p, c, b, err);
}

template <int D, class T>
cudaError_t launch_width(int row_tile, const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CacheView& c, const BatchView& b, int* err, cudaStream_t stream) {
    if (row_tile == 8) return launch_one<D, T, 1>(p, tk, tv, c, b, err, stream);
    if (row_tile == 16) return launch_one<D, T, 2>(p, tk, tv, c, b, err, stream);
    return cudaErrorInvalidValue;
}

template <class T>
cudaError_t launch_type(int row_tile, const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                        const CacheView& c, const BatchView& b, int* err, cudaStream_t stream) {
    switch (c.head_dim) {
        case 64: return launch_width<64, T>(row_tile, p, tk, tv, c, b, err, stream);
        case 128: return launch_width<128, T>(row_tile, p, tk, tv, c, b, err, stream);
        case 256: return launch_width<256, T>(row_tile, p, tk, tv, c, b, err, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_attention_mma(int row_tile, const AttnParams& p, const void* tk, const void* tv, const CacheView& c,
                                 const BatchView& b, bool bf16, int* err, cudaStream_t stream) {
    const CUtensorMap& mk = *static_cast<const CUtensorMap*>(tk);
    const CUtensorMap& mv = *static_cast<const CUtensorMap*>(tv);
    return bf16 ? launch_type<KvBf16>(row_tile, p, mk, mv, c, b, err, stream)
                : launch_type<KvF16>(row_tile, p, mk, mv, c, b, err, stream);
}

}  // namespace iq4xs
