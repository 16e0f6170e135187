// attention_mma.cu -- tree attention for few rows a key/value head (single
// tokens, short drafts): warp-level MMA (m16n8k16) on 16-row tiles.
//
// Few rows make the cache the whole cost: 4 D bytes a key against 4 D flops
// a row and key, so HBM bounds it and the rest has to stay out of the way.
// One producer warp streams 64-key tiles of K and V through a ring in shared
// memory by TMA (boxes of 64 channels x a page's slots, 128-byte swizzle);
// four consumer warps own 16 keys of every tile each, with a running maximum,
// sum and 16 x D output of their own, so that no warp waits for another until
// the item ends: scores stay in the MMA's accumulator layout, which is the
// next MMA's A operand.
//
// Weights go into the second product as the sum of 16-bit parts (two for
// fp16, three for bf16: hi = round(w), lo = round(w - hi), ...), so that
// rounding them costs less than fp32 accumulation does.
#include "attention.cuh"

namespace iq4xs {
namespace {

constexpr int kRowTile = MmaForm::kRows, kKeyTile = MmaForm::kKeys;
constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kWarpKeys = kKeyTile / kConsumers;
static_assert(kWarpKeys == 16, "a warp's keys are one k16 step of the second product");

template <int D>
struct MmaAttn {
    static constexpr int kChunks = D / 64;
    static constexpr int kTileBytes = kKeyTile * D * 2;      // K or V of a tile
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kCtas = D == 256 ? 1 : 2;           // resident a SM
    static constexpr int kStages = D == 256 ? 3 : D == 128 ? 3 : 6;
    static constexpr int kQBytes = kRowTile * D * 2;
    static constexpr int kJoinCols = 32;                     // channels of the warps' outputs joined at a time
    static constexpr int kJoinBytes = kConsumers * kRowTile * kJoinCols * 4;
    static constexpr int kJoin = kStages * kStageBytes + kQBytes;
    static constexpr int kMl = kJoin + kJoinBytes;           // per warp and row: max, sum; then joined
    static constexpr int kBars = kMl + (kConsumers + 1) * kRowTile * 8;
    static constexpr int kSmem = kBars + 3 * kStages * 8 + 16 + 1024;  // + alignment
    static constexpr bool kQInRegs = D <= 64;
    static_assert(kSmem <= (kCtas == 1 ? 227 : 113) * 1024, "shared memory of the resident CTAs");
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
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
static_assert(kConsumers * 32 == 128, "the consumers' barrier");

template <int D, class T>
__global__ void __launch_bounds__(kThreads, MmaAttn<D>::kCtas)
    attention_mma_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                         const AttnParams p, const CacheView c, const BatchView b, int* err) {
    using C = MmaAttn<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);  // swizzle atoms
    const uint32_t base = smem_u32(smem);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kBars);
    uint64_t* v_full = k_full + C::kStages;
    uint64_t* slot_free = v_full + C::kStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(slot_free + C::kStages);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = blockIdx.x;
    const Bc bc = bc_open(err);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(k_full + i, 1);
            mbar_init(v_full + i, 1);
            mbar_init(slot_free + i, kConsumers);
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
    WorkWalk<MmaForm> w;
    w.start(p, b, g, err);

    if (warp == kConsumers) {
        // ---------------------------------------------------------- producer
        const int box_slots = min(c.page_size, kKeyTile);
        const int boxes = kKeyTile / box_slots * C::kChunks;  // of K (or V) a full tile
        const uint32_t box_bytes = box_slots * kChunkBytes;
        int it = 0;
        bool live = true;
        for (; live && w.valid(); w.next(p, b, g, err)) {
            const int end = w.seen_tiles(p);
            const int keys = w.w.len + w.w.tokens;
            const int held = min(b.held[w.s], b.table_width);
            const int32_t* table = b.page_table + w.s * b.table_stride;
            // Page ids of 32 pages from page0 on, one a lane, the next 32 on their way.
            int page0 = (w.tile0 * kKeyTile) >> c.page_shift;
            int ids = page0 + lane < held ? table[page0 + lane] : -1;
            int ids2 = page0 + 32 + lane < held ? table[page0 + 32 + lane] : -1;
            for (int tile = w.tile0; tile < end; ++tile, ++it) {
                const int st = it % C::kStages, pos0 = tile * kKeyTile;
                if (it >= C::kStages && !warp_wait(slot_free + st, ((it / C::kStages) - 1) & 1, abort_flag, err,
                                                   kDevErrTimeoutKvSlot)) {
                    live = false;
                    break;
                }
                while ((pos0 >> c.page_shift) >= page0 + 32) {
                    page0 += 32;
                    ids = ids2;
                    ids2 = page0 + 32 + lane < held ? table[page0 + 32 + lane] : -1;
                }
                // boxes that hold a key: those of slots at or behind the end stay out
                const int used = min(boxes, (min(kKeyTile, keys - pos0) + box_slots - 1) / box_slots * C::kChunks);
                const bool skip = it == p.skip_stage;
                if (lane == 0 && !skip) {
                    mbar_arrive_expect_tx(k_full + st, used * box_bytes);
                    mbar_arrive_expect_tx(v_full + st, used * box_bytes);
                }
                __syncwarp();
                for (int i0 = 0; i0 < used; i0 += 32) {
                    const int i = i0 + lane;
                    const int sub = i / C::kChunks, chunk = i % C::kChunks;
                    const int pos = pos0 + sub * box_slots;
                    int page = __shfl_sync(0xffffffffu, ids, ((pos >> c.page_shift) - page0) & 31);
                    if (i < used && !skip) {
                        if (page < 0 || page >= c.pages) {
                            data_error(err, kDataPage);
                            page = c.pages;  // outside the map: zeros
                        }
                        const int slot = pos & (c.page_size - 1);
                        const int y = p.slot_axis == 1 ? slot : w.head, z = p.slot_axis == 1 ? w.head : slot;
                        const uint32_t dst = base + st * C::kStageBytes + chunk * kKeyTile * kChunkBytes +
                                             sub * box_bytes;
                        bc_tma(bc, chunk * 64, 2, 64, D, slot, c.page_size, kBcAttnKv, kBcAttnKv);
                        tma_load_4d(dst, &tk, chunk * 64, y, z, page, k_full + st);
                        tma_load_4d(dst + C::kTileBytes, &tv, chunk * 64, y, z, page, v_full + st);
                    }
                }
                __syncwarp();
            }
        }
        // No copy may be in flight when the CTA ends; the consumers wait for
        // every stage, unless a wait ran out.
        if (*abort_flag) {
            for (int i = max(0, it - C::kStages); i < it; ++i)
                if (i != p.skip_stage) {
                    int no_abort = 0;
                    mbar_wait(k_full + i % C::kStages, (i / C::kStages) & 1, &no_abort, err, kDevErrTimeoutKv);
                    kv_wait(v_full + i % C::kStages, (i / C::kStages) & 1, &no_abort, err, kDevErrTimeoutKv);
                }
        }
        return;
    }

    // ------------------------------------------------------------ consumers
    const uint32_t q_s = base + C::kStages * C::kStageBytes;
    float* join = reinterpret_cast<float*>(smem + C::kJoin);
    float2* ml = reinterpret_cast<float2*>(smem + C::kMl);
    const int rg = lane >> 2, ct = lane & 3;  // fragment row and column pair
    int it = 0;
    for (; w.valid(); w.next(p, b, g, err)) {
        const int end = w.seen_tiles(p);
        const int rows = min(kRowTile, w.w.tokens * p.group - w.row_tile * kRowTile);
        const int keys = w.w.len + w.w.tokens;
        // q of the item's rows
        constexpr int kQUnits = kRowTile * (D / 8) / (32 * kConsumers);
        uint4 qv[kQUnits];
#pragma unroll
        for (int i = 0; i < kQUnits; ++i) {
            // (behind the last row the last one again, instead of a branch:
            // all loads are in flight together)
            const int u = threadIdx.x + i * 32 * kConsumers, col = u % (D / 8);
            const int row = w.row_tile * kRowTile + min(u / (D / 8), rows - 1), t = token_of(p, row);
            const uint16_t* src = p.q + (w.w.row0 + t) * p.q_row_stride +
                                  ((int64_t)w.head * p.group + row - t * p.group) * D + col * 8;
            qv[i] = make_uint4(0, 0, 0, 0);
            if (bc_global(bc, src, 16, p.q,
                          2 * ((p.rows - 1) * p.q_row_stride + (int64_t)p.group * p.kv_heads * D), kBcAttnQ))
                qv[i] = *reinterpret_cast<const uint4*>(src);
        }
#pragma unroll
        for (int i = 0; i < kQUnits; ++i) {
            const int u = threadIdx.x + i * 32 * kConsumers;
            sts_u128(q_s + unit_at(u / (D / 8), u % (D / 8), kRowTile), sign_q(p, qv[i]));
        }
        consumer_sync();
        uint32_t qf[C::kQInRegs ? D / 16 : 1][4];
        const uint32_t q_row = q_s;
        if constexpr (C::kQInRegs) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) ldsm4(q_row + unit_at(lane & 15, 2 * k + (lane >> 4), kRowTile), qf[k]);
        }

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows rg, rg + 8
        int tok[2];  // the rows' tokens (rows behind the last: the last token)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            tok[i] = min(w.w.tokens - 1, token_of(p, w.row_tile * kRowTile + rg + 8 * i));

        for (int tile = w.tile0; tile < end; ++tile, ++it) {
            const int st = it % C::kStages, par = (it / C::kStages) & 1;
            const uint32_t k_s = base + st * C::kStageBytes, v_s = k_s + C::kTileBytes;
            const int key0 = tile * kKeyTile + warp * kWarpKeys;  // the warp's first position
            const int have = min(kWarpKeys, keys - key0);          // its positions before the end
            kv_wait(k_full + st, par, abort_flag, err, kDevErrTimeoutKv);
            if (have > 0) {
                float s[2][2][4];  // [even, odd k step][8 keys][fragment]
#pragma unroll
                for (int i = 0; i < 16; ++i) (&s[0][0][0])[i] = 0.f;
                const int kr = warp * kWarpKeys + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t kf[4];
                    ldsm4(k_s + unit_at(kr, 2 * k + ((lane >> 3) & 1), kKeyTile), kf);
                    uint32_t qt[4];
                    const uint32_t* a = qt;
                    if constexpr (C::kQInRegs) a = qf[k];
                    else ldsm4(q_row + unit_at(lane & 15, 2 * k + (lane >> 4), kRowTile), qt);
                    mma16816<T>(s[k & 1][0], a, kf[0], kf[1]);
                    mma16816<T>(s[k & 1][1], a, kf[2], kf[3]);
                }
                float x[2][4];  // [row][key: 2 ct, 2 ct + 1, 8 + 2 ct, 8 + 2 ct + 1]
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[r][k] = (s[0][k >> 1][2 * r + (k & 1)] + s[1][k >> 1][2 * r + (k & 1)]) * p.scale_log2;
                bool hidden = false;  // a new token of this strip that some row does not see
                if (key0 + kWarpKeys > w.w.len) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int key = (k >> 1) * 8 + 2 * ct + (k & 1), j = key0 + key - w.w.len;
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const bool inside = key < have;
                            const bool see = inside && (j < 0 || sees_new(p, w.w.row0 + tok[r], tok[r], j));
                            hidden |= inside && !see;
                            if (!see) x[r][k] = -INFINITY;
                        }
                    }
                    hidden = __any_sync(0xffffffffu, hidden);
                }
                // running maximum (lazily) and weights
                float mx[2];
                bool rise = false;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    mx[r] = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
                    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
                    rise |= mx[r] > m[r] + kLazy;
                }
                if (__any_sync(0xffffffffu, rise)) {
                    float f[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const bool up = mx[r] > m[r] + kLazy;
                        f[r] = up ? fast_exp2(m[r] - mx[r]) : 1.f;
                        m[r] = up ? mx[r] : m[r];
                        l[r] *= f[r];
                    }
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        o[i][0] *= f[0];
                        o[i][1] *= f[0];
                        o[i][2] *= f[1];
                        o[i][3] *= f[1];
                    }
                }
                float e[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float shift = m[r] == -INFINITY ? 0.f : kWeightBits - m[r];
#pragma unroll
                    for (int k = 0; k < 4; ++k) e[r][k] = fast_exp2(x[r][k] + shift);
                    l[r] += (e[r][0] + e[r][1]) + (e[r][2] + e[r][3]);
                }

                kv_wait(v_full + st, par, abort_flag, err, kDevErrTimeoutKv);
                if (hidden || have < kWarpKeys) {
                    // Slots behind the end may hold anything, and so may tokens
                    // that a row does not see: a zero weight would still carry
                    // their NaN and infinities into the sum.  Such values leave
                    // the tile; those of tokens that a row does see are added
                    // to it here.
                    const uint32_t strip = v_s;
                    for (int key = 0; key < kWarpKeys; ++key) {
                        const int vr = warp * kWarpKeys + key;
                        bool odd = key >= have;
                        if (!odd && hidden) {
                            for (int u = lane; u < D / 8; u += 32) {
                                uint4 v;
                                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                             : "r"(strip + unit_at(vr, u, kKeyTile)));
                                const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float2 f = T::unpack(wd[i]);
                                    odd |= !isfinite(f.x) || !isfinite(f.y);
                                }
                            }
                            odd = __any_sync(0xffffffffu, odd);
                            if (odd) {
                                const int src = rg * 4 + ((key & 7) >> 1);
                                float pk[2], xk[2];
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    const float e0 = __shfl_sync(0xffffffffu, key < 8 ? e[r][0] : e[r][2], src);
                                    const float e1 = __shfl_sync(0xffffffffu, key < 8 ? e[r][1] : e[r][3], src);
                                    const float x0 = __shfl_sync(0xffffffffu, key < 8 ? x[r][0] : x[r][2], src);
                                    const float x1 = __shfl_sync(0xffffffffu, key < 8 ? x[r][1] : x[r][3], src);
                                    pk[r] = key & 1 ? e1 : e0;
                                    xk[r] = key & 1 ? x1 : x0;
                                }
#pragma unroll
                                for (int i = 0; i < D / 8; ++i) {
                                    const float2 f = T::unpack(lds_u32_ordered(strip + unit_at(vr, i, kKeyTile) + 4 * ct));
#pragma unroll
                                    for (int r = 0; r < 2; ++r)
                                        if (xk[r] != -INFINITY) {
                                            o[i][2 * r] = fmaf(pk[r], f.x, o[i][2 * r]);
                                            o[i][2 * r + 1] = fmaf(pk[r], f.y, o[i][2 * r + 1]);
                                        }
                                }
                            }
                        }
                        __syncwarp();
                        if (odd)
                            for (int u = lane; u < D / 8; u += 32)
                                sts_u128(strip + unit_at(vr, u, kKeyTile), make_uint4(0, 0, 0, 0));
                    }
                    __syncwarp();
                    fence_proxy_async_smem();  // these writes come before the slot's next copy
                }
                uint32_t pf[4][Parts<T>::kN], pn[Parts<T>::kN][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i & 1, k = (i >> 1) * 2;
                    Parts<T>::split(make_float2(e[r][k], e[r][k + 1]), pf[i]);
#pragma unroll
                    for (int n = 0; n < Parts<T>::kN; ++n) pn[n][i] = pf[i][n];
                }
                const int vr = warp * kWarpKeys + (lane & 15);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t vf[4];
                    ldsm4_t(v_s + unit_at(vr, 2 * i + (lane >> 4), kKeyTile), vf);
                    // A product of its own, smallest parts first, added to o by
                    // rounded fp32 adds: the MMA cuts its sums off instead of
                    // rounding them, which over thousands of tiles would lean
                    // all to one side (4e-5 of the result at 131k tokens).
                    float t[2][4];
#pragma unroll
                    for (int n = 0; n < 8; ++n) (&t[0][0])[n] = 0.f;
#pragma unroll
                    for (int n = Parts<T>::kN - 1; n >= 0; --n) {
                        mma16816<T>(t[0], pn[n], vf[0], vf[1]);
                        mma16816<T>(t[1], pn[n], vf[2], vf[3]);
                    }
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        o[2 * i][n] += t[0][n];
                        o[2 * i + 1][n] += t[1][n];
                    }
                }
            } else {
                kv_wait(v_full + st, par, abort_flag, err, kDevErrTimeoutKv);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(slot_free + st);
        }

        // Join the warps' results.
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (ct == 0) ml[warp * kRowTile + rg + 8 * r] = make_float2(m[r], l[r]);
        }
        consumer_sync();
        float f[2], top[2], sum[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            top[r] = -INFINITY;
            sum[r] = 0.f;
            for (int i = 0; i < kConsumers; ++i) top[r] = fmaxf(top[r], ml[i * kRowTile + rg + 8 * r].x);
            for (int i = 0; i < kConsumers; ++i) {
                const float2 t = ml[i * kRowTile + rg + 8 * r];
                // (a maximum of -inf: the warp saw nothing, sum 0, or only NaN)
                sum[r] += t.x == -INFINITY ? t.y : t.y * fast_exp2(t.x - top[r]);
            }
            f[r] = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - top[r]);
        }
        if (warp == 0 && ct == 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = rg + 8 * r;
                ml[kConsumers * kRowTile + row] = make_float2(top[r], sum[r]);
                if (!w.whole && row < rows)
                    p.part_ml[(int64_t)w.slot * p.slot_rows + row] = make_float2(top[r], sum[r]);
            }
        }
        constexpr int kCols = C::kJoinCols;
#pragma unroll
        for (int ch = 0; ch < D / kCols; ++ch) {
#pragma unroll
            for (int i = 0; i < kCols / 8; ++i) {
                const float* v = o[ch * (kCols / 8) + i];
                float* to = join + warp * kRowTile * kCols + i * 8 + 2 * ct;
                *reinterpret_cast<float2*>(to + rg * kCols) = make_float2(v[0] * f[0], v[1] * f[0]);
                *reinterpret_cast<float2*>(to + (rg + 8) * kCols) = make_float2(v[2] * f[1], v[3] * f[1]);
            }
            consumer_sync();
            for (int u = threadIdx.x; u < rows * (kCols / 4); u += 32 * kConsumers) {
                const int r = u / (kCols / 4), col = u % (kCols / 4) * 4;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kConsumers; ++i) {
                    const float4 t = *reinterpret_cast<const float4*>(join + (i * kRowTile + r) * kCols + col);
                    v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
                }
                if (w.whole) {
                    const float sum_r = ml[kConsumers * kRowTile + r].y;
                    const float inv = sum_r == 0.f ? 0.f : 1.f / sum_r;  // a row that sees nothing: zeros
                    const int row = w.row_tile * kRowTile + r, t = token_of(p, row);
                    float* dst = p.out + (w.w.row0 + t) * p.out_row_stride +
                                 ((int64_t)w.head * p.group + row - t * p.group) * D + ch * kCols + col;
                    if (bc_global(bc, dst, 16, p.out,
                                  4 * ((p.rows - 1) * p.out_row_stride + (int64_t)p.group * p.kv_heads * D), kBcAttnOut))
                        *reinterpret_cast<float4*>(dst) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                } else {
                    float* dst = p.part_o + ((int64_t)w.slot * p.slot_rows + r) * D + ch * kCols + col;
                    *reinterpret_cast<float4*>(dst) = v;
                }
            }
            consumer_sync();
        }
    }
}

template <int D, class T>
cudaError_t launch_one(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, const CacheView& c,
                       const BatchView& b, int* err, cudaStream_t stream) {
    const cudaError_t e = allow_smem<attention_mma_kernel<D, T>>(MmaAttn<D>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_chained(attention_mma_kernel<D, T>, dim3((unsigned)p.ctas), dim3(kThreads), MmaAttn<D>::kSmem, stream,
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

cudaError_t launch_attention_mma(const AttnParams& p, const void* tk, const void* tv, const CacheView& c,
                                 const BatchView& b, bool bf16, int* err, cudaStream_t stream) {
    const CUtensorMap& mk = *static_cast<const CUtensorMap*>(tk);
    const CUtensorMap& mv = *static_cast<const CUtensorMap*>(tv);
    return bf16 ? launch_type<KvBf16>(p, mk, mv, c, b, err, stream) : launch_type<KvF16>(p, mk, mv, c, b, err, stream);
}

}  // namespace iq4xs
