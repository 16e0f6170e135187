// verify.cu -- which drafted tokens the target's probabilities accept, and the
// token behind them (include/iq4xs.h).
//
// The walk down the tree takes single probabilities: a cluster's first CTA
// looks them all up at once and walks in shared memory.  Whole rows of the
// vocabulary are summed where a drafter's distribution is taken off after a
// rejection, and once for the draw; a cluster shares them.  The sums are of
// whole numbers (values times 2^61), so that neither the order nor the split
// changes them: a draw near the border of two tokens always falls alike.
//
// Few bytes are read (a row or two of probabilities a sequence): what it takes
// is the chain of launch, tree, probabilities, sums, and the draw's search, whose barriers
// warps wait at (8.0 stalls an issue; for instructions 1.5): 12 trees of 8
// over 131,073 tokens 11.0 us (17 with cold caches), a chain of four with a drafter's
// probabilities over 32,000 10.2.  (CTAs of 256, 512 and 1,024 threads: 13.1, 12.3 and 12.4 before the loads
// were grouped.)  With a drafter's probabilities every rejection sums two rows again: 12
// chains of 4 over 131,073 16.6 us, 12 trees of 8 34.8, 45 177.8.
#include <type_traits>

#include "delta.cuh"

namespace iq4xs {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;
constexpr int kVerifyRows = 1024;
constexpr int kRun = 256;  // values that a warp sums at a time, eight a lane
constexpr int kMaxRuns = (1 << 20) / kVerifyCluster / kRun;

struct VerifyParams {
    const float* probs;
    const float* draft;
    int64_t probs_stride, draft_stride;
    const int32_t* tokens;
    const uint64_t* tree_mask;
    const float* accept_u;
    const float* draw_u;
    int32_t* paths;
    int32_t* accepted;
    int32_t* next;
    int mask_words, rows, vocab, path_width, ranks;
};

// What the first CTA tells the others to do next.
struct __align__(16) Order {
    int what;   // kSum, kDraw, kEnd
    int node;   // row of the batch whose probabilities they are
    int taken;  // times that the drafter's distribution comes off
    int gone;   // without one: rejected tokens in the first CTA's list; -1: the sums of before hold
};
enum { kSum, kDraw, kEnd };

struct VerifyShared {
    int parent[kVerifyRows], token[kVerifyRows];
    float u[kVerifyRows], p[kVerifyRows], q[kVerifyRows];
    unsigned char again[kVerifyRows];              // a sibling before has the same token
    int gone[kVerifyRows];                         // tokens rejected at the row
    unsigned long long mass[kVerifyRows];          // m before each subtraction
    unsigned long long parts[kVerifyCluster];      // the CTAs' sums
    unsigned long long runs[kMaxRuns];             // this CTA's, run by run
    Order order;
    int count;  // rows accepted
};

__device__ __forceinline__ float in_unit(float p) { return p > 0.f ? fminf(p, 1.f) : 0.f; }  // (NaN: 0)
// p in 0..1 as a whole number of 2^-61.
__device__ __forceinline__ unsigned long long whole(float p) {
    if (!(p > 0.f)) return 0;
    const uint32_t bits = __float_as_uint(fminf(p, 1.f));
    const int e = max((int)(bits >> 23), 1);  // value = mantissa * 2^(e - 150)
    const unsigned long long m = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);
    const int shift = e - 150 + 61;
    return shift >= 0 ? m << shift : shift > -32 ? m >> -shift : 0;
}
__device__ __forceinline__ double real(unsigned long long w) { return (double)w * 0x1p-61; }
// max(r - m q, 0)
__device__ __forceinline__ unsigned long long take_off(unsigned long long r, unsigned long long m, unsigned long long q) {
    const unsigned long long off = __umul64hi(m << 1, q << 2);
    return r > off ? r - off : 0;
}
// What is left of p behind `taken` subtractions of q (the first m is 1).
__device__ __forceinline__ unsigned long long left_of(float p, float q_at, int taken, const unsigned long long* mass) {
    const unsigned long long q = whole(q_at);
    unsigned long long r = whole(p);
    r = r > q ? r - q : 0;
#pragma unroll 1
    for (int x = 1; x < taken; ++x) r = take_off(r, mass[x], q);
    return r;
}
// Sums of eight.  (Out of line: a step calls this kernel once, its instructions
// come from L2 or HBM, and unrolled for every run they were most of its time.)
__device__ __noinline__ unsigned long long whole8(float a, float b, float c, float d, float e, float f, float g, float h) {
    return ((whole(a) + whole(b)) + (whole(c) + whole(d))) + ((whole(e) + whole(f)) + (whole(g) + whole(h)));
}
__device__ __noinline__ unsigned long long left8(float a, float b, float c, float d, float e, float f, float g, float h, float qa, float qb,
                                                 float qc, float qd, float qe, float qf, float qg, float qh, int taken,
                                                 const unsigned long long* mass) {
    const float p[8] = {a, b, c, d, e, f, g, h}, q[8] = {qa, qb, qc, qd, qe, qf, qg, qh};
    unsigned long long sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += left_of(p[k], q[k], taken, mass);
    return sum;
}
__device__ __forceinline__ uint32_t at_rank(const void* p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void st_rank(const void* p, int rank, unsigned long long v) {
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(at_rank(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ int ld_rank(const int* p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(at_rank(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();  // (the barrier wants warps whole, and threads of their own have been at work)
    cluster_arrive_release();
    cluster_wait();
}

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p, const BatchView b, int* err) {
    __shared__ VerifyShared sh;
    cluster_arrive_relaxed();
    griddep_launch_dependents();
    griddep_wait();
    const Bc bc = bc_open(err);
    const int rank = blockIdx.x % p.ranks, s = blockIdx.x / p.ranks;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t p_extent = 4 * ((p.rows - 1) * p.probs_stride + p.vocab);
    const int64_t q_extent = 4 * ((p.rows - 1) * p.draft_stride + p.vocab);
    const int64_t path_extent = 4 * (int64_t)b.sequences * p.path_width;
    int32_t* const path = p.paths + (int64_t)s * p.path_width;
    int first = 0, n = 0;
    if (rank == 0) {
        n = batch_rows(b, s, p.rows, &first, err);
        if (n > kVerifyRows) {
            if (tid == 0) data_error(err, kDataCount);
            n = 0;
        }
        // Every row: parent, token, random number, and its token's probabilities behind its parent.
        for (int t = tid; t < n; t += kVerifyThreads) {
            int parent = t - 1;
            if (p.tree_mask != nullptr) {
                parent = -1;
                for (int i = min(p.mask_words - 1, t >> 6); i >= 0 && parent < 0; --i) {
                    const uint64_t* from = p.tree_mask + (int64_t)(first + t) * p.mask_words + i;
                    uint64_t bits =
                        bc_global(bc, from, 8, p.tree_mask, 8 * (int64_t)p.rows * p.mask_words, kBcVerifyRow) ? *from : 0;
                    if (i == t >> 6) bits &= (1ull << (t & 63)) - 1;
                    if (bits != 0) parent = 64 * i + 63 - __clzll(bits);
                }
            }
            int token = -1;
            float u = 0.f, pr = 0.f, qr = 0.f;
            if (bc_global(bc, p.tokens + first + t, 4, p.tokens, 4 * (int64_t)p.rows, kBcVerifyRow))
                token = p.tokens[first + t];
            if (bc_global(bc, p.accept_u + first + t, 4, p.accept_u, 4 * (int64_t)p.rows, kBcVerifyRow))
                u = p.accept_u[first + t];
            if (token < 0 || token >= p.vocab) token = -1;
            if (parent >= 0 && token >= 0) {
                const float* from = p.probs + (first + parent) * p.probs_stride + token;
                if (bc_global(bc, from, 4, p.probs, p_extent, kBcVerifyProbs)) pr = *from;
                if (p.draft != nullptr) {
                    from = p.draft + (first + parent) * p.draft_stride + token;
                    if (bc_global(bc, from, 4, p.draft, q_extent, kBcVerifyProbs)) qr = *from;
                }
            }
            sh.parent[t] = parent;
            sh.token[t] = token;
            sh.u[t] = u;
            sh.p[t] = pr;
            sh.q[t] = qr;
        }
        __syncthreads();
        if (p.draft == nullptr)
            for (int t = tid; t < n; t += kVerifyThreads) {
                bool again = false;
                for (int i = t - 1; i > sh.parent[t] && !again; --i)
                    again = sh.parent[i] == sh.parent[t] && sh.token[i] == sh.token[t];
                sh.again[t] = again;
            }
        __syncthreads();
    }
    // Thread 0 of the first CTA: where the walk stands.
    constexpr unsigned long long kOne = 1ull << 61;
    int node = 0, t = 1, count = 1, taken = 0, gone = 0;
    bool summed = false;  // what is left behind the node has been summed
    unsigned long long mass = kOne;
    float near_mass = 1.f;
    auto accept = [&] {
        node = t;
        if (bc_global(bc, path + count, 4, p.paths, path_extent, kBcVerifyOut)) path[count] = t;
        ++count;
        taken = gone = 0;
        mass = kOne;
        near_mass = 1.f;
        summed = false;
    };
    auto walk = [&]() -> int {
        for (; t < n && count < p.path_width; ++t) {
            if (sh.parent[t] != node) continue;
            // (the same comparisons whatever the token: one outside has no chance and nothing to take off)
            unsigned long long r = whole(sh.p[t]);
            const double u = (double)sh.u[t];
            if (p.draft != nullptr) {
                const unsigned long long q = whole(sh.q[t]);
                for (int i = 0; i < taken; ++i) r = take_off(r, sh.mass[i], q);
                // (at first by the values themselves, whose product 64 bits hold)
                if (sh.token[t] >= 0 && (taken == 0 ? u * (double)in_unit(sh.q[t]) < (double)in_unit(sh.p[t])
                                                    : u * real(mass) * real(q) < real(r))) {
                    accept();
                    continue;
                }
                for (int k = 0; k < p.ranks; ++k) st_rank(&sh.mass[taken], k, mass);
                ++taken;
                ++t;
                summed = true;
                return kSum;
            }
            if (sh.token[t] < 0) continue;
            if (sh.again[t]) r = 0;
            // (In fp32 where that is far from a tie: its mass is off by 2^-24 a sibling, 1024 of them at most.)
            const float chance = sh.again[t] ? 0.f : in_unit(sh.p[t]), bar = sh.u[t] * near_mass;
            const bool far = fabsf(bar - chance) > 0x1p-12f;
            if (gone == 0 ? sh.u[t] < chance : far ? bar < chance : u * real(mass) < real(r)) {
                accept();
                continue;
            }
            mass -= min(mass, r);
            near_mass = fmaxf(near_mass - chance, 0.f);
            if (!sh.again[t]) sh.gone[gone++] = sh.token[t];
        }
        return kDraw;
    };
    // The part of a row of the vocabulary that this CTA sums, in runs that go round its warps.
    const int each = ((p.vocab + p.ranks - 1) / p.ranks + kRun - 1) / kRun * kRun;
    const int begin = min(p.vocab, rank * each), end = min(p.vocab, begin + each), runs = (end - begin + kRun - 1) / kRun;
    const int some = (runs + 31) / 32;
    unsigned long long upto = 0;  // the first warp's sums up to and with a lane's runs
    float draw = 0.f;
    if (bc_global(bc, p.draw_u + s, 4, p.draw_u, 4 * (int64_t)b.sequences, kBcVerifyRow)) draw = p.draw_u[s];
    bool plain = false;
    __syncwarp();
    cluster_wait();  // (every CTA has begun: its shared memory may be written)
    for (;;) {
        if (rank == 0 && tid == 0) {
            Order o = {kEnd, 0, 0, 0};
            if (n > 0) {
                o.what = plain ? kDraw : walk();
                o.node = first + node;
                o.taken = plain ? 0 : taken;
                o.gone = plain ? 0 : o.what == kDraw && summed ? -1 : gone;
            }
            const unsigned long long* w = reinterpret_cast<const unsigned long long*>(&o);
            for (int k = 0; k < p.ranks; ++k) {
                st_rank(&sh.order, k, w[0]);
                st_rank(reinterpret_cast<unsigned long long*>(&sh.order) + 1, k, w[1]);
            }
        }
        cluster_sync();
        const Order o = sh.order;
        if (o.what == kEnd) break;
        // What is left behind the row of values i0, i0 + step, ... (0 behind the part's end).
        const float* const p_row = p.probs + o.node * p.probs_stride;
        const float* const q_row = p.draft + o.node * p.draft_stride;
        auto ask = [&](const float* row, const float* base, int64_t extent, int i) {
            return i < end && bc_global(bc, row + i, 4, base, extent, kBcVerifyProbs) ? row[i] : 0.f;
        };
        // Sums of `kRuns` runs from `run` on, their loads in flight together.
        auto sum_runs = [&](auto runs_tag, int run) {
            constexpr int kRuns = decltype(runs_tag)::value;
            float pr[kRuns][8], qr[kRuns][8];
            auto ask_runs = [&](float (&to)[kRuns][8], const float* row, const float* base, int64_t extent) {
                const int i0 = begin + run * kRun + lane;
                const float* const from = row + i0;
                if (!kBoundsCheck && i0 - lane + ((kRuns - 1) * kVerifyWarps + 1) * kRun <= end) {  // (all inside: no test a value)
#pragma unroll
                    for (int y = 0; y < kRuns; ++y)
#pragma unroll
                        for (int k = 0; k < 8; ++k) to[y][k] = from[y * kVerifyWarps * kRun + 32 * k];
                } else {
#pragma unroll
                    for (int y = 0; y < kRuns; ++y)
#pragma unroll
                        for (int k = 0; k < 8; ++k) to[y][k] = ask(row, base, extent, i0 + y * kVerifyWarps * kRun + 32 * k);
                }
            };
            ask_runs(pr, p_row, p.probs, p_extent);
            if (o.taken > 0) ask_runs(qr, q_row, p.draft, q_extent);
            unsigned long long sum[kRuns];
#pragma unroll
            for (int y = 0; y < kRuns; ++y) {
                const float(&a)[8] = pr[y], (&e)[8] = qr[y];
                sum[y] = o.taken > 0 ? left8(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], e[0], e[1], e[2], e[3], e[4], e[5],
                                             e[6], e[7], o.taken, sh.mass)
                                     : whole8(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7]);
            }
#pragma unroll
            for (int k = 16; k > 0; k >>= 1)
#pragma unroll
                for (int y = 0; y < kRuns; ++y) sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], k);
            if (lane == 0)
#pragma unroll
                for (int y = 0; y < kRuns; ++y)
                    if (run + y * kVerifyWarps < runs) sh.runs[run + y * kVerifyWarps] = sum[y];
        };
        if (o.gone >= 0) {
            if (p.draft != nullptr) {
                for (int run = warp; run < runs; run += 2 * kVerifyWarps) sum_runs(std::integral_constant<int, 2>{}, run);
            } else {
                for (int run = warp; run < runs; run += 4 * kVerifyWarps) sum_runs(std::integral_constant<int, 4>{}, run);
            }
            __syncthreads();
            for (int i = tid; i < o.gone; i += kVerifyThreads) {
                const int x = rank != 0 ? ld_rank(&sh.gone[i], 0) : sh.gone[i];
                if (rank != 0) sh.gone[i] = x;
                if (x >= begin && x < end && bc_global(bc, p_row + x, 4, p.probs, p_extent, kBcVerifyProbs))
                    atomicAdd(&sh.runs[(x - begin) / kRun], 0ull - whole(p_row[x]));
            }
            __syncthreads();
            // Lane l of the first warp: runs l * some .. of the part.
            upto = 0;
            if (warp == 0) {
                for (int i = lane * some; i < min(runs, (lane + 1) * some); ++i) upto += sh.runs[i];
#pragma unroll
                for (int k = 1; k < 32; k <<= 1) {
                    const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, k);
                    if (lane >= k) upto += y;
                }
                const unsigned long long all = __shfl_sync(0xffffffffu, upto, 31);
                if (lane < p.ranks) st_rank(&sh.parts[rank], lane, all);
            }
            cluster_sync();
        }
        unsigned long long total = 0, before = 0;
        for (int k = 0; k < p.ranks; ++k) {
            before += k < rank ? sh.parts[k] : 0;
            total += sh.parts[k];
        }
        if (o.what == kSum) {
            mass = total;
            continue;
        }
        if (total == 0 && !plain) {  // nothing is left: from the row itself
            plain = true;
            cluster_sync();  // (sums of before: no other barrier keeps the next order from overtaking the looks at this one)
            continue;
        }
        if (total == 0) {
            if (rank == 0 && tid == 0 && bc_global(bc, p.next + s, 4, p.next, 4 * (int64_t)b.sequences, kBcVerifyOut))
                p.next[s] = -1;
            break;
        }
        const double at = (double)fminf(fmaxf(draw, 0.f), 1.f) * (double)total;
        unsigned long long wanted = at < (double)total ? (unsigned long long)at : total - 1;
        wanted = min(wanted, total - 1);  // the first value whose running sum is above it
        if (wanted < before || wanted - before >= sh.parts[rank]) break;
        wanted -= before;
        if (warp != 0) break;
        const int at_lane = __ffs(__ballot_sync(0xffffffffu, upto > wanted)) - 1;
        const unsigned long long below = __shfl_up_sync(0xffffffffu, upto, 1);
        if (at_lane > 0) wanted -= __shfl_sync(0xffffffffu, below, at_lane);
        int run = at_lane * some;
        for (; run < min(runs, (at_lane + 1) * some) - 1 && wanted >= sh.runs[run]; ++run) wanted -= sh.runs[run];
        // Eight neighbouring values a lane.
        const int i0 = begin + run * kRun + 8 * lane;
        unsigned long long r[8], sum = 0;
        float pr[8], qr[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) pr[k] = ask(p_row, p.probs, p_extent, i0 + k);
        if (o.taken > 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) qr[k] = ask(q_row, p.draft, q_extent, i0 + k);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = o.taken > 0 ? left_of(pr[k], qr[k], o.taken, sh.mass) : whole(pr[k]);
        for (int k = 0; k < o.gone; ++k)
#pragma unroll
            for (int x = 0; x < 8; ++x) r[x] = sh.gone[k] == i0 + x ? 0 : r[x];
#pragma unroll
        for (int x = 0; x < 8; ++x) sum += r[x];
        unsigned long long with = sum;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, with, k);
            if (lane >= k) with += y;
        }
        if (lane == __ffs(__ballot_sync(0xffffffffu, with > wanted)) - 1) {
            unsigned long long so_far = with - sum;
            int x = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                so_far += r[k];
                x += so_far <= wanted;
            }
            if (bc_global(bc, p.next + s, 4, p.next, 4 * (int64_t)b.sequences, kBcVerifyOut)) p.next[s] = i0 + x;
        }
        break;
    }
    if (rank == 0) {
        if (tid == 0) {
            sh.count = n > 0 ? count : 0;
            if (bc_global(bc, p.accepted + s, 4, p.accepted, 4 * (int64_t)b.sequences, kBcVerifyOut))
                p.accepted[s] = n > 0 ? count : 0;
            if (n > 0 && bc_global(bc, path, 4, p.paths, path_extent, kBcVerifyOut)) path[0] = 0;
            if (n == 0 && bc_global(bc, p.next + s, 4, p.next, 4 * (int64_t)b.sequences, kBcVerifyOut)) p.next[s] = -1;
        }
        __syncthreads();
        for (int i = sh.count + tid; i < p.path_width; i += kVerifyThreads)
            if (bc_global(bc, path + i, 4, p.paths, path_extent, kBcVerifyOut)) path[i] = 0;
    }
}

}  // namespace

cudaError_t launch_verify_drafts(const iq4xs_verify_drafts_args& a, const BatchView& b, int* err, int num_sms,
                                 cudaStream_t stream) {
    VerifyParams p;
    p.probs = a.probs;
    p.draft = a.draft_probs;
    p.probs_stride = a.probs_stride;
    p.draft_stride = a.draft_probs ? a.draft_stride : 0;
    p.tokens = a.tokens;
    p.tree_mask = a.tree_mask;
    p.accept_u = a.accept_u;
    p.draw_u = a.draw_u;
    p.paths = a.paths;
    p.accepted = a.accepted;
    p.next = a.next;
    p.mask_words = (int)a.mask_words;
    p.rows = (int)a.rows;
    p.vocab = (int)a.vocab;
    p.path_width = (int)a.path_width;
    p.ranks = 1;
    // A run for half of a CTA's warps, and a CTA an SM: 131,073 tokens, 12 sequences 18.5,
    // 13.6 and 10.9 us by 2, 4 and 8 CTAs each, 45 18.5, 24.6 and 28.7; 701 tokens
    // and a drafter's probabilities, 12 sequences 9.4 by one and 10.7 by two.  (At
    // least as many as the sums' runs need.)
    while (p.ranks < kVerifyCluster &&
           (p.vocab > (int64_t)p.ranks * kMaxRuns * kRun ||
            (p.ranks * 8 * kRun < p.vocab && 2 * (int64_t)p.ranks * b.sequences <= num_sms)))
        p.ranks *= 2;
    return launch_chained(verify_kernel, dim3((unsigned)(b.sequences * p.ranks)), dim3(kVerifyThreads), 0, stream, p.ranks,
                          p, b, err);
}

}  // namespace iq4xs
