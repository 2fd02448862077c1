// Around the experts of a mixture: the choice of experts with its gradient, the
// slots sorted by expert, tokens copied to their experts' rows, and the experts'
// outputs added up for the tokens, with the gradients.  (Dispatch's gradient is a
// combine without weights.)  Slot s = token * k + j is a token's j-th choice.
#include <cuda_runtime.h>

#include <mutex>

#include "f32x2.cuh"
#include "ptx.cuh"
#include "row_ops.cuh"
#include "temx_internal.h"

namespace temx {

namespace {

// ---------------------------------------------------------------- router

// A warp per token; lane l holds experts l, l + 32, ... (kN of them).
//   key[e] = fl32(logit[e] + bias[e]);  the k largest keys, ties to the lowest index.
//   p = softmax of the logits over all experts, or the logistic function of each;
//   weight = scale p, or scale p / (the chosen experts' sum of p).
// Keys are compared as integers in the order of the numbers; NaN comes last, after
// -inf, so the indices are always k different experts.  Instructions bound it (the
// bytes of 16384 x 128 bf16 take 0.6 us): a key of 16 bits (bf16 or fp16 logits without
// a bias: kPacked) shares a word with its index, so that one maximum over the warp
// gives both, and the chosen logits are read again at the end (16384 x 128 bf16, k = 8,
// both directions, unsorted: 12.0 us; with two maxima over the warp and a shuffle per choice 16.2).
// For enough choices a lane first sorts its words: a round then looks at one of them (both
// directions 11.1).  On either side of the rule, forward, 16384 tokens, us (this, without the
// sorted path in the kernel): 128 experts k = 8 6.5, 7.6, k = 1 4.8, 5.3; 256 k = 4 8.4, 8.8,
// k = 3 7.9, 8.1; 512 k = 8 16.7, 18.4, but below the rule k = 7 17.0, 16.4, k = 3 12.4, 11.8.
// Keys of 32 bits with their index are pairs, and sorted as such were slower (16384 x 256
// fp32, k = 4: 12.6, 11.0).
constexpr int kRouteWarps = 8;

__device__ __forceinline__ uint32_t ordered_key(float v) {
    if (v != v) return 1u;                                 // (0: taken already)
    const uint32_t b = __float_as_uint(v + 0.0f);          // (-0 and 0 are equal)
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;       // -inf: 0x007FFFFF
}

__device__ __forceinline__ float logistic(float v) { return 1.0f / (1.0f + expf(-v)); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

template <typename T, int kN>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t token, int lane, float (&l)[kN]) {
    const T* p = static_cast<const T*>(a.logits) + token * a.ld_logits;
#pragma unroll
    for (int i = 0; i < kN; ++i) l[i] = lane + 32 * i < a.experts ? to_f32(p[lane + 32 * i]) : -INFINITY;
}

// Largest logit of the row and the sum of exp(logit - largest).
template <int kN>
__device__ __forceinline__ void softmax_sum(const float (&l)[kN], float& most, float& sum) {
    float m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < kN; ++i) s += l[i] == -INFINITY ? 0.0f : expf(l[i] - m);
    most = m;
    sum = warp_sum(s);
}

// A chosen logit's share of the logistic scores of the chosen (-inf in lanes without a
// choice); 0 where all are -inf.  Scores vanish below -88, so they are taken relative to
// e^top, s e^-top = 1 / (e^top + e^(top - v)), with top the largest chosen logit if that is
// negative, else 0: the factor cancels, and the largest is at least 1/2.  (-top is the least
// of max(-v, 0), whose bits are in the order of the numbers: one reduction.)  `rest`: 1 - s,
// e^(top - v) times s e^-top; 1 where that is 0.
__device__ __forceinline__ float logistic_share(float logit, float& rest) {
    const float top = -__uint_as_float(__reduce_min_sync(0xFFFFFFFFu, __float_as_uint(fmaxf(-logit, 0.0f))));
    const float e = expf(top - logit), s = logit == -INFINITY ? 0.0f : 1.0f / (expf(top) + e), sum = warp_sum(s);
    rest = s == 0.0f ? 1.0f : e * s;
    return sum == 0.0f ? 0.0f : s / sum;
}

// The bits of a 16-bit float in the order of the numbers, NaN last (1), -0 as 0.
template <typename T> __device__ __forceinline__ uint32_t ordered_key16(float v) {
    if (v != v) return 1u;
    const T h = from_f32<T>(v + 0.0f);                     // (v is a T)
    const uint32_t b = *reinterpret_cast<const uint16_t*>(&h);
    return (b & 0x8000u) ? ~b & 0xFFFFu : b | 0x8000u;
}

// A lane's keys in falling order (Batcher's merge exchange; kN a power of two).
template <int kN> __device__ __forceinline__ void sort_falling(uint32_t (&key)[kN]) {
#pragma unroll
    for (int p = 1; p < kN; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int i = 0; i + k < kN; ++i)
                if (i >= k % p && (i - k % p) / k % 2 == 0 && i / (2 * p) == (i + k) / (2 * p)) {
                    const uint32_t x = key[i], y = key[i + k];
                    key[i] = max(x, y);
                    key[i + k] = min(x, y);
                }
}

template <typename T, int kN, bool kPacked>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_kernel(const RouteArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t token = int64_t(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (token >= a.tokens) return;
    float l[kN];
    load_logits<T, kN>(a, token, lane, l);
    uint32_t key[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int e = lane + 32 * i;
        if constexpr (kPacked) key[i] = ordered_key16<T>(l[i]) << 16 | uint32_t(0xFFFF - e);
        else key[i] = ordered_key(a.bias && e < a.experts ? l[i] + a.bias[e] : l[i]);
        if (e >= a.experts) key[i] = 0u;
    }
    int mine = 0;                                          // lane j: the j-th choice
    if (kPacked && kN <= 16 && a.k >= kN / 2) {            // (sorted once, a lane's largest key is its first)
        sort_falling(key);
        for (int j = 0; j < a.k; ++j) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, key[0]);
            const bool won = key[0] == top;
#pragma unroll
            for (int i = 0; i < kN; ++i) key[i] = !won ? key[i] : i + 1 < kN ? key[i + 1] : 0u;
            if (lane == j) mine = int(0xFFFFu - (top & 0xFFFFu));
        }
    } else {
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < kN; ++i) best = max(best, key[i]);
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
            uint32_t e;
            if constexpr (kPacked) {
                e = 0xFFFFu - (top & 0xFFFFu);
#pragma unroll
                for (int i = 0; i < kN; ++i) key[i] = key[i] == top ? 0u : key[i];
            } else {
                uint32_t at = 0xFFFFFFFFu;
#pragma unroll
                for (int i = kN - 1; i >= 0; --i)
                    if (key[i] == top) at = uint32_t(lane + 32 * i);
                e = __reduce_min_sync(0xFFFFFFFFu, at);
#pragma unroll
                for (int i = 0; i < kN; ++i)
                    if (e == uint32_t(lane + 32 * i)) key[i] = 0u;
            }
            if (lane == j) mine = int(e);
        }
    }
    const float logit = lane < a.k ? to_f32((static_cast<const T*>(a.logits) + token * a.ld_logits)[mine]) : -INFINITY;
    const bool chosen = lane < a.k;
    float w;
    if (a.scoring == TE_MX_SCORE_SOFTMAX) {
        float most, sum;
        if (a.renormalise) {                               // of the chosen ones alone: the others' sum cancels
            most = warp_max(logit);
            const float p = chosen && logit != -INFINITY ? expf(logit - most) : 0.0f;
            sum = warp_sum(p);
            w = p;
        } else {
            softmax_sum(l, most, sum);
            w = logit != -INFINITY ? expf(logit - most) : 0.0f;
        }
        w = sum == 0.0f ? 0.0f : w / sum;
    } else {
        float rest;
        w = a.renormalise ? logistic_share(logit, rest) : logistic(logit);
    }
    if (chosen) {
        a.index[token * a.k + lane] = mine;
        a.weight[token * a.k + lane] = w * a.scale;
    }
}

// Gradient of the logits from that of the weights (g = scale dweight, w before the
// scale, p and s the scores):
//   softmax, renormalised   dl_i = w_i (g_i - sum_j w_j g_j)          chosen i, else 0
//   softmax                 dl_e = p_e ([e chosen] g_e - sum_j p_j g_j)
//   logistic, renormalised  dl_i = w_i (1 - s_i) (g_i - sum_j w_j g_j)
//   logistic                dl_i = s_i (1 - s_i) g_i
// An index outside the experts takes no part in any of it, the sums of w included: a choice
// that was never made.  (One dropped after the weights were made has its index and g = 0.)
template <typename T, int kN>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_backward_kernel(const RouteArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t token = int64_t(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (token >= a.tokens) return;
    const T* row = static_cast<const T*>(a.logits) + token * a.ld_logits;
    int e = -1;
    float g = 0.0f, logit = -INFINITY;
    if (lane < a.k) {
        e = a.index[token * a.k + lane];
        if (e < 0 || e >= a.experts) e = -1;
        else {
            g = a.weight[token * a.k + lane] * a.scale;
            logit = to_f32(row[e]);
        }
    }
    float d[kN];                                           // the gradients of what was not chosen
#pragma unroll
    for (int i = 0; i < kN; ++i) d[i] = 0.0f;
    float mine;                                            // a chosen expert's
    if (a.scoring == TE_MX_SCORE_SOFTMAX) {
        if (a.renormalise) {
            const float most = warp_max(logit);
            const float p = logit != -INFINITY ? expf(logit - most) : 0.0f;
            const float sum = warp_sum(p), w = sum == 0.0f ? 0.0f : p / sum;
            mine = w * (g - warp_sum(w * g));
        } else {
            float l[kN], most, sum;
            load_logits<T, kN>(a, token, lane, l);
            softmax_sum(l, most, sum);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const float p = logit != -INFINITY ? expf(logit - most) * inv : 0.0f;
            const float total = warp_sum(p * g);
            mine = p * (g - total);
#pragma unroll
            for (int i = 0; i < kN; ++i) d[i] = l[i] == -INFINITY ? 0.0f : -total * (expf(l[i] - most) * inv);
        }
    } else {
        if (a.renormalise) {
            float rest;
            const float w = logistic_share(logit, rest), total = warp_sum(w * g);
            mine = e < 0 ? 0.0f : w * rest * (g - total);
        } else {
            mine = e < 0 ? 0.0f : logistic(logit) * logistic(-logit) * g;
        }
    }
    // the whole row, then the chosen experts' over it (the warp's stores in order)
    T* out = static_cast<T*>(a.dlogits) + token * a.ld_dlogits;
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (lane + 32 * i < a.experts) out[lane + 32 * i] = from_f32<T>(d[i]);
    __syncwarp();
    if (e >= 0) out[e] = from_f32<T>(mine);
}

// ---------------------------------------------------------------- slots sorted by expert

// A stable counting sort in one launch: a cluster of blocks, each with a contiguous
// part of the slots, each warp with a contiguous part of its block's.  A warp goes
// through its slots 32 at a time: the slots of one expert find each other with a ballot
// for each bit of its index, and each takes the warp's count of that expert (in shared
// memory of the warp's own, so no atomic's order matters) and its place among them as
// its rank.  The counts are then summed over the warps and, through distributed shared
// memory, over the blocks, and a slot's row is its rank behind what comes before its
// warp.  The inverse leaves through shared memory, where the block's slots are sorted,
// so that an expert's slots are written side by side (scattered one by one from 8 SMs
// 131072 slots took 2 us more).  A warp holds its slots in registers,
// 16 groups of 32; more slots than all warps hold are sorted in rounds, after a pass
// that counts the experts' slots in all of them.
constexpr int kSortWarps = 32;                   // of a block
constexpr int kSortFewWarps = 8;                 // of a block alone, for few slots and experts
constexpr int kSortCluster = 16;                 // blocks at most (8 without the wide clusters)
constexpr int kMaxExperts = 1024;
constexpr int kSortHeld = 16;                    // groups of 32 slots in a warp's registers
constexpr int kSortBlockSlots = 32 * kSortWarps * kSortHeld;
// (a round's groups times its warps: products of both are ints)
static_assert(int64_t(kSortCluster) * kSortBlockSlots / 32 * (kSortCluster * kSortWarps) < int64_t(1) << 31);

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int32_t remote_load(const int32_t* p, uint32_t rank) {
    uint32_t addr;
    int32_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Inclusive sum over the block's threads; `sums`: a slot for each warp.
template <int kWarps> __device__ __forceinline__ int32_t block_scan(int32_t v, int32_t* sums, int warp, int lane) {
    auto warp_scan = [&](int32_t x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    v = warp_scan(v);
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    const int32_t w = warp_scan(lane < kWarps ? sums[lane] : 0);
    const int32_t before = __shfl_sync(0xFFFFFFFFu, w, warp == 0 ? 0 : warp - 1);
    return warp == 0 ? v : v + before;
}

template <int kBits, int kWarps>                 // of an expert's index, of a block
__global__ void __launch_bounds__(32 * kWarps, 1)
moe_sort_kernel(const int32_t* __restrict__ index, int64_t slots, int32_t experts, int blocks, int32_t* __restrict__ group_m,
                int32_t* __restrict__ row, int32_t* __restrict__ slot, unsigned int* status) {
    constexpr int kThreads = 32 * kWarps, kSlots = kThreads * kSortHeld;
    extern __shared__ int32_t shared[];
    uint32_t* sorted = reinterpret_cast<uint32_t*>(shared);            // [kSlots]: expert << 16 | slot
    int32_t* counts = shared + kSlots;                     // [kWarps][experts]: counts, then first places
    __shared__ int32_t total[2][kMaxExperts];              // of this block's slots (read by the other blocks)
    __shared__ int32_t to_row[kMaxExperts];                // from a place in `sorted` to a row
    __shared__ int32_t sums[2][kWarps];
    __shared__ int32_t here_kept, all_kept;
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = int(threadIdx.x), lane = t & 31, warp = t >> 5;
    const uint32_t rank = blocks > 1 ? cluster_rank() : 0u;
    const int64_t per_round = int64_t(blocks) * kSlots, rounds = slots > per_round ? (slots + per_round - 1) / per_round : 1;
    auto sync_blocks = [&] {
        if (blocks > 1) cluster_sync_all();
        else __syncthreads();
    };
    // expert t's slots in the blocks before this one, and in all
    auto across_blocks = [&](const int32_t* of_block, int32_t& before) {
        int32_t v[kSortCluster], all = 0;
        before = 0;
        if (t >= experts) return all;
#pragma unroll
        for (int b = 0; b < kSortCluster; ++b) v[b] = b >= blocks ? 0 : blocks == 1 ? of_block[t] : remote_load(&of_block[t], uint32_t(b));
#pragma unroll
        for (int b = 0; b < kSortCluster; ++b) {
            if (b < int(rank)) before += v[b];
            all += v[b];
        }
        return all;
    };
    int32_t all = 0, start = 0, done = 0;                  // expert t's slots, its first row, its slots in earlier rounds
    if (rounds > 1) {
        total[1][t] = 0;
        __syncthreads();
        for (int64_t s = int64_t(rank) * kThreads + t; s < slots; s += int64_t(blocks) * kThreads) {
            const int32_t e = index[s];
            if (e >= 0 && e < experts) atomicAdd(&total[1][e], 1);
        }
        sync_blocks();
        int32_t before;
        all = across_blocks(total[1], before);
        const int32_t upto = block_scan<kWarps>(all, sums[0], warp, lane);
        start = upto - all;
        if (t == kThreads - 1) all_kept = upto;
    }
    for (int64_t round = 0; round < rounds; ++round) {
        // this block's slots of the round, and this warp's, whole groups of 32
        const int64_t first = round * per_round;
        const int in_round = int(slots - first < per_round ? slots - first : per_round);
        const int groups = (in_round + 31) / 32, parts = blocks * kWarps, part = int(rank) * kWarps + warp;
        const int g0 = groups * part / parts, n = groups * (part + 1) / parts - g0;    // (n: at most kSortHeld)
        const int of_block = 32 * (groups * (int(rank) * kWarps) / parts), s0 = 32 * g0 + lane;
        const int32_t* from = index + first + s0;
        int32_t of[kSortHeld];                             // expert << 16 | rank; -1: none
#pragma unroll
        for (int i = 0; i < kSortHeld; ++i) of[i] = i < n && s0 + 32 * i < in_round ? from[32 * i] : -1;
        for (int i = t; i < kWarps * experts; i += kThreads) counts[i] = 0;
        __syncthreads();
        int32_t* mine = counts + warp * experts;
#pragma unroll
        for (int i = 0; i < kSortHeld; ++i) {
            if (i < n) {
                int32_t e = of[i];
                if (e >= experts) {
                    set_device_status(status, kStatusBadArg);
                    e = -1;
                }
                uint32_t peers = __ballot_sync(0xFFFFFFFFu, e >= 0);   // the slots of the same expert
#pragma unroll
                for (int b = 0; b < kBits; ++b) {
                    const bool one = e & (1 << b);
                    const uint32_t set = __ballot_sync(0xFFFFFFFFu, one);
                    peers &= one ? set : ~set;
                }
                int32_t r = 0;
                if (e >= 0) r = mine[e] + __popc(peers & ((1u << lane) - 1u));
                __syncwarp();
                if (e >= 0 && lane == 31 - __clz(peers)) mine[e] = r + 1;
                __syncwarp();
                of[i] = e < 0 ? -1 : e << 16 | r;          // (r < 512)
            }
        }
        __syncthreads();
        // over the warps
        int32_t here = 0;
        if (t < experts) {
            for (int w0 = 0; w0 < kWarps; w0 += 8) {
                int32_t c[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) c[w] = counts[(w0 + w) * experts + t];
#pragma unroll
                for (int w = 0; w < 8; ++w) here += c[w];
            }
        }
        total[round & 1][t] = here;
        // over the blocks, and over the experts
        sync_blocks();
        int32_t before;
        const int32_t of_round = across_blocks(total[round & 1], before);
        if (rounds == 1) {
            all = of_round;
            const int32_t upto = block_scan<kWarps>(all, sums[0], warp, lane);
            start = upto - all;
            if (t == kThreads - 1) all_kept = upto;
        }
        const int32_t place_upto = block_scan<kWarps>(here, sums[1], warp, lane);
        if (t == kThreads - 1) here_kept = place_upto;
        if (t < experts) {
            int32_t p = place_upto - here;                 // the expert's first place in `sorted`
            to_row[t] = start + done + before - p;
            for (int w0 = 0; w0 < kWarps; w0 += 8) {
                int32_t c[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) c[w] = counts[(w0 + w) * experts + t];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    counts[(w0 + w) * experts + t] = p;
                    p += c[w];
                }
            }
            done += of_round;
        }
        __syncthreads();
        int32_t* to = row + first + s0;
#pragma unroll
        for (int i = 0; i < kSortHeld; ++i) {
            if (i < n && s0 + 32 * i < in_round) {
                int32_t r = -1;
                if (of[i] >= 0) {
                    const int32_t e = of[i] >> 16, p = (of[i] & 0xFFFF) + mine[e];
                    sorted[p] = uint32_t(e) << 16 | uint32_t(s0 + 32 * i - of_block);
                    r = p + to_row[e];
                }
                to[32 * i] = r;
            }
        }
        __syncthreads();
        const int32_t base = int32_t(first) + of_block;
        for (int p = t; p < here_kept; p += kThreads) {
            const uint32_t v = sorted[p];
            slot[p + to_row[v >> 16]] = base + int32_t(v & 0xFFFFu);
        }
    }
    if (rank == 0 && t < experts) group_m[t] = all;
    // rows without a slot
    for (int64_t r = all_kept + int64_t(rank) * kThreads + t; r < slots; r += int64_t(blocks) * kThreads) slot[r] = -1;
    if (blocks > 1) cluster_sync_all();                    // no block leaves while another may still read its counts
}

// ---------------------------------------------------------------- dispatch

// Every token's row is read once and written to the rows of its slots (16384 x 8 rows of
// 8 KB: 178 us, the floor).  A block takes
// a token's part of kCopyThreads * kCopyPieces pieces of kBytes bytes; the scales of MXFP8 rows go
// byte by byte with the first part.
constexpr int kCopyThreads = 128;
template <int kBytes> constexpr int kCopyPieces = kBytes == 16 ? 4 : 8;      // per thread
template <int kBytes> struct PieceOf;
template <> struct PieceOf<16> { using Type = uint4; };
template <> struct PieceOf<4> { using Type = uint32_t; };
template <> struct PieceOf<2> { using Type = uint16_t; };
template <> struct PieceOf<1> { using Type = uint8_t; };

template <int kBytes>
__global__ void __launch_bounds__(kCopyThreads)
moe_dispatch_kernel(const DispatchArgs a, int parts, unsigned int* status) {
    using Piece = typename PieceOf<kBytes>::Type;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t token = int64_t(blockIdx.x) / parts;
    const int part = int(int64_t(blockIdx.x) % parts);
    const int64_t pieces = a.row_bytes / kBytes, p0 = int64_t(part) * kCopyThreads * kCopyPieces<kBytes> + threadIdx.x;
    const Piece* x = reinterpret_cast<const Piece*>(a.x + token * a.ld_x);
    Piece v[kCopyPieces<kBytes>];
#pragma unroll
    for (int i = 0; i < kCopyPieces<kBytes>; ++i)
        if (p0 + i * kCopyThreads < pieces) v[i] = x[p0 + i * kCopyThreads];
    for (int j = 0; j < a.k; ++j) {
        const int64_t r = a.row[token * a.k + j];
        if (r < 0) continue;
        if (r >= a.total_rows) {
            if (threadIdx.x == 0) set_device_status(status, kStatusBadArg);
            continue;
        }
        Piece* out = reinterpret_cast<Piece*>(a.out + r * a.ld_out);
#pragma unroll
        for (int i = 0; i < kCopyPieces<kBytes>; ++i)
            if (p0 + i * kCopyThreads < pieces) out[p0 + i * kCopyThreads] = v[i];
        if (a.scales && part == 0)
            for (int64_t b = threadIdx.x; b < a.scale_bytes; b += kCopyThreads)
                a.out_scales[r * a.ld_out_scales + b] = a.scales[token * a.ld_scales + b];
    }
}

// ---------------------------------------------------------------- combine

// out[t] = sum_j weight[t][j] y[row[t][j]] + residual[t], in fp32, the choices in
// order, rounded once.  Persistent: a block's warps take parts of 32 kN pieces of a
// token side by side, a piece a 16-byte vector (kVec: rows on 16-byte boundaries) or an element, from kJ rows at
// a time; lane j holds the j-th row and weight, loaded a token ahead.  The loads in
// flight are what it lives on, so few choices take more pieces.  16384 x 8 x 4096 bf16
// with a residual: 200 us (floor 198; a block of 256 threads per token and part, one
// vector per thread, 231); 4096 x 2 x 2048 15.5 (9.9; 20); 4096 x 4 x 2047 27 (15; 87).
constexpr int kCombineThreads = 128;             // at most
constexpr int kCombineWarps = 24;                // of an SM, resident
template <typename T, bool kVec, int kN, int kJ>
__global__ void __launch_bounds__(kCombineThreads, kCombineWarps * 32 / kCombineThreads)
moe_combine_kernel(const CombineArgs a, unsigned int* status) {
    using V = Vec<T>;
    using Piece = typename std::conditional<kVec, uint4, T>::type;
    constexpr int kPairs = kVec ? V::kPairs : 1;           // (an element: the low half)
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int pieces = kVec ? int(a.hidden / V::kN) : int(a.hidden);
    const int i0 = int(blockIdx.y * blockDim.x + threadIdx.x - lane) * kN + lane;
    if (i0 - lane >= pieces) return;                       // (no part of the rows for this warp)
    auto pair = [](const Piece& w, int q) {
        if constexpr (kVec) return V::pair(w, q);
        else return f32x2::pack(to_f32(w), 0.0f);
    };
    int32_t row = -1, row_next = -1;
    float weight = 0.0f, weight_next = 0.0f;
    auto load_side = [&](int64_t token) {
        row_next = lane < a.k ? a.row[token * a.k + lane] : -1;
        weight_next = lane < a.k && a.weight ? a.weight[token * a.k + lane] : 1.0f;
    };
    load_side(blockIdx.x);
    for (int64_t token = blockIdx.x; token < a.tokens; token += gridDim.x) {
        row = row_next;
        weight = weight_next;
        if (row >= a.total_rows) {
            set_device_status(status, kStatusBadArg);
            row = -1;
        }
        if (token + gridDim.x < a.tokens) load_side(token + gridDim.x);
        const Piece* res = a.residual ? reinterpret_cast<const Piece*>(static_cast<const T*>(a.residual) + token * a.ld_residual) : nullptr;
        Piece add[kN];
        uint64_t s[kN][kPairs];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            if (res && i0 + 32 * n < pieces) add[n] = res[i0 + 32 * n];
#pragma unroll
            for (int q = 0; q < kPairs; ++q) s[n][q] = 0;
        }
        for (int j0 = 0; j0 < a.k; j0 += kJ) {
            Piece w[kJ][kN];
            int32_t r[kJ];
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                r[j] = __shfl_sync(0xFFFFFFFFu, row, (j0 + j) & 31);
                if (j0 + j >= a.k) r[j] = -1;
                if (r[j] >= 0) {
                    const Piece* y = reinterpret_cast<const Piece*>(static_cast<const T*>(a.y) + r[j] * a.ld_y) + i0;
#pragma unroll
                    for (int n = 0; n < kN; ++n)
                        if (i0 + 32 * n < pieces) w[j][n] = y[32 * n];
                }
            }
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const uint64_t f = f32x2::both(__shfl_sync(0xFFFFFFFFu, weight, (j0 + j) & 31));
                if (r[j] >= 0) {
#pragma unroll
                    for (int n = 0; n < kN; ++n)
                        if (i0 + 32 * n < pieces) {
#pragma unroll
                            for (int q = 0; q < kPairs; ++q) s[n][q] = f32x2::fma(pair(w[j][n], q), f, s[n][q]);
                        }
                }
            }
        }
        Piece* out = reinterpret_cast<Piece*>(static_cast<T*>(a.out) + token * a.ld_out) + i0;
#pragma unroll
        for (int n = 0; n < kN; ++n)
            if (i0 + 32 * n < pieces) {
                if (res) {
#pragma unroll
                    for (int q = 0; q < kPairs; ++q) s[n][q] = f32x2::add(s[n][q], pair(add[n], q));
                }
                if constexpr (kVec) out[32 * n] = V::from_pairs(s[n]);
                else out[32 * n] = from_f32<T>(f32x2::lo(s[n][0]));
            }
    }
}

// dy[row[t][j]] = weight[t][j] dout[t],  dweight[t][j] = <dout[t], y[row[t][j]]>.  A
// warp per slot, so that a row's product stays in the warp; the warps of a token read
// its dout from L1.  HBM bounds it: 4099 x 6 rows of 2048 fp16 34.4 us (floor 32.3); element
// by element 4096 x 4 rows of 2047 bf16 41 (22).  dweight of a slot without a row is 0.
constexpr int kSlotWarps = 8;
template <typename T, bool kVec>
__global__ void __launch_bounds__(kSlotWarps * 32)
moe_combine_backward_kernel(const CombineArgs a, unsigned int* status) {
    using V = Vec<T>;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t s = int64_t(blockIdx.x) * kSlotWarps + (threadIdx.x >> 5);
    if (s >= a.tokens * a.k) return;
    const int64_t token = s / a.k;
    int64_t r = a.row[s];
    if (r >= a.total_rows) {
        set_device_status(status, kStatusBadArg);
        r = -1;
    }
    if (r < 0) {
        if (a.dweight && lane == 0) a.dweight[s] = 0.0f;
        return;
    }
    const T* dout = static_cast<const T*>(a.dout) + token * a.ld_dout;
    const T* y = static_cast<const T*>(a.y) + r * a.ld_y;
    T* dy = a.dy ? static_cast<T*>(a.dy) + r * a.ld_dy : nullptr;
    const float w = a.weight[s];
    float dot = 0.0f;
    if constexpr (kVec) {
        const uint64_t w2 = f32x2::both(w);
        const int64_t nvec = a.hidden / V::kN;
        uint64_t sum = 0;
        constexpr int kAhead = 4;                          // vectors in flight
        for (int64_t i0 = lane; i0 < nvec; i0 += 32 * kAhead) {
            uint4 d[kAhead], v[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int64_t i = i0 + 32 * q;
                d[q] = i < nvec ? reinterpret_cast<const uint4*>(dout)[i] : make_uint4(0, 0, 0, 0);
                if (a.dweight) v[q] = i < nvec ? reinterpret_cast<const uint4*>(y)[i] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int64_t i = i0 + 32 * q;
                if (i >= nvec) break;
                uint64_t o[V::kPairs];
#pragma unroll
                for (int p = 0; p < V::kPairs; ++p) {
                    const uint64_t dp = V::pair(d[q], p);
                    o[p] = f32x2::mul(dp, w2);
                    if (a.dweight) sum = f32x2::fma(dp, V::pair(v[q], p), sum);
                }
                if (dy) reinterpret_cast<uint4*>(dy)[i] = V::from_pairs(o);
            }
        }
        dot = f32x2::lo(sum) + f32x2::hi(sum);
    } else {
        constexpr int kAhead = 8;                          // elements in flight
        for (int64_t i0 = lane; i0 < a.hidden; i0 += 32 * kAhead) {
            T d[kAhead], v[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const bool live = i0 + 32 * q < a.hidden;
                d[q] = live ? dout[i0 + 32 * q] : from_f32<T>(0.0f);
                if (a.dweight) v[q] = live ? y[i0 + 32 * q] : from_f32<T>(0.0f);
            }
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                if (i0 + 32 * q >= a.hidden) break;
                const float f = to_f32(d[q]);
                if (a.dweight) dot = fmaf(f, to_f32(v[q]), dot);
                if (dy) dy[i0 + 32 * q] = from_f32<T>(f * w);
            }
        }
    }
    if (a.dweight) {
        dot = warp_sum(dot);
        if (lane == 0) a.dweight[s] = dot;
    }
}

// ---------------------------------------------------------------- launches

template <typename T, int kN>
cudaError_t route_n(const RouteArgs& a, bool backward, cudaStream_t stream) {
    const dim3 grid(unsigned((a.tokens + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
    if (backward) return launch_dependent(route_backward_kernel<T, kN>, grid, block, stream, a);
    if constexpr (sizeof(T) == 2)
        if (!a.bias) return launch_dependent(route_kernel<T, kN, true>, grid, block, stream, a);
    return launch_dependent(route_kernel<T, kN, false>, grid, block, stream, a);
}

template <typename T>
cudaError_t route_t(const RouteArgs& a, bool backward, cudaStream_t stream) {
    if (a.experts <= 32) return route_n<T, 1>(a, backward, stream);
    if (a.experts <= 64) return route_n<T, 2>(a, backward, stream);
    if (a.experts <= 128) return route_n<T, 4>(a, backward, stream);
    if (a.experts <= 256) return route_n<T, 8>(a, backward, stream);
    if (a.experts <= 512) return route_n<T, 16>(a, backward, stream);
    return route_n<T, 32>(a, backward, stream);
}

te_mx_status route_any(const RouteArgs& a, bool backward, cudaStream_t stream) {
    cudaError_t e = a.dtype == TE_MX_FP32   ? route_t<float>(a, backward, stream)
                    : a.dtype == TE_MX_FP16 ? route_t<__half>(a, backward, stream)
                                            : route_t<__nv_bfloat16>(a, backward, stream);
    return cuda_status(e, "router kernel launch");
}

template <int kBytes>
cudaError_t dispatch_launch(const DispatchArgs& a, unsigned int* status, cudaStream_t stream) {
    const int64_t per = int64_t(kCopyThreads) * kCopyPieces<kBytes>, pieces = a.row_bytes / kBytes;
    const int64_t parts = pieces > per ? (pieces + per - 1) / per : 1;
    return launch_dependent(moe_dispatch_kernel<kBytes>, dim3(unsigned(a.tokens * parts)), dim3(kCopyThreads), stream, a,
                            int(parts), status);
}

template <typename T, bool kVec, int kN, int kJ>
cudaError_t combine_launch(const CombineArgs& a, int sms, unsigned int* status, cudaStream_t stream) {
    const int64_t pieces = kVec ? a.hidden / Vec<T>::kN : a.hidden, parts = (pieces + 32 * kN - 1) / (32 * kN);
    // All blocks resident (a second wave of persistent blocks would take as long as the
    // first); a block is one warp, so that every warp has a part whatever their number, or up
    // to four where all the work is resident at once (64 x 8 x 7168 bf16: 2.6 us, 2.8 with
    // one; 9044 x 6 x 2816 59.8, 57.4; 8192 x 2 x 5120 62.5, 60.0) or the parts are so many
    // that a few warps without one do not count (a grid has 65535 rows of blocks at most)
    const int64_t resident = int64_t(sms) * kCombineWarps;
    const int64_t most_warps = a.tokens * parts <= resident || parts > 1024 ? kCombineThreads / 32 : 1;
    const int64_t rows_of_blocks = (parts + most_warps - 1) / most_warps;
    const int warps = int((parts + rows_of_blocks - 1) / rows_of_blocks);
    const int64_t most = resident / warps > rows_of_blocks ? resident / warps / rows_of_blocks : 1;
    return launch_dependent(moe_combine_kernel<T, kVec, kN, kJ>, dim3(unsigned(a.tokens < most ? a.tokens : most), unsigned(rows_of_blocks)),
                            dim3(unsigned(32 * warps)), stream, a, status);
}

template <typename T>
cudaError_t combine(const CombineArgs& a, bool backward, int sms, unsigned int* status, cudaStream_t stream) {
    auto fits = [&](const void* p, int64_t ld, int64_t rows) { return !p || rows_on16(p, ld, rows, sizeof(T)); };
    const bool vec = a.hidden % Vec<T>::kN == 0 && fits(a.y, a.ld_y, a.total_rows) && fits(a.residual, a.ld_residual, a.tokens) &&
                     fits(a.out, a.ld_out, a.tokens) && fits(a.dout, a.ld_dout, a.tokens) && fits(a.dy, a.ld_dy, a.total_rows);
    if (backward) {
        const dim3 grid(unsigned((a.tokens * a.k + kSlotWarps - 1) / kSlotWarps)), block(kSlotWarps * 32);
        return vec ? launch_dependent(moe_combine_backward_kernel<T, true>, grid, block, stream, a, status)
                   : launch_dependent(moe_combine_backward_kernel<T, false>, grid, block, stream, a, status);
    }
    if (!vec) return combine_launch<T, false, 8, 4>(a, sms, status, stream);
    if (a.k <= 2) return combine_launch<T, true, 4, 2>(a, sms, status, stream);
    if (a.k <= 4) return combine_launch<T, true, 2, 4>(a, sms, status, stream);
    return combine_launch<T, true, 1, 8>(a, sms, status, stream);
}

te_mx_status combine_any(const CombineArgs& a, bool backward, cudaStream_t stream) {
    unsigned int* status = nullptr;
    int sms = 0;
    te_mx_status st = device_status_ptr(&status);
    if (st != TE_MX_OK || (st = device_sm_count(&sms)) != TE_MX_OK) return st;
    cudaError_t e = a.dtype == TE_MX_FP32   ? combine<float>(a, backward, sms, status, stream)
                    : a.dtype == TE_MX_FP16 ? combine<__half>(a, backward, sms, status, stream)
                                            : combine<__nv_bfloat16>(a, backward, sms, status, stream);
    return cuda_status(e, "combine kernel launch");
}

}  // namespace

te_mx_status route_launch(const RouteArgs& a, cudaStream_t stream) { return route_any(a, false, stream); }
te_mx_status route_backward_launch(const RouteArgs& a, cudaStream_t stream) { return route_any(a, true, stream); }

// Blocks of the sort: one up to where a cluster is faster (2048 slots: 6.3 us, 8 blocks
// 6.4; 8192: 12, 6.7; with up to 256 experts one of 8 warps: 400 slots 4.3 us, 32 warps 5.4), eight, and sixteen, if the device takes such clusters, from where
// those are faster (16384: 7.2, 7.4; 32768: 8.7, 8.0; 131072: 15.8, 11.3).
constexpr int64_t kSortAlone = 2048, kSortEight = 16384;

// Whether the device launches the kernel in clusters of 16 blocks, with the shared memory
// of the most experts that it takes; looked up once per kernel and device, and the
// attribute for it set then.
static bool wide_clusters(const void* kern, int which, cudaLaunchConfig_t cfg) {
    static std::mutex mu;
    static int8_t known[5][64];                            // 0: not looked up, 1: yes, -1: no
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lock(mu);
    int8_t& k = known[which][dev];
    if (k == 0) {
        int n = 0;
        cfg.dynamicSmemBytes = size_t(kSortBlockSlots + kSortWarps * (which == 4 ? kMaxExperts : 32 << which)) * 4;
        const bool ok = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0;
        if (!ok) (void)cudaGetLastError();
        k = ok ? 1 : -1;
    }
    return k > 0;
}

te_mx_status moe_sort_launch(const int32_t* index, int64_t slots, int32_t experts, int32_t* group_m, int32_t* row,
                             int32_t* slot, cudaStream_t stream) {
    unsigned int* status = nullptr;
    te_mx_status st = device_status_ptr(&status);
    if (st != TE_MX_OK) return st;
    const int which = experts <= 32 ? 0 : experts <= 64 ? 1 : experts <= 128 ? 2 : experts <= 256 ? 3 : 4;
    auto kern = which == 0 ? moe_sort_kernel<5, kSortWarps> : which == 1 ? moe_sort_kernel<6, kSortWarps>
                : which == 2 ? moe_sort_kernel<7, kSortWarps> : which == 3 ? moe_sort_kernel<8, kSortWarps>
                                                                           : moe_sort_kernel<10, kSortWarps>;
    int warps = kSortWarps;
    if (slots <= kSortAlone && experts <= 32 * kSortFewWarps) {
        kern = moe_sort_kernel<8, kSortFewWarps>;
        warps = kSortFewWarps;
    }
    cudaError_t e = set_smem_attribute_once(reinterpret_cast<const void*>(kern), (kSortBlockSlots + kSortWarps * kMaxExperts) * 4);
    if (e != cudaSuccess) return cuda_status(e, "expert sort kernel attributes");
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(unsigned(32 * warps));
    cfg.dynamicSmemBytes = size_t(32 * warps * kSortHeld + warps * experts) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    int blocks = 1;
    auto clusters_of = [&](int n) {
        blocks = n;
        cfg.gridDim = dim3(unsigned(n));
        attr[1].val.clusterDim.x = unsigned(n);
        cfg.numAttrs = n > 1 ? 2 : 1;
    };
    clusters_of(slots <= kSortAlone ? 1 : slots <= kSortEight ? 8 : kSortCluster);
    if (blocks == kSortCluster && !wide_clusters(reinterpret_cast<const void*>(kern), which, cfg)) clusters_of(8);
    e = cudaLaunchKernelEx(&cfg, kern, index, slots, experts, blocks, group_m, row, slot, status);
    return cuda_status(e, "expert sort kernel launch");
}

te_mx_status moe_dispatch_launch(const DispatchArgs& a, cudaStream_t stream) {
    unsigned int* status = nullptr;
    te_mx_status st = device_status_ptr(&status);
    if (st != TE_MX_OK) return st;
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) | uintptr_t(a.row_bytes) |
                          (a.tokens > 1 ? uintptr_t(a.ld_x) : 0) | (a.total_rows > 1 ? uintptr_t(a.ld_out) : 0);
    cudaError_t e = all % 16 == 0  ? dispatch_launch<16>(a, status, stream)
                    : all % 4 == 0 ? dispatch_launch<4>(a, status, stream)
                    : all % 2 == 0 ? dispatch_launch<2>(a, status, stream)
                                   : dispatch_launch<1>(a, status, stream);
    return cuda_status(e, "dispatch kernel launch");
}

te_mx_status moe_combine_launch(const CombineArgs& a, cudaStream_t stream) { return combine_any(a, false, stream); }
te_mx_status moe_combine_backward_launch(const CombineArgs& a, cudaStream_t stream) { return combine_any(a, true, stream); }

}  // namespace temx
