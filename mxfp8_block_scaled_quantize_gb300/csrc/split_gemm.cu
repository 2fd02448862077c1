// MXFP8 GEMM for few tokens or few output tiles, plain, gated or gated over
// experts (whose blocks of tokens are found on the device): where the 256-
// column tiles of gemm.cu leave SMs idle, and where the bytes of the weights are
// what the call costs.
//
// The operands change places: rows of the weights are the MMA's M = 128 rows,
// tokens its N columns (a block of up to 128, rounded up to 16), so a block
// reads 16 KB of weights per 128 of K whatever the tokens are, and tiles are 128
// weight rows each: 128 output columns, or for the gated GEMM the 64 gate rows
// and the 64 up rows of 64 output columns.  Where even those leave SMs idle, K is
// split over a cluster of up to 8 blocks, which add up their accumulators
// through distributed shared memory in rank order (deterministic).  Two blocks
// fit on an SM.  Measured (us; the bytes' floor, here, the tiles of gemm.cu):
//   gated, 1 token, 7168 -> 2 x 18432       40.1   43.3   56
//   gated, 1 token, 4096 -> 2 x 1024         1.3    6     17
//   gated, 300 tokens, 4096 -> 2 x 1024      1.7   11.4   20
//   grouped, 1 token to 8 of 128 experts, 4096 -> 2 x 768
//                                            7.7   14.0   27.8
//   plain, 1 x 7168 x 18432                 20.1   24.4   94
//   plain, 1000 x 1024 x 8192                2.8   15.7   29.6
//
// One tile per block, 8 warps:
//   warp 0     TMA producer: weights (128-byte swizzle) and tokens into a ring;
//   warp 1     TMEM owner and MMA issuer (tcgen05.mma.kind::mxf8f6f4.block_scale);
//   warp 2     scale factors: a group is 4 K-steps; row-major scale tiles are
//              turned into the tcgen05 layout in place and copied into TMEM;
//   warps 4-7  the accumulator's 128 lanes -> shared memory, [token][row] fp32;
//   all        8 output columns per thread: summed over the cluster, bias,
//              activation and product (gated), 16-byte stores.
// Every mbarrier wait is bounded; a wait that gives up aborts the block cleanly
// and sets the device status word.
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "f32x2.cuh"
#include "gated_act.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "temx_internal.h"

namespace temx {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsW = 128;                  // weight rows per tile = accumulator lanes
template <bool kGated> constexpr int kCols = kGated ? kRowsW / 2 : kRowsW;       // output columns per tile
constexpr int kTokens = 128;                 // tokens per tile, at most
constexpr int kK = 128;                      // K per stage (bytes of E4M3)
constexpr int kWBytes = kRowsW * kK;
constexpr int kMaxStages = 8;
constexpr int kSfSlots = 3;                  // scale groups in shared memory, and in TMEM
constexpr int kSfAhead = 2;                  // groups loaded ahead of the one being prepared
constexpr int kSfSlotBytes = 2 * kRowsW * 16;        // the weights' 128 rows, then up to 128 tokens' x 16 scale bytes
constexpr int kSmemBytes = 112 * 1024;       // per block (two per SM)
constexpr uint32_t kTmemCols = 256;          // accumulator [0, 128), scale factors from 128: 12 K-step slots of 8
constexpr uint32_t kSfCol0 = 128;
constexpr int kTilePitch = kRowsW + 4;       // floats per token of the accumulator tile in shared memory
constexpr int kMaxSplit = 8;

struct SplitParams {
    int32_t M, N, K;         // M: tokens in all; N: output columns (gated: W has 2N rows, per group)
    int32_t groups;          // 0: dense
    const int32_t* group_m;  // device
    int32_t n;               // tokens of a tile, rounded up to 16
    int32_t n_tiles;         // tiles along N; the tile index goes through them first
    int32_t k_iters;         // K / 128
    int32_t split;           // blocks of a cluster, each with its part of K
    int32_t stages;
    const uint16_t* bias;    // bf16 [N] (gated: [2N], per group) or null
    uint16_t* D;             // bf16 [M x N]
    uint16_t* aux;           // gated: bf16 [M x 2N] or null
    int32_t act;
    unsigned int* status;
};

struct __align__(16) SplitShared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t sf_full[kSfSlots];              // a group's scale bytes landed
    uint64_t sf_ready[kSfSlots];             // its scale factors are in TMEM
    uint64_t grp_done[kSfSlots];             // its MMAs completed
    uint64_t acc_full;                       // every MMA completed
    uint32_t tmem_base;
    int32_t abort;
    int32_t group, m0, row_end;              // grouped: this block's tokens (group < 0: none)
};

// Grouped: finds the `want`-th block of up to 128 tokens among the groups' rows
// (one warp).  Sizes are clamped so that no group reaches past M; a negative size
// or a sum above M sets the status word, once per launch.
__device__ __forceinline__ void find_block(const SplitParams& p, SplitShared& sh, int32_t want, int lane) {
    const int per = (p.groups + 31) / 32, lo = min(p.groups, lane * per), hi = min(p.groups, lo + per);
    bool bad = false;
    int64_t rows = 0;
    for (int g = lo; g < hi; ++g) {
        bad |= p.group_m[g] < 0;
        rows += max(p.group_m[g], 0);
    }
    int64_t incl = rows;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    bad |= lane == 31 && incl > p.M;
    const int64_t first = incl - rows, M = p.M;
    auto blocks_of = [&](int64_t row, int32_t m) { return int32_t((min(row + m, M) - min(row, M) + kTokens - 1) / kTokens); };
    int32_t blocks = 0;
    int64_t row = first;
    for (int g = lo; g < hi; ++g) {
        const int32_t m = max(p.group_m[g], 0);
        blocks += blocks_of(row, m);
        row += m;
    }
    int32_t b = blocks;
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xFFFFFFFFu, b, o);
        if (lane >= o) b += v;
    }
    if (lane == 31 && want >= b) sh.group = -1;
    b -= blocks;                                          // blocks before this lane's groups
    if (want >= b && want < b + blocks) {
        row = first;
        for (int g = lo; g < hi; ++g) {
            const int32_t m = max(p.group_m[g], 0), n = blocks_of(row, m);
            if (want >= b && want < b + n) {
                sh.group = g;
                sh.m0 = int32_t(row) + (want - b) * kTokens;
                sh.row_end = int32_t(min(row + m, M));
            }
            b += n;
            row += m;
        }
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0 && blockIdx.x == 0) set_device_status(p.status, kStatusBadArg);
}

// Bounded mbarrier wait that also returns false once another role aborted.
__device__ __forceinline__ bool wait_or_abort(const uint64_t& b, uint32_t parity, SplitShared& sh, unsigned int* status) {
    const uint32_t bar = smem_u32(&b);
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    volatile int32_t* abort_flag = &sh.abort;
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            set_device_status(status, kStatusTimeout);
            *abort_flag = 1;
            return false;
        }
    }
}

// Raw scale rows (row r: 16 bytes = 4 words, word c = the 4 scale bytes of
// K-step c) of a 128-row atom -> scale-factor layout for tcgen05.cp 32x128b:
// for K-step c 512 bytes where byte j*16 + i*4 + b is scale byte b of row 32i +
// j.  In place; the whole warp reads before anyone writes.
__device__ __forceinline__ void sf_layout(uint32_t sf, int lane) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lds128(sf + (32 * i + lane) * 16);
    __syncwarp();
    sts128(sf + 0 * 512 + lane * 16, v[0].x, v[1].x, v[2].x, v[3].x);
    sts128(sf + 1 * 512 + lane * 16, v[0].y, v[1].y, v[2].y, v[3].y);
    sts128(sf + 2 * 512 + lane * 16, v[0].z, v[1].z, v[2].z, v[3].z);
    sts128(sf + 3 * 512 + lane * 16, v[0].w, v[1].w, v[2].w, v[3].w);
}

// 32 lanes x 16 consecutive 32-bit columns -> 16 registers per thread.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}

// 16 bytes of the same shared-memory variable in block `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t to_bf16x2(uint64_t v) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f32x2::hi(v)), "f"(f32x2::lo(v)));
    return r;
}

template <bool kGated, bool kGrouped>
__global__ void __launch_bounds__(kThreads, 2)
split_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_sw, const __grid_constant__ CUtensorMap map_sx,
                  const SplitParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ SplitShared sh;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // (broadcast: the compiler then knows them to be the same in all lanes)
    const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = __shfl_sync(0xFFFFFFFFu, p.split > 1 ? cluster_ctarank() : 0u, 0);
    constexpr int kTileCols = kCols<kGated>;
    const int32_t tile = int32_t(blockIdx.x) / p.split;
    const int32_t f0 = tile % p.n_tiles * kTileCols;     // first output column
    const uint32_t stage_bytes = uint32_t(kWBytes + p.n * kK);
    const uint32_t sf_ring = smem_u32(smem) + uint32_t(p.stages) * stage_bytes;
    // this block's scale groups (4 K-steps each) and K-steps
    const int32_t groups = (p.k_iters + 3) / 4;
    const int32_t g0 = int32_t(int64_t(groups) * rank / p.split), g1 = int32_t(int64_t(groups) * (rank + 1) / p.split);
    const int32_t k0 = 4 * g0, k1 = min(4 * g1, p.k_iters);

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        for (int s = 0; s < kSfSlots; ++s) {
            mbar_init(smem_u32(&sh.sf_full[s]), 1);
            mbar_init(smem_u32(&sh.sf_ready[s]), 1);
            mbar_init(smem_u32(&sh.grp_done[s]), 1);
        }
        mbar_init(smem_u32(&sh.acc_full), 1);
        sh.abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_sw);
        tma_prefetch_desc(&map_sx);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (kGrouped && warp == 3) find_block(p, sh, tile / p.n_tiles, lane);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem_base, 0);
    if (kGrouped && sh.group < 0) {                      // (every block of a cluster)
        if (warp == 1) tmem_dealloc(tmem, kTmemCols);
        return;
    }
    // first token, end of the tile's tokens, group, its first row of W
    const int32_t m0 = kGrouped ? sh.m0 : tile / p.n_tiles * kTokens, row_end = kGrouped ? sh.row_end : p.M;
    const int32_t group = kGrouped ? sh.group : 0, w0 = group * (kGated ? 2 : 1) * p.N + f0;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            int32_t s = 0;
            uint32_t phase = 1;                          // (the first pass finds every stage free)
            for (int32_t k = k0; k < k1; ++k) {
                if (!wait_or_abort(sh.empty[s], phase, sh, p.status)) break;
                const uint32_t dst = smem_u32(smem) + uint32_t(s) * stage_bytes, bar = smem_u32(&sh.full[s]);
                mbar_arrive_expect_tx(bar, stage_bytes);
                tma_load_2d(dst, &map_w, bar, k * kK, w0);
                if constexpr (kGated)                    // (the box is 64 rows: gate, then up)
                    tma_load_2d(dst + kWBytes / 2, &map_w, bar, k * kK, p.N + w0);
                tma_load_2d(dst + kWBytes, &map_x, bar, k * kK, m0);
                if (++s == p.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (sh.abort)                                // gave up: let the loads in flight land
                for (int i = 0; i < p.stages; ++i)
                    for (uint32_t q = 0; q < 2; ++q) mbar_wait(smem_u32(&sh.full[i]), q, p.status, 1000000ull);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (the warp together, lane 0 issues)
        const uint32_t issue = lane == 0 ? 1u : 0u;
        // kind::mxf8f6f4 with block scaling: E4M3 A and B, both K-major, N >> 3 at
        // bit 17, UE8M0 scales (bit 23), M >> 4 at bit 24; scale-factor byte ids
        // at bits 4..5 (B) and 29..30 (A)
        const uint32_t idesc = (uint32_t(p.n >> 3) << 17) | (1u << 23) | (uint32_t(kRowsW >> 4) << 24);
        // Every value of the loop is warp-uniform, and the next barriers are tested
        // between a K-step's MMAs and its commits: 4 MMAs cost 255 ns however few
        // tokens they have, and cost 348 ns without.
        uint32_t s = 0, phase = 0, slot = 0, sf_phase = 0;
        bool ok = true, landed = false, sf_landed = false;
        for (int32_t k = k0; k < k1; k += 4) {           // a scale group
            const int32_t steps = min(4, k1 - k);
            const uint32_t next_slot = slot + 1 == kSfSlots ? 0 : slot + 1;
            const uint32_t next_sf_phase = sf_phase ^ (next_slot == 0 ? 1u : 0u);
            for (int32_t c = 0; c < steps; ++c) {
                ok = __all_sync(0xFFFFFFFFu, landed) || __all_sync(0xFFFFFFFFu, wait_or_abort(sh.full[s], phase, sh, p.status));
                if (ok && c == 0) {
                    ok = __all_sync(0xFFFFFFFFu, sf_landed) ||
                         __all_sync(0xFFFFFFFFu, wait_or_abort(sh.sf_ready[slot], sf_phase, sh, p.status));
                    tc_fence_after();
                }
                if (!ok) break;
                const uint32_t st = smem_u32(smem) + s * stage_bytes;
                const uint64_t a_desc = smem_desc(st, 16, 1024, 2), b_desc = smem_desc(st + kWBytes, 16, 1024, 2);
                const uint32_t sf = tmem + kSfCol0 + (slot * 4 + uint32_t(c)) * 8;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)           // (+32 bytes along K = +2 in the address field)
                    mma_mxf8_if(tmem, a_desc + 2 * kk, b_desc + 2 * kk, idesc | (uint32_t(kk) << 4) | (uint32_t(kk) << 29), sf,
                                sf + 4, (k - k0) | c | kk ? 1u : 0u, issue);
                const uint32_t next = s + 1 == uint32_t(p.stages) ? 0 : s + 1;
                const uint32_t next_phase = phase ^ (next == 0 ? 1u : 0u);
                landed = mbar_test(smem_u32(&sh.full[next]), next_phase);
                if (c == steps - 1) sf_landed = mbar_test(smem_u32(&sh.sf_ready[next_slot]), next_sf_phase);
                tc_commit_if(smem_u32(&sh.empty[s]), issue);
                if (c == steps - 1) tc_commit_if(smem_u32(&sh.grp_done[slot]), issue);
                s = next;
                phase = next_phase;
            }
            if (!ok) break;
            slot = next_slot;
            sf_phase = next_sf_phase;
        }
        tc_commit_if(smem_u32(&sh.acc_full), issue);
        if (!ok && lane == 0)                            // gave up: let the MMAs in flight end before TMEM is freed
            mbar_wait(smem_u32(&sh.acc_full), 0, p.status, 1000000ull);
    } else if (warp == 2) {
        // ------------------------------------------------ scale factors
        auto load = [&](int32_t j) {                     // group j (of this block), by lane 0
            const uint32_t bar = smem_u32(&sh.sf_full[j % kSfSlots]), dst = sf_ring + uint32_t(j % kSfSlots) * kSfSlotBytes;
            mbar_arrive_expect_tx(bar, uint32_t(16 * (kRowsW + p.n)));
            tma_load_2d(dst, &map_sw, bar, (g0 + j) * 16, w0);
            if constexpr (kGated) tma_load_2d(dst + kRowsW * 8, &map_sw, bar, (g0 + j) * 16, p.N + w0);
            tma_load_2d(dst + kRowsW * 16, &map_sx, bar, (g0 + j) * 16, m0);
        };
        const int32_t n_groups = g1 - g0;
        if (lane == 0)
            for (int32_t j = 0; j < kSfAhead && j < n_groups; ++j) load(j);
        for (int32_t j = 0; j < n_groups; ++j) {
            const int32_t slot = j % kSfSlots;
            const uint32_t bit = uint32_t(j / kSfSlots) & 1u;
            bool ok = __all_sync(0xFFFFFFFFu, wait_or_abort(sh.sf_full[slot], bit, sh, p.status));
            if (ok) {
                const uint32_t sf = sf_ring + uint32_t(slot) * kSfSlotBytes;
                sf_layout(sf, lane);
                sf_layout(sf + kRowsW * 16, lane);       // (rows past the tokens: bytes that no MMA reads)
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    // the slot's columns are free once the MMAs of the group before in it completed
                    if (j >= kSfSlots) ok = wait_or_abort(sh.grp_done[slot], bit ^ 1u, sh, p.status);
                    if (ok) {
                        tc_fence_after();
                        const int32_t steps = min(4, k1 - k0 - 4 * j);
                        for (int32_t c = 0; c < steps; ++c) {
                            const uint32_t col = tmem + kSfCol0 + uint32_t(slot * 4 + c) * 8;
                            tc_cp_32x128b_warpx4(col, smem_desc(sf + c * 512, 0, 128, 0));
                            tc_cp_32x128b_warpx4(col + 4, smem_desc(sf + kRowsW * 16 + c * 512, 0, 128, 0));
                        }
                        tc_commit(smem_u32(&sh.sf_ready[slot]));
                        // group j + 2 takes the slot of group j - 1, once its copies have landed
                        if (j + kSfAhead < n_groups) {
                            if (j > 0) ok = wait_or_abort(sh.sf_ready[(j - 1) % kSfSlots], uint32_t((j - 1) / kSfSlots) & 1u, sh,
                                                          p.status);
                            if (ok) load(j + kSfAhead);
                        }
                    }
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            }
            if (!ok) break;
        }
        if (sh.abort && lane == 0)                       // gave up: let the scale loads in flight land
            for (int i = 0; i < kSfSlots; ++i)
                for (uint32_t q = 0; q < 2; ++q) mbar_wait(smem_u32(&sh.sf_full[i]), q, p.status, 1000000ull);
    } else if (warp >= 4) {
        // ------------------------------------------------ accumulator -> [token][row] fp32
        if (__all_sync(0xFFFFFFFFu, wait_or_abort(sh.acc_full, 0, sh, p.status))) {
            tc_fence_after();
            const int q = warp & 3;
            float* acc = reinterpret_cast<float*>(smem) + 32 * q + lane;           // (every stage has been read)
            for (int32_t c = 0; c < p.n; c += 16) {
                uint32_t v[16];
                tmem_ld_x16(tmem + (uint32_t(32 * q) << 16) + uint32_t(c), v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[(c + i) * kTilePitch] = __uint_as_float(v[i]);
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (p.split > 1) cluster_sync();                     // every block's partial accumulators are in its shared memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    // Items (token, 8 columns), a contiguous part of them per block of the cluster
    // (neighbouring threads read neighbouring bytes: 128 tokens, 4096 -> 2 x 1024,
    // 14.9 us; 19.5 us with a token per thread)
    constexpr int kChunks = kTileCols / 8;
    const int32_t items = min(kTokens, row_end - m0) * kChunks, i1 = int32_t(int64_t(items) * (rank + 1) / p.split);
    for (int32_t i = int32_t(int64_t(items) * rank / p.split) + int32_t(threadIdx.x); i < i1; i += kThreads) {
        const int32_t m = i / kChunks, c = i % kChunks * 8, f = f0 + c;
        if (f >= p.N) continue;                          // (N % 16 == 0: 8 columns are in or out together)
        uint64_t v[kGated ? 2 : 1][4];                   // (gate, up)
#pragma unroll
        for (int half = 0; half < (kGated ? 2 : 1); ++half) {
            const uint32_t off = uint32_t(m * kTilePitch + half * kTileCols + c) * 4;
            float4 a = make_float4(0, 0, 0, 0), b = a;
            if (p.split == 1) {
                a = *reinterpret_cast<const float4*>(smem + off);
                b = *reinterpret_cast<const float4*>(smem + off + 16);
            } else {
                const uint32_t addr = smem_u32(smem) + off;
                float4 x[kMaxSplit], y[kMaxSplit];       // (every load in flight before the first is added)
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r)
                    if (r < p.split) {
                        x[r] = ld_cluster(addr, uint32_t(r));
                        y[r] = ld_cluster(addr + 16, uint32_t(r));
                    }
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r)
                    if (r < p.split) {
                        a.x += x[r].x; a.y += x[r].y; a.z += x[r].z; a.w += x[r].w;
                        b.x += y[r].x; b.y += y[r].y; b.z += y[r].z; b.w += y[r].w;
                    }
            }
            v[half][0] = f32x2::pack(a.x, a.y);
            v[half][1] = f32x2::pack(a.z, a.w);
            v[half][2] = f32x2::pack(b.x, b.y);
            v[half][3] = f32x2::pack(b.z, b.w);
            if (p.bias) {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.bias + ((kGated ? 2 : 1) * group + half) * int64_t(p.N) + f));
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) v[half][k] = f32x2::add(v[half][k], f32x2::pack(bf16_lo(ww[k]), bf16_hi(ww[k])));
            }
            if (kGated && p.aux)
                st_global_v4(p.aux + (2 * int64_t(m0 + m) + half) * p.N + f, to_bf16x2(v[half][0]), to_bf16x2(v[half][1]),
                             to_bf16x2(v[half][2]), to_bf16x2(v[half][3]));
        }
        if constexpr (kGated)
            gated::with(p.act, [&](auto act) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[0][k] = f32x2::mul(gated::act2<decltype(act)::value>(v[0][k]), v[1][k]);
            });
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = to_bf16x2(v[0][k]);
        st_global_v4(p.D + int64_t(m0 + m) * p.N + f, o[0], o[1], o[2], o[3]);
    }
    if (p.split > 1) cluster_sync();                     // no block leaves while another may still read its shared memory
}

// Blocks of up to 128 tokens that M tokens can make in `groups` groups (or one).
int64_t token_blocks(int64_t M, int64_t groups) {
    if (groups == 0) return (M + kTokens - 1) / kTokens;
    return (M < groups ? M : groups) + M / kTokens;
}

template <bool kGated, bool kGrouped>
te_mx_status launch(const GemmArgs& a, int sms, cudaStream_t stream) {
    SplitParams p{};
    p.M = int32_t(a.M); p.N = int32_t(a.N); p.K = int32_t(a.K);
    p.n = p.M < kTokens ? (p.M + 15) / 16 * 16 : kTokens;
    p.n_tiles = (p.N + kCols<kGated> - 1) / kCols<kGated>;
    p.k_iters = p.K / kK;
    p.groups = a.groups;
    p.group_m = a.group_m;
    p.bias = static_cast<const uint16_t*>(a.has_bias ? a.bias : nullptr);
    p.D = static_cast<uint16_t*>(a.D);
    p.aux = static_cast<uint16_t*>(a.aux);
    p.act = a.act;
    te_mx_status st = device_status_ptr(&p.status);
    if (st != TE_MX_OK) return st;
    // Split K while two blocks per SM are not there, down to one scale group (512
    // of K) per block; with several blocks of tokens, whose accumulators are
    // whole tiles to add up, at most four ways and past two only up to a block
    // per SM (512 x 1024 x 4096: 19 us eight ways, 10.6 four ways)
    const int64_t tiles = int64_t(p.n_tiles) * token_blocks(p.M, p.groups), groups = (p.k_iters + 3) / 4;
    const bool few = p.M <= kTokens;
    p.split = 1;
    while (p.split < (few ? kMaxSplit : 4) && 2 * p.split <= groups &&
           tiles * 2 * p.split <= (few || p.split == 1 ? 2 * sms : sms))
        p.split *= 2;
    const int stage = kWBytes + p.n * kK;
    p.stages = (kSmemBytes - 1024 - kSfSlots * kSfSlotBytes) / stage;
    if (p.stages > kMaxStages) p.stages = kMaxStages;

    // (rows of scales are at least 16 bytes: their pitch is)
    const uint64_t K = uint64_t(p.K), sf_cols = uint64_t(p.K / 32) < 16 ? 16 : uint64_t(p.K / 32);
    const uint64_t w_rows = uint64_t(p.N) * (kGated ? 2 : 1) * uint64_t(kGrouped ? p.groups : 1);
    CUtensorMap mw, mx, msw, msx;
    if ((st = encode_tensor_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, K, w_rows, K, kK, kCols<kGated>,
                                   CU_TENSOR_MAP_SWIZZLE_128B)) != TE_MX_OK) return st;
    if ((st = encode_tensor_map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, K, uint64_t(p.M), K, kK, uint32_t(p.n),
                                   CU_TENSOR_MAP_SWIZZLE_128B)) != TE_MX_OK) return st;
    if ((st = encode_tensor_map_2d(&msw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.sB, sf_cols, w_rows, uint64_t(a.ld_sB), 16,
                                   kCols<kGated>, CU_TENSOR_MAP_SWIZZLE_NONE)) != TE_MX_OK) return st;
    if ((st = encode_tensor_map_2d(&msx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.sA, sf_cols, uint64_t(p.M), uint64_t(a.ld_sA), 16,
                                   uint32_t(p.n), CU_TENSOR_MAP_SWIZZLE_NONE)) != TE_MX_OK) return st;

    auto kern = split_gemm_kernel<kGated, kGrouped>;
    cudaError_t e = set_smem_attribute_once(reinterpret_cast<const void*>(kern), kSmemBytes);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(split GEMM)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(tiles * p.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(p.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, mw, mx, msw, msx, p), "split GEMM kernel launch");
}

}  // namespace

bool split_gemm_takes(const GemmArgs& a, int sms) {
    if (a.wgrad || a.acc_f32 || a.f32_scales || a.gelu || a.dgelu) return false;
    // grouped: few tokens, in few enough blocks for the GPU to hold all at once
    // (the sizes are on the device: as many as there can be).  Measured (us; here,
    // the tiles of gemm.cu), 4096 -> 2 x 768: 1 token to 8 of 128 experts 14.0, 27.8;
    // 32 rows of 8 experts 13.9, 19.4; 512 rows 19.3, 20.3; 1200 rows of 16 experts,
    // 1024 -> 2 x 256: 11.4, 10.0
    if (a.groups > 0)
        return a.gated && a.M <= 4 * kTokens && token_blocks(a.M, a.groups) * ((a.N + kCols<true> - 1) / kCols<true>) <= 2 * int64_t(sms);
    // (a plain GEMM below 16 K-steps has its sums in one order in gemm.cu, and keeps it)
    if (!a.gated && a.K < 16 * kK) return false;
    // plain, 65 to 128 tokens at fewer than 28 K-steps, where a tile's start and join
    // are not small beside its loop: with few tiles, split over K; with up to two
    // per SM where those fill the SMs, or up to 96 tokens.  Measured (us; here, those
    // tiles), K = 2048: 128 x 4096 10.5, 13.5; 128 x 8192 16.0, 14.1; 96 x 16384 13.9,
    // 15.3; 128 x 32768 18.7, 20.1; 128 x 65536 36.2, 32.4; 96 x 131072 59.5, 56.7;
    // K = 3584: 128 x 8192 17.6, 21.7; 128 x 65536 50.1, 51.3
    if (!a.gated && a.M > 64 && a.M <= kTokens && a.K < 28 * kK) {
        const int64_t tiles = (a.N + kCols<false> - 1) / kCols<false>;
        return 4 * tiles <= sms || (tiles <= 2 * int64_t(sms) && (a.M <= 96 || tiles > sms));
    }
    if (a.M <= kTokens) return true;
    // more tokens: while the tiles of gemm.cu (256 rows per pair of SMs, or 128
    // per SM, by 256 accumulator columns) leave half of the SMs idle, three
    // quarters with fewer than 32 K-steps.  Measured (us; here, those tiles):
    // plain 1000 x 2048 x 8192 23.4, 29.8; gated 512 tokens, 4096 -> 2 x 2048 17.6,
    // 19.4, -> 2 x 4096 20.6, 21.6; 300 tokens, 1024 -> 2 x 1024 8.7, 10.4; 1000
    // tokens 11.7, 10.6; plain 1000 x 2048 x 2048 13.0, 12.2
    const int64_t rows = a.M >= 256 ? 256 : 128, units = a.M >= 256 ? sms / 2 : sms, cols = a.gated ? 128 : 256;
    return (a.K >= 32 * kK ? 2 : 4) * ((a.M + rows - 1) / rows) * ((a.N + cols - 1) / cols) <= units;
}

te_mx_status split_gemm_launch(const GemmArgs& a, int sms, cudaStream_t stream) {
    if (a.groups > 0) return launch<true, true>(a, sms, stream);
    return a.gated ? launch<true, false>(a, sms, stream) : launch<false, false>(a, sms, stream);
}

}  // namespace temx
