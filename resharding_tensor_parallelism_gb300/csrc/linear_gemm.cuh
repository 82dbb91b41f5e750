// Products of the gated feed-forward block and of the linear layers on a
// virtual mesh of P ranks (ColossalAI "1D tensor parallelism" page, sections 2,
// 2.1 and 2.2: column-parallel and row-parallel layers and their gradients),
// with what follows the product in its epilogue:
//   LIN_OUT    out = act(acc + bias) + residual, and optionally h = acc + bias
//   LIN_GLU    y = act(X Ag) * (X Au): both projections and their product in one
//              kernel, and optionally the two pre-activations
//   LIN_DGLU   acc = dY = dZ B^T: dHg = dY * Hu * act'(Hg), dHu = dY * act(Hg)
//
// The tensor pipe bounds them: 2 rows cols kdim operations. A cluster of 2 CTAs
// (2 SMs) computes one 256 x 256 accumulator tile per step, as in the plain
// tensor-parallel MLP: warp 0 of each CTA loads its 128 rows of A and its 128
// columns of B by TMA into a 6-stage ring, one thread of the leader issues
// tcgen05.mma.cta_group::2 (256 x 256 x 16), and the other warps turn one of two TMEM
// accumulators into outputs while the next tile is multiplied. Measured on the gated
// 4096 x 4096 x 16384 block, training: tensor pipe 88 % busy in both of its kernels. For LIN_GLU the
// leader's CTA loads 128 gate columns and its peer the same 128 up columns, so
// the accumulator's two halves hold gate and up of one output column in the same
// TMEM lane: the epilogue thread of a row has both without any exchange, and X
// is read once for the two projections. A fused sum over ranks (and, for the
// input gradient, over gate and up) walks all operand pairs in one K loop.
//
// An epilogue warp takes 32 columns of its 32 rows at a time: outputs are staged in
// swizzled shared memory and leave by TMA tensor stores; the residual (or the kept
// gate and up) comes in the same way, into the same slots, while the tile is still
// being multiplied, and the bias in one load per lane. Each output is rounded to bf16
// once; Y is computed from the float32 accumulators, not from the kept, rounded
// pre-activations.
//
// SPLIT: when a product has so few tiles that two to four pairs per tile fit the GPU
// at once, a cluster of that many pairs shares a tile: each pair multiplies one part
// of the K range, leaves its float32 accumulator in its (now free) operand ring, and
// the pairs then add up every other chunk of 32 columns over distributed shared
// memory, in the order of the parts, on the way into the same epilogue.
#pragma once

#include <atomic>
#include <cstring>

#include "activation.cuh"
#include "linear.h"
#include "tcgen05.cuh"

namespace rtp {

struct LinArgs {
    CUtensorMap ta[LIN_MAX_GROUPS], tb[LIN_MAX_GROUPS];  // LIN_GLU: tb[g] gate, tb[LIN_MAX_RANKS + g] up
    CUtensorMap to[LIN_MAX_GROUPS], to2[LIN_MAX_RANKS], to3[LIN_MAX_RANKS];
    CUtensorMap ti[LIN_MAX_RANKS], ti2[LIN_MAX_RANKS];   // read by the epilogue: residual, or gate and up
    const __nv_bfloat16* bias[LIN_MAX_RANKS];
    const __nv_bfloat16* residual[LIN_MAX_RANKS];
    __nv_bfloat16* h[LIN_MAX_RANKS];  // the buffers of to2 (LIN_OUT)
    int64_t ld;  // output row stride, elements
    int32_t groups, fused, kb_per_group, m_tiles, n_tiles, rows, cols;
    int32_t total_tiles, group_m, groups_in_n;
    int32_t act, has_bias, has_residual, keep;
    int32_t kbs;    // K blocks of a tile (of all operand pairs when fused)
    int32_t split;  // SPLIT kernels: K parts of a tile, over a cluster of `split` pairs
};

namespace {

constexpr int BM = LIN_TILE_ROWS, BN = LIN_TILE_COLS;
constexpr uint32_t SUB = 64 * BK * 2;  // one 64 x 64 box, 8 KB
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr uint32_t A_BYTES = 128 * BK * 2, B_BYTES = 128 * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr uint32_t SLOT_BYTES = 2048;  // one staging slot: 32 rows x 32 bf16 columns


constexpr int LIN_NOT_SPLIT = 1;     // (positive: not a status)
constexpr int SPLIT_COST = 12;       // K blocks of time (0.28 us each) that a sum over the parts costs
// CFG_ACT: the activation's code is compiled in (LIN_OUT; a branch around so much
// code costs an instruction fetch in every step of the epilogue)
enum : int { CFG_A_T = 1, CFG_B_T = 2, CFG_F32 = 4, CFG_ACT = 8, CFG_EPI_SHIFT = 4 };

// 16 or 32 accumulator columns of this warp's 32 lanes; the registers are valid
// after tmem_wait.
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_16cols(taddr, r); }
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) { tmem_ld_wait(r); }
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_32cols(taddr, r); }
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) { tmem_ld_wait(r); }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// The barrier at the same address in both CTAs of a pair (mask: their ranks in the cluster).
__device__ __forceinline__ void mma_commit_both(uint32_t bar, uint16_t mask)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(mask)
                 : "memory");
}

// Epilogue warps and shared memory of a kernel: the operand ring and, per epilogue
// warp, a ring of staging slots (64-byte swizzled as the TMA reads and writes them; a
// float32 chunk takes two, 128-byte swizzled).
// Whole tiles: 4 warps with 4 slots, and 6 stages. 8 warps halve an epilogue, which
// is bound by instruction latency, but next to a running product they cost power and
// issue slots (8192 x 4096 x 16384 gated, training: 2.5-3 % slower).
// SPLIT: nothing runs beside the one epilogue, so 8 warps; 5 stages where the
// epilogue moves two to four times the data (LIN_GLU, LIN_DGLU) and has 4 slots.
template <int CFG, bool SPLIT>
struct Layout {
    static constexpr bool deep = (CFG >> CFG_EPI_SHIFT) != LIN_OUT;
    static constexpr int epi_warps = SPLIT ? 8 : 4, threads = 64 + 32 * epi_warps;
    static constexpr int stages = SPLIT && deep ? 5 : 6, slots = SPLIT && !deep ? 2 : 4;
    static constexpr uint32_t warp_bytes = slots * SLOT_BYTES;
    static constexpr size_t bytes = stages * STAGE_BYTES + 1024 + epi_warps * warp_bytes + 1024;  // barriers, alignment
    static_assert(bytes <= 232448, "at most 227 KB of shared memory per CTA");
};

// Instruction descriptor of tcgen05.mma kind::f16 (float32 D, bf16 A and B):
// bit 15 A M-major, bit 16 B N-major, N >> 3 from bit 17, M >> 4 from bit 24.
__host__ __device__ constexpr uint32_t idesc(bool a_t, bool b_t)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_t ? 1u : 0u) << 15) | ((b_t ? 0u : 1u) << 16) |
           ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

// Tile index -> (group, M tile, N tile): blocks of group_m M tiles, N tile after
// N tile within a block; the groups are the outermost index, or, when they
// share A, part of the N range, so that a block of A rows stays in L2 while
// every group's B columns stream past it.
__device__ __forceinline__ void tile_coords(const LinArgs& a, int tile, int& g, int& mt, int& nt)
{
    const int per_group = a.fused || a.groups_in_n ? 0 : a.m_tiles * a.n_tiles;
    g = per_group ? tile / per_group : 0;
    const int r = tile - g * per_group;
    const int span = a.group_m * (a.groups_in_n ? a.groups * a.n_tiles : a.n_tiles);
    const int first_m = (r / span) * a.group_m;
    const int rows = min(a.m_tiles - first_m, a.group_m);
    const int w = r % span;
    mt = first_m + w % rows;
    nt = w / rows;
    if (a.groups_in_n) {
        g = nt / a.n_tiles;
        nt -= g * a.n_tiles;
    }
}

template <int N>
__device__ __forceinline__ void bulk_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Barriers as in the plain tensor-parallel MLP kernel: full[s] in the leader
// (both CTAs' TMA bytes), empty[s] in both (the leader's commit), acc_full[x] in
// both, acc_empty[x] in the leader (the 4 epilogue warps of each CTA).
template <int CFG, bool SPLIT>
__global__ void __launch_bounds__(Layout<CFG, SPLIT>::threads, 1) linear_gemm_kernel(const __grid_constant__ LinArgs a)
{
    constexpr bool A_T = (CFG & CFG_A_T) != 0, B_T = (CFG & CFG_B_T) != 0, F32 = (CFG & CFG_F32) != 0;
    constexpr int EPI = CFG >> CFG_EPI_SHIFT;
    constexpr bool PLAIN = EPI == LIN_OUT && (A_T || B_T);  // gradients: the accumulator alone
    constexpr bool ACT = EPI != LIN_OUT || (CFG & CFG_ACT) != 0;
    constexpr int TILE_COLS = EPI == LIN_GLU ? BN / 2 : BN;
    using L = Layout<CFG, SPLIT>;
    constexpr int STAGES = L::stages, SLOTS = L::slots, EPI_WARPS = L::epi_warps;
    constexpr int HALVES = EPI_WARPS / 4;                                // column ranges of the epilogue warps
    constexpr int WARP_COLS = TILE_COLS / HALVES, CHUNKS = WARP_COLS / 32;  // of an epilogue warp
    // Columns a step, one or two steps a chunk. 32 halve the steps' fixed latency in a
    // whole tile's epilogue (4096 x 512 x 4096 with SiLU: 41.0 us at 16, 33.6 at 32);
    // beside the long products of LIN_GLU, and with 8 warps, 16 measured better (8192 x
    // 4096 x 16384, training: 1932 us against 1975; 256 x 2048 x 2048, split: 11.2 against
    // 12.7).
    constexpr int STEP = SPLIT || EPI == LIN_GLU ? 16 : 32;
    constexpr int PER = 32 / STEP;
    constexpr uint32_t PART_BYTES = 128 * BN * 4;  // SPLIT: a part's accumulator in shared memory
    static_assert(!SPLIT || PART_BYTES + L::epi_warps * 4096u <= L::stages * STAGE_BYTES, "in the operand ring's memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5 + SLOTS * EPI_WARPS);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(STAGES + s); };
    auto acc_full = [&](int x) { return bar0 + 8u * (uint32_t)(2 * STAGES + x); };
    auto acc_empty = [&](int x) { return bar0 + 8u * (uint32_t)(2 * STAGES + 2 + x); };
    const uint32_t drain_bar = bar0 + 8u * (uint32_t)(2 * STAGES + 4);
    auto slot_bar = [&](int w, int s) { return bar0 + 8u * (uint32_t)(2 * STAGES + 5 + SLOTS * w + s); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // SPLIT: a cluster of `split` pairs has one tile, each pair one part of its K
    // range. Otherwise a cluster is one pair, and takes tiles in turn.
    const uint32_t rank = cluster_rank(), cta = SPLIT ? rank & 1u : rank, leader = SPLIT ? rank & ~1u : 0u;
    const int parts = SPLIT ? a.split : 1, part = SPLIT ? (int)(rank >> 1) : 0;
    const int first = (int)cluster_id(), stride = SPLIT ? a.total_tiles : (int)num_clusters();
    const int kb0 = SPLIT ? (int)((int64_t)a.kbs * part / parts) : 0;
    const int kb1 = SPLIT ? (int)((int64_t)a.kbs * (part + 1) / parts) : a.kbs;
    // one barrier a thread: full and empty, acc_full, acc_empty, drain, the slots
    constexpr int NBARS = 2 * STAGES + 5 + SLOTS * EPI_WARPS;
    if (threadIdx.x < NBARS) {
        const int b = (int)threadIdx.x;
        mbar_init(bar0 + 8u * (uint32_t)b, b == 2 * STAGES + 2 || b == 2 * STAGES + 3 ? 2 * EPI_WARPS : 1);
        if (b == 0) *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        for (int g = 0; g < a.groups; ++g) {
            prefetch_map(&a.ta[g]);
            prefetch_map(&a.tb[EPI == LIN_GLU ? (int)cta * LIN_MAX_RANKS + g : g]);
        }
    }
    if (warp == 2 && lane == 0) {
        for (int g = 0; g < (a.fused ? 1 : a.groups); ++g) prefetch_map(&a.to[g]);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers are initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // launched as a programmatic dependent: the previous kernel of the stream
    // completes, and its writes are visible, before any global memory access
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Every CTA of this grid is on an SM once they have all come here, so the next
    // kernel's CTAs may take SMs as this grid's leave them, and run their set-up.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ---------------- TMA producer (one lane per CTA) ----------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_parity = 0;
            bool ok = true;
            const uint32_t smem0 = smem_u32(smem);
            const uint32_t leader_full0 = map_to_rank(full_bar(0), leader);
            for (int tile = first; ok && tile < a.total_tiles; tile += stride) {
                int g, mt, nt;
                tile_coords(a, tile, g, mt, nt);
                const int row = mt * BM + (int)cta * 128;
                const int col = EPI == LIN_GLU ? nt * TILE_COLS : nt * BN + (int)cta * 128;
                int gg = a.fused ? kb0 / a.kb_per_group : g;
                int kk = a.fused ? kb0 - gg * a.kb_per_group : kb0;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_bar(empty_bar(stage), phase ^ 1u, abort_flag, ERR_PRODUCER)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = smem0 + (uint32_t)stage * STAGE_BYTES, sb = sa + A_BYTES;
                    const uint32_t fb = leader_full0 + 8u * (uint32_t)stage;
                    if (cta == 0) mbar_expect_tx(full_bar(stage), 2 * STAGE_BYTES);
                    const CUtensorMap* am = &a.ta[gg];
                    const CUtensorMap* bm = &a.tb[EPI == LIN_GLU ? (int)cta * LIN_MAX_RANKS + gg : gg];
                    if constexpr (A_T) {  // two 64(M) x 64(K) boxes
                        tma_load_2d_pair(sa, am, fb, row, kk * BK);
                        tma_load_2d_pair(sa + SUB, am, fb, row + 64, kk * BK);
                    } else {  // one 128(M) x 64(K) box
                        tma_load_2d_pair(sa, am, fb, kk * BK, row);
                    }
                    if constexpr (B_T) {  // one 128(N) x 64(K) box
                        tma_load_2d_pair(sb, bm, fb, kk * BK, col);
                    } else {  // two 64(N) x 64(K) boxes
                        tma_load_2d_pair(sb, bm, fb, col, kk * BK);
                        tma_load_2d_pair(sb + SUB, bm, fb, col + 64, kk * BK);
                    }
                    issued |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                    if (++kk == a.kb_per_group) {  // next operand pair (fused sum)
                        kk = 0;
                        ++gg;
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                if (cta == 0) {
                    for (int s = 0; s < STAGES; ++s)
                        if ((issued >> s) & 1u) drain_wait(full_bar(s), (issued_parity >> s) & 1u);
                } else {
                    // the follower cannot wait on the leader's barrier: give its
                    // last loads (microseconds) time to land
                    const uint64_t t0 = global_ns();
                    while (global_ns() - t0 < 2000000ull) {
                    }
                }
            }
        }
        __syncwarp();
        if (SPLIT) cluster_sync();  // with the epilogue warps, before the parts are summed
    } else if (warp == 1) {
        // ---------------- MMA issuer (one lane of the leader) ----------------
        if (lane == 0 && cta == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            // K-major: 32-byte steps (16 bf16) in the 128-byte swizzle row, 8-row
            // groups 1024 bytes apart. M/N-major: 2048-byte steps (16 K rows), the
            // two 64-wide boxes SUB bytes apart.
            constexpr uint32_t a_step = A_T ? 2048u : 32u, b_step = B_T ? 32u : 2048u;
            const uint64_t desc_a0 = smem_desc(smem_u32(smem), A_T ? SUB : 16u, 1024u);
            const uint64_t desc_b0 = smem_desc(smem_u32(smem) + A_BYTES, B_T ? 16u : SUB, 1024u);
            bool ok = true;
            // (a constant for whole tiles: a mask in a register costs them 2 %)
            const uint16_t both = SPLIT ? (uint16_t)(3u << leader) : (uint16_t)3;
            for (int tile = first; ok && tile < a.total_tiles; tile += stride) {
                if (!wait_bar(acc_empty(acc), acc_phase ^ 1u, abort_flag, ERR_MMA_ACC)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_bar(full_bar(stage), phase, abort_flag, ERR_MMA_STAGE)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t off = (uint64_t)((uint32_t)stage * STAGE_BYTES >> 4);
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        mma_bf16_pair(d_tmem, desc_a0 + off + (uint64_t)(a_step * k >> 4),
                                      desc_b0 + off + (uint64_t)(b_step * k >> 4), idesc(A_T, B_T),
                                      (kb > kb0 || k > 0) ? 1u : 0u);
                    mma_commit_both(empty_bar(stage), both);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_both(acc_full(acc), both);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            if (!ok || *abort_flag) {
                mma_commit_pair_local(drain_bar);
                drain_wait(drain_bar, 0);
            }
        }
        __syncwarp();
        if (SPLIT) cluster_sync();
    } else {
        // ---------------- epilogue (both CTAs) ----------------
        const uint32_t stage_epi = smem_u32(smem) + STAGES * STAGE_BYTES + 1024u + (uint32_t)(warp - 2) * L::warp_bytes;
        const int quarter = warp & 3, half = (warp - 2) >> 2;  // TMEM lanes; columns of the tile
        int acc = 0;
        uint32_t acc_phase = 0;
        uint32_t slot = 0;                     // first staging slot of the next chunk (warp-uniform)
        uint32_t in_phase = 0;                 // bit s: parity of the next TMA load into slot s
        uint32_t in_flight = 0;                // bit s: a load into slot s is not yet waited for (lane 0)
        const bool has_in = EPI == LIN_DGLU || (EPI == LIN_OUT && !PLAIN && !F32 && a.has_residual);
        const bool has_bias = EPI == LIN_OUT && !PLAIN && a.has_bias;
        const bool keep = !PLAIN && EPI != LIN_DGLU && a.keep;
        // Slots a chunk takes: 1, with a second operand or output, or in float32, 2
        // (LIN_GLU with kept pre-activations 3).
        const uint32_t per_chunk = EPI == LIN_DGLU || F32 || (EPI == LIN_OUT && keep) ? 2u : EPI == LIN_GLU && keep ? 3u : 1u;
        for (int tile = first; tile < a.total_tiles; tile += stride) {
            int g, mt, nt;
            tile_coords(a, tile, g, mt, nt);
            // this warp's 32 rows: lane l holds row row0 + l of the accumulator
            const int row0 = mt * BM + (int)cta * 128 + quarter * 32;
            const int64_t row = row0 + lane;
            // The warp's chunks of 32 columns: its half of the tile, or, SPLIT, its share of
            // this part's: every `parts`-th chunk of the tile belongs to one part.
            const int tile_col = nt * TILE_COLS;
            auto chunk_at = [&](int k) { return SPLIT ? 32 * ((HALVES * k + half) * parts + part) : half * WARP_COLS + 32 * k; };
            int chunks = 0;  // warp-uniform
            if (row0 < a.rows)
                while (chunks < CHUNKS && chunk_at(chunks) < min(TILE_COLS, a.cols - tile_col)) ++chunks;
            auto slot_addr = [&](uint32_t s) { return stage_epi + (s & (SLOTS - 1)) * SLOT_BYTES; };
            // Operands of chunk c into its slots, by TMA: they cross the memory while
            // the tile is still being multiplied. One lane.
            auto fetch = [&](int c) {
                const uint32_t s = (slot + (uint32_t)c * per_chunk) & (SLOTS - 1);
                in_flight |= 1u << s;
                mbar_expect_tx(slot_bar(warp - 2, (int)s), EPI == LIN_DGLU ? 2 * SLOT_BYTES : SLOT_BYTES);
                tma_load_2d(slot_addr(s), &a.ti[g], slot_bar(warp - 2, (int)s), tile_col + chunk_at(c), row0);
                if (EPI == LIN_DGLU) tma_load_2d(slot_addr(s + 1), &a.ti2[g], slot_bar(warp - 2, (int)s), tile_col + chunk_at(c), row0);
            };
            const int depth = (int)(SLOTS / per_chunk);  // chunks whose slots exist at once
            if (has_in && lane == 0 && chunks > 0) {
                bulk_wait_read<0>();  // the last tile's stores have read the slots
                for (int c = 0; c < min(chunks, depth); ++c) fetch(c);
            }
            // bias of the warp's columns: lane l holds 8 columns from 8 (l % 4) of chunk l / 4
            uint4 bias = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (EPI == LIN_OUT && !PLAIN) {
                const int at = chunk_at(lane >> 2) + 8 * (lane & 3);
                if (has_bias && (lane >> 2) < CHUNKS && at < TILE_COLS && tile_col + at < a.cols)
                    bias = __ldg(reinterpret_cast<const uint4*>(a.bias[g] + tile_col + at));
            }
            int ok = 1;
            if (lane == 0) ok = wait_bar(acc_full(acc), acc_phase, abort_flag, ERR_EPILOGUE) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) {
                if (SPLIT) cluster_sync();
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * BN);

            // 16-byte unit u of this lane's row, as the TMA swizzles it: u ^ (r / 2 % 4)
            // of a 64-byte row, u ^ (r % 8) of a float32 chunk's 128-byte row
            auto unit = [&](uint32_t s, int u) {
                return slot_addr(s) + (uint32_t)lane * 64u + 16u * (uint32_t)(u ^ ((lane >> 1) & 3));
            };
            auto unit_f32 = [&](uint32_t s, int u) {
                return slot_addr(s) + (uint32_t)lane * 128u + 16u * (uint32_t)(u ^ (lane & 7));
            };
            // columns of step c (its first one is c % PER steps into the chunk)
            auto put_bf16 = [&](uint32_t s, int c, const float (&v)[STEP]) {
#pragma unroll
                for (int q = 0; q < STEP / 8; ++q)
                    st_shared_v4(unit(s, STEP / 8 * (c & (PER - 1)) + q), bf16x2(v[8 * q], v[8 * q + 1]),
                                 bf16x2(v[8 * q + 2], v[8 * q + 3]), bf16x2(v[8 * q + 4], v[8 * q + 5]),
                                 bf16x2(v[8 * q + 6], v[8 * q + 7]));
            };
            auto put_f32 = [&](uint32_t s, int c, const float (&v)[STEP]) {
#pragma unroll
                for (int q = 0; q < STEP / 4; ++q)
                    st_shared_v4(unit_f32(s, STEP / 4 * (c & (PER - 1)) + q), __float_as_uint(v[4 * q]),
                                 __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
            };
            auto unpack8 = [](const uint4& w, float* x) {
                x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
                x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
            };
            auto get_bf16 = [&](uint32_t s, int c, float (&x)[STEP]) {
#pragma unroll
                for (int q = 0; q < STEP / 8; ++q) unpack8(ld_shared_v4(unit(s, STEP / 8 * (c & (PER - 1)) + q)), x + 8 * q);
            };
            // Until the stores that used this chunk's slots have read them. The slots go
            // round, so only the newest stores may be pending, as many as fit beside this
            // chunk (a store is one group of this lane, a float32 one reads two slots).
            auto acquire = [&]() {
                if (lane == 0) {
                    if constexpr (SLOTS == 2) {
                        if (per_chunk == 1) bulk_wait_read<1>();
                        else bulk_wait_read<0>();
                    } else {
                        if (per_chunk == 1) bulk_wait_read<3>();
                        else if (!F32 && per_chunk == 2) bulk_wait_read<2>();
                        else bulk_wait_read<1>();
                    }
                }
                __syncwarp();
            };
            auto flush = [&]() {
                fence_async_shared();
                __syncwarp();
            };
            auto store = [&](const CUtensorMap* map, uint32_t s, int c0) {
                if (lane == 0) {
                    tma_store_2d(map, slot_addr(s), c0, row0);
                    bulk_commit();
                }
            };
            auto wait_in = [&](uint32_t s) {  // the chunk's operands have landed in slot s (and s + 1)
                s &= SLOTS - 1;
                int got = 1;
                if (lane == 0) got = wait_bar(slot_bar(warp - 2, (int)s), (in_phase >> s) & 1u, abort_flag, ERR_EPILOGUE) ? 1 : 0;
                if (got) {
                    in_phase ^= 1u << s;
                    in_flight &= ~(1u << s);
                }
                return __shfl_sync(0xffffffffu, got, 0) != 0;
            };
            // The operands of a later chunk, once the chunk before this one has left its
            // slots (where the slots do not hold the warp's whole part of the tile).
            auto refill = [&](int c) {
                if (!has_in || c < 1 || c - 1 + depth >= chunks || depth < 2) return;
                if (lane == 0) {
                    bulk_wait_read<0>();
                    fetch(c - 1 + depth);
                }
                __syncwarp();
            };

            // Loops that are not unrolled: the straight-line form fetched its code anew
            // for every tile. The accumulator columns of the next step are on their way
            // while a step is computed.
            const int steps = PER * chunks;
            bool good = true;
            // Accumulator columns of step c: from tensor memory (columns + `up` for the up
            // projection), in flight until take(), or, SPLIT, from every part's shared
            // memory, added in the order of the parts.
            uint32_t ra[STEP], rb[STEP];
            const uint32_t smem0 = smem_u32(smem);
            auto column = [&](int c) { return chunk_at(c / PER) + STEP * (c % PER); };
            auto start = [&](int c, int up, uint32_t (&r)[STEP]) {
                if constexpr (!SPLIT) tmem_load(taddr + (uint32_t)(column(c) + up), r);
            };
            auto take = [&](int c, int up, uint32_t (&r)[STEP], float (&v)[STEP]) {
                if constexpr (SPLIT) {
                    // Summed in 128-byte pieces of a column (a request of 32 scattered 16-byte
                    // pieces takes the cluster's network many times as long), and turned to
                    // one row a lane in the warp's own 4 KB behind the accumulator.
                    const uint32_t in_col = 16u * (uint32_t)(lane & 7), own = smem0 + PART_BYTES + (uint32_t)(warp - 2) * 4096u +
                                                                              (up ? 128u * STEP : 0u);
                    const uint32_t at = smem0 + 512u * (uint32_t)(column(c) + up + (lane >> 3)) + 128u * (uint32_t)quarter + in_col;
                    float4 sum[STEP / 4];
                    for (int p = 0; p < parts; ++p) {
                        const uint32_t from = map_to_rank(at, (uint32_t)(2 * p) + cta);
                        float4 w[STEP / 4];
#pragma unroll
                        for (int q = 0; q < STEP / 4; ++q) w[q] = ld_cluster_f4(from + 2048u * q);
#pragma unroll
                        for (int q = 0; q < STEP / 4; ++q)
                            sum[q] = p ? make_float4(sum[q].x + w[q].x, sum[q].y + w[q].y, sum[q].z + w[q].z, sum[q].w + w[q].w) : w[q];
                    }
                    __syncwarp();  // the last step's columns have been read
#pragma unroll
                    for (int q = 0; q < STEP / 4; ++q)
                        st_shared_v4(own + 128u * (uint32_t)(4 * q + (lane >> 3)) + in_col, __float_as_uint(sum[q].x),
                                     __float_as_uint(sum[q].y), __float_as_uint(sum[q].z), __float_as_uint(sum[q].w));
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < STEP; ++j)
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[j]) : "r"(own + 128u * (uint32_t)j + 4u * (uint32_t)lane) : "memory");
                } else {
                    tmem_wait(r);
#pragma unroll
                    for (int j = 0; j < STEP; ++j) v[j] = __uint_as_float(r[j]);
                }
            };
            if constexpr (SPLIT) {
                // this part's accumulator to the operand ring's memory (every load has landed
                // and every MMA is done): column c, row r at float 128 c + r
                const uint32_t dst = smem0 + 4u * (uint32_t)(quarter * 32 + lane);
#pragma unroll 1
                for (int c = half * (BN / HALVES); c < (half + 1) * (BN / HALVES); c += STEP) {
                    tmem_load(taddr + (uint32_t)c, ra);
                    tmem_wait(ra);
#pragma unroll
                    for (int j = 0; j < STEP; ++j)
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 512u * (uint32_t)(c + j)), "r"(ra[j]) : "memory");
                }
                cluster_sync();
            }
            if constexpr (EPI == LIN_OUT) {
                if (steps > 0) start(0, 0, ra);
#pragma unroll 1
                for (int c = 0; c < steps; ++c) {
                    const uint32_t s = slot + (uint32_t)(c / PER) * per_chunk;
                    float v[STEP];
                    take(c, 0, ra, v);
                    if (c + 1 < steps) start(c + 1, 0, ra);
                    if (c % PER == 0) {
                        if (!has_in) acquire();  // else the slots were free when the operands were fetched
                        else if (!(good = wait_in(s))) break;
                    }
                    if constexpr (!PLAIN) {
                        if (has_bias) {
#pragma unroll
                            for (int q = 0; q < STEP / 8; ++q) {
                                const uint32_t w[4] = {bias.x, bias.y, bias.z, bias.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t b = __shfl_sync(0xffffffffu, w[e], STEP / 8 * c + q);
                                    v[8 * q + 2 * e] += bf16_lo(b);
                                    v[8 * q + 2 * e + 1] += bf16_hi(b);
                                }
                            }
                        }
                        if constexpr (F32) {  // the output takes both slots: h goes straight to memory
                            if (keep && row < a.rows) {
#pragma unroll
                                for (int q = 0; q < STEP / 8; ++q) {
                                    const int cq = tile_col + column(c) + 8 * q;
                                    if (cq < a.cols)
                                        *reinterpret_cast<uint4*>(a.h[g] + row * a.ld + cq) =
                                            make_uint4(bf16x2(v[8 * q], v[8 * q + 1]), bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                                       bf16x2(v[8 * q + 4], v[8 * q + 5]), bf16x2(v[8 * q + 6], v[8 * q + 7]));
                                }
                            }
                        } else if (keep) {
                            put_bf16(s + 1, c, v);
                        }
                        if constexpr (ACT)
                            with_act(a.act, [&](auto tag) {
#pragma unroll
                                for (int j = 0; j < STEP; ++j) v[j] = act_value<decltype(tag)::value, F32>(v[j]);
                            });
                        if (F32 ? a.has_residual != 0 : has_in) {
                            float x[STEP] = {};
                            if constexpr (F32) {
#pragma unroll
                                for (int q = 0; q < STEP / 8; ++q) {
                                    const int cq = tile_col + column(c) + 8 * q;
                                    if (row < a.rows && cq < a.cols)
                                        unpack8(__ldg(reinterpret_cast<const uint4*>(a.residual[g] + row * a.ld + cq)), x + 8 * q);
                                }
                            } else {
                                get_bf16(s, c, x);
                            }
#pragma unroll
                            for (int j = 0; j < STEP; ++j) v[j] += x[j];
                        }
                    }
                    const int c0 = tile_col + chunk_at(c / PER);
                    if constexpr (F32) put_f32(s, c, v);
                    else put_bf16(s, c, v);
                    if (c % PER == PER - 1) {
                        refill(c / PER);
                        flush();
                        store(&a.to[g], s, c0);
                        if (!F32 && keep) store(&a.to2[g], s + 1, c0);
                        if (has_in && depth < 2 && c + 1 < steps) {  // one chunk at a time (a kept h beside it)
                            if (lane == 0) {
                                bulk_wait_read<0>();
                                fetch(c / PER + 1);
                            }
                            __syncwarp();
                        }
                    }
                }
            } else if constexpr (EPI == LIN_GLU) {
                // accumulator columns 0-127 hold the gate, 128-255 the up projection
                if (steps > 0) {
                    start(0, 0, ra);
                    start(0, TILE_COLS, rb);
                }
#pragma unroll 1
                for (int c = 0; c < steps; ++c) {
                    const uint32_t s = slot + (uint32_t)(c / PER) * per_chunk;
                    float v[STEP], u[STEP];
                    take(c, 0, ra, v);
                    take(c, TILE_COLS, rb, u);
                    if (c + 1 < steps) {
                        start(c + 1, 0, ra);
                        start(c + 1, TILE_COLS, rb);
                    }
                    if (c % PER == 0) acquire();
                    if (keep) {
                        put_bf16(s + 1, c, v);
                        put_bf16(s + 2, c, u);
                    }
                    with_act(a.act, [&](auto tag) {
#pragma unroll
                        for (int j = 0; j < STEP; ++j) v[j] = act_value<decltype(tag)::value>(v[j]);
                    });
#pragma unroll
                    for (int j = 0; j < STEP; ++j) v[j] *= u[j];
                    put_bf16(s, c, v);
                    if (c % PER == PER - 1) {
                        const int c0 = tile_col + chunk_at(c / PER);
                        flush();
                        store(&a.to[g], s, c0);
                        if (keep) {
                            store(&a.to2[g], s + 1, c0);
                            store(&a.to3[g], s + 2, c0);
                        }
                    }
                }
            } else {  // LIN_DGLU: slots s, s + 1 hold gate and up, and take the two gradients in their place
                if (steps > 0) start(0, 0, ra);
#pragma unroll 1
                for (int c = 0; c < steps; ++c) {
                    const uint32_t s = slot + (uint32_t)(c / PER) * per_chunk;
                    float dy[STEP], hg[STEP], hu[STEP];
                    take(c, 0, ra, dy);
                    if (c + 1 < steps) start(c + 1, 0, ra);
                    if (c % PER == 0 && !(good = wait_in(s))) break;
                    get_bf16(s, c, hg);
                    get_bf16(s + 1, c, hu);
                    with_act(a.act, [&](auto tag) {
#pragma unroll
                        for (int j = 0; j < STEP; ++j) {
                            float av, dv;
                            act_both<decltype(tag)::value>(hg[j], av, dv);
                            hg[j] = dy[j] * hu[j] * dv;
                            hu[j] = dy[j] * av;
                        }
                    });
                    put_bf16(s, c, hg);
                    put_bf16(s + 1, c, hu);
                    if (c % PER == PER - 1) {
                        const int c0 = tile_col + chunk_at(c / PER);
                        refill(c / PER);
                        flush();
                        store(&a.to[g], s, c0);
                        store(&a.to2[g], s + 1, c0);
                    }
                }
            }
            if (!good) {
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");  // the next step's columns
                break;
            }
            slot = (slot + (uint32_t)chunks * per_chunk) & (SLOTS - 1);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(acc_empty(acc), leader));
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (lane == 0)  // after an abort: the loads still in flight land before the CTA leaves
            for (int s = 0; s < SLOTS; ++s)
                if ((in_flight >> s) & 1u) drain_wait(slot_bar(warp - 2, s), (in_phase >> s) & 1u);
        if (lane == 0) bulk_wait_all();  // every output tile written before the CTA leaves
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still signal or read it
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
}

// ---- launch -----------------------------------------------------------------------

inline cudaLaunchAttribute cluster_of(int ctas)
{
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = (unsigned)ctas;
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
    return a;
}

// Resident clusters of `ctas` CTAs on the current device, 0 where none fits (a device
// or partition may have no such group of SMs), asked once per device and size (racing
// first calls compute the same value); sets the kernel's shared-memory limit on the way.
template <int CFG, bool SPLIT>
int resident_clusters(const char* fn, int ctas, int* n)
{
    static std::atomic<int> known[64][5];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fail(RTP_ECUDA, "%s: no CUDA device", fn);
    std::atomic<int>& slot = known[dev][ctas / 2];
    *n = slot.load(std::memory_order_acquire) - 1;  // 0: not asked yet
    if (*n >= 0) return RTP_OK;
    cudaError_t e = cudaFuncSetAttribute(linear_gemm_kernel<CFG, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<CFG, SPLIT>::bytes);
    if (e != cudaSuccess) return fail(RTP_ECUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = cluster_of(ctas);
    cfg.gridDim = dim3((unsigned)(ctas * 64));
    cfg.blockDim = dim3(Layout<CFG, SPLIT>::threads);
    cfg.dynamicSmemBytes = Layout<CFG, SPLIT>::bytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(n, linear_gemm_kernel<CFG, SPLIT>, &cfg);
    if (e != cudaSuccess || *n < 0) {
        cudaGetLastError();
        *n = 0;
    }
    slot.store(*n + 1, std::memory_order_release);
    return RTP_OK;
}

template <int CFG, bool SPLIT>
int launch_t(const char* fn, LinArgs& args, cudaStream_t stream)
{
    int ctas = 2, clusters = 0;
    if constexpr (SPLIT) {
        // As many parts as leave every cluster resident at once, while a part saves
        // more K blocks than adding it up costs.
        args.split = 1;
        double best = args.kbs;
        int64_t none_from = INT64_MAX;  // CTAs of the clusters that are taken not to fit
        take_hook(RTP_HOOK_NO_CLUSTERS, &none_from);
        for (int s = 2; s <= 4; ++s) {
            const double cost = (double)args.kbs / s + SPLIT_COST + s;
            if (args.kbs < 4 * s || cost >= best || 2 * s >= none_from) continue;
            int n = 0, st = resident_clusters<CFG, SPLIT>(fn, 2 * s, &n);
            if (st) return st;
            if (args.total_tiles > n) continue;
            best = cost;
            args.split = s;
        }
        if (args.split == 1) return LIN_NOT_SPLIT;
        ctas = 2 * args.split;
        clusters = args.total_tiles;
    } else {
        int st = resident_clusters<CFG, SPLIT>(fn, 2, &clusters);
        if (st) return st;
        if (clusters <= 0) return fail(RTP_ECUDA, "%s: no pair of SMs fits a product's cluster", fn);
        if (args.total_tiles < clusters) clusters = args.total_tiles;
    }
    if (clusters <= 0) return RTP_OK;
    cudaLaunchAttribute attr[2] = {cluster_of(ctas), {}};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas * clusters));
    cfg.blockDim = dim3(Layout<CFG, SPLIT>::threads);
    cfg.dynamicSmemBytes = Layout<CFG, SPLIT>::bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, linear_gemm_kernel<CFG, SPLIT>, args);
    if (e != cudaSuccess) return fail(RTP_ECUDA, "%s: product launch failed: %s", fn, cudaGetErrorString(e));
    ++product_launches[SPLIT ? args.split : RTP_PRODUCT_WHOLE];
    return RTP_OK;
}

template <bool SPLIT>
int launch_cfg(const char* fn, int cfg, LinArgs& a, cudaStream_t stream)
{
    switch (cfg) {
    case LIN_GLU << CFG_EPI_SHIFT: return launch_t<LIN_GLU << CFG_EPI_SHIFT, SPLIT>(fn, a, stream);
    case (LIN_DGLU << CFG_EPI_SHIFT) | CFG_B_T: return launch_t<(LIN_DGLU << CFG_EPI_SHIFT) | CFG_B_T, SPLIT>(fn, a, stream);
    case 0: return launch_t<0, SPLIT>(fn, a, stream);
    case CFG_ACT: return launch_t<CFG_ACT, SPLIT>(fn, a, stream);
    case CFG_F32: return launch_t<CFG_F32, SPLIT>(fn, a, stream);
    case CFG_F32 | CFG_ACT: return launch_t<CFG_F32 | CFG_ACT, SPLIT>(fn, a, stream);
    case CFG_A_T: return launch_t<CFG_A_T, SPLIT>(fn, a, stream);
    case CFG_A_T | CFG_F32: return launch_t<CFG_A_T | CFG_F32, SPLIT>(fn, a, stream);
    case CFG_B_T: return launch_t<CFG_B_T, SPLIT>(fn, a, stream);
    case CFG_B_T | CFG_F32: return launch_t<CFG_B_T | CFG_F32, SPLIT>(fn, a, stream);
    default: return fail(RTP_EUNSUPPORTED, "%s: no product for transposed operands of this kind", fn);
    }
}

}  // namespace

// linear_gemm_split.cu: launches the product with its tiles' K ranges split, or
// returns LIN_NOT_SPLIT when that does not pay.
int launch_linear_split(const char* fn, int cfg, LinArgs& a, cudaStream_t stream);

}  // namespace rtp
