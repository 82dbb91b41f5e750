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
// tcgen05.mma.cta_group::2 (256 x 256 x 16), and warps 2-5 turn one of two TMEM
// accumulators into outputs while the next tile is multiplied. For LIN_GLU the
// leader's CTA loads 128 gate columns and its peer the same 128 up columns, so
// the accumulator's two halves hold gate and up of one output column in the same
// TMEM lane: the epilogue thread of a row has both without any exchange, and X
// is read once for the two projections. A fused sum over ranks (and, for the
// input gradient, over gate and up) walks all operand pairs in one K loop.
//
// Outputs leave in bf16 chunks of 32 x 32 (2 KB) by TMA tensor stores from a ring
// of 4 staging slots per epilogue warp. A kept pre-activation is rounded to bf16
// once; Y is computed from the float32 accumulators, not from the rounded ones.
#include <atomic>
#include <cstring>

#include "activation.cuh"
#include "linear.h"
#include "tcgen05.cuh"

namespace rtp {

namespace {

constexpr int BM = 256, BN = 256;
constexpr uint32_t SUB = 64 * BK * 2;  // one 64 x 64 box, 8 KB
constexpr int EPI_WARPS = 4;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr int STAGES = 6;
constexpr uint32_t A_BYTES = 128 * BK * 2, B_BYTES = 128 * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr uint32_t SLOT_BYTES = 2048;                 // one 32 x 32 bf16 chunk
constexpr uint32_t EPI_WARP_BYTES = 4 * SLOT_BYTES;   // or two 32 x 32 float32 chunks
constexpr size_t SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + EPI_WARPS * EPI_WARP_BYTES + 1024;
static_assert(SMEM_BYTES <= 232448, "at most 227 KB of shared memory per CTA");

enum : int { CFG_A_T = 1, CFG_B_T = 2, CFG_F32 = 4, CFG_EPI_SHIFT = 3 };

struct Args {
    CUtensorMap ta[LIN_MAX_GROUPS], tb[LIN_MAX_GROUPS];  // LIN_GLU: tb[g] gate, tb[LIN_MAX_RANKS + g] up
    CUtensorMap to[LIN_MAX_GROUPS], to2[LIN_MAX_RANKS], to3[LIN_MAX_RANKS];
    const __nv_bfloat16* bias[LIN_MAX_RANKS];
    const __nv_bfloat16* residual[LIN_MAX_RANKS];
    const __nv_bfloat16* aux[LIN_MAX_RANKS];
    const __nv_bfloat16* aux2[LIN_MAX_RANKS];
    int64_t ld;  // output row stride, elements
    int32_t groups, fused, kb_per_group, m_tiles, n_tiles, rows, cols;
    int32_t total_tiles, group_m, groups_in_n;
    int32_t act, has_bias, has_residual, keep;
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
__device__ __forceinline__ void tile_coords(const Args& a, int tile, int& g, int& mt, int& nt)
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
template <int CFG>
__global__ void __launch_bounds__(THREADS, 1) linear_gemm_kernel(const __grid_constant__ Args a)
{
    constexpr bool A_T = (CFG & CFG_A_T) != 0, B_T = (CFG & CFG_B_T) != 0, F32 = (CFG & CFG_F32) != 0;
    constexpr int EPI = CFG >> CFG_EPI_SHIFT;
    constexpr bool PLAIN = EPI == LIN_OUT && (A_T || B_T);  // gradients: the accumulator alone
    constexpr int TILE_COLS = EPI == LIN_GLU ? BN / 2 : BN;
    constexpr int CHUNKS = TILE_COLS / 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(STAGES + s); };
    auto acc_full = [&](int x) { return bar0 + 8u * (uint32_t)(2 * STAGES + x); };
    auto acc_empty = [&](int x) { return bar0 + 8u * (uint32_t)(2 * STAGES + 2 + x); };
    const uint32_t drain_bar = bar0 + 8u * (uint32_t)(2 * STAGES + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t cta = cluster_rank();
    const int pair = (int)cluster_id(), npairs = (int)num_clusters();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(acc_full(x), 1);
            mbar_init(acc_empty(x), 2 * EPI_WARPS);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
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
    const int kbs = a.fused ? a.groups * a.kb_per_group : a.kb_per_group;

    if (warp == 0) {
        // ---------------- TMA producer (one lane per CTA) ----------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_parity = 0;
            bool ok = true;
            const uint32_t smem0 = smem_u32(smem);
            const uint32_t leader_full0 = map_to_rank(full_bar(0), 0);
            for (int tile = pair; ok && tile < a.total_tiles; tile += npairs) {
                int g, mt, nt;
                tile_coords(a, tile, g, mt, nt);
                const int row = mt * BM + (int)cta * 128;
                const int col = EPI == LIN_GLU ? nt * TILE_COLS : nt * BN + (int)cta * 128;
                int gg = a.fused ? 0 : g, kk = 0;
                for (int kb = 0; kb < kbs; ++kb) {
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
            for (int tile = pair; ok && tile < a.total_tiles; tile += npairs) {
                if (!wait_bar(acc_empty(acc), acc_phase ^ 1u, abort_flag, ERR_MMA_ACC)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
                for (int kb = 0; kb < kbs; ++kb) {
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
                                      (kb > 0 || k > 0) ? 1u : 0u);
                    mma_commit_pair(empty_bar(stage));
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_pair(acc_full(acc));
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
    } else {
        // ---------------- epilogue (both CTAs) ----------------
        const uint32_t stage_epi = smem_u32(smem) + STAGES * STAGE_BYTES + 1024u + (uint32_t)(warp - 2) * EPI_WARP_BYTES;
        const int quarter = warp & 3;
        int acc = 0;
        uint32_t acc_phase = 0;
        uint32_t slot = 0;  // next staging slot (warp-uniform): the stores take the 4 slots in turn
        for (int tile = pair; tile < a.total_tiles; tile += npairs) {
            int g, mt, nt;
            tile_coords(a, tile, g, mt, nt);
            int ok = 1;
            if (lane == 0) ok = wait_bar(acc_full(acc), acc_phase, abort_flag, ERR_EPILOGUE) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            tc_fence_after();
            // this warp's 32 rows: lane l holds row row0 + l of the accumulator
            const int row0 = mt * BM + (int)cta * 128 + quarter * 32;
            const int64_t row = row0 + lane;
            const int col = nt * TILE_COLS;
            const bool row_ok = row < a.rows;
            const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * BN);

            // 32 bf16 of this lane's row of a [rows, cols] operand at column c0 (zeros outside)
            auto load_row = [&](const __nv_bfloat16* base, int c0, uint4 (&v)[4]) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = row_ok && c0 + 8 * q < a.cols
                               ? __ldg(reinterpret_cast<const uint4*>(base + row * a.ld + c0 + 8 * q))
                               : make_uint4(0u, 0u, 0u, 0u);
            };
            auto row_at = [](const uint4 (&v)[4], int j) {
                const uint4& u = v[j >> 3];
                const uint32_t w = (j & 6) == 0 ? u.x : (j & 6) == 2 ? u.y : (j & 6) == 4 ? u.z : u.w;
                return (j & 1) ? bf16_hi(w) : bf16_lo(w);
            };
            // Staging: the lane's row of a chunk goes to a slot in the TMA's swizzled
            // layout (16-byte unit u of row r at u ^ (r / 2 % 4) of a 64-byte row, or
            // u ^ (r % 8) of a 128-byte float32 row), and one lane stores it.
            auto put_bf16 = [&](uint32_t s, const float (&v)[32]) {
                const uint32_t rb = stage_epi + s * SLOT_BYTES + (uint32_t)lane * 64u;
                const int sw = (lane >> 1) & 3;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    st_shared_v4(rb + 16u * (uint32_t)(q ^ sw), pack_bf16(v[8 * q], v[8 * q + 1]),
                                 pack_bf16(v[8 * q + 2], v[8 * q + 3]), pack_bf16(v[8 * q + 4], v[8 * q + 5]),
                                 pack_bf16(v[8 * q + 6], v[8 * q + 7]));
            };
            auto put_f32 = [&](uint32_t s, const float (&v)[32]) {
                const uint32_t rb = stage_epi + s * SLOT_BYTES + (uint32_t)lane * 128u;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    st_shared_v4(rb + 16u * (uint32_t)(q ^ (lane & 7)), __float_as_uint(v[4 * q]),
                                 __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                                 __float_as_uint(v[4 * q + 3]));
            };
            // before N slots are written: the stores that used them have read them
            // (the wait counts this lane's store groups, one per slot or float32 pair)
            auto flush = [&]() {
                fence_async_shared();
                __syncwarp();
            };
            auto store = [&](const CUtensorMap* map, uint32_t s, int c0) {
                if (lane == 0) {
                    tma_store_2d(map, stage_epi + s * SLOT_BYTES, c0, row0);
                    bulk_commit();
                }
            };

            if constexpr (EPI == LIN_OUT) {
                auto emit = [&](int c, const uint32_t (&r)[32], const uint4 (&res)[4]) {
                    const int c0 = col + 32 * c;
                    if (c0 >= a.cols || row0 >= a.rows) return;  // warp-uniform
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                    bool keep = false;
                    if constexpr (!PLAIN) {
                        keep = a.keep != 0;
                        if (a.has_bias) {
                            uint4 b[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                b[q] = c0 + 8 * q < a.cols ? __ldg(reinterpret_cast<const uint4*>(a.bias[g] + c0 + 8 * q))
                                                           : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] += row_at(b, j);
                        }
                    }
                    uint32_t s = slot;
                    if (keep) {
                        if (lane == 0) {
                            if constexpr (F32) bulk_wait_read<0>();
                            else bulk_wait_read<2>();
                        }
                        __syncwarp();
                        put_bf16(s, v);
                        s = F32 ? 2u : (s + 1) & 3u;
                    } else {
                        if (lane == 0) {
                            if constexpr (F32) bulk_wait_read<1>();
                            else bulk_wait_read<3>();
                        }
                        __syncwarp();
                    }
                    if constexpr (!PLAIN) {
                        if (a.act != RTP_ACT_NONE)
                            with_act(a.act, [&](auto tag) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) v[j] = act_value<decltype(tag)::value>(v[j]);
                            });
                        if (a.has_residual) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] += row_at(res, j);
                        }
                    }
                    if constexpr (F32) put_f32(s, v);
                    else put_bf16(s, v);
                    flush();
                    if (keep) store(&a.to2[g], slot, c0);
                    store(&a.to[g], s, c0);
                    // float32 chunks alternate between slots 0-1 and 2-3 (with h kept: h
                    // in slot 0, the output in 2-3)
                    if constexpr (F32) slot = keep ? 0u : slot ^ 2u;
                    else slot = (s + 1) & 3u;
                };
                auto load_res = [&](int c, uint4 (&v)[4]) {
                    if constexpr (!PLAIN) {
                        if (a.has_residual) load_row(a.residual[g], col + 32 * c, v);
                    }
                };
                uint32_t ra[32], rb[32];
                uint4 ha[4], hb[4];
                load_res(0, ha);
                tmem_ld_32cols(taddr, ra);
                tmem_ld_wait(ra);
                for (int c = 0; c < CHUNKS; c += 2) {
                    tmem_ld_32cols(taddr + 32u * (c + 1), rb);
                    load_res(c + 1, hb);
                    emit(c, ra, ha);
                    tmem_ld_wait(rb);
                    if (c + 2 < CHUNKS) {
                        tmem_ld_32cols(taddr + 32u * (c + 2), ra);
                        load_res(c + 2, ha);
                    }
                    emit(c + 1, rb, hb);
                    if (c + 2 < CHUNKS) tmem_ld_wait(ra);
                }
            } else if constexpr (EPI == LIN_GLU) {
                // accumulator columns 0-127 hold the gate, 128-255 the up projection
                for (int c = 0; c < CHUNKS; ++c) {
                    const int c0 = col + 32 * c;
                    if (c0 >= a.cols || row0 >= a.rows) break;  // warp-uniform
                    uint32_t rg[32], ru[32];
                    tmem_ld_32cols(taddr + 32u * c, rg);
                    tmem_ld_32cols(taddr + (uint32_t)TILE_COLS + 32u * c, ru);
                    tmem_ld_wait(rg);
                    tmem_ld_wait(ru);
                    float v[32], u[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        v[j] = __uint_as_float(rg[j]);
                        u[j] = __uint_as_float(ru[j]);
                    }
                    const bool keep = a.keep != 0;
                    if (lane == 0) {
                        if (keep) bulk_wait_read<1>();
                        else bulk_wait_read<3>();
                    }
                    __syncwarp();
                    const uint32_t s0 = slot, s1 = (slot + 1) & 3u, s2 = (slot + 2) & 3u;
                    if (keep) {
                        put_bf16(s1, v);
                        put_bf16(s2, u);
                    }
                    with_act(a.act, [&](auto tag) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = act_value<decltype(tag)::value>(v[j]) * u[j];
                    });
                    put_bf16(s0, v);
                    flush();
                    store(&a.to[g], s0, c0);
                    if (keep) {
                        store(&a.to2[g], s1, c0);
                        store(&a.to3[g], s2, c0);
                    }
                    slot = (slot + (keep ? 3u : 1u)) & 3u;
                }
            } else {  // LIN_DGLU
                for (int c = 0; c < CHUNKS; ++c) {
                    const int c0 = col + 32 * c;
                    if (c0 >= a.cols || row0 >= a.rows) break;  // warp-uniform
                    uint4 hg[4], hu[4];
                    load_row(a.aux[g], c0, hg);
                    load_row(a.aux2[g], c0, hu);
                    uint32_t r[32];
                    tmem_ld_32cols(taddr + 32u * c, r);
                    tmem_ld_wait(r);
                    float dg[32], du[32];
                    with_act(a.act, [&](auto tag) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float dy = __uint_as_float(r[j]);
                            float av, dv;
                            act_both<decltype(tag)::value>(row_at(hg, j), av, dv);
                            dg[j] = dy * row_at(hu, j) * dv;
                            du[j] = dy * av;
                        }
                    });
                    if (lane == 0) bulk_wait_read<2>();
                    __syncwarp();
                    const uint32_t s0 = slot, s1 = (slot + 1) & 3u;
                    put_bf16(s0, dg);
                    put_bf16(s1, du);
                    flush();
                    store(&a.to[g], s0, c0);
                    store(&a.to2[g], s1, c0);
                    slot = (slot + 2) & 3u;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(acc_empty(acc), 0));
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (lane == 0) bulk_wait_all();  // every output tile written before the CTA leaves
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cluster_sync();  // no CTA leaves while its peer may still signal or read it
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
}

// ---- host side --------------------------------------------------------------------

template <int CFG>
int launch_t(const char* fn, Args& args, cudaStream_t stream)
{
    // per device: resident 2-SM clusters (0 = not yet queried); racing first
    // calls compute the same value
    static std::atomic<int> max_clusters[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fail(RTP_ECUDA, "%s: no CUDA device", fn);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int nclusters = max_clusters[dev].load(std::memory_order_acquire);
    if (!nclusters) {
        cudaError_t e = cudaFuncSetAttribute(linear_gemm_kernel<CFG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
        if (e != cudaSuccess) return fail(RTP_ECUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
        cfg.gridDim = dim3(2 * 64);
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, linear_gemm_kernel<CFG>, &cfg);
        if (e != cudaSuccess || n <= 0) return fail(RTP_ECUDA, "%s: cudaOccupancyMaxActiveClusters: %s", fn, cudaGetErrorString(e));
        max_clusters[dev].store(n, std::memory_order_release);
        nclusters = n;
    }
    const int clusters = args.total_tiles < nclusters ? args.total_tiles : nclusters;
    if (clusters <= 0) return RTP_OK;
    cfg.gridDim = dim3(2 * clusters);
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, linear_gemm_kernel<CFG>, args);
    if (e != cudaSuccess) return fail(RTP_ECUDA, "%s: product launch failed: %s", fn, cudaGetErrorString(e));
    return RTP_OK;
}

// Encodes a map, or copies the previous group's when it is of the same buffer
// (a shared operand is encoded once).
int operand_map(CUtensorMap* maps, const void* const* ptrs, int i, int64_t rows, int64_t cols, int box_rows)
{
    if (i > 0 && ptrs[i] == ptrs[i - 1]) {
        maps[i] = maps[i - 1];
        return RTP_OK;
    }
    return make_map(&maps[i], ptrs[i], rows, cols, box_rows);
}

}  // namespace

int launch_linear_gemm(const char* fn, const LinGemm& p, cudaStream_t stream)
{
    static thread_local Args a;
    std::memset(&a, 0, sizeof a);
    const int tile_cols = p.epi == LIN_GLU ? BN / 2 : BN;
    int st;
    for (int g = 0; g < p.groups; ++g) {
        if (p.a_t) st = operand_map(a.ta, p.A, g, p.kdim, p.rows, 64);
        else st = operand_map(a.ta, p.A, g, p.rows, p.kdim, 128);
        if (st) return st;
        if (p.b_t) st = operand_map(a.tb, p.B, g, p.cols, p.kdim, 128);
        else st = operand_map(a.tb, p.B, g, p.kdim, p.cols, BK);
        if (st) return st;
        if (p.epi == LIN_GLU && (st = make_map(&a.tb[LIN_MAX_RANKS + g], p.B2[g], p.kdim, p.cols, BK))) return st;
    }
    const int outs = p.fused ? 1 : p.groups;
    a.keep = p.epi == LIN_DGLU || p.out2[0] != nullptr;
    for (int g = 0; g < outs; ++g) {
        if ((st = encode_out_map(&a.to[g], p.out[g], p.rows, p.cols, p.cols, p.out_f32))) return st;
        if (a.keep && (st = encode_out_map(&a.to2[g], p.out2[g], p.rows, p.cols, p.cols, false))) return st;
        if (a.keep && p.epi == LIN_GLU && (st = encode_out_map(&a.to3[g], p.out3[g], p.rows, p.cols, p.cols, false))) return st;
    }
    for (int g = 0; g < LIN_MAX_RANKS; ++g) {
        a.bias[g] = static_cast<const __nv_bfloat16*>(p.bias[g]);
        a.residual[g] = static_cast<const __nv_bfloat16*>(p.residual[g]);
        a.aux[g] = static_cast<const __nv_bfloat16*>(p.aux[g]);
        a.aux2[g] = static_cast<const __nv_bfloat16*>(p.aux2[g]);
    }
    a.has_bias = p.bias[0] != nullptr;
    a.has_residual = p.residual[0] != nullptr;
    a.act = p.act;
    a.ld = p.cols;
    a.groups = p.groups;
    a.fused = p.fused;
    a.groups_in_n = p.a_shared && !p.fused;
    a.rows = (int)p.rows;
    a.cols = (int)p.cols;
    a.m_tiles = (int)((p.rows + BM - 1) / BM);
    a.n_tiles = (int)((p.cols + tile_cols - 1) / tile_cols);
    a.kb_per_group = (int)((p.kdim + BK - 1) / BK);
    a.total_tiles = outs * a.m_tiles * a.n_tiles;
    // Short K: tall blocks of M tiles, whose A rows stay in L2 while the B columns
    // stream past; long K: near-square waves, which read the fewest panels (as
    // measured for the plain tensor-parallel MLP's products).
    const int64_t k_extent = (int64_t)(p.fused ? p.groups : 1) * a.kb_per_group * BK;
    a.group_m = k_extent >= 8192 ? 8 : 16;
    const int f32 = p.out_f32 ? CFG_F32 : 0;
    if (p.epi == LIN_GLU) return launch_t<LIN_GLU << CFG_EPI_SHIFT>(fn, a, stream);
    if (p.epi == LIN_DGLU) return launch_t<(LIN_DGLU << CFG_EPI_SHIFT) | CFG_B_T>(fn, a, stream);
    switch ((p.a_t ? CFG_A_T : 0) | (p.b_t ? CFG_B_T : 0) | f32) {
    case 0: return launch_t<0>(fn, a, stream);
    case CFG_F32: return launch_t<CFG_F32>(fn, a, stream);
    case CFG_A_T: return launch_t<CFG_A_T>(fn, a, stream);
    case CFG_A_T | CFG_F32: return launch_t<CFG_A_T | CFG_F32>(fn, a, stream);
    case CFG_B_T: return launch_t<CFG_B_T>(fn, a, stream);
    case CFG_B_T | CFG_F32: return launch_t<CFG_B_T | CFG_F32>(fn, a, stream);
    default: return fail(RTP_EUNSUPPORTED, "%s: no product with both operands transposed", fn);
    }
}

int take_linear_gemm_error(void* stream, uint32_t* code)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_tp_error, sizeof v, 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_tp_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return fail(RTP_ECUDA, "rtp_device_error: %s", cudaGetErrorString(cudaGetLastError()));
    *code = v;
    return RTP_OK;
}

}  // namespace rtp
