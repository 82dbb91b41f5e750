// Host side of the pair products (linear_gemm.cuh): tensor maps, tile counts, and the
// kernels whose clusters take whole tiles.
#include "linear_gemm.cuh"

namespace rtp {

namespace {

// Map of a whole row-major [rows, cols] buffer that the epilogue stores to or reads from.
int epi_map(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, bool f32)
{
    return encode_out_map(m, ptr, rows, cols, cols, f32);
}

// Encodes a map, or copies the previous group's when it is of the same buffer
// (a shared operand is encoded once).
int operand_map(CUtensorMap* maps, const void* const* ptrs, int i, int64_t rows, int64_t cols, int box_rows, int64_t ld)
{
    if (i > 0 && ptrs[i] == ptrs[i - 1]) {
        maps[i] = maps[i - 1];
        return RTP_OK;
    }
    return make_map(&maps[i], ptrs[i], rows, cols, box_rows, ld);
}

}  // namespace

int launch_linear_gemm(const char* fn, const LinGemm& p, cudaStream_t stream)
{
    static thread_local LinArgs a;
    std::memset(&a, 0, sizeof a);
    const int tile_cols = p.epi == LIN_GLU ? BN / 2 : BN;
    int st;
    for (int g = 0; g < p.groups; ++g) {
        if (p.a_t) st = operand_map(a.ta, p.A, g, p.kdim, p.rows, 64, p.lda);
        else st = operand_map(a.ta, p.A, g, p.rows, p.kdims[g] ? p.kdims[g] : p.kdim, 128, p.lda);
        if (st) return st;
        if (p.b_t) st = operand_map(a.tb, p.B, g, p.cols, p.kdims[g] ? p.kdims[g] : p.kdim, 128, p.ldb);
        else st = operand_map(a.tb, p.B, g, p.kdim, p.cols, BK, p.ldb);
        if (st) return st;
        if (p.epi == LIN_GLU && (st = make_map(&a.tb[LIN_MAX_RANKS + g], p.B2[g], p.kdim, p.cols, BK))) return st;
    }
    const int outs = p.fused ? 1 : p.groups;
    a.keep = p.epi == LIN_DGLU || p.out2[0] != nullptr;
    for (int g = 0; g < outs; ++g) {
        if (p.epi == LIN_EXP) st = encode_out_map(&a.to[g], p.out[g], p.rows, p.cols, p.ldo ? p.ldo : p.cols, false);
        else if (p.epi != LIN_LSE) st = epi_map(&a.to[g], p.out[g], p.rows, p.cols, p.out_f32);
        if (st) return st;
        if (a.keep && (st = epi_map(&a.to2[g], p.out2[g], p.rows, p.cols, false))) return st;
        if (a.keep && p.epi == LIN_GLU && (st = epi_map(&a.to3[g], p.out3[g], p.rows, p.cols, false))) return st;
        const void* in = p.epi == LIN_DGLU ? p.aux[g] : g < LIN_MAX_RANKS ? p.residual[g] : nullptr;
        if (in && (st = epi_map(&a.ti[g], in, p.rows, p.cols, false))) return st;
        if (p.epi == LIN_DGLU && (st = epi_map(&a.ti2[g], p.aux2[g], p.rows, p.cols, false))) return st;
    }
    for (int g = 0; g < LIN_MAX_RANKS; ++g) {
        a.bias[g] = static_cast<const __nv_bfloat16*>(p.bias[g]);
        a.residual[g] = static_cast<const __nv_bfloat16*>(p.residual[g]);
        a.h[g] = static_cast<__nv_bfloat16*>(p.out2[g]);
    }
    a.has_bias = p.bias[0] != nullptr;
    a.has_residual = p.residual[0] != nullptr;
    a.act = p.act;
    a.accumulate = p.accumulate;
    a.row_scale = p.row_scale;
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
    a.softmax = softmax_args(p.softmax, outs * a.n_tiles);
    // Short K: tall blocks of M tiles, whose A rows stay in L2 while the B columns
    // stream past; long K: near-square waves, which read the fewest panels (as
    // measured for the plain tensor-parallel MLP's products).
    const int64_t k_extent = (int64_t)(p.fused ? p.groups : 1) * a.kb_per_group * BK;
    a.group_m = k_extent >= 8192 ? 8 : 16;
    a.kbs = (p.fused ? p.groups : 1) * a.kb_per_group;
    const int cfg = (int)p.epi << CFG_EPI_SHIFT | (p.a_t ? CFG_A_T : 0) | (p.b_t ? CFG_B_T : 0) |
                    (p.out_f32 ? CFG_F32 : 0) | (p.epi == LIN_OUT && p.act ? CFG_ACT : 0);
    st = launch_linear_split(fn, cfg, a, stream);
    return st == LIN_NOT_SPLIT ? launch_cfg<false>(fn, cfg, a, stream) : st;
}

int take_linear_gemm_error(void* stream, uint32_t* code)
{
    uint32_t split = 0;
    int st = take_tp_error(stream, code);
    if (st || (st = take_linear_split_error(stream, &split))) return st;
    if (!*code) *code = split;
    return RTP_OK;
}

}  // namespace rtp
