// gemm_act8.cu -- the forward grouped GEMM with the fused SwiGLU whose pre-activation is
// kept in 8 bits: the engine's epilogue finds each row's largest |y| of 32 columns in the
// registers that hold them (the accumulators come 32 columns of one row a thread) and
// writes codes in place of bf16 rows, half the bytes.  Bound by the tensor cores: 16384 rows
// of 4096 -> 28672 over 8 experts take 2.00-2.11 ms (1.8-1.9 PFLOP/s, by the power cap),
// gg_forward_swiglu 2.15-2.22; 131072 rows of 2048 -> 1536 over 128 experts 470-494 us and
// 540-630.  Its pair
// kernels run producer and issuer as whole warps (2.23 -> 2.12 ms) and eight epilogue warps
// (2.12 -> 2.00 ms; 16384 rows of 1024 -> 4096 150 -> 84 us).
#include "gemm_launch.cuh"

using namespace gg;

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Upper bound on the expert-order row tiles (matmul_ogs.py, RoutingData.n_blocks).
int64_t row_tile_bound(int64_t R, int E) {
    if (R <= E) return R;
    return (R - E + 1 + kBM - 1) / kBM + E - 1;
}

template <int EPI>
int launch_kept(const gg_bf16* X, const gg_bf16* W, int64_t T, int E, int64_t N, int64_t K, int permute_x,
                GemmParams& p, cudaStream_t st) {
    CUtensorMap mA{}, mB{};
    const int64_t bound = row_tile_bound(p.R, E) * ((N + kBN - 1) / kBN);
    if (permute_x) {
        if (!encode_map_3d(&mB, W, K, N, E, K, N * K, kBK, kBN)) return GG_ERR_CUDA;
        p.ga = GatherSrc{X, K, T, K, ROW_TOKEN};
        return launch_gemm<KIND_RAGGED_M, false, false, true, false, false, EPI>(mB, mB, mB, mB, p, bound, st);
    }
    if (!encode_map_3d(&mB, W, K, N, E, K, N * K, kBK, kBN / 2)) return GG_ERR_CUDA;
    if (!encode_map_2d(&mA, X, K, p.R, K, kBK, kBM)) return GG_ERR_CUDA;
    return launch_gemm<KIND_RAGGED_M, false, false, false, false, true, EPI>(mA, mB, mA, mB, p, bound, st);
}

}  // namespace

extern "C" int gg_forward_swiglu_act8(const gg_bf16* X, const gg_bf16* W, const int32_t* m_sizes,
                                      const int32_t* gather_idx, int64_t T, int topk, int E, int64_t N, int64_t K,
                                      int permute_x, int fmt, uint8_t* codes, uint8_t* scales, gg_bf16* A,
                                      int32_t* status, void* stream) {
    if (T < 0 || topk < 1 || E < 1 || N < 0 || K < 0) return GG_ERR_INVALID_ARG;
    if (fmt != GG_ACT8_INT8 && fmt != GG_ACT8_E4M3) return GG_ERR_INVALID_ARG;
    if (topk > GG_MAX_TOPK || E > GG_MAX_EXPERTS || N % 16 || K % 8) return GG_ERR_UNSUPPORTED;
    const int64_t R = T * topk;
    if (R >= (int64_t(1) << 31) || N >= (int64_t(1) << 30) || K >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
    if (permute_x && !gather_idx) return GG_ERR_INVALID_ARG;
    if (R == 0 || N == 0) return GG_OK;
    if (!m_sizes || !codes || !scales || !A) return GG_ERR_INVALID_ARG;
    if (!al16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3u) || !al16(A)) return GG_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(m_sizes) | reinterpret_cast<uintptr_t>(gather_idx)) & 3u) return GG_ERR_UNSUPPORTED;
    if (K > 0 && (!X || !W)) return GG_ERR_INVALID_ARG;  // with K == 0 they have no elements
    if (K > 0 && (!al16(X) || !al16(W))) return GG_ERR_UNSUPPORTED;
    if (K > 0 && (N > INT64_MAX / 2 / E / K || R > INT64_MAX / 2 / K)) return GG_ERR_UNSUPPORTED;
    const Span outs[] = {{codes, R * act8_code_pitch(N)}, {scales, R * act8_scale_pitch(N)}, {A, R * N}};
    const Span ins[] = {{X, (permute_x ? T : R) * K * 2}, {W, E * N * K * 2}, {m_sizes, int64_t(E) * 4}, {gather_idx, R * 4}};
    if (outputs_overlap(outs, ins)) return GG_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) {  // y = 0: codes of 0 under the least scale
        int rc = cuda_result(cudaMemsetAsync(A, 0, static_cast<size_t>(R * (N / 2)) * 2, st));
        if (rc == GG_OK) rc = cuda_result(cudaMemsetAsync(codes, 0, static_cast<size_t>(R * act8_code_pitch(N)), st));
        if (rc == GG_OK) rc = cuda_result(cudaMemsetAsync(scales, 10, static_cast<size_t>(R * act8_scale_pitch(N)), st));
        return rc;
    }
    GemmParams p{};
    p.E = E;
    p.topk = topk;
    p.R = R;
    p.m_sizes = m_sizes;
    p.gather_idx = gather_idx;
    p.status = status;
    p.N = static_cast<int>(N);
    p.Kred = static_cast<int>(K);
    p.act_out = A;
    p.ld_act = N / 2;
    p.codes = codes;
    p.scales = scales;
    p.ld_codes = act8_code_pitch(N);
    p.ld_scales = act8_scale_pitch(N);
    return fmt == GG_ACT8_INT8 ? launch_kept<EPI_ACT8_INT8>(X, W, T, E, N, K, permute_x, p, st)
                               : launch_kept<EPI_ACT8_E4M3>(X, W, T, E, N, K, permute_x, p, st);
}
