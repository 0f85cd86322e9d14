// lora.cu -- entry points of the low-rank adapters beside a shared projection:
// argument checks and the order of the launches.  The kernels are in lora_plan.cu
// (the batch's plan), lora_shrink.cu (low-rank products), lora_project.cu (projections of few rows),
// lora_pair.cu (projections of many rows) and lora_grad.cu (adapter gradients).
#include "lora.cuh"

using namespace gg;

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// Sizes shared by the calls: GG_OK, or the code to return.
int check_sizes(int64_t T, int L, int r, int64_t N, int64_t K) {
    if (T < 0 || L < 1 || r < 1 || N < 0 || K < 0) return GG_ERR_INVALID_ARG;
    if (L > GG_MAX_EXPERTS || r > GG_LORA_MAX_RANK || r % 8 || N % 8 || K % 8) return GG_ERR_UNSUPPORTED;
    if (T >= (int64_t(1) << 31) - kUnit || N >= (int64_t(1) << 30) || K >= (int64_t(1) << 30)) return GG_ERR_UNSUPPORTED;
    return GG_OK;
}

// The backward's workspace: V, V in two parts, the gradients' counters and partial sums.
size_t v_bytes(int64_t T, int r) { return (static_cast<size_t>(T) * r * 2 + 255) / 256 * 256; }
constexpr size_t kCounterBytes = (kGradWords * sizeof(uint32_t) + 255) / 256 * 256;

// Y (or dX) from its operands: tiles with a split reduction, or 2-CTA tiles.  Splitting
// pays for few rows (whole forwards, split and 2-CTA: 64 rows of 4096 x 4096 15.6 and
// 19.5 us; 48 of 2048 x 2048, 32 mixed adapters 13.5 and 18.9; 64 in runs 12.4 and 13.0),
// and for a long reduction, the adapters' blocks among it, whose 2-CTA tiles leave half of
// the GPU idle.  The two meet near 44 blocks (one adapter, 128 to 513 rows, 8 to 26 tiles: at
// 40 blocks 14.9-16.4 and 15.0-15.9, at 52 15.5-17.4 and 17.2-18.2; 512 mixed rows of
// 4096 -> 2048, 32 adapters of rank 128: 33.0 and 44.8, 4 of rank 64: 17.7 and 14.8).
// Known to be off: 28 to 36 tiles of one adapter (256 rows of 4096 -> 7168: 24.1 and
// 21.6; 300 rows of 4096 x 4096 22.2 and 20.7, with four adapters 22.5 and 25.4), and many
// adapters of which few occur, which the host does not know (300 rows of 2048 x 2048, one
// of 256 adapters of rank 64: 19.2 and 16.8).
int project(bool b_mn, const uint16_t* X, const uint16_t* W, const uint16_t* U, const uint16_t* ad,
            const PlanView& plan, int64_t Kred, int64_t ncols, int r, uint16_t* out, uint32_t* ready, int32_t* status,
            cudaStream_t st) {
    const int64_t pairs = plan.units * ((ncols + 255) / 256);
    // reduction blocks of a tile, with those of the adapters that can occur in it
    const int64_t rchunks = (r + 63) / 64, per = 64 / rank_pad(r);
    const int64_t rows = plan.T < kUnit ? plan.T : kUnit;
    const int64_t adapters = (plan.L < rows ? plan.L : rows) * rchunks / per;
    const int64_t blocks = (Kred + 63) / 64 + adapters;
    if (plan.T <= 64 || (pairs * 4 < num_sms() && blocks > 44))
        return lora_project_launch(b_mn, X, W, U, ad, plan, Kred, ncols, r, out, ready, status, st);
    return lora_pair_launch(b_mn, X, W, U, ad, plan, Kred, ncols, r, out, ready, status, st);
}

}  // namespace

extern "C" {

size_t gg_lora_plan_size(int64_t T, int L) {
    if (T < 0 || L < 1 || L > GG_MAX_EXPERTS || T >= (int64_t(1) << 31) - kUnit) return 0;
    return plan_bytes_of(T, L);
}

int gg_lora_plan(const int32_t* ids, int64_t T, int L, void* plan, size_t plan_bytes, int32_t* status, void* stream) {
    if (T < 0 || L < 1) return GG_ERR_INVALID_ARG;
    if (L > GG_MAX_EXPERTS || T >= (int64_t(1) << 31) - kUnit) return GG_ERR_UNSUPPORTED;
    if (T == 0) return GG_OK;
    if (!ids) return GG_ERR_INVALID_ARG;
    if (!plan || plan_bytes < plan_bytes_of(T, L) || !al16(plan)) return GG_ERR_WORKSPACE;
    return lora_plan_launch(ids, plan_view(plan, T, L), status, as_stream(stream));
}

int gg_lora_forward(const gg_bf16* X, const gg_bf16* W, const gg_bf16* A, const gg_bf16* B, const float* scale,
                    const void* plan, int64_t T, int L, int r, int64_t N, int64_t K, gg_bf16* Y, gg_bf16* U,
                    int32_t* status, void* stream) {
    const int rc = check_sizes(T, L, r, N, K);
    if (rc != GG_OK) return rc;
    if (T == 0) return GG_OK;
    if (!plan || !U || (N > 0 && !Y)) return GG_ERR_INVALID_ARG;
    if (!al16(plan) || !al16(U) || !al16(Y)) return GG_ERR_UNSUPPORTED;
    cudaStream_t st = as_stream(stream);
    if (K == 0) {  // X, W and A have no elements
        int e = cuda_result(cudaMemsetAsync(U, 0, static_cast<size_t>(T) * r * 2, st));
        if (e == GG_OK && N > 0) e = cuda_result(cudaMemsetAsync(Y, 0, static_cast<size_t>(T * N) * 2, st));
        return e;
    }
    if (!X || !A || (N > 0 && (!W || !B))) return GG_ERR_INVALID_ARG;
    if (!al16(X) || !al16(W) || !al16(A) || !al16(B)) return GG_ERR_UNSUPPORTED;
    const PlanView v = plan_view(const_cast<void*>(plan), T, L);
    const int e = lora_shrink_launch(false, X, A, scale, v, K, r, U, nullptr, 0, nullptr, 0, status, st);
    if (e != GG_OK || N == 0) return e;
    return project(false, X, W, U, B, v, K, N, r, Y, nullptr, status, st);
}

size_t gg_lora_backward_workspace_size(int64_t T, int r) {
    if (T < 0 || r < 1) return 0;
    return 3 * v_bytes(T, r) + kCounterBytes + static_cast<size_t>(2 * kGradCtas) * 128 * r * sizeof(float);
}

int gg_lora_backward(const gg_bf16* dY, const gg_bf16* X, const gg_bf16* W, const gg_bf16* A, const gg_bf16* B,
                     const float* scale, const void* plan, const gg_bf16* U, int64_t T, int L, int r, int64_t N,
                     int64_t K, gg_bf16* dX, gg_bf16* dA, gg_bf16* dB, void* workspace, size_t workspace_bytes,
                     int32_t* status, void* stream) {
    const int rc = check_sizes(T, L, r, N, K);
    if (rc != GG_OK) return rc;
    if (!dX && !dA && !dB) return GG_OK;
    if (!al16(dX) || !al16(dA) || !al16(dB)) return GG_ERR_UNSUPPORTED;
    cudaStream_t st = as_stream(stream);
    const size_t lr = static_cast<size_t>(L) * r;
    if (T == 0 || N == 0 || K == 0) {  // nothing to sum: every gradient that has elements is zero
        int e = GG_OK;
        if (dX && T * K > 0) e = cuda_result(cudaMemsetAsync(dX, 0, static_cast<size_t>(T * K) * 2, st));
        if (e == GG_OK && dA && K > 0) e = cuda_result(cudaMemsetAsync(dA, 0, lr * K * 2, st));
        // (K == 0: U is zero, and so is dB)
        if (e == GG_OK && dB && N > 0) e = cuda_result(cudaMemsetAsync(dB, 0, lr * N * 2, st));
        return e;
    }
    if (!plan || !dY || !B || (dX && (!W || !A)) || (dA && !X) || (dB && !U)) return GG_ERR_INVALID_ARG;
    if (!al16(plan) || !al16(dY) || !al16(X) || !al16(W) || !al16(A) || !al16(B) || !al16(U)) return GG_ERR_UNSUPPORTED;
    if (!workspace || !al16(workspace) || workspace_bytes < gg_lora_backward_workspace_size(T, r)) return GG_ERR_WORKSPACE;
    const PlanView v = plan_view(const_cast<void*>(plan), T, L);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint16_t* V = reinterpret_cast<uint16_t*>(ws);
    const int64_t part = static_cast<int64_t>(v_bytes(T, r) / sizeof(uint16_t));
    uint16_t* parts = V + part;
    uint32_t* counters = reinterpret_cast<uint32_t*>(ws + 3 * v_bytes(T, r));
    float* sums = reinterpret_cast<float*>(ws + 3 * v_bytes(T, r) + kCounterBytes);
    int e;
    if (dX || dA)
        e = lora_shrink_launch(true, dY, B, scale, v, N, r, V, dA ? parts : nullptr, part, counters, kGradWords, status, st);
    else
        e = cuda_result(cudaMemsetAsync(counters, 0, kGradWords * sizeof(uint32_t), st));
    if (e == GG_OK && dX) e = project(true, dY, W, V, A, v, N, K, r, dX, dA || dB ? counters + kGradCtas : nullptr, status, st);
    if (e == GG_OK && (dA || dB))
        e = lora_grad_launch(X, dY, U, parts, parts + part, v, K, N, r, dA, dB, counters, sums,
                             dX ? GRAD_AFTER_DX : (dA ? GRAD_AFTER_V : GRAD_AFTER_OTHER), status, st);
    return e;
}

}  // extern "C"
