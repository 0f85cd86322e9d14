// block_norm_bwd.cu -- the gradients of the norms around a block (gg.h, "norms around a
// block"; block_norm.cu has the forward).
//
// Measured between graph nodes, both kernels (4.7 us of each are a launch's own, 6 the
// vectors' sums): 8192 x 4096 with a bf16 stream from int8 65 us, 5.7 TB/s; from bf16 72 us,
// 5.6 TB/s; with an fp32 stream from int8 95 us, 6.0 TB/s; 4097 x 2056 fp32 from e4m3 32 us.
// Bound by HBM behind those; 2048 x 16384 from int8, two CTAs a row: 82 us.  The norm of the
// stream alone, 8192 x 4096: 50 us bf16, 77 fp32 (5.4, 6.1 TB/s).
#include "block_norm.cuh"

namespace gg {
namespace {

struct NormBwd {
    const void* dh;
    const uint16_t* dx;
    const void* h;
    const uint16_t* y;
    const uint8_t *codes, *scales;
    const float *w_post, *gate, *token_gate, *w_pre;
    float res_scale, eps;
    int64_t T;
    int K, half;  // columns, and those of a row's first half (all, if it is not split)
    void* out_dh;
    uint16_t* dy;
    float *dtoken_gate, *part;
    int32_t* status;
    int stages, stage_bytes, st32;
    // a stage: h', dh', dx, y, its scales, the token's gate (those that the call has): the
    // bytes of each's rows, and where a stage has them
    int h_bytes, dh_bytes, dx_bytes, y_bytes, sc_bytes;
    int dh_at, dx_at, y_at, sc_at, tg_at;
    float inv_k;
    Probe probe;
};

enum KeptY { Y_NONE = 0, Y_BF16 = 1, Y_INT8 = 2, Y_E4M3 = 3 };

// One reduction a row.  With r, q the norms' factors and c = r^3 mean(w_pre dx h'),
//   G = dh' + r w_pre dx - c h',   sum(w G y) = A + r B - c C
// (w = w_post gate; A, B, C the sums of w y dh', w y w_pre dx, w y h'), so all six sums
// come from the rows as loaded, and the second pass over the stage writes both outputs.
//
// ALL: dh, dx and both row outputs are there.  Tests for absent tensors, uniform as they are,
// cut the loads of a row's halves apart: 8192 x 4096 from int8 took 77 us with them, 67
// without.  (Units of 8 columns and twice the threads, 64 registers each: 91 us, for a row's
// sums and factors are every thread's.)
// SPLIT: a cluster's two CTAs have halves of each row.
template <bool F32, int YK, bool SPLIT, bool FULL, bool ALL, bool PROBE = false>
__global__ void __launch_bounds__(kMaxThreads, 1) block_norm_bwd_kernel(const NormBwd p) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int hs = F32 ? 4 : 2;
    constexpr int FMT = YK == Y_E4M3 ? GG_ACT8_E4M3 : GG_ACT8_INT8;
    Ctl* ctl = reinterpret_cast<Ctl*>(smem);
    uint8_t* ring = smem + sizeof(Ctl);
    // K columns from column col0 are this CTA's
    const uint32_t side = SPLIT ? cluster_ctarank() : 0u;
    const int col0 = side ? p.half : 0, K = !SPLIT ? p.K : side ? p.K - p.half : p.half;
    const int64_t first = SPLIT ? cluster_id_x() : blockIdx.x, step = SPLIT ? nclusters_x() : gridDim.x;
    const bool has_dx = ALL || p.dx != nullptr, has_dh = ALL || p.dh != nullptr;
    const bool small = YK >= Y_INT8 || p.token_gate;
    // what this CTA copies of each row, and from where
    const int in_stream = K * hs, in_y = YK == Y_BF16 ? 2 * K : static_cast<int>(act8_code_pitch(K));
    const int h_copied = SPLIT ? (has_dx ? in_stream : 0) : p.h_bytes, dh_copied = SPLIT ? (has_dh ? in_stream : 0) : p.dh_bytes;
    const int dx_copied = SPLIT ? (has_dx ? 2 * K : 0) : p.dx_bytes, y_copied = SPLIT ? (YK == Y_NONE ? 0 : in_y) : p.y_bytes;
    const int sc_copied = SPLIT ? static_cast<int>(act8_scale_pitch(K)) : p.sc_bytes;
    const uint8_t* from_h = static_cast<const uint8_t*>(p.h) + col0 * hs;
    const uint8_t* from_dh = static_cast<const uint8_t*>(p.dh) + col0 * hs;
    const uint8_t* from_dx = reinterpret_cast<const uint8_t*>(p.dx + col0);
    const uint8_t* from_y = YK == Y_BF16 ? reinterpret_cast<const uint8_t*>(p.y + col0) : p.codes + col0;
    const uint8_t* from_sc = p.scales + col0 / kActBlock;
    if (!FULL) {
        const int area_k = SPLIT ? p.half : K;
        for (int s = 0; s < p.stages; ++s) {
            uint8_t* at = ring + s * p.stage_bytes;
            if (has_dx) zero_pad(at, h_copied, stream_area(F32, area_k));
            if (has_dh) zero_pad(at + p.dh_at, dh_copied, stream_area(F32, area_k));
            if (has_dx) zero_pad(at + p.dx_at, dx_copied, bf16_area(F32, area_k));
            if (YK != Y_NONE) zero_pad(at + p.y_at, y_copied, YK == Y_BF16 ? bf16_area(F32, area_k) : code_area(F32, area_k));
        }
    }
    init_ring(ctl, p.stages, small ? 33 : 1, !SPLIT ? 0 : YK == Y_NONE ? 2 : 6);

    int64_t t_in = first;
    int s_in = 0;
    Account<PROBE> account;
    constexpr uint64_t limit = PROBE ? kProbeWaitNs : kWaitLimitNs;
    // Warp 0 loads: lane 0 the rows, all of them the scales and the gate in words (rows of
    // scales have no 16-byte alignment), whose arrivals the barrier counts as they land.
    auto refill = [&]() {
        if (warp_id() != 0 || t_in >= p.T) return;
        uint8_t* to = ring + s_in * p.stage_bytes;
        uint64_t* bar = &ctl->full[s_in];
        if constexpr (PROBE) account.fill(ctl, p.stages, (t_in - first) / step);
        const bool held = PROBE && t_in == p.probe.withheld && side == 0;
        if (lane_id() == 0) {
            mbar_arrive_expect_tx(bar, h_copied + dh_copied + dx_copied + y_copied);
            if (h_copied && !held) bulk_row(to, from_h + t_in * p.h_bytes, h_copied, bar);
            if (dh_copied) bulk_row(to + p.dh_at, from_dh + t_in * p.dh_bytes, dh_copied, bar);
            if (dx_copied) bulk_row(to + p.dx_at, from_dx + t_in * p.dx_bytes, dx_copied, bar);
            if (YK != Y_NONE) bulk_row(to + p.y_at, from_y + t_in * p.y_bytes, y_copied, bar);
        }
        if (small) {
            if (YK >= Y_INT8)
                for (int b = 4 * lane_id(); b < sc_copied; b += 128) copy_word(to + p.sc_at + b, from_sc + t_in * p.sc_bytes + b);
            if (p.token_gate && lane_id() == 0) copy_word(to + p.tg_at, p.token_gate + t_in);
            cp_async_mbar_arrive(bar);
        }
        t_in += step;
        if (++s_in == p.stages) s_in = 0;
    };
    for (int s = 0; s < p.stages; ++s) refill();

    Cols<F32, FULL> cols;
    Unit wp, wx, pre, post;
    cols.init(K);
#pragma unroll
    for (int k = 0; k < 8; ++k) pre.v[k] = post.v[k] = 0;
    cols.get_weight(p.w_pre ? p.w_pre + col0 : nullptr, wx);
    cols.get_weights(p.w_post ? p.w_post + col0 : nullptr, p.gate ? p.gate + col0 : nullptr, wp);
    const f32x2 a2 = pair(p.res_scale, p.res_scale);
    // A unit of neighbouring columns lies in one block of y, whose factor its sums take;
    // quads lie in four.
    constexpr int SC = F32 ? 4 : 1;
    int stage = 0;
    uint32_t parity = 0, calls = 0;
    bool at_first = true, left = false;
    for (int64_t t = first; t < p.T; t += step) {
        const uint8_t* rows = ring + stage * p.stage_bytes;
        wait_row(&ctl->full[stage], parity, ctl, p.status, limit);
        account.waited();
        const float tg = p.token_gate ? *reinterpret_cast<const float*>(rows + p.tg_at) : 1.f;
        auto scale = [&](int j) { return cols.holds(j) ? rows[p.sc_at + (cols.column(j) >> 5)] : uint8_t(0); };
        const float factor = YK >= Y_INT8 && !F32 ? act8_factor(scale(0)) : 1.f;
        float quad_factor[SC];
#pragma unroll
        for (int j = 0; j < SC; ++j) quad_factor[j] = YK >= Y_INT8 && F32 ? act8_factor(scale(j)) : 1.f;
        // y (bf16 stream: but for its block's factor)
        auto get_y = [&](int half, f32x2 (&y)[4]) {
            if constexpr (YK == Y_BF16) {
                cols.get_bf16(rows + p.y_at, half, y);
            } else {
                uint32_t w[2];
                cols.get_codes(rows + p.y_at, half, w);
                code_pairs<FMT>(w[0], y[0], y[1]);
                code_pairs<FMT>(w[1], y[2], y[3]);
                if constexpr (F32) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float f = quad_factor[2 * half + (k >> 1)];
                        y[k] = mul2(y[k], pair(f, f));
                    }
                }
            }
        };
        float sum[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        f32x2 s[6] = {0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            f32x2 h[4], d[4], y[4];
            if (has_dx) {
                cols.get_stream(rows, half, h);
                cols.get_bf16(rows + p.dx_at, half, d);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    d[k] = mul2(d[k], wx.v[4 * half + k]);
                    s[0] = fma2(h[k], h[k], s[0]);
                    s[1] = fma2(d[k], h[k], s[1]);
                }
            }
            if (YK != Y_NONE) {
                const f32x2* w = wp.v + 4 * half;
                get_y(half, y);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s[2] = fma2(y[k], y[k], s[2]);
                    y[k] = mul2(y[k], w[k]);
                }
                if (has_dx) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        s[4] = fma2(y[k], d[k], s[4]);
                        s[5] = fma2(y[k], h[k], s[5]);
                    }
                }
                if (has_dh) {
                    cols.get_stream(rows + p.dh_at, half, h);
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[3] = fma2(y[k], h[k], s[3]);
                }
            }
        }
        sum[0] += both(s[0]);
        sum[1] += both(s[1]);
        if (YK != Y_NONE) {
            sum[2] += YK == Y_BF16 ? both(s[2]) : factor * (factor * both(s[2]));
#pragma unroll
            for (int k = 3; k < 6; ++k) sum[k] += factor * both(s[k]);
        }
        if (YK == Y_NONE) {
            float two[2] = {sum[0], sum[1]};
            left = row_sum<2, SPLIT>(two, ctl, calls, p.status);
            sum[0] = two[0], sum[1] = two[1];
        } else {
            left = row_sum<6, SPLIT>(sum, ctl, calls, p.status);
        }
        if (left) break;
        // past this barrier the previous row's stage has been read by all
        if (!at_first && p.stages > 1) refill();
        at_first = false;
        const float r = has_dx ? rsqrtf(fmaf(sum[0], p.inv_k, p.eps)) : 0.f;
        const float c = has_dx ? r * (r * (r * (sum[1] * p.inv_k))) : 0.f;  // (r^3 alone can pass the largest float)
        const float q = p.w_post ? rsqrtf(fmaf(sum[2], p.inv_k, p.eps)) : 1.f;
        const float z = sum[3] + r * sum[4] - c * sum[5];
        if (p.dtoken_gate && threadIdx.x == 0 && side == 0) p.dtoken_gate[t] = z * q;
        const float cy = p.w_post ? q * (q * (q * (tg * (z * p.inv_k)))) : 0.f;
        const f32x2 r2 = pair(r, r), c2 = pair(-c, -c), q2 = pair(q * tg, q * tg);
        uint8_t* to_dy = reinterpret_cast<uint8_t*>(p.dy + col0) + t * (2 * p.K);
        uint8_t* to_dh = static_cast<uint8_t*>(p.out_dh) + col0 * hs + t * (p.K * hs);
        const float fy = -cy * factor, fq = q * tg * factor;
        const f32x2 fy2 = pair(fy, fy), fq2 = pair(fq, fq);
        Unit G, m;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            f32x2 h[4], d[4], y[4];
            f32x2* g = G.v + 4 * half;
            if (has_dh) {
                cols.get_stream(rows + p.dh_at, half, g);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) g[k] = 0;
            }
            if (has_dx) {
                cols.get_stream(rows, half, h);
                cols.get_bf16(rows + p.dx_at, half, d);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int x = 4 * half + k;
                    d[k] = mul2(d[k], r2);
                    pre.v[x] = fma2(d[k], h[k], pre.v[x]);
                    g[k] = fma2(d[k], wx.v[x], g[k]);
                    g[k] = fma2(h[k], c2, g[k]);
                }
            }
            if (YK != Y_NONE) {
                const f32x2* w = wp.v + 4 * half;
                get_y(half, y);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int x = 4 * half + k;
                    post.v[x] = fma2(mul2(g[k], y[k]), fq2, post.v[x]);
                    m.v[x] = fma2(y[k], fy2, mul2(mul2(g[k], w[k]), q2));
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) g[k] = mul2(g[k], a2);
        }
        if (YK != Y_NONE && (ALL || p.dy)) cols.put_bf16(to_dy, p.st32, m);
        if (ALL || p.out_dh) cols.put_stream(to_dh, p.st32, G);
        if (p.stages == 1) {
            __syncthreads();
            refill();
        }
        if (++stage == p.stages) {
            stage = 0;
            parity ^= 1u;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;");
    // (left: a CTA whose own waits all ended leaves as well when the other half's gave up)
    if (left && threadIdx.x == 0) {
        drain_ring(ctl, p.stages, (t_in - first) / step, limit);
        account.drained();
    }
    account.put(p.probe, left, (t_in - first) / step);
    if (p.part) {
        float* to = p.part + first * 2 * p.K + col0;
        cols.put_sums(to, pre);
        cols.put_sums(to + p.K, post);
    }
    if (SPLIT) leave_pair();
}

// dw_pre, dw_post, dgate from the CTAs' partial sums [ctas][2][K]: a CTA takes 8 columns
// of both kinds (a sector of each row; whole lines of one kind were 1-9 us slower but for
// 8192 columns), two lanes a row; what a lane summed is joined over
// the lanes and then the warps, in their order.  256 threads up to 512 rows, a few loads
// each, 512 for more (narrow rows have up to 2432; 128, 256 or 512 threads made 0.4 us of
// difference for 304 rows of 4096 columns).
constexpr int kSumThreads = 512;
constexpr int kSumCols = 8;
__global__ void __launch_bounds__(kSumThreads)
block_norm_sum_kernel(const float* __restrict__ part, int ctas, int K, const float* w_post, const float* gate,
                      float* dw_post, float* dw_pre, float* dgate) {
    __shared__ float s[kSumThreads / 32][2][kSumCols];
    const int lane = lane_id(), c = blockIdx.x * kSumCols + 4 * (lane & 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = threadIdx.x >> 1; i < ctas; i += blockDim.x / 2) {
        const float* from = part + static_cast<int64_t>(i) * 2 * K + c;
        const float4 a = __ldcg(reinterpret_cast<const float4*>(from)), b = __ldcg(reinterpret_cast<const float4*>(from + K));
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int d = 16; d > 1; d >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
        if (lane < 2) s[warp_id()][k >> 2][4 * lane + (k & 3)] = v[k];
    }
    __syncthreads();
    if (threadIdx.x >= 2 * kSumCols) return;
    const int kind = threadIdx.x >> 3, col = threadIdx.x & 7, at = blockIdx.x * kSumCols + col;
    float sum = 0.f;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) sum += s[w][kind][col];
    if (kind == 0) {
        if (dw_pre) dw_pre[at] = sum;
    } else {
        if (dw_post) dw_post[at] = gate ? gate[at] * sum : sum;
        if (dgate) dgate[at] = w_post ? w_post[at] * sum : sum;
    }
}

// Rows of partial sums.
int64_t bwd_parts(int64_t T, int64_t K) {
    const int64_t n = norm_rows(K, norm_per_sm(K));
    return T < n ? T : n;
}

struct Launch {
    bool split, full, all;
    unsigned rows;
    int threads;
    size_t smem;
    cudaStream_t st;
};
template <bool F32, int YK, bool SPLIT, bool FULL, bool ALL>
int launch_bwd(const NormBwd& p, const Launch& l) {
    static std::atomic<uint64_t> done;
    return launch(block_norm_bwd_kernel<F32, YK, SPLIT, FULL, ALL>, done, p, SPLIT, l.rows, l.threads, l.smem, l.st);
}
template <bool F32, int YK>
int launch_bwd(const NormBwd& p, const Launch& l) {
    if (l.split) return l.all ? launch_bwd<F32, YK, true, false, true>(p, l) : launch_bwd<F32, YK, true, false, false>(p, l);
    return l.full  ? launch_bwd<F32, YK, false, true, true>(p, l)
           : l.all ? launch_bwd<F32, YK, false, false, true>(p, l)
                   : launch_bwd<F32, YK, false, false, false>(p, l);
}
// The diagnostic form: a bf16 stream and y.
template <bool SPLIT>
int launch_probe(const NormBwd& p, const Launch& l) {
    static std::atomic<uint64_t> done;
    return launch(block_norm_bwd_kernel<false, Y_BF16, SPLIT, false, true, true>, done, p, SPLIT, l.rows, l.threads, l.smem, l.st);
}

size_t workspace_size(int64_t T, int64_t K) {
    if (T <= 0 || K <= 0 || K > GG_NORM_MAX_K) return 0;
    return static_cast<size_t>(bwd_parts(T, K)) * 2 * static_cast<size_t>(K) * sizeof(float);
}

int block_norm_bwd(const void* dh, const gg_bf16* dx, const void* h, int h_dtype, const gg_bf16* y, const uint8_t* y_codes,
                   const uint8_t* y_scales, int fmt, const float* w_post, const float* gate, const float* token_gate,
                   float res_scale, const float* w_pre, float eps, int64_t T, int64_t K, void* out_dh, gg_bf16* dy,
                   float* dw_post, float* dw_pre, float* dgate, float* dtoken_gate, void* workspace,
                   size_t workspace_bytes, int32_t* status, void* stream, const Probe* probe) {
    if (T < 0 || K < 0) return GG_ERR_INVALID_ARG;
    if (h_dtype != GG_DTYPE_BF16 && h_dtype != GG_DTYPE_F32) return GG_ERR_INVALID_ARG;
    if (fmt != GG_ACT8_INT8 && fmt != GG_ACT8_E4M3) return GG_ERR_INVALID_ARG;
    if (!(eps > 0.f && eps < INFINITY)) return GG_ERR_INVALID_ARG;
    if (K % 8 || K > GG_NORM_MAX_K || T >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
    if (!y_codes != !y_scales || (y_codes && y)) return GG_ERR_INVALID_ARG;
    const bool has_y = y || y_codes, sums = dw_post || dw_pre || dgate;
    if (T > 0 && K > 0) {
        if (!dx != !w_pre || (dw_pre && !dx)) return GG_ERR_INVALID_ARG;
        if (!has_y && (w_post || gate || token_gate || dy || dw_post || dgate || dtoken_gate)) return GG_ERR_INVALID_ARG;
        if (dw_post && !w_post) return GG_ERR_INVALID_ARG;
        if (dx && !h) return GG_ERR_INVALID_ARG;
    }
    const void* ptrs[] = {dh, dx, h, y, y_codes, w_post, gate, w_pre, out_dh, dy, dw_post, dw_pre, dgate, workspace};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return GG_ERR_UNSUPPORTED;
    const void* words[] = {y_scales, token_gate, dtoken_gate};
    for (const void* q : words)
        if (!aligned(q, 4)) return GG_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0 || T == 0) {  // empty sums
        float* vec[] = {dw_post, dw_pre, dgate};
        for (float* q : vec)
            if (q && K > 0) {
                const int rc = cuda_result(cudaMemsetAsync(q, 0, static_cast<size_t>(K) * 4, st));
                if (rc != GG_OK) return rc;
            }
        return dtoken_gate && T > 0 ? cuda_result(cudaMemsetAsync(dtoken_gate, 0, static_cast<size_t>(T) * 4, st)) : GG_OK;
    }
    if (sums && (!workspace || workspace_bytes < workspace_size(T, K))) return GG_ERR_WORKSPACE;
    const bool f32 = h_dtype == GG_DTYPE_F32;
    {
        const int64_t hb = T * K * (f32 ? 4 : 2), xb = T * K * 2, vb = K * 4;
        // out_dh may be dh itself; the other rows may then be dh too
        const int64_t row = hb / T;
        const Span outs[] = {{dy, xb}, {dw_post, vb}, {dw_pre, vb}, {dgate, vb}, {dtoken_gate, T * 4},
                             {sums ? workspace : nullptr, static_cast<int64_t>(workspace_size(T, K))},
                             {out_dh, hb, out_dh == dh ? row : 0}};
        const Span ins[] = {{dh, hb, row}, {dx, xb, 2 * K}, {h, hb, row}, {y, xb, 2 * K}, {y_codes, T * act8_code_pitch(K)},
                            {y_scales, T * act8_scale_pitch(K)}, {w_post, vb}, {gate, vb}, {w_pre, vb}, {token_gate, T * 4}};
        if (outputs_overlap(outs, ins)) return GG_ERR_INVALID_ARG;
    }
    // without a block h' is h: the scale is the residual's beside one
    NormBwd p{dh, dx, h, y, y_codes, y_scales, w_post, gate, token_gate, w_pre, has_y ? res_scale : 1.f, eps, T,
              static_cast<int>(K), static_cast<int>(norm_half(K)), out_dh, dy, dtoken_gate, sums ? static_cast<float*>(workspace) : nullptr, status,
              0, 0, K % 16 == 0 && aligned(out_dh, 32) && aligned(dy, 32)};
    const int k = p.K, part = p.half;
    auto place = [&p](int area) {
        const int at = p.stage_bytes;
        p.stage_bytes += area;
        return at;
    };
    p.inv_k = 1.f / static_cast<float>(k);
    if (dx) {
        p.h_bytes = k * (f32 ? 4 : 2);
        place(stream_area(f32, part));
    }
    if (dh) {
        p.dh_bytes = k * (f32 ? 4 : 2);
        p.dh_at = place(stream_area(f32, part));
    }
    if (dx) {
        p.dx_bytes = 2 * k;
        p.dx_at = place(bf16_area(f32, part));
    }
    if (y) {
        p.y_bytes = 2 * k;
        p.y_at = place(bf16_area(f32, part));
    } else if (y_codes) {
        p.y_bytes = static_cast<int>(act8_code_pitch(K));
        p.y_at = place(code_area(f32, part));
        p.sc_bytes = static_cast<int>(act8_scale_pitch(K));
        p.sc_at = place((static_cast<int>(act8_scale_pitch(part)) + 15) / 16 * 16);
    }
    if (token_gate) p.tg_at = place(16);
    if (p.stage_bytes == 0) p.stage_bytes = 16;  // nothing given: zeros go out
    int per_sm = norm_per_sm(K);
    const int threads = norm_threads(K);
    p.stages = ring_stages(p.stage_bytes, per_sm);
    const int64_t most = norm_rows(K, per_sm);
    const bool all = dh && dx && out_dh && (dy || !has_y);
    const Launch l{norm_split(K), all && p.st32 && K == 16 * threads, all, static_cast<unsigned>(T < most ? T : most), threads,
                   sizeof(Ctl) + static_cast<size_t>(p.stages) * p.stage_bytes, st};
    if (probe) {
        p.probe = *probe;
        return l.split ? launch_probe<true>(p, l) : launch_probe<false>(p, l);
    }
    const int kind = y ? Y_BF16 : !y_codes ? Y_NONE : fmt == GG_ACT8_INT8 ? Y_INT8 : Y_E4M3;
#define GG_BWD(F)                                        \
    (kind == Y_NONE   ? launch_bwd<F, Y_NONE>(p, l)      \
     : kind == Y_BF16 ? launch_bwd<F, Y_BF16>(p, l)      \
     : kind == Y_INT8 ? launch_bwd<F, Y_INT8>(p, l)      \
                      : launch_bwd<F, Y_E4M3>(p, l))
    const int rc = f32 ? GG_BWD(true) : GG_BWD(false);
#undef GG_BWD
    if (rc != GG_OK || !sums) return rc;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(K / kSumCols));
    cfg.blockDim = dim3(l.rows <= 512 ? 256 : kSumThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_result(cudaLaunchKernelEx(&cfg, block_norm_sum_kernel, static_cast<const float*>(p.part),
                                          static_cast<int>(l.rows), p.K, w_post, gate, dw_post, dw_pre, dgate));
}

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

size_t gg_block_norm_bwd_workspace_size(int64_t T, int64_t K) { return workspace_size(T, K); }

int gg_block_norm_bwd(const void* dh, const gg_bf16* dx, const void* h, int h_dtype, const gg_bf16* y,
                      const uint8_t* y_codes, const uint8_t* y_scales, int fmt, const float* w_post,
                      const float* gate, const float* token_gate, float res_scale, const float* w_pre, float eps,
                      int64_t T, int64_t K, void* out_dh, gg_bf16* dy, float* dw_post, float* dw_pre, float* dgate,
                      float* dtoken_gate, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    return block_norm_bwd(dh, dx, h, h_dtype, y, y_codes, y_scales, fmt, w_post, gate, token_gate, res_scale, w_pre, eps, T,
                          K, out_dh, dy, dw_post, dw_pre, dgate, dtoken_gate, workspace, workspace_bytes, status, stream,
                          nullptr);
}

int gg_selftest_block_norm_bwd_wait(const gg_bf16* dx, const gg_bf16* h, const gg_bf16* y, const float* w, int64_t T,
                                    int64_t K, int64_t withheld, gg_bf16* out_dh, gg_bf16* dy, int32_t* record,
                                    int32_t* status, void* stream) {
    if (!dx || !y || !w || !out_dh || !dy || !record || !status || withheld < 0 || withheld >= T) return GG_ERR_INVALID_ARG;
    if (!aligned(record, 4) || !aligned(status, 4)) return GG_ERR_UNSUPPORTED;
    Probe probe;
    probe.withheld = withheld;
    probe.record = record;
    return block_norm_bwd(dx, dx, h, GG_DTYPE_BF16, y, nullptr, nullptr, GG_ACT8_INT8, w, nullptr, nullptr, 1.f, w, 1e-6f, T,
                          K, out_dh, dy, nullptr, nullptr, nullptr, nullptr, nullptr, 0, status, stream, &probe);
}

}  // extern "C"
