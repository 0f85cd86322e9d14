// block_norm.cu -- the norms around a block, fused with the top-k combine of its rows, its
// gates and the scaled residual (gg.h, "norms around a block"); block_norm_bwd.cu has the
// gradients.
//
// Measured between graph nodes (4.7 us of each are a launch's own): 8192 x 4096 bf16 50 us,
// 5.4 TB/s (41 us alone, 18 instructions an element); with a stream of fp32 71 us, 5.7 TB/s;
// eight expert rows of 2048 columns combined for 16384 tokens, fp32 stream, y kept in int8:
// 138 us, 6.6 TB/s; two rows of 4096 for 8192 tokens: 59 us, 5.6 TB/s; 2048 x 16384, two CTAs a
// row: 56 us.  The norm of the stream alone, 8192 x 4096: 22 us bf16, 33 fp32 (6.0, 6.2 TB/s).
#include "block_norm.cuh"

namespace gg {
namespace {

struct NormFwd {
    const void* h;
    const uint16_t* Y;
    const int32_t* map;
    const float* topk_w;
    int topk;
    const float *w_post, *gate, *token_gate, *w_pre;
    float res_scale, eps;
    int64_t T;
    int K, half;  // columns, and those of a row's first half (all, if it is not split)
    void* out_h;
    uint16_t *out_x, *out_y;
    uint8_t *codes, *scales;
    int32_t* status;
    int stages, stage_bytes, slots, groups;  // expert rows a stage, stages a token
    int st32;                                // output rows start 32-byte aligned
    Probe probe;
};

enum Keep { KEEP_NONE = 0, KEEP_BF16 = 1, KEEP_INT8 = 2, KEEP_E4M3 = 3 };
// y: none, a row as it is, a sum of few rows, of more
enum Source { SRC_NONE = 0, SRC_ROW = 1, SRC_FEW = 2, SRC_SLOTS = 3 };

constexpr int kFewRows = 3;    // up to these SRC_FEW
constexpr int kMinStages = 2;  // of a sum's rows

// A thread's 16 columns of y in 8 bits: the block's largest |y| from the lanes that share
// it (whole warps call this: two neighbours, or of each quad eight).
template <bool F32, bool FULL, int FMT>
__device__ __forceinline__ void keep_unit(const Cols<F32, FULL>& cols, const Unit& y, uint8_t* codes, uint8_t* scales,
                                          int code_pitch) {
    float f[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) split(y.v[k], f[2 * k], f[2 * k + 1]);
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) m = amax_nan(m, f[4 * j + k]);
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) m = amax_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
            const uint32_t s = act8_scale<FMT>(m), c = cols.column(j);
            if (FULL || c < static_cast<uint32_t>(code_pitch)) {
                *reinterpret_cast<uint32_t*>(codes + c) =
                    act8_code4<FMT>(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3], act8_inverse(s));
                if ((c & 31) == 0) scales[c >> 5] = static_cast<uint8_t>(s);
            }
        }
    } else {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) m = amax_nan(m, f[k]);
        m = amax_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const uint32_t s = act8_scale<FMT>(m), c = cols.column(0);
        const float inv = act8_inverse(s);
        if (FULL || c < static_cast<uint32_t>(code_pitch)) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = act8_code4<FMT>(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3], inv);
            *reinterpret_cast<uint4*>(codes + c) = make_uint4(w[0], w[1], w[2], w[3]);
            if ((c & 31) == 0) scales[c >> 5] = static_cast<uint8_t>(s);
        }
    }
}

// Two rows are done at once unless y is a sum, whose rows fill the ring by themselves.
// Sums of up to three rows take 80 registers, so that three CTAs of 256 threads share an SM
// (8192 x 4096 with two rows a token: 69 us with two CTAs, 59 with three; eight rows of 2048
// columns: 138 and 150); the others two.  SPLIT: a cluster's two CTAs have halves of each row.
template <bool F32, int KEEP, bool SPLIT, bool FULL, int SRC, bool PROBE = false>
__global__ void __maxnreg__(SRC == SRC_FEW ? 80 : 128) block_norm_kernel(const NormFwd p) {
    constexpr bool SUM = SRC >= SRC_FEW;
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int ROWS = SUM ? 1 : 2;
    constexpr int hs = F32 ? 4 : 2;
    Ctl* ctl = reinterpret_cast<Ctl*>(smem);
    uint8_t* ring = smem + sizeof(Ctl);
    const int lane = lane_id();
    // K columns from column col0 are this CTA's
    const uint32_t side = SPLIT ? cluster_ctarank() : 0u;
    const int col0 = side ? p.half : 0, K = !SPLIT ? p.K : side ? p.K - p.half : p.half;
    const int64_t first = SPLIT ? cluster_id_x() : blockIdx.x, step = SPLIT ? nclusters_x() : gridDim.x;
    const int row_bytes = 2 * K, row_area = bf16_area(F32, SPLIT ? p.half : K);
    const int h_at = SRC == SRC_NONE ? 0 : SRC == SRC_ROW ? row_area : p.slots * row_area;
    const int groups = SUM ? p.groups : 1;
    const float inv_k = 1.f / p.K;
    const uint16_t* from_y = p.Y + col0;
    const uint8_t* from_h = static_cast<const uint8_t*>(p.h) + col0 * hs;
    const float *w_post = p.w_post ? p.w_post + col0 : nullptr, *gate = p.gate ? p.gate + col0 : nullptr;
    const float* w_pre = p.w_pre ? p.w_pre + col0 : nullptr;
    if (!FULL) {
        for (int s = 0; s < p.stages; ++s) {
            uint8_t* at = ring + s * p.stage_bytes;
            for (int j = 0; SRC != SRC_NONE && j < (SRC == SRC_ROW ? 1 : p.slots); ++j)
                zero_pad(at + j * row_area, row_bytes, row_area);
            zero_pad(at + h_at, K * hs, stream_area(F32, SPLIT ? p.half : K));
        }
    }
    init_ring(ctl, p.stages, SUM ? 32 : 1, SPLIT ? ROWS : 0);

    // Warp 0 loads: thread 0 a token's rows; of a sum lane j the j-th expert row of the
    // stage's group, lane 0 the residual row with a token's last group.  The number and
    // weight of an expert row are read one stage before they are needed.
    int64_t t_in = first;
    int g_in = 0, s_in = 0;
    auto issued = [&]() { return (t_in - first) / step * groups + g_in; };
    Account<PROBE> account;
    constexpr uint64_t limit = PROBE ? kProbeWaitNs : kWaitLimitNs;
    int32_t row_in = -1;
    float w_in = 1.f;
    auto look_up = [&]() {
        const int j = g_in * p.slots + lane;
        row_in = -1;
        if (t_in < p.T && lane < p.slots && j < p.topk) {
            const int64_t f = t_in * p.topk + j;
            row_in = p.map ? p.map[f] : static_cast<int32_t>(f);
            w_in = p.topk_w ? p.topk_w[f] : 1.f;
        }
    };
    auto issue = [&]() {
        if (t_in >= p.T) return;
        uint8_t* stage = ring + s_in * p.stage_bytes;
        uint64_t* bar = &ctl->full[s_in];
        if constexpr (PROBE) account.fill(ctl, p.stages, issued());
        if constexpr (SUM) {
            const bool held = PROBE && t_in == p.probe.withheld && g_in == 0 && side == 0;
            const bool slot = lane < p.slots && g_in * p.slots + lane < p.topk;
            const bool ok = slot && row_in >= 0 && row_in < p.T * p.topk;
            if (slot) {
                if (!ok) set_status(p.status, GG_DEV_BAD_ROW_INDEX);
                ctl->slot[s_in][lane] = Slot{w_in, ok};
            }
            const uint32_t hb = lane == 0 && g_in == groups - 1 ? K * hs : 0;
            mbar_arrive_expect_tx(bar, (ok ? row_bytes : 0) + hb);
            if (ok && !held) bulk_row(stage + lane * row_area, from_y + static_cast<int64_t>(row_in) * p.K, row_bytes, bar);
            if (hb) bulk_row(stage + h_at, from_h + t_in * (p.K * hs), hb, bar);
            if (++g_in == groups) {
                g_in = 0;
                t_in += step;
            }
        } else {
            mbar_arrive_expect_tx(bar, (SRC == SRC_ROW ? row_bytes : 0) + K * hs);
            if (SRC == SRC_ROW) bulk_row(stage, from_y + t_in * p.K, row_bytes, bar);
            bulk_row(stage + h_at, from_h + t_in * (p.K * hs), K * hs, bar);
            t_in += step;
        }
        if (++s_in == p.stages) s_in = 0;
    };
    auto refill = [&]() {
        if (SUM ? warp_id() == 0 : threadIdx.x == 0) {
            issue();
            if (SUM) look_up();
        }
    };
    if (SUM && warp_id() == 0) look_up();
    for (int s = 0; s < p.stages; ++s) refill();

    Cols<F32, FULL> cols;
    Unit wp, wx;
    cols.init(K);
    cols.get_weights(w_post, gate, wp);
    cols.get_weight(w_pre, wx);
    const f32x2 a2 = pair(p.res_scale, p.res_scale);
    const int code_pitch = static_cast<int>(act8_code_pitch(p.K)), scale_pitch = static_cast<int>(act8_scale_pitch(p.K));
    int stage = 0;
    uint32_t parity = 0, calls = 0;
    bool left = false;
    for (int64_t t = first; t < p.T; t += ROWS * step) {
        const int rows = ROWS == 1 || t + step < p.T ? ROWS : 1;
        float tg[ROWS];
        Unit y[ROWS], h[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (r >= rows) {  // the last row of an odd count: not stored twice
                tg[r] = 0.f;
                y[r] = y[0];
                h[r] = h[0];
                continue;
            }
            tg[r] = p.token_gate ? p.token_gate[t + r * step] : 1.f;
            if constexpr (SUM) {
#pragma unroll
                for (int k = 0; k < 8; ++k) y[r].v[k] = 0;
            }
            for (int g = 0; g < groups; ++g) {
                const uint8_t* at = ring + stage * p.stage_bytes;
                wait_row(&ctl->full[stage], parity, ctl, p.status, limit);
                account.waited();
                if constexpr (SUM) {
                    const int n = min(p.slots, p.topk - g * p.slots);
                    for (int j = 0; j < n; ++j) {
                        const Slot sl = ctl->slot[stage][j];
                        if (!sl.ok) continue;
                        const f32x2 w2 = pair(sl.w, sl.w);
                        Unit u;
                        cols.get_bf16(at + j * row_area, 0, u.v);
                        cols.get_bf16(at + j * row_area, 1, u.v + 4);
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[r].v[k] = fma2(w2, u.v[k], y[r].v[k]);
                    }
                }
                const bool last = g == groups - 1;
                if (last) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (SRC == SRC_ROW) cols.get_bf16(at, i, y[r].v + 4 * i);
                        cols.get_stream(at + h_at, i, h[r].v + 4 * i);
                    }
                }
                if (++stage == p.stages) {
                    stage = 0;
                    parity ^= 1u;
                }
                // a stage that the next row or group needs before the row sums' barrier
                if (!last || (ROWS == 2 && r == 0 && p.stages == 1)) {
                    __syncthreads();
                    if (!given_up(ctl)) refill();
                }
            }
        }
        float q[ROWS];
        if (SPLIT || (SRC != SRC_NONE && p.w_post)) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                f32x2 s2 = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) s2 = SRC != SRC_NONE ? fma2(y[r].v[k], y[r].v[k], s2) : s2;
                q[r] = both(s2);
            }
            left = row_sum<ROWS, SPLIT>(q, ctl, calls, p.status);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) q[r] = SPLIT && !p.w_post ? 1.f : rsqrtf(fmaf(q[r], inv_k, p.eps));
        } else {
            __syncthreads();
            left = given_up(ctl);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) q[r] = 1.f;
        }
        if (left) break;
        // every thread holds the rows in registers
        refill();
        if (ROWS == 2 && rows == 2 && p.stages > 1) refill();
        if constexpr (SRC != SRC_NONE) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                if (r >= rows) continue;
                const int64_t tr = t + r * step;
                uint8_t* to_h = static_cast<uint8_t*>(p.out_h) + col0 * hs + tr * (p.K * hs);
                if constexpr (KEEP == KEEP_BF16) {
                    cols.put_bf16(reinterpret_cast<uint8_t*>(p.out_y + col0) + tr * (2 * p.K), p.st32, y[r]);
                } else if constexpr (KEEP != KEEP_NONE) {
                    constexpr int FMT = KEEP == KEEP_INT8 ? GG_ACT8_INT8 : GG_ACT8_E4M3;
                    keep_unit<F32, FULL, FMT>(cols, y[r], p.codes + col0 + tr * code_pitch,
                                              p.scales + col0 / kActBlock + tr * scale_pitch,
                                              static_cast<int>(act8_code_pitch(K)));
                }
                const f32x2 q2 = pair(q[r] * tg[r], q[r] * tg[r]);
#pragma unroll
                for (int k = 0; k < 8; ++k) h[r].v[k] = fma2(mul2(y[r].v[k], wp.v[k]), q2, mul2(h[r].v[k], a2));
                cols.put_stream(to_h, p.st32, h[r]);
            }
        }
        if (!p.out_x) continue;
        float n[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            f32x2 s2 = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) s2 = fma2(h[r].v[k], h[r].v[k], s2);
            n[r] = both(s2);
        }
        // (not left here, which took rows of 9000 columns and more 1.5% longer: a row whose sums did
        // not come is stored from half of them, under a status that says so, and the next row leaves)
        (void)row_sum<ROWS, SPLIT>(n, ctl, calls, p.status);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (r >= rows) continue;
            const int64_t tr = t + r * step;
            const float f = rsqrtf(fmaf(n[r], inv_k, p.eps));
            const f32x2 f2 = pair(f, f);
            uint8_t* to_x = reinterpret_cast<uint8_t*>(p.out_x + col0) + tr * (2 * p.K);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[r].v[k] = mul2(h[r].v[k], mul2(f2, wx.v[k]));
            cols.put_bf16(to_x, p.st32, h[r]);
        }
    }
    if (left && threadIdx.x == 0) {
        drain_ring(ctl, p.stages, issued(), limit);
        account.drained();
    }
    account.put(p.probe, left, issued());
    if (SPLIT) leave_pair();
}

// One instantiation each: whole or half rows, rows that fill their threads (FULL), what is
// kept of y, the stream's type.  FULL rows without bounds: 16384 x 2048 fp32 with eight rows
// 133 us, 139 with bounds; 8192 x 4096 with two rows 58 and 61, one row 48.7 and 49.4, none (the
// stream alone) 22.4 and 24.1; 16384 x 512 12.2 and 13.1; only 8192 x 8192 is the same, 88.
struct Launch {
    bool split, full;
    unsigned rows;
    int threads;
    size_t smem;
    cudaStream_t st;
};
template <bool F32, int KEEP, int SRC>
int launch_fwd(const NormFwd& p, const Launch& l) {
    static std::atomic<uint64_t> done[3];
    if constexpr (SRC != SRC_FEW) {
        if (l.split) return launch(block_norm_kernel<F32, KEEP, true, false, SRC>, done[0], p, true, l.rows, l.threads, l.smem, l.st);
    }
    return l.full ? launch(block_norm_kernel<F32, KEEP, false, true, SRC>, done[1], p, false, l.rows, l.threads, l.smem, l.st)
                  : launch(block_norm_kernel<F32, KEEP, false, false, SRC>, done[2], p, false, l.rows, l.threads, l.smem, l.st);
}
template <bool F32, int SRC>
int launch_fwd(int keep, const NormFwd& p, const Launch& l) {
    switch (keep) {
        case KEEP_NONE: return launch_fwd<F32, KEEP_NONE, SRC>(p, l);
        case KEEP_BF16: return launch_fwd<F32, KEEP_BF16, SRC>(p, l);
        case KEEP_INT8: return launch_fwd<F32, KEEP_INT8, SRC>(p, l);
        default: return launch_fwd<F32, KEEP_E4M3, SRC>(p, l);
    }
}
template <bool F32>
int launch_fwd(int keep, const NormFwd& p, const Launch& l) {
    if (!p.Y) return launch_fwd<F32, KEEP_NONE, SRC_NONE>(p, l);
    if (p.topk == 1 && !p.map && !p.topk_w) return launch_fwd<F32, SRC_ROW>(keep, p, l);
    if (p.topk <= kFewRows && !l.split) return launch_fwd<F32, SRC_FEW>(keep, p, l);
    return launch_fwd<F32, SRC_SLOTS>(keep, p, l);
}
// The diagnostic form: sums of more rows, a bf16 stream.
int launch_probe(const NormFwd& p, const Launch& l) {
    static std::atomic<uint64_t> done[2];
    return l.split ? launch(block_norm_kernel<false, KEEP_NONE, true, false, SRC_SLOTS, true>, done[0], p, true, l.rows, l.threads, l.smem, l.st)
                   : launch(block_norm_kernel<false, KEEP_NONE, false, false, SRC_SLOTS, true>, done[1], p, false, l.rows, l.threads, l.smem, l.st);
}

int block_norm(const void* h, int h_dtype, const gg_bf16* Y, const int32_t* row_id_map, const float* topk_w, int topk,
               const float* w_post, const float* gate, const float* token_gate, float res_scale, const float* w_pre,
               float eps, int64_t T, int64_t K, void* out_h, gg_bf16* out_x, gg_bf16* out_y, uint8_t* y_codes,
               uint8_t* y_scales, int fmt, int32_t* status, void* stream, const Probe* probe) {
    if (T < 0 || K < 0 || topk < 1) return GG_ERR_INVALID_ARG;
    if (h_dtype != GG_DTYPE_BF16 && h_dtype != GG_DTYPE_F32) return GG_ERR_INVALID_ARG;
    if (fmt != GG_ACT8_INT8 && fmt != GG_ACT8_E4M3) return GG_ERR_INVALID_ARG;
    if (!(eps > 0.f && eps < INFINITY)) return GG_ERR_INVALID_ARG;
    if (K % 8 || K > GG_NORM_MAX_K || topk > GG_MAX_TOPK) return GG_ERR_UNSUPPORTED;
    if (T >= (int64_t(1) << 31) || T * topk >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
    if (!y_codes != !y_scales || (y_codes && out_y)) return GG_ERR_INVALID_ARG;
    if (!w_pre != !out_x) return GG_ERR_INVALID_ARG;
    if (!Y && (row_id_map || topk_w || topk > 1 || w_post || gate || token_gate || out_y || y_codes || !out_x))
        return GG_ERR_INVALID_ARG;
    if (T == 0 || K == 0) return GG_OK;
    if (!h || (Y && !out_h)) return GG_ERR_INVALID_ARG;
    const void* ptrs[] = {h, Y, w_post, gate, w_pre, out_h, out_x, out_y, y_codes};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return GG_ERR_UNSUPPORTED;
    const void* words[] = {y_scales, row_id_map, topk_w, token_gate};
    for (const void* q : words)
        if (!aligned(q, 4)) return GG_ERR_UNSUPPORTED;
    const bool f32 = h_dtype == GG_DTYPE_F32;
    const int64_t hb = T * K * (f32 ? 4 : 2), xb = T * K * 2, pitch = act8_code_pitch(K), spitch = act8_scale_pitch(K);
    {
        // out_h may be h itself; Y may then be h too, where its rows are the tokens'
        const int64_t row = hb / T, y_row = topk == 1 && !row_id_map ? 2 * K : 0;
        const Span outs[] = {{out_x, xb}, {out_y, xb}, {y_codes, T * pitch}, {y_scales, T * spitch}, {Y ? out_h : nullptr, hb, out_h == h ? row : 0}};
        const Span ins[] = {{h, hb, row}, {Y, xb * topk, y_row}, {w_post, K * 4}, {gate, K * 4}, {w_pre, K * 4}, {token_gate, T * 4},
                            {row_id_map, T * topk * 4}, {topk_w, T * topk * 4}};
        if (outputs_overlap(outs, ins)) return GG_ERR_INVALID_ARG;
    }
    NormFwd p{h, Y, row_id_map, topk_w, topk, w_post, gate, token_gate, w_pre, res_scale, eps, T,
              static_cast<int>(K), static_cast<int>(norm_half(K)), out_h, out_x, out_y, y_codes, y_scales, status, 0, 0, 1, 1,
              K % 16 == 0 && aligned(out_h, 32) && aligned(out_x, 32) && aligned(out_y, 32)};
    int per_sm = norm_per_sm(K);
    if (Y && (topk > 1 || row_id_map || topk_w) && topk <= kFewRows && !norm_split(K)) per_sm = per_sm * 3 / 2;
    // A stage holds as many of a token's expert rows (a lane each) as leave two stages to
    // every CTA of an SM: each group of rows ends in a barrier.  16384 x 2048 (fp32 stream)
    // with eight rows took 138 us with four a stage, 150 with two, 186 with all eight and
    // half the CTAs; 5255 x 5384 211 us with one a stage, 133 with five, 121 with all eight.
    // (Three stages with fewer rows each: 5-12% slower.)
    const int h_area = stream_area(f32, p.half);
    if (Y) {
        const int area = bf16_area(f32, p.half);
        for (p.slots = topk < kMaxSlots ? topk : kMaxSlots; p.slots > 1; --p.slots)
            if (ring_room(per_sm) >= kMinStages * (static_cast<int64_t>(p.slots) * area + h_area)) break;
        p.groups = (topk + p.slots - 1) / p.slots;
        p.slots = (topk + p.groups - 1) / p.groups;
        p.stage_bytes = p.slots * area + h_area;
    } else {
        p.stage_bytes = h_area;
    }
    p.stages = ring_stages(p.stage_bytes, per_sm);
    const int64_t most = norm_rows(K, per_sm);
    const int threads = norm_threads(K);
    const Launch l{norm_split(K), p.st32 && K == 16 * threads, static_cast<unsigned>(T < most ? T : most), threads,
                   sizeof(Ctl) + static_cast<size_t>(p.stages) * p.stage_bytes, static_cast<cudaStream_t>(stream)};
    if (probe) {
        p.probe = *probe;
        return launch_probe(p, l);
    }
    const int keep = out_y ? KEEP_BF16 : !y_codes ? KEEP_NONE : fmt == GG_ACT8_INT8 ? KEEP_INT8 : KEEP_E4M3;
    return f32 ? launch_fwd<true>(keep, p, l) : launch_fwd<false>(keep, p, l);
}

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

int gg_block_norm(const void* h, int h_dtype, const gg_bf16* Y, const int32_t* row_id_map, const float* topk_w,
                  int topk, const float* w_post, const float* gate, const float* token_gate, float res_scale,
                  const float* w_pre, float eps, int64_t T, int64_t K, void* out_h, gg_bf16* out_x, gg_bf16* out_y,
                  uint8_t* y_codes, uint8_t* y_scales, int fmt, int32_t* status, void* stream) {
    return block_norm(h, h_dtype, Y, row_id_map, topk_w, topk, w_post, gate, token_gate, res_scale, w_pre, eps, T, K, out_h,
                      out_x, out_y, y_codes, y_scales, fmt, status, stream, nullptr);
}

int gg_selftest_block_norm_wait(const gg_bf16* h, const gg_bf16* Y, int topk, const float* w, int64_t T, int64_t K,
                                int64_t withheld, gg_bf16* out_h, gg_bf16* out_x, int32_t* record, int32_t* status,
                                void* stream) {
    if (!Y || !w || !record || !status || withheld < 0 || withheld >= T || topk <= kFewRows) return GG_ERR_INVALID_ARG;
    if (!aligned(record, 4) || !aligned(status, 4)) return GG_ERR_UNSUPPORTED;
    Probe probe;
    probe.withheld = withheld;
    probe.record = record;
    return block_norm(h, GG_DTYPE_BF16, Y, nullptr, nullptr, topk, w, nullptr, nullptr, 1.f, w, 1e-6f, T, K, out_h, out_x,
                      nullptr, nullptr, nullptr, GG_ACT8_INT8, status, stream, &probe);
}

}  // extern "C"
