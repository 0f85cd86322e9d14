// lora_grad.cu -- gradients of the adapters, a ragged reduction over each
// adapter's tokens:
//   dA[a] = sum_{t: ids[t] = a} V[t]^T X[t]    [r, K]
//   dB[a] = sum_{t: ids[t] = a} dY[t]^T U[t]   [N, r]
// Both are one problem: a wide source (X, dY) read along its columns against a
// narrow one (V, U), for a 128-column chunk of the wide source and one adapter.
// Bound by reading X and dY once; the MMAs run with the wide columns as M and the
// rank as N.
//
// The rows are the plan's tiles, in blocks of 64 rows of one adapter.  A block whose
// rows are neighbours in memory (a sequence's) is copied by TMA; any other (ids
// in no order, the adapter's last rows) is gathered row by row with cp.async, rows
// past the end as zeros, so nothing of another adapter's rows enters the sums.
// Blocks are split over a cluster and the partial sums joined as in lora_shrink.cu.
#include "lora.cuh"

namespace gg {
namespace {

constexpr int kGM = 128;            // columns of the wide source
constexpr int kGK = 64;             // rows of a block
constexpr int kGThreads = 192;      // producer, issuer, four gather / epilogue warps
constexpr int kGWide = kGM * kGK * 2;
constexpr int kGMaxStages = 6;
// the partial sums fit the drained ring
static_assert(73728 >= 4 * kGM * (32 + 4) && 73728 >= 4 * 32 * (kGM + 4), "ring");
static_assert(98304 >= 4 * kGM * (64 + 4) && 98304 >= 4 * 64 * (kGM + 4), "ring");
static_assert(196608 >= 4 * kGM * (kLoraMaxRank + 4) && 196608 >= 4 * kLoraMaxRank * (kGM + 4), "ring");


struct GradSide {
    const uint16_t* wide;      // [T, cols]
    const uint16_t* narrow[2]; // [T, r]: the operand and its rounding's remainder
    int parts;                 // 1 or 2 of them
    int cols;
    int tiles;                 // 128-column chunks
    uint16_t* out;
};

struct GradParams {
    PlanView plan;
    GradSide side[2];          // dA, dB
    int r, chunk, nc;          // rank; width (16, 32, 64) and number of its pieces
    int stages;
    int stage_bytes;
    int32_t* status;
};

struct GradCtl {
    uint64_t full[kGMaxStages];
    uint64_t empty[kGMaxStages];
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
};

struct GradMaps {
    CUtensorMap wide[2];
    CUtensorMap narrow[3];     // V, V's remainder, U
};

// RING: bytes of the operand ring; CTAS: resident on an SM
template <int RING, int CTAS>
__global__ void __launch_bounds__(kGThreads, CTAS)
grad_kernel(const __grid_constant__ GradMaps maps, const GradParams p, const int S) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    __shared__ GradCtl ctl_s;
    GradCtl* ctl = &ctl_s;
    volatile int* abort_flag = &ctl->abort_flag;
    const int warp = warp_id(), lane = lane_id();
    const int rank = static_cast<int>(cluster_ctarank());
    const int64_t item = blockIdx.x / S;
    const int tiles = p.side[0].tiles + p.side[1].tiles;
    const int a = static_cast<int>(item / tiles);
    const int tile = static_cast<int>(item % tiles);
    const int sd = tile < p.side[0].tiles ? 0 : 1;
    const GradSide side = p.side[sd];
    const int col0 = (sd == 0 ? tile : tile - p.side[0].tiles) * kGM;
    const int ncols = p.chunk * p.nc;  // accumulator columns
    const uint32_t piece_bytes = static_cast<uint32_t>(p.chunk) * kGK * 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&ctl->full[s], 1 + 128);  // the producer, every gather thread
            mbar_init(&ctl->empty[s], 1);
        }
        mbar_init(&ctl->done, 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.wide[sd]);
    }
    const int tcols = ncols <= 32 ? 32 : (ncols <= 64 ? 64 : (ncols <= 128 ? 128 : 256));
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, tcols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int count = p.plan.goff[a + 1] - p.plan.goff[a];
    const int4* tiles_a = p.plan.tile + p.plan.toff[a];
    const int nb = (count + kGK - 1) / kGK;
    const int act = min(S, nb);  // ranks with blocks
    const int lo = rank < act ? static_cast<int>(static_cast<int64_t>(nb) * rank / act) : 0;
    const int hi = rank < act ? static_cast<int>(static_cast<int64_t>(nb) * (rank + 1) / act) : 0;
    const uint32_t tmem = ctl->tmem_base;
    const uint32_t ring0 = smem_u32(ring);
    const int nnarrow = p.nc * side.parts;
    // Block b is half b & 1 of tile b / 2.  Each role walks the tiles with the next
    // one's entry already loaded.
    static_assert(kTileRows == 2 * kGK, "two blocks a tile");
    int4 cur = make_int4(0, 0, 0, 0), next = cur;
    if (hi > lo) {
        cur = tiles_a[lo / 2];
        if (lo / 2 < (hi - 1) / 2) next = tiles_a[lo / 2 + 1];
    }
    auto advance = [&](int b) {  // to block b + 1
        if ((b & 1) && b + 1 < hi) {
            cur = next;
            if ((b + 1) / 2 < (hi - 1) / 2) next = tiles_a[(b + 1) / 2 + 1];
        }
    };
    auto by_tma = [&](int b) { return cur.w >= 0 && cur.z >= ((b & 1) + 1) * kGK; };

    if (warp == 0) {
        // --------------------------------------------------- TMA producer --
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int b = lo; b < hi; ++b) {
                if (!mbar_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status)) break;
                uint64_t* bar = &ctl->full[stage];
                if (by_tma(b)) {
                    uint8_t* s = ring + stage * p.stage_bytes;
                    const int32_t t = cur.w + (b & 1) * kGK;
                    mbar_arrive_expect_tx(bar, kGWide + piece_bytes * nnarrow);
                    tma_load_2d(s, &maps.wide[sd], bar, col0, t);
                    tma_load_2d(s + kGWide / 2, &maps.wide[sd], bar, col0 + 64, t);
                    for (int k = 0; k < nnarrow; ++k)
                        tma_load_2d(s + kGWide + k * piece_bytes, &maps.narrow[sd == 0 ? k / p.nc : 2], bar,
                                    (k % p.nc) * p.chunk, t);
                } else {
                    mbar_arrive(bar);
                }
                advance(b);
                ++issued;
                if (++stage == p.stages) { stage = 0; phase ^= 1u; }
            }
            // every copy has landed before the ring is reused or the CTA exits
            for (int j = 0; j < min(issued, p.stages); ++j) {
                if (--stage < 0) { stage = p.stages - 1; phase ^= 1u; }
                int dummy = 0;
                mbar_wait(&ctl->full[stage], phase, reinterpret_cast<volatile int*>(&dummy), p.status);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------- MMA issuer --
        if (lane == 0 && hi > lo) {
            const uint32_t idesc = idesc_bf16_f32_n(kGM, ncols, 1, 1);
            int stage = 0;
            uint32_t phase = 0;
            bool any_mma = false;
            for (int b = lo; b < hi; ++b) {
                if (!mbar_wait(&ctl->full[stage], phase, abort_flag, p.status)) break;
                tc_fence_after();
                fence_proxy_async_smem();  // gathered rows are generic-proxy writes
                const uint32_t s = ring0 + stage * p.stage_bytes;
                for (int part = 0; part < side.parts; ++part) {
                    const uint32_t sN = s + kGWide + part * p.nc * piece_bytes;
#pragma unroll
                    for (int ks = 0; ks < kGK / 16; ++ks)
                        umma_bf16(tmem, smem_desc(s + ks * 2048, kGWide / 2, 1024, kLayoutSw128),
                                  mnmajor_desc(sN + ks * 32 * p.chunk, 2 * p.chunk, piece_bytes), idesc,
                                  (b > lo || part > 0 || ks > 0) ? 1u : 0u);
                }
                umma_commit(&ctl->empty[stage]);
                any_mma = true;
                if (++stage == p.stages) { stage = 0; phase ^= 1u; }
            }
            if (any_mma) umma_commit(&ctl->done);
            else mbar_arrive(&ctl->done);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- row gathers --
        const int gt = threadIdx.x - 64;  // 0 .. 127
        int stage = 0;
        uint32_t phase = 0;
        for (int b = lo; b < hi; ++b) {
            if (!warp_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status, 32)) break;
            if (by_tma(b)) {
                mbar_arrive(&ctl->full[stage]);
            } else {
                const uint32_t s = ring0 + stage * p.stage_bytes;
                const int off = (b & 1) * kGK, valid = cur.z - off;
                auto token = [&](int rr) {  // of the block's row rr
                    return rr >= valid ? -1 : (cur.w >= 0 ? cur.w + off + rr : p.plan.order[cur.y + off + rr]);
                };
                // 16 pieces of 8 columns a row of the wide source, 8 rows a step
                const int pc = gt & 15;
                const bool in = col0 + pc * 8 < side.cols;
                int32_t tok[kGK / 8];
#pragma unroll
                for (int j = 0; j < kGK / 8; ++j) tok[j] = token((gt >> 4) + 8 * j);
#pragma unroll
                for (int j = 0; j < kGK / 8; ++j) {
                    const int rr = (gt >> 4) + 8 * j;
                    const bool v = in && tok[j] >= 0;
                    cp_async_16(s + (pc >> 3) * (kGWide / 2) + rr * 128 + (((pc & 7) ^ (rr & 7)) << 4),
                                v ? side.wide + static_cast<int64_t>(tok[j]) * side.cols + col0 + pc * 8 : side.wide,
                                v ? 16u : 0u);
                }
                // narrow: chunk / 8 pieces a row, swizzled over the row's width as TMA does
                // (16-byte piece index XOR address bits 7 and up)
                const int npc = p.chunk / 8;
                const int np = gt % npc, rows_a_step = 128 / npc;
                for (int rr = gt / npc; rr < kGK; rr += rows_a_step) {
                    const int32_t t = token(rr);
                    const uint32_t flip = static_cast<uint32_t>((rr * p.chunk * 2) >> 7) & (npc - 1);
                    for (int k = 0; k < nnarrow; ++k) {
                        const int c = (k % p.nc) * p.chunk + np * 8;
                        const uint16_t* src = side.narrow[k / p.nc];
                        const bool v = t >= 0 && c < p.r;
                        cp_async_16(s + kGWide + k * piece_bytes + rr * p.chunk * 2 + ((np ^ flip) << 4),
                                    v ? src + static_cast<int64_t>(t) * p.r + c : src, v ? 16u : 0u);
                    }
                }
                cp_async_mbar_arrive(&ctl->full[stage]);
            }
            advance(b);
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
        cp_async_wait<0>();
    }

    // -------------------------------------------- partial sums to the cluster --
    bool good = true;
    if (hi > lo) good = warp_wait(&ctl->done, 0, abort_flag, p.status);
    tc_fence_after();
    __syncthreads();
    float* part = reinterpret_cast<float*>(ring);
    // dA is stored along the wide columns (pitch kGM), dB along the rank
    const int pitch = sd == 0 ? kGM + 4 : p.r + 4;
    if (warp >= 2 && hi > lo) {
        const int q = warp & 3, row = q * 32 + lane;
        for (int c = 0; c < p.r; c += 8) {
            uint32_t v[8];
            tmem_ld_32x32b_x8(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, v);
            tmem_ld_wait();
            if (sd == 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k) part[(c + k) * pitch + row] = __uint_as_float(v[k]);
            } else {
                *reinterpret_cast<uint4*>(part + row * pitch + c) = make_uint4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<uint4*>(part + row * pitch + c + 4) = make_uint4(v[4], v[5], v[6], v[7]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (good) {
        const int wide = min(kGM, side.cols - col0);
        if (sd == 0) {
            const int quads = wide / 4;
            for (int i = rank * kGThreads + threadIdx.x; i < p.r * quads; i += S * kGThreads) {
                const int c = i / quads, k = (i % quads) * 4;
                *reinterpret_cast<uint2*>(side.out + (static_cast<int64_t>(a) * p.r + c) * side.cols + col0 + k) =
                    pack_bf16x4(cluster_sum4(smem_u32(part + c * pitch + k), act));
            }
        } else {
            const int quads = p.r / 4;
            for (int i = rank * kGThreads + threadIdx.x; i < wide * quads; i += S * kGThreads) {
                const int n = i / quads, c = (i % quads) * 4;
                *reinterpret_cast<uint2*>(side.out + (static_cast<int64_t>(a) * side.cols + col0 + n) * p.r + c) =
                    pack_bf16x4(cluster_sum4(smem_u32(part + n * pitch + c), act));
            }
        }
    }
    __syncthreads();
    cluster_sync();  // no CTA leaves while another may still read its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, tcols);
    }
}

template <int RING, int CTAS>
int launch_grad(const GradMaps& m, GradParams p, cudaStream_t st) {
    constexpr size_t smem = 1024 + RING;
    static ClusterRoom rooms;
    int room[kMaxCluster + 1];
    const int rc = rooms.get(grad_kernel<RING, CTAS>, smem, room);
    if (rc != GG_OK) return rc;
    p.stages = RING / p.stage_bytes;
    if (p.stages > kGMaxStages) p.stages = kGMaxStages;
    // The split: until the CTAs fill the GPU twice, at least two blocks of a mean
    // adapter each.
    const int64_t items = static_cast<int64_t>(p.plan.L) * (p.side[0].tiles + p.side[1].tiles);
    const int64_t blocks = p.plan.T / kGK / p.plan.L;
    int S = kMaxCluster;
    while (S > 1 && (items > 2 * room[S] || S * 2 > blocks)) S /= 2;
    if (items * S >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
    ClusterLaunch l(items * S, kGThreads, smem, S, false, st);
    clear_pending_launch_error();
    const cudaError_t err = cudaLaunchKernelEx(&l.cfg, grad_kernel<RING, CTAS>, m, p, S);
    if (err != cudaSuccess) { record_cuda_error(err); return GG_ERR_CUDA; }
    return launch_result();
}

}  // namespace

int lora_grad_launch(const uint16_t* X, const uint16_t* dY, const uint16_t* U, const uint16_t* V, const uint16_t* V_lo,
                     const PlanView& plan, int64_t K, int64_t N, int r, uint16_t* dA, uint16_t* dB, int32_t* status,
                     cudaStream_t st) {
    GradParams p{};
    p.plan = plan;
    p.r = r;
    p.chunk = rank_pad(r);
    p.nc = (r + p.chunk - 1) / p.chunk;
    p.status = status;
    if (dA)
        p.side[0] = GradSide{X, {V, V_lo}, 2, static_cast<int>(K), static_cast<int>((K + kGM - 1) / kGM), dA};
    if (dB)
        p.side[1] = GradSide{dY, {U, nullptr}, 1, static_cast<int>(N), static_cast<int>((N + kGM - 1) / kGM), dB};
    p.stage_bytes = kGWide + p.chunk * kGK * 2 * p.nc * (dA ? 2 : 1);
    GradMaps m{};
    if (dA) {
        if (!encode_map_2d(&m.wide[0], X, K, plan.T, K, 64, kGK)) return GG_ERR_CUDA;
        if (!encode_map_2d(&m.narrow[0], V, r, plan.T, r, p.chunk, kGK)) return GG_ERR_CUDA;
        if (!encode_map_2d(&m.narrow[1], V_lo, r, plan.T, r, p.chunk, kGK)) return GG_ERR_CUDA;
    }
    if (dB) {
        if (!encode_map_2d(&m.wide[1], dY, N, plan.T, N, 64, kGK)) return GG_ERR_CUDA;
        if (!encode_map_2d(&m.narrow[2], U, r, plan.T, r, p.chunk, kGK)) return GG_ERR_CUDA;
    }
    // rings of at least three stages while two CTAs fit an SM (ranks up to 64), three
    // CTAs for ranks up to 32
    if (p.chunk <= 32) return launch_grad<73728, 3>(m, p, st);
    return p.nc == 1 ? launch_grad<98304, 2>(m, p, st) : launch_grad<196608, 1>(m, p, st);
}

}  // namespace gg
