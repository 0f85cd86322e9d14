// lora_project.cu -- the shared projection with its adapters for few rows (decode,
// short prompts): Y = X W^T + U B[a]^T and dX = dY W + V A[a].  Longer batches take
// the 2-CTA tiles of lora_pair.cu.
//
// Bound by streaming W, which takes every SM: each 128 x 128 tile's reduction is
// split over a cluster whose CTAs' partial sums are joined in rank order through
// distributed shared memory (as in lora_shrink.cu).  Row slots hold the rows there
// are, so that few rows leave the shared memory to W's blocks in flight, and W's
// first blocks are asked for before anything else is read: the kernel may start
// while the low-rank product runs and waits for it only at the adapters' blocks.
//
// Rows stay in token order.  An adapter's part is added to the tile's accumulators
// by MMAs masked to its rows, rank_pad(r) reduction columns each; a ring stage
// holds as many adapters as fit.
//
// 1 row of 4096 -> 6144 at rank 16, with the low-rank product before it: 15.4-16.0 us (graph
// replay; 18-22 a call); W's 50 MB take 8 of them at 6.5 TB/s, the rest is the join and two
// launches.  48 rows with 32 adapters: 20.3 us.
#include "lora.cuh"

namespace gg {
namespace {

constexpr int kRM = 128;              // rows of a tile
constexpr int kRN = 128;              // columns of a tile
constexpr int kRK = 64;               // reduction block
constexpr int kRMaxStages = 6;
constexpr int kRThreads = 192;        // producer, issuer, four epilogue warps
constexpr int kRSlot = kRN * kRK * 2; // W's, or adapters', columns
constexpr int kRRing = 98304;         // two CTAs an SM

struct ProjectParams {
    PlanView plan;
    int Kred;            // shared reduction length
    int ncols;           // output columns
    int r;               // rank
    int rpad, epb;       // width of an adapter block, adapters a stage holds
    int mtiles;
    int xrows;           // rows of the X boxes (a multiple of 8, at most 128)
    int stages;
    uint16_t* out;
    uint32_t* ready;     // to release once U (V) can be read (or null)
    int32_t* status;
};

struct ProjectCtl {
    uint64_t full[kRMaxStages];
    uint64_t empty[kRMaxStages];
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
    int nent;                   // adapters that occur in this row tile
    int32_t gid[kRM];
    alignas(16) uint32_t mask[kRM][4];
};

constexpr int kProjectSmem = 1024 + kRRing + 4096;
static_assert(sizeof(ProjectCtl) <= 4096, "control block");
static_assert(kRRing >= kRM * kRN * 4, "partial sums fit the drained ring");

// B_MN: W and the adapters are read along their columns (dX).
template <bool B_MN>
__global__ void __launch_bounds__(kRThreads, 2)
project_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
               const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmE, const ProjectParams p,
               const int S) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    ProjectCtl* ctl = reinterpret_cast<ProjectCtl*>(ring + kRRing);
    volatile int* abort_flag = &ctl->abort_flag;
    const int warp = warp_index(), lane = lane_id();
    const int rank = static_cast<int>(cluster_ctarank());
    const int64_t item = blockIdx.x / S;
    // a column tile's row tiles are neighbours: they read the same W
    const int64_t mt = item % p.mtiles;
    const int n0 = static_cast<int>(item / p.mtiles) * kRN;
    const int64_t row0 = mt * kRM;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kRM), p.plan.T - row0));
    const int nb = (p.Kred + kRK - 1) / kRK;
    const int b_lo = static_cast<int>(static_cast<int64_t>(nb) * rank / S);  // at least one block: S <= nb
    const int b_hi = static_cast<int>(static_cast<int64_t>(nb) * (rank + 1) / S);
    const int nbase = b_hi - b_lo;
    const int a_slot = p.xrows * 128;
    const int stage_bytes = a_slot + kRSlot;
    const int stages = p.stages;

    // shared block i of this CTA into its stage
    auto load_base = [&](int i, int stage) {
        uint8_t* sA = ring + stage * stage_bytes;
        uint8_t* sB = sA + a_slot;
        uint64_t* bar = &ctl->full[stage];
        const int red = (b_lo + i) * kRK;
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(a_slot) + kRSlot);
        if (B_MN) {
            tma_load_2d(sB, &tmW, bar, n0, red);
            tma_load_2d(sB + kRSlot / 2, &tmW, bar, n0 + 64, red);
        } else {
            tma_load_2d(sB, &tmW, bar, red, n0);
        }
        tma_load_2d(sA, &tmX, bar, red, static_cast<int32_t>(row0));
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        mbar_init(&ctl->done, 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();  // the barriers, before TMA completes on them
        for (int i = 0; i < min(nbase, stages); ++i) load_base(i, i);
        tma_prefetch_desc(&tmU);
        tma_prefetch_desc(&tmE);
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, kRN);
        tmem_relinquish();
    }
    if (warp == 2) {
        // the unit's entries that have rows in this half of it, in order
        const int64_t u = mt >> 1;
        const int half = static_cast<int>(mt & 1) * 4;
        const int cnt = p.plan.cnt[u];
        int n = 0;
        for (int j0 = 0; j0 < cnt; j0 += 32) {
            const int j = j0 + lane;
            uint4 m = make_uint4(0, 0, 0, 0);
            if (j < cnt) m = *reinterpret_cast<const uint4*>(p.plan.mask + (u * p.plan.slots + j) * kUnitWords + half);
            const bool has = (m.x | m.y | m.z | m.w) != 0;
            const uint32_t b = __ballot_sync(0xffffffffu, has);
            if (has) {
                const int k = n + __popc(b & ((1u << lane) - 1u));  // below 128: each entry has a row of its own
                ctl->gid[k] = p.plan.gid[u * p.plan.slots + j];
                ctl->mask[k][0] = m.x;
                ctl->mask[k][1] = m.y;
                ctl->mask[k][2] = m.z;
                ctl->mask[k][3] = m.w;
            }
            n += __popc(b);
        }
        if (lane == 0) ctl->nent = n;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // this rank's share of the adapters' blocks, after its share of the shared ones
    const int ne = ctl->nent;
    const int rchunks = (p.r + 63) / 64;
    const int xb = p.r <= 64 ? (ne + p.epb - 1) / p.epb : ne * rchunks;
    const int x_lo = xb * rank / S, x_hi = xb * (rank + 1) / S;
    const int nblk = nbase + x_hi - x_lo;
    const uint32_t tmem = ctl->tmem_base;
    const uint32_t ring0 = smem_u32(ring);
    const uint32_t eb = 256u * p.rpad;  // bytes of an adapter's columns in a stage
    // the first adapter block's entry and rank columns; the next block's
    const int ef0 = p.r <= 64 ? x_lo * p.epb : x_lo / rchunks, rc0 = p.r <= 64 ? 0 : (x_lo % rchunks) * 64;
    auto next_block = [&](int& ef, int& rc) {
        if ((rc += 64) >= p.r) {
            rc = 0;
            ef += p.epb;
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------- producer --
        const bool elect = elect_one();
        int issued = min(nbase, stages);
        int stage = issued % stages;
        uint32_t phase = issued == stages ? 1u : 0u;
        int ef = ef0, rc = rc0;
        bool waited = false;
        for (int i = issued; i < nblk; ++i) {
            if (!all_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status)) break;
            if (i < nbase) {
                if (elect) load_base(i, stage);
            } else {
                if (!waited) {
                    pdl_wait();  // U (V) of the kernel before
                    waited = true;
                    release_ready(p.ready);
                    pdl_launch_dependents();  // (the next kernel may read it too)
                }
                uint8_t* sA = ring + stage * stage_bytes;
                uint8_t* sB = sA + a_slot;
                uint64_t* bar = &ctl->full[stage];
                const int en = min(p.epb, ne - ef);
                if (elect) {
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.xrows) * p.rpad * 2u + eb * en);
                    tma_load_2d(sA, &tmU, bar, rc, static_cast<int32_t>(row0));
                    for (int e = 0; e < en; ++e) {
                        const int g = ctl->gid[ef + e];
                        if (B_MN) {
                            tma_load_3d(sB + e * eb, &tmE, bar, n0, rc, g);
                            tma_load_3d(sB + e * eb + eb / 2, &tmE, bar, n0 + 64, rc, g);
                        } else {
                            tma_load_3d(sB + e * eb, &tmE, bar, rc, n0, g);
                        }
                    }
                }
                next_block(ef, rc);
            }
            ++issued;
            if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        if (!waited) {
            pdl_wait();  // the launch before this one has finished before this grid can
            release_ready(p.ready);
            pdl_launch_dependents();
        }
        // every copy has landed before the ring is reused or the CTA exits
        for (int j = 0; j < min(issued, stages); ++j) {
            if (--stage < 0) { stage = stages - 1; phase ^= 1u; }
            int dummy = 0;
            mbar_wait(&ctl->full[stage], phase, reinterpret_cast<volatile int*>(&dummy), p.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------- MMA issuer --
        const bool elect = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        bool any_mma = false;
        constexpr uint32_t idesc = idesc_bf16_f32(kRM, kRN, 0, B_MN ? 1 : 0);
        const Desc dX(smem_desc(ring0, 16, 1024, kLayoutSw128));
        const Desc dW(B_MN ? smem_desc(ring0 + a_slot, kRSlot / 2, 1024, kLayoutSw128)
                           : smem_desc(ring0 + a_slot, 16, 1024, kLayoutSw128));
        const Desc dU(kmajor_desc(ring0, p.rpad * 2));
        const Desc dE(B_MN ? smem_desc(ring0 + a_slot, eb / 2, 1024, kLayoutSw128) : kmajor_desc(ring0 + a_slot, p.rpad * 2));
        constexpr uint32_t kStep = B_MN ? 128 : 2;  // 16 reduction columns of the right operand
        int ef = ef0, rc = rc0;
        for (int i = 0; i < nblk; ++i) {
            if (!all_wait(&ctl->full[stage], phase, abort_flag, p.status)) break;
            tc_fence_after();
            const uint32_t at = stage * (stage_bytes / 16);
            if (i < nbase) {
                if (elect) {
#pragma unroll
                    for (int ks = 0; ks < kRK / 16; ++ks)
                        umma_at<false>(tmem, dX, at + 2 * ks, dW, at + kStep * ks, idesc, (i > 0 || ks > 0) ? 1u : 0u);
                }
            } else {
                const int en = min(p.epb, ne - ef);
                const int steps = (min(64, p.r - rc) + 15) / 16;
                if (elect) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (e >= en) break;
                        const uint4 m = *reinterpret_cast<const uint4*>(&ctl->mask[ef + e][0]);
                        const uint32_t keep[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (ks < steps)
                                umma_rows_at(tmem, dU, at + 2 * ks, dE, at + e * (eb / 16) + kStep * ks, idesc, keep);
                    }
                }
                next_block(ef, rc);
            }
            if (elect) umma_commit(&ctl->empty[stage]);
            any_mma = true;
            if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        if (elect) {
            if (any_mma) umma_commit(&ctl->done);
            else mbar_arrive(&ctl->done);
        }
        __syncwarp();
    }

    // -------------------------------------------- partial sums to the cluster --
    const bool good = warp_wait(&ctl->done, 0, abort_flag, p.status);
    tc_fence_after();
    __syncthreads();  // the copies have landed, the MMAs have completed: the ring is free
    float* part = reinterpret_cast<float*>(ring);
    const int q = warp & 3;
    const int row = q * 32 + lane;
    // 4-column pieces of a row are rotated by the row, against bank conflicts
    if (warp >= 2 && q * 32 < rows) {
#pragma unroll 1
        for (int c = 0; c < kRN; c += 32) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, v);
            tmem_ld_wait();
            if (row < rows) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4*>(part + row * kRN + (((c / 4 + k) ^ (row & 31)) << 2)) =
                        make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (good) {
        // a warp sums and stores one row's 128 columns at a time
        for (int i = rank * kRThreads + threadIdx.x; i < rows * (kRN / 4); i += S * kRThreads) {
            const int rr = i / (kRN / 4), g = i % (kRN / 4);
            const int col = n0 + g * 4;
            if (col >= p.ncols) continue;
            const float4 s = cluster_sum4(smem_u32(part + rr * kRN + ((g ^ (rr & 31)) << 2)), S);
            *reinterpret_cast<uint2*>(p.out + (row0 + rr) * p.ncols + col) = pack_bf16x4(s);
        }
    }
    __syncthreads();
    cluster_sync();  // no CTA leaves while another may still read its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kRN);
    }
}

template <bool B_MN>
int launch_project(const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& u, const CUtensorMap& e,
                   const ProjectParams& p, cudaStream_t st) {
    static ClusterRoom rooms;
    int room[kMaxCluster + 1];
    const int rc = rooms.get(project_kernel<B_MN>, kProjectSmem, room);
    if (rc != GG_OK) return rc;
    // The widest split whose clusters are resident at once with an eighth to spare: the
    // low-rank product may still hold some SMs, and a cluster that starts late runs
    // alone (300 rows of 4096 x 4096: 29 us at 96 of 97 clusters of 3, 25 in clusters of 2).
    const int64_t nb = (p.Kred + kRK - 1) / kRK;
    const int64_t tiles = static_cast<int64_t>(p.mtiles) * ((p.ncols + kRN - 1) / kRN);
    int S = kMaxCluster;
    while (S > 1 && (tiles * 8 > room[S] * 7 || S > nb)) --S;
    if (tiles * S >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
    ClusterLaunch l(tiles * S, kRThreads, kProjectSmem, S, true, st);
    clear_pending_launch_error();
    const cudaError_t err = cudaLaunchKernelEx(&l.cfg, project_kernel<B_MN>, x, w, u, e, p, S);
    if (err != cudaSuccess) { record_cuda_error(err); return GG_ERR_CUDA; }
    return launch_result();
}

}  // namespace

int lora_project_launch(bool b_mn, const uint16_t* X, const uint16_t* W, const uint16_t* U, const uint16_t* ad,
                        const PlanView& plan, int64_t Kred, int64_t ncols, int r, uint16_t* out, uint32_t* ready,
                        int32_t* status, cudaStream_t st) {
    ProjectParams p{};
    p.plan = plan;
    p.Kred = static_cast<int>(Kred);
    p.ncols = static_cast<int>(ncols);
    p.r = r;
    p.rpad = rank_pad(r);
    p.epb = 64 / p.rpad;
    p.mtiles = static_cast<int>((plan.T + kRM - 1) / kRM);
    p.xrows = plan.T >= kRM ? kRM : static_cast<int>((plan.T + 7) / 8 * 8);
    // (the MMA reads 128 rows from every row slot: what follows it stays in the ring,
    // the last stage's column slot being as large)
    p.stages = kRRing / (p.xrows * 128 + kRSlot);
    if (p.stages > kRMaxStages) p.stages = kRMaxStages;
    p.out = out;
    p.ready = ready;
    p.status = status;
    CUtensorMap mX{}, mW{}, mU{}, mE{};
    if (!encode_map_2d(&mX, X, Kred, plan.T, Kred, kRK, p.xrows)) return GG_ERR_CUDA;
    if (!encode_map_2d(&mU, U, r, plan.T, r, p.rpad, p.xrows)) return GG_ERR_CUDA;
    if (b_mn) {  // W [Kred, ncols], ad [L, r, ncols]
        if (!encode_map_2d(&mW, W, ncols, Kred, ncols, 64, kRK)) return GG_ERR_CUDA;
        if (!encode_map_3d(&mE, ad, ncols, r, plan.L, ncols, ncols * r, 64, p.rpad)) return GG_ERR_CUDA;
        return launch_project<true>(mX, mW, mU, mE, p, st);
    }
    if (!encode_map_2d(&mW, W, Kred, ncols, Kred, kRK, kRN)) return GG_ERR_CUDA;
    if (!encode_map_3d(&mE, ad, r, ncols, plan.L, r, ncols * r, p.rpad, kRN)) return GG_ERR_CUDA;
    return launch_project<false>(mX, mW, mU, mE, p, st);
}

}  // namespace gg
