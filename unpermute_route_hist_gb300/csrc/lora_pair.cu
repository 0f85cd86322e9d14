// lora_pair.cu -- the shared projection with its adapters for batches of many
// rows: Y = X W^T + U B[a]^T and dX = dY W + V A[a], persistent 2-CTA tiles of
// 256 x 256 (cta_group::2 tcgen05 MMAs, accumulators double-buffered in tensor
// memory, TMA-fed six-stage ring).
//
// Rows stay in token order: the shared product is one dense GEMM, bound by the
// tensor rate.  A tile's last ring blocks are its adapters': for each adapter that
// occurs among the tile's 256 rows one block of rank_pad(r) reduction columns (U's
// rows against B[a]'s) is accumulated into those rows' lanes alone.  A batch of
// sequences has one or two adapters a tile, so that adds 1-2 blocks to K / 64.
// Sorting rows by adapter instead would read and write X and Y once more, or
// gather X (2.5x slower loads here), and break tiles at every adapter's end.
//
// A shared block costs 517-525 SM cycles and an adapter block of rank 64 523 (one round of 76
// tiles, by the kernel's cycles at 32, 64 and 128 blocks and at 1 to 33 adapters; the MMAs'
// own time is 512): an adapter's id and row masks wait in shared memory, copied while the
// shared blocks run (read from global memory a block ahead: 512 mixed rows of 32 adapters of
// rank 128 took 63 us instead of 46).
//
// 8192 rows of 4096 -> 6144 at rank 32, with the low-rank product before it: 231-239 us by box
// (graph replay), 1.75-1.81 PFLOP/s, 262-270 us a call at the power cap; the tensor pipe is
// active 88% of this kernel's time.
//
// Warp 0: TMA producer; warp 1: tensor memory and, in the even CTA, MMA issue;
// warps 2-5: epilogue (tensor memory -> bf16 -> 32-byte row pieces).  Every wait
// is bounded (GG_DEV_TIMEOUT).
#include "lora.cuh"

namespace gg {
namespace {

constexpr int kPM = 128, kPN = 256, kPK = 64;
constexpr int kPStages = 6;
constexpr int kPThreads = 192;
constexpr int kPSlot = 128 * kPK * 2;  // A rows, or the CTA's half of the B columns
constexpr int kPStage = 2 * kPSlot;
constexpr int kPGroup = 8;             // 256-row units of a raster group

struct PairParams {
    PlanView plan;
    int Kred, ncols, r, rpad, epb;
    int ntiles;        // column tiles
    int64_t whole;     // tiles done whole; the rest are cut into column pieces
    int cuts;          // pieces of those: 1 or 2
    int64_t items;     // tiles and pieces
    uint16_t* out;
    uint32_t* ready;   // to release once U (V) can be read (or null)
    int st32;          // output rows start 32-byte aligned
    int32_t* status;
};

struct PairCtl {
    uint64_t full[kPStages];
    uint64_t empty[kPStages];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    alignas(16) uint32_t mask[kUnit][kUnitWords];  // the issuer's tile: rows of each entry
    int32_t gid[kUnit];                            // the producer's tile: its adapters
};
constexpr int kPairSmem = 1024 + kPStages * kPStage + sizeof(PairCtl);

// Item t: groups of kPGroup units sweep every column tile, rows fastest, so the tiles
// in flight share W's columns and X's rows in L2.  The tiles of the last round, when
// they are few, are cut into column pieces that more clusters share.
struct PairTile {
    int64_t unit;
    int n0, width;
};
__device__ __forceinline__ PairTile pair_tile(int64_t t, const PairParams& p) {
    int piece = 0, width = kPN;
    if (t >= p.whole) {
        width = kPN / p.cuts;
        piece = static_cast<int>((t - p.whole) % p.cuts);
        t = p.whole + (t - p.whole) / p.cuts;
    }
    const int64_t per = static_cast<int64_t>(kPGroup) * p.ntiles;
    const int64_t group = t / per, first = group * kPGroup;
    const int64_t left = p.plan.units - first;
    const int h = static_cast<int>(left < kPGroup ? left : kPGroup);
    const int loc = static_cast<int>(t - group * per);
    return {first + loc % h, (loc / h) * kPN + piece * width, width};
}

template <bool B_MN>
__global__ void __launch_bounds__(kPThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
            const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmE,
            const __grid_constant__ CUtensorMap tmWp, const __grid_constant__ CUtensorMap tmEp, const PairParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    PairCtl* ctl = reinterpret_cast<PairCtl*>(ring + kPStages * kPStage);
    volatile int* abort_flag = &ctl->abort_flag;
    const int warp = warp_index(), lane = lane_id();
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int64_t slot = cluster_id_x(), nslot = nclusters_x();

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPStages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tmem_full[b], 1);
            mbar_init(&ctl->tmem_empty[b], 8);  // the epilogue warps of both CTAs
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmU);
        tma_prefetch_desc(&tmE);
    }
    if (warp == 1) {
        tmem_alloc_pair(&ctl->tmem_base, 2 * kPN);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const uint32_t ring0 = smem_u32(ring);
    const int nb = (p.Kred + kPK - 1) / kPK;
    const int rchunks = (p.r + 63) / 64;
    // adapter blocks of a unit with ne entries
    auto ext_blocks = [&](int ne) { return p.r <= 64 ? (ne + p.epb - 1) / p.epb : ne * rchunks; };

    if (warp == 0) {
        // ------------------------------------------------------- producer --
        {
            const bool elect = elect_one();
            int stage = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            bool ok = true, waited = false;
            const uint32_t eb = 256u * p.rpad;  // bytes of an adapter's columns, and of the rows' U
            for (int64_t t = slot; t < p.items && ok; t += nslot) {
                const PairTile ti = pair_tile(t, p);
                if (ti.n0 >= p.ncols) continue;  // a piece past the last column
                const int32_t arow = static_cast<int32_t>(ti.unit * kUnit + rank * kPM);
                const int half = ti.width / 2;  // columns of one CTA
                const int32_t nh = ti.n0 + static_cast<int32_t>(rank) * half;
                const bool whole = ti.width == kPN;
                const CUtensorMap* mW = whole ? &tmW : &tmWp;
                const CUtensorMap* mE = whole ? &tmE : &tmEp;
                const int ne = p.plan.cnt[ti.unit];
                const int32_t* gid = p.plan.gid + ti.unit * p.plan.slots;
                const int fetch_at = min(nb, kPStages) - 1;  // with the ring full of loads
                for (int i = 0; i < nb; ++i) {
                    if (!all_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    uint8_t* sA = ring + stage * kPStage;
                    uint8_t* sB = sA + kPSlot;
                    const uint32_t bar = mapa_u32(&ctl->full[stage], 0);
                    const int32_t red = i * kPK;
                    if (elect) {
                        if (leader) mbar_arrive_expect_tx(&ctl->full[stage], 2u * (kPSlot + half * kPK * 2));
                        tma_load_2d_pair(sA, &tmX, bar, red, arow);
                        if (B_MN) {
                            tma_load_2d_pair(sB, mW, bar, nh, red);
                            if (whole) tma_load_2d_pair(sB + 8192, mW, bar, nh + 64, red);
                        } else {
                            tma_load_2d_pair(sB, mW, bar, red, nh);
                        }
                    }
                    if (i == fetch_at) {
                        for (int e = lane; e < ne; e += 32)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&ctl->gid[e])), "l"(gid + e) : "memory");
                        cp_async_commit();
                    }
                    ++issued;
                    if (++stage == kPStages) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                const int xb = ext_blocks(ne);
                cp_async_wait<0>();
                __syncwarp();
                int ef = 0, rc = 0;  // first entry of the block, its rank columns
                for (int xi = 0; xi < xb; ++xi) {
                    const int en = min(p.epb, ne - ef);
                    if (!all_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    if (!waited) {
                        pdl_wait();  // U (V) of the kernel before
                        waited = true;
                        release_ready(p.ready);
                        pdl_launch_dependents();  // (the next kernel may read it too)
                    }
                    uint8_t* sA = ring + stage * kPStage;
                    uint8_t* sB = sA + kPSlot;
                    const uint32_t bar = mapa_u32(&ctl->full[stage], 0);
                    if (elect) {
                        if (leader) mbar_arrive_expect_tx(&ctl->full[stage], 2u * (eb + half * p.rpad * 2 * en));
                        tma_load_2d_pair(sA, &tmU, bar, rc, arow);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (e >= en) break;
                            if (B_MN) {
                                tma_load_3d_pair(sB + e * eb, mE, bar, nh, rc, ctl->gid[ef + e]);
                                if (whole) tma_load_3d_pair(sB + e * eb + eb / 2, mE, bar, nh + 64, rc, ctl->gid[ef + e]);
                            } else {
                                tma_load_3d_pair(sB + e * eb, mE, bar, rc, nh, ctl->gid[ef + e]);
                            }
                        }
                    }
                    if ((rc += 64) >= p.r) {
                        rc = 0;
                        ef += p.epb;
                    }
                    ++issued;
                    if (++stage == kPStages) { stage = 0; phase ^= 1u; }
                }
                __syncwarp();  // every lane has read its ids before the next tile's arrive
            }
            if (!waited) {
                pdl_wait();  // the launch before this one has finished before this grid can
                release_ready(p.ready);
                pdl_launch_dependents();
            }
            // The even CTA's barriers count both CTAs' copies: let them land.
            if (leader) {
                const int64_t pend = issued < kPStages ? issued : kPStages;
                for (int64_t j = 0; j < pend; ++j) {
                    if (--stage < 0) { stage = kPStages - 1; phase ^= 1u; }
                    int dummy = 0;
                    mbar_wait(&ctl->full[stage], phase, reinterpret_cast<volatile int*>(&dummy), p.status);
                }
            }
        }
    } else if (warp == 1) {
        // ----------------------------------------------------- MMA issuer --
        if (leader) {
            const bool elect = elect_one();
            // stage 0's operands: the shared product's, the adapters'
            const uint32_t eb = 256u * p.rpad;
            const Desc dX(smem_desc(ring0, 16, 1024, kLayoutSw128));
            const Desc dW(B_MN ? smem_desc(ring0 + kPSlot, 8192, 1024, kLayoutSw128)
                               : smem_desc(ring0 + kPSlot, 16, 1024, kLayoutSw128));
            const Desc dU(kmajor_desc(ring0, p.rpad * 2));
            const Desc dE(B_MN ? smem_desc(ring0 + kPSlot, eb / 2, 1024, kLayoutSw128) : kmajor_desc(ring0 + kPSlot, p.rpad * 2));
            constexpr uint32_t kStep = B_MN ? 128 : 2;  // 16 reduction columns of the right operand
            int stage = 0;
            uint32_t phase = 0, acc = 0;
            bool ok = true, any_mma = false;
            for (int64_t t = slot; t < p.items && ok; t += nslot) {
                const PairTile ti = pair_tile(t, p);
                if (ti.n0 >= p.ncols) continue;
                const uint32_t idesc = idesc_bf16_f32_n(2 * kPM, ti.width, 0, B_MN ? 1 : 0);
                const int ne = p.plan.cnt[ti.unit];
                const uint4* masks = reinterpret_cast<const uint4*>(p.plan.mask + ti.unit * p.plan.slots * kUnitWords);
                const uint32_t buf = acc & 1u;
                if (!all_wait(&ctl->tmem_empty[buf], ((acc >> 1) & 1u) ^ 1u, abort_flag, p.status, true)) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * kPN;
                for (int i = 0; i < nb; ++i) {
                    if (!all_wait(&ctl->full[stage], phase, abort_flag, p.status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t at = stage * (kPStage / 16);
                    if (elect) {
#pragma unroll
                        for (int ks = 0; ks < kPK / 16; ++ks)
                            umma_at<true>(d, dX, at + 2 * ks, dW, at + kStep * ks, idesc, (i > 0 || ks > 0) ? 1u : 0u);
                        umma_commit_pair(&ctl->empty[stage], 0x3);
                    }
                    if (i == 0) {  // the masks, while the shared product runs
                        for (int e = lane; e < 2 * ne; e += 32)
                            cp_async_16(smem_u32(&ctl->mask[0][0]) + 16 * e, masks + e, 16u);
                        cp_async_commit();
                    }
                    any_mma = true;
                    if (++stage == kPStages) { stage = 0; phase ^= 1u; }
                }
                const int xb = ext_blocks(ne);
                cp_async_wait<0>();
                __syncwarp();
                int ef = 0, rc = 0;
                for (int xi = 0; xi < xb && ok; ++xi) {
                    const int en = min(p.epb, ne - ef);
                    const int steps = (min(64, p.r - rc) + 15) / 16;
                    if (!all_wait(&ctl->full[stage], phase, abort_flag, p.status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t at = stage * (kPStage / 16);
                    if (elect) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (e >= en) break;
                            const uint4 m0 = *reinterpret_cast<const uint4*>(&ctl->mask[ef + e][0]);
                            const uint4 m1 = *reinterpret_cast<const uint4*>(&ctl->mask[ef + e][4]);
                            const uint32_t keep[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                if (ks < steps)
                                    umma_rows_pair_at(d, dU, at + 2 * ks, dE, at + e * (eb / 16) + kStep * ks, idesc, keep);
                        }
                        umma_commit_pair(&ctl->empty[stage], 0x3);
                    }
                    if ((rc += 64) >= p.r) {
                        rc = 0;
                        ef += p.epb;
                    }
                    if (++stage == kPStages) { stage = 0; phase ^= 1u; }
                }
                __syncwarp();  // every mask has been read before the next tile's arrive
                if (ok && elect) umma_commit_pair(&ctl->tmem_full[buf], 0x3);
                ++acc;
            }
            if (any_mma) {
                if (elect) umma_commit_pair(&ctl->drain, 0x1);
                int dummy = 0;
                mbar_wait(&ctl->drain, 0, reinterpret_cast<volatile int*>(&dummy), p.status);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- epilogue --
        const int q = warp & 3;
        const uint64_t pol = l2_policy_evict_first();
        uint32_t acc = 0;
        for (int64_t t = slot; t < p.items; t += nslot) {
            const PairTile ti = pair_tile(t, p);
            if (ti.n0 >= p.ncols) continue;
            const int end = min(p.ncols, ti.n0 + ti.width);
            const int64_t row = ti.unit * kUnit + rank * kPM + q * 32 + lane;
            uint16_t* orow = row < p.plan.T ? p.out + row * p.ncols : nullptr;
            const uint32_t buf = acc & 1u;
            if (!warp_wait(&ctl->tmem_full[buf], (acc >> 1) & 1u, abort_flag, p.status, 64, true)) break;
            tc_fence_after();
            const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * kPN;
#pragma unroll 1
            for (int c = 0; c < ti.width; c += 128) {
                __syncwarp();
                uint32_t v[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld_32x32b_x32(ta + c + 32 * k, v[k]);
                tmem_ld_wait();
                if (c + 128 >= ti.width) {
                    // every column is in registers: hand the accumulator back
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader) mbar_arrive(&ctl->tmem_empty[buf]);
                        else mbar_arrive_remote(&ctl->tmem_empty[buf], 0);
                    }
                }
                if (!orow) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int pc = 0; pc < 32; pc += 16) {
                        const int col = ti.n0 + c + 32 * k + pc;
                        uint4 o[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t* x = &v[k][pc + 8 * h];
                            o[h] = make_uint4(pack_bf16x2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                              pack_bf16x2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                                              pack_bf16x2(__uint_as_float(x[4]), __uint_as_float(x[5])),
                                              pack_bf16x2(__uint_as_float(x[6]), __uint_as_float(x[7])));
                        }
                        if (p.st32 && col + 8 < end) {
                            st_global_32_policy(orow + col, o[0], o[1], pol);
                        } else {
                            if (col < end) st_global_16_policy(orow + col, o[0], pol);
                            if (col + 8 < end) st_global_16_policy(orow + col + 8, o[1], pol);
                        }
                    }
            }
            ++acc;
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still signal it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 2 * kPN);
}

// Clusters resident at once.
template <bool B_MN>
int pair_room(int* clusters) {
    static ClusterRoom rooms;
    int room[kMaxCluster + 1];
    const int rc = rooms.get(pair_kernel<B_MN>, kPairSmem, room);
    if (rc == GG_OK) *clusters = room[2];
    return rc;
}

// X, W, U, adapters; W's and the adapters' columns of a piece
template <bool B_MN>
int launch_pair(const CUtensorMap (&m)[6], const PairParams& p, int clusters, cudaStream_t st) {
    ClusterLaunch l(2 * (p.items < clusters ? p.items : clusters), kPThreads, kPairSmem, 2, true, st);
    clear_pending_launch_error();
    const cudaError_t err = cudaLaunchKernelEx(&l.cfg, pair_kernel<B_MN>, m[0], m[1], m[2], m[3], m[4], m[5], p);
    if (err != cudaSuccess) { record_cuda_error(err); return GG_ERR_CUDA; }
    return launch_result();
}

}  // namespace

int lora_pair_launch(bool b_mn, const uint16_t* X, const uint16_t* W, const uint16_t* U, const uint16_t* ad,
                     const PlanView& plan, int64_t Kred, int64_t ncols, int r, uint16_t* out, uint32_t* ready,
                     int32_t* status, cudaStream_t st) {
    PairParams p{};
    p.plan = plan;
    p.Kred = static_cast<int>(Kred);
    p.ncols = static_cast<int>(ncols);
    p.r = r;
    p.rpad = rank_pad(r);
    p.epb = 64 / p.rpad;
    int clusters = 0;
    const int rc = b_mn ? pair_room<true>(&clusters) : pair_room<false>(&clusters);
    if (rc != GG_OK) return rc;
    p.ntiles = static_cast<int>((ncols + kPN - 1) / kPN);
    // The last round's tiles, if they are at most half of the clusters, in halves: a round
    // takes as long as its widest item (2600 rows of 4096 x 2056: 52 us whole, 45 cut; in
    // quarters, whose blocks are bound by their row loads, no less).
    const int64_t tiles = plan.units * p.ntiles, rest = tiles % clusters;
    p.cuts = rest * 2 <= clusters ? 2 : 1;
    p.whole = tiles - rest;
    p.items = p.whole + rest * p.cuts;
    p.out = out;
    p.ready = ready;
    p.st32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 && ncols % 16 == 0;
    p.status = status;
    CUtensorMap m[6] = {};
    if (!encode_map_2d(&m[0], X, Kred, plan.T, Kred, kPK, kPM)) return GG_ERR_CUDA;
    if (!encode_map_2d(&m[2], U, r, plan.T, r, p.rpad, kPM)) return GG_ERR_CUDA;
    if (b_mn) {  // W [Kred, ncols], ad [L, r, ncols]: 64-column pieces in either case
        if (!encode_map_2d(&m[1], W, ncols, Kred, ncols, 64, kPK)) return GG_ERR_CUDA;
        if (!encode_map_3d(&m[3], ad, ncols, r, plan.L, ncols, ncols * r, 64, p.rpad)) return GG_ERR_CUDA;
        m[4] = m[1];
        m[5] = m[3];
        return launch_pair<true>(m, p, clusters, st);
    }
    if (!encode_map_2d(&m[1], W, Kred, ncols, Kred, kPK, kPN / 2)) return GG_ERR_CUDA;
    if (!encode_map_3d(&m[3], ad, r, ncols, plan.L, r, ncols * r, p.rpad, kPN / 2)) return GG_ERR_CUDA;
    m[4] = m[1];
    m[5] = m[3];
    if (p.cuts > 1 && rest > 0) {
        const uint32_t half = kPN / 2 / p.cuts;
        if (!encode_map_2d(&m[4], W, Kred, ncols, Kred, kPK, half)) return GG_ERR_CUDA;
        if (!encode_map_3d(&m[5], ad, r, ncols, plan.L, r, ncols * r, p.rpad, half)) return GG_ERR_CUDA;
    }
    return launch_pair<false>(m, p, clusters, st);
}

}  // namespace gg
