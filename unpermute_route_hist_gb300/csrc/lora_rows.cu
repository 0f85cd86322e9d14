// lora_rows.cu -- the adapter path's products over 128-row tiles with the
// reduction split over a cluster.
//
//  shrink   U[t] = scale[a] X[t] A[a]^T (forward; A [L, r, K] read along K) and
//           V[t] = scale[a] dY[t] B[a]  (backward; B [L, N, r] read along r).
//           A tile multiplies its rows by every adapter that occurs among them and
//           each row keeps its own adapter's columns.  Bound by reading X (dY)
//           once; rank r output columns, so the reduction is all there is to split.
//  project  Y = X W^T + U B[a]^T and dX = dY W + V A[a] for few row tiles (decode,
//           short prompts): bound by streaming W, which takes every SM, so each
//           128 x 128 tile's reduction is split over the cluster.  Longer batches
//           take the 2-CTA tiles of lora_pair.cu.
//
// A CTA computes its share of the reduction into tensor memory (TMA ring -> one
// issuing thread -> fp32 accumulators), writes it to shared memory, and after a
// cluster barrier each CTA sums its part of the tile over the cluster's CTAs in
// rank order: one rounding, the same bits on every run, no atomics, no scratch in
// device memory.
#include <atomic>

#include "lora.cuh"

namespace gg {
namespace {

constexpr int kRM = 128;              // rows of a tile
constexpr int kRN = 128;              // columns of a tile (project) or of a chunk (shrink)
constexpr int kRK = 64;               // reduction block
constexpr int kRStages = 3;           // two CTAs an SM
constexpr int kRThreads = 192;        // producer, issuer, four epilogue warps
constexpr int kRSlot = 128 * kRK * 2; // bytes of an operand slot
constexpr int kRStage = 2 * kRSlot;
constexpr int kMaxCluster = 8;

enum RowsMode { ROWS_SHRINK = 0, ROWS_PROJECT = 1 };

struct RowsParams {
    PlanView plan;
    int Kred;            // shared reduction length
    int ncols;           // project: output columns
    int r;               // rank
    int width;           // shrink: columns of one entry in a chunk (accumulator columns)
    int take;            // shrink: rank columns a chunk computes of an entry (r, or 128 of a larger rank)
    int subs;            // shrink: chunks a large rank is cut into
    int epc;             // shrink: entries of a chunk
    int nchunk;          // chunks (shrink) or column tiles (project) a row tile has
    int mtiles;
    int rpad, epb;       // project: width of an adapter block, adapters a ring stage holds
    int xrows;           // rows of the X boxes (a multiple of 8, at most 128)
    const float* scale;
    uint16_t* out;
    uint16_t* out_lo;    // shrink: the rounding's remainder, in bf16 (or null)
    int32_t* status;
};

struct RowsCtl {
    uint64_t full[kRStages];
    uint64_t empty[kRStages];
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
    int nent;                   // entries of this row tile
    uint32_t any[4];            // rows that have an adapter
    int32_t gid[kRM];
    uint32_t mask[kRM][4];
    int32_t own[kRM];           // shrink: the row's entry within the chunk, or -1
};

constexpr int kRowsSmem = 1024 + kRStages * kRStage + sizeof(RowsCtl);
static_assert(kRStages * kRStage >= kRM * (kRN + 4) * 4, "partial sums fit the drained ring");

// B_MN: the right operands are read along their columns (dY B and dY W + V A).
template <int MODE, bool B_MN>
__global__ void __launch_bounds__(kRThreads, 2)
rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
            const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmE, const RowsParams p,
            const int S) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    RowsCtl* ctl = reinterpret_cast<RowsCtl*>(ring + kRStages * kRStage);
    volatile int* abort_flag = &ctl->abort_flag;
    const int warp = warp_id(), lane = lane_id();
    const int rank = static_cast<int>(cluster_ctarank());
    const int64_t item = blockIdx.x / S;
    // shrink: a row tile's chunks are neighbours (they read the same X); project: a
    // column tile's row tiles are (they read the same W)
    const int64_t mt = MODE == ROWS_SHRINK ? item / p.nchunk : item % p.mtiles;
    const int chunk = static_cast<int>(MODE == ROWS_SHRINK ? item % p.nchunk : item / p.mtiles);
    const int64_t row0 = mt * kRM;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kRM), p.plan.T - row0));
    const int n0 = chunk * kRN;  // project

    if (MODE == ROWS_SHRINK) pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRStages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        mbar_init(&ctl->done, 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmE);
        if (MODE == ROWS_PROJECT) {
            tma_prefetch_desc(&tmW);
            tma_prefetch_desc(&tmU);
        }
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
        uint32_t any[4] = {0, 0, 0, 0};
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
            any[0] |= m.x;
            any[1] |= m.y;
            any[2] |= m.z;
            any[3] |= m.w;
            n += __popc(b);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t o = __reduce_or_sync(0xffffffffu, any[w]);
            if (lane == 0) ctl->any[w] = o;
        }
        if (lane == 0) ctl->nent = n;
    }
    if (MODE == ROWS_SHRINK && threadIdx.x < kRM) ctl->own[threadIdx.x] = -1;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int nent = ctl->nent;
    // shrink: this chunk's entries and the columns of their rank it takes
    const int e0 = MODE == ROWS_SHRINK ? (chunk / p.subs) * p.epc : 0;
    const int ne = MODE == ROWS_SHRINK ? max(0, min(p.epc, nent - e0)) : nent;
    const int c0 = MODE == ROWS_SHRINK ? (chunk % p.subs) * p.take : 0;
    // this rank's reduction blocks: a share of the shared product's, then of the adapters'
    const int nb = (p.Kred + kRK - 1) / kRK;
    const int rchunks = (p.r + 63) / 64;
    const int xb = MODE == ROWS_PROJECT ? (p.r <= 64 ? (ne + p.epb - 1) / p.epb : ne * rchunks) : 0;
    const bool work = MODE == ROWS_PROJECT || ne > 0;
    const int b_lo = work ? static_cast<int>(static_cast<int64_t>(nb) * rank / S) : 0;
    const int b_hi = work ? static_cast<int>(static_cast<int64_t>(nb) * (rank + 1) / S) : 0;
    const int x_lo = static_cast<int>(static_cast<int64_t>(xb) * rank / S);
    const int x_hi = static_cast<int>(static_cast<int64_t>(xb) * (rank + 1) / S);
    const int nblk = (b_hi - b_lo) + (x_hi - x_lo);
    const uint32_t tmem = ctl->tmem_base;
    const uint32_t ring0 = smem_u32(ring);

    if (warp == 0) {
        // ------------------------------------------------------- producer --
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            bool ok = true;
            const uint32_t xbytes = static_cast<uint32_t>(p.xrows) * 128u;
            for (int i = 0; i < nblk; ++i) {
                if (!mbar_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
                uint8_t* sA = ring + stage * kRStage;
                uint8_t* sB = sA + kRSlot;
                uint64_t* bar = &ctl->full[stage];
                if (i < b_hi - b_lo) {
                    const int red = (b_lo + i) * kRK;
                    if (MODE == ROWS_SHRINK) {
                        const int boxes = B_MN ? p.width / 64 : 1;
                        const uint32_t ebytes = B_MN ? 8192u * boxes : static_cast<uint32_t>(p.width) * 128u;
                        mbar_arrive_expect_tx(bar, xbytes + ebytes * ne);
                        tma_load_2d(sA, &tmX, bar, red, static_cast<int32_t>(row0));
                        for (int e = 0; e < ne; ++e) {
                            if (B_MN) {
                                for (int c = 0; c < boxes; ++c)
                                    tma_load_3d(sB + e * ebytes + c * 8192, &tmE, bar, c0 + c * 64, red, ctl->gid[e0 + e]);
                            } else {
                                tma_load_3d(sB + e * ebytes, &tmE, bar, red, c0, ctl->gid[e0 + e]);
                            }
                        }
                    } else {
                        mbar_arrive_expect_tx(bar, xbytes + kRSlot);
                        tma_load_2d(sA, &tmX, bar, red, static_cast<int32_t>(row0));
                        if (B_MN) {
                            tma_load_2d(sB, &tmW, bar, n0, red);
                            tma_load_2d(sB + 8192, &tmW, bar, n0 + 64, red);
                        } else {
                            tma_load_2d(sB, &tmW, bar, red, n0);
                        }
                    }
                } else {
                    if (i == b_hi - b_lo) pdl_wait();  // U (V) of the kernel before
                    const int xi = x_lo + i - (b_hi - b_lo);
                    const int ef = p.r <= 64 ? xi * p.epb : xi / rchunks;
                    const int en = p.r <= 64 ? min(p.epb, ne - ef) : 1;
                    const int rc = p.r <= 64 ? 0 : (xi % rchunks) * 64;
                    const uint32_t eb = 256u * p.rpad;
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
                ++issued;
                if (++stage == kRStages) { stage = 0; phase ^= 1u; }
            }
            // the launch before this one has finished before this grid can
            if (MODE == ROWS_PROJECT) pdl_wait();
            // every copy has landed before the ring is reused or the CTA exits
            (void)ok;
            for (int j = 0; j < min(issued, kRStages); ++j) {
                if (--stage < 0) { stage = kRStages - 1; phase ^= 1u; }
                int dummy = 0;
                mbar_wait(&ctl->full[stage], phase, reinterpret_cast<volatile int*>(&dummy), p.status);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------- MMA issuer --
        if (lane == 0 && nblk > 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool any_mma = false;
            const int mma_n = MODE == ROWS_SHRINK ? (ne * p.width + 15) / 16 * 16 : kRN;
            const uint32_t idesc = idesc_bf16_f32(kRM, 16, 0, B_MN ? 1 : 0) - (2u << 17) +
                                   (static_cast<uint32_t>(mma_n >> 3) << 17);
            for (int i = 0; i < nblk; ++i) {
                if (!mbar_wait(&ctl->full[stage], phase, abort_flag, p.status)) break;
                tc_fence_after();
                const uint32_t sA = ring0 + stage * kRStage, sB = sA + kRSlot;
                if (i < b_hi - b_lo) {
#pragma unroll
                    for (int ks = 0; ks < kRK / 16; ++ks) {
                        const uint64_t ad = smem_desc(sA + ks * 32, 16, 1024, kLayoutSw128);
                        const uint64_t bd = B_MN ? smem_desc(sB + ks * 2048, 8192, 1024, kLayoutSw128)
                                                 : smem_desc(sB + ks * 32, 16, 1024, kLayoutSw128);
                        umma_bf16(tmem, ad, bd, idesc, (i > 0 || ks > 0) ? 1u : 0u);
                    }
                } else {
                    const int xi = x_lo + i - (b_hi - b_lo);
                    const int ef = p.r <= 64 ? xi * p.epb : xi / rchunks;
                    const int en = p.r <= 64 ? min(p.epb, ne - ef) : 1;
                    const int left = p.r <= 64 ? p.r : min(64, p.r - (xi % rchunks) * 64);
                    const uint32_t eb = 256u * p.rpad;
                    for (int e = 0; e < en; ++e) {
                        const uint32_t keep[4] = {ctl->mask[ef + e][0], ctl->mask[ef + e][1], ctl->mask[ef + e][2],
                                                  ctl->mask[ef + e][3]};
                        for (int ks = 0; ks < (left + 15) / 16; ++ks) {
                            const uint64_t ad = kmajor_desc(sA + ks * 32, p.rpad * 2);
                            const uint64_t bd = B_MN ? smem_desc(sB + e * eb + ks * 2048, eb / 2, 1024, kLayoutSw128)
                                                     : kmajor_desc(sB + e * eb + ks * 32, p.rpad * 2);
                            umma_bf16_rows(tmem, ad, bd, idesc, keep);
                        }
                    }
                }
                umma_commit(&ctl->empty[stage]);
                any_mma = true;
                if (++stage == kRStages) { stage = 0; phase ^= 1u; }
            }
            if (any_mma) umma_commit(&ctl->done);
            else mbar_arrive(&ctl->done);
        }
        __syncwarp();
    }

    // -------------------------------------------- partial sums to the cluster --
    // (every warp: the ring is free once the MMAs have completed)
    bool good = true;
    if (nblk > 0) good = warp_wait(&ctl->done, 0, abort_flag, p.status);
    tc_fence_after();
    __syncthreads();  // the producer has seen its copies land
    float* part = reinterpret_cast<float*>(ring);
    const int q = warp & 3;
    const int row = q * 32 + lane;
    const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if (MODE == ROWS_SHRINK) {
        const int pitch = p.take + 4;
        if (warp >= 2 && nblk > 0 && q * 32 < rows) {
            for (int e = 0; e < ne; ++e) {
                const uint32_t m = ctl->mask[e0 + e][q];
                if (m == 0) continue;
                const bool mine = (m >> lane) & 1u;
                if (mine) ctl->own[row] = e;
                for (int c = 0; c < p.take; c += 8) {
                    uint32_t v[8];
                    tmem_ld_32x32b_x8(tq + e * p.width + c, v);
                    tmem_ld_wait();
                    if (mine) {
                        *reinterpret_cast<uint4*>(part + row * pitch + c) = make_uint4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<uint4*>(part + row * pitch + c + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                    }
                    __syncwarp();
                }
            }
        }
        tc_fence_before();
        __syncthreads();
        cluster_sync();
        const int groups = min(p.take, p.r - c0) / 8;
        if (ne > 0 && good) {
            for (int i = rank * kRThreads + threadIdx.x; i < rows * groups; i += S * kRThreads) {
                const int rr = i / groups, c = (i % groups) * 8;
                const int e = ctl->own[rr];
                if (e < 0) continue;
                float s[8];
                cluster_sum8(smem_u32(part + rr * pitch + c), S, s);
                const float sc = p.scale ? p.scale[ctl->gid[e0 + e]] : 1.0f;
                float lo[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s[k] *= sc;
                    const float hi = __bfloat162float(__float2bfloat16(s[k]));
                    lo[k] = fabsf(hi) < __int_as_float(0x7f800000) ? s[k] - hi : 0.f;
                }
                const int64_t at = (row0 + rr) * p.r + c0 + c;
                // U (V) is the tensor cores' operand: bf16, and for the adapter gradients,
                // which sum it over tokens, its remainder as a second bf16
                *reinterpret_cast<uint4*>(p.out + at) = pack_bf16x8(s);
                if (p.out_lo) *reinterpret_cast<uint4*>(p.out_lo + at) = pack_bf16x8(lo);
            }
        }
        // rows without an adapter keep zeros
        if (chunk == 0) {
            for (int i = rank * kRThreads + threadIdx.x; i < rows * (p.r / 8); i += S * kRThreads) {
                const int rr = i / (p.r / 8), c = (i % (p.r / 8)) * 8;
                if ((ctl->any[rr >> 5] >> (rr & 31)) & 1u) continue;
                *reinterpret_cast<uint4*>(p.out + (row0 + rr) * p.r + c) = make_uint4(0, 0, 0, 0);
                if (p.out_lo) *reinterpret_cast<uint4*>(p.out_lo + (row0 + rr) * p.r + c) = make_uint4(0, 0, 0, 0);
            }
        }
    } else {
        // 16-byte pieces of a row rotated by the row, so neither side has bank conflicts
        if (warp >= 2 && q * 32 < rows) {
#pragma unroll 1
            for (int c = 0; c < kRN; c += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tq + c, v);
                tmem_ld_wait();
                if (row < rows) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // pieces in pairs: a group of 8 columns stays together
                        const int piece = (((c / 8 + k / 2) ^ (row & 15)) << 1) | (k & 1);
                        *reinterpret_cast<uint4*>(part + row * kRN + piece * 4) =
                            make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        __syncthreads();
        cluster_sync();
        if (good) {
            // rank s takes the 8-column groups g with g % S == s
            const int mine = (kRN / 8 - rank + S - 1) / S;
            for (int i = threadIdx.x; i < rows * mine; i += kRThreads) {
                const int rr = i / mine, g = (i % mine) * S + rank;
                const int col = n0 + g * 8;
                if (col >= p.ncols) continue;
                float s[8];
                cluster_sum8(smem_u32(part + rr * kRN + ((g ^ (rr & 15)) << 3)), S, s);
                *reinterpret_cast<uint4*>(p.out + (row0 + rr) * p.ncols + col) = pack_bf16x8(s);
            }
        }
    }
    __syncthreads();
    cluster_sync();  // no CTA leaves while another may still read its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kRN);
    }
}

template <int MODE, bool B_MN>
int launch_rows(const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& u, const CUtensorMap& e,
                const RowsParams& p, int S, bool pdl, cudaStream_t st) {
    auto kern = rows_kernel<MODE, B_MN>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) { record_cuda_error(err); return GG_ERR_CUDA; }
    if (dev < 0 || dev >= 64) dev = 0;
    static std::atomic<bool> smem_set[64];
    if (!smem_set[dev].load(std::memory_order_acquire)) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
        if (err != cudaSuccess) { record_cuda_error(err); return GG_ERR_CUDA; }
        smem_set[dev].store(true, std::memory_order_release);
    }
    const int64_t grid = static_cast<int64_t>(p.mtiles) * p.nchunk * S;
    if (grid >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(S);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kRThreads);
    cfg.dynamicSmemBytes = kRowsSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    clear_pending_launch_error();
    err = cudaLaunchKernelEx(&cfg, kern, x, w, u, e, p, S);
    if (err != cudaSuccess) { record_cuda_error(err); return GG_ERR_CUDA; }
    return launch_result();
}

int box_rows(int64_t T) { return T >= kRM ? kRM : static_cast<int>((T + 7) / 8 * 8); }

}  // namespace

int lora_shrink_launch(bool b_mn, const uint16_t* X, const uint16_t* ad, const float* scale, const PlanView& plan,
                       int64_t Kred, int r, uint16_t* out, uint16_t* out_lo, int32_t* status, cudaStream_t st) {
    RowsParams p{};
    p.plan = plan;
    p.Kred = static_cast<int>(Kred);
    p.r = r;
    p.mtiles = static_cast<int>((plan.T + kRM - 1) / kRM);
    p.xrows = box_rows(plan.T);
    p.scale = scale;
    p.out = out;
    p.out_lo = out_lo;
    p.status = status;
    p.take = r < kRN ? r : kRN;
    p.subs = (r + kRN - 1) / kRN;
    p.width = b_mn ? (p.take + 63) / 64 * 64 : p.take;
    const int64_t nb = (Kred + kRK - 1) / kRK;
    const int64_t most = plan.L < (plan.T < kRM ? plan.T : kRM) ? plan.L : (plan.T < kRM ? plan.T : kRM);
    // Entries a chunk takes: up to 128 accumulator columns, fewer while the chunks
    // that can be in use leave SMs idle (few rows, many adapters).
    p.epc = p.subs > 1 ? 1 : (kRN / p.width < 1 ? 1 : kRN / p.width);
    while (p.epc > 1 && p.mtiles * ((most + p.epc - 1) / p.epc) * kMaxCluster < 2 * num_sms()) p.epc = (p.epc + 1) / 2;
    p.nchunk = static_cast<int>((most + p.epc - 1) / p.epc) * p.subs;
    // The reduction's split: enough CTAs for two an SM, at least two blocks each.
    int S = kMaxCluster;
    while (S > 1 && (static_cast<int64_t>(p.mtiles) * S > 4 * num_sms() || S * 2 > nb)) S /= 2;
    CUtensorMap mX{}, mE{};
    if (!encode_map_2d(&mX, X, Kred, plan.T, Kred, kRK, p.xrows)) return GG_ERR_CUDA;
    if (b_mn) {
        if (!encode_map_3d(&mE, ad, r, Kred, plan.L, r, Kred * r, 64, kRK)) return GG_ERR_CUDA;
        return launch_rows<ROWS_SHRINK, true>(mX, mX, mX, mE, p, S, false, st);
    }
    if (!encode_map_3d(&mE, ad, Kred, r, plan.L, Kred, Kred * r, kRK, p.take)) return GG_ERR_CUDA;
    return launch_rows<ROWS_SHRINK, false>(mX, mX, mX, mE, p, S, false, st);
}

int lora_project_launch(bool b_mn, const uint16_t* X, const uint16_t* W, const uint16_t* U, const uint16_t* ad,
                        const PlanView& plan, int64_t Kred, int64_t ncols, int r, uint16_t* out, int32_t* status,
                        cudaStream_t st) {
    RowsParams p{};
    p.plan = plan;
    p.Kred = static_cast<int>(Kred);
    p.ncols = static_cast<int>(ncols);
    p.r = r;
    p.rpad = rank_pad(r);
    p.epb = 64 / p.rpad;
    p.mtiles = static_cast<int>((plan.T + kRM - 1) / kRM);
    p.nchunk = static_cast<int>((ncols + kRN - 1) / kRN);
    p.xrows = box_rows(plan.T);
    p.out = out;
    p.status = status;
    const int64_t nb = (Kred + kRK - 1) / kRK;
    const int64_t tiles = static_cast<int64_t>(p.mtiles) * p.nchunk;
    int S = static_cast<int>(2 * num_sms() / tiles);
    if (S > kMaxCluster) S = kMaxCluster;
    if (S > nb) S = static_cast<int>(nb);
    if (S < 1) S = 1;
    CUtensorMap mX{}, mW{}, mU{}, mE{};
    if (!encode_map_2d(&mX, X, Kred, plan.T, Kred, kRK, p.xrows)) return GG_ERR_CUDA;
    if (!encode_map_2d(&mU, U, r, plan.T, r, p.rpad, p.xrows)) return GG_ERR_CUDA;
    if (b_mn) {  // W [Kred, ncols], ad [L, r, ncols]
        if (!encode_map_2d(&mW, W, ncols, Kred, ncols, 64, kRK)) return GG_ERR_CUDA;
        if (!encode_map_3d(&mE, ad, ncols, r, plan.L, ncols, ncols * r, 64, p.rpad)) return GG_ERR_CUDA;
        return launch_rows<ROWS_PROJECT, true>(mX, mW, mU, mE, p, S, true, st);
    }
    if (!encode_map_2d(&mW, W, Kred, ncols, Kred, kRK, kRN)) return GG_ERR_CUDA;
    if (!encode_map_3d(&mE, ad, r, ncols, plan.L, r, ncols * r, p.rpad, kRN)) return GG_ERR_CUDA;
    return launch_rows<ROWS_PROJECT, false>(mX, mW, mU, mE, p, S, true, st);
}

}  // namespace gg
