// lora_shrink.cu -- the low-rank products of the adapters:
//   U[t] = scale[a] X[t] A[a]^T   (forward; A [L, r, K] read along K)
//   V[t] = scale[a] dY[t] B[a]    (backward; B [L, N, r] read along r)
//
// Bound by reading X (dY) once.  A tile is up to 128 rows of one adapter in the
// plan's order, so nothing is computed for another adapter: neighbouring rows (a
// sequence's) come by TMA, scattered ones are gathered row by row with cp.async.
// Rank r leaves few output columns, so the reduction is split over a cluster; each
// CTA accumulates its share in tensor memory, and after a cluster barrier every
// CTA sums its part of the tile over the cluster's CTAs in rank order: one
// rounding, the same bits on every run, no atomics, no scratch in device memory.
//
// 8192 x 4096 at rank 32: 16 us, 4.2 TB/s, of which the plan's entry, the first loads and
// the join are 8; a bare ring of bulk loads of the same 67 MB, any tile shape (16 to 128
// rows), split (1 to 8) and depth, took 18-20 us by itself (inputs cold, events around it).
#include "lora.cuh"

namespace gg {
namespace {

constexpr int kSM = kTileRows;
constexpr int kSN = 128;             // rank columns of a tile (larger ranks: several tiles)
constexpr int kSK = 64;              // reduction block
constexpr int kSMaxStages = 6;
constexpr int kSThreads = 192;       // producer, issuer, four gather / epilogue warps
constexpr int kSRing = 98304;        // two CTAs an SM

struct ShrinkParams {
    PlanView plan;
    const uint16_t* X;
    int Kred, r;
    int take;          // rank columns of a tile
    int subs;          // tiles the rank is cut into
    int chunk;         // columns of an MN-major piece of the adapter (16, 32 or 64)
    int a_slot;        // bytes of a stage's row slot
    int stage_bytes, stages;
    const float* scale;
    uint16_t* out;
    uint16_t* parts;   // the product as two bf16 (below), [2][T, r] (or null)
    int64_t part;      // elements from one part to the other
    uint32_t* zero;    // words to clear for the kernels after
    int zero_words;
    int32_t* status;
};

struct ShrinkCtl {
    uint64_t full[kSMaxStages];
    uint64_t empty[kSMaxStages];
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
    int32_t row[kSM];  // the tile's rows
};

// v as two bf16 whose sum is v to 2^-16 and which have v's sign, both zero only if v is: the
// bits above bf16's last, and the rest (2^-24 of v if there is none).  A product with an
// infinity then is the same infinity for both (a rounded v and its remainder would give
// inf - inf or inf 0); an infinite or NaN v is both parts.
__device__ __forceinline__ void two_parts(float v, float& hi, float& lo) {
    hi = lo = v;
    if (fabsf(v) < __int_as_float(0x7f800000)) {
        hi = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
        lo = v - hi;
        if (lo == 0.f) lo = v * 0x1p-24f;
    }
}

constexpr int kShrinkSmem = 1024 + kSRing + 1024;
static_assert(sizeof(ShrinkCtl) <= 1024, "control block");
static_assert(kSRing >= kSM * (kSN + 4) * 4, "partial sums fit the drained ring");

template <bool B_MN>
__global__ void __launch_bounds__(kSThreads, 2)
shrink_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmE, const ShrinkParams p,
              const int S) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    ShrinkCtl* ctl = reinterpret_cast<ShrinkCtl*>(ring + kSRing);
    volatile int* abort_flag = &ctl->abort_flag;
    const int warp = warp_index(), lane = lane_id();
    const int rank = static_cast<int>(cluster_ctarank());
    const int64_t item = blockIdx.x / S;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmE);
    }
    // rows without an adapter get zeros, 32 rows a warp over the grid's warps 2-5 while the
    // others load (a CTA a unit after its sums made 2048 rows of 4096, half of them a run without, 16.3 us; now 7.7)
    auto zero_bare_rows = [&]() {
        const int64_t first = static_cast<int64_t>(blockIdx.x) * 4 + warp - 2, step = static_cast<int64_t>(gridDim.x) * 4;
        for (int64_t i = first * 32 + lane; i < p.zero_words; i += step * 32) p.zero[i] = 0;
        const int per = p.r / 8, at_once = 32 / per, sub = lane / per;  // 16-byte pieces of a row, rows of a warp
        for (int64_t w = first; w * 32 < p.plan.T; w += step) {
            uint32_t bare = ~p.plan.any[w];
            const int64_t left = p.plan.T - w * 32;
            if (left < 32) bare &= (1u << left) - 1u;
            if (!bare || sub >= at_once) continue;
            for (int row = sub; row < 32; row += at_once) {
                if (!(bare >> row & 1u)) continue;
                const int64_t at = (w * 32 + row) * p.r + (lane - sub * per) * 8;
                *reinterpret_cast<uint4*>(p.out + at) = make_uint4(0, 0, 0, 0);
                if (p.parts) {
                    *reinterpret_cast<uint4*>(p.parts + at) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(p.parts + p.part + at) = make_uint4(0, 0, 0, 0);
                }
            }
        }
        __syncwarp();
    };
    // (the grid has a cluster for every tile there could be: the entry exists)
    const int4 tile = p.plan.tile[item / p.subs];
    if (item >= static_cast<int64_t>(*p.plan.ntile) * p.subs) {  // the whole cluster
        if (warp >= 2) zero_bare_rows();
        return;
    }
    const int a = tile.x, n = tile.z;
    const bool gather = tile.w < 0;
    const int c0 = static_cast<int>(item % p.subs) * p.take;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&ctl->full[s], gather ? 1 + 128 : 1);
            mbar_init(&ctl->empty[s], 1);
        }
        mbar_init(&ctl->done, 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, kSN);
        tmem_relinquish();
    }
    if (threadIdx.x >= 64) {
        const int i = threadIdx.x - 64;
        if (i < n) ctl->row[i] = gather ? p.plan.order[tile.y + i] : tile.w + i;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int nb = (p.Kred + kSK - 1) / kSK;
    const int lo = static_cast<int>(static_cast<int64_t>(nb) * rank / S);
    const int hi = static_cast<int>(static_cast<int64_t>(nb) * (rank + 1) / S);  // at least one block: S <= nb
    const uint32_t tmem = ctl->tmem_base;
    const uint32_t ring0 = smem_u32(ring);
    const int pieces = (p.take + p.chunk - 1) / p.chunk;   // MN-major pieces of the adapter
    const uint32_t piece_bytes = static_cast<uint32_t>(p.chunk) * kSK * 2;

    if (warp == 0) {
        // ------------------------------------------------------- producer --
        const bool elect = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        int issued = 0;
        const uint32_t ebytes = B_MN ? piece_bytes * pieces : static_cast<uint32_t>(p.take) * 128u;
        for (int b = lo; b < hi; ++b) {
            if (!all_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status)) break;
            uint8_t* sA = ring + stage * p.stage_bytes;
            uint8_t* sB = sA + p.a_slot;
            uint64_t* bar = &ctl->full[stage];
            if (elect) {
                mbar_arrive_expect_tx(bar, ebytes + (gather ? 0u : static_cast<uint32_t>(p.a_slot)));
                if (!gather) tma_load_2d(sA, &tmX, bar, b * kSK, tile.w);
                if (B_MN) {
                    for (int c = 0; c < pieces; ++c)
                        tma_load_3d(sB + c * piece_bytes, &tmE, bar, c0 + c * p.chunk, b * kSK, a);
                } else {
                    tma_load_3d(sB, &tmE, bar, b * kSK, c0, a);
                }
            }
            ++issued;
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
        // every copy has landed before the ring is reused or the CTA exits
        for (int j = 0; j < min(issued, p.stages); ++j) {
            if (--stage < 0) { stage = p.stages - 1; phase ^= 1u; }
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
        const int cols = B_MN ? pieces * p.chunk : (p.take + 15) / 16 * 16;
        const uint32_t idesc = idesc_bf16_f32_n(kSM, cols, 0, B_MN ? 1 : 0);
        const Desc dX(smem_desc(ring0, 16, 1024, kLayoutSw128));
        const Desc dE(B_MN ? mnmajor_desc(ring0 + p.a_slot, 2 * p.chunk, piece_bytes)
                           : smem_desc(ring0 + p.a_slot, 16, 1024, kLayoutSw128));
        const uint32_t step = B_MN ? 2 * p.chunk : 2;  // 16 reduction columns of the adapter
        for (int b = lo; b < hi; ++b) {
            if (!all_wait(&ctl->full[stage], phase, abort_flag, p.status)) break;
            tc_fence_after();
            const uint32_t at = stage * (p.stage_bytes / 16);
            if (elect) {
                if (gather) fence_proxy_async_smem();  // gathered rows are generic-proxy writes
#pragma unroll
                for (int ks = 0; ks < kSK / 16; ++ks)
                    umma_at<false>(tmem, dX, at + 2 * ks, dE, at + step * ks, idesc, (b > lo || ks > 0) ? 1u : 0u);
                umma_commit(&ctl->empty[stage]);
            }
            any_mma = true;
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
        if (elect) {
            if (any_mma) umma_commit(&ctl->done);
            else mbar_arrive(&ctl->done);
        }
        __syncwarp();
    } else if (gather) {
        // ---------------------------------------------------- row gathers --
        // thread: 16-byte piece gt & 7 of rows gt / 8 + 16 j; rows past the tile's
        // end are left as they are (their accumulator rows are not stored)
        const int gt = threadIdx.x - 64;
        const int pc = gt & 7;
        const uint16_t* src[kSM / 16];
#pragma unroll
        for (int j = 0; j < kSM / 16; ++j) {
            const int rr = (gt >> 3) + 16 * j;
            src[j] = rr < n ? p.X + static_cast<int64_t>(ctl->row[rr]) * p.Kred + pc * 8 : nullptr;
        }
        int stage = 0;
        uint32_t phase = 0;
        for (int b = lo; b < hi; ++b) {
            if (!warp_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status, 32)) break;
            const uint32_t sA = ring0 + stage * p.stage_bytes;
            const bool in = b * kSK + pc * 8 < p.Kred;
#pragma unroll
            for (int j = 0; j < kSM / 16; ++j) {
                const int rr = (gt >> 3) + 16 * j;
                if (rr < n)
                    cp_async_16(sA + rr * 128 + ((pc ^ (rr & 7)) << 4), in ? src[j] + b * kSK : p.X, in ? 16u : 0u);
            }
            cp_async_mbar_arrive(&ctl->full[stage]);
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
        cp_async_wait<0>();
    }
    if (warp >= 2) zero_bare_rows();

    // -------------------------------------------- partial sums to the cluster --
    const bool good = warp_wait(&ctl->done, 0, abort_flag, p.status);
    tc_fence_after();
    __syncthreads();  // the copies have landed, the MMAs have completed: the ring is free
    float* part = reinterpret_cast<float*>(ring);
    const int groups = min(p.take, p.r - c0) / 8;
    const int pitch = p.take + 4;
    const int q = warp & 3;
    if (warp >= 2 && q * 32 < n) {
        for (int c = 0; c < 8 * groups; c += 8) {
            uint32_t v[8];
            tmem_ld_32x32b_x8(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, v);
            tmem_ld_wait();
            float* d = part + (q * 32 + lane) * pitch + c;
            *reinterpret_cast<uint4*>(d) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4*>(d + 4) = make_uint4(v[4], v[5], v[6], v[7]);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (good) {
        const float sc = p.scale ? p.scale[a] : 1.0f;
        const int quads = groups * 2;
        for (int i = rank * kSThreads + threadIdx.x; i < n * quads; i += S * kSThreads) {
            const int rr = i / quads, c = (i % quads) * 4;
            float4 s = cluster_sum4(smem_u32(part + rr * pitch + c), S);
            s = make_float4(s.x * sc, s.y * sc, s.z * sc, s.w * sc);
            // U (V) is an operand of the tensor cores: bf16, which moves Y and dX by 0.0006 to
            // 0.0011 of their norm (their own rounding: 0.0017).  The adapter gradients sum V
            // over tokens: they take it as two bf16
            const int64_t at = static_cast<int64_t>(ctl->row[rr]) * p.r + c0 + c;
            *reinterpret_cast<uint2*>(p.out + at) = pack_bf16x4(s);
            if (p.parts) {
                float4 hi, lo;
                two_parts(s.x, hi.x, lo.x);
                two_parts(s.y, hi.y, lo.y);
                two_parts(s.z, hi.z, lo.z);
                two_parts(s.w, hi.w, lo.w);
                *reinterpret_cast<uint2*>(p.parts + at) = pack_bf16x4(hi);
                *reinterpret_cast<uint2*>(p.parts + p.part + at) = pack_bf16x4(lo);
            }
        }
    }
    __syncthreads();
    cluster_sync();  // no CTA leaves while another may still read its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kSN);
    }
}

template <bool B_MN>
int launch_shrink(const CUtensorMap& x, const CUtensorMap& e, const ShrinkParams& p, cudaStream_t st) {
    static ClusterRoom rooms;
    int room[kMaxCluster + 1];
    int rc = rooms.get(shrink_kernel<B_MN>, kShrinkSmem, room);
    if (rc != GG_OK) return rc;
    // The split: as many CTAs as are resident at once for the tiles a batch of
    // sequences has (whole tiles and half of the adapters' ragged ones).
    const int64_t nb = (p.Kred + kSK - 1) / kSK;
    const int64_t ragged = p.plan.max_tiles - p.plan.T / kTileRows;
    const int64_t tiles = (p.plan.T / kTileRows + (ragged + 1) / 2) * p.subs;
    int S = kMaxCluster;
    while (S > 1 && (tiles > room[S] || S > nb)) --S;
    const int64_t grid = p.plan.max_tiles * p.subs * S;
    if (grid >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
    ClusterLaunch l(grid, kSThreads, kShrinkSmem, S, false, st);
    clear_pending_launch_error();
    const cudaError_t err = cudaLaunchKernelEx(&l.cfg, shrink_kernel<B_MN>, x, e, p, S);
    if (err != cudaSuccess) { record_cuda_error(err); return GG_ERR_CUDA; }
    return launch_result();
}

}  // namespace

int lora_shrink_launch(bool b_mn, const uint16_t* X, const uint16_t* ad, const float* scale, const PlanView& plan,
                       int64_t Kred, int r, uint16_t* out, uint16_t* parts, int64_t part, uint32_t* zero,
                       int zero_words, int32_t* status, cudaStream_t st) {
    ShrinkParams p{};
    p.plan = plan;
    p.X = X;
    p.Kred = static_cast<int>(Kred);
    p.r = r;
    p.take = r < kSN ? r : kSN;
    p.subs = (r + kSN - 1) / kSN;
    p.chunk = rank_pad(p.take);
    p.scale = scale;
    p.out = out;
    p.parts = parts;
    p.part = part;
    p.zero = zero;
    p.zero_words = zero ? zero_words : 0;
    p.status = status;
    const int rows = plan.T >= kSM ? kSM : static_cast<int>((plan.T + 7) / 8 * 8);
    p.a_slot = rows * 128;
    // adapter slot: rank rows of 128 bytes, or MN-major pieces of kSK rows; at least
    // what the MMA reads past it of the row slot stays inside the ring
    const int e = b_mn ? (p.take + p.chunk - 1) / p.chunk * p.chunk * kSK * 2 : (p.take + 15) / 16 * 16 * 128;
    p.stage_bytes = (p.a_slot + e + 1023) / 1024 * 1024;
    p.stages = (kSRing - kSM * 128) / p.stage_bytes;
    if (p.stages > kSMaxStages) p.stages = kSMaxStages;
    CUtensorMap mX{}, mE{};
    if (!encode_map_2d(&mX, X, Kred, plan.T, Kred, kSK, rows)) return GG_ERR_CUDA;
    if (b_mn) {
        if (!encode_map_3d(&mE, ad, r, Kred, plan.L, r, Kred * r, p.chunk, kSK)) return GG_ERR_CUDA;
        return launch_shrink<true>(mX, mE, p, st);
    }
    if (!encode_map_3d(&mE, ad, Kred, r, plan.L, Kred, Kred * r, kSK, p.take)) return GG_ERR_CUDA;
    return launch_shrink<false>(mX, mE, p, st);
}

}  // namespace gg
