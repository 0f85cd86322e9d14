// lora_grad.cu -- gradients of the adapters, a ragged reduction over each
// adapter's tokens:
//   dA[a] = sum_{t: ids[t] = a} V[t]^T X[t]    [r, K]
//   dB[a] = sum_{t: ids[t] = a} dY[t]^T U[t]   [N, r]
// Both are one problem: a wide source (X, dY) read along its columns against a
// narrow one (V, U), for a 128-column chunk of the wide source and one adapter.
// Bound by reading X and dY once; the MMAs run with the wide columns as M and the
// rank as N.
//
// The rows are the plan's blocks of up to 64 rows of one adapter.  A block whose
// rows are neighbours in memory (a sequence's) is copied by TMA; any other (ids
// in no order, the adapter's last rows) is gathered row by row with cp.async, rows
// past the end as zeros, so nothing of another adapter's rows enters the sums.
//
// All blocks of all (adapter, chunk) items are one list, cut into equal shares, one
// a CTA: adapters differ widely in tokens, and an item a CTA left the largest
// adapter's items running alone (65 against 47 us for two draws of 8192 tokens).
// The ring runs on from item to item; accumulators are double-buffered, so an item's
// epilogue overlaps the next one's loads.  An item that ends in another CTA than it
// began leaves fp32 partial sums, and whichever of its CTAs comes last adds them in
// block order: nothing waits, and the bits do not depend on who that was.
//
// 8192 tokens, 8 adapters of rank 32, 4096 and 6144 columns: 56 us with V's product before it,
// 4.8 TB/s of X and of dY twice; 12 us after dX, beside whose last tiles it starts.
#include "lora.cuh"

namespace gg {
namespace {

constexpr int kGM = 128;            // columns of the wide source
constexpr int kGK = kBlockRows;     // rows of a block
constexpr int kGThreads = 320;      // producer, issuer, four gather and four epilogue warps
constexpr int kGWide = kGM * kGK * 2;
constexpr int kGMaxStages = 8;
constexpr int kGMinBlocks = 2;      // of a CTA's share

struct GradSide {
    const uint16_t* wide;      // [T, cols]
    const uint16_t* narrow[2]; // [T, r]: the operand, in one or two parts
    int parts;                 // 1 or 2 of them
    int cols;
    int tiles;                 // 128-column chunks
    uint16_t* out;
};

struct GradParams {
    PlanView plan;
    GradSide side[2];          // dA, dB
    int r, nc;                 // rank; number of its pieces
    int stages;
    int stage_bytes;
    uint32_t* counter;         // [CTA]: arrivals of the item that CTA began and did not end
    float* sums;               // [CTA][2][r][128]
    uint32_t* ready;           // released by dX's kernel once V and the cleared counters can be read (or null)
    int32_t* status;
};

struct GradCtl {
    uint64_t full[kGMaxStages];
    uint64_t empty[kGMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int last;
    int ready;              // V can be read: nothing to wait for
    int kind[kGMaxStages];  // of the stage's block: kGathered | kItemEnd | kTwoParts
};

constexpr int kGathered = 1;  // by cp.async
constexpr int kItemEnd = 2;   // the last of its item here
constexpr int kTwoParts = 4;  // of the narrow operand

struct GradMaps {
    CUtensorMap wide[2];
    CUtensorMap narrow[3];     // V's two parts, U
};

// A CTA's share of the list, walked item by item: adapter a, chunk `tile` of both
// sides' together, block b of the adapter's nb.
struct GradWalk {
    int a, tile, b, nb;
    int64_t at;  // position in the list
};

// Whether ok holds in all 128 threads of the epilogue (a barrier of theirs).
__device__ __forceinline__ bool all_of_128(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1u : 0u)
        : "memory");
    return r != 0;
}

// RING: bytes of the operand ring; CTAS: resident on an SM; CHUNK: rank columns of a
// narrow piece (16, 32 or 64)
template <int RING, int CTAS, int CHUNK>
__global__ void __launch_bounds__(kGThreads, CTAS)
grad_kernel(const __grid_constant__ GradMaps maps, const GradParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    __shared__ GradCtl ctl_s;
    GradCtl* ctl = &ctl_s;
    volatile int* abort_flag = &ctl->abort_flag;
    const int warp = warp_index(), lane = lane_id();
    const int tiles = p.side[0].tiles + p.side[1].tiles;
    const int ncols = CHUNK * p.nc;  // accumulator columns
    const int buf_cols = ncols <= 16 ? 16 : (ncols <= 32 ? 32 : (ncols <= 64 ? 64 : (ncols <= 128 ? 128 : 256)));
    constexpr uint32_t piece_bytes = CHUNK * kGK * 2;

    // adapters without tokens get zeros, a piece from every CTA: a lane looks at an
    // adapter, the warp clears those found
    for (int a0 = warp * 32; a0 < p.plan.L; a0 += kGThreads) {
        const int mine = a0 + lane;
        const bool empty = mine < p.plan.L && p.plan.boff[mine + 1] == p.plan.boff[mine];
        for (uint32_t found = __ballot_sync(0xffffffffu, empty); found; found &= found - 1) {
            const int a = a0 + __ffs(found) - 1;
            for (int k = 0; k < 2; ++k) {
                if (!p.side[k].tiles) continue;
                const int64_t n = static_cast<int64_t>(p.r) * p.side[k].cols;
                for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * 8; i < n;
                     i += static_cast<int64_t>(gridDim.x) * 256)
                    *reinterpret_cast<uint4*>(p.side[k].out + a * n + i) = make_uint4(0, 0, 0, 0);
            }
        }
    }
    const int nblocks = p.plan.boff[p.plan.L];
    const int64_t total = static_cast<int64_t>(nblocks) * tiles;
    // the CTAs that share the list: none without a block, else kGMinBlocks each
    const int64_t fit = total / kGMinBlocks > 1 ? total / kGMinBlocks : 1;
    const int64_t G = fit < gridDim.x ? fit : gridDim.x;
    if (blockIdx.x >= G) {
        pdl_wait();
        return;
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&ctl->full[s], 1 + 128);  // the producer, every gather thread
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->acc_full[b], 1);
            mbar_init(&ctl->acc_empty[b], 4);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        for (int k = 0; k < 2; ++k)
            if (p.side[k].tiles) tma_prefetch_desc(&maps.wide[k]);
    }
    if (threadIdx.x == 64) ctl->ready = p.ready && acquire_ready(p.ready);
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, 2 * buf_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Launched while the kernel before runs.  That is the one that makes V and clears the
    // counters, to be waited for, or dX's, which makes both visible by its flag: then nothing
    // here depends on it, and these CTAs fill the SMs its last tiles leave idle.
    if (!ctl->ready) pdl_wait();
    else if (warp == 0) fence_proxy_async();  // V's stores, before the producer's TMA reads of them
    const uint32_t tmem = ctl->tmem_base;
    const uint32_t ring0 = smem_u32(ring);
    // Share j ends where share j + 1 begins, at total (j + 1) / G or at an end of the item
    // there if that is near: an eighth of a share more work costs less than joining parts.
    const int64_t near = total / G / 8 > 1 ? total / G / 8 : 1;
    auto snap = [&](int64_t x, int64_t begin, int64_t end) {  // x in the item [begin, end)
        if (x - begin <= near && x - begin <= end - x) return begin;
        return end - x <= near ? end : x;
    };
    auto bound = [&](int64_t j) {
        const int64_t x = total * j / G;
        if (x >= total) return total;  // (and with no blocks at all)
        const int64_t tile = x / nblocks, base = tile * nblocks;
        const int a = p.plan.block[x - base].x;
        return snap(x, base + p.plan.boff[a], base + p.plan.boff[a + 1]);
    };
    const int64_t lo = bound(blockIdx.x), hi = bound(blockIdx.x + 1);

    // The list runs chunk by chunk through all adapters' blocks, so that blocks that have
    // to be gathered (3x a copied one's time) fall to all CTAs alike.
    // (the epilogue's walk, an item a step)
    auto start = [&]() {
        GradWalk w{0, 0, 0, 0, lo};
        if (lo < hi) {
            w.tile = static_cast<int>(lo / nblocks);
            const int in = static_cast<int>(lo - static_cast<int64_t>(w.tile) * nblocks);
            w.a = p.plan.block[in].x;
            w.b = in - p.plan.boff[w.a];
            w.nb = p.plan.boff[w.a + 1] - p.plan.boff[w.a];
        }
        return w;
    };
    auto next_item = [&](GradWalk& w) {  // past the last block of the item that is this CTA's
        w.at += w.nb - w.b;
        if (w.at >= hi) return;
        w.b = 0;
        do {
            if (++w.a == p.plan.L) {
                w.a = 0;
                ++w.tile;
            }
            w.nb = p.plan.boff[w.a + 1] - p.plan.boff[w.a];
        } while (w.nb == 0);
    };
    auto by_tma = [&](const int4& e) { return e.w >= 0 && (e.z & (kLastBlock - 1)) == kGK; };

    if (warp == 0) {
        // --------------------------------------------------- TMA producer --
        const bool elect = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        int64_t issued = 0;
        int tile = lo < hi ? static_cast<int>(lo / nblocks) : 0;
        int in = static_cast<int>(lo - static_cast<int64_t>(tile) * nblocks);
        int4 next = lo < hi ? p.plan.block[in] : make_int4(0, 0, 0, 0);
        for (int64_t at = lo; at < hi; ++at) {
            const int4 e = next;
            const int t = tile;
            if (++in == nblocks) { in = 0; ++tile; }
            next = p.plan.block[in];  // on its way while this one waits
            const int sd = t < p.side[0].tiles ? 0 : 1;
            const int col0 = (sd == 0 ? t : t - p.side[0].tiles) * kGM;
            const int parts = sd == 0 ? p.side[0].parts : p.side[1].parts;
            if (!all_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status)) break;
            uint64_t* bar = &ctl->full[stage];
            const bool tma = by_tma(e);
            if (elect) {
                ctl->kind[stage] = (tma ? 0 : kGathered) | ((e.z & kLastBlock) || at + 1 == hi ? kItemEnd : 0) |
                                   (parts == 2 ? kTwoParts : 0);
                if (tma) {
                    uint8_t* s = ring + stage * p.stage_bytes;
                    mbar_arrive_expect_tx(bar, kGWide + piece_bytes * (p.nc * parts));
                    tma_load_2d(s, &maps.wide[sd], bar, col0, e.w);
                    tma_load_2d(s + kGWide / 2, &maps.wide[sd], bar, col0 + 64, e.w);
                    s += kGWide;
                    for (int part = 0; part < parts; ++part)
                        for (int k = 0; k < p.nc; ++k, s += piece_bytes)
                            tma_load_2d(s, &maps.narrow[sd == 0 ? part : 2], bar, k * CHUNK, e.w);
                } else {
                    mbar_arrive(bar);
                }
            }
            ++issued;
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
        // every copy has landed before the CTA exits
        const int64_t pend = issued < p.stages ? issued : p.stages;
        for (int64_t j = 0; j < pend; ++j) {
            if (--stage < 0) { stage = p.stages - 1; phase ^= 1u; }
            int dummy = 0;
            mbar_wait(&ctl->full[stage], phase, reinterpret_cast<volatile int*>(&dummy), p.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------- MMA issuer --
        const bool elect = elect_one();
        const uint32_t idesc = idesc_bf16_f32_n(kGM, ncols, 1, 1);
        const Desc dWide(smem_desc(ring0, kGWide / 2, 1024, kLayoutSw128));
        const Desc dNarrow(mnmajor_desc(ring0 + kGWide, 2 * CHUNK, piece_bytes));
        constexpr uint32_t kStep = 2 * CHUNK;  // 16 rows of the narrow operand (the wide one's: 128)
        const uint32_t part_step = p.nc * piece_bytes / 16;
        int stage = 0;
        uint32_t phase = 0, item = 0;
        bool any_mma = false, first = true;
        for (int64_t at = lo; at < hi; ++at) {
            const uint32_t buf = item & 1u;
            if (first && !all_wait(&ctl->acc_empty[buf], ((item >> 1) & 1u) ^ 1u, abort_flag, p.status)) break;
            if (!all_wait(&ctl->full[stage], phase, abort_flag, p.status)) break;
            tc_fence_after();
            const int kind = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&ctl->kind[stage]), 0);
            const uint32_t off = stage * (p.stage_bytes / 16);
            const uint32_t d = tmem + buf * buf_cols;
            const bool end = (kind & kItemEnd) != 0;
            if (elect) {
                if (kind & kGathered) fence_proxy_async_smem();  // gathered rows are generic-proxy writes
#pragma unroll
                for (int ks = 0; ks < kGK / 16; ++ks)
                    umma_at<false>(d, dWide, off + ks * 128, dNarrow, off + ks * kStep, idesc, (!first || ks > 0) ? 1u : 0u);
                if (kind & kTwoParts) {
#pragma unroll
                    for (int ks = 0; ks < kGK / 16; ++ks)
                        umma_at<false>(d, dWide, off + ks * 128, dNarrow, off + part_step + ks * kStep, idesc, 1u);
                }
                umma_commit(&ctl->empty[stage]);
                if (end) umma_commit(&ctl->acc_full[buf]);
            }
            any_mma = true;
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
            first = end;
            if (end) ++item;
        }
        if (any_mma) {
            if (elect) umma_commit(&ctl->drain);
            int dummy = 0;
            mbar_wait(&ctl->drain, 0, reinterpret_cast<volatile int*>(&dummy), p.status);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ---------------------------------------------------- row gathers --
        const int gt = threadIdx.x - 64;  // 0 .. 127
        int stage = 0;
        uint32_t phase = 0;
        // wide: 16 pieces of 8 columns a row, 8 rows a step; narrow: CHUNK / 8 pieces a
        // row, kStep rows a step.  A block's rows are loaded one block ahead, its entry
        // two.
        constexpr int kPieces = CHUNK / 8, kStep = 128 / kPieces, kSteps = kGK / kStep < 1 ? 1 : kGK / kStep;
        const int pc = gt & 15, np = gt % kPieces, nr = gt / kPieces;
        int32_t wide[kGK / 8], narrow[kSteps];
        auto load_rows = [&](const int4& e) {
            const int n = e.z & (kLastBlock - 1);
            auto token = [&](int rr) {  // of the block's row rr
                return rr >= n ? -1 : (e.w >= 0 ? e.w + rr : p.plan.order[e.y + rr]);
            };
#pragma unroll
            for (int j = 0; j < kGK / 8; ++j) wide[j] = token((gt >> 4) + 8 * j);
#pragma unroll
            for (int j = 0; j < kSteps; ++j) narrow[j] = token(nr + kStep * j);
        };
        int tile = lo < hi ? static_cast<int>(lo / nblocks) : 0;
        int in = static_cast<int>(lo - static_cast<int64_t>(tile) * nblocks);
        int4 e = make_int4(0, 0, 0, 0), next = e;
        if (lo < hi) {
            e = p.plan.block[in];
            if (!by_tma(e)) load_rows(e);
            next = p.plan.block[in + 1 == nblocks ? 0 : in + 1];
        }
        // swizzled places of this thread's pieces: 16-byte piece index XOR the address bits
        // 7 and up, as TMA does (narrow rows are 2 CHUNK bytes)
        const uint32_t wide_to = (pc >> 3) * (kGWide / 2) + (gt >> 4) * 128 + (((pc & 7) ^ ((gt >> 4) & 7)) << 4);
        for (int64_t at = lo; at < hi; ++at) {
            const bool tma = by_tma(e);
            const int t = tile;
            if (!warp_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, p.status, 32)) break;
            if (tma) {
                mbar_arrive(&ctl->full[stage]);
            } else {
                const int sd = t < p.side[0].tiles ? 0 : 1;
                const int col = (sd == 0 ? t : t - p.side[0].tiles) * kGM + pc * 8;
                const uint16_t* src = sd == 0 ? p.side[0].wide : p.side[1].wide;
                const int cols = sd == 0 ? p.side[0].cols : p.side[1].cols;
                const uint32_t s = ring0 + stage * p.stage_bytes;
                const bool inside = col < cols;
                src += inside ? col : 0;
#pragma unroll
                for (int j = 0; j < kGK / 8; ++j)
                    cp_async_16(s + wide_to + j * 1024, src + static_cast<int64_t>(max(wide[j], 0)) * cols,
                                inside && wide[j] >= 0 ? 16u : 0u);
                const int parts = sd == 0 ? p.side[0].parts : p.side[1].parts;
                for (int part = 0; part < parts; ++part) {
                    const uint16_t* nsrc = sd == 1 ? p.side[1].narrow[0] : (part == 0 ? p.side[0].narrow[0] : p.side[0].narrow[1]);
                    for (int k = 0; k < p.nc; ++k) {
                        const int c = k * CHUNK + np * 8;
                        const uint32_t to = s + kGWide + (part * p.nc + k) * piece_bytes;
#pragma unroll
                        for (int j = 0; j < kSteps; ++j) {
                            const int rr = nr + kStep * j;
                            const uint32_t flip = static_cast<uint32_t>((rr * CHUNK * 2) >> 7) & (kPieces - 1);
                            if (kStep <= kGK || rr < kGK)
                                cp_async_16(to + rr * CHUNK * 2 + ((np ^ flip) << 4),
                                            nsrc + static_cast<int64_t>(max(narrow[j], 0)) * p.r + (c < p.r ? c : 0),
                                            narrow[j] >= 0 && c < p.r ? 16u : 0u);
                        }
                    }
                }
                cp_async_mbar_arrive(&ctl->full[stage]);
            }
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
            if (++in == nblocks) { in = 0; ++tile; }
            e = next;
            if (at + 1 < hi && !by_tma(e)) load_rows(e);
            next = p.plan.block[in + 1 == nblocks ? 0 : in + 1];
        }
        cp_async_wait<0>();
    } else {
        // ------------------------------------------------------- epilogue --
        constexpr int kCols = 16;  // rank columns a step
        const int q = warp & 3, row = q * 32 + lane;  // this thread's wide column
        uint32_t item = 0;
        GradWalk w = start();
        while (w.at < hi) {
            const uint32_t buf = item & 1u, round = (item >> 1) & 1u;
            ++item;
            // the item, and (if it is not all this CTA's) the CTAs that hold its blocks
            const int a = w.a, tile = w.tile;
            const int64_t i_lo = w.at - w.b, i_hi = i_lo + w.nb;
            int64_t c_lo = blockIdx.x, c_hi = blockIdx.x;
            if (i_lo < lo || i_hi > hi) {
                // (the shares at its ends, but for those whose bounds went to its ends)
                c_lo = ((i_lo + 1) * G - 1) / total;
                c_hi = (i_hi * G - 1) / total;
                for (int64_t x; (x = total * (c_lo + 1) / G) < i_hi && snap(x, i_lo, i_hi) == i_lo;) ++c_lo;
                for (int64_t x; (x = total * c_hi / G) > i_lo && snap(x, i_lo, i_hi) == i_hi;) --c_hi;
            }
            next_item(w);  // (its loads before the wait)
            const int sd = tile < p.side[0].tiles ? 0 : 1;
            const GradSide& side = p.side[sd];
            const int col = (sd == 0 ? tile : tile - p.side[0].tiles) * kGM + row;
            // kCols rank columns of this wide column to the gradient
            auto store = [&](int c0, const float (&v)[kCols]) {
                if (col >= side.cols) return;
#pragma unroll
                for (int g = 0; g < kCols; g += 8) {
                    const int c = c0 + g;
                    if (c >= p.r) break;
                    if (sd == 0) {
                        uint16_t* o = side.out + (static_cast<int64_t>(a) * p.r + c) * side.cols + col;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            reinterpret_cast<__nv_bfloat16*>(o)[static_cast<int64_t>(k) * side.cols] = __float2bfloat16(v[g + k]);
                    } else {
                        *reinterpret_cast<uint4*>(side.out + (static_cast<int64_t>(a) * side.cols + col) * p.r + c) =
                            make_uint4(pack_bf16x2(v[g], v[g + 1]), pack_bf16x2(v[g + 2], v[g + 3]),
                                       pack_bf16x2(v[g + 4], v[g + 5]), pack_bf16x2(v[g + 6], v[g + 7]));
                    }
                }
            };
            const size_t slot = static_cast<size_t>(kGM) * p.r;
            // slot 1 of the CTA an item begins in, slot 0 of those it goes on in
            float* mine = c_lo == c_hi ? nullptr : p.sums + (2 * blockIdx.x + (blockIdx.x == c_lo ? 1 : 0)) * slot + row;
            // the four warps go on, or give up, together
            const bool ok = warp_wait(&ctl->acc_full[buf], round, abort_flag, p.status, 64);
            if (!all_of_128(ok)) break;
            tc_fence_after();
            for (int c = 0; c < p.r; c += kCols) {
                uint32_t u[kCols];
                const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * buf_cols + c;
                tmem_ld_32x32b_x16(ta, u);
                tmem_ld_wait();
                float v[kCols];
#pragma unroll
                for (int k = 0; k < kCols; ++k) v[k] = __uint_as_float(u[k]);
                if (mine) {
#pragma unroll
                    for (int k = 0; k < kCols; ++k)
                        if (c + (k & ~7) < p.r) __stcg(mine + (c + k) * kGM, v[k]);
                } else {
                    store(c, v);
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->acc_empty[buf]);
            if (mine) {
                // the four warps' sums are out before the arrival is counted
                __threadfence();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (warp == 6 && lane == 0) {
                    uint32_t before;
                    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.counter + c_lo) : "memory");
                    ctl->last = before == static_cast<uint32_t>(c_hi - c_lo) ? 1 : 0;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                const bool last = *reinterpret_cast<volatile int*>(&ctl->last) != 0;
                if (last) {
                    __threadfence();
                    // in block order; a part's columns are all in flight together, and the
                    // next part's with them
                    for (int c = 0; c < p.r; c += kCols) {
                        auto load = [&](int64_t j, float (&x)[kCols]) {
                            const float* part = p.sums + (2 * j + (j == c_lo ? 1 : 0)) * slot + row;
#pragma unroll
                            for (int k = 0; k < kCols; ++k) x[k] = c + (k & ~7) < p.r ? __ldcg(part + (c + k) * kGM) : 0.f;
                        };
                        float v[kCols], x[kCols];
                        load(c_lo, v);
                        load(c_lo + 1, x);  // (at least two parts)
                        for (int64_t j = c_lo + 1; j <= c_hi; ++j) {
                            float y[kCols];
                            if (j < c_hi) load(j + 1, y);
#pragma unroll
                            for (int k = 0; k < kCols; ++k) {
                                v[k] += x[k];
                                x[k] = y[k];
                            }
                        }
                        store(c, v);
                    }
                }
                // (ctl->last is rewritten only after the next item's first barrier, which
                // every reader reaches after reading it)
            }
        }
    }

    pdl_wait();  // this grid does not end before the one before it
    // (a CTA that starts after this finds no flag and waits, for a grid that has ended)
    if (p.ready && blockIdx.x == 0 && threadIdx.x == 0) *p.ready = 0;
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * buf_cols);
    }
}

template <int RING, int CTAS, int CHUNK>
int launch_grad(const GradMaps& m, GradParams p, bool after_kernel, cudaStream_t st) {
    constexpr size_t smem = 1024 + RING;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) { record_cuda_error(e); return GG_ERR_CUDA; }
    if (dev < 0 || dev >= 64) dev = 0;
    static std::atomic<bool> smem_set[64];
    if (!smem_set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(grad_kernel<RING, CTAS, CHUNK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem));
        if (e != cudaSuccess) { record_cuda_error(e); return GG_ERR_CUDA; }
        smem_set[dev].store(true, std::memory_order_release);
    }
    p.stages = RING / p.stage_bytes;
    if (p.stages > kGMaxStages) p.stages = kGMaxStages;
    int64_t G = int64_t(CTAS) * num_sms();  // every CTA resident at once
    if (G > kGradCtas) G = kGradCtas;
    ClusterLaunch l(G, kGThreads, smem, 1, after_kernel, st);
    clear_pending_launch_error();
    e = cudaLaunchKernelEx(&l.cfg, grad_kernel<RING, CTAS, CHUNK>, m, p);
    if (e != cudaSuccess) { record_cuda_error(e); return GG_ERR_CUDA; }
    return launch_result();
}

}  // namespace

int lora_grad_launch(const uint16_t* X, const uint16_t* dY, const uint16_t* U, const uint16_t* V_hi, const uint16_t* V_lo,
                     const PlanView& plan, int64_t K, int64_t N, int r, uint16_t* dA, uint16_t* dB, uint32_t* counters,
                     float* sums, GradAfter after, int32_t* status, cudaStream_t st) {
    GradParams p{};
    const bool kernel = after != GRAD_AFTER_OTHER;
    p.plan = plan;
    p.r = r;
    const int chunk = rank_pad(r);
    p.nc = (r + chunk - 1) / chunk;
    p.counter = counters;
    p.ready = after == GRAD_AFTER_DX ? counters + kGradCtas : nullptr;
    p.sums = sums;
    p.status = status;
    if (dA)
        p.side[0] = GradSide{X, {V_hi, V_lo}, 2, static_cast<int>(K), static_cast<int>((K + kGM - 1) / kGM), dA};
    if (dB)
        p.side[1] = GradSide{dY, {U, nullptr}, 1, static_cast<int>(N), static_cast<int>((N + kGM - 1) / kGM), dB};
    p.stage_bytes = kGWide + chunk * kGK * 2 * p.nc * (dA ? 2 : 1);
    GradMaps m{};
    if (dA) {
        if (!encode_map_2d(&m.wide[0], X, K, plan.T, K, 64, kGK)) return GG_ERR_CUDA;
        if (!encode_map_2d(&m.narrow[0], V_hi, r, plan.T, r, chunk, kGK)) return GG_ERR_CUDA;
        if (!encode_map_2d(&m.narrow[1], V_lo, r, plan.T, r, chunk, kGK)) return GG_ERR_CUDA;
    }
    if (dB) {
        if (!encode_map_2d(&m.wide[1], dY, N, plan.T, N, 64, kGK)) return GG_ERR_CUDA;
        if (!encode_map_2d(&m.narrow[2], U, r, plan.T, r, chunk, kGK)) return GG_ERR_CUDA;
    }
    // two CTAs an SM for ranks up to 64, one above
    if (chunk == 16) return launch_grad<98304, 2, 16>(m, p, kernel, st);
    if (chunk == 32) return launch_grad<98304, 2, 32>(m, p, kernel, st);
    return p.nc == 1 ? launch_grad<98304, 2, 64>(m, p, kernel, st) : launch_grad<196608, 1, 64>(m, p, kernel, st);
}

}  // namespace gg
