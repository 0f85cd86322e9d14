// block_norm.cuh -- what the norms around a block and their gradients share (gg.h, "norms
// around a block"; block_norm.cu, block_norm_bwd.cu).
//
// Both directions read and write each row once and are bound by HBM.  A CTA takes token
// rows t, t + grid, ...: their rows come into a ring of shared-memory stages by bulk
// copies a few rows ahead (a combined token's expert rows by one copy each, issued by as
// many lanes), so loads never wait for a row's sums.  A thread owns the same 16 columns (a
// unit; half a block of the 8-bit form) of every row: the weights' and the column sums'
// registers live as long as the CTA.  Rows of more than 8192
// columns are shared by the two CTAs of a cluster.  Row sums are reduced in a fixed order, column sums
// in token order within a CTA and then over CTAs: results repeat bit for bit.
//
// With the loads hidden, instructions are what is left to run out of (a row of 4096
// columns moves in some 1400 SM cycles forward, 2000 backward), hence the packed fp32
// arithmetic, the instantiations without bounds (FULL), and two rows an iteration in the
// forward, whose sums share their exchanges and barriers.
#pragma once

#include <atomic>
#include <cmath>

#include "act8.cuh"

namespace gg {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxStages = 8;
constexpr int kMaxSlots = 32;           // expert rows of a stage, one lane each
constexpr int kSmemBudget = 228 * 1024;  // an SM's shared memory, for all its CTAs
constexpr int kGridSms = 152;  // (a constant: the workspace's size is asked for without a device)

struct Slot {
    float w;
    int ok;
};
// The head of a CTA's shared memory; the stages follow.
struct Ctl {
    uint64_t full[kMaxStages];
    uint64_t sent[2];  // the other CTA's sums have landed
    float few[2][2][kMaxThreads / 32];  // of one or two sums; zeros for warps that are not
    float red[2][kMaxThreads / 32][8];
    Slot slot[kMaxStages][kMaxSlots];
    float other[2][8];  // the sums of the CTA that has the row's other half, and whether it gave up
    int abort_flag;
    int pad[3];
};
static_assert(sizeof(Ctl) % 16 == 0, "stages are 16-byte aligned");

// ------------------------------------------------------------- pairs of fp32 --

using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pair(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(f32x2 p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float both(f32x2 p) {
    float a, b;
    split(p, a, b);
    return a + b;
}

// Sixteen columns as eight pairs.
struct Unit {
    f32x2 v[8];
};
__device__ __forceinline__ void bf16_pairs(uint32_t w, f32x2& v) {
    v = pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t bf16_pair(f32x2 p) {
    float a, b;
    split(p, a, b);
    return pack_bf16x2(a, b);
}

// Which 16 columns of a row a thread's unit is.
//   bf16 stream  columns 16 u ..: one 32-byte store, half a block of the 8-bit form
//   fp32 stream  four quads, columns 4 (u + j threads) ..: rows of 4-byte elements are
//                then read from shared memory without bank conflicts (16 neighbouring
//                ones are a 4-way conflict: 116 us for the backward of 8192 x 4096, int8)
// Shared-memory rows are followed by zeros up to one more unit (quad), where units past
// the row's end read, so reads have no bounds; stores have, unless FULL.
template <bool F32, bool FULL>
struct Cols {
    uint32_t at[F32 ? 4 : 1];  // where to read: unit or quad numbers
    uint32_t first, step;      // where they lie: unit, or first quad and its distance to the next
    int inside;                // halves, or a bit for each quad, inside the row

    __device__ __forceinline__ void init(int K) {
        if constexpr (F32) {
            step = blockDim.x;
            first = threadIdx.x;
            inside = 0;
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const uint32_t q = first + j * step;
                if (q < K / 4u) inside |= 1 << j;
                at[j] = min(q, K / 4u);
            }
        } else {
            step = 0;
            first = threadIdx.x;
            inside = max(0, min(2, (K - 16 * static_cast<int>(first)) / 8));
            at[0] = min(first, (K + 15) / 16u);
        }
    }
    __device__ __forceinline__ uint32_t quad(int j) const { return FULL ? first + j * step : at[F32 ? j : 0]; }
    __device__ __forceinline__ uint32_t unit() const { return FULL ? first : at[0]; }

    // columns 8 half .. 8 half + 7 of the unit from a row in shared memory
    __device__ __forceinline__ void get_bf16(const uint8_t* row, int half, f32x2* v) const {
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint2 w = *reinterpret_cast<const uint2*>(row + 8 * quad(2 * half + j));
                bf16_pairs(w.x, v[2 * j]);
                bf16_pairs(w.y, v[2 * j + 1]);
            }
        } else {
            const uint4 w = *reinterpret_cast<const uint4*>(row + 32 * unit() + 16 * half);
            bf16_pairs(w.x, v[0]);
            bf16_pairs(w.y, v[1]);
            bf16_pairs(w.z, v[2]);
            bf16_pairs(w.w, v[3]);
        }
    }
    // the same of a row of the residual stream
    __device__ __forceinline__ void get_stream(const uint8_t* row, int half, f32x2* v) const {
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 f = *reinterpret_cast<const float4*>(row + 16 * quad(2 * half + j));
                v[2 * j] = pair(f.x, f.y);
                v[2 * j + 1] = pair(f.z, f.w);
            }
        } else {
            get_bf16(row, half, v);
        }
    }
    // eight codes
    __device__ __forceinline__ void get_codes(const uint8_t* row, int half, uint32_t (&w)[2]) const {
        if constexpr (F32) {
            w[0] = *reinterpret_cast<const uint32_t*>(row + 4 * quad(2 * half));
            w[1] = *reinterpret_cast<const uint32_t*>(row + 4 * quad(2 * half + 1));
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(row + 16 * unit() + 8 * half);
            w[0] = u.x, w[1] = u.y;
        }
    }

    // fp32 vectors in global memory: weights (ones where there are none) ...
    __device__ __forceinline__ void get_weight(const float* w, Unit& u) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
            if (w && holds(j)) f = *reinterpret_cast<const float4*>(w + column(j));
            u.v[2 * j] = pair(f.x, f.y);
            u.v[2 * j + 1] = pair(f.z, f.w);
        }
    }
    __device__ __forceinline__ void get_weights(const float* w, const float* g, Unit& u) const {
        get_weight(w, u);
        if (g) {
            Unit x;
            get_weight(g, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) u.v[i] = mul2(u.v[i], x.v[i]);
        }
    }
    // ... and sums
    __device__ __forceinline__ void put_sums(float* to, const Unit& u) const {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (holds(j))
                asm volatile("st.global.v2.b64 [%0], {%1, %2};" ::"l"(to + column(j)), "l"(u.v[2 * j]), "l"(u.v[2 * j + 1])
                             : "memory");
    }

    // columns 4 j .. 4 j + 3 of the unit: inside the row, and which of the row
    __device__ __forceinline__ bool holds(int j) const { return FULL || (F32 ? (inside >> j) & 1 : j / 2 < inside); }
    __device__ __forceinline__ uint32_t column(int j) const { return F32 ? 4 * (first + j * step) : 16 * first + 4 * j; }

    // bf16 outputs; whole 32-byte sectors where the rows start at them (st32)
    __device__ __forceinline__ void put_bf16(uint8_t* row, int st32, const Unit& u) const {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = bf16_pair(u.v[i]);
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (holds(j)) *reinterpret_cast<uint2*>(row + 2 * column(j)) = make_uint2(w[2 * j], w[2 * j + 1]);
        } else if (FULL || (st32 && inside == 2)) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + 32 * first), "r"(w[0]),
                         "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        } else {
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (half < inside)
                    *reinterpret_cast<uint4*>(row + 32 * first + 16 * half) =
                        make_uint4(w[4 * half], w[4 * half + 1], w[4 * half + 2], w[4 * half + 3]);
        }
    }
    __device__ __forceinline__ void put_stream(uint8_t* row, int st32, const Unit& u) const {
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (holds(j))
                    asm volatile("st.global.v2.b64 [%0], {%1, %2};" ::"l"(row + 4 * column(j)), "l"(u.v[2 * j]),
                                 "l"(u.v[2 * j + 1])
                                 : "memory");
        } else {
            put_bf16(row, st32, u);
        }
    }
};

// Bytes of a row in shared memory: what is copied, then zeros up to one more unit of
// `unit` bytes, rounded to the next row's alignment.
__host__ __device__ constexpr int row_area(int copied, int unit) {
    return ((copied + unit - 1) / unit * unit + unit + 15) / 16 * 16;
}
__host__ __device__ constexpr int bf16_area(bool f32, int K) { return row_area(2 * K, f32 ? 8 : 32); }
__host__ __device__ constexpr int stream_area(bool f32, int K) { return row_area(f32 ? 4 * K : 2 * K, f32 ? 16 : 32); }
__host__ __device__ constexpr int code_area(bool f32, int K) {
    return row_area(static_cast<int>(act8_code_pitch(K)), f32 ? 4 : 16);
}
// The zeros behind a row's copied bytes.
__device__ __forceinline__ void zero_pad(uint8_t* row, int copied, int area) {
    for (int b = copied + 4 * static_cast<int>(threadIdx.x); b < area; b += 4 * static_cast<int>(blockDim.x))
        *reinterpret_cast<uint32_t*>(row + b) = 0;
}

// The integers that four int8 codes are, or four e4m3 codes' values: what they stand for
// but for their block's factor.
template <int FMT>
__device__ __forceinline__ void code_pairs(uint32_t w, f32x2& a, f32x2& b) {
    float f[4];
    act8_value4<FMT>(w, 1.f, f);
    a = pair(f[0], f[1]);
    b = pair(f[2], f[3]);
}

// ---------------------------------------------------------------------- rows --

// A whole row into shared memory; the bytes complete on the barrier.
__device__ __forceinline__ void bulk_row(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Four bytes into shared memory, asynchronously.
__device__ __forceinline__ void copy_word(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Sums of N = 1, 2 or up to 8 values over the CTA, the same bits in every thread, one
// barrier a call.  Within a warp halves of the lanes take halves of the values (9
// exchanges for eight values, not 40); then every warp adds the warps' sums itself.
// `turn` alternates between two buffers: one is written again only past the next
// call's barrier.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], Ctl* ctl, int turn) {
    constexpr int P = N <= 1 ? 1 : N <= 2 ? 2 : 8;  // values exchanged
    const int lane = lane_id(), warps = blockDim.x >> 5;
    float x[P];
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = i < N ? v[i < N ? i : 0] : 0.f;
    int bit = 16;
#pragma unroll
    for (int half = P / 2; half > 0; half >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = up ? x[i] : x[i + half], keep = up ? x[i + half] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
        }
    }
#pragma unroll
    for (int d = 16 / P; d > 0; d >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], d);
    // value i now lies in the 32 / P lanes from 32 / P * i on
    constexpr int L = 32 / P;
    if (warps == 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x[0], L * i);
        __syncwarp();
        return;
    }
    if constexpr (P <= 2) {
        // one or two values: every thread reads the warps' sums itself
        if ((lane & (L - 1)) == 0) ctl->few[turn][lane / L][warp_id()] = x[0];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
            for (int w = 0; w < warps; w += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&ctl->few[turn][i][w]);
                v[i] += (f.x + f.y) + (f.z + f.w);
            }
        }
    } else {
        if ((lane & (L - 1)) == 0) ctl->red[turn][warp_id()][lane / L] = x[0];
        __syncthreads();
        // lane l: value l % 8 of warps l / 8, l / 8 + 4, ...
        float s = 0.f;
        for (int w = lane / P; w < warps; w += L) s += ctl->red[turn][w][lane & (P - 1)];
#pragma unroll
        for (int d = 16; d >= P; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, s, i);
    }
}


// The barrier's phase, with a limit.  A wait that runs out raises the CTA's flag, which
// every thread reads behind the next barrier: the CTA leaves as one, and until it does
// nothing more is copied (the stage's phase is not over: a second fill would arrive on it).
__device__ __forceinline__ void wait_row(uint64_t* bar, uint32_t parity, Ctl* ctl, int32_t* status,
                                         uint64_t limit_ns = kWaitLimitNs) {
    (void)mbar_wait(bar, parity, &ctl->abort_flag, status, 0, limit_ns);
}
__device__ __forceinline__ bool given_up(const Ctl* ctl) {
    return *reinterpret_cast<const volatile int*>(&ctl->abort_flag) != 0;
}

// Row sums: over the CTA, or with SPLIT over the two CTAs of a cluster that have a row's
// halves (at most seven).  Each sends its sums to the other's shared memory, where they
// complete on a barrier (`call` counts the calls: two buffers in turn, each used again only
// behind the other's next sums).  Both add the same two numbers, so they hold the same bits.
// True: the caller drains its ring and leaves.  With the sums a CTA says whether it had given
// up, so the other leaves with the same row; one whose wait for the sums themselves runs out
// has sent its own already, and the other leaves when the next do not come.  (A barrier of
// the cluster in its place waits for the stores of the row before: 2048 x 16384 76 us forward
// and 90 backward from int8.)
template <int N, bool SPLIT>
__device__ __forceinline__ bool row_sum(float (&v)[N], Ctl* ctl, uint32_t& call, int32_t* status) {
    const uint32_t turn = call & 1u;
    cta_sum(v, ctl, turn);
    bool left = given_up(ctl);
    if constexpr (SPLIT) {
        if (threadIdx.x <= N) {
            float x = left ? 1.f : 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (threadIdx.x == i) x = v[i];
            st_async_u32_signal(&ctl->other[turn][threadIdx.x], &ctl->sent[turn], cluster_ctarank() ^ 1u, __float_as_uint(x));
        }
        if (threadIdx.x == 0) {
            int late = 0;
            if (!mbar_wait(&ctl->sent[turn], (call >> 1) & 1u, &late, status, 0, kWaitLimitNs, true))
                *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
        }
        __syncthreads();
        const volatile float* other = ctl->other[turn];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += other[i];
        left = given_up(ctl) || other[N] != 0.f;
    }
    ++call;
    return left;
}

// Behind a wait that ran out, here or in the CTA that has the rows' other halves: the copies
// issued so far land (or their waits run out as well) before the CTA leaves its shared memory.
// The thread that issued them.  (Not inline: its registers would spill others of the loops in
// front of it.)
__device__ __noinline__ void drain_ring(Ctl* ctl, int stages, int64_t issued, uint64_t limit_ns = kWaitLimitNs) {
    for (int s = 0; s < stages; ++s) {
        const int64_t n = issued / stages + (s < issued % stages ? 1 : 0);
        int dummy = 0;
        if (n > 0) (void)mbar_wait(&ctl->full[s], static_cast<uint32_t>(n - 1) & 1u, &dummy, nullptr, 0, limit_ns);
    }
}

// The diagnostic form of the kernels (gg_selftest_block_norm_wait, _bwd_wait): of one token's
// rows (their first stage, the first half) the copies are left out, so that the wait for them
// runs out, and each CTA records how it left.
constexpr uint64_t kProbeWaitNs = 20000000ull;  // for rows; 2 s still for the other CTA's sums
struct Probe {
    int64_t withheld = -1;
    int32_t* record = nullptr;  // [CTAs][3]: left early; stages filled and not waited for; fills of unfinished phases
};
// Thread 0's account of a CTA's ring.
template <bool ON>
struct Account {
    __device__ __forceinline__ void fill(Ctl*, int, int64_t) {}
    __device__ __forceinline__ void waited() {}
    __device__ __forceinline__ void drained() {}
    __device__ __forceinline__ void put(const Probe&, bool, int64_t) const {}
};
template <>
struct Account<true> {
    int64_t waits = 0;
    int bad = 0;
    bool drain = false;
    // the n-th fill of the ring is about to be issued
    __device__ __forceinline__ void fill(Ctl* ctl, int stages, int64_t n) {
        if (threadIdx.x == 0 && n >= stages)
            bad += mbar_try_wait(&ctl->full[n % stages], static_cast<uint32_t>(n / stages - 1) & 1u) ? 0 : 1;
    }
    __device__ __forceinline__ void waited() { ++waits; }
    __device__ __forceinline__ void drained() { drain = true; }
    __device__ __forceinline__ void put(const Probe& p, bool left, int64_t fills) const {
        if (threadIdx.x != 0) return;
        int32_t* r = p.record + 3 * static_cast<int64_t>(blockIdx.x);
        r[0] = left;
        r[1] = drain ? 0 : static_cast<int32_t>(fills - waits);
        r[2] = bad;
    }
};

// `sums`: the sums of a row that a cluster's two CTAs send each other, 0 where a CTA has whole rows.
__device__ __forceinline__ void init_ring(Ctl* ctl, int stages, uint32_t arrivals, int sums) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&ctl->full[s], arrivals);
        if (sums) {
            mbar_init(&ctl->sent[0], sums + 1);
            mbar_init(&ctl->sent[1], sums + 1);
        }
        ctl->abort_flag = 0;
        fence_barrier_init();
    }
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(ctl->few) / 4); i += blockDim.x) (&ctl->few[0][0][0])[i] = 0.f;
    if (sums) {  // (the other's barriers are there before anything is sent)
        __syncwarp();
        cluster_sync();
    } else {
        __syncthreads();
    }
}
// A CTA leaves only when what the other sends it has landed, or will not be sent.
__device__ __forceinline__ void leave_pair() {
    __syncwarp();
    cluster_sync();
}

// ---------------------------------------------------------------------- host --

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows of up to 8192 columns are one CTA's, wider ones two CTAs' of a cluster, each with the
// weights of its half in registers: the first's half is whole blocks of the 8-bit form and
// whole words of their scales.  (One CTA with two units a thread read its weights from L2 for
// every row: 2048 x 16384 95 us forward, 190 backward from int8.)
inline bool norm_split(int64_t K) { return K > 16 * kMaxThreads; }
inline int64_t norm_half(int64_t K) { return norm_split(K) ? (K / 2 + 127) / 128 * 128 : K; }
inline int norm_threads(int64_t K) { return static_cast<int>((norm_half(K) + 511) / 512 * 32); }
// CTAs that share an SM: 512 threads' worth, 16 at most.
inline int norm_per_sm(int64_t K) {
    const int n = kMaxThreads / norm_threads(K);
    return n < 16 ? n : 16;
}
// Stages of a CTA when per_sm CTAs share an SM, each with the 1 KB that every CTA takes;
// per_sm falls until there are at least two.
inline int64_t ring_room(int per_sm) { return kSmemBudget / per_sm - static_cast<int64_t>(sizeof(Ctl)) - 1024; }
// Rows under way at once.
inline int64_t norm_rows(int64_t K, int per_sm) { return norm_split(K) ? kGridSms * per_sm / 2 : kGridSms * per_sm; }
inline int ring_stages(int64_t stage_bytes, int& per_sm) {
    for (;; --per_sm) {
        const int64_t n = ring_room(per_sm) / stage_bytes;
        if (n >= 2 || per_sm == 1) return static_cast<int>(n < 1 ? 1 : n > kMaxStages ? kMaxStages : n);
    }
}

// The shared-memory opt-in, once per kernel and device.
inline int opt_in(const void* kern, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_result(e);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return GG_OK;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return cuda_result(e);
    done.fetch_or(bit, std::memory_order_release);
    return GG_OK;
}

// `rows` CTAs, or clusters of two.
template <typename P>
int launch(void (*kern)(const P), std::atomic<uint64_t>& done, const P& p, bool split, unsigned rows, int threads,
           size_t smem, cudaStream_t st) {
    const int rc = opt_in(reinterpret_cast<const void*>(kern), done);
    if (rc != GG_OK) return rc;
    clear_pending_launch_error();
    if (!split) {
        kern<<<rows, threads, smem, st>>>(p);
        return launch_result();
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * rows);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_result(cudaLaunchKernelEx(&cfg, kern, p));
}
}  // namespace
}  // namespace gg
