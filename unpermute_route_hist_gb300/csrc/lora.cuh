// lora.cuh -- what the low-rank adapter kernels share: the plan of a batch's
// adapter ids (which adapters occur among which rows), masked tensor-core
// products, and the reads of a cluster partner's shared memory.
//
// Low-rank adapters beside a shared projection: token t with adapter a has
//   U[t] = scale[a] X[t] A[a]^T,   Y[t] = X[t] W^T + U[t] B[a]^T.
// Rows stay in token order.  The shared product is one dense GEMM; an adapter's
// part is added to the same accumulator by one masked MMA per (row tile, adapter
// that occurs in it), whose mask keeps the other rows' accumulators untouched
// (not multiplied by zero: an infinity in one adapter never reaches another
// request's rows).
#pragma once

#include <atomic>

#include "common.cuh"

namespace gg {

constexpr int kUnit = 256;          // rows of a plan unit (one 2-CTA tile)
constexpr int kUnitWords = kUnit / 32;
constexpr int kLoraMaxRank = 256;

// The plan of one batch's ids, as laid out in the caller's buffer.
//   slots    entries a unit has room for: min(L, 256)
//   ntile    [1]                row tiles in adapter order (below)
//   cnt      [units]            adapters that occur in the unit's rows
//   gid      [units][slots]     those adapters, ascending
//   mask     [units][slots][8]  the rows of each, a bit a row
//   any      [units][8]         the rows that have an adapter
//   start    [units][slots]     rows of that adapter in earlier units
//   goff     [L + 1]            first position of each adapter's rows in order
//   toff     [L + 1]            first tile of each adapter
//   boff     [L + 1]            64-row blocks of the adapters before each
//   block    [max_blocks] int4  {adapter, position in order, rows, first row if the
//                               rows are neighbours, else -1}: up to 64 rows of one
//                               adapter; of an adapter's last, rows + kLastBlock
//   order    [T]                rows sorted by adapter, ascending inside one
//   tile     [max_tiles] int4   {adapter, position in order, rows, first row if the
//                               rows are neighbours in memory, else -1}: up to 128
//                               rows of one adapter
struct PlanView {
    int64_t T;
    int L, slots;
    int64_t units, max_tiles, max_blocks;
    int32_t* ntile;
    int32_t* cnt;
    int32_t* gid;
    uint32_t* mask;
    uint32_t* any;
    int32_t* start;
    int32_t* goff;
    int32_t* toff;
    int32_t* boff;
    int32_t* order;
    int4* tile;
    int4* block;
};

constexpr int kTileRows = 128;
constexpr int kBlockRows = 64;
constexpr int kLastBlock = 1 << 16;

// The plan's layout over buf (null: only the size matters); its bytes in *bytes.
inline PlanView plan_view(void* buf, int64_t T, int L, size_t* bytes = nullptr) {
    PlanView v{};
    v.T = T;
    v.L = L;
    v.units = (T + kUnit - 1) / kUnit;
    v.slots = L < kUnit ? L : kUnit;
    v.max_tiles = T / kTileRows + (T < L ? T : L);
    v.max_blocks = T / kBlockRows + (T < L ? T : L);
    size_t at = 0;
    auto take = [&](int64_t n, int64_t size) {
        void* p = static_cast<uint8_t*>(buf) + at;
        at += static_cast<size_t>((n * size + 255) / 256 * 256);
        return p;
    };
    v.ntile = static_cast<int32_t*>(take(1, 4));
    v.cnt = static_cast<int32_t*>(take(v.units, 4));
    v.gid = static_cast<int32_t*>(take(v.units * v.slots, 4));
    v.mask = static_cast<uint32_t*>(take(v.units * v.slots, 32));
    v.any = static_cast<uint32_t*>(take(v.units, 32));
    v.start = static_cast<int32_t*>(take(v.units * v.slots, 4));
    v.goff = static_cast<int32_t*>(take(static_cast<int64_t>(L) + 1, 4));
    v.toff = static_cast<int32_t*>(take(static_cast<int64_t>(L) + 1, 4));
    v.boff = static_cast<int32_t*>(take(static_cast<int64_t>(L) + 1, 4));
    v.order = static_cast<int32_t*>(take(T, 4));
    v.tile = static_cast<int4*>(take(v.max_tiles, 16));
    v.block = static_cast<int4*>(take(v.max_blocks, 16));
    if (bytes) *bytes = at;
    return v;
}
inline size_t plan_bytes_of(int64_t T, int L) {
    size_t b = 0;
    plan_view(nullptr, T, L, &b);
    return b;
}

// Width, in reduction columns, of an adapter's block beside the shared product:
// the rank rounded up to 16, 32 or 64 (ranks above 64: chunks of 64).  64 / rpad
// adapters share one stage of the operand ring.
__host__ __device__ constexpr int rank_pad(int r) { return r <= 16 ? 16 : (r <= 32 ? 32 : 64); }

// Shared-memory descriptor layout code of a K-major tile whose rows are rpad bf16.
constexpr uint32_t kLayoutSw32 = 6;
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t addr, int row_bytes) {
    const uint32_t layout = row_bytes == 32 ? kLayoutSw32 : (row_bytes == 64 ? kLayoutSw64 : kLayoutSw128);
    return smem_desc(addr, 16, 8 * row_bytes, layout);
}

// The same for an operand read along its columns (MN-major): reduction rows of
// row_bytes (32, 64 or 128), chunks of that width chunk_bytes apart.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t addr, int row_bytes, uint32_t chunk_bytes) {
    const uint32_t layout = row_bytes == 32 ? kLayoutSw32 : (row_bytes == 64 ? kLayoutSw64 : kLayoutSw128);
    return smem_desc(addr, chunk_bytes, 8 * row_bytes, layout);
}

// idesc_bf16_f32 for a column count known at run time.
__device__ __forceinline__ uint32_t idesc_bf16_f32_n(int M, int N, int a_mn_major, int b_mn_major) {
    return (idesc_bf16_f32(M, 0, a_mn_major, b_mn_major)) | (static_cast<uint32_t>(N >> 3) << 17);
}

// The producer and issuer warps run as whole warps: every lane walks the loop and
// waits, one elected lane issues.  Addresses and descriptors then are the same in every
// lane, which lets them live in uniform registers; with lane 0 alone on a divergent
// path 8192 rows of 4096 -> 6144 took 256 us, 239 this way, and 777 rows 20 and 18.6.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// Every lane waits for the phase; true if all of them saw it (bounded, as mbar_wait).
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status,
                                         bool cluster_scope = false) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status, 0, kWaitLimitNs, cluster_scope));
}

// A descriptor as its two halves: addresses advance the low one (16-byte units).
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ explicit Desc(uint64_t d) : lo(static_cast<uint32_t>(d)), hi(static_cast<uint32_t>(d >> 32)) {}
};

// D[tmem] (+)= A[smem] * B[smem]^T, a and b units of 16 bytes past the descriptors.
template <bool PAIR>
__device__ __forceinline__ void umma_at(uint32_t d_tmem, const Desc& A, uint32_t a, const Desc& B, uint32_t b,
                                        uint32_t idesc, uint32_t accumulate) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
            "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
            "r"(A.lo + a), "r"(A.hi), "r"(B.lo + b), "r"(B.hi), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
            "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
            "r"(A.lo + a), "r"(A.hi), "r"(B.lo + b), "r"(B.hi), "r"(idesc), "r"(accumulate)
            : "memory");
}
// D[tmem] += A[smem] * B[smem]^T for the rows whose mask bit is set; the other rows'
// accumulators are not written (the MMA's disable-output-lane operand).
__device__ __forceinline__ void umma_rows_at(uint32_t d_tmem, const Desc& A, uint32_t a, const Desc& B, uint32_t b,
                                             uint32_t idesc, const uint32_t (&keep)[4]) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, 1, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, {%6, %7, %8, %9}, p;\n\t}" ::"r"(d_tmem),
        "r"(A.lo + a), "r"(A.hi), "r"(B.lo + b), "r"(B.hi), "r"(idesc), "r"(~keep[0]), "r"(~keep[1]), "r"(~keep[2]),
        "r"(~keep[3])
        : "memory");
}
__device__ __forceinline__ void umma_rows_pair_at(uint32_t d_tmem, const Desc& A, uint32_t a, const Desc& B, uint32_t b,
                                                  uint32_t idesc, const uint32_t (&keep)[8]) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, 1, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, {%6, %7, %8, %9, %10, %11, %12, %13}, p;\n\t}" ::"r"(d_tmem),
        "r"(A.lo + a), "r"(A.hi), "r"(B.lo + b), "r"(B.hi), "r"(idesc), "r"(~keep[0]), "r"(~keep[1]), "r"(~keep[2]),
        "r"(~keep[3]), "r"(~keep[4]), "r"(~keep[5]), "r"(~keep[6]), "r"(~keep[7])
        : "memory");
}

// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Four floats of a cluster CTA's shared memory (a shared::cluster address).
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t mapa_addr(uint32_t addr, uint32_t cta) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(cta));
    return remote;
}

// This thread's reads through the async proxy (TMA) come after what is visible to it here.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Programmatic dependent launch: let the next kernel of the stream start its
// prologue; wait until the previous one has finished and its writes are visible
// (at once when this kernel was launched without the attribute).
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    fence_proxy_async();  // its stores, before this thread's TMA reads of them
}

// A kernel started beside the one before it (dX's) that reads what the launch before that
// one wrote (V): the launch order starts it late enough, but only griddepcontrol.wait or a
// release it has acquired makes the writes visible, and the wait would last until dX's end.
// So dX's kernel, once it has waited itself, releases a flag (its first CTA's producer:
// the wait covers the whole grid before), and the reader acquires it, or waits after all
// where the flag is not there.  V's kernel clears the flag, and the reader when it ends.
constexpr uint32_t kReadyFlag = 0x56d2a91eu;
// A whole warp, after pdl_wait() and before pdl_launch_dependents().
__device__ __forceinline__ void release_ready(uint32_t* flag) {
    if (flag && blockIdx.x == 0 && lane_id() == 0) {
        asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(flag), "r"(kReadyFlag) : "memory");
        __threadfence();  // performed before the launch that looks for it
    }
    __syncwarp();
}
__device__ __forceinline__ bool acquire_ready(const uint32_t* flag) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    return v == kReadyFlag;
}

// The sum of four floats at the same shared-memory offset in CTAs 0 .. n-1 of the
// cluster (at most 8), in that order; all reads are in flight together.
__device__ __forceinline__ float4 cluster_sum4(uint32_t addr, int n) {
    float4 x[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c < n) x[c] = ld_cluster_f32x4(mapa_addr(addr, static_cast<uint32_t>(c)));
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        if (c < n) {
            s.x += x[c].x;
            s.y += x[c].y;
            s.z += x[c].z;
            s.w += x[c].w;
        }
    }
    return s;
}

__device__ __forceinline__ uint2 pack_bf16x4(const float4& s) {
    return make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

// ------------------------------------------------------------------ host --

bool encode_map_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                   uint64_t row_stride_elems, uint32_t box_inner, uint32_t box_outer);
bool encode_map_3d(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                   uint64_t stride1_elems, uint64_t stride2_elems, uint32_t b0, uint32_t b1);
int num_sms();

// Launch of a kernel in clusters of S CTAs.
struct ClusterLaunch {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    ClusterLaunch(int64_t grid, int threads, size_t smem, int S, bool after_start, cudaStream_t st) : cfg{} {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(S);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        // may start while the kernel before it runs (griddepcontrol)
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = after_start ? 2 : 1;
    }
    ClusterLaunch(const ClusterLaunch&) = delete;
};

constexpr int kMaxCluster = 8;

// An empty kernel of the same block shape: the occupancy query answers one CTA an SM
// for every kernel that allocates tensor memory, although two are resident at once
// (measured: 304 CTAs of 100 KB, each with 128 TMEM columns, ran together).
static __global__ void __launch_bounds__(192, 2) cluster_room_kernel() {}

// Per kernel: the shared-memory opt-in and how many clusters of 1 .. 8 CTAs of 192
// threads are resident at once with smem bytes, asked once per device.  GG_OK or an
// error code.
struct ClusterRoom {
    std::atomic<int> n[64][kMaxCluster + 1];  // 0: not asked yet
    template <typename K>
    int get(K kern, size_t smem, int (&room)[kMaxCluster + 1]) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) { record_cuda_error(e); return GG_ERR_CUDA; }
        if (dev < 0 || dev >= 64) dev = 0;
        if (n[dev][kMaxCluster].load(std::memory_order_acquire) == 0) {
            const int bytes = static_cast<int>(smem);
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(cluster_room_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
            for (int S = 1; S <= kMaxCluster && e == cudaSuccess; ++S) {
                ClusterLaunch l(int64_t(S) * 1024, 192, smem, S, false, nullptr);
                int c = 0;
                e = cudaOccupancyMaxActiveClusters(&c, cluster_room_kernel, &l.cfg);
                if (e == cudaSuccess && c < 1) e = cudaErrorInvalidConfiguration;
                if (e == cudaSuccess) n[dev][S].store(c, std::memory_order_release);
            }
            if (e != cudaSuccess) { record_cuda_error(e); return GG_ERR_CUDA; }
        }
        for (int S = 1; S <= kMaxCluster; ++S) room[S] = n[dev][S].load(std::memory_order_acquire);
        return GG_OK;
    }
};

// U = scale X A^T (B_MN false; A [L, r, K]) or V = scale dY B (B_MN true; B [L, N, r]).
// parts (if any): the product as two bf16, the second `part` elements after the first.
// zero (if any): zero_words 32-bit words that the launch also clears.
int lora_shrink_launch(bool b_mn, const uint16_t* X, const uint16_t* ad, const float* scale, const PlanView& plan,
                       int64_t Kred, int r, uint16_t* out, uint16_t* parts, int64_t part, uint32_t* zero,
                       int zero_words, int32_t* status, cudaStream_t st);
// Y = X W^T + U B^T (b_mn false) or dX = dY W + V A (b_mn true): split-reduction
// clusters for few row tiles, 2-CTA pair tiles otherwise.  ready (or null): a cleared word
// to release once U (V) can be read, for the gradients' kernel.
int lora_project_launch(bool b_mn, const uint16_t* X, const uint16_t* W, const uint16_t* U, const uint16_t* ad,
                        const PlanView& plan, int64_t Kred, int64_t ncols, int r, uint16_t* out, uint32_t* ready,
                        int32_t* status, cudaStream_t st);
int lora_pair_launch(bool b_mn, const uint16_t* X, const uint16_t* W, const uint16_t* U, const uint16_t* ad,
                     const PlanView& plan, int64_t Kred, int64_t ncols, int r, uint16_t* out, uint32_t* ready,
                     int32_t* status, cudaStream_t st);
// dA, dB (either may be null) from V's two parts and U; counters: kGradCtas zeroed words, and the flag that dX's
// kernel releases; sums: the CTAs' partial sums, 2 x kGradCtas x 128 x r floats.
constexpr int kGradCtas = 320;
constexpr int kGradWords = kGradCtas + 1;
// What was launched just before: V's kernel, dX's (itself after V's), or something else.
enum GradAfter { GRAD_AFTER_V, GRAD_AFTER_DX, GRAD_AFTER_OTHER };
int lora_grad_launch(const uint16_t* X, const uint16_t* dY, const uint16_t* U, const uint16_t* V_hi, const uint16_t* V_lo,
                     const PlanView& plan, int64_t K, int64_t N, int r, uint16_t* dA, uint16_t* dB, uint32_t* counters,
                     float* sums, GradAfter after, int32_t* status, cudaStream_t st);
int lora_plan_launch(const int32_t* ids, const PlanView& plan, int32_t* status, cudaStream_t st);

}  // namespace gg
