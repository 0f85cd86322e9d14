// lora_plan.cu -- the plan of a batch's adapter ids: for every unit of 256 rows
// the adapters that occur in it with the rows of each as a bit mask, and all rows
// sorted by adapter.  Integer work on 4 bytes a token; made once a batch and used
// by every projection of every layer.  The result is the same on every run: an
// entry's place is the rank of its adapter id in the unit's bitmap, a row's place
// the rank of its bit, no atomic hands out places.
//
// Bound by launches: up to 256 rows one CTA does everything in one launch (13 us a
// call from Python, 3 on the device), more take five (22 us at 8192 rows, 12 on the
// device).  Each of those needs the one before over all units: the units' entries, each
// adapter's rows over the units, the adapters' offsets, the rows' places, the tiles.
#include "lora.cuh"

namespace gg {
namespace {

constexpr int kBitWords = GG_MAX_EXPERTS / 32;

struct UnitShared {
    uint32_t bits[kBitWords];      // adapters that occur
    int32_t before[kBitWords];     // occurring adapters in earlier words
    uint32_t rows[kUnit][kUnitWords];
    // rank of adapter a among the occurring ones (a up to one past the last adapter)
    __device__ int rank(int a) const {
        if (a >= 32 * kBitWords) return before[kBitWords - 1] + __popc(bits[kBitWords - 1]);
        return before[a >> 5] + __popc(bits[a >> 5] & ((1u << (a & 31)) - 1u));
    }
};

// Unit u by 256 threads, a thread per row: its entries to the plan.  Returns this row's
// entry (-1: no adapter); their number in *n.
__device__ __forceinline__ int plan_unit(const int32_t* __restrict__ ids, const PlanView& v, int64_t u, UnitShared& s,
                                         int* n, int32_t* status) {
    const int tid = threadIdx.x;
    const int64_t t = u * kUnit + tid;
    for (int i = tid; i < kBitWords; i += kUnit) s.bits[i] = 0;
    for (int i = tid; i < kUnit * kUnitWords; i += kUnit) (&s.rows[0][0])[i] = 0;
    __syncthreads();
    int a = t < v.T ? ids[t] : -1;
    if (a < -1 || a >= v.L) {
        set_status(status, GG_DEV_BAD_ADAPTER_ID);
        a = -1;
    }
    if (a >= 0) atomicOr(&s.bits[a >> 5], 1u << (a & 31));
    __syncthreads();
    if (tid < 32) {  // exclusive prefix of the words' counts: two words a lane
        static_assert(kBitWords == 64, "two bitmap words a lane");
        const int c0 = __popc(s.bits[2 * tid]), c1 = __popc(s.bits[2 * tid + 1]);
        int x = c0 + c1;
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (tid >= d) x += y;
        }
        s.before[2 * tid] = x - c0 - c1;
        s.before[2 * tid + 1] = x - c1;
        if (tid == 31) v.cnt[u] = x;
    }
    __syncthreads();
    int j = -1;
    if (a >= 0) {
        j = s.rank(a);
        atomicOr(&s.rows[j][tid >> 5], 1u << (tid & 31));
        v.gid[u * v.slots + j] = a;  // the same value from every row of the adapter
    }
    __syncthreads();
    *n = s.rank(32 * kBitWords);
    for (int i = tid; i < *n * kUnitWords; i += kUnit) v.mask[u * v.slots * kUnitWords + i] = (&s.rows[0][0])[i];
    const uint32_t with = __ballot_sync(0xffffffffu, a >= 0);
    if ((tid & 31) == 0) v.any[u * kUnitWords + (tid >> 5)] = with;
    return j;
}

__global__ void __launch_bounds__(kUnit) plan_units_kernel(const int32_t* __restrict__ ids, PlanView v, int32_t* status) {
    __shared__ UnitShared s;
    int n;
    plan_unit(ids, v, blockIdx.x, s, &n, status);
}

// A batch of one unit (decode, short prompts): the whole plan in one CTA, one launch
// instead of five.
__global__ void __launch_bounds__(kUnit) plan_one_unit_kernel(const int32_t* __restrict__ ids, PlanView v, int32_t* status) {
    __shared__ UnitShared s;
    __shared__ int32_t rows[kUnit + 1], tiles[kUnit + 1], blocks[kUnit + 1];  // of the entries before each
    __shared__ int32_t order[kUnit];
    __shared__ int32_t sums[3][kUnit / 32];
    const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
    int n;
    const int j = plan_unit(ids, v, 0, s, &n, status);
    int c = 0;
    if (tid < n)
        for (int w = 0; w < kUnitWords; ++w) c += __popc(s.rows[tid][w]);
    // exclusive prefixes over the entries, a thread each
    int x[3] = {c, (c + kTileRows - 1) / kTileRows, (c + kBlockRows - 1) / kBlockRows};
    const int own[3] = {x[0], x[1], x[2]};
    for (int k = 0; k < 3; ++k) {
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x[k], d);
            if (lane >= d) x[k] += y;
        }
        if (lane == 31) sums[k][warp] = x[k];
    }
    __syncthreads();
    for (int k = 0; k < 3; ++k)
        for (int w = 0; w < warp; ++w) x[k] += sums[k][w];
    rows[tid] = x[0] - own[0];
    tiles[tid] = x[1] - own[1];
    blocks[tid] = x[2] - own[2];
    if (tid == kUnit - 1) {
        rows[kUnit] = x[0];
        tiles[kUnit] = x[1];
        blocks[kUnit] = x[2];
        *v.ntile = x[1];
    }
    __syncthreads();
    if (j >= 0) {
        int pos = rows[j];
        for (int w = 0; w < warp; ++w) pos += __popc(s.rows[j][w]);
        pos += __popc(s.rows[j][warp] & ((1u << lane) - 1u));
        order[pos] = tid;
        v.order[pos] = tid;
    }
    if (tid < n) v.start[tid] = 0;
    for (int a = tid; a <= v.L; a += kUnit) {  // (entries past the last hold its totals)
        const int k = s.rank(a);
        v.goff[a] = rows[k];
        v.toff[a] = tiles[k];
        v.boff[a] = blocks[k];
    }
    __syncthreads();
    if (tid < n) {
        const int a = v.gid[tid];
        auto entry = [&](int at, int m, int flags) {
            return make_int4(a, at, m + flags, order[at + m - 1] - order[at] == m - 1 ? order[at] : -1);
        };
        for (int i = 0; i * kTileRows < c; ++i)
            v.tile[tiles[tid] + i] = entry(rows[tid] + i * kTileRows, min(kTileRows, c - i * kTileRows), 0);
        for (int i = 0; i * kBlockRows < c; ++i)
            v.block[blocks[tid] + i] = entry(rows[tid] + i * kBlockRows, min(kBlockRows, c - i * kBlockRows),
                                             (i + 1) * kBlockRows >= c ? kLastBlock : 0);
    }
}

// One warp per adapter: its rows in each unit, summed in unit order into start;
// goff[a + 1] receives its total (the scan below makes offsets of them).
__global__ void __launch_bounds__(128) plan_groups_kernel(PlanView v) {
    const int a = static_cast<int>((static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5);
    const int lane = lane_id();
    if (a >= v.L) return;
    int run = 0;
    for (int64_t u0 = 0; u0 < v.units; u0 += 32) {
        const int64_t u = u0 + lane;
        int c = 0;
        int64_t at = -1;
        if (u < v.units) {
            int lo = 0, hi = v.cnt[u];
            const int32_t* g = v.gid + u * v.slots;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (g[mid] < a) lo = mid + 1; else hi = mid;
            }
            if (lo < v.cnt[u] && g[lo] == a) {
                at = u * v.slots + lo;
                for (int w = 0; w < kUnitWords; ++w) c += __popc(v.mask[at * kUnitWords + w]);
            }
        }
        int x = c;
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (at >= 0) v.start[at] = run + x - c;
        run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) v.goff[a + 1] = run;
}

// One warp: exclusive prefixes of the adapters' rows (in place), tiles and blocks.
__global__ void __launch_bounds__(32) plan_scan_kernel(PlanView v) {
    const int lane = lane_id();
    int rows = 0, tiles = 0, blocks = 0;
    for (int a0 = 0; a0 < v.L; a0 += 32) {
        const int a = a0 + lane;
        const int c = a < v.L ? v.goff[a + 1] : 0;
        int x = c, y = (c + kTileRows - 1) / kTileRows, z = (c + kBlockRows - 1) / kBlockRows;
        for (int d = 1; d < 32; d <<= 1) {
            const int xs = __shfl_up_sync(0xffffffffu, x, d), ys = __shfl_up_sync(0xffffffffu, y, d);
            const int zs = __shfl_up_sync(0xffffffffu, z, d);
            if (lane >= d) {
                x += xs;
                y += ys;
                z += zs;
            }
        }
        if (a < v.L) {
            v.goff[a + 1] = rows + x;
            v.toff[a + 1] = tiles + y;
            v.boff[a + 1] = blocks + z;
        }
        rows += __shfl_sync(0xffffffffu, x, 31);
        tiles += __shfl_sync(0xffffffffu, y, 31);
        blocks += __shfl_sync(0xffffffffu, z, 31);
    }
    if (lane == 0) {
        v.goff[0] = 0;
        v.toff[0] = 0;
        v.boff[0] = 0;
        *v.ntile = tiles;
    }
}

// Rows into adapter order: one CTA per unit, a warp per entry in turn, each lane
// placing its bit of every mask word.
__global__ void __launch_bounds__(kUnit) plan_order_kernel(PlanView v) {
    const int64_t u = blockIdx.x;
    const int lane = lane_id();
    for (int j = warp_id(); j < v.cnt[u]; j += kUnit / 32) {
        const int64_t at = u * v.slots + j;
        int32_t pos = v.goff[v.gid[at]] + v.start[at];
        for (int w = 0; w < kUnitWords; ++w) {
            const uint32_t m = v.mask[at * kUnitWords + w];
            if ((m >> lane) & 1u)
                v.order[pos + __popc(m & ((1u << lane) - 1u))] = static_cast<int32_t>(u * kUnit + w * 32 + lane);
            pos += __popc(m);
        }
    }
}

// The row tiles and blocks, a thread each: its adapter by bisection of the offsets.
__global__ void __launch_bounds__(128) plan_tiles_kernel(PlanView v) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    auto entry = [&](const int32_t* off, int rows, bool mark_last) {
        int lo = 0, hi = v.L - 1;  // the last adapter whose first entry is not past i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (off[mid] <= i) lo = mid; else hi = mid - 1;
        }
        const int at = v.goff[lo] + static_cast<int>(i - off[lo]) * rows;
        const int left = v.goff[lo + 1] - at, n = min(rows, left);
        const int first = v.order[at];
        return make_int4(lo, at, n + (mark_last && left <= rows ? kLastBlock : 0),
                         v.order[at + n - 1] - first == n - 1 ? first : -1);
    };
    if (i < v.toff[v.L]) v.tile[i] = entry(v.toff, kTileRows, false);
    if (i < v.boff[v.L]) v.block[i] = entry(v.boff, kBlockRows, true);
}

}  // namespace

int lora_plan_launch(const int32_t* ids, const PlanView& v, int32_t* status, cudaStream_t st) {
    clear_pending_launch_error();
    if (v.units == 1) {
        plan_one_unit_kernel<<<1, kUnit, 0, st>>>(ids, v, status);
        return launch_result();
    }
    plan_units_kernel<<<static_cast<unsigned>(v.units), kUnit, 0, st>>>(ids, v, status);
    plan_groups_kernel<<<static_cast<unsigned>((v.L + 3) / 4), 128, 0, st>>>(v);
    plan_scan_kernel<<<1, 32, 0, st>>>(v);
    plan_order_kernel<<<static_cast<unsigned>(v.units), kUnit, 0, st>>>(v);
    plan_tiles_kernel<<<static_cast<unsigned>((v.max_blocks + 127) / 128), 128, 0, st>>>(v);
    return launch_result();
}

}  // namespace gg
