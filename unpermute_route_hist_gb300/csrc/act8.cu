// act8.cu -- activations kept in 8 bits: rows to codes and back (optionally gathered into
// expert order), and the gated activation's backward from the kept pre-activation.
// The forward that keeps it is the grouped GEMM's (gemm_act8.cu).
//
// All three stream their tensors once and are bound by HBM.  Work is flat over pieces of
// 16 columns (8 where rows or addresses have no 32-byte alignment; 8 activations) of all
// rows, so narrow rows fill warps as wide ones do; a CTA finds the row of its first piece
// by one 64-bit division, the others from it by a multiplication.
#include <type_traits>

#include "act8.cuh"

namespace gg {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 2;  // pieces a thread, their loads in flight together
constexpr int kUnpackVecs = 4;

__device__ __forceinline__ uint4 ld_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// the same with an L2 policy; codes, W = 16 or 8 of them
__device__ __forceinline__ uint64_t l2_policy_evict_last() {
    uint64_t pol;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}
template <int W>
__device__ __forceinline__ uint4 ld_codes(const void* p, uint64_t pol) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if constexpr (W == 16)
        asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p), "l"(pol));
    else
        asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v2.u32 {%0, %1}, [%2], %3;"
                     : "=r"(v.x), "=r"(v.y)
                     : "l"(p), "l"(pol));
    return v;
}

__device__ __forceinline__ void bf16x2_floats(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
}

__device__ __forceinline__ void ld_stream32(const void* p, uint4& a, uint4& b) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
}
__device__ __forceinline__ void st_32(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// W elements as loaded, 16 bytes at a time, or whole 32-byte sectors (W = 16: aligned).
template <int DT, int W>
struct Raw {
    static constexpr int kQuads = W * (DT == GG_DTYPE_F32 ? 4 : 2) / 16;
    uint4 q[kQuads];
    __device__ __forceinline__ void load(const void* p, int64_t elem) {
        const char* at = static_cast<const char*>(p) + elem * (DT == GG_DTYPE_F32 ? 4 : 2);
        if constexpr (W == 16) {
#pragma unroll
            for (int i = 0; i < kQuads; i += 2) ld_stream32(at + 16 * i, q[i], q[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < kQuads; ++i) q[i] = ld_stream(at + 16 * i);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) q[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void floats(float (&f)[W]) const {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (DT == GG_DTYPE_F32) {
                    f[4 * i + k] = __uint_as_float(w[k]);
                } else if constexpr (DT == GG_DTYPE_BF16) {
                    bf16x2_floats(w[k], f[8 * i + 2 * k], f[8 * i + 2 * k + 1]);
                } else {
                    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                    f[8 * i + 2 * k] = p.x;
                    f[8 * i + 2 * k + 1] = p.y;
                }
            }
        }
    }
};

template <int DT, int W>
__device__ __forceinline__ void store(void* p, int64_t elem, const float (&f)[W], uint64_t pol) {
    constexpr int kQuads = W * (DT == GG_DTYPE_F32 ? 4 : 2) / 16;
    char* at = static_cast<char*>(p) + elem * (DT == GG_DTYPE_F32 ? 4 : 2);
    uint4 q[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (DT == GG_DTYPE_F32) {
                w[k] = __float_as_uint(f[4 * i + k]);
            } else if constexpr (DT == GG_DTYPE_BF16) {
                w[k] = pack_bf16x2(f[8 * i + 2 * k], f[8 * i + 2 * k + 1]);
            } else {
                const __half2 h = __floats2half2_rn(f[8 * i + 2 * k], f[8 * i + 2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if constexpr (W == 16) {
#pragma unroll
        for (int i = 0; i < kQuads; i += 2) st_global_32_policy(at + 16 * i, q[i], q[i + 1], pol);
    } else {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) st_global_16_policy(at + 16 * i, q[i], pol);
    }
}

// (row, vector) of this thread's vectors u = 0.. of the CTA's kThreads * VECS.
template <int VECS>
struct FlatRows {
    int64_t row0;
    uint32_t v0;
    FastDiv per_row;
    __device__ __forceinline__ FlatRows(const FastDiv& q) : per_row(q) {
        const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * VECS);
        row0 = first / q.d;
        v0 = static_cast<uint32_t>(first - row0 * q.d);
    }
    __device__ __forceinline__ void at(int u, int64_t& row, uint32_t& v) const {
        const uint32_t x = v0 + u * kThreads + threadIdx.x;
        const uint32_t r = x / per_row;
        row = row0 + r;
        v = x - r * per_row.d;
    }
};

// A thread takes W columns; the neighbours of its block (pieces a row are padded to whole
// blocks, so one warp's) find the block's largest |x| by exchanges.  8192 x 4096 bf16: 17 us,
// 6.0 TB/s (with 8 columns a thread 18.3).
template <int DT, int FMT, int W>
__global__ void __launch_bounds__(kThreads)
act8_pack_kernel(const void* __restrict__ X, int64_t rows, int C, FastDiv vecs, uint8_t* __restrict__ codes,
                 uint8_t* __restrict__ scales, int scale_pitch) {
    const FlatRows<kVecs> flat(vecs);
    Raw<DT, W> raw[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        int64_t row;
        uint32_t v;
        flat.at(u, row, v);
        if (row < rows && W * v < static_cast<uint32_t>(C)) raw[u].load(X, row * C + W * v);
        else raw[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        int64_t row;
        uint32_t v;
        flat.at(u, row, v);
        float f[W], m = 0.f;
        raw[u].floats(f);
#pragma unroll
        for (int i = 0; i < W; ++i) m = amax_nan(m, f[i]);
#pragma unroll
        for (int d = 1; d < kActBlock / W; d <<= 1) m = amax_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
        const uint32_t s = act8_scale<FMT>(m);
        const float inv = act8_inverse(s);
        if (row >= rows) continue;
        uint32_t w[W / 4];
#pragma unroll
        for (int i = 0; i < W / 4; ++i) w[i] = act8_code4<FMT>(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], inv);
        uint8_t* to = codes + (row * vecs.d + v) * W;
        if constexpr (W == 16) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        if (v % (kActBlock / W) == 0) scales[row * scale_pitch + v / (kActBlock / W)] = static_cast<uint8_t>(s);
    }
}

// A thread writes W columns of an output row from its source row's codes and scale.  Bound
// by HBM: 8192 x 4096 as it is 17 us, each row twice in another order 29 us, 16384 x 2048 each
// row eight times 91 us (the copy rate: 15, 25, 84; 4.7 us are a launch's own).  Outputs leave
// L2 first and gathered codes last, or the outputs push out rows that are read again (34 and
// 122 us); gathered rows want four pieces' loads in flight (30 and 97 us with two).  What runs
// behind takes as long as with codes that leave like any line (dW of 8192 x 4096 twice 2.29 and
// 2.28 ms within a span of 2.13-2.32, of 16384 x 2048 eight times 657-672 and 671-682 us).
template <int DT, int FMT, int W>
__global__ void __launch_bounds__(kThreads)
act8_unpack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t src_rows, int C,
                   FastDiv vecs, int64_t code_pitch, int scale_pitch, const int32_t* __restrict__ gather_idx,
                   FastDiv div, int64_t rows, void* __restrict__ out, int32_t* status) {
    const FlatRows<kUnpackVecs> flat(vecs);
    int64_t from[kUnpackVecs];
#pragma unroll
    for (int u = 0; u < kUnpackVecs; ++u) {
        int64_t row;
        uint32_t v;
        flat.at(u, row, v);
        from[u] = row < rows ? row : -1;
        if (gather_idx && row < rows) {
            const int32_t f = gather_idx[row];
            from[u] = f < 0 ? -1 : static_cast<int64_t>(static_cast<uint32_t>(f) / div);
            if (from[u] < 0 || from[u] >= src_rows) {
                set_status(status, GG_DEV_BAD_ROW_INDEX);
                from[u] = -1;
            }
        }
    }
    const uint64_t first_out = l2_policy_evict_first(), keep = gather_idx ? l2_policy_evict_last() : first_out;
    uint4 w[kUnpackVecs];
    uint32_t s[kUnpackVecs];
#pragma unroll
    for (int u = 0; u < kUnpackVecs; ++u) {
        int64_t row;
        uint32_t v;
        flat.at(u, row, v);
        w[u] = make_uint4(0, 0, 0, 0);
        s[u] = 10;
        if (from[u] < 0) continue;
        w[u] = ld_codes<W>(codes + from[u] * code_pitch + W * v, keep);
        s[u] = scales[from[u] * scale_pitch + v / (kActBlock / W)];
    }
#pragma unroll
    for (int u = 0; u < kUnpackVecs; ++u) {
        int64_t row;
        uint32_t v;
        flat.at(u, row, v);
        if (row >= rows) continue;
        const float f = act8_factor(s[u]);
        const uint32_t word[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        float all[W];
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            float four[4];
            act8_value4<FMT>(word[i], f, four);
#pragma unroll
            for (int k = 0; k < 4; ++k) all[4 * i + k] = four[k];
        }
        store<DT, W>(out, row * C + W * v, all, first_out);
    }
}

// A thread takes 8 activations: 16 codes (gate, up interleaved; half a block) and 8 of
// dA give 16 columns of dH and, when wanted, the activation again.  16384 x 14336 from int8:
// 337 us with the activation, 7.0 TB/s of its 2.36 GB, 282 without.  With four pieces a
// thread (72 registers) 362 us and with IEEE divisions 391: too few warps to hide the loads.
template <int FMT, bool AL32>
__global__ void __launch_bounds__(kThreads)
swiglu_bwd_act8_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                       const uint16_t* __restrict__ dA, int64_t rows, FastDiv vecs, int64_t code_pitch,
                       int scale_pitch, uint16_t* __restrict__ dH, uint16_t* __restrict__ A) {
    const FlatRows<kVecs> flat(vecs);
    uint4 w[kVecs], d[kVecs];
    uint32_t s[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        int64_t row;
        uint32_t v;
        flat.at(u, row, v);
        if (row < rows) {
            w[u] = ld_stream(codes + row * code_pitch + 16 * v);
            d[u] = ld_stream(dA + (row * vecs.d + v) * 8);
            s[u] = scales[row * scale_pitch + (v >> 1)];
        }
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        int64_t row;
        uint32_t v;
        flat.at(u, row, v);
        if (row >= rows) continue;
        const float f = act8_factor(s[u]);
        const uint32_t cw[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        const uint32_t dw[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
        uint32_t oh[8], oa[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float gu[4], da[2], a[2];
            act8_value4<FMT>(cw[i], f, gu);
            bf16x2_floats(dw[i], da[0], da[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float g = gu[2 * j], up = gu[2 * j + 1];
                const float sg = __fdividef(1.0f, 1.0f + __expf(-g));  // two steps off at most; 0 past 2^126
                oh[2 * i + j] = pack_bf16x2(da[j] * up * sg * (1.0f + g * (1.0f - sg)), da[j] * g * sg);
                a[j] = g * sg * up;
            }
            oa[i] = pack_bf16x2(a[0], a[1]);
        }
        const int64_t at = (row * vecs.d + v) * 8;
        const uint4 h0 = make_uint4(oh[0], oh[1], oh[2], oh[3]), h1 = make_uint4(oh[4], oh[5], oh[6], oh[7]);
        if constexpr (AL32) {
            st_32(dH + 2 * at, h0, h1);
        } else {
            reinterpret_cast<uint4*>(dH + 2 * at)[0] = h0;
            reinterpret_cast<uint4*>(dH + 2 * at)[1] = h1;
        }
        if (A) *reinterpret_cast<uint4*>(A + at) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
    }
}

// CTAs for rows of `vecs` vectors; 0: more than a grid takes.
unsigned flat_grid(int64_t rows, int64_t vecs, int pieces) {
    const int64_t per = kThreads * pieces;
    if (rows > INT64_MAX / vecs - per) return 0;
    const int64_t n = (rows * vecs + per - 1) / per;
    return n < (int64_t(1) << 31) ? static_cast<unsigned>(n) : 0;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// fn(dtype, fmt, width), each a constant.
template <typename F, typename FMT, typename W>
int by_type(int dtype, FMT fmt, W w, F fn) {
    if (dtype == GG_DTYPE_BF16) return fn(std::integral_constant<int, GG_DTYPE_BF16>(), fmt, w);
    if (dtype == GG_DTYPE_F16) return fn(std::integral_constant<int, GG_DTYPE_F16>(), fmt, w);
    return fn(std::integral_constant<int, GG_DTYPE_F32>(), fmt, w);
}
template <typename F, typename W>
int by_type(int dtype, int fmt, W w, F fn) {
    return fmt == GG_ACT8_INT8 ? by_type(dtype, std::integral_constant<int, GG_ACT8_INT8>(), w, fn)
                               : by_type(dtype, std::integral_constant<int, GG_ACT8_E4M3>(), w, fn);
}
template <typename F>
int by_type(int dtype, int fmt, bool wide, F fn) {
    return wide ? by_type(dtype, fmt, std::integral_constant<int, 16>(), fn)
                : by_type(dtype, fmt, std::integral_constant<int, 8>(), fn);
}

bool known(int dtype, int fmt) {
    return (dtype == GG_DTYPE_BF16 || dtype == GG_DTYPE_F16 || dtype == GG_DTYPE_F32) &&
           (fmt == GG_ACT8_INT8 || fmt == GG_ACT8_E4M3);
}

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

int gg_act8_pack(const void* X, int dtype, int64_t rows, int64_t C, int fmt, uint8_t* codes, uint8_t* scales,
                 void* stream) {
    if (rows < 0 || C < 0 || !known(dtype, fmt)) return GG_ERR_INVALID_ARG;
    if (C % 8 || C >= (int64_t(1) << 30)) return GG_ERR_UNSUPPORTED;
    if (rows == 0 || C == 0) return GG_OK;
    if (!X || !codes || !scales) return GG_ERR_INVALID_ARG;
    if (!al16(X) || !al16(codes) || !al4(scales)) return GG_ERR_UNSUPPORTED;
    const int64_t size = dtype == GG_DTYPE_F32 ? 4 : 2;
    if (rows > INT64_MAX / (2 * C * size)) return GG_ERR_UNSUPPORTED;
    const Span out[] = {{codes, rows * act8_code_pitch(C)}, {scales, rows * act8_scale_pitch(C)}}, in[] = {{X, rows * C * size}};
    if (outputs_overlap(out, in)) return GG_ERR_INVALID_ARG;
    const bool wide = C % 16 == 0 && al32(X);
    const int64_t vecs = act8_code_pitch(C) / (wide ? 16 : 8);
    const unsigned grid = flat_grid(rows, vecs, kVecs);
    if (!grid) return GG_ERR_UNSUPPORTED;
    clear_pending_launch_error();
    return by_type(dtype, fmt, wide, [&](auto dt, auto f, auto w) {
        act8_pack_kernel<dt(), f(), w()><<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            X, rows, static_cast<int>(C), fast_div(static_cast<uint32_t>(vecs)), codes, scales,
            static_cast<int>(act8_scale_pitch(C)));
        return launch_result();
    });
}

int gg_act8_unpack(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t src_rows, int64_t C,
                   const int32_t* gather_idx, int div, int64_t rows, void* out, int dtype, int32_t* status,
                   void* stream) {
    if (rows < 0 || src_rows < 0 || C < 0 || !known(dtype, fmt)) return GG_ERR_INVALID_ARG;
    if (gather_idx ? div < 1 : rows != src_rows) return GG_ERR_INVALID_ARG;
    if (C % 8 || C >= (int64_t(1) << 30)) return GG_ERR_UNSUPPORTED;
    if (rows == 0 || C == 0) return GG_OK;
    if (!out || (src_rows > 0 && (!codes || !scales))) return GG_ERR_INVALID_ARG;
    if (!al16(out) || !al16(codes) || !al4(scales) || !al4(gather_idx)) return GG_ERR_UNSUPPORTED;
    const int64_t size = dtype == GG_DTYPE_F32 ? 4 : 2;
    if (rows > INT64_MAX / (2 * C * size) || src_rows > INT64_MAX / (2 * C * size)) return GG_ERR_UNSUPPORTED;
    const Span outs[] = {{out, rows * C * size}};
    const Span ins[] = {{codes, src_rows * act8_code_pitch(C)}, {scales, src_rows * act8_scale_pitch(C)}, {gather_idx, rows * 4}};
    if (outputs_overlap(outs, ins)) return GG_ERR_INVALID_ARG;
    const bool wide = C % 16 == 0 && al32(out);
    const int64_t vecs = C / (wide ? 16 : 8);
    const unsigned grid = flat_grid(rows, vecs, kUnpackVecs);
    if (!grid) return GG_ERR_UNSUPPORTED;
    clear_pending_launch_error();
    return by_type(dtype, fmt, wide, [&](auto dt, auto f, auto w) {
        act8_unpack_kernel<dt(), f(), w()><<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            codes, scales, src_rows, static_cast<int>(C), fast_div(static_cast<uint32_t>(vecs)), act8_code_pitch(C),
            static_cast<int>(act8_scale_pitch(C)), gather_idx, fast_div(static_cast<uint32_t>(gather_idx ? div : 1)),
            rows, out, status);
        return launch_result();
    });
}

int gg_swiglu_bwd_act8(const uint8_t* codes, const uint8_t* scales, int fmt, const gg_bf16* dA, int64_t rows,
                       int64_t I, gg_bf16* dH, gg_bf16* A, void* stream) {
    if (rows < 0 || I < 0 || !known(GG_DTYPE_BF16, fmt)) return GG_ERR_INVALID_ARG;
    if (I % 8 || I >= (int64_t(1) << 29)) return GG_ERR_UNSUPPORTED;
    if (rows == 0 || I == 0) return GG_OK;
    if (!codes || !scales || !dA || !dH) return GG_ERR_INVALID_ARG;
    if (!al16(codes) || !al4(scales) || !al16(dA) || !al16(dH) || !al16(A)) return GG_ERR_UNSUPPORTED;
    const unsigned grid = flat_grid(rows, I / 8, kVecs);
    if (!grid) return GG_ERR_UNSUPPORTED;
    clear_pending_launch_error();
    if (rows > INT64_MAX / (8 * I)) return GG_ERR_UNSUPPORTED;
    const Span outs[] = {{dH, rows * I * 4}, {A, rows * I * 2}};
    const Span ins[] = {{codes, rows * act8_code_pitch(2 * I)}, {scales, rows * act8_scale_pitch(2 * I)}, {dA, rows * I * 2}};
    if (outputs_overlap(outs, ins)) return GG_ERR_INVALID_ARG;
    const bool a32 = al32(dH);
    auto kern = fmt == GG_ACT8_INT8
                    ? (a32 ? swiglu_bwd_act8_kernel<GG_ACT8_INT8, true> : swiglu_bwd_act8_kernel<GG_ACT8_INT8, false>)
                    : (a32 ? swiglu_bwd_act8_kernel<GG_ACT8_E4M3, true> : swiglu_bwd_act8_kernel<GG_ACT8_E4M3, false>);
    kern<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        codes, scales, dA, rows, fast_div(static_cast<uint32_t>(I / 8)), act8_code_pitch(2 * I),
        static_cast<int>(act8_scale_pitch(2 * I)), dH, A);
    return launch_result();
}

}  // extern "C"
