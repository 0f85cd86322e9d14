// rope.cu -- rotary positions on the heads of a projection, in place or not
// (wall_x backend.py: rope, rope_bwd, one position or one per axis and token).
//
// Pair i of a head turns by the angle pos[t] * f_i: x1' = m (x1 cos - x2 sin),
// x2' = m (x2 cos + x1 sin); the backward turns the gradient by the opposite
// angle.  Bound by reading and writing the heads once; q and k go in one launch.
//
// The angle: frequencies come as 64-bit fractions of a turn, so pos * f modulo one
// turn is the low half of a 64-bit integer product, exact for every position
// (a 32-bit product loses 2^-24 of the angle: 0.008 rad at position 131072), and
// cos and sin are taken of a reduced argument in fp32.  Each CTA computes them
// once for its tokens (shared memory) and applies them to all heads.
//
// 16384 tokens of 40 heads of 128 in place: 52 us on the device (graph replay), 6.4 TB/s, 94% of
// the rate of a copy; 54 us a call, 91%.
//
// A thread takes PV pairs at a time, the widest power of two that the rotated
// width, the head width, strides and addresses allow (16-byte accesses for
// ordinary heads, single elements for odd ones).
#include "common.cuh"

#include <cuda_fp16.h>

namespace gg {

int num_sms();

namespace {

constexpr int kRopeThreads = 128;  // 52 us against 54 with 256 on 16384 tokens of 40 heads, 28 against 30 out of place
constexpr int kRopeMaxTokens = 8;    // of a CTA
constexpr int kRopeMaxRot = 1024;

struct RopeHeads {
    const void* x;
    void* out;
    int64_t xt, xh, ot, oh;  // token and head strides, elements
    int n;
};

struct RopeParams {
    RopeHeads q, k;
    const int32_t* pos;   // [axes, T]
    const int64_t* step;  // [rot / 2] turns a position, 2^-64 each
    float m;
    int64_t T;
    int half;             // pairs of a head
    int tail;             // elements past the rotated part to copy (0: in place)
    int bound[3];         // first pair of axes 1, 2, 3
    int tokens;           // of a CTA
    int backward;
};

template <typename E> __device__ __forceinline__ float to_f(E x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename E> __device__ __forceinline__ E from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16(x); }

// The two products' roundings are spelled out, so that every variant gives the same bits.
__device__ __forceinline__ float turn1(float x1, float x2, float2 cs) { return fmaf(x1, cs.x, -__fmul_rn(x2, cs.y)); }
__device__ __forceinline__ float turn2(float x1, float x2, float2 cs) { return fmaf(x2, cs.x, __fmul_rn(x1, cs.y)); }

// N elements moved as one access of at most 16 bytes.
template <typename E, int N>
struct alignas(sizeof(E) * N) Vec {
    static_assert(sizeof(E) * N <= 16, "one access");
    E e[N];
};

// Division of a 31-bit number by a number fixed at launch.
struct FastDiv {
    uint32_t d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t x) : d(x), shift(0) {
        while ((uint64_t(1) << shift) < x) ++shift;
        mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - x)) / x + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// Dynamic shared memory: cos and sin of the CTA's tokens, [tokens][half] float2.  A
// token's pairs are stored two by two across its pieces (pair k of piece v at
// (k / 2) pieces + v), so that neighbouring threads read neighbouring 16 bytes:
// in pair order every 16-byte read meets a 4-way bank conflict, which bound the
// kernel.
template <typename E, int PV, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const RopeParams p, const FastDiv per, const FastDiv heads, const FastDiv half) {
    extern __shared__ __align__(16) float2 cs[];
    using V = Vec<E, PV>;
    constexpr int kPairs = PV > 1 ? 2 : 1;  // of a 16-byte read
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
    const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.T - t0));
    const uint32_t turns = static_cast<uint32_t>(p.half / PV);  // rotated pieces of a head; then copied ones
    for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(nt * p.half); i += kRopeThreads) {
        const uint32_t t = half.div(i);
        const int j = static_cast<int>(i - t * half.d);
        const int axis = (j >= p.bound[0]) + (j >= p.bound[1]) + (j >= p.bound[2]);
        const int64_t pos = p.pos[axis * p.T + t0 + t];
        // modulo one turn, as a signed fraction in [-1/2, 1/2)
        const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(pos) * static_cast<uint64_t>(p.step[j]));
        float s, c;
        sincospif(__ll2float_rn(turn) * 0x1p-63f, &s, &c);
        const uint32_t v = j / PV, k = j % PV;
        cs[t * p.half + ((k / kPairs) * turns + v) * kPairs + k % kPairs] = make_float2(p.m * c, p.backward ? -p.m * s : p.m * s);
    }
    __syncthreads();
    const uint32_t items = static_cast<uint32_t>(nt) * heads.d * per.d;
    for (uint32_t i = threadIdx.x; i < items; i += kRopeThreads) {
        const uint32_t th = per.div(i), v = i - th * per.d;
        const uint32_t t = heads.div(th), h = th - t * heads.d;
        const bool isq = h < static_cast<uint32_t>(p.q.n);
        const RopeHeads& g = isq ? p.q : p.k;
        const int64_t hh = isq ? h : h - p.q.n;
        const E* x = static_cast<const E*>(g.x) + (t0 + t) * g.xt + hh * g.xh;
        E* o = static_cast<E*>(g.out) + (t0 + t) * g.ot + hh * g.oh;
        if (v >= turns) {  // copied: two pieces, half of the copied part apart
            const uint32_t tail = static_cast<uint32_t>(p.tail / PV), copies = (tail + 1) / 2, c = v - turns;
            const V* s = reinterpret_cast<const V*>(x + 2 * p.half);
            V* d = reinterpret_cast<V*>(o + 2 * p.half);
            const V z1 = s[c];
            if (c + copies < tail) d[c + copies] = s[c + copies];
            d[c] = z1;
            continue;
        }
        // the piece's two parts: pairs' first and second elements, or (interleaved) PV
        // neighbouring elements and the PV after them
        const uint32_t at = INTER ? 2 * v * PV : v * PV, off = INTER ? PV : p.half;
        V z1 = *reinterpret_cast<const V*>(x + at), z2 = *reinterpret_cast<const V*>(x + at + off);
        const float2* a = cs + t * p.half + v * kPairs;
        E y[2 * PV];
        if (INTER) {
#pragma unroll
            for (int k = 0; k < PV; ++k) {
                y[k] = z1.e[k];
                y[PV + k] = z2.e[k];
            }
        }
#pragma unroll
        for (int k = 0; k < PV; k += kPairs) {
            float2 c[kPairs];
            if constexpr (kPairs == 2) {
                const float4 c2 = *reinterpret_cast<const float4*>(a + k * turns);
                c[0] = make_float2(c2.x, c2.y);
                c[1] = make_float2(c2.z, c2.w);
            } else {
                c[0] = a[0];
            }
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                E& first = INTER ? y[2 * (k + e)] : z1.e[k + e];
                E& second = INTER ? y[2 * (k + e) + 1] : z2.e[k + e];
                const float x1 = to_f(first), x2 = to_f(second);
                first = from_f<E>(turn1(x1, x2, c[e]));
                second = from_f<E>(turn2(x1, x2, c[e]));
            }
        }
        if (INTER) {
#pragma unroll
            for (int k = 0; k < PV; ++k) {
                z1.e[k] = y[k];
                z2.e[k] = y[PV + k];
            }
        }
        *reinterpret_cast<V*>(o + at) = z1;
        *reinterpret_cast<V*>(o + at + off) = z2;
    }
}

template <typename E, int PV>
void launch_pv(const RopeParams& p, bool inter, unsigned grid, size_t smem, cudaStream_t st) {
    const FastDiv per(static_cast<uint32_t>(p.half / PV + (p.tail / PV + 1) / 2));
    const FastDiv heads(static_cast<uint32_t>(p.q.n + p.k.n));
    const FastDiv half(static_cast<uint32_t>(p.half > 0 ? p.half : 1));
    if (inter) rope_kernel<E, PV, true><<<grid, kRopeThreads, smem, st>>>(p, per, heads, half);
    else rope_kernel<E, PV, false><<<grid, kRopeThreads, smem, st>>>(p, per, heads, half);
}

template <typename E>
int launch_rope(RopeParams p, bool inter, cudaStream_t st) {
    // the widest piece everything is a multiple of: pairs, the copied tail, strides
    // and addresses
    constexpr int kMost = 16 / sizeof(E);
    auto fits = [&](int pv) {
        if (p.half % pv || p.tail % pv) return false;
        const uintptr_t bytes = sizeof(E) * pv;  // of an access
        for (const RopeHeads* g : {&p.q, &p.k}) {
            if (g->n == 0) continue;
            const uintptr_t all = reinterpret_cast<uintptr_t>(g->x) | reinterpret_cast<uintptr_t>(g->out) |
                                  static_cast<uintptr_t>((g->xt | g->ot | g->xh | g->oh) * static_cast<int64_t>(sizeof(E)));
            if (all % bytes) return false;
        }
        return true;
    };
    int pv = kMost;
    while (pv > 1 && !fits(pv)) pv /= 2;
    // tokens of a CTA: about two pieces a thread, while enough CTAs remain
    const int64_t per = static_cast<int64_t>(p.q.n + p.k.n) * (p.half / pv + (p.tail / pv + 1) / 2);
    int64_t tok = (2 * kRopeThreads + per - 1) / per;
    if (tok > kRopeMaxTokens) tok = kRopeMaxTokens;
    while (tok > 1 && (p.T + tok - 1) / tok < 2 * num_sms()) --tok;
    p.tokens = static_cast<int>(tok);
    const int64_t grid = (p.T + tok - 1) / tok;
    const size_t smem = static_cast<size_t>(tok) * p.half * sizeof(float2);
    if (grid >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
    clear_pending_launch_error();
    const unsigned gr = static_cast<unsigned>(grid);
    if constexpr (kMost == 8)
        if (pv == 8) { launch_pv<E, 8>(p, inter, gr, smem, st); return launch_result(); }
    if (pv == 4) launch_pv<E, 4>(p, inter, gr, smem, st);
    else if (pv == 2) launch_pv<E, 2>(p, inter, gr, smem, st);
    else launch_pv<E, 1>(p, inter, gr, smem, st);
    return launch_result();
}

}  // namespace
}  // namespace gg

using namespace gg;

extern "C" {

int gg_rope(const void* q, int64_t q_tok, int64_t q_head, int n_q, const void* k, int64_t k_tok, int64_t k_head,
            int n_k, void* out_q, int64_t oq_tok, int64_t oq_head, void* out_k, int64_t ok_tok, int64_t ok_head,
            const int32_t* positions, int axes, const int32_t* sections, const int64_t* steps, float attention_scale,
            int64_t T, int D, int rot, int interleaved, int dtype, int backward, void* stream) {
    if (T < 0 || D < 0 || rot < 0 || n_q < 0 || n_k < 0) return GG_ERR_INVALID_ARG;
    if (rot > D || rot % 2 || axes < 1 || axes > GG_ROPE_MAX_AXES) return GG_ERR_INVALID_ARG;
    if (dtype != GG_DTYPE_BF16 && dtype != GG_DTYPE_F16 && dtype != GG_DTYPE_F32) return GG_ERR_INVALID_ARG;
    if (q_tok < 0 || q_head < 0 || k_tok < 0 || k_head < 0 || oq_tok < 0 || oq_head < 0 || ok_tok < 0 || ok_head < 0)
        return GG_ERR_INVALID_ARG;
    if (axes > 1) {
        if (!sections) return GG_ERR_INVALID_ARG;
        int64_t sum = 0;
        for (int i = 0; i < axes; ++i) {
            if (sections[i] < 0) return GG_ERR_INVALID_ARG;
            sum += sections[i];
        }
        if (sum != rot / 2) return GG_ERR_INVALID_ARG;
    }
    const int64_t heads = static_cast<int64_t>(n_q) + n_k;
    // (a CTA's elements are counted in 32 bits)
    if (rot > kRopeMaxRot || heads > GG_ROPE_MAX_HEADS || heads * D > (int64_t(1) << 27)) return GG_ERR_UNSUPPORTED;
    if (T == 0 || D == 0 || heads == 0) return GG_OK;
    if ((n_q && (!q || !out_q)) || (n_k && (!k || !out_k))) return GG_ERR_INVALID_ARG;
    if (rot > 0 && (!positions || !steps)) return GG_ERR_INVALID_ARG;
    const uintptr_t size = dtype == GG_DTYPE_F32 ? 4 : 2;
    auto odd = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % size != 0; };
    if ((n_q && (odd(q) || odd(out_q))) || (n_k && (odd(k) || odd(out_k)))) return GG_ERR_UNSUPPORTED;
    const bool same = (!n_q || (q == out_q && q_tok == oq_tok && q_head == oq_head)) &&
                      (!n_k || (k == out_k && k_tok == ok_tok && k_head == ok_head));
    if (same && rot == 0) return GG_OK;
    // an output's heads may not overlap one another: neighbours are as far apart as what is written
    const int wide = same ? rot : D;
    auto overlap = [&](int n, int64_t tok, int64_t head) { return (T > 1 && n > 0 && tok < wide) || (n > 1 && head < wide); };
    if (overlap(n_q, oq_tok, oq_head) || overlap(n_k, ok_tok, ok_head)) return GG_ERR_INVALID_ARG;
    RopeParams p{};
    p.q = RopeHeads{q, out_q, q_tok, q_head, oq_tok, oq_head, n_q};
    p.k = RopeHeads{k, out_k, k_tok, k_head, ok_tok, ok_head, n_k};
    p.pos = positions;
    p.step = steps;
    p.m = attention_scale;
    p.T = T;
    p.half = rot / 2;
    p.tail = same ? 0 : D - rot;
    int b = axes > 1 ? sections[0] : p.half;
    for (int i = 0; i < 3; ++i) {
        p.bound[i] = i + 1 < axes ? b : p.half;
        if (i + 1 < axes) b += sections[i + 1];
    }
    p.backward = backward ? 1 : 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == GG_DTYPE_BF16) return launch_rope<__nv_bfloat16>(p, interleaved != 0, st);
    if (dtype == GG_DTYPE_F16) return launch_rope<__half>(p, interleaved != 0, st);
    return launch_rope<float>(p, interleaved != 0, st);
}

}  // extern "C"
