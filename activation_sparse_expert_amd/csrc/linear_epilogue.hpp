// Epilogue of the linear layer: bias, activation, gate, residual, one rounding.
#pragma once
#include "linear.hpp"
#include "mfma_stream.hpp"
#include "rows.hpp"

#include <type_traits>

namespace moeffn {
namespace le {

template <int U>
using Args = std::conditional_t<U == st::kI8, LinearQ8Args, LinearArgs>;

// v sigmoid(z) with the hardware reciprocal (one unit in the last place, which an
// fp32 division would cost ten instructions to remove)
__device__ __forceinline__ float gate_by(float v, float z)
{
    return v * __builtin_amdgcn_rcpf(1.f + __expf(-z));
}

// moe_act.  Every form takes the infinities of a product that overflowed the
// way its formula does in fp32.
template <int ACT>
__device__ __forceinline__ float activate(float v)
{
    if constexpr (ACT == 1) return v != v ? v : fmaxf(v, 0.f);                      // ReLU (a NaN stays one)
    // GELU: 1 + erf z = erfc(-z), which does not cancel where v is negative (at -5
    // the sum is off by a tenth of itself, several steps of a bf16 y)
    else if constexpr (ACT == 2) return 0.5f * v * erfcf(v * -0.70710678118654752f);
    // GELU, tanh form: 0.5 v (1 + tanh z) = v sigmoid(2 z)
    else if constexpr (ACT == 3) return gate_by(v, 1.59576912160573072f * (v + 0.044715f * v * v * v));
    else if constexpr (ACT == 4) return gate_by(v, v);                              // SiLU
    else return v;
}

// Q outputs from their products: v with W (and the results), g with Wg, biases added.
template <int Q, int ACT>
__device__ __forceinline__ void values_as(const LinearArgs &p, float (&v)[Q], const float (&g)[Q])
{
#pragma unroll
    for (int i = 0; i < Q; ++i) v[i] = p.wg ? v[i] * activate<ACT>(g[i]) : activate<ACT>(v[i]);
}
template <int Q>
__device__ __forceinline__ void values(const LinearArgs &p, float (&v)[Q], const float (&g)[Q])
{
    switch (p.act) {
    case 1: values_as<Q, 1>(p, v, g); break;
    case 2: values_as<Q, 2>(p, v, g); break;
    case 3: values_as<Q, 3>(p, v, g); break;
    case 4: values_as<Q, 4>(p, v, g); break;
    default: values_as<Q, 0>(p, v, g); break;
    }
}

// Element (t, n) from its product(s): a with W, g with Wg.
__device__ __forceinline__ void finish(const LinearArgs &p, int t, int n, float a, float g)
{
    float v[1] = {p.b ? a + p.b[n] : a};
    const float gb[1] = {p.bg ? g + p.bg[n] : g};
    values<1>(p, v, gb);
    if (p.r) v[0] += st::load_el(p.r, p.ydt, (size_t)t * p.rs + n);
    st::store_el(p.y, p.ydt, (size_t)t * p.ys + n, v[0]);
}

// Whether four outputs of a token can be read and written together (finish_cols4, add_store4)
template <int U>
bool quads(const Args<U> &p)
{
    if constexpr (U == st::kI8)
        if ((((uintptr_t)p.sw | (uintptr_t)p.sg) & 15) != 0) return false;
    const size_t al = p.ydt == 2 ? 16 : 8;
    auto ok = [&](const void *q, long long stride) { return ((uintptr_t)q & (al - 1)) == 0 && stride % 4 == 0; };
    return p.N % 4 == 0 && ok(p.y, p.ys) && (!p.r || ok(p.r, p.rs)) && ((uintptr_t)p.b & 15) == 0 &&
           ((uintptr_t)p.bg & 15) == 0;
}

// The same from sums of the matrix instructions: of 16-bit products as they are, of codes as
// integers times the token's and the output's scale, the latter first (a weight's scale
// is far from the ends of fp32).
template <int U, class S>
__device__ __forceinline__ void finish_sum(const Args<U> &p, int t, int n, S a, S g)
{
    if constexpr (U == st::kI8) {
        const float sx = p.sx[t];
        finish(p, t, n, (float)a * p.sw[n] * sx, p.wg ? (float)g * p.sg[n] * sx : 0.f);
    } else {
        finish(p, t, n, a, g);
    }
}

// Sums that pass through LDS or the workspace as the bits of a float
__device__ __forceinline__ float bits(float v) { return v; }
__device__ __forceinline__ float bits(int v) { return __int_as_float(v); }

template <int U>
__device__ __forceinline__ float add_bits(float a, float b)
{
    if constexpr (U == st::kI8) return __int_as_float(__float_as_int(a) + __float_as_int(b));
    else return a + b;
}

template <int U>
__device__ __forceinline__ void finish_bits(const Args<U> &p, int t, int n, float a, float g)
{
    if constexpr (U == st::kI8) finish_sum<U>(p, t, n, __float_as_int(a), __float_as_int(g));
    else finish(p, t, n, a, g);
}

// What the outputs n .. n + 3 need of their rows of W and Wg: scales and biases.  A lane of a
// tile's epilogue has the same outputs of many tokens and loads this once.
struct Cols {
    float w[4], g[4], b[4], bg[4];
};

__device__ __forceinline__ void cols4(float (&v)[4], const float *p, int n, int N, bool quads)
{
    if (quads) {
        const float4 q = *(const float4 *)(p + n);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = p[min(n + x, N - 1)];
    }
}

template <int U>
__device__ __forceinline__ void load_cols(const Args<U> &p, Cols &c, int n, bool quads)
{
    if constexpr (U == st::kI8) {
        cols4(c.w, p.sw, n, p.N, quads);
        if (p.wg) cols4(c.g, p.sg, n, p.N, quads);
    }
    if (p.b) cols4(c.b, p.b, n, p.N, quads);
    if (p.bg) cols4(c.bg, p.bg, n, p.N, quads);
}

// The residual of four outputs of a token, at ar, before its conversion (m of them exist)
__device__ __forceinline__ uint4 load_residual(const LinearArgs &p, size_t ar, int m, bool quads)
{
    uint4 r = make_uint4(0, 0, 0, 0);
    if (quads) {
        if (p.ydt == 2) {
            r = *(const uint4 *)((const float *)p.r + ar);
        } else {
            const uint2 q = *(const uint2 *)((const uint16_t *)p.r + ar);
            r.x = q.x; r.y = q.y;
        }
    } else if (p.ydt == 2) {
        const uint32_t *q = (const uint32_t *)p.r + ar;
        r = make_uint4(q[0], m > 1 ? q[1] : 0, m > 2 ? q[2] : 0, m > 3 ? q[3] : 0);
    } else {
        const uint16_t *q = (const uint16_t *)p.r + ar;
        r.x = q[0] | (m > 1 ? (uint32_t)q[1] << 16 : 0);
        r.y = (m > 2 ? q[2] : 0) | (m > 3 ? (uint32_t)q[3] << 16 : 0);
    }
    return r;
}

// Four outputs of a token with scale sx from their sums v (and g) as bits, residual aside; ACT:
// moe_act, or -1 for p.act
template <int U, int ACT>
__device__ __forceinline__ void apply_cols(const Args<U> &p, const Cols &c, float sx, float (&v)[4], float (&g)[4])
{
    if constexpr (U == st::kI8) {
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = (float)__float_as_int(v[x]) * c.w[x] * sx;
        if (p.wg)
#pragma unroll
            for (int x = 0; x < 4; ++x) g[x] = (float)__float_as_int(g[x]) * c.g[x] * sx;
    }
    if (p.b)
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] += c.b[x];
    if (p.bg)
#pragma unroll
        for (int x = 0; x < 4; ++x) g[x] += c.bg[x];
    if constexpr (ACT < 0) values<4>(p, v, g);
    else values_as<4, ACT>(p, v, g);
}

// Adds the residual's bits r (RES: there is one) and stores; YDT: p.ydt
template <int YDT, bool RES>
__device__ __forceinline__ void add_store4(const LinearArgs &p, const uint4 &r, size_t at, int m, bool quads, float (&v)[4])
{
    if constexpr (RES) {
        if constexpr (YDT == 2) {
            v[0] += __uint_as_float(r.x); v[1] += __uint_as_float(r.y);
            v[2] += __uint_as_float(r.z); v[3] += __uint_as_float(r.w);
        } else {
            v[0] += lo16_to_float<YDT == 1>(r.x); v[1] += hi16_to_float<YDT == 1>(r.x);
            v[2] += lo16_to_float<YDT == 1>(r.y); v[3] += hi16_to_float<YDT == 1>(r.y);
        }
    }
    if (!quads) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (x < m) st::store_el(p.y, YDT, at + x, v[x]);
    } else if constexpr (YDT == 2) {
        *(float4 *)((float *)p.y + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *(uint2 *)((uint16_t *)p.y + at) =
            make_uint2(st::to16<YDT == 1>(v[0]) | (uint32_t)st::to16<YDT == 1>(v[1]) << 16,
                       st::to16<YDT == 1>(v[2]) | (uint32_t)st::to16<YDT == 1>(v[3]) << 16);
    }
}

// Outputs n .. n + 3 (n a multiple of 4, all below N) of token t, with scale sx and residual r
template <int U>
__device__ __forceinline__ void finish_cols4(const Args<U> &p, const Cols &c, float sx, const uint4 &r, int t, int n,
                                             float (&v)[4], float (&g)[4])
{
    apply_cols<U, -1>(p, c, sx, v, g);
    const size_t at = (size_t)t * p.ys + n;
    auto store = [&](auto res) {
        constexpr bool R = decltype(res)::value;
        if (p.ydt == 2) add_store4<2, R>(p, r, at, 4, true, v);
        else if (p.ydt == 1) add_store4<1, R>(p, r, at, 4, true, v);
        else add_store4<0, R>(p, r, at, 4, true, v);
    };
    if (p.r) store(std::true_type());
    else store(std::false_type());
}

}  // namespace le
}  // namespace moeffn
