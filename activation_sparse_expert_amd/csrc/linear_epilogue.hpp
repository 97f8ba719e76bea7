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

// Whether four outputs of a token can be read and written together (finish4)
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

template <bool BF16>
__device__ __forceinline__ void residual_store4(const LinearArgs &p, size_t at, size_t ar, float (&v)[4])
{
    if (p.r) {
        const uint2 r = *(const uint2 *)((const uint16_t *)p.r + ar);
        v[0] += lo16_to_float<BF16>(r.x);
        v[1] += hi16_to_float<BF16>(r.x);
        v[2] += lo16_to_float<BF16>(r.y);
        v[3] += hi16_to_float<BF16>(r.y);
    }
    *(uint2 *)((uint16_t *)p.y + at) =
        make_uint2(st::to16<BF16>(v[0]) | (uint32_t)st::to16<BF16>(v[1]) << 16,
                   st::to16<BF16>(v[2]) | (uint32_t)st::to16<BF16>(v[3]) << 16);
}

// Outputs n .. n + 3 (n a multiple of 4, all below N) of token t
__device__ __forceinline__ void finish4(const LinearArgs &p, int t, int n, float (&v)[4], float (&g)[4])
{
    if (p.b) {
        const float4 b = *(const float4 *)(p.b + n);
        v[0] += b.x; v[1] += b.y; v[2] += b.z; v[3] += b.w;
    }
    if (p.bg) {
        const float4 b = *(const float4 *)(p.bg + n);
        g[0] += b.x; g[1] += b.y; g[2] += b.z; g[3] += b.w;
    }
    values<4>(p, v, g);
    const size_t at = (size_t)t * p.ys + n, ar = (size_t)t * p.rs + n;
    if (p.ydt == 1) {
        residual_store4<true>(p, at, ar, v);
    } else if (p.ydt == 0) {
        residual_store4<false>(p, at, ar, v);
    } else {
        if (p.r) {
            const float4 r = *(const float4 *)((const float *)p.r + ar);
            v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
        }
        *(float4 *)((float *)p.y + at) = make_float4(v[0], v[1], v[2], v[3]);
    }
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

template <int U>
__device__ __forceinline__ void finish_bits4(const Args<U> &p, int t, int n, float (&v)[4], float (&g)[4])
{
    if constexpr (U == st::kI8) {
        const float sx = p.sx[t];
        const float4 w = *(const float4 *)(p.sw + n);
        v[0] = (float)__float_as_int(v[0]) * w.x * sx; v[1] = (float)__float_as_int(v[1]) * w.y * sx;
        v[2] = (float)__float_as_int(v[2]) * w.z * sx; v[3] = (float)__float_as_int(v[3]) * w.w * sx;
        if (p.wg) {
            const float4 s = *(const float4 *)(p.sg + n);
            g[0] = (float)__float_as_int(g[0]) * s.x * sx; g[1] = (float)__float_as_int(g[1]) * s.y * sx;
            g[2] = (float)__float_as_int(g[2]) * s.z * sx; g[3] = (float)__float_as_int(g[3]) * s.w * sx;
        }
    }
    finish4(p, t, n, v, g);
}

}  // namespace le
}  // namespace moeffn
