// Epilogue of the linear layer: bias, activation, gate, residual, one rounding.
#pragma once
#include "linear.hpp"
#include "mfma_stream.hpp"

namespace moeffn {
namespace le {

// moe_act.  Every form takes the infinities of a product that overflowed the
// way its formula does in fp32.
__device__ __forceinline__ float activate(float v, int act)
{
    switch (act) {
    case 1: return v != v ? v : fmaxf(v, 0.f);                              // ReLU (a NaN stays one)
    case 2: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));       // GELU
    case 3: {                                                               // GELU, tanh form:
        // 0.5 v (1 + tanh z) = v sigmoid(2 z)
        const float z = 0.79788456080286536f * (v + 0.044715f * v * v * v);
        return v / (1.f + __expf(-2.f * z));
    }
    case 4: return silu(v);
    default: return v;
    }
}

// Element (t, n) from its product(s): a with W, g with Wg.
__device__ __forceinline__ float value(const LinearArgs &p, float a, float g, float b, float bg)
{
    a += b;
    return p.wg ? a * activate(g + bg, p.act) : activate(a, p.act);
}

__device__ __forceinline__ void finish(const LinearArgs &p, int t, int n, float a, float g)
{
    float v = value(p, a, g, p.b ? p.b[n] : 0.f, p.bg ? p.bg[n] : 0.f);
    if (p.r) v += st::load_el(p.r, p.ydt, (size_t)t * p.rs + n);
    st::store_el(p.y, p.ydt, (size_t)t * p.ys + n, v);
}

// Whether four outputs of a token can be read and written together (finish4)
inline bool quads(const LinearArgs &p)
{
    const size_t al = p.ydt == 2 ? 16 : 8;
    auto ok = [&](const void *q, long long stride) { return ((uintptr_t)q & (al - 1)) == 0 && stride % 4 == 0; };
    return p.N % 4 == 0 && ok(p.y, p.ys) && (!p.r || ok(p.r, p.rs)) && ((uintptr_t)p.b & 15) == 0 &&
           ((uintptr_t)p.bg & 15) == 0;
}

// Outputs n .. n + 3 (n a multiple of 4, all below N) of token t
__device__ __forceinline__ void finish4(const LinearArgs &p, int t, int n, const float (&a)[4], const float (&g)[4])
{
    float v[4];
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 b = p.b ? *(const float4 *)(p.b + n) : zero, bg = p.bg ? *(const float4 *)(p.bg + n) : zero;
    const float bb[4] = {b.x, b.y, b.z, b.w}, gg[4] = {bg.x, bg.y, bg.z, bg.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = value(p, a[i], g[i], bb[i], gg[i]);
    const size_t at = (size_t)t * p.ys + n, ar = (size_t)t * p.rs + n;
    if (p.ydt == 2) {
        if (p.r) {
            const float4 r = *(const float4 *)((const float *)p.r + ar);
            v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
        }
        *(float4 *)((float *)p.y + at) = make_float4(v[0], v[1], v[2], v[3]);
        return;
    }
    const bool bf = p.ydt == 1;
    if (p.r) {
        const uint2 r = *(const uint2 *)((const uint16_t *)p.r + ar);
        const uint32_t w[2] = {r.x, r.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint16_t h = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            v[i] += bf ? st::from16<true>(h) : st::from16<false>(h);
        }
    }
    uint32_t o[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i >> 1] |= (uint32_t)(bf ? st::to16<true>(v[i]) : st::to16<false>(v[i])) << (16 * (i & 1));
    *(uint2 *)((uint16_t *)p.y + at) = make_uint2(o[0], o[1]);
}

}  // namespace le
}  // namespace moeffn
