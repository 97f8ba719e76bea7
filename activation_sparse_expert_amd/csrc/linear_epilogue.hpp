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
__device__ __forceinline__ void finish(const LinearArgs &p, int t, int n, float a, float g)
{
    if (p.b) a += p.b[n];
    if (p.wg) {
        if (p.bg) g += p.bg[n];
        a *= activate(g, p.act);
    } else {
        a = activate(a, p.act);
    }
    if (p.r) a += st::load_el(p.r, p.ydt, (size_t)t * p.rs + n);
    st::store_el(p.y, p.ydt, (size_t)t * p.ys + n, a);
}

}  // namespace le
}  // namespace moeffn
