// Norms between two blocks: y = rs r + bs g (.) Npost(o), out = Npre(y), one row a workgroup,
// kept in LDS in fp32.
#include "codes.hpp"
#include "mfma_stream.hpp"
#include "rows.hpp"

namespace moeffn {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

__device__ __forceinline__ float block_sum(float v, float *lds)
{
    v = seg_sum<64>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kWaves; ++i) v += lds[i];
    return v;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, float *lds)
{
    for (int s = 32; s > 0; s >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, s));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = __uint_as_float(v);
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) v = max(v, __float_as_uint(lds[i]));
    return v;
}

// The row's norm in place; each thread touches its own elements only.  Where the squares
// pass fp32 everything is taken of values 2^-80 as large, beside which eps is nothing.
__device__ void norm_row(float *row, int d, int layer, float eps, const void *w, const void *b, int wdt, float add, float *lds)
{
    float k = 1.f, m = 0.f, ss = 0.f;
    for (;;) {
        if (layer) {
            m = 0.f;
            for (int i = threadIdx.x; i < d; i += kThreads) m += row[i] * k;
            m = block_sum(m, lds) / (float)d;
        }
        ss = 0.f;
        for (int i = threadIdx.x; i < d; i += kThreads) ss += (row[i] * k - m) * (row[i] * k - m);
        ss = block_sum(ss, lds);
        if (ss < INFINITY || k != 1.f) break;
        k = 0x1p-80f;
    }
    const float f = 1.f / sqrtf(ss / (float)d + (k == 1.f ? eps : 0.f));
    for (int i = threadIdx.x; i < d; i += kThreads) {
        float v = (row[i] * k - m) * f;
        if (w) v *= st::load_el(w, wdt, i) + add;
        if (b) v += st::load_el(b, wdt, i);
        row[i] = v;
    }
}

__global__ void __launch_bounds__(kThreads)
norm_kernel(NormArgs a)
{
    extern __shared__ float row[];
    __shared__ float lds[kWaves];
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        if (a.o) {
            for (int i = threadIdx.x; i < a.d; i += kThreads) row[i] = st::load_el(a.o, a.odt, (size_t)t * a.os + i);
            if (a.post) norm_row(row, a.d, a.layer, a.eps, a.pw, a.pb, a.wdt, a.add, lds);
        }
        for (int i = threadIdx.x; i < a.d; i += kThreads) {
            float v = a.r ? a.rscale * st::load_el(a.r, a.rdt, (size_t)t * a.rs + i) : 0.f;
            if (a.o) v += a.bscale * (row[i] * (a.g ? st::load_el(a.g, a.odt, (size_t)t * a.gs + i) : 1.f));
            if (a.y) st::store_el(a.y, a.rdt, (size_t)t * a.ys + i, v);
            row[i] = v;
        }
        if (!a.out) continue;
        norm_row(row, a.d, a.layer, a.eps, a.w, a.b, a.wdt, a.add, lds);
        if (a.ndt != 3) {
            for (int i = threadIdx.x; i < a.d; i += kThreads) st::store_el(a.out, a.ndt, (size_t)t * a.ns + i, row[i]);
            continue;
        }
        uint32_t most = 0;
        for (int i = threadIdx.x; i < a.d; i += kThreads) most = max(most, codes::magnitude(row[i]));
        const codes::Row c = codes::row(block_max(most, lds));
        for (int i = threadIdx.x; i < a.d; i += kThreads)
            ((int8_t *)a.out)[(size_t)t * a.ns + i] = (int8_t)codes::code(row[i], c);
        if (threadIdx.x == 0) a.out_scale[t] = c.scale;
    }
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(norm_kernel, dim3((unsigned)(a.T < 65536 ? a.T : 65536)), dim3(kThreads), a.d * 4, s, a);
    return hipGetLastError();
}

}  // namespace moeffn
