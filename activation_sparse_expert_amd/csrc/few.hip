// A whole dense MoE layer for at most 32 tokens (MoE-Infinity review, "A3 背景"
// and FloE review, "MoE 专家前向计算": top-k routing, SwiGLU experts):
//   y_t = r_t + sum_s w_ts a_e(t,s)(x_t) + sum_i a_E+i(x_t),
//   a_e(x) = (SiLU(x G_e) (.) (x U_e)) D_e.
// Bound by the weights of the chosen experts, read once: two kernels stream
// them through the matrix cores (mfma_stream.hpp), all tokens of the call as
// the other operand, so an expert's weights serve its tokens together without
// gathering them.  A column of D that belongs to a token the expert was not
// chosen for is dropped (its operand repeats one of the expert's own tokens, so that
// nothing of another token, nor an infinity in these weights, reaches it).
//   gate/up: a wave takes 16 channels of an expert and a slice of d;
//            h = SiLU(g) u goes to the workspace;
//   down:    a workgroup takes 16 columns of y over all listed experts, its
//            waves an equal share each of the experts' channels laid end to end, so
//            no partial rows leave the workgroup.
// h is kept as the sum of two values of the 16-bit type (hi = its rounding,
// lo = the rounding of the rest): the products with W^down are then good to
// about 2^-17 (bf16) or 2^-22 (fp16) of h, and the rounding of y is the only one
// that shows.  One more MFMA per step is free under the weight stream.
#include "linear.hpp"
#include "mfma_stream.hpp"

namespace moeffn {

namespace {

using st::floatx4;

// The listed experts in LDS, in ascending order, and their tokens.
struct List {
    int *expert;                        // [amax]
    uint32_t *mask;                     // [amax]
    int *off;                           // [amax]
    int n;
};

// Made by every workgroup from the T k choices.  em [E] and n [1]: LDS scratch.
__device__ __forceinline__ void make_list(const FewArgs &a, List &l, uint32_t *em, int *n)
{
    const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 63;
    for (int e = tid; e < a.E; e += nthr) em[e] = 0u;
    __syncthreads();
    for (int p = tid; p < a.T * a.k; p += nthr) atomicOr(&em[a.topk_idx[p]], 1u << (p / a.k));
    __syncthreads();
    if (tid < 64) {
        int na = 0, rows = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            const uint32_t m = e0 + lane < a.E ? em[e0 + lane] : 0u;
            const unsigned long long b = __ballot(m != 0u);
            int c = __popc(m), incl = c;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(incl, o, 64);
                if (lane >= o) incl += v;
            }
            if (m) {
                const int i = na + __popcll(b & ((1ull << lane) - 1ull));
                l.expert[i] = e0 + lane;
                l.mask[i] = m;
                l.off[i] = rows + incl - c;
            }
            na += __popcll(b);
            rows += __shfl(incl, 63, 64);
        }
        const uint32_t all = a.T == 32 ? 0xFFFFFFFFu : (1u << a.T) - 1u;
        for (int i = lane; i < a.S; i += 64) {
            l.expert[na + i] = a.E + i;
            l.mask[na + i] = all;
            l.off[na + i] = rows + i * a.T;
        }
        if (lane == 0) *n = na + a.S;
    }
    __syncthreads();
    l.n = *n;
}

// What the down product and the trace need of the list (one workgroup writes it).
__device__ __forceinline__ void export_list(const FewArgs &a, const List &l, const uint32_t *em)
{
    const int tid = threadIdx.x, nthr = blockDim.x;
    if (tid == 0) *a.tab.n = l.n;
    for (int i = tid; i < l.n; i += nthr) {
        const int e = l.expert[i], off = l.off[i];
        a.tab.expert[i] = e;
        a.tab.mask[i] = l.mask[i];
        a.tab.off[i] = off;
        if (e >= a.E) {
            for (int t = 0; t < a.T; ++t) a.tab.wt[off + t] = 1.f;
            continue;
        }
        for (uint32_t m = l.mask[i], r = 0; m; m &= m - 1, ++r) {
            const int t = __ffs(m) - 1;
            float w = 0.f;
            for (int s = 0; s < a.k; ++s)
                if (a.topk_idx[t * a.k + s] == e) w = a.topk_w[t * a.k + s];
            a.tab.wt[off + r] = w;
        }
    }
    for (int e = tid; e < a.E; e += nthr) {
        const int c = __popc(em[e]);
        if (a.count) a.count[e] = c;
        if (a.eam_row) a.eam_row[e] += c;
        if (a.expert_dense) a.expert_dense[e] = c > 0 ? 1 : 0;
    }
}

__device__ __forceinline__ int row_of(uint32_t mask, int off, int t)
{
    return off + __popc(mask & ((1u << t) - 1u));
}

template <bool BF16, int NB, int U>
__global__ void __launch_bounds__(1024)
few_gateup_kernel(FewArgs a, int P, int slice)
{
    extern __shared__ __align__(16) float smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
    float *red = smem;                              // [2][waves][2][NB][64 lanes][4]
    List l;
    l.expert = (int *)(red + 2 * waves * 2 * NB * 256);
    l.mask = (uint32_t *)(l.expert + a.amax);
    l.off = (int *)(l.mask + a.amax);
    uint32_t *em = (uint32_t *)(l.off + a.amax);    // [E]
    make_list(a, l, em, (int *)(em + a.E));
    if (blockIdx.x == 0) export_list(a, l, em);

    const int G = waves / P, g = wave / P, p = wave - g * P;
    const int fb = (a.f + 15) / 16, units = l.n * fb;
    const int li = lane & 15, kq = 8 * (lane >> 4);
    const int s0 = p * slice, s1 = min(s0 + slice, (a.d + 31) / 32);
    for (int u0 = blockIdx.x * G, it = 0; u0 < units; u0 += gridDim.x * G, ++it) {
        floatx4 acc[2][NB];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[m][j] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (u0 + g < units && s0 < s1) {
            const int i = (u0 + g) / fb, c = (u0 + g) - i * fb;
            const uint32_t mask = l.mask[i];
            const int row = min(16 * c + li, a.f - 1);
            const size_t at = ((size_t)l.expert[i] * a.f + row) * a.d + kq;
            const uint16_t *w[2] = {a.gate + at, a.up + at}, *x[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int t = 16 * j + li;
                x[j] = a.x + (size_t)((mask >> t) & 1u ? t : __ffs(mask) - 1) * a.d + kq;
            }
            st::stream<BF16, 2, NB, 1, U>(acc, w, x, s0, s1, a.d, kq);
        }
        float *rd = red + (it & 1) * waves * 2 * NB * 256;   // two halves: one barrier per round
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                *(floatx4 *)&rd[((wave * 2 + m) * NB + j) * 256 + 4 * lane] = acc[m][j];
        __syncthreads();
        for (int q = tid; q < G * NB * 256; q += blockDim.x) {
            const int gg = q / (NB * 256), e = q - gg * NB * 256;
            const int t = e >> 4, r = e & 15;
            if (u0 + gg >= units) continue;
            const int i = (u0 + gg) / fb, c = (u0 + gg) - i * fb;
            const int ch = 16 * c + r;
            const uint32_t mask = l.mask[i];
            if (ch >= a.f || !((mask >> t) & 1u)) continue;
            const int pos = (t >> 4) * 256 + 4 * ((t & 15) + 16 * (r >> 2)) + (r & 3);
            float v[2] = {0.f, 0.f};
            for (int z = 0; z < P; ++z)
#pragma unroll
                for (int m = 0; m < 2; ++m) v[m] += rd[((gg * P + z) * 2 + m) * NB * 256 + pos];
            const float h = silu(v[0]) * v[1];
            const uint16_t hi = st::to16<BF16>(h);
            const float back = st::from16<BF16>(hi);
            // an infinite or NaN h stands in hi alone
            const uint16_t lo = fabsf(back) < INFINITY ? st::to16<BF16>(h - back) : (uint16_t)0;
            uint16_t *dst = a.h + ((size_t)row_of(mask, l.off[i], t) * a.f + (ch & ~7)) * 2 + (ch & 7);
            dst[0] = hi;
            dst[8] = lo;
        }
    }
}

template <bool BF16, int NB, int U>
__global__ void __launch_bounds__(1024)
few_down_kernel(FewArgs a)
{
    extern __shared__ __align__(16) float red[];    // [waves][NB][64 lanes][4]
    const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, kq = 8 * (lane >> 4);
    const int n0 = 16 * blockIdx.x;
    const int col = min(n0 + li, a.d - 1);
    const int n = *a.tab.n;
    const int spe = (a.f + 31) / 32;                // steps of 32 channels per expert
    const int total = n * spe;
    const int beg = (int)((long long)total * wave / waves), end = (int)((long long)total * (wave + 1) / waves);

    floatx4 y[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) y[j] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int s = beg; s < end;) {
        const int i = s / spe, s0 = s - i * spe, s1 = min(spe, s0 + end - s);
        s += s1 - s0;
        const uint32_t mask = a.tab.mask[i];
        const int off = a.tab.off[i];
        const uint16_t *w[1] = {a.down_t + ((size_t)a.tab.expert[i] * a.d + col) * a.f + kq};
        const uint16_t *h[2 * NB];
        float wt[NB];
        bool mine[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int t = 16 * j + li;
            mine[j] = (mask >> t) & 1u;
            const int row = mine[j] ? row_of(mask, off, t) : off;
            wt[j] = a.tab.wt[row];
            h[2 * j] = a.h + (size_t)row * a.f * 2 + 2 * kq;
            h[2 * j + 1] = h[2 * j] + 8;
        }
        floatx4 acc[1][NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[0][j] = floatx4{0.f, 0.f, 0.f, 0.f};
        st::stream<BF16, 1, 2 * NB, 2, U>(acc, w, h, s0, s1, a.f, kq);
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) y[j][r] = mine[j] ? y[j][r] + wt[j] * acc[0][j][r] : y[j][r];
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) *(floatx4 *)&red[(wave * NB + j) * 256 + 4 * lane] = y[j];
    __syncthreads();
    for (int q = tid; q < NB * 256; q += blockDim.x) {
        const int t = q >> 4, r = q & 15, c = n0 + r;
        if (t >= a.T || c >= a.d) continue;
        const int pos = (t >> 4) * 256 + 4 * ((t & 15) + 16 * (r >> 2)) + (r & 3);
        float v = 0.f;
        for (int z = 0; z < waves; ++z) v += red[z * NB * 256 + pos];
        const size_t at = (size_t)t * a.d + c;
        if (a.r) v += st::load_el(a.r, a.ydt, at);
        st::store_el(a.y, a.ydt, at, v);
    }
}

template <bool BF16, int NB>
hipError_t gateup(const FewArgs &a, hipStream_t s)
{
    constexpr int U = NB == 1 ? 8 : 4, W = 16;
    const int steps = (a.d + 31) / 32, fb = (a.f + 15) / 16;
    const long long units = (long long)fb * a.amax;
    int P = 1;
    while (P < W && units * P < 4096 && steps >= 2 * U * P) P *= 2;
    const int G = W / P, slice = (steps + P - 1) / P;
    long long grid = (units + G - 1) / G;
    if (grid > 1024) grid = 1024;
    const size_t lds = (size_t)W * 2 * 2 * NB * 1024 + (size_t)a.amax * 12 + (size_t)a.E * 4 + 4;
    const void *kern = (const void *)few_gateup_kernel<BF16, NB, U>;
    hipError_t e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((few_gateup_kernel<BF16, NB, U>), dim3((unsigned)grid), dim3(64 * W), lds, s, a, P, slice);
    return hipGetLastError();
}

template <bool BF16, int NB>
hipError_t down(const FewArgs &a, hipStream_t s)
{
    constexpr int U = NB == 1 ? 8 : 4, W = 16;
    hipLaunchKernelGGL((few_down_kernel<BF16, NB, U>), dim3((unsigned)((a.d + 15) / 16)), dim3(64 * W),
                       (size_t)W * NB * 1024, s, a);
    return hipGetLastError();
}

bool args_ok(const FewArgs &a)
{
    return a.T >= 1 && a.T <= kFewTokens && a.d >= 8 && a.d % 8 == 0 && a.f >= 8 && a.f % 8 == 0 && a.E >= 1 &&
           a.E <= 1024 && a.S >= 0 && (long long)a.T * (a.k + a.S) <= kFewRows && a.amax >= 1 && a.amax <= kFewRows;
}

}  // namespace

hipError_t launch_few_gateup(const FewArgs &a, hipStream_t s)
{
    if (!args_ok(a)) return hipErrorInvalidValue;
    if (a.T <= 16) return a.bf16 ? gateup<true, 1>(a, s) : gateup<false, 1>(a, s);
    return a.bf16 ? gateup<true, 2>(a, s) : gateup<false, 2>(a, s);
}

hipError_t launch_few_down(const FewArgs &a, hipStream_t s)
{
    if (!args_ok(a)) return hipErrorInvalidValue;
    if (a.T <= 16) return a.bf16 ? down<true, 1>(a, s) : down<false, 1>(a, s);
    return a.bf16 ? down<true, 2>(a, s) : down<false, 2>(a, s);
}

}  // namespace moeffn
