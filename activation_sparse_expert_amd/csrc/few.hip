// A whole dense MoE layer for at most 32 tokens (MoE-Infinity review, "A3 背景"
// and FloE review, "MoE 专家前向计算": top-k routing, SwiGLU experts):
//   y_t = r_t + sum_s w_ts a_e(t,s)(x_t) + sum_i a_E+i(x_t),
//   a_e(x) = (SiLU(x G_e) (.) (x U_e)) D_e.
// Bound by the weights of the chosen experts, read once past the tokens that
// chose each (mfma_stream.hpp):
//   rank:    one workgroup ranks the router's logits and lists the experts
//            with their tokens;
//   gate/up: a wave takes 16 channels of a listed expert and a slice of d;
//            h = SiLU(g) u goes to the workspace;
//   down:    a workgroup takes 16 columns of y over all listed experts, its
//            waves an equal share each of the experts' channels laid end to end, so
//            no partial rows leave the workgroup.
// h is kept as the sum of two values of the 16-bit type (hi = its rounding,
// lo = the rounding of the rest): the products with W^down are then good to
// about 2^-17 (bf16) or 2^-22 (fp16) of h, and the rounding of y is the only one
// that shows.  hi and lo go through the matrix core as two tokens, which mostly fill
// columns that would idle.  A column of the matrix core depends on its own token
// alone, so infinities and NaN stay with the tokens whose experts hold them.
#include "linear.hpp"
#include "mfma_stream.hpp"
#include "route_common.hpp"

namespace moeffn {

namespace {

using st::floatx4;

// One workgroup: wave w ranks tokens w, w + 16, ...; then the list.
__global__ void __launch_bounds__(1024)
few_rank_kernel(FewArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 63, wave = tid >> 6, waves = nthr >> 6;
    const int E = a.E, E4 = (E + 3) & ~3, k = a.k;
    float *lg = (float *)smem;                      // [T][E4], padded with -inf
    int *sel = (int *)(lg + a.T * E4);              // [T][k]
    float *w = (float *)(sel + a.T * k);            // [T][k]
    uint32_t *em = (uint32_t *)(w + a.T * k);       // [E] bit t: token t goes to the expert
    int *eo = (int *)(em + E);                      // [E] first row
    for (int i = tid; i < a.T * E4; i += nthr) {
        const int t = i / E4, e = i - t * E4;
        const float v = e < E ? a.lg[(size_t)t * E + e] : -INFINITY;
        lg[i] = v;
        if (a.logits && e < E) a.logits[(size_t)t * E + e] = v;
    }
    for (int e = tid; e < E; e += nthr) em[e] = 0u;
    __syncthreads();
    for (int t = wave; t < a.T; t += waves) rc::rank_topk(lg + t * E4, E, k, sel + t * k, lane, 64);
    __syncthreads();
    for (int t = wave; t < a.T; t += waves) {
        const float *l = lg + t * E4;
        const int *st = sel + t * k;
        const float m = l[st[0]], den = rc::gate_den(l, st, E, k, a.renorm, m, lane);
        for (int s = lane; s < k; s += 64) {
            const float v = __expf(l[st[s]] - m) / den;
            w[t * k + s] = v;
            if (a.topk_idx) a.topk_idx[t * k + s] = st[s];
            if (a.topk_w) a.topk_w[t * k + s] = v;
            atomicOr(&em[st[s]], 1u << t);
        }
    }
    __syncthreads();
    if (wave == 0) {
        int na = 0, rows = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const uint32_t m = e0 + lane < E ? em[e0 + lane] : 0u;
            const unsigned long long b = __ballot(m != 0u);
            const int c = __popc(m);
            int incl = c;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(incl, o, 64);
                if (lane >= o) incl += v;
            }
            if (m) {
                const int i = na + __popcll(b & ((1ull << lane) - 1ull));
                a.tab.expert[i] = e0 + lane;
                a.tab.off[i] = rows + incl - c;
                eo[e0 + lane] = rows + incl - c;
            }
            na += __popcll(b);
            rows += __shfl(incl, 63, 64);
        }
        for (int i = lane; i <= a.S; i += 64) {
            if (i < a.S) a.tab.expert[na + i] = E + i;
            a.tab.off[na + i] = rows + i * a.T;
        }
        if (lane == 0) *a.tab.n = na + a.S;
    }
    __syncthreads();
    for (int p = tid; p < a.T * k; p += nthr) {
        const int t = p / k, e = sel[p];
        const int row = eo[e] + __popc(em[e] & ((1u << t) - 1u));
        a.tab.tok[row] = t;
        a.tab.wt[row] = w[p];
    }
    for (int p = tid; p < a.T * a.S; p += nthr) {
        a.tab.tok[a.T * k + p] = p % a.T;
        a.tab.wt[a.T * k + p] = 1.f;
    }
    for (int e = tid; e < E; e += nthr) {
        const int c = __popc(em[e]);
        if (a.count) a.count[e] = c;
        if (a.eam_row) a.eam_row[e] += c;
        if (a.expert_dense) a.expert_dense[e] = c > 0 ? 1 : 0;
    }
}

// Gate and up products of one wave: 16 channels, the expert's n tokens (at most
// 8 XI), into red [2][NB][64 lanes][4] of its own once every ring is done with.
template <bool BF16, int XI, int D>
__device__ __forceinline__ void gateup_wave(const FewArgs &a, unsigned char *ring, int e, int c, int off, int n,
                                            int b0, int b1, int blocks, int lane, floatx4 (&out)[2][2])
{
    using R = st::Ring<2, XI>;
    floatx4 acc[2][R::kFrag];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < R::kFrag; ++j) acc[m][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int r = st::copy_row(lane), k = 64 * b0 + st::copy_k(lane);
    const uint16_t *src[R::kCopies];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ch = min(16 * c + 8 * (i & 1) + r, a.f - 1);
        src[i] = (i < 2 ? a.gate : a.up) + ((size_t)e * a.f + ch) * a.d + k;
    }
#pragma unroll
    for (int i = 0; i < XI; ++i) src[4 + i] = a.x + (size_t)a.tab.tok[off + min(8 * i + r, n - 1)] * a.d + k;
    st::stream<BF16, 2, XI, D>(acc, ring, src, b1 - b0, b1 == blocks ? a.d - 64 * (blocks - 1) : 64, lane);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < R::kFrag; ++j) out[m][j] = acc[m][j];
}

// XM: groups of 8 tokens that an expert can have (1, 2 or 4); P waves share 16 channels
template <bool BF16, int XM, int D>
__global__ void __launch_bounds__(1024)
few_gateup_kernel(FewArgs a, int P, int slice)
{
    constexpr int NB = (XM + 1) / 2;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
    const int G = waves / P, g = wave / P, p = wave - g * P;
    const int fb = (a.f + 15) / 16, units = *a.tab.n * fb;
    const int u0 = blockIdx.x * G;
    if (u0 >= units) return;
    const int blocks = (a.d + 63) / 64, b0 = p * slice, b1 = min(b0 + slice, blocks);
    floatx4 acc[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[m][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (u0 + g < units && b0 < b1) {
        const int i = (u0 + g) / fb, c = (u0 + g) - i * fb;
        const int e = a.tab.expert[i], off = a.tab.off[i], n = a.tab.off[i + 1] - off;
        unsigned char *ring = smem + wave * D * st::Ring<2, XM>::kBlock;
        if (XM == 1 || n <= 8) gateup_wave<BF16, 1, D>(a, ring, e, c, off, n, b0, b1, blocks, lane, acc);
        else if (XM == 2 || n <= 16) gateup_wave<BF16, 2, D>(a, ring, e, c, off, n, b0, b1, blocks, lane, acc);
        else gateup_wave<BF16, 4, D>(a, ring, e, c, off, n, b0, b1, blocks, lane, acc);
    }
    __syncthreads();                                // the rings are done with
    float *red = (float *)smem;                     // [waves][2][NB][64 lanes][4]
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j) *(floatx4 *)&red[((wave * 2 + m) * NB + j) * 256 + 4 * lane] = acc[m][j];
    __syncthreads();
    for (int q = tid; q < G * NB * 256; q += blockDim.x) {
        const int gg = q / (NB * 256), el = q - gg * NB * 256;
        const int t = el >> 4, r = el & 15;         // the expert's t-th token, channel of the group
        if (u0 + gg >= units) continue;
        const int i = (u0 + gg) / fb, ch = 16 * (u0 + gg - i * fb) + r;
        const int off = a.tab.off[i];
        if (ch >= a.f || t >= a.tab.off[i + 1] - off) continue;
        const int pos = (t >> 4) * 256 + 4 * ((t & 15) + 16 * (r >> 2)) + (r & 3);
        float v[2] = {0.f, 0.f};
        for (int z = 0; z < P; ++z)
#pragma unroll
            for (int m = 0; m < 2; ++m) v[m] += red[((gg * P + z) * 2 + m) * NB * 256 + pos];
        const float h = silu(v[0]) * v[1];
        const uint16_t hi = st::to16<BF16>(h);
        const float back = st::from16<BF16>(hi);
        // an infinite or NaN h stands in hi alone
        const uint16_t lo = fabsf(back) < INFINITY ? st::to16<BF16>(h - back) : (uint16_t)0;
        uint16_t *dst = a.h + (size_t)(off + t) * 2 * a.f + ch;
        dst[0] = hi;
        dst[a.f] = lo;
    }
}

// One wave's share of one expert: 16 columns, blocks [b0, b1) of its channels;
// the 2 n columns of the matrix core are hi, then lo of its n tokens.  The
// weighted sum goes into y [T][16], this wave's own LDS.
template <bool BF16, int XI, int D>
__device__ __forceinline__ void down_wave(const FewArgs &a, unsigned char *ring, float *y, int e, int col, int off,
                                          int n, int b0, int b1, int blocks, int lane)
{
    using R = st::Ring<1, XI>;
    floatx4 acc[1][R::kFrag];
#pragma unroll
    for (int j = 0; j < R::kFrag; ++j) acc[0][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int r = st::copy_row(lane), k = 64 * b0 + st::copy_k(lane);
    const uint16_t *src[R::kCopies];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        src[i] = a.down_t + ((size_t)e * a.d + min(col + 8 * i + r, a.d - 1)) * a.f + k;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int v = min(8 * i + r, 2 * n - 1);
        src[2 + i] = a.h + ((size_t)(off + (v < n ? v : v - n)) * 2 + (v < n ? 0 : 1)) * a.f + k;
    }
    st::stream<BF16, 1, XI, D>(acc, ring, src, b1 - b0, b1 == blocks ? a.f - 64 * (blocks - 1) : 64, lane);
    // the hi columns first, then the lo ones: two lanes never add to one place at once
    const int q = lane >> 4;
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int j = 0; j < R::kFrag; ++j) {
            const int v = 16 * j + (lane & 15), t = v - part * n;
            if (t >= 0 && t < n) {
                const float w = a.tab.wt[off + t];
                float *p = y + a.tab.tok[off + t] * 16 + 4 * q;
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] += w * acc[0][j][i];
            }
        }
}

// XM: groups of 8 hi and lo columns that an expert can have (1, 2, 4 or 8)
template <bool BF16, int XM, int D>
__global__ void __launch_bounds__(1024)
few_down_kernel(FewArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    unsigned char *ring = smem + wave * D * st::Ring<1, XM>::kBlock;
    float *ys = (float *)(smem + waves * D * st::Ring<1, XM>::kBlock);  // [waves][T][16]
    float *y = ys + wave * a.T * 16;
    for (int i = lane; i < a.T * 16; i += 64) y[i] = 0.f;
    const int n0 = 16 * blockIdx.x;
    const int n = *a.tab.n, blocks = (a.f + 63) / 64, total = n * blocks;
    const int beg = (int)((long long)total * wave / waves), end = (int)((long long)total * (wave + 1) / waves);
    for (int s = beg; s < end;) {
        const int i = s / blocks, b0 = s - i * blocks, b1 = min(blocks, b0 + end - s);
        s += b1 - b0;
        const int e = a.tab.expert[i], off = a.tab.off[i], m = a.tab.off[i + 1] - off;
        if (XM == 1 || m <= 4) down_wave<BF16, 1, D>(a, ring, y, e, n0, off, m, b0, b1, blocks, lane);
        else if (XM == 2 || m <= 8) down_wave<BF16, 2, D>(a, ring, y, e, n0, off, m, b0, b1, blocks, lane);
        else if (XM == 4 || m <= 16) down_wave<BF16, 4, D>(a, ring, y, e, n0, off, m, b0, b1, blocks, lane);
        else down_wave<BF16, 8, D>(a, ring, y, e, n0, off, m, b0, b1, blocks, lane);
    }
    __syncthreads();
    for (int q = tid; q < a.T * 16; q += blockDim.x) {
        const int t = q >> 4, c = n0 + (q & 15);
        if (c >= a.d) continue;
        float v = 0.f;
        for (int z = 0; z < waves; ++z) v += ys[z * a.T * 16 + q];
        const size_t at = (size_t)t * a.d + c;
        if (a.r) v += st::load_el(a.r, a.ydt, at);
        st::store_el(a.y, a.ydt, at, v);
    }
}

hipError_t allow_lds(const void *k, size_t lds)
{
    if (lds <= 64 * 1024) return hipSuccess;
    return hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
}

template <bool BF16, int XM, int D>
hipError_t gateup(const FewArgs &a, hipStream_t s)
{
    const int blocks = (a.d + 63) / 64, fb = (a.f + 15) / 16;
    const long long units = (long long)fb * a.amax;
    int P = 4;
    while (P < 8 && units * P < 2048 && blocks >= 8 * P) P *= 2;
    while (P > 1 && blocks < P) P /= 2;
    const int G = P < 4 ? 4 / P : 1, slice = (blocks + P - 1) / P;
    constexpr size_t ring = (size_t)D * st::Ring<2, XM>::kBlock, red = (XM + 1) / 2 * 2048;
    const size_t lds = G * P * (ring > red ? ring : red);
    const hipError_t e = allow_lds((const void *)few_gateup_kernel<BF16, XM, D>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((few_gateup_kernel<BF16, XM, D>), dim3((unsigned)((units + G - 1) / G)), dim3(64 * G * P), lds, s,
                       a, P, slice);
    return hipGetLastError();
}

template <bool BF16, int XM, int D, int W>
hipError_t down(const FewArgs &a, hipStream_t s)
{
    const size_t lds = (size_t)W * (D * st::Ring<1, XM>::kBlock + a.T * 64);
    const hipError_t e = allow_lds((const void *)few_down_kernel<BF16, XM, D>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((few_down_kernel<BF16, XM, D>), dim3((unsigned)((a.d + 15) / 16)), dim3(64 * W), lds, s, a);
    return hipGetLastError();
}

bool args_ok(const FewArgs &a)
{
    return a.T >= 1 && a.T <= kFewTokens && a.d >= 8 && a.d % 8 == 0 && a.f >= 8 && a.f % 8 == 0 && a.E >= 1 &&
           a.E <= 1024 && a.k >= 1 && a.k <= a.E && a.S >= 0 && (long long)a.T * (a.k + a.S) <= kFewRows && a.amax >= 1 && a.amax <= kFewRows;
}

}  // namespace

hipError_t launch_few_rank(const FewArgs &a, hipStream_t s)
{
    if (!args_ok(a)) return hipErrorInvalidValue;
    const size_t lds = (size_t)a.T * (((a.E + 3) & ~3) + 2 * a.k) * 4 + (size_t)a.E * 8;
    const hipError_t e = allow_lds((const void *)few_rank_kernel, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(few_rank_kernel, dim3(1), dim3(1024), lds, s, a);
    return hipGetLastError();
}

hipError_t launch_few_gateup(const FewArgs &a, hipStream_t s)
{
    if (!args_ok(a)) return hipErrorInvalidValue;
    if (a.T <= 8) return a.bf16 ? gateup<true, 1, 3>(a, s) : gateup<false, 1, 3>(a, s);
    if (a.T <= 16) return a.bf16 ? gateup<true, 2, 3>(a, s) : gateup<false, 2, 3>(a, s);
    return a.bf16 ? gateup<true, 4, 3>(a, s) : gateup<false, 4, 3>(a, s);
}

hipError_t launch_few_down(const FewArgs &a, hipStream_t s)
{
    if (!args_ok(a)) return hipErrorInvalidValue;
    if (a.T <= 4) return a.bf16 ? down<true, 1, 4, 8>(a, s) : down<false, 1, 4, 8>(a, s);
    if (a.T <= 8) return a.bf16 ? down<true, 2, 4, 8>(a, s) : down<false, 2, 4, 8>(a, s);
    if (a.T <= 16) return a.bf16 ? down<true, 4, 3, 8>(a, s) : down<false, 4, 3, 8>(a, s);
    return a.bf16 ? down<true, 8, 3, 4>(a, s) : down<false, 8, 3, 4>(a, s);
}

}  // namespace moeffn
