// A whole dense MoE layer for at most 32 tokens (MoE-Infinity review, "A3 背景"
// and FloE review, "MoE 专家前向计算": top-k routing, SwiGLU experts):
//   y_t = r_t + sum_s w_ts a_e(t,s)(x_t) + sum_i a_E+i(x_t),
//   a_e(x) = (SiLU(x G_e) (.) (x U_e)) D_e.
// Bound by the weights of the chosen experts, streamed past the tokens that chose
// each (mfma_stream.hpp), in two kernels:
//   gate/up: a wave takes 16 channels of a listed expert and a slice of d;
//            h = SiLU(g) u goes to the workspace;
//   down:    a workgroup takes 16 columns of y and a share of the listed
//            experts' channels laid end to end; the last of a column's
//            workgroups to finish adds their partial sums in order.
// Before them the router, unless it is so small that every gate/up workgroup
// works it out for itself (see launch_few).
// 64 experts of 2048 x 1408, top-6, and 2 shared ones: one token 32 us (139 MB in
// kernels of 3.1 + 18.3 + 12.5 us, short streams), 32 tokens 200-209 us (1.1 GB, 5.3
// TB/s: 4.5 + 10.6 + 125 + 68).  8 of 4096 x 14336, top-2, 4 tokens (5 or 6 of them
// chosen): 297-351 us, gate/up at 6.1-6.3 TB/s.
// h is kept as a sum of terms of the 16-bit type, each the rounding of what those
// before it leave: three, which hold the 24 bits of fp32 (two of bf16 hold 17, which
// turns one rounding of a bf16 y in a thousand), or two where the layer and y are both
// fp16: 22 bits, of which y shows 11.  In fp16 the second is kept times 2^11 and the
// third times 2^22 (kTermScale), since the rest of an h below 2^-3 lies among fp16's
// subnormals, whose steps are coarser than 2^-22 of it; of an h down to 2^-14 the
// second then loses nothing.
// The terms go through the matrix core as tokens of their own, which mostly fill
// columns that would idle.  A column of the matrix core depends on its own token
// alone, so infinities and NaN stay with the tokens whose experts hold them.
#include "internal.hpp"
#include "linear.hpp"
#include "mfma_stream.hpp"
#include "route_common.hpp"
#include <type_traits>

namespace moeffn {

namespace {

using st::floatx4;

// What each term of h is kept times, over the one before.  The rest of a term is at
// most half a step of it, 16, so that its product stays below fp16's 65504; bf16
// has fp32's exponents.
template <bool BF16>
constexpr float kTermScale = BF16 ? 1.f : 2048.f;

// A listed expert, one 16-byte load: {expert or -1, its tokens as bits, first row,
// down_cost of the experts before it}.  Its r-th token is the r-th set bit and has row
// first + r.
__device__ __forceinline__ int nth_bit(uint32_t mask, int r)
{
    for (; r > 0; --r) mask &= mask - 1;
    return __ffs(mask) - 1;
}

// Rows of h that a pass of the down product over m <= 16 tokens copies
__device__ __forceinline__ int down_rows(int m, int terms)
{
    const int r = m * terms;
    return r <= 8 ? 8 : r <= 16 ? 16 : terms == 2 ? 32 : r <= 24 ? 24 : 48;
}

// What a block of an expert with n tokens costs in the down product, in half KB of
// weights copied from HBM and, at half the price, of rows of h from L2.
__device__ __forceinline__ int down_cost(int n, int terms)
{
    auto pass = [=](int m) { return 4 + down_rows(m, terms) / 8; };
    return n <= 16 ? pass(n) : pass(16) + pass(n - 16);
}

// The largest of the wave's 64 values, in every lane
__device__ __forceinline__ float wave_max(float v)
{
    // lanes l ^ 1, l ^ 2, then the mirror images within 8 and 16 lanes, then rows
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, false)));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, false)));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, false)));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, false)));
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The k best of E <= 64 N experts by one wave, in registers, in the order that
// rank_topk ranks by: larger logit, then lower index, NaN as -inf.  emit(s, e)
// gets them best first; took[j] are the experts 64 j + bit among them.  k rounds
// of an arg-max over the lanes: for a few choices far fewer instructions than
// counting, for each expert, those ahead of it.
constexpr int kSelect = 16;                         // choices up to which this is the shorter way
template <int N, class F>
__device__ __forceinline__ void select(const float *lg, int E, int k, int lane, unsigned long long (&took)[N], F emit)
{
    float v[N];                                     // logit of expert 64 j + lane
    bool left[N];                                   // and whether it may still be chosen
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = lane + 64 * j;
        left[j] = e < E;
        took[j] = 0ull;
        const float l = left[j] ? lg[e] : -INFINITY;
        v[j] = l != l ? -INFINITY : l;
    }
    for (int s = 0; s < k; ++s) {
        float best = -INFINITY;
#pragma unroll
        for (int j = 0; j < N; ++j) best = fmaxf(best, left[j] ? v[j] : -INFINITY);
        best = wave_max(best);
        int e = -1;
#pragma unroll
        for (int j = N - 1; j >= 0; --j) {          // the lowest that has it
            const unsigned long long b = __ballot(left[j] && v[j] == best);
            e = b ? 64 * j + __ffsll(b) - 1 : e;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const bool it = e == 64 * j + lane;
            left[j] = left[j] && !it;
            took[j] |= __ballot(it);
        }
        emit(s, e);
    }
}

template <int N>
__device__ __forceinline__ void select_to(const float *lg, int E, int k, int lane, int *to)
{
    unsigned long long took[N];
    select<N>(lg, E, k, lane, took, [&](int s, int e) { if (lane == 0) to[s] = e; });
}

// One token: the i-th in ascending order of its k <= kSelect best experts
template <int N>
__device__ __forceinline__ int pick_of(const float *lg, int E, int k, int i, int lane)
{
    unsigned long long took[N];
    select<N>(lg, E, k, lane, took, [](int, int) {});
    int e = -1;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = __popcll(took[j]);
        if (e < 0 && i < c) {
            unsigned long long b = took[j];
            for (; i > 0; --i) b &= b - 1;
            e = 64 * j + __ffsll(b) - 1;
        }
        i -= c;
    }
    return e;
}

__device__ __forceinline__ int pick(const float *lg, int E, int k, int i, int lane)
{
    if (E <= 64) return pick_of<1>(lg, E, k, i, lane);
    return E <= 256 ? pick_of<4>(lg, E, k, i, lane) : pick_of<16>(lg, E, k, i, lane);
}

// Bytes of LDS that route() works in
__host__ __device__ inline size_t route_bytes(int T, int E, int k)
{
    return (size_t)T * ((E + 3) & ~3) * 4 + (size_t)T * k * 8 + (size_t)E * 8 + 16;
}

// Ranks the logits and lists the experts, by one workgroup.  LOGITS: forms the
// logits too.  rec [amax + 1] (LDS or global); wt: the rows' router weights, or null
// where another workgroup writes them with the call's exports.
template <bool BF16, bool LOGITS>
__device__ void route(const FewArgs &a, int4 *rec, unsigned char *smem, bool exports)
{
    const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 63, wave = tid >> 6, waves = nthr >> 6;
    const int E = a.E, E4 = (E + 3) & ~3, k = a.k;
    float *lg = (float *)smem;                      // [T][E4], padded with -inf
    int *sel = (int *)(lg + a.T * E4);              // [T][k]
    float *w = (float *)(sel + a.T * k);            // [T][k]
    uint32_t *em = (uint32_t *)(w + a.T * k);       // [E] bit t: token t goes to the expert
    int *eo = (int *)(em + E);                      // [E] first row
    int *count = eo + E;
    for (int e = tid; e < E; e += nthr) em[e] = 0u;
    if constexpr (LOGITS) {
        for (int i = wave; i < a.T * E; i += waves) {
            const int t = i / E, e = i - t * E;
            const float v = rc::wave_logit_rows<BF16 ? 1 : 0>(a.x + (size_t)t * a.d, a.rw, a.rdt, a.d, a.rbias, e, lane);
            if (lane == 0) lg[t * E4 + e] = v;
        }
        for (int i = tid; i < a.T * (E4 - E); i += nthr) lg[i / (E4 - E) * E4 + E + i % (E4 - E)] = -INFINITY;
    } else {
        for (int i = tid; i < a.T * E4; i += nthr) {
            const int t = i / E4, e = i - t * E4;
            lg[i] = e < E ? a.lg[(size_t)t * E + e] : -INFINITY;
        }
    }
    __syncthreads();
    for (int t = wave; t < a.T; t += waves) {
        int *to = sel + t * k;
        if (k > kSelect) rc::rank_topk(lg + t * E4, E, k, to, lane, 64);
        else if (E <= 64) select_to<1>(lg + t * E4, E, k, lane, to);
        else if (E <= 256) select_to<4>(lg + t * E4, E, k, lane, to);
        else select_to<16>(lg + t * E4, E, k, lane, to);
    }
    __syncthreads();
    for (int t = wave; t < a.T; t += waves) {
        const float *row = lg + t * E4;
        const int *st = sel + t * k;
        const float m = row[st[0]], den = rc::gate_den(row, st, E, k, a.renorm, m, lane);
        for (int s = lane; s < k; s += 64) {
            w[t * k + s] = __expf(row[st[s]] - m) / den;
            atomicOr(&em[st[s]], 1u << t);
        }
    }
    __syncthreads();
    if (wave == 0) {
        int na = 0, rows = 0, cost = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const uint32_t m = e0 + lane < E ? em[e0 + lane] : 0u;
            const unsigned long long b = __ballot(m != 0u);
            // rows (at most 32 x 64 here) and costs, scanned together
            const int c = __popc(m), v0 = c | (m ? down_cost(c, a.terms) : 0) << 16;
            int incl = v0;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(incl, o, 64);
                if (lane >= o) incl += v;
            }
            if (m) {
                const int off = rows + ((incl - v0) & 0xFFFF);
                rec[na + __popcll(b & ((1ull << lane) - 1ull))] = make_int4(e0 + lane, (int)m, off, cost + ((incl - v0) >> 16));
                eo[e0 + lane] = off;
            }
            na += __popcll(b);
            const int sum = __shfl(incl, 63, 64);
            rows += sum & 0xFFFF;
            cost += sum >> 16;
        }
        const uint32_t all = 0xFFFFFFFFu >> (32 - a.T);
        for (int i = na + lane; i <= a.amax; i += 64) {
            const int sh = i - na;
            const int w = cost + min(sh, a.S) * down_cost(a.T, a.terms);
            rec[i] = sh < a.S ? make_int4(E + sh, (int)all, rows + sh * a.T, w) : make_int4(-1, 0, 0, w);
        }
        if (lane == 0) *count = na + a.S;
    }
    __syncthreads();
    if (exports) {
        if (tid == 0) *a.tab.n = *count;
        for (int p = tid; p < a.T * k; p += nthr) {
            const int t = p / k, e = sel[p];
            a.tab.wt[eo[e] + __popc(em[e] & ((1u << t) - 1u))] = w[p];
            if (a.topk_idx) a.topk_idx[p] = e;
            if (a.topk_w) a.topk_w[p] = w[p];
        }
        for (int p = tid; p < a.T * a.S; p += nthr) a.tab.wt[a.T * k + p] = 1.f;
        if (a.logits)
            for (int i = tid; i < a.T * E; i += nthr) a.logits[i] = lg[i / E * E4 + i % E];
        for (int e = tid; e < E; e += nthr) {
            const int c = __popc(em[e]);
            if (a.count) a.count[e] = c;
            if (a.eam_row) a.eam_row[e] += c;
            if (a.expert_dense) a.expert_dense[e] = c > 0 ? 1 : 0;
        }
        for (int i = tid; i < (a.d + 15) / 16; i += nthr) a.tab.done[i] = 0;
    }
    __syncthreads();                                // the scratch is free, the list complete
}

__global__ void __launch_bounds__(1024)
few_rank_kernel(FewArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    route<false, false>(a, a.tab.rec, smem, true);
}

// Gate and up products of one wave: 16 channels from c, the expert's n tokens (at
// most XR), blocks [b0, b1) of d.
template <bool BF16, int XR, int D>
__device__ __forceinline__ void gateup_wave(const FewArgs &a, unsigned char *ring, int e, uint32_t mask, int n, int c,
                                            int b0, int b1, int blocks, int lane, floatx4 (&out)[2][2])
{
    using R = st::Ring<2, XR>;
    floatx4 acc[2][R::kFrag];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < R::kFrag; ++j) acc[m][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int r = st::copy_row(lane), k = 64 * b0 + st::copy_k(lane);
    const uint16_t *src[R::kCopies];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ch = min(c + 8 * (i & 1) + r, a.f - 1);
        src[i] = (i < 2 ? a.gate : a.up) + ((size_t)e * a.f + ch) * a.d + k;
    }
#pragma unroll
    for (int i = 0; i < R::kTok; ++i) src[4 + i] = a.x + (size_t)nth_bit(mask, min(8 * i + r, n - 1)) * a.d + k;
    st::stream<BF16, 2, XR, D>(acc, ring, src, b1 - b0, b1 == blocks ? a.d - 64 * (blocks - 1) : 64, lane);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < R::kFrag; ++j) out[m][j] = acc[m][j];
}

// Bytes of a wave's ring in a kernel for at most xm token rows (rows of h in the
// down product), and its depth where blocks hold xr of them: 3 or 4
// blocks at xm rows, as many as fit with fewer.  (Three terms take 3, so that as
// many workgroups share a compute unit as with two.)
constexpr int kUpRing(int xm) { return 3 * (4096 + 128 * xm); }
constexpr int kUpDepth(int xm, int xr) { return kUpRing(xm) / (4096 + 128 * xr); }
constexpr int kDownM(int xm) { return xm <= 24 ? 1 : 2; }  // groups of 16 columns
constexpr int kDownRing(int terms, int xm)
{
    return (terms == 3 && xm > 8 ? 3 : 4) * (2048 * kDownM(xm) + 128 * xm);
}
constexpr int kDownDepth(int terms, int xm, int xr) { return kDownRing(terms, xm) / (2048 * kDownM(xm) + 128 * xr); }

// Where the gate/up kernel has the list from
enum { kFromList = 0, kFromLogits = 1, kFromRouter = 2 };

// XM: tokens that an expert can have (1, 8, 16 or 32); P waves share 16 channels
template <bool BF16, int XM, int ROUTE>
__global__ void __launch_bounds__(512)
few_gateup_kernel(FewArgs a, int P, int slice)
{
    constexpr int NB = (XM + 15) / 16;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
    const int G = waves / P, g = wave / P, p = wave - g * P;
    const int fb = (a.f + 15) / 16, units = a.amax * fb;
    const int u0 = blockIdx.x * G;
    unsigned char *rings = smem;
    const int4 *list = a.tab.rec;
    if constexpr (ROUTE == kFromRouter) {
        int4 *own = (int4 *)smem;
        rings += 16 * (size_t)(a.amax + 1);
        route<BF16, true>(a, own, rings, blockIdx.x == 0);
        if (blockIdx.x == 0)
            for (int i = tid; i <= a.amax; i += blockDim.x) a.tab.rec[i] = own[i];
        list = own;
    }
    if constexpr (ROUTE == kFromLogits) {
        // one workgroup lists the experts for the down product
        if (blockIdx.x == 0) route<BF16, false>(a, a.tab.rec, smem, true);
    }
    const int blocks = (a.d + 63) / 64, b0 = p * slice, b1 = min(b0 + slice, blocks);
    auto record = [&](int i) -> int4 {
        if constexpr (ROUTE == kFromLogits)         // one token: expert i in row i
            return make_int4(i < a.k ? pick(a.lg, a.E, a.k, i, lane) : a.E + i - a.k, 1, i, 0);
        return list[i];
    };
    floatx4 acc[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[m][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (u0 + g < units && b0 < b1) {
        const int i = (u0 + g) / fb, c = 16 * (u0 + g - i * fb);
        const int4 rec = record(i);
        const int e = __builtin_amdgcn_readfirstlane(rec.x);
        const uint32_t mask = __builtin_amdgcn_readfirstlane(rec.y);
        const int n = __popc(mask);
        unsigned char *ring = rings + wave * kUpRing(XM);
        if (e >= 0) {
            if constexpr (XM == 1)
                gateup_wave<BF16, 1, kUpDepth(1, 1)>(a, ring, e, mask, n, c, b0, b1, blocks, lane, acc);
            else if (XM == 8 || n <= 8)
                gateup_wave<BF16, 8, kUpDepth(XM, 8)>(a, ring, e, mask, n, c, b0, b1, blocks, lane, acc);
            else if (XM == 16 || n <= 16)
                gateup_wave<BF16, 16, kUpDepth(XM, 16)>(a, ring, e, mask, n, c, b0, b1, blocks, lane, acc);
            else gateup_wave<BF16, 32, kUpDepth(XM, 32)>(a, ring, e, mask, n, c, b0, b1, blocks, lane, acc);
        }
    }
    __syncthreads();                                // the rings are done with
    float *red = (float *)rings;                    // [waves][2][NB][64 lanes][4]
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
        int off = i, n = 1;
        if constexpr (ROUTE != kFromLogits) {
            off = list[i].z;
            n = list[i].x < 0 ? 0 : __popc((uint32_t)list[i].y);
        }
        if (ch >= a.f || t >= n) continue;
        const int pos = (t >> 4) * 256 + 4 * ((t & 15) + 16 * (r >> 2)) + (r & 3);
        float v[2] = {0.f, 0.f};
        for (int z = 0; z < P; ++z)
#pragma unroll
            for (int m = 0; m < 2; ++m) v[m] += red[((gg * P + z) * 2 + m) * NB * 256 + pos];
        float h = silu(v[0]) * v[1];
        uint16_t *dst = a.h + (size_t)(off + t) * a.terms * a.f + ch;
        for (int z = 0; z < a.terms; ++z) {
            const uint16_t term = st::to16<BF16>(h);
            const float back = st::from16<BF16>(term);
            dst[(size_t)z * a.f] = term;
            // an infinite or NaN h stands in the first term alone
            h = fabsf(back) < INFINITY ? (h - back) * kTermScale<BF16> : 0.f;
        }
    }
}

// One wave's share of one expert: 16 NM columns from col, blocks [b0, b1) of its
// channels, tokens first .. first + n - 1 of the expert's; the TERMS n columns of the
// matrix core are the first terms of the n tokens' h, then the second, then the third.
// The weighted sum goes into y [T][16 NM], this wave's own LDS.
template <bool BF16, int TERMS, int NM, int XR, int D>
__device__ __forceinline__ void down_wave(const FewArgs &a, unsigned char *ring, float *y, int4 rec, int first, int n,
                                          int col, int b0, int b1, int blocks, int lane)
{
    using R = st::Ring<NM, XR>;
    floatx4 acc[NM][R::kFrag];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int j = 0; j < R::kFrag; ++j) acc[m][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int off = rec.z + first;
    const int r = st::copy_row(lane), k = 64 * b0 + st::copy_k(lane);
    const uint16_t *src[R::kCopies];
#pragma unroll
    for (int i = 0; i < 2 * NM; ++i)
        src[i] = a.down_t + ((size_t)rec.x * a.d + min(col + 8 * i + r, a.d - 1)) * a.f + k;
#pragma unroll
    for (int i = 0; i < R::kTok; ++i) {
        const int v = min(8 * i + r, TERMS * n - 1), z = v < n ? 0 : v < 2 * n ? 1 : 2;
        src[2 * NM + i] = a.h + ((size_t)(off + v - z * n) * TERMS + z) * a.f + k;
    }
    // this lane's columns: their term (TERMS: none), factor and place in y
    int at[R::kFrag], term[R::kFrag];
    float w[R::kFrag];
#pragma unroll
    for (int j = 0; j < R::kFrag; ++j) {
        const int v = 16 * j + (lane & 15), z = v < n ? 0 : v < 2 * n ? 1 : v < 3 * n ? 2 : 3, t = v - z * n;
        constexpr float s = 1.f / kTermScale<BF16>;
        term[j] = min(z, TERMS);
        at[j] = z < TERMS ? nth_bit((uint32_t)rec.y, first + t) * 16 * NM + 4 * (lane >> 4) : 0;
        w[j] = z < TERMS ? a.tab.wt[off + t] * (z == 0 ? 1.f : z == 1 ? s : s * s) : 0.f;
        // arrived here: else the compiler waits for it inside the stream, and for the
        // copies with it (13 tokens, 8 experts of 4096 x 14336: 150 us against 210)
        asm volatile("" : "+v"(w[j]));
    }
    st::stream<BF16, NM, XR, D>(acc, ring, src, b1 - b0, b1 == blocks ? a.f - 64 * (blocks - 1) : 64, lane);
    // the columns of the first terms, then of the second, then of the third: those of
    // a token lie in different lanes, whose sums must not be read before the
    // others' are written.  Where an infinite weight has made a sum infinite (or NaN)
    // it stays so: a later term times that weight may be an infinity of the other
    // sign, or 0 times it, a NaN.
#pragma unroll
    for (int h = 0; h < TERMS; ++h) {
#pragma unroll
        for (int j = 0; j < R::kFrag; ++j)
            if (term[j] == h)
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = y[at[j] + 16 * m + i];
                        const float c = w[j] * acc[m][j][i];
                        y[at[j] + 16 * m + i] = v + (h == 0 || fabsf(v) < INFINITY ? c : 0.f);
                    }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// XM: rows of h that a pass can have (2, 8, 16 or 32 by two terms, 4, 8, 16, 24 or 48
// by three): an expert with more than 16 tokens takes two passes over its weights.
// Workgroup b takes columns
// C (b % nblk) .. and part b / nblk of `parts`; the waves of all parts take
// equal shares of the blocks' costs, in the order of the list.
template <bool BF16, int TERMS, int XM>
__global__ void __launch_bounds__(256)
few_down_kernel(FewArgs a, int parts)
{
    constexpr int NM = kDownM(XM), C = 16 * NM;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    unsigned char *ring = smem + wave * kDownRing(TERMS, XM);
    float *ys = (float *)(smem + waves * kDownRing(TERMS, XM));    // [waves][T][C]
    float *y = ys + wave * a.T * C;
    for (int i = lane; i < a.T * C; i += 64) y[i] = 0.f;
    const int nblk = (a.d + C - 1) / C, part = blockIdx.x / nblk, blk = blockIdx.x - part * nblk;
    const int n0 = C * blk;
    const int blocks = (a.f + 63) / 64, share = part * waves + wave, shares = parts * waves;
    if constexpr (XM < 8) {
        // one token: every listed expert has it
        const long long total = (long long)a.amax * blocks;
        const int beg = (int)(total * share / shares), end = (int)(total * (share + 1) / shares);
        for (int s = beg; s < end;) {
            const int i = s / blocks, b0 = s - i * blocks, b1 = min(blocks, b0 + end - s);
            s += b1 - b0;
            down_wave<BF16, TERMS, NM, XM, kDownDepth(TERMS, XM, XM)>(a, ring, y, a.tab.rec[i], 0, 1, n0, b0, b1, blocks, lane);
        }
    } else {
        // a list entry's w is the cost of the blocks of one column before it / blocks
        const int n = *a.tab.n;
        const long long total = (long long)a.tab.rec[n].w * blocks;
        const long long beg = total * share / shares, end = total * (share + 1) / shares;
        int i = -1;                                 // the last entry at or before beg
        for (int i0 = 0; i0 < n; i0 += 64)
            i += __popcll(__ballot(i0 + lane < n && (long long)a.tab.rec[i0 + min(lane, n - 1 - i0)].w * blocks <= beg));
        for (; i < n; ++i) {
            const int4 rec = a.tab.rec[i];
            const int all = __popc((uint32_t)rec.y), cost = down_cost(all, TERMS);
            const long long at = (long long)rec.w * blocks;
            if (at >= end) break;
            // the blocks that begin within the share
            const int b0 = beg > at ? (int)((beg - at + cost - 1) / cost) : 0;
            const int b1 = (int)min((long long)blocks, (end - at + cost - 1) / cost);
            if (b0 >= b1) continue;
            for (int first = 0; first < all; first += 16) {
                const int m = min(16, all - first);
                const int rows = down_rows(m, TERMS);
                auto pass = [&](auto xr) {
                    constexpr int XR = decltype(xr)::value;
                    down_wave<BF16, TERMS, NM, XR, kDownDepth(TERMS, XM, XR)>(a, ring, y, rec, first, m, n0, b0, b1, blocks, lane);
                };
                if (XM == 8 || rows == 8) pass(std::integral_constant<int, 8>());
                else if (XM == 16 || rows == 16) pass(std::integral_constant<int, XM < 16 ? XM : 16>());
                else if (XM == 24 || rows == 24) pass(std::integral_constant<int, XM < 24 ? XM : 24>());
                else pass(std::integral_constant<int, XM>());
            }
        }
    }
    __syncthreads();
    auto finish = [&](int t, int c, float v) {
        const size_t at = (size_t)t * a.d + c;
        if (a.r) v += st::load_el(a.r, a.ydt, at);
        st::store_el(a.y, a.ydt, at, v);
    };
    for (int q = tid; q < a.T * C; q += blockDim.x) {
        const int t = q / C, c = n0 + q % C;
        if (c >= a.d) continue;
        float v = 0.f;
        for (int z = 0; z < waves; ++z) v += ys[z * a.T * C + q];
        if (parts == 1) finish(t, c, v);
        else store_coherent(a.part + ((size_t)part * a.T + t) * a.d + c, v);
    }
    if (parts == 1) return;
    // The parts are written and read by device-scope accesses, which go past the
    // caches of one XCD, and each thread waits for its stores to arrive before its
    // workgroup is counted: no fence, which would write back and drop the L2 that the
    // other workgroups stream through (68 us against 13 on the fine-grained layer).
    // The workgroup that counts last adds the parts in order, so which one that
    // is does not show.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(a.tab.done + blk, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
    __syncthreads();
    if (!last) return;
    for (int q = tid; q < a.T * C; q += blockDim.x) {
        const int t = q / C, c = n0 + q % C;
        if (c >= a.d) continue;
        float v = 0.f;
        for (int z = 0; z < parts; ++z) v += load_coherent(a.part + ((size_t)z * a.T + t) * a.d + c);
        finish(t, c, v);
    }
}

hipError_t allow_lds(const void *k, size_t lds)
{
    if (lds <= 64 * 1024) return hipSuccess;
    return hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
}

template <bool BF16, int XM, int ROUTE>
hipError_t gateup(const FewArgs &a, hipStream_t s)
{
    const int blocks = (a.d + 63) / 64, fb = (a.f + 15) / 16;
    const long long units = (long long)fb * a.amax;
    constexpr int kMost = 160 * 1024;
    static_assert(4 * kUpRing(XM) <= kMost, "four waves' rings fit a compute unit");
    const size_t rb = ROUTE == kFromList ? 0 : route_bytes(a.T, a.E, a.k);
    const size_t list = ROUTE == kFromRouter ? 16 * (size_t)(a.amax + 1) : 0;
    // slices of d, as the linear layer's of K
    int P = 4;
    if (8 * kUpRing(XM) + list <= kMost && units * P < 2048 && blocks >= 8 * P) P = 8;
    while (P > 1 && blocks < P) P /= 2;
    const int G = P < 4 ? 4 / P : 1, slice = (blocks + P - 1) / P;
    static_assert(kUpRing(XM) >= (XM + 15) / 16 * 2048, "the sums fit the rings");
    size_t lds = (size_t)G * P * kUpRing(XM);
    if (rb > lds) lds = rb;
    lds += list;
    const hipError_t e = allow_lds((const void *)few_gateup_kernel<BF16, XM, ROUTE>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((few_gateup_kernel<BF16, XM, ROUTE>), dim3((unsigned)((units + G - 1) / G)), dim3(64 * G * P),
                       lds, s, a, P, slice);
    return hipGetLastError();
}

template <bool BF16>
hipError_t gateup_for(const FewArgs &a, int route, hipStream_t s)
{
    if (a.T == 1) {
        if (route == kFromRouter) return gateup<BF16, 1, kFromRouter>(a, s);
        return route == kFromLogits ? gateup<BF16, 1, kFromLogits>(a, s) : gateup<BF16, 1, kFromList>(a, s);
    }
    if (a.T <= 8) return route == kFromRouter ? gateup<BF16, 8, kFromRouter>(a, s) : gateup<BF16, 8, kFromList>(a, s);
    return a.T <= 16 ? gateup<BF16, 16, kFromList>(a, s) : gateup<BF16, 32, kFromList>(a, s);
}

template <bool BF16, int TERMS, int XM>
hipError_t down(const FewArgs &a, hipStream_t s)
{
    constexpr int W = 4;
    constexpr int C = 16 * kDownM(XM);
    const size_t lds = (size_t)W * (kDownRing(TERMS, XM) + a.T * C * 4);
    const hipError_t e = allow_lds((const void *)few_down_kernel<BF16, TERMS, XM>, lds);
    if (e != hipSuccess) return e;
    const int parts = few_parts(a.T, a.d, a.f, a.E, a.k, a.S);
    hipLaunchKernelGGL((few_down_kernel<BF16, TERMS, XM>), dim3((unsigned)((a.d + C - 1) / C * parts)), dim3(64 * W), lds, s,
                       a, parts);
    return hipGetLastError();
}

template <bool BF16>
hipError_t down_for(const FewArgs &a, hipStream_t s)
{
    if constexpr (!BF16)
        if (a.terms == 2) {
            if (a.T == 1) return down<BF16, 2, 2>(a, s);
            if (a.T <= 4) return down<BF16, 2, 8>(a, s);
            return a.T <= 8 ? down<BF16, 2, 16>(a, s) : down<BF16, 2, 32>(a, s);
        }
    if (a.T == 1) return down<BF16, 3, 4>(a, s);
    if (a.T <= 2) return down<BF16, 3, 8>(a, s);
    if (a.T <= 5) return down<BF16, 3, 16>(a, s);
    return a.T <= 8 ? down<BF16, 3, 24>(a, s) : down<BF16, 3, 48>(a, s);
}

bool args_ok(const FewArgs &a)
{
    return a.T >= 1 && a.T <= kFewTokens && a.d >= 8 && a.d % 8 == 0 && a.f >= 8 && a.f % 8 == 0 && a.E >= 1 &&
           a.E <= 1024 && a.k >= 1 && a.k <= a.E && a.S >= 0 && (long long)a.T * (a.k + a.S) <= kFewRows && a.amax >= 1 && a.amax <= kFewRows;
}

}  // namespace

int few_amax(int T, int E, int k, int S) { return (E < T * k ? E : T * k) + S; }

// Workgroups per column block of y (16 columns, 32 from 9 tokens on): about three
// per compute unit in all, one where their rings fill it, while each of the 4 waves keeps 6
// blocks of 64 channels
int few_parts(int T, int d, int f, int E, int k, int S)
{
    const int c = T <= 8 ? 16 : 32, nblk = (d + c - 1) / c, want = T <= 8 ? 768 : 256;
    const long long most = (long long)few_amax(T, E, k, S) * ((f + 63) / 64) / 24;
    int p = (want + nblk - 1) / nblk;
    if (p > most) p = most < 1 ? 1 : (int)most;
    if (p > 32) p = 32;
    // one token: shares that start and end with an expert, where a count near p gives them
    const int n = few_amax(T, E, k, S);
    if (T == 1)
        for (int d1 = 0; d1 <= p / 3; ++d1) {
            if (4 * (p + d1) % n == 0 && p + d1 <= 32 && p + d1 <= most) return p + d1;
            if (4 * (p - d1) % n == 0) return p - d1;
        }
    return p;
}

// (the layer in us, two terms and an fp16 y, three and an fp32 y: 64 experts of 2048 x
// 1408, top-6, 4 tokens 82 and 83, 32 224 and 231; 8 of 4096 x 14336, top-2, 312 and 315,
// 491 and 511)
static int few_terms(int bf16, int ydt) { return !bf16 && ydt == 0 ? 2 : kFewTerms; }

hipError_t launch_few(const FewArgs &args, hipStream_t s)
{
    if (!args_ok(args)) return hipErrorInvalidValue;
    FewArgs a = args;
    a.terms = few_terms(a.bf16, a.ydt);
    // Who works the router out.  Every gate/up workgroup for itself where that
    // takes less than a kernel more: all of it up to 32768 products, for one token the choice
    // alone; both only in layers of about one round of workgroups (1024), since each pays.
    const long long units = (long long)a.amax * ((a.f + 15) / 16);
    int route = kFromList;
    if (units <= 1024) {
        if (a.T <= 8 && (long long)a.T * a.E * a.d <= 32768) route = kFromRouter;
        else if (a.T == 1 && a.k <= kSelect) route = kFromLogits;
    }
    hipError_t e = hipSuccess;
    if (route != kFromRouter) {
        RouteArgs r{};
        r.x = a.x; r.xdt = a.bf16; r.T = a.T; r.d = a.d;
        r.rw = a.rw; r.rdt = a.rdt; r.bias = a.rbias;
        r.E = a.E;
        r.lg_buf = a.lg;
        e = launch_route_logits(r, s);
        if (e != hipSuccess) return e;
    }
    if (route == kFromList) {
        const size_t lds = route_bytes(a.T, a.E, a.k);
        e = allow_lds((const void *)few_rank_kernel, lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(few_rank_kernel, dim3(1), dim3(1024), lds, s, a);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    e = a.bf16 ? gateup_for<true>(a, route, s) : gateup_for<false>(a, route, s);
    if (e != hipSuccess) return e;
    return a.bf16 ? down_for<true>(a, s) : down_for<false>(a, s);
}

}  // namespace moeffn
