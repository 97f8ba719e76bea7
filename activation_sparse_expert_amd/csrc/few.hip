// A whole dense MoE layer for at most 32 tokens (MoE-Infinity review, "A3 背景"
// and FloE review, "MoE 专家前向计算": top-k routing, SwiGLU experts):
//   y_t = r_t + sum_s w_ts a_e(t,s)(x_t) + sum_i a_E+i(x_t),
//   a_e(x) = (SiLU(x G_e) (.) (x U_e)) D_e.
// Bound by the weights of the chosen experts, read once past the tokens that
// chose each (mfma_stream.hpp), in two kernels:
//   gate/up: a wave takes 16 channels of a listed expert and a slice of d;
//            h = SiLU(g) u goes to the workspace;
//   down:    a workgroup takes 16 columns of y and a share of the listed
//            experts' channels laid end to end; the last of a column's
//            workgroups to finish adds their partial sums in order.
// Before them the router, unless it is so small that every gate/up workgroup
// works it out for itself (see launch_few).
// h is kept as the sum of two values of the 16-bit type (hi = its rounding,
// lo = the rounding of the rest): the products with W^down are then good to
// about 2^-17 (bf16) or 2^-22 (fp16) of h, and the rounding of y is the only one
// that shows.  hi and lo go through the matrix core as two tokens, which mostly fill
// columns that would idle.  A column of the matrix core depends on its own token
// alone, so infinities and NaN stay with the tokens whose experts hold them.
#include "internal.hpp"
#include "linear.hpp"
#include "mfma_stream.hpp"
#include "route_common.hpp"

namespace moeffn {

namespace {

using st::floatx4;

// A listed expert, one 16-byte load: {expert or -1, its tokens as bits, first row, -}.
// Its r-th token is the r-th set bit and has row first + r.
__device__ __forceinline__ int nth_bit(uint32_t mask, int r)
{
    for (; r > 0; --r) mask &= mask - 1;
    return __ffs(mask) - 1;
}

// Bytes of LDS that route() works in
__host__ __device__ inline size_t route_bytes(int T, int E, int k)
{
    return (size_t)T * ((E + 3) & ~3) * 4 + (size_t)T * k * 8 + (size_t)E * 8 + 16;
}

// Ranks the logits and lists the experts, by one workgroup.  LOGITS: forms the
// logits too.  rec [amax] (LDS or global); wt: the rows' router weights, or null
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
    for (int t = wave; t < a.T; t += waves) rc::rank_topk(lg + t * E4, E, k, sel + t * k, lane, 64);
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
                rec[na + __popcll(b & ((1ull << lane) - 1ull))] = make_int4(e0 + lane, (int)m, rows + incl - c, 0);
                eo[e0 + lane] = rows + incl - c;
            }
            na += __popcll(b);
            rows += __shfl(incl, 63, 64);
        }
        const uint32_t all = 0xFFFFFFFFu >> (32 - a.T);
        for (int i = na + lane; i < a.amax; i += 64) {
            const int sh = i - na;
            rec[i] = sh < a.S ? make_int4(E + sh, (int)all, rows + sh * a.T, 0) : make_int4(-1, 0, 0, 0);
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

// One token, E <= 64 kPickLanes: the i-th in ascending order of its k best experts, found by each
// wave in registers (k rounds of an arg-max over the lanes), in the order that
// rank_topk ranks by: larger logit, then lower index; NaN as -inf, -0 as 0.
constexpr int kPick = 8;                            // logits per lane
__device__ __forceinline__ int pick(const float *lg, int E, int k, int i, int lane)
{
    unsigned long long key[kPick];
#pragma unroll
    for (int j = 0; j < kPick; ++j) {
        const int e = lane + 64 * j;
        key[j] = 0ull;                              // below every expert
        if (64 * j < E && e < E) {
            float v = lg[e];
            v = v != v ? -INFINITY : v + 0.f;
            const uint32_t b = __float_as_uint(v);
            key[j] = (unsigned long long)((b & 0x80000000u) ? ~b : b | 0x80000000u) << 32 | (0xFFFFFFFFu - (uint32_t)e);
        }
    }
    uint32_t took = 0u;
    for (int s = 0; s < k; ++s) {
        unsigned long long best = key[0];
#pragma unroll
        for (int j = 1; j < kPick; ++j) best = key[j] > best ? key[j] : best;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const unsigned long long v = __shfl_xor(best, o, 64);
            best = v > best ? v : best;
        }
#pragma unroll
        for (int j = 0; j < kPick; ++j)
            if (key[j] == best) {
                key[j] = 0ull;
                took |= 1u << j;
            }
    }
    int e = -1;
#pragma unroll
    for (int j = 0; j < kPick; ++j) {
        unsigned long long b = __ballot((took >> j) & 1u);
        const int c = __popcll(b);
        if (e < 0 && i < c) {
            for (; i > 0; --i) b &= b - 1;
            e = 64 * j + __ffsll(b) - 1;
        }
        i -= c;
    }
    return __builtin_amdgcn_readfirstlane(e);
}

// Gate and up products of one wave: 16 channels from c, the expert's n tokens (at
// most 8 XI), blocks [b0, b1) of d.
template <bool BF16, int XI, int D>
__device__ __forceinline__ void gateup_wave(const FewArgs &a, unsigned char *ring, int e, uint32_t mask, int n, int c,
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
        const int ch = min(c + 8 * (i & 1) + r, a.f - 1);
        src[i] = (i < 2 ? a.gate : a.up) + ((size_t)e * a.f + ch) * a.d + k;
    }
#pragma unroll
    for (int i = 0; i < XI; ++i) src[4 + i] = a.x + (size_t)nth_bit(mask, min(8 * i + r, n - 1)) * a.d + k;
    st::stream<BF16, 2, XI, D>(acc, ring, src, b1 - b0, b1 == blocks ? a.d - 64 * (blocks - 1) : 64, lane);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < R::kFrag; ++j) out[m][j] = acc[m][j];
}

// Bytes of a wave's ring, and its depth where blocks have XI token rows of 8
constexpr int kUpRing(int xm) { return 3 * st::Ring<2, 1>::kBlock + (xm - 1) * 3 * 1024; }
constexpr int kUpDepth(int xm, int xi) { return kUpRing(xm) / (1024 * (4 + xi)) < 4 ? kUpRing(xm) / (1024 * (4 + xi)) : 4; }
constexpr int kDownRing(int xm) { return xm == 1 ? 12 * 1024 : xm == 2 ? 16 * 1024 : 18 * 1024; }
constexpr int kDownDepth(int xm, int xi) { return kDownRing(xm) / (1024 * (2 + xi)); }

// Where the gate/up kernel has the list from
enum { kFromList = 0, kFromLogits = 1, kFromRouter = 2 };

// XM: groups of 8 tokens that an expert can have (1, 2 or 4); P waves share 16 channels
template <bool BF16, int XM, int ROUTE>
__global__ void __launch_bounds__(512)
few_gateup_kernel(FewArgs a, int P, int slice)
{
    constexpr int NB = (XM + 1) / 2;
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
        rings += 16 * (size_t)a.amax;
        route<BF16, true>(a, own, rings, blockIdx.x == 0);
        if (blockIdx.x == 0)
            for (int i = tid; i < a.amax; i += blockDim.x) a.tab.rec[i] = own[i];
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
            if (XM == 1 || n <= 8)
                gateup_wave<BF16, 1, kUpDepth(XM, 1)>(a, ring, e, mask, n, c, b0, b1, blocks, lane, acc);
            else if (XM == 2 || n <= 16)
                gateup_wave<BF16, 2, kUpDepth(XM, 2)>(a, ring, e, mask, n, c, b0, b1, blocks, lane, acc);
            else gateup_wave<BF16, 4, kUpDepth(XM, 4)>(a, ring, e, mask, n, c, b0, b1, blocks, lane, acc);
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

// One wave's share of one expert: 16 columns from col, blocks [b0, b1) of its
// channels, tokens first .. first + n - 1 of the expert's; the 2 n columns of the matrix
// core are hi, then lo of the n tokens.  The weighted sum goes into y [T][16],
// this wave's own LDS.
template <bool BF16, int XI, int D>
__device__ __forceinline__ void down_wave(const FewArgs &a, unsigned char *ring, float *y, int4 rec, int first, int n,
                                          int col, int b0, int b1, int blocks, int lane)
{
    using R = st::Ring<1, XI>;
    floatx4 acc[1][R::kFrag];
#pragma unroll
    for (int j = 0; j < R::kFrag; ++j) acc[0][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int off = rec.z + first;
    const int r = st::copy_row(lane), k = 64 * b0 + st::copy_k(lane);
    const uint16_t *src[R::kCopies];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        src[i] = a.down_t + ((size_t)rec.x * a.d + min(col + 8 * i + r, a.d - 1)) * a.f + k;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int v = min(8 * i + r, 2 * n - 1);
        src[2 + i] = a.h + ((size_t)(off + (v < n ? v : v - n)) * 2 + (v < n ? 0 : 1)) * a.f + k;
    }
    // this lane's columns: whether hi (0) or lo (1), their router weight and place in y
    int at[R::kFrag], part[R::kFrag];
    float w[R::kFrag];
#pragma unroll
    for (int j = 0; j < R::kFrag; ++j) {
        const int v = 16 * j + (lane & 15), t = v < n ? v : v - n;
        part[j] = v < n ? 0 : v < 2 * n ? 1 : 2;
        at[j] = part[j] < 2 ? nth_bit((uint32_t)rec.y, first + t) * 16 + 4 * (lane >> 4) : 0;
        w[j] = part[j] < 2 ? a.tab.wt[off + t] : 0.f;
    }
    st::stream<BF16, 1, XI, D>(acc, ring, src, b1 - b0, b1 == blocks ? a.f - 64 * (blocks - 1) : 64, lane);
    // the hi columns first, then the lo ones: a token's two columns lie in two
    // lanes, whose sums must not be read before the other's are written
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < R::kFrag; ++j)
            if (part[j] == h)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[at[j] + i] += w[j] * acc[0][j][i];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// XM: groups of 8 hi and lo columns that a pass can have (1, 2 or 4): an expert
// with more than 16 tokens takes two passes over its weights.  Workgroup b takes
// columns 16 (b % nblk) .. and part b / nblk of `parts`.
template <bool BF16, int XM>
__global__ void __launch_bounds__(256)
few_down_kernel(FewArgs a, int parts)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    unsigned char *ring = smem + wave * kDownRing(XM);
    float *ys = (float *)(smem + waves * kDownRing(XM));    // [waves][T][16]
    float *y = ys + wave * a.T * 16;
    for (int i = lane; i < a.T * 16; i += 64) y[i] = 0.f;
    const int nblk = (a.d + 15) / 16, part = blockIdx.x / nblk, blk = blockIdx.x - part * nblk;
    const int n0 = 16 * blk;
    const int n = a.T == 1 ? a.amax : *a.tab.n, blocks = (a.f + 63) / 64;
    const long long total = (long long)n * blocks, share = part * waves + wave, shares = (long long)parts * waves;
    const int beg = (int)(total * share / shares), end = (int)(total * (share + 1) / shares);
    for (int s = beg; s < end;) {
        const int i = s / blocks, b0 = s - i * blocks, b1 = min(blocks, b0 + end - s);
        s += b1 - b0;
        const int4 rec = a.tab.rec[i];
        const int all = __popc((uint32_t)rec.y);
        for (int first = 0; first < all; first += 16) {
            const int m = min(16, all - first);
            if (XM == 1 || m <= 4)
                down_wave<BF16, 1, kDownDepth(XM, 1)>(a, ring, y, rec, first, m, n0, b0, b1, blocks, lane);
            else if (XM == 2 || m <= 8)
                down_wave<BF16, 2, kDownDepth(XM, 2)>(a, ring, y, rec, first, m, n0, b0, b1, blocks, lane);
            else down_wave<BF16, 4, kDownDepth(XM, 4)>(a, ring, y, rec, first, m, n0, b0, b1, blocks, lane);
        }
    }
    __syncthreads();
    auto finish = [&](int t, int c, float v) {
        const size_t at = (size_t)t * a.d + c;
        if (a.r) v += st::load_el(a.r, a.ydt, at);
        st::store_el(a.y, a.ydt, at, v);
    };
    for (int q = tid; q < a.T * 16; q += blockDim.x) {
        const int t = q >> 4, c = n0 + (q & 15);
        if (c >= a.d) continue;
        float v = 0.f;
        for (int z = 0; z < waves; ++z) v += ys[z * a.T * 16 + q];
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
    for (int q = tid; q < a.T * 16; q += blockDim.x) {
        const int t = q >> 4, c = n0 + (q & 15);
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
    int P = 4;
    while (P < 8 && units * P < 2048 && blocks >= 8 * P) P *= 2;
    while (P > 1 && blocks < P) P /= 2;
    const int G = P < 4 ? 4 / P : 1, slice = (blocks + P - 1) / P;
    static_assert(kUpRing(XM) >= (XM + 1) / 2 * 2048, "the sums fit the rings");
    size_t lds = (size_t)G * P * kUpRing(XM);
    const size_t rb = ROUTE == kFromList ? 0 : route_bytes(a.T, a.E, a.k);
    if (rb > lds) lds = rb;
    if (ROUTE == kFromRouter) lds += 16 * (size_t)a.amax;
    const hipError_t e = allow_lds((const void *)few_gateup_kernel<BF16, XM, ROUTE>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((few_gateup_kernel<BF16, XM, ROUTE>), dim3((unsigned)((units + G - 1) / G)), dim3(64 * G * P),
                       lds, s, a, P, slice);
    return hipGetLastError();
}

template <bool BF16>
hipError_t gateup_for(const FewArgs &a, int route, hipStream_t s)
{
    if (a.T <= 8) {
        if (route == kFromRouter) return gateup<BF16, 1, kFromRouter>(a, s);
        return route == kFromLogits ? gateup<BF16, 1, kFromLogits>(a, s) : gateup<BF16, 1, kFromList>(a, s);
    }
    return a.T <= 16 ? gateup<BF16, 2, kFromList>(a, s) : gateup<BF16, 4, kFromList>(a, s);
}

template <bool BF16, int XM>
hipError_t down(const FewArgs &a, hipStream_t s)
{
    constexpr int W = 4;
    const size_t lds = (size_t)W * (kDownRing(XM) + a.T * 64);
    const hipError_t e = allow_lds((const void *)few_down_kernel<BF16, XM>, lds);
    if (e != hipSuccess) return e;
    const int parts = few_parts(a.T, a.d, a.f, a.E, a.k, a.S);
    hipLaunchKernelGGL((few_down_kernel<BF16, XM>), dim3((unsigned)((a.d + 15) / 16 * parts)), dim3(64 * W), lds, s, a,
                       parts);
    return hipGetLastError();
}

bool args_ok(const FewArgs &a)
{
    return a.T >= 1 && a.T <= kFewTokens && a.d >= 8 && a.d % 8 == 0 && a.f >= 8 && a.f % 8 == 0 && a.E >= 1 &&
           a.E <= 1024 && a.k >= 1 && a.k <= a.E && a.S >= 0 && (long long)a.T * (a.k + a.S) <= kFewRows && a.amax >= 1 && a.amax <= kFewRows;
}

}  // namespace

int few_amax(int T, int E, int k, int S) { return (E < T * k ? E : T * k) + S; }

// Workgroups per 16 columns of y: about three per compute unit in all, while
// each of its 4 waves keeps 4 blocks of 64 channels
int few_parts(int T, int d, int f, int E, int k, int S)
{
    const int nblk = (d + 15) / 16;
    const long long most = (long long)few_amax(T, E, k, S) * ((f + 63) / 64) / 16;
    int p = (768 + nblk - 1) / nblk;
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

hipError_t launch_few(const FewArgs &a, hipStream_t s)
{
    if (!args_ok(a)) return hipErrorInvalidValue;
    // Who works the router out.  Every gate/up workgroup for itself where that
    // takes less than a kernel more: all of it up to 32768 products, for one token the choice
    // alone; both only in layers of about one round of workgroups (1024), since each pays.
    const long long units = (long long)a.amax * ((a.f + 15) / 16);
    int route = kFromList;
    if (units <= 1024) {
        if (a.T <= 8 && (long long)a.T * a.E * a.d <= 32768) route = kFromRouter;
        else if (a.T == 1 && a.E <= 64 * kPick && a.k <= 16) route = kFromLogits;
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
    if (a.T <= 4) return a.bf16 ? down<true, 1>(a, s) : down<false, 1>(a, s);
    if (a.T <= 8) return a.bf16 ? down<true, 2>(a, s) : down<false, 2>(a, s);
    return a.bf16 ? down<true, 4>(a, s) : down<false, 4>(a, s);
}

}  // namespace moeffn
