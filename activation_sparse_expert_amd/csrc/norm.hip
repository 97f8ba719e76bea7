// Norms between two blocks: y = rs r + bs g (.) Npost(o), out = Npre(y).  Bound by HBM: a row
// is held in registers by the lanes of part of a wave, or by a workgroup, so that each
// operand is read and written once, and mean and squares are two passes over registers.
// 131072 x 128, bf16: 12.7 us, 5.3 TB/s; 4096 x 6144 between two norms to codes: 41.7 us, 4.2 TB/s
// (three reductions over a workgroup a row, the next row's loads under way); one row 3.0 us, the
// launch.  Layer norms have more to do a value and are bound by instructions where rows are
// short of a block: 8192 x 2048 alone 15.4 us, RMS 14.0.
#include "row_io.hpp"
#include "rows.hpp"

#include <cfloat>

namespace moeffn {

namespace {

// All loads so far have landed.  Which of them a later instruction would wait for depends on operands that
// may be null and on their types, and where the compiler cannot tell it waits for all loads, the
// next row's among them: it is told here, where all are needed.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// The norm of a row in place, n[c] of whose elements each group of this lane holds.  Where a sum
// or the squares pass fp32 everything is taken of values 2^-80 as large, eps of 2^-160 of itself
// (0 below 2^11: beside squares that pass fp32 that is nothing, and of equal values,
// whose sum alone does, v - m is 0 and what is under the root need only not be).
// The mean m is off by what its sum was rounded to, some units in its last place.  Where it is larger
// than the deviation that may be much of what is left of a value, and all of it where values are
// equal: there e = v - m is summed too, its mean `off` is what m is off by, and the squares about
// m + off are sum e^2 - off sum e.  (Of equal values e is a few units in the last place, these sums
// are exact and the norm is 0.)  Only such rows take the third sum: 8192 x 2048 around 5 takes
// 18.1 us, around 0 15.4.
// LAYER: layer norms, whose registers the RMS norms would otherwise hold too (4096 x 6144 between
// two RMS norms to codes: 46 us in one instance with them, 43 apart).
template <bool LAYER, int L, int C, bool WIDE, bool FULL>
__device__ __forceinline__ void norm_row(float (&v)[C][8], const int (&n)[C], rio::Team<L> &team, const NormArgs &a,
                                         const void *w, const rio::Raw<WIDE> (&wr)[C], const void *b)
{
    float m = 0.f, ss, k = 1.f;
    // s / d, which is exact where fp32 holds it
    auto mean = [&](float s) {
        const float q = s * a.inv;
        return fmaf(fmaf(-q, a.len, s), a.inv, q);
    };
    // the row's sum of g(v - m) (RMS: of g(v)) over its own elements; whole groups count or do not
    auto sum = [&](auto g) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = LAYER ? v[c][j] - m : v[c][j];
                t = g(FULL || !LAYER || j < n[c] ? e : 0.f, t);
            }
            s += !FULL || n[c] > 0 ? t : 0.f;
        }
        return team.sum(s);
    };
    const auto plain = [](float e, float t) { return t + e; };
    const auto square = [](float e, float t) { return fmaf(e, e, t); };
    auto stats = [&]() {
        if constexpr (LAYER) {
            m = 0.f;
            m = mean(sum(plain));
        }
        ss = sum(square);
    };
    stats();
    if (__any(!(ss < INFINITY))) {
        k = ss < INFINITY ? 1.f : 0x1p-80f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] *= k;
        stats();
    }
    if constexpr (LAYER) {
        const bool far = m != 0.f && !(m * m < ss * a.inv);             // (so where both are 0 by underflow)
        if (__any(far)) {
            const float s = sum(plain), off = mean(s), sq = fmaf(-s, off, ss);
            ss = far ? (sq < 0.f ? 0.f : sq) : ss;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[c][j] = far ? v[c][j] - m - off : v[c][j];
            m = far ? 0.f : m;
        }
    }
    const float var = ss * a.inv + a.eps * k * k;
    const float f = __builtin_amdgcn_rsqf(var < FLT_MIN ? FLT_MIN : var);      // (a NaN stays one)
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = LAYER ? (v[c][j] - m) * f : v[c][j] * f;
        if (w) {
            float x[8];
            rio::floats<WIDE>(wr[c], a.wdt, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] *= x[j] + a.add;
        }
        if (b) {
            float x[8];
            const rio::Raw<WIDE> br = rio::load<WIDE, FULL>(b, a.wdt, 8 * (team.lane() + c * team.lanes()), n[c], a.d & 7);
            loads_done();
            rio::floats<WIDE>(br, a.wdt, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] += x[j];
        }
        if (!FULL)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] = j < n[c] ? v[c][j] : 0.f;
    }
}

// L, C: lanes of a row and groups of 8 a lane (row_io.hpp); WIDE: some input has 32 bits; FULL:
// d is a multiple of 8; BARE: no block
template <bool LAYER, int L, int C, bool WIDE, bool FULL, bool BARE>
__global__ void __launch_bounds__(L ? 256 : 1024)
norm_kernel(NormArgs a)
{
    __shared__ __align__(16) rio::Slots slots;
    rio::Team<L> team(&slots);
    constexpr int G = L ? 256 / (L ? L : 1) : 1;
    int n[C], at[C];
    rio::Raw<WIDE> rr[C], orw[C], gr[C], wr[C], pwr[C];
    auto load_block = [&](long long t) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            n[c] = t < a.T ? a.d - at[c] : 0;
            if (!BARE) orw[c] = rio::load<WIDE, FULL>(rio::at(a.o, a.odt, t * a.os), a.odt, at[c], n[c], a.d & 7);
        }
    };
    auto load_rest = [&](long long t, bool first) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (a.r) rr[c] = rio::load<WIDE, FULL>(rio::at(a.r, a.rdt, t * a.rs), a.rdt, at[c], n[c], a.d & 7);
            if (!BARE && a.g && (first || a.gs)) gr[c] = rio::load<WIDE, FULL>(rio::at(a.g, a.odt, t * a.gs), a.odt, at[c], n[c], a.d & 7);
        }
    };
    long long base = blockIdx.x;
#pragma unroll
    for (int c = 0; c < C; ++c) at[c] = 8 * (team.lane() + c * team.lanes());
    load_block(base * G + team.row());
    load_rest(base * G + team.row(), true);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (!BARE && a.pw) pwr[c] = rio::load<WIDE, FULL>(a.pw, a.wdt, at[c], a.d - at[c], a.d & 7);
        if (a.w) wr[c] = rio::load<WIDE, FULL>(a.w, a.wdt, at[c], a.d - at[c], a.d & 7);
    }
    for (; base * G < a.T; base += gridDim.x) {
        const long long t = base * G + team.row();
        const bool live = t < a.T;
        loads_done();
        int m[C];                                   // n of this row (n is the next one's from its loads on)
        float v[C][8];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            m[c] = n[c];
            if constexpr (C > 1 || (WIDE && !FULL)) {
                rio::stay_packed<WIDE>(wr[c]);
                if (!BARE) rio::stay_packed<WIDE>(pwr[c]);
                if (!BARE) rio::stay_packed<WIDE>(gr[c]);
            }
        }
        if (!BARE) {
#pragma unroll
            for (int c = 0; c < C; ++c) rio::floats<WIDE>(orw[c], a.odt, v[c]);
        }
        // The next row of these lanes is on its way while this one is finished, its block from before
        // the block's norm where that hides more than the registers cost: 4096 x 6144 between norms to
        // codes 43.2 us against 44.9, but in one group of 16-bit numbers 131072 x 128 26.7 against 25.7.
        constexpr bool kEarly = C > 1 || WIDE;
        const long long next = t + (long long)gridDim.x * G;
        const bool more = (base + gridDim.x) * G < a.T;
        if (kEarly && more) load_block(next);
        if (!BARE) {
            if (a.post) norm_row<LAYER, L, C, WIDE, FULL>(v, m, team, a, a.pw, pwr, a.pb);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!BARE && a.g) {
                float g[8];
                rio::floats<WIDE>(gr[c], a.odt, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[c][j] *= g[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] = BARE ? 0.f : a.bscale * v[c][j];
            if (a.r) {
                float r[8];
                rio::floats<WIDE>(rr[c], a.rdt, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[c][j] += a.rscale * r[j];
            }
        }
        if (!kEarly && more) load_block(next);
        if (more) load_rest(next, false);
        if (a.y) {
#pragma unroll
            for (int c = 0; c < C; ++c) rio::store<FULL>(rio::at(a.y, a.rdt, t * a.ys), a.rdt, at[c], m[c], a.d & 7, v[c]);
        }
        if (!a.out) continue;
        norm_row<LAYER, L, C, WIDE, FULL>(v, m, team, a, a.w, wr, a.b);
        if (a.ndt != 3) {
#pragma unroll
            for (int c = 0; c < C; ++c) rio::store<FULL>(rio::at(a.out, a.ndt, t * a.ns), a.ndt, at[c], m[c], a.d & 7, v[c]);
            continue;
        }
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t of = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) of = rio::umax(of, codes::magnitude(v[c][j]));
            most = rio::umax(most, m[c] > 0 ? of : 0);
        }
        const codes::Row r = codes::row(team.max(most));
        const double f = codes::factor64(r);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = codes::code64(v[c][j], f);
            rio::store_codes<FULL>((int8_t *)a.out + t * a.ns, at[c], m[c], a.d & 7, q, r.ok);
        }
        if (team.lane() == 0 && live) a.out_scale[t] = r.scale;
    }
}

template <bool LAYER, int L, int C, bool WIDE, bool FULL, bool BARE>
hipError_t launch_as(const NormArgs &a, const rio::Shape &h, hipStream_t s)
{
    static const int waves = rio::held_waves((const void *)norm_kernel<LAYER, L, C, WIDE, FULL, BARE>);
    hipLaunchKernelGGL((norm_kernel<LAYER, L, C, WIDE, FULL, BARE>), dim3(rio::grid(h, a.T, waves)), dim3(h.threads), 0, s, a);
    return hipGetLastError();
}

template <bool LAYER, bool WIDE, bool FULL, bool BARE>
hipError_t launch(const NormArgs &a, hipStream_t s)
{
    // two groups a lane: 2048 x 8192 between norms to 8 bits 28.7 us against 30.8 in one, 4096 x 3001 28.3
    // against 40.3, but layer norms of 4096 x 5000 40.7 against 35.5; 4096 x 4096 alike.  With 32-bit
    // operands two groups need more than the 128 registers that 16 waves leave (8 to 50 go to scratch) and
    // are taken where one does not hold the row, above 8192: 2048 x 16384 on an fp32 stream 79 us, 5.1 TB/s,
    // layer norms of bf16 rows with fp32 weights 88 us, 3.0 TB/s, of 2048 x 16383 142 us.
    const rio::Shape h = rio::shape(a.d, WIDE || a.T <= 512 ? rio::kGroups : FULL ? 512 : 256);
    switch (h.lanes) {
    case 8: return launch_as<LAYER, 8, 1, WIDE, FULL, BARE>(a, h, s);
    case 16: return launch_as<LAYER, 16, 1, WIDE, FULL, BARE>(a, h, s);
    case 32: return launch_as<LAYER, 32, 1, WIDE, FULL, BARE>(a, h, s);
    case 64: return launch_as<LAYER, 64, 1, WIDE, FULL, BARE>(a, h, s);
    }
    return h.groups == 1 ? launch_as<LAYER, 0, 1, WIDE, FULL, BARE>(a, h, s) : launch_as<LAYER, 0, 2, WIDE, FULL, BARE>(a, h, s);
}

template <bool WIDE, bool FULL>
hipError_t launch_of(const NormArgs &a, hipStream_t s)
{
    if (a.layer) return a.o ? launch<true, WIDE, FULL, false>(a, s) : launch<true, WIDE, FULL, true>(a, s);
    return a.o ? launch<false, WIDE, FULL, false>(a, s) : launch<false, WIDE, FULL, true>(a, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs &given, hipStream_t s)
{
    NormArgs a = given;
    a.len = (float)a.d;
    a.inv = 1.f / a.len;
    if (a.d < 1 || a.d > rio::kHeld) return hipErrorInvalidValue;
    const bool weights = a.w || a.b || a.pw || a.pb;
    const bool wide = (a.r && a.rdt == 2) || (a.o && a.odt == 2) || (weights && a.wdt == 2);
    if (wide) return a.d % 8 ? launch_of<true, false>(a, s) : launch_of<true, true>(a, s);
    return a.d % 8 ? launch_of<false, false>(a, s) : launch_of<false, true>(a, s);
}

}  // namespace moeffn
