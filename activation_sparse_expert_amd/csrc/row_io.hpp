// Eight neighbouring elements of a row at a time, of any type and at any address: whole
// groups are loads and stores of 16 bytes (8 for codes), which gfx950 takes at the
// alignment of an element; a row's last elements go by four, two and one.
#pragma once
#include "codes.hpp"
#include "mfma_stream.hpp"

namespace moeffn {
namespace rio {

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The bits of 8 elements; WIDE: of any type, else of a 16-bit type
template <bool WIDE>
struct Raw {
    uint4 a;
};
template <>
struct Raw<true> {
    uint4 a, b;                         // 16-bit types: a alone
};

// Element i of an array of type dt
__device__ __forceinline__ const void *at(const void *p, int dt, long long i) { return (const char *)p + (i << (dt == 2 ? 2 : 1)); }
__device__ __forceinline__ void *at(void *p, int dt, long long i) { return (char *)p + (i << (dt == 2 ? 2 : 1)); }

__device__ __forceinline__ uint4 load16(const void *p)
{
    uint4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

template <class T>
__device__ __forceinline__ T read_any(const void *p)
{
    T v;
    __builtin_memcpy(&v, p, sizeof(T));
    return v;
}
template <class T>
__device__ __forceinline__ void write_any(void *p, T v) { __builtin_memcpy(p, &v, sizeof(T)); }

// Elements i .. i + 7 of a row, or where n < 8 the row's last n, zeros past them; none if n <= 0.
// `tail` is what n is wherever 0 < n < 8, the same for all lanes: those elements go by
// four, two and one.  FULL: there is no such n.
template <bool WIDE, bool FULL = false>
__device__ __forceinline__ Raw<WIDE> load(const void *p, int dt, uint32_t i, int n, int tail)
{
    Raw<WIDE> r{};
    if (n >= 8) {
        if (!WIDE || dt != 2) {
            r.a = load16((const uint16_t *)p + i);
        } else if constexpr (WIDE) {
            r.a = load16((const float *)p + i);
            r.b = load16((const float *)p + i + 4);
        }
    } else if (!FULL && n > 0) {
        if (!WIDE || dt != 2) {
            const uint16_t *q = (const uint16_t *)p + i;
            uint2 four = make_uint2(0, 0);
            uint32_t two = 0, one = 0;
            if (tail & 4) four = read_any<uint2>(q);
            if (tail & 2) two = read_any<uint32_t>(q + (tail & 4));
            if (tail & 1) one = q[tail & 6];
            if (tail & 4) r.a = tail & 2 ? make_uint4(four.x, four.y, two, one) : make_uint4(four.x, four.y, one, 0);
            else r.a = tail & 2 ? make_uint4(two, one, 0, 0) : make_uint4(one, 0, 0, 0);
        } else if constexpr (WIDE) {
            const uint32_t *q = (const uint32_t *)p + i;
            uint4 four = make_uint4(0, 0, 0, 0);
            uint2 two = make_uint2(0, 0);
            uint32_t one = 0;
            if (tail & 4) four = read_any<uint4>(q);
            if (tail & 2) two = read_any<uint2>(q + (tail & 4));
            if (tail & 1) one = q[tail & 6];
            const uint4 rest = tail & 2 ? make_uint4(two.x, two.y, one, 0) : make_uint4(one, 0, 0, 0);
            if (tail & 4) {
                r.a = four;
                r.b = rest;
            } else {
                r.a = rest;
            }
        }
    }
    return r;
}

// Keeps the compiler from unpacking r before a loop, which would hold it in twice the registers.  (Four
// registers at once: by members, some are copied as soon as they are loaded, and the load waited for.)
template <bool WIDE>
__device__ __forceinline__ void stay_packed(Raw<WIDE> &r)
{
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 a = __builtin_bit_cast(u32x4, r.a);
    asm volatile("" : "+v"(a));
    r.a = __builtin_bit_cast(uint4, a);
    if constexpr (WIDE) {
        u32x4 b = __builtin_bit_cast(u32x4, r.b);
        asm volatile("" : "+v"(b));
        r.b = __builtin_bit_cast(uint4, b);
    }
}

template <bool BF16>
__device__ __forceinline__ void halves(const uint4 &a, float (&v)[8])
{
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = lo16_to_float<BF16>(w[j]);
        v[2 * j + 1] = hi16_to_float<BF16>(w[j]);
    }
}

template <bool WIDE>
__device__ __forceinline__ void floats(const Raw<WIDE> &r, int dt, float (&v)[8])
{
    if constexpr (WIDE)
        if (dt == 2) {
            const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
            return;
        }
    if (dt == 1) halves<true>(r.a, v);
    else halves<false>(r.a, v);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pair16(float a, float b)
{
    return st::to16<BF16>(a) | (uint32_t)st::to16<BF16>(b) << 16;
}

// As load
template <bool FULL = false>
__device__ __forceinline__ void store(void *p, int dt, uint32_t i, int n, int tail, const float (&v)[8])
{
    if (dt == 2) {
        float *q = (float *)p + i;
        if (n >= 8) {
            __builtin_memcpy(q, v, 32);
        } else if (!FULL && n > 0) {
            // (named, so that the choice is between registers and not between places of an array)
            const float v0 = v[0], v1 = v[1], v2 = v[2], v4 = v[4], v5 = v[5], v6 = v[6];
            const bool f = tail & 4, t = tail & 2;
            const float a = f ? v4 : v0, b = f ? v5 : v1, c = f ? v6 : v2;
            if (f) write_any(q, make_float4(v0, v1, v2, v[3]));
            if (t) write_any(q + (tail & 4), make_float2(a, b));
            if (tail & 1) q[tail & 6] = t ? c : a;
        }
        return;
    }
    uint4 w;
    if (dt == 1) w = make_uint4(pair16<true>(v[0], v[1]), pair16<true>(v[2], v[3]), pair16<true>(v[4], v[5]), pair16<true>(v[6], v[7]));
    else w = make_uint4(pair16<false>(v[0], v[1]), pair16<false>(v[2], v[3]), pair16<false>(v[4], v[5]), pair16<false>(v[6], v[7]));
    uint16_t *q = (uint16_t *)p + i;
    if (n >= 8) {
        write_any(q, w);
    } else if (!FULL && n > 0) {
        const bool f = tail & 4, t = tail & 2;
        if (f) write_any(q, make_uint2(w.x, w.y));
        if (t) write_any(q + (tail & 4), f ? w.z : w.x);
        if (tail & 1) q[tail & 6] = (uint16_t)(f ? (t ? w.w : w.z) : t ? w.y : w.x);
    }
}

// Codes from the bits that codes::code gives, zeros unless ok
template <bool FULL = false>
__device__ __forceinline__ void store_codes(int8_t *p, uint32_t i, int n, int tail, const uint32_t (&q)[8], bool ok)
{
    uint2 w = make_uint2(codes::pack4(q[0], q[1], q[2], q[3]), codes::pack4(q[4], q[5], q[6], q[7]));
    if (!ok) w = make_uint2(0, 0);
    p += i;
    if (n >= 8) {
        write_any(p, w);
    } else if (!FULL && n > 0) {
        const uint32_t r = tail & 4 ? w.y : w.x;
        if (tail & 4) write_any(p, w.x);
        if (tail & 2) write_any(p + (tail & 4), (uint16_t)r);
        if (tail & 1) p[tail & 6] = (int8_t)(tail & 2 ? r >> 16 : r);
    }
}

// The largest |x| of 8 elements, as codes::magnitude; their bits still in a 16-bit type are
// compared in pairs
template <bool WIDE>
__device__ __forceinline__ uint32_t most(const Raw<WIDE> &r, int dt)
{
    if constexpr (WIDE) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, w[j] & 0x7FFFFFFFu);
        return m;
    } else {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
        u16x2 m = {0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[j] & 0x7FFF7FFFu));
        const uint16_t h = m.x > m.y ? m.x : m.y;
        return codes::magnitude(dt == 1 ? bf16_bits_to_float(h) : half_bits_to_float(h));
    }
}

// ---- the lanes of a row ----------------------------------------------------
// A row is held by L lanes of a wave (8 to 64) or, with L 0, by a whole workgroup of up to 16
// waves.  There, partial results go through two sets of LDS slots in turn, so that one
// barrier does: who writes a set again has passed a barrier after everyone read it.
template <int S>
__device__ __forceinline__ uint32_t bfly_max(uint32_t v)
{
    if constexpr (S == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return umax(r[0], r[1]);
    } else if constexpr (S == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return umax(r[0], r[1]);
    } else {
        return umax(v, __float_as_uint(xor_lane<S>(__uint_as_float(v))));
    }
}
template <int SEG, int S = SEG / 2>
__device__ __forceinline__ uint32_t seg_max(uint32_t v)
{
    if constexpr (S == 0) return v;
    else return seg_max<SEG, S / 2>(bfly_max<S>(v));
}

struct Slots {
    uint32_t v[2][16];
};

template <int L>
struct Team {
    Slots *s;
    int set;

    __device__ __forceinline__ Team(Slots *slots) : s(slots), set(0)
    {
        if constexpr (L == 0) {
            if (threadIdx.x < 32) ((uint32_t *)s)[threadIdx.x] = 0;     // slots of waves that there are not
            __syncthreads();
        }
    }
    // this lane's place in the row's lanes, their number, and the rows of a workgroup
    __device__ __forceinline__ int lane() const { return L ? threadIdx.x & (L - 1) : threadIdx.x; }
    __device__ __forceinline__ int lanes() const { return L ? L : blockDim.x; }
    __device__ __forceinline__ int row() const { return L ? threadIdx.x / (L ? L : 1) : 0; }

    __device__ __forceinline__ const uint4 *exchange(uint32_t v)
    {
        set ^= 1;
        if ((threadIdx.x & 63) == 0) s->v[set][threadIdx.x >> 6] = v;
        __syncthreads();
        return (const uint4 *)s->v[set];
    }
    __device__ __forceinline__ float sum(float v)
    {
        if constexpr (L != 0) return seg_sum<L>(v);
        const uint4 *p = exchange(__float_as_uint(seg_sum<64>(v)));
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 q = p[i];
            t += (__uint_as_float(q.x) + __uint_as_float(q.y)) + (__uint_as_float(q.z) + __uint_as_float(q.w));
        }
        return t;
    }
    __device__ __forceinline__ uint32_t max(uint32_t v)
    {
        if constexpr (L != 0) return seg_max<L>(v);
        const uint4 *p = exchange(seg_max<64>(v));
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 q = p[i];
            t = umax(t, umax(umax(q.x, q.y), umax(q.z, q.w)));
        }
        return t;
    }
};

constexpr int kGroups = 1024;           // groups of 8 that a workgroup's lanes hold one each of
constexpr int kHeld = 2 * 8 * kGroups;  // elements of a row that its registers hold

// The lanes, threads of a workgroup and groups of 8 a lane for rows of k elements.  A workgroup
// waits for its loads, then for its sums: a lane for each group has the least latency;
// with two groups a lane (rows of more than `two` groups) a compute unit holds more rows.
struct Shape {
    int lanes, threads, groups;
};
inline Shape shape(int k, int two)
{
    const int n8 = (k + 7) / 8;
    int l = 8;
    while (l < n8) l *= 2;
    if (l <= 64) return {l, 256, 1};
    const int groups = n8 > two ? 2 : 1;
    return {0, 64 * ((n8 + 64 * groups - 1) / (64 * groups)), groups};
}

// Waves of a kernel that a compute unit holds
inline int held_waves(const void *kernel)
{
    int n = 0;
    return hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, 64, 0) == hipSuccess && n > 0 ? n : 16;
}

// Workgroups for T rows: where one has a row, no more than the chip's 256 compute units hold at a time,
// `waves` each, which then take rows one after another, the next one's loads under way.  (With
// twice as many, of which half wait, 8192 x 1411 between blocks took 32 us instead of 28.)
// Rows of part of a wave: 16 workgroups a unit, which holds 5 to 8 of them (300000 x 64 29 us so, 30.4
// with those; 100000 x 100 26.4, 22.7 with those).
inline unsigned grid(const Shape &h, int T, int waves)
{
    const long long wgs = h.lanes ? ((long long)T + 256 / h.lanes - 1) / (256 / h.lanes) : T;
    const int unit = h.lanes ? 16 : waves / (h.threads / 64);
    const long long held = 256ll * (unit > 1 ? unit : 1);
    return (unsigned)(wgs < held ? wgs : held);
}

}  // namespace rio
}  // namespace moeffn
