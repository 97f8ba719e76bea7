// Rows to 8-bit codes and back (codes.hpp has the arithmetic).  Bound by HBM: a row is read
// once, its largest |x| found while it is held in registers.  4096 x 14336 bf16 to codes 37 us,
// 4.7 TB/s, and back 28 us, 6.3 TB/s, whose codes are still in the Infinity Cache; one row 3 us,
// the launch.
#include "row_io.hpp"
#include "rows.hpp"

#include <algorithm>

namespace moeffn {

namespace {

// XDT: type of x; L, C: lanes of a row and groups of 8 a lane (row_io.hpp)
template <int XDT, int L, int C>
__global__ void __launch_bounds__(L ? 256 : 1024)
quantize_kernel(QuantizeArgs a)
{
    __shared__ __align__(16) rio::Slots slots;
    rio::Team<L> team(&slots);
    constexpr int G = L ? 256 / (L ? L : 1) : 1;
    int n[C], at[C];
    rio::Raw<XDT == 2> raw[C];
    auto load_row = [&](long long t) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            n[c] = t < a.T ? a.k - at[c] : 0;
            raw[c] = rio::load<XDT == 2>(rio::at(a.x, XDT, t * a.xs), XDT, at[c], n[c], a.k & 7);
        }
    };
#pragma unroll
    for (int c = 0; c < C; ++c) at[c] = 8 * (team.lane() + c * team.lanes());
    long long b = blockIdx.x;
    load_row(b * G + team.row());
    for (; b * G < a.T; b += gridDim.x) {
        const long long t = b * G + team.row();
        int m[C];
        float v[C][8];
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            m[c] = n[c];
            rio::floats<XDT == 2>(raw[c], XDT, v[c]);
            most = rio::umax(most, rio::most<XDT == 2>(raw[c], XDT));
        }
        // the next row of these lanes is on its way while this one is finished
        if ((b + gridDim.x) * G < a.T) load_row(t + (long long)gridDim.x * G);
        const codes::Row r = codes::row(team.max(most));
        const double f = XDT == 2 ? codes::factor64(r) : 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = XDT == 2 ? codes::code64(v[c][j], f) : codes::code(v[c][j], r);
            rio::store_codes(a.q + t * a.qs, at[c], m[c], a.k & 7, q, r.ok);
        }
        if (team.lane() == 0 && t < a.T) a.scale[t] = r.scale;
    }
}

// Rows longer than registers hold: read twice
template <int XDT>
__global__ void __launch_bounds__(1024)
quantize_long_kernel(QuantizeArgs a)
{
    __shared__ __align__(16) rio::Slots slots;
    rio::Team<0> team(&slots);
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        const void *x = rio::at(a.x, XDT, t * a.xs);
        int8_t *qr = a.q + t * a.qs;
        uint32_t most = 0;
        for (int i = 8 * threadIdx.x; i < a.k; i += 8 * 1024) {
            most = rio::umax(most, rio::most<XDT == 2>(rio::load<XDT == 2>(x, XDT, i, a.k - i, a.k & 7), XDT));
        }
        const codes::Row r = codes::row(team.max(most));
        const double f = XDT == 2 ? codes::factor64(r) : 0.0;
        for (int i = 8 * threadIdx.x; i < a.k; i += 8 * 1024) {
            float v[8];
            uint32_t q[8];
            rio::floats<XDT == 2>(rio::load<XDT == 2>(x, XDT, i, a.k - i, a.k & 7), XDT, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = XDT == 2 ? codes::code64(v[j], f) : codes::code(v[j], r);
            rio::store_codes(qr, i, a.k - i, a.k & 7, q, r.ok);
        }
        if (threadIdx.x == 0) a.scale[t] = r.scale;
    }
}

// L lanes a row; `parts` workgroups take pieces of 8 L elements of a row each
template <int L>
__global__ void __launch_bounds__(256)
dequantize_kernel(DequantizeArgs a, int parts)
{
    constexpr int G = 256 / L;
    const long long b = blockIdx.x / parts;
    const int first = 8 * (threadIdx.x % L + L * (blockIdx.x % parts));
    for (long long t = b * G + threadIdx.x / L; t < a.T; t += (long long)(gridDim.x / parts) * G) {
        const float s = a.scale[t];
        for (int i = first; i < a.k; i += 8 * L * parts) {
            const int8_t *p = a.q + t * a.qs + i;
            uint2 q = make_uint2(0, 0);
            if (a.k - i >= 8) {
                q = rio::read_any<uint2>(p);
            } else {
                const int tail = a.k & 7;
                uint32_t rest = 0;
                if (tail & 4) q.x = rio::read_any<uint32_t>(p);
                if (tail & 2) rest = rio::read_any<uint16_t>(p + (tail & 4));
                if (tail & 1) rest |= (uint32_t)(uint8_t)p[tail & 6] << (tail & 2 ? 16 : 0);
                if (tail & 4) q.y = rest;
                else q.x = rest;
            }
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)((j < 4 ? q.x : q.y) >> 8 * (j & 3)) * s;
            rio::store(rio::at(a.y, a.ydt, t * a.ys), a.ydt, i, a.k - i, a.k & 7, v);
        }
    }
}

constexpr int kMaxGrid = 1 << 20;       // workgroups

unsigned grid_of(int T, int rows) { return (unsigned)std::min<long long>(((long long)T + rows - 1) / rows, kMaxGrid); }

template <int XDT>
hipError_t quantize(const QuantizeArgs &a, hipStream_t s)
{
    if (a.k > rio::kHeld) {
        hipLaunchKernelGGL(quantize_long_kernel<XDT>, dim3(grid_of(a.T, 1)), dim3(1024), 0, s, a);
        return hipGetLastError();
    }
    // two groups a lane: 14336 x 4096 35 us against 36.5
    const rio::Shape h = rio::shape(a.k, a.T <= 512 ? rio::kGroups : 256);
    const dim3 g(rio::grid(h, a.T, 24)), b(h.threads);
    switch (h.lanes) {
    case 8: hipLaunchKernelGGL((quantize_kernel<XDT, 8, 1>), g, b, 0, s, a); break;
    case 16: hipLaunchKernelGGL((quantize_kernel<XDT, 16, 1>), g, b, 0, s, a); break;
    case 32: hipLaunchKernelGGL((quantize_kernel<XDT, 32, 1>), g, b, 0, s, a); break;
    case 64: hipLaunchKernelGGL((quantize_kernel<XDT, 64, 1>), g, b, 0, s, a); break;
    default:
        if (h.groups == 1) hipLaunchKernelGGL((quantize_kernel<XDT, 0, 1>), g, b, 0, s, a);
        else hipLaunchKernelGGL((quantize_kernel<XDT, 0, 2>), g, b, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const QuantizeArgs &a, hipStream_t s)
{
    return a.xdt == 2 ? quantize<2>(a, s) : a.xdt == 1 ? quantize<1>(a, s) : quantize<0>(a, s);
}

hipError_t launch_dequantize_rows(const DequantizeArgs &a, hipStream_t s)
{
    // few long rows: a piece of a row for each workgroup
    const int parts = a.T < 512 && a.k > 2048 ? (a.k + 2047) / 2048 : 1;
    const int lanes = rio::shape(a.k, rio::kGroups).lanes;
    const dim3 b(256);
    switch (lanes) {
    case 8: hipLaunchKernelGGL(dequantize_kernel<8>, dim3(grid_of(a.T, 32)), b, 0, s, a, 1); break;
    case 16: hipLaunchKernelGGL(dequantize_kernel<16>, dim3(grid_of(a.T, 16)), b, 0, s, a, 1); break;
    case 32: hipLaunchKernelGGL(dequantize_kernel<32>, dim3(grid_of(a.T, 8)), b, 0, s, a, 1); break;
    case 64: hipLaunchKernelGGL(dequantize_kernel<64>, dim3(grid_of(a.T, 4)), b, 0, s, a, 1); break;
    default: hipLaunchKernelGGL(dequantize_kernel<256>, dim3(grid_of(a.T, 1) * parts), b, 0, s, a, parts);
    }
    return hipGetLastError();
}

}  // namespace moeffn
