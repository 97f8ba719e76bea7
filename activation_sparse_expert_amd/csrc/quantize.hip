// Rows to 8-bit codes and back (codes.hpp has the arithmetic).  Bound by HBM: a row is read
// once, its largest |x| found while it is held in registers.
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
    for (long long b = blockIdx.x; b * G < a.T; b += gridDim.x) {
        const long long t = b * G + team.row();
        const void *x = rio::at(a.x, XDT, t * a.xs);
        int8_t *qr = a.q + t * a.qs;
        rio::Raw<XDT == 2> raw[C];
        int n[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (team.lane() + c * team.lanes());
            n[c] = t < a.T ? a.k - i : 0;
            raw[c] = rio::load<XDT == 2>(x, XDT, i, n[c]);
        }
        float v[C][8];
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            rio::floats<XDT == 2>(raw[c], XDT, v[c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) most = rio::umax(most, codes::magnitude(v[c][j]));
        }
        const codes::Row r = codes::row(team.max(most));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            int q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = XDT == 2 ? codes::code64(v[c][j], r) : codes::code(v[c][j], r);
            rio::store_codes(qr, 8 * (team.lane() + c * team.lanes()), n[c], q);
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
            float v[8];
            rio::floats<XDT == 2>(rio::load<XDT == 2>(x, XDT, i, a.k - i), XDT, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) most = rio::umax(most, codes::magnitude(v[j]));
        }
        const codes::Row r = codes::row(team.max(most));
        for (int i = 8 * threadIdx.x; i < a.k; i += 8 * 1024) {
            float v[8];
            int q[8];
            rio::floats<XDT == 2>(rio::load<XDT == 2>(x, XDT, i, a.k - i), XDT, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = XDT == 2 ? codes::code64(v[j], r) : codes::code(v[j], r);
            rio::store_codes(qr, i, a.k - i, q);
        }
        if (threadIdx.x == 0) a.scale[t] = r.scale;
    }
}

template <int L>
__global__ void __launch_bounds__(256)
dequantize_kernel(DequantizeArgs a)
{
    constexpr int G = 256 / L;
    for (long long b = blockIdx.x; b * G < a.T; b += gridDim.x) {
        const long long t = b * G + threadIdx.x / L;
        if (t >= a.T) continue;
        const float s = a.scale[t];
        for (int i = 8 * (threadIdx.x % L); i < a.k; i += 8 * L) {
            const int8_t *p = a.q + (size_t)t * a.qs + i;
            int8_t q[8] = {};
            if (a.k - i >= 8) {
                __builtin_memcpy(q, p, 8);
            } else {
#pragma unroll
                for (int j = 0; j < 7; ++j)
                    if (j < a.k - i) q[j] = p[j];
            }
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (float)q[j] * s;
            rio::store(rio::at(a.y, a.ydt, t * a.ys), a.ydt, i, a.k - i, v);
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
    const rio::Shape h = rio::shape(a.k, a.T > 256);
    const dim3 g(grid_of(a.T, h.lanes ? 256 / h.lanes : 1)), b(h.threads);
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
    const int lanes = rio::shape(a.k, a.T > 256).lanes;
    const dim3 b(256);
    switch (lanes) {
    case 8: hipLaunchKernelGGL(dequantize_kernel<8>, dim3(grid_of(a.T, 32)), b, 0, s, a); break;
    case 16: hipLaunchKernelGGL(dequantize_kernel<16>, dim3(grid_of(a.T, 16)), b, 0, s, a); break;
    case 32: hipLaunchKernelGGL(dequantize_kernel<32>, dim3(grid_of(a.T, 8)), b, 0, s, a); break;
    case 64: hipLaunchKernelGGL(dequantize_kernel<64>, dim3(grid_of(a.T, 4)), b, 0, s, a); break;
    default: hipLaunchKernelGGL(dequantize_kernel<256>, dim3(grid_of(a.T, 1)), b, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace moeffn
