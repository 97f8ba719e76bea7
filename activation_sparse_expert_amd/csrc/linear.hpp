// Host-side declarations of the linear layer and the few-token MoE layer.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moeffn {

// y = r + act(x W^T + b), or gated: y = r + act(x Wg^T + bg) (.) (x W^T + b)
struct LinearArgs {
    int T, K, N;
    int bf16;                           // 16-bit type of x and the weights: 1 bf16, 0 fp16
    int act;                            // moe_act
    int ydt;                            // type of y and the residual (0 f16, 1 bf16, 2 f32)
    const uint16_t *x;                  // [T] rows at stride xs (elements)
    long long xs;
    const uint16_t *w, *wg;             // [N][K]; wg null: not gated
    const float *b, *bg;                // [N] or null
    const void *r;                      // [T] rows at stride rs, or null
    long long rs;
    void *y;                            // [T] rows at stride ys
    long long ys;
    float *part;                        // split of K: partial products (workspace)
};

// Rows up to which a call streams the weights past all tokens at once.
constexpr int kStreamTokens = 32;

hipError_t launch_linear_stream(const LinearArgs &a, hipStream_t s);    // T <= kStreamTokens
hipError_t launch_linear_tile(const LinearArgs &a, hipStream_t s);      // any T
size_t linear_tile_ws_bytes(int T, int K, int N);       // the larger of the plain and the gated call's

// The few-token MoE layer: the call's experts and their tokens, made by every
// gate/up workgroup from the routing, and kept for the down product by one.
// Experts with tokens are listed in ascending order, the shared ones last; a
// token's place in expert a is row off[a] + (set bits of mask[a] below it).
struct FewTab {
    int32_t *n;                         // [1] experts listed
    int32_t *expert;                    // [A]
    uint32_t *mask;                     // [A] bit t: token t goes to the expert
    int32_t *off;                       // [A] first row
    float *wt;                          // [T (k + S)] router weight of each row
};

struct FewArgs {
    int T, d, f, E, k, S;
    int bf16, ydt;
    const uint16_t *x;                  // [T][d]
    const uint16_t *gate, *up;          // [E+S][f][d]
    const uint16_t *down_t;             // [E+S][d][f]
    const int32_t *topk_idx;            // [T][k]
    const float *topk_w;                // [T][k]
    FewTab tab;
    int amax;                           // bound of the listed experts: min(E, T k) + S
    uint16_t *h;                        // [T (k + S)][f / 8][8 hi, 8 lo] (workspace)
    const void *r;                      // [T][d] or null
    void *y;                            // [T][d]
    int32_t *count, *eam_row;           // trace exports or null
    uint8_t *expert_dense;
};

constexpr int kFewTokens = 32;          // bits of a token mask
constexpr int kFewRows = 2048;          // T (k + S)
hipError_t launch_few_gateup(const FewArgs &a, hipStream_t s);
hipError_t launch_few_down(const FewArgs &a, hipStream_t s);

}  // namespace moeffn
