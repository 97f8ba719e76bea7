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

hipError_t launch_linear(const LinearArgs &a, hipStream_t s);
hipError_t launch_linear_stream(const LinearArgs &a, hipStream_t s);    // no workspace
// The parts of K of a call (0: streamed) and its tile
int linear_parts(int T, int K, int N, bool gated, int *bm, int *bn);
size_t linear_ws_bytes(int T, int K, int N);            // enough for the plain and the gated call

// The few-token MoE layer: the experts of a call and their tokens, made from the
// routing once.  Experts with tokens are listed in ascending order, the shared ones
// last; an expert's tokens have consecutive rows.
struct FewTab {
    int32_t *n;                         // [1] experts listed
    int4 *rec;                          // [A + 1] {expert (-1 past the list), token bits, first row, cost before}
    float *wt;                          // [T (k + S)] router weight of each row (shared experts: 1)
    int32_t *done;                      // [ceil(d / 16)] parts of a column block that are written
};

struct FewArgs {
    int T, d, f, E, k, S;
    int bf16, ydt;
    const uint16_t *x;                  // [T][d]
    const uint16_t *gate, *up;          // [E+S][f][d]
    const uint16_t *down_t;             // [E+S][d][f]
    const void *rw;                     // [E][d] router in rdt
    int rdt;
    const float *rbias;                 // [E] or null
    int renorm;
    float *lg;                          // [T][E] logits (workspace)
    FewTab tab;
    int amax;                           // bound of the listed experts: min(E, T k) + S
    int terms;                          // that h is kept in (launch_few sets it)
    uint16_t *h;                        // [T (k + S)][terms][f] (workspace)
    float *part;                        // [few_parts][T][d] (workspace)
    const void *r;                      // [T][d] or null
    void *y;                            // [T][d]
    int32_t *topk_idx;                  // trace exports or null
    float *topk_w, *logits;
    int32_t *count, *eam_row;
    uint8_t *expert_dense;
};

constexpr int kFewTokens = 32;
constexpr int kFewTerms = 3;            // the most
constexpr int kFewRows = 2048;          // T (k + S)
int few_amax(int T, int E, int k, int S);
int few_parts(int T, int d, int f, int E, int k, int S);
hipError_t launch_few(const FewArgs &a, hipStream_t s);

}  // namespace moeffn
