// Host-side declarations of the operators on rows of tokens: 8-bit codes and back, the norms
// between two blocks, and the linear layer on 8-bit codes.
#pragma once
#include "linear.hpp"

namespace moeffn {

// Types of row operands: moe_dtype (0 f16, 1 bf16, 2 f32, 3 8-bit codes)
inline int type_bytes(int dt) { return dt == 2 ? 4 : dt == 3 ? 1 : 2; }

struct QuantizeArgs {
    int T, k;
    const void *x;                      // [T] rows at stride xs (elements), type xdt (0, 1, 2)
    int xdt;
    long long xs;
    int8_t *q;                          // [T] rows at stride qs
    long long qs;
    float *scale;                       // [T]
};
hipError_t launch_quantize_rows(const QuantizeArgs &a, hipStream_t s);

struct DequantizeArgs {
    int T, k;
    const int8_t *q;                    // [T] rows at stride qs
    long long qs;
    const float *scale;                 // [T]
    void *y;                            // [T] rows at stride ys, type ydt (0, 1, 2)
    int ydt;
    long long ys;
};
hipError_t launch_dequantize_rows(const DequantizeArgs &a, hipStream_t s);

// y = rs r + bs g (.) Npost(o), out = Npre(y) (of the unrounded y)
struct NormArgs {
    int T, d;
    int layer;                          // 1: layer norms, 0: RMS norms
    float eps;
    int wdt;                            // type of the weights and biases
    const void *w, *b;                  // [d] or null (1, 0): of the norm before the next block
    int post;                           // whether the block's output is normed
    const void *pw, *pb;                // [d] or null
    float add;                          // added to the weights (0 or 1)
    float rscale, bscale;
    const void *r;                      // [T] rows, type rdt (y's too), or null (0)
    int rdt;
    long long rs;
    const void *o;                      // [T] rows, type odt (the gate's too), or null
    int odt;
    long long os;
    const void *g;                      // [T] rows at stride gs (0: one row for all), or null
    long long gs;
    void *y;                            // [T] rows or null
    long long ys;
    void *out;                          // [T] rows or null, type ndt (3: codes, with out_scale)
    int ndt;
    long long ns;
    float *out_scale;                   // [T]
    float len, inv;                     // d and 1 / d (launch_norm sets them)
};
hipError_t launch_norm(const NormArgs &a, hipStream_t s);

// The linear layer on codes: products of the base's x and w (codes; strides and K in
// elements, that is bytes) times sx[t] sw[j], then as the linear layer.
struct LinearQ8Args : LinearArgs {
    int xdt;                            // type of x: 3 codes, else one token that the kernel makes codes of
    const float *sx;                    // [T] (codes)
    const float *sw, *sg;               // [N] scales of w and wg
};
hipError_t launch_linear_q8(const LinearQ8Args &a, hipStream_t s);
bool linear_q8_own_codes(int T, int K, int xdt);        // whether it makes codes of such tokens
// The parts of K of a call (0: streamed) and its tile
int linear_q8_parts(int T, int K, int N, bool gated, int *bm, int *bn);
size_t linear_q8_split_bytes(int T, int K, int N);      // partial products, enough for the plain and the gated call

}  // namespace moeffn
