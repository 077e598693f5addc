// dense.h -- launcher interface between the C ABI (dense_abi.hip) and the
// kernels of the experts' layer for a few tokens and of the matrix product
// with its backward pass.  Not installed; callers use include/ep.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ep {

// ---------------------------------------------------------------- a few tokens

constexpr int kFewTokens = 64;   // a lane for every token

struct FewShape {
    int T, H, I, E, k;
    bool f8;   // weights e4m3 with block scales, else bf16
};

// Some tokens (16 at most) that share an expert: what one pass of the second
// kernel over the expert's weights serves.
struct FewSegment {
    uint64_t tokens;     // bit t: token t has a row; rows are in the order of the bits
    int32_t expert;
    int32_t rows;
    uint32_t pair[8];    // 16 bits each, row r in half r % 2 of word r / 2: t k + j of the row, where its h lies
    uint32_t pad[4];
};
static_assert(sizeof(FewSegment) == 64, "one line");

// The second kernel's blocks have 32 columns of y.  Up to 128 of them, where at
// least two for each fit the 256 CUs, each has several blocks with a part of the
// segments, and the last of them adds up the parts (with parts / without, the layer,
// us: 64 tokens, 96 experts, 2048 wide, 176 / 260; 4096 wide, 64 experts 233 / 287; 7
// tokens, 1000 wide, 24 / 32).  From 129 on, two for each come in a second round and
// cost more than the CUs that one leaves idle: 4224 wide, 64 tokens, top-8 of 32
// experts 317 / 304, 5120 wide 350 / 346, 7168 wide 384 / 373; one token 50 / 43, 55 /
// 51, 76 / 71.
constexpr int kFewColumns = 32, kFewJoins = 128;
inline int few_columns(const FewShape &s) { return (s.H + kFewColumns - 1) / kFewColumns; }
inline int few_parts(const FewShape &s) {
    const int cols = few_columns(s), most = s.T * s.k;   // as many as there can be segments
    const int parts = cols <= kFewJoins ? (256 / cols < 16 ? 256 / cols : 16) : 1;
    return parts < most ? parts : most;
}

// Workspace: the number of segments, the counts of blocks that are done, the
// segments, h as two bf16 parts [T k][2][I], the parts of y [parts][T][H].
constexpr size_t kFewHead = 256 + kFewJoins * 4;
inline size_t few_h_offset(const FewShape &s) { return kFewHead + (size_t)s.T * s.k * sizeof(FewSegment); }
inline size_t few_partial_offset(const FewShape &s) { return few_h_offset(s) + (size_t)s.T * s.k * s.I * 4; }
inline size_t few_workspace(const FewShape &s) {
    const int parts = s.T > 0 ? few_parts(s) : 1;
    return few_partial_offset(s) + (parts > 1 ? (size_t)parts * s.T * s.H * 4 : 0);
}

hipError_t launch_few(const FewShape &s, const uint16_t *x, const int64_t *idx, const float *w, const void *up,
                      const float *ups, const void *down, const float *downs, const uint16_t *residual, uint16_t *y,
                      uint8_t *ws, hipStream_t stream);

// ---------------------------------------------------------------- the product

enum Activation { kActNone = 0, kActRelu, kActSilu, kActGelu, kActGeluTanh };

struct LinearShape {
    int64_t M;
    int K, N;     // N: width of y; gated: w has 2 N rows
    int act;
    bool gated;
    bool f32;     // y (and its gradient) fp32, else bf16
    bool w32;     // the weights' gradient fp32, else bf16
    __host__ __device__ int wide() const { return gated ? 2 * N : N; }
    // the gradient over z is dy itself
    bool plain() const { return act == kActNone && !gated && !f32; }
};

// Workspace of the backward pass: dz in bf16 (in two parts from an fp32 dy, in
// three for an fp32 gradient of the weights) unless it is dy itself, the bias' sums
// of runs of rows.
// Rows of a run, by 512 columns for a block: 64, or fewer (4 at least) where the
// blocks would not fill the chip (100 rows of 512: 64 rows 15 us, 4 rows 5).
inline int dz_rows(const LinearShape &s) {
    int r = 64;
    while (r > 4 && (s.M + r - 1) / r * ((s.N + 511) / 512) < 1024) r /= 2;
    return r;
}
inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
inline int dz_parts(const LinearShape &s) { return s.plain() ? 0 : (s.w32 ? 3 : (s.f32 ? 2 : 1)); }
inline size_t linear_sums_offset(const LinearShape &s) {
    return align256((size_t)dz_parts(s) * s.M * s.wide() * 2);
}
inline size_t linear_workspace(const LinearShape &s) {
    return linear_sums_offset(s) + (size_t)((s.M + dz_rows(s) - 1) / dz_rows(s)) * s.wide() * 4;
}

hipError_t launch_linear(const LinearShape &s, const uint16_t *x, const uint16_t *w, const float *bias,
                         const uint16_t *residual, void *y, uint16_t *z, hipStream_t stream);
hipError_t launch_linear_backward(const LinearShape &s, const void *dy, const uint16_t *x, const uint16_t *w,
                                  const uint16_t *z, uint16_t *grad_x, void *grad_w, float *grad_bias, uint8_t *ws,
                                  hipStream_t stream);

}  // namespace ep
