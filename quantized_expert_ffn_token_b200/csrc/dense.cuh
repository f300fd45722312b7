// Internal declarations of the dense feed-forward operators (dense_api.cu,
// dense_gemm.cu, quant_s8.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace qeffn {

int set_error(int status, const char *what);   // message for moe_last_error(), returns status (moe_api.cu)

constexpr int DT_S8 = 4;   // operand type beside moe_dtype's: 8-bit integers

// What happens to a finished tile of the product.
enum GemmEpi {
    EPI_STORE = 0,      // out = C (with scales and bias for 8-bit operands)
    EPI_GATE = 1,       // C0 = A b[0]^T, C1 = A b[1]^T: out = act(C0) * C1; out1, out2 = C0, C1 if wanted
    EPI_GATE_BWD = 2    // C = dh: out = dg, out1 = du, out2 = h from in1 = g, in2 = u
};

// C [M][N] = sum over segments s of A_s [M][K] . B_s [N][K]^T.  An operand is
// stored with its reduction index contiguous ([M][K], [N][K]) or, where a_mn /
// b_mn is set, with its row index contiguous ([K][M], [K][N]).
struct GemmArgs {
    int type = MOE_BF16;          // operand type: MOE_BF16, MOE_FP16 or DT_S8
    int M = 0, N = 0, K = 0;      // K of one segment
    int segs = 1;                 // 1 or 2
    const void *a[2] = {nullptr, nullptr};
    const void *b[2] = {nullptr, nullptr};   // EPI_GATE: gate and up (one segment)
    long long lda = 0, ldb = 0;   // elements
    bool a_mn = false, b_mn = false;
    int epi = EPI_STORE;
    int act = 0;
    void *out = nullptr, *out1 = nullptr, *out2 = nullptr;
    int out_dtype = MOE_BF16;     // of out; out1 and out2 have the operand type
    long long ldo = 0;            // of out; out1, out2, in1, in2 are contiguous rows of N
    const void *in1 = nullptr, *in2 = nullptr;
    const float *row_scale = nullptr;                    // 8-bit operands: [M]
    const float *col_scale[2] = {nullptr, nullptr};      // [N], EPI_GATE: of gate and up
    const float *bias = nullptr;                         // [N] or NULL
    bool add = false;             // EPI_STORE with fp32 out: out += C
    bool b_ready = false;         // a later kernel of its call, and B is an input of the call
};

// Kernels of one call and of calls after each other overlap.  Every kernel here is launched programmatically: it starts
// while the kernel before it drains, waits for that one's results before it touches them, and only then lets the next
// kernel start; so when a later kernel of a call runs, everything before the call is complete.  A call's first kernel
// reads nothing before its wait, because the kernel before it may be the one that writes its inputs; a later one may load
// operands that are inputs of the call (GemmArgs::b_ready).
int launch_gemm(const GemmArgs &g, cudaStream_t st);
int launch_rows(const GemmArgs &g, cudaStream_t st);
constexpr int kGroup = 4;
// The gradients' products (dx may be NULL, n_dw at most 3), in one launch or two.
int launch_gradients(const GemmArgs *dx, const GemmArgs *dw, int n_dw, cudaStream_t st);
bool rows_fit(const GemmArgs &g);   // the product streams its weights (dense_rows.cu) rather than tiling them
int read_dense_error(int *code);   // reads and clears the error word of the current device
int launch_quantize_s8(const void *x, int dtype, long long ld, int rows, int cols, int8_t *q, float *scale,
                       cudaStream_t st);

// act(z) and act'(z).  With P(z) the gate's weight (a sigmoid, or the normal
// distribution function), act = z P and act' = P + z P'.  The fast exponential
// and division are off by a few fp32 ulp (the exponential by |x| ulp at large
// arguments), far inside the 16-bit or 8-bit rounding that follows.  The
// division gives 0 once its divisor is above 2^126: silu(z) is 0 below
// z = -87.3, where it is smaller than 1e-36.
__device__ __forceinline__ float fast_sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

constexpr float kGeluC = 1.5957691216057308f;   // 2 sqrt(2/pi): (1 + tanh v)/2 is the sigmoid of 2 v

__device__ __forceinline__ float act_fwd(int act, float z) {
    if (act == MOE_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
    if (act == MOE_ACT_GELU_TANH) return z * fast_sigmoid(kGeluC * z * (1.f + 0.044715f * z * z));
    return z * (0.5f * erfcf(-0.70710678118654752f * z));
}

// a = act(z), d = act'(z).
__device__ __forceinline__ void act_bwd(int act, float z, float &a, float &d) {
    if (act == MOE_ACT_SILU) {
        const float s = fast_sigmoid(z);
        a = z * s;
        d = s * (1.f + z * (1.f - s));
    } else if (act == MOE_ACT_GELU_TANH) {
        const float s = fast_sigmoid(kGeluC * z * (1.f + 0.044715f * z * z));
        // s (1 - s) is zero in fp32 beyond |z| = 16, where z^3 may overflow
        const float c = fabsf(z) > 16.f ? 0.f : z * kGeluC * (1.f + 0.134145f * z * z);
        a = z * s;
        d = s + s * (1.f - s) * c;
    } else {
        const float s = 0.5f * erfcf(-0.70710678118654752f * z);
        // e^(-z^2/2) is zero in fp32 beyond |z| = 16, where z^2 may overflow
        const float p = fabsf(z) > 16.f ? 0.f : z * 0.3989422804014327f * __expf(-0.5f * z * z);
        a = z * s;
        d = s + p;
    }
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

}  // namespace qeffn
