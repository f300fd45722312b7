// Rows to 8-bit codes with one scale a row.
#include "dense.cuh"
#include "moe_internal.cuh"

namespace qeffn {

namespace {

constexpr int Q_NT = 256;

// A CTA per row, two passes: the largest magnitude, then the codes.  The scale and the quotients use
// correctly rounded divisions, so that the codes are the same wherever they are computed.
template <class T>
__global__ void __launch_bounds__(Q_NT) k_quantize_s8(const T *x, long long ld, int cols, int8_t *q, float *scale) {
    const long long r = blockIdx.x;
    const T *xr = x + r * ld;
    int8_t *qr = q + r * cols;
    // |x| as bits: positive fp32 order like integers, infinities and NaNs above every finite value
    unsigned top = 0;
    for (int i = threadIdx.x; i < cols; i += Q_NT) top = max(top, __float_as_uint(to_f32(xr[i])) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xffffffffu, top);
    __shared__ unsigned part[Q_NT / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int w = 0; w < Q_NT / 32; ++w) top = max(top, part[w]);
    const bool finite = top < 0x7F800000u;
    const float s = finite ? __fdiv_rn(__uint_as_float(top), 127.f) : __uint_as_float(0x7FC00000u);
    const bool live = finite && s > 0.f;
    for (int i = threadIdx.x; i < cols; i += Q_NT)
        qr[i] = live ? (int8_t)__float2int_rn(__fdiv_rn(to_f32(xr[i]), s)) : (int8_t)0;
    if (threadIdx.x == 0) scale[r] = s;
}

}  // namespace

int launch_quantize_s8(const void *x, int dtype, long long ld, int rows, int cols, int8_t *q, float *scale,
                       cudaStream_t st) {
    if (dtype == MOE_BF16) k_quantize_s8<<<rows, Q_NT, 0, st>>>((const __nv_bfloat16 *)x, ld, cols, q, scale);
    else if (dtype == MOE_FP16) k_quantize_s8<<<rows, Q_NT, 0, st>>>((const __half *)x, ld, cols, q, scale);
    else k_quantize_s8<<<rows, Q_NT, 0, st>>>((const float *)x, ld, cols, q, scale);
    QE_CHECK_LAUNCH("k_quantize_s8");
    return MOE_OK;
}

}  // namespace qeffn
