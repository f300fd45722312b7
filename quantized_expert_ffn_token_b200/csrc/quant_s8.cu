// Rows to 8-bit codes with one scale a row: s = max|x| / 127, q = rint(x / s).
//
// Bound by HBM: a row is read once into registers (16-byte loads), reduced over the CTA, scaled and written.  Rows whose
// address does not allow 16-byte accesses are read twice, the second time from L1/L2.  With 16 loads a thread a part of
// the row goes through local memory instead (a 1024-thread CTA's 64 registers a thread spill 340 bytes, 512 threads' 128
// spill 60): rows of more than 4096 loads while there are at most 148 of them, and those too long for 8 loads of 384 threads otherwise.
// The codes are those of correctly rounded divisions, so that they are the same wherever they are computed: the product
// with a reciprocal decides where it lies 1e-4 or more from a half (its error is below 127 * 2^-21), a division the rest.
#include "dense.cuh"
#include "moe_internal.cuh"

namespace qeffn {

namespace {

template <class T>
struct Vec { static constexpr int N = 16 / (int)sizeof(T); };   // elements of a 16-byte load

__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Elements of one 16-byte load, widened.
template <class T>
__device__ __forceinline__ void widen(const uint4 &w, float (&f)[Vec<T>::N]) {
    const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) f[i] = to_f32(e[i]);
}

struct RowScale {
    float s, inv, limit;   // a code is decided by the reciprocal up to this distance from a whole number
    bool live;
};
// Scale of a row whose largest magnitude has the bits `top`.
__device__ __forceinline__ RowScale row_scale(unsigned top) {
    const bool finite = top < 0x7F800000u;
    const float s = finite ? __fdiv_rn(__uint_as_float(top), 127.f) : __uint_as_float(0x7FC00000u);
    // a subnormal scale's reciprocal overflows or lacks bits: every code by division
    return s > 1e-37f ? RowScale{s, __fdiv_rn(1.f, s), 0.4999f, finite} : RowScale{s, 0.f, -1.f, finite && s > 0.f};
}

// A code by division.  A subnormal scale is rounded to whole units of 2^-149, by up to a third of itself: quotients reach
// 190 there (a maximum of 190 units has the scale 1), and their codes are held at 127.
__device__ __forceinline__ int code_exact(float v, float s) { return max(-127, min(127, __float2int_rn(__fdiv_rn(v, s)))); }
// Four of them, for values next to a half (kept out of line: inlined, its copies did not fit the instruction cache and the
// kernel took five times as long).
__device__ __noinline__ uint32_t codes_exact(float a, float b, float c, float d, float s) {
    return (uint32_t)(code_exact(a, s) & 255) | (uint32_t)(code_exact(b, s) & 255) << 8 |
           (uint32_t)(code_exact(c, s) & 255) << 16 | (uint32_t)(code_exact(d, s) & 255) << 24;
}
// Four codes.  Adding 1.5 * 2^23 rounds the product with the reciprocal to a whole number (half to even) in the sum's
// low bits.
__device__ __forceinline__ uint32_t codes(const float *f, const RowScale &r) {
    constexpr float kMagic = 12582912.f;
    float m[4], far = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m[k] = fmaf(f[k], r.inv, kMagic);
        far = fmaxf(far, fabsf(fmaf(f[k], r.inv, kMagic - m[k])));
    }
    uint32_t b = __byte_perm(__byte_perm(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0040),
                             __byte_perm(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0040), 0x5410);
    if (far > r.limit) b = codes_exact(f[0], f[1], f[2], f[3], r.s);
    return b;
}

// The codes of one 16-byte load.
template <class T>
__device__ __forceinline__ void put_codes(int8_t *q, int i, const uint4 &w, const RowScale &r) {
    float f[Vec<T>::N];
    widen<T>(w, f);
    if constexpr (Vec<T>::N == 8) reinterpret_cast<uint2 *>(q)[i] = r.live ? make_uint2(codes(f, r), codes(f + 4, r)) : make_uint2(0, 0);
    else reinterpret_cast<uint32_t *>(q)[i] = r.live ? codes(f, r) : 0;
}
template <class T>
__device__ __forceinline__ unsigned top_of(const uint4 &w, unsigned top) {
    float f[Vec<T>::N];
    widen<T>(w, f);
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e) top = max(top, mag(f[e]));
    return top;
}

// LANES threads a row (a warp, or the whole CTA of NT).  NV: 16-byte loads a thread holds (0: element by element, read
// twice).
template <class T, int NT, int LANES, int NV>
__global__ void __launch_bounds__(NT) k_quantize_s8(const T *x, long long ld, int rows, int cols, int8_t *q, float *scale) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const long long row = (long long)blockIdx.x * (NT / LANES) + threadIdx.x / LANES;
    const int at = threadIdx.x % LANES;
    if (LANES == 32 && row >= rows) return;
    const T *xr = x + row * ld;
    int8_t *qr = q + row * cols;
    const int nvec = cols / Vec<T>::N;   // NV > 0: cols is a multiple
    unsigned top = 0;                    // |x| as bits: they order like integers, infinities and NaNs above every finite value
    uint4 held[NV ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = at + j * LANES;
            held[j] = i < nvec ? reinterpret_cast<const uint4 *>(xr)[i] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) top = top_of<T>(held[j], top);
    } else {
        for (int i = at; i < cols; i += LANES) top = max(top, mag(to_f32(xr[i])));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (LANES > 32) {
        __shared__ unsigned part[NT / 32];
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) top = max(top, part[w]);
    }
    const RowScale r = row_scale(top);
    if (at == 0) scale[row] = r.s;
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * LANES < nvec) put_codes<T>(qr, at + j * LANES, held[j], r);
    } else {
        for (int i = at; i < cols; i += LANES) qr[i] = r.live ? (int8_t)code_exact(to_f32(xr[i]), r.s) : (int8_t)0;
    }
}

template <class T, int NT, int LANES, int NV>
int launch_as(const T *x, long long ld, int rows, int cols, int8_t *q, float *scale, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((rows + NT / LANES - 1) / (NT / LANES));
    cfg.blockDim = dim3(NT);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    QE_CHECK(cudaLaunchKernelEx(&cfg, k_quantize_s8<T, NT, LANES, NV>, x, ld, rows, cols, q, scale));
    QE_CHECK_LAUNCH("k_quantize_s8");
    return MOE_OK;
}

template <class T>
int launch_type(const T *x, long long ld, int rows, int cols, int8_t *q, float *scale, cudaStream_t st) {
    constexpr int V = Vec<T>::N;
    const bool vec = cols % V == 0 && ld % V == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(q) % 8 == 0;
    const int n = cols / V;   // loads a row
    if (!vec || n > 16 * 1024) return launch_as<T, 1024, 1024, 0>(x, ld, rows, cols, q, scale, st);
    // few rows: a wide CTA on each, for latency; many: a warp or a small CTA with four to eight loads a thread, measured on
    // 4096 rows: 4096 bf16 128 x 4 5940 GB/s (256 x 2 5290, 512 x 1 4060, 32 x 16 3680), 12288 fp32 384 x 8 6550 (512 x 8
    // 6070, 1024 x 4 3700), 512 fp32 32 x 4 2890 (128 x 1 2030)
    if (rows <= 148 || n > 16 * 512) {
        if (n <= 1024) return launch_as<T, 1024, 1024, 1>(x, ld, rows, cols, q, scale, st);
        if (n <= 4 * 1024) return launch_as<T, 1024, 1024, 4>(x, ld, rows, cols, q, scale, st);
        return launch_as<T, 1024, 1024, 16>(x, ld, rows, cols, q, scale, st);
    }
    if (n <= 4 * 32) return launch_as<T, 256, 32, 4>(x, ld, rows, cols, q, scale, st);
    if (n <= 4 * 128) return launch_as<T, 128, 128, 4>(x, ld, rows, cols, q, scale, st);
    if (n <= 8 * 128) return launch_as<T, 128, 128, 8>(x, ld, rows, cols, q, scale, st);
    if (n <= 8 * 384) return launch_as<T, 384, 384, 8>(x, ld, rows, cols, q, scale, st);
    return launch_as<T, 512, 512, 16>(x, ld, rows, cols, q, scale, st);
}

}  // namespace

int launch_quantize_s8(const void *x, int dtype, long long ld, int rows, int cols, int8_t *q, float *scale,
                       cudaStream_t st) {
    if (dtype == MOE_BF16) return launch_type((const __nv_bfloat16 *)x, ld, rows, cols, q, scale, st);
    if (dtype == MOE_FP16) return launch_type((const __half *)x, ld, rows, cols, q, scale, st);
    return launch_type((const float *)x, ld, rows, cols, q, scale, st);
}

}  // namespace qeffn
