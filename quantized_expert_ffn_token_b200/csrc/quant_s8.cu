// Rows to 8-bit codes with one scale a row: s = max|x| / 127, q = rint(x / s).
//
// Bound by HBM: a row is read once into registers (16-byte loads), reduced over the CTA, scaled and written.  Rows too
// long for the registers, or whose address does not allow 16-byte accesses, are read twice, the second time from L1/L2.
// The codes are those of correctly rounded divisions, so that they are the same wherever they are computed: the product
// with a reciprocal decides where it lies 1e-4 or more from a half (its error is below 127 * 2^-21), a division the rest.
#include "dense.cuh"
#include "moe_internal.cuh"

namespace qeffn {

namespace {

template <class T>
struct Vec { static constexpr int N = 16 / (int)sizeof(T); };   // elements of a 16-byte load

__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ int code(float v, float s, float inv) {
    const float t = v * inv, r = rintf(t);
    if (fabsf(t - r) < 0.4999f) return (int)r;
    return __float2int_rn(__fdiv_rn(v, s));
}

// Elements of one 16-byte load, widened.
template <class T>
__device__ __forceinline__ void widen(const uint4 &w, float (&f)[Vec<T>::N]) {
    const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) f[i] = to_f32(e[i]);
}

// A CTA per row.  NV: 16-byte loads a thread holds (0: element by element, read twice).
template <class T, int NT, int NV>
__global__ void __launch_bounds__(NT) k_quantize_s8(const T *x, long long ld, int cols, int8_t *q, float *scale) {
    constexpr int V = Vec<T>::N;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const long long row = blockIdx.x;
    const T *xr = x + row * ld;
    int8_t *qr = q + row * cols;
    const int nvec = cols / V;   // NV > 0: cols is a multiple of V
    unsigned top = 0;            // |x| as bits: they order like integers, infinities and NaNs above every finite value
    uint4 held[NV ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + j * NT;
            held[j] = i < nvec ? reinterpret_cast<const uint4 *>(xr)[i] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float f[V];
            widen<T>(held[j], f);
#pragma unroll
            for (int e = 0; e < V; ++e) top = max(top, mag(f[e]));
        }
    } else {
        for (int i = threadIdx.x; i < cols; i += NT) top = max(top, mag(to_f32(xr[i])));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    __shared__ unsigned part[NT / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) top = max(top, part[w]);
    const bool finite = top < 0x7F800000u;
    const float s = finite ? __fdiv_rn(__uint_as_float(top), 127.f) : __uint_as_float(0x7FC00000u);
    if (threadIdx.x == 0) scale[row] = s;
    const bool live = finite && s > 0.f;
    // a reciprocal that overflows or loses bits to a subnormal scale leaves every code to the division
    const float inv = s > 1e-37f ? __fdiv_rn(1.f, s) : __uint_as_float(0x7FC00000u);
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + j * NT;
            if (i >= nvec) break;
            float f[V];
            widen<T>(held[j], f);
            uint32_t out[V / 4];
#pragma unroll
            for (int e = 0; e < V / 4; ++e) {
                uint32_t b = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) b |= (uint32_t)(live ? code(f[4 * e + k], s, inv) & 255 : 0) << (8 * k);
                out[e] = b;
            }
            if constexpr (V == 8) reinterpret_cast<uint2 *>(qr)[i] = make_uint2(out[0], out[1]);
            else reinterpret_cast<uint32_t *>(qr)[i] = out[0];
        }
    } else {
        for (int i = threadIdx.x; i < cols; i += NT) qr[i] = live ? (int8_t)code(to_f32(xr[i]), s, inv) : (int8_t)0;
    }
}

template <class T, int NT, int NV>
int launch_as(const T *x, long long ld, int rows, int cols, int8_t *q, float *scale, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3(rows);
    cfg.blockDim = dim3(NT);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    QE_CHECK(cudaLaunchKernelEx(&cfg, k_quantize_s8<T, NT, NV>, x, ld, cols, q, scale));
    QE_CHECK_LAUNCH("k_quantize_s8");
    return MOE_OK;
}

template <class T>
int launch_type(const T *x, long long ld, int rows, int cols, int8_t *q, float *scale, cudaStream_t st) {
    constexpr int V = Vec<T>::N;
    const bool vec = cols % V == 0 && ld % V == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(q) % 8 == 0;
    const int n = cols / V;
    if (!vec || n > 16 * 1024) return launch_as<T, 1024, 0>(x, ld, rows, cols, q, scale, st);
    // few rows: the widest CTA there is, for latency; many: four loads a thread, eight CTAs an SM
    if (rows <= 148 || n > 16 * 256) {
        if (n <= 1024) return launch_as<T, 1024, 1>(x, ld, rows, cols, q, scale, st);
        if (n <= 4 * 1024) return launch_as<T, 1024, 4>(x, ld, rows, cols, q, scale, st);
        return launch_as<T, 1024, 16>(x, ld, rows, cols, q, scale, st);
    }
    if (n <= 2 * 256) return launch_as<T, 256, 2>(x, ld, rows, cols, q, scale, st);
    if (n <= 4 * 256) return launch_as<T, 256, 4>(x, ld, rows, cols, q, scale, st);
    return launch_as<T, 256, 16>(x, ld, rows, cols, q, scale, st);
}

}  // namespace

int launch_quantize_s8(const void *x, int dtype, long long ld, int rows, int cols, int8_t *q, float *scale,
                       cudaStream_t st) {
    if (dtype == MOE_BF16) return launch_type((const __nv_bfloat16 *)x, ld, rows, cols, q, scale, st);
    if (dtype == MOE_FP16) return launch_type((const __half *)x, ld, rows, cols, q, scale, st);
    return launch_type((const float *)x, ld, rows, cols, q, scale, st);
}

}  // namespace qeffn
