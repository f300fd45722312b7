// Matrix products of the dense feed-forward operators.
#include "dense.cuh"
#include "moe_internal.cuh"

namespace qeffn {

namespace {

constexpr int SG_T = 64, SG_K = 16;   // tile and k step

template <class T>
struct AccOf { using type = float; };
template <>
struct AccOf<int8_t> { using type = int; };

__device__ __forceinline__ float mac(float c, __nv_bfloat16 a, __nv_bfloat16 b) { return fmaf(to_f32(a), to_f32(b), c); }
__device__ __forceinline__ float mac(float c, __half a, __half b) { return fmaf(to_f32(a), to_f32(b), c); }
__device__ __forceinline__ int mac(int c, int8_t a, int8_t b) { return c + (int)a * (int)b; }

__device__ __forceinline__ void put(void *p, int dtype, long long i, float v) {
    if (dtype == MOE_BF16) ((__nv_bfloat16 *)p)[i] = from_f32<__nv_bfloat16>(v);
    else if (dtype == MOE_FP16) ((__half *)p)[i] = from_f32<__half>(v);
    else ((float *)p)[i] = v;
}

// One 64 x 64 tile of C a CTA, 16 x 16 threads with 4 x 4 outputs each, operands through shared memory.
template <class T, int EPI>
__global__ void __launch_bounds__(256) k_gemm_simple(const GemmArgs g) {
    using Acc = typename AccOf<T>::type;
    constexpr int NB = EPI == EPI_GATE ? 2 : 1;
    __shared__ T sa[SG_K][SG_T + 2], sb[NB][SG_K][SG_T + 2];
    const int m0 = blockIdx.y * SG_T, n0 = blockIdx.x * SG_T, tid = threadIdx.x;
    const int tx = tid & 15, ty = tid >> 4;
    Acc acc[NB][4][4] = {};
    for (int s = 0; s < g.segs; ++s)
        for (int k0 = 0; k0 < g.K; k0 += SG_K) {
            for (int i = tid; i < SG_K * SG_T; i += 256) {
                int r = g.a_mn ? i % SG_T : i / SG_K, k = g.a_mn ? i / SG_T : i % SG_K;
                const T *a = (const T *)g.a[s];
                const bool in = m0 + r < g.M && k0 + k < g.K;
                sa[k][r] = in ? a[g.a_mn ? (k0 + k) * g.lda + m0 + r : (m0 + r) * g.lda + k0 + k] : T(0);
                r = g.b_mn ? i % SG_T : i / SG_K, k = g.b_mn ? i / SG_T : i % SG_K;
                const bool inb = n0 + r < g.N && k0 + k < g.K;
                for (int j = 0; j < NB; ++j) {
                    const T *b = (const T *)g.b[NB == 2 ? j : s];
                    sb[j][k][r] = inb ? b[g.b_mn ? (k0 + k) * g.ldb + n0 + r : (n0 + r) * g.ldb + k0 + k] : T(0);
                }
            }
            __syncthreads();
            for (int k = 0; k < SG_K; ++k)
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            acc[j][r][c] = mac(acc[j][r][c], sa[k][ty * 4 + r], sb[j][k][tx * 4 + c]);
            __syncthreads();
        }
    for (int r = 0; r < 4; ++r)
        for (int c = 0; c < 4; ++c) {
            const long long m = m0 + ty * 4 + r, n = n0 + tx * 4 + c;
            if (m >= g.M || n >= g.N) continue;
            float v = (float)acc[0][r][c], v1 = (float)acc[NB - 1][r][c];
            if (g.type == DT_S8) {
                v *= g.row_scale[m] * g.col_scale[0][n];
                if (EPI == EPI_GATE) v1 *= g.row_scale[m] * g.col_scale[1][n];
                if (g.bias) v += g.bias[n];
            }
            if (EPI == EPI_STORE) {
                if (g.add) v += ((float *)g.out)[m * g.ldo + n];
                put(g.out, g.out_dtype, m * g.ldo + n, v);
            } else if (EPI == EPI_GATE) {
                put(g.out, g.out_dtype, m * g.ldo + n, act_fwd(g.act, v) * v1);
                if (g.out1) {
                    put(g.out1, g.type, m * g.N + n, v);
                    put(g.out2, g.type, m * g.N + n, v1);
                }
            } else {
                float z = 0.f, u = 0.f, a, d;
                if constexpr (sizeof(T) == 2) z = to_f32(((const T *)g.in1)[m * g.N + n]), u = to_f32(((const T *)g.in2)[m * g.N + n]);
                act_bwd(g.act, z, a, d);
                put(g.out, g.out_dtype, m * g.ldo + n, v * u * d);
                put(g.out1, g.type, m * g.N + n, v * a);
                if (g.out2) put(g.out2, g.type, m * g.N + n, a * u);
            }
        }
}

template <class T>
void run_simple(const GemmArgs &g, cudaStream_t st) {
    const dim3 grid((g.N + SG_T - 1) / SG_T, (g.M + SG_T - 1) / SG_T);
    if (g.epi == EPI_GATE) k_gemm_simple<T, EPI_GATE><<<grid, 256, 0, st>>>(g);
    else if (g.epi == EPI_GATE_BWD) k_gemm_simple<T, EPI_GATE_BWD><<<grid, 256, 0, st>>>(g);
    else k_gemm_simple<T, EPI_STORE><<<grid, 256, 0, st>>>(g);
}

}  // namespace

int launch_gemm(const GemmArgs &g, cudaStream_t st) {
    if (g.type == MOE_BF16) run_simple<__nv_bfloat16>(g, st);
    else if (g.type == MOE_FP16) run_simple<__half>(g, st);
    else run_simple<int8_t>(g, st);
    QE_CHECK_LAUNCH("k_gemm_simple");
    return MOE_OK;
}

}  // namespace qeffn
