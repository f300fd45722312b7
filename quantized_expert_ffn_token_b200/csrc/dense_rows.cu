// Products of few rows (a decode step's tokens): C [T][N] = x [T][K] . W [N][K]^T, T at most 32.
//
// Bound by reading W once from HBM.  A CTA owns 8 G rows of W (gated products: as many gate rows and the up rows of the
// same index) and its KW warps split the reduction index in 128-byte blocks, dealt round robin; several CTAs share an SM, so
// that one's start and end hide behind the others' streams.  Weights go from global memory straight into mma.sync
// operands: lane (g, c) of a warp loads 16 consecutive bytes of row g, block part c, and uses them as the B fragments of
// two MMAs; that permutes the reduction index within the block, which is harmless because the token operand (A
// fragments, read the same way, from L1 after the SM's first CTA) is permuted alike.  One MMA covers 16 tokens and 8
// rows of W.  A warp has the loads of U blocks in flight at once.  The warps' partial sums meet in shared memory in
// warp order, so results do not depend on timing.
//
// The second kernel of a call starts while the first one drains (programmatic launch): its first weights are on their
// way before it waits for the first one's results.
#include "dense.cuh"
#include "moe_internal.cuh"

namespace qeffn {

namespace {

struct RowsArgs {
    const uint8_t *w0, *w1;     // rows of Kb bytes (w1: up, gated products)
    const uint8_t *x;           // token rows, ldx bytes apart
    long long ldx;
    int T, N, Kb;               // Kb: bytes of a row of W
    int act;
    void *out, *out1, *out2;
    int out_dtype, type;
    long long ldo;
    const float *row_scale, *col_scale0, *col_scale1, *bias;
    int first;                  // first kernel of its call: nothing is read before the wait
};

__device__ __forceinline__ uint4 ldg_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <int TYPE>
struct AccT { using type = float; };
template <>
struct AccT<DT_S8> { using type = int; };

// D (16 tokens x 8 rows) += A . B over 32 bytes of the reduction index.
template <int TYPE>
__device__ __forceinline__ void mma(typename AccT<TYPE>::type (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    if constexpr (TYPE == MOE_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else if constexpr (TYPE == MOE_FP16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void put(void *p, int dtype, long long i, float v) {
    if (dtype == MOE_BF16) ((__nv_bfloat16 *)p)[i] = from_f32<__nv_bfloat16>(v);
    else if (dtype == MOE_FP16) ((__half *)p)[i] = from_f32<__half>(v);
    else ((float *)p)[i] = v;
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// TT: groups of 8 tokens (1, 2 or 4).  G: groups of 8 rows.  KW: warps, U: blocks in flight per warp, MB: CTAs per SM.
template <int TYPE, int TT, bool GATE, int G, int KW, int U, int MB>
__global__ void __launch_bounds__(KW * 32, MB) k_rows(const RowsArgs p) {
    using Acc = typename AccT<TYPE>::type;
    constexpr int NW = GATE ? 2 : 1;
    constexpr int S = G * NW;               // weight streams: stream s is row group s % G of matrix s / G
    constexpr int MT = (TT + 1) / 2;        // 16-token tiles
    constexpr int NA = TT == 1 ? 2 : 4;     // accumulator values with tokens in them
    __shared__ Acc red[KW][S][MT][NA][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int r0 = 8 * G * blockIdx.x;
    const int nblk = (p.Kb + 127) >> 7;     // 128-byte blocks of a row
    const uint8_t *w0 = p.w0 + (size_t)(r0 + g) * p.Kb + 16 * c;
    const uint8_t *w1 = GATE ? p.w1 + (size_t)(r0 + g) * p.Kb + 16 * c : nullptr;
    const uint8_t *x = p.x + g * p.ldx + 16 * c;
    Acc acc[S][MT][4] = {};
    bool waited = false;
    if (p.first) {   // the kernel before may be anyone's: bring the first weights as far as L2, then wait
        for (int s = 0; s < S; ++s)
            if (r0 + 8 * (s % G) + g < p.N && 128 * warp + 16 * c < p.Kb)
                prefetch_l2((s >= G ? w1 : w0) + (size_t)8 * (s % G) * p.Kb + 128 * warp);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;");
        waited = true;
    }
    for (int b0 = warp; b0 < nblk || !waited; b0 += KW * U) {
        uint4 wv[U][2][S];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const int off = 128 * (b0 + u * KW) + 64 * h;
                    wv[u][h][s] = r0 + 8 * (s % G) + g < p.N && off + 16 * c < p.Kb
                                      ? ldg_stream((s >= G ? w1 : w0) + (size_t)8 * (s % G) * p.Kb + off)
                                      : make_uint4(0, 0, 0, 0);
                }
        if (!waited) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;");
            waited = true;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int off = 128 * (b0 + u * KW) + 64 * h;
                const bool in = off + 16 * c < p.Kb;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                    if (in && 16 * m + g < p.T) lo = *reinterpret_cast<const uint4 *>(x + 16 * m * p.ldx + off);
                    if (TT > 1 && in && 16 * m + 8 + g < p.T) hi = *reinterpret_cast<const uint4 *>(x + (16 * m + 8) * p.ldx + off);
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        mma<TYPE>(acc[s][m], lo.x, hi.x, lo.y, hi.y, wv[u][h][s].x, wv[u][h][s].y);
                        mma<TYPE>(acc[s][m], lo.z, hi.z, lo.w, hi.w, wv[u][h][s].z, wv[u][h][s].w);
                    }
                }
            }
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NA; ++i) red[warp][s][m][i][lane] = acc[s][m][i];
    __syncthreads();
    // sums over the warps, in warp order
    for (int e = threadIdx.x; e < G * MT * NA * 32; e += KW * 32) {
        const int ln = e & 31, i = (e >> 5) % NA, m = (e >> 5) / NA % MT, s = (e >> 5) / (NA * MT);
        Acc v = 0, v1 = 0;
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            v += red[k][s][m][i][ln];
            if (GATE) v1 += red[k][(NW - 1) * G + s][m][i][ln];
        }
        const int t = 16 * m + (ln >> 2) + 8 * (i >> 1);
        const long long r = r0 + 8 * s + 2 * (ln & 3) + (i & 1);
        if (t >= p.T || r >= p.N) continue;
        float f = (float)v, f1 = (float)v1;
        if (TYPE == DT_S8) {
            f *= p.row_scale[t] * p.col_scale0[r];
            if (GATE) f1 *= p.row_scale[t] * p.col_scale1[r];
            else if (p.bias) f += p.bias[r];
        }
        if (GATE) {
            put(p.out, p.out_dtype, t * p.ldo + r, act_fwd(p.act, f) * f1);
            if (p.out1) {
                put(p.out1, p.type, (long long)t * p.N + r, f);
                put(p.out2, p.type, (long long)t * p.N + r, f1);
            }
        } else {
            put(p.out, p.out_dtype, t * p.ldo + r, f);
        }
    }
}

template <int TYPE, int TT, bool GATE, int G, int KW, int U, int MB>
int launch_rows_as(const RowsArgs &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((p.N + 8 * G - 1) / (8 * G));
    cfg.blockDim = dim3(KW * 32);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    QE_CHECK(cudaLaunchKernelEx(&cfg, k_rows<TYPE, TT, GATE, G, KW, U, MB>, p));
    QE_CHECK_LAUNCH("k_rows");
    return MOE_OK;
}

// Shapes, measured on B200 in us (launches back to back, each waiting for the last; rows x bytes a row).  A block is 128
// bytes of a row; `brief` rows have fewer than 32.
//   gate and up, one token: 8 warps, 2 CTAs an SM 10240 x 5120 17.5 (3 CTAs 18.6, 4 warps x 6 19.9, 16 x 2 20.5); many brief
//   rows 4 warps with 2 blocks in flight 5000 x 1024 3.6 (8 warps 4.5), 6000 x 2048 6.3 (6.5), at 16 tokens 4
//   warps x 6 CTAs 7.0 (8.0); but 2048 x 2048 8 warps, 3.5 (3.6 and more)
//   a grid below the SM count: 16 warps (2 x 512 x 5120 3.3, 8 warps 3.7; 1024 x 12000, 12 tokens 6.2, 8 warps 7.7)
//   one matrix, one token: 2560 x 20480 8 warps with 4 blocks in flight 11.8 (2 blocks 13.1, 4 warps 16.5, 16 warps 13.7);
//   two row groups a CTA for more rows, 16 warps 12288 x 8192 18.7 (20.3), and for brief rows, 4 warps 10240 x 2560 6.0 (7.3)
//   one matrix, several tokens: two row groups a CTA, because the token operand costs as much as the weights; 16 warps for
//   up to 4096 rows or rows of 64 blocks (2048 x 2048, 32 tokens 2.9, one group 3.8; 2560 x 20480, 16 tokens 16.9, 8 warps
//   20.9), else 4 warps (10240 x 2560 8-bit, 16 tokens 8.0, one group 9.5, 16 warps 10.8)
template <int TYPE, int TT>
int launch_rows_t(const RowsArgs &p, bool gate, cudaStream_t st) {
    const bool few = p.N <= 8 * 148, brief = p.Kb < 32 * 128;
    if (gate) {
        if (few) return launch_rows_as<TYPE, TT, true, 1, 16, 1, 1>(p, st);
        if (!brief || p.N <= 4096) return launch_rows_as<TYPE, TT, true, 1, 8, 1, 2>(p, st);
        if constexpr (TT == 1) return launch_rows_as<TYPE, TT, true, 1, 4, 2, 4>(p, st);
        return launch_rows_as<TYPE, TT, true, 1, 4, 1, 6>(p, st);
    }
    if (few) return launch_rows_as<TYPE, TT, false, 1, 16, 2, 1>(p, st);
    if constexpr (TT == 1) {
        if (brief) return launch_rows_as<TYPE, TT, false, 2, 4, 2, 4>(p, st);
        return p.N > 4096 ? launch_rows_as<TYPE, TT, false, 2, 16, 1, 2>(p, st) : launch_rows_as<TYPE, TT, false, 1, 8, 4, 3>(p, st);
    }
    if (p.N <= 4096 || p.Kb >= 64 * 128) return launch_rows_as<TYPE, TT, false, 2, 16, 1, 2>(p, st);
    return launch_rows_as<TYPE, TT, false, 2, 4, 1, 6>(p, st);
}

template <int TYPE>
int launch_rows_type(const RowsArgs &p, bool gate, cudaStream_t st) {
    if (p.T <= 8) return launch_rows_t<TYPE, 1>(p, gate, st);
    return p.T <= 16 ? launch_rows_t<TYPE, 2>(p, gate, st) : launch_rows_t<TYPE, 4>(p, gate, st);
}

}  // namespace

// Which products these are.  Up to 16 rows always; up to 32 while the weights are few, where the launch counts.  A bf16
// block at 32 rows, us: 512 x 512 4.5 (tensor-core tiles 8.6), 1024 x 2048 8.4 (13.7), 2560 x 5120 32 (26), 2560 x 10240 56
// (39).  The limit is a product's, not the block's: 2048 x 4096 tiles its gate and up and streams its down projection,
// 29 (22 with both streamed).
bool rows_fit(const GemmArgs &g) {
    if (g.a_mn || g.b_mn || g.segs != 1) return false;
    const long long bytes = (long long)g.N * g.K * (g.type == DT_S8 ? 1 : 2) * (g.epi == EPI_GATE ? 2 : 1);
    return g.M <= 16 || (g.M <= 32 && bytes <= 24LL << 20);
}

int launch_rows(const GemmArgs &g, cudaStream_t st) {
    const int size = g.type == DT_S8 ? 1 : 2;
    RowsArgs p = {};
    p.w0 = (const uint8_t *)g.b[0], p.w1 = (const uint8_t *)g.b[1];
    p.x = (const uint8_t *)g.a[0];
    p.ldx = g.lda * size;
    p.T = g.M, p.N = g.N, p.Kb = g.K * size;
    p.act = g.act;
    p.out = g.out, p.out1 = g.out1, p.out2 = g.out2, p.out_dtype = g.out_dtype, p.type = g.type, p.ldo = g.ldo;
    p.row_scale = g.row_scale, p.col_scale0 = g.col_scale[0], p.col_scale1 = g.col_scale[1], p.bias = g.bias;
    p.first = !g.b_ready;
    const bool gate = g.epi == EPI_GATE;
    if (g.type == DT_S8) return launch_rows_type<DT_S8>(p, gate, st);
    return g.type == MOE_FP16 ? launch_rows_type<MOE_FP16>(p, gate, st) : launch_rows_type<MOE_BF16>(p, gate, st);
}

}  // namespace qeffn
