// Matrix products of the dense feed-forward operators on the tensor cores.
//
// C [M][N] = A . B^T with fp32 (8-bit operands: int32) accumulators in TMEM.  One persistent kernel, a CTA pair on two
// SMs per output tile of 256 x 256: each CTA holds 128 rows of A and 128 rows of B of every k step, and the pair's MMA
// (M = 256, N = 256) reads both halves, so an operand byte is loaded into shared memory once per 256 rows of the other
// operand.  A k step is 128 bytes of the reduction index (64 16-bit or 128 8-bit values), staged by TMA through a ring
// of shared-memory stages with the 128-byte swizzle.  Operands may be stored with either index contiguous (the
// gradients read weights and activations as they lie; the MMA's transpose bits do the rest), and rows, columns and
// reduction tails past the end read as zeros (TMA) and are clipped on the way out.
//
//   warp 0: TMA producer (one lane)         warp 1: MMA issuer (one lane of the pair's first CTA)
//   warp 2: TMEM allocation                 warps 4..7: epilogue (TMEM lane quarter = warp % 4)
//
// TMEM holds two 256-column accumulators, so a tile's epilogue runs while the next tile's MMAs do.  The gated forward
// product takes 128 gate columns from the first CTA's B and the 128 up columns of the same index from the second's:
// column c and column 128 + c of a row meet in one thread.
#include <algorithm>

#include "dense.cuh"
#include "dense_ptx.cuh"
#include "moe_internal.cuh"

namespace qeffn {

using namespace dense;

namespace {

constexpr int GT_NT = 256;
constexpr int GT_N = 256;                   // accumulator columns of a tile
constexpr int GT_KB = 128;                  // bytes of the reduction index per stage
constexpr int GT_STAGES = 5;
constexpr int GT_HALF = 128 * GT_KB;        // 128 operand rows of a stage
constexpr int GT_STAGE = 2 * GT_HALF;       // A and B of one CTA
constexpr int GT_EPI_W0 = 4;
constexpr int GT_BUF = 4096;                // an epilogue warp's store tile: 32 rows of 128 bytes
constexpr int GT_NBUF = 3;                  // tiles in flight per epilogue warp
constexpr int GT_SMEM = 1024 + GT_STAGES * GT_STAGE + 4 * GT_NBUF * GT_BUF + 256;

struct Maps {
    CUtensorMap a[2], b[2], out[3];
};

struct TileArgs {
    int M, N, kblocks, segs;    // kblocks: k steps of one segment
    int tiles_m, tiles_n;
    int act;
    int fp16;                   // 16-bit operands (and out1, out2): fp16 rather than bf16
    int out_dtype;
    int add;
    int extra;                  // out1 and out2 wanted (EPI_GATE: both, EPI_GATE_BWD: out2)
    const void *in1, *in2;
    const float *row_scale, *col_scale0, *col_scale1, *bias;
};

struct GtBars {
    uint64_t full[GT_STAGES], empty[GT_STAGES], acc_full[2], acc_empty[2], mma_done;
    uint32_t tmem;
};

__device__ __forceinline__ uint32_t pack16(float a, float b, int fp16) {
    if (fp16) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack16(uint32_t v, int fp16) {
    if (fp16) return __half22float2(*reinterpret_cast<__half2 *>(&v));
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
}

// 32 values of this lane's row into half `half` (32 16-bit columns) of a swizzled 32 x 64 store tile.
__device__ __forceinline__ void stage16(uint8_t *buf, int lane, int half, const float (&v)[32], int fp16) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 w = make_uint4(pack16(v[8 * c], v[8 * c + 1], fp16), pack16(v[8 * c + 2], v[8 * c + 3], fp16),
                                   pack16(v[8 * c + 4], v[8 * c + 5], fp16), pack16(v[8 * c + 6], v[8 * c + 7], fp16));
        *reinterpret_cast<uint4 *>(buf + lane * 128 + (((4 * half + c) ^ (lane & 7)) << 4)) = w;
    }
}
// 32 fp32 values: the whole row of a 32 x 32 store tile.
__device__ __forceinline__ void stage32(uint8_t *buf, int lane, const float (&v)[32]) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<float4 *>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}

template <bool S8>
__device__ __forceinline__ void load_acc(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    tmem_ld32(taddr, r);
    tmem_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = S8 ? (float)(int)r[i] : __uint_as_float(r[i]);
}

// v[i] *= rs * cs[n + i]: the scales' product first, as the plain form has it.
__device__ __forceinline__ void apply_scale(float (&v)[32], float rs, const float *cs, int n, int N) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= rs * (n + i < N ? __ldg(cs + n + i) : 0.f);
}

// The store tiles of one epilogue warp: a ring of GT_NBUF buffers, each free again once its copy has been read.
struct StoreRing {
    uint8_t *base;
    int lane, at = 0;
    __device__ uint8_t *acquire() {
        if (lane == 0) tma_wait_read<GT_NBUF - 1>();
        __syncwarp();
        return base + at * GT_BUF;
    }
    __device__ void release(const CUtensorMap *m, int x, int y, bool in, bool add = false) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (in) {
                if (add) tma_add(m, x, y, base + at * GT_BUF);
                else tma_store(m, x, y, base + at * GT_BUF);
            }
            tma_commit();
        }
        at = at + 1 == GT_NBUF ? 0 : at + 1;
    }
};

template <bool S8, bool A_MN, bool B_MN, int EPI, int CG>
__global__ void __launch_bounds__(GT_NT, 1) k_gemm_tc(const __grid_constant__ Maps maps, const __grid_constant__ TileArgs p) {
    constexpr int BK = S8 ? 128 : 64;             // reduction values per stage
    constexpr int TM = 128 * CG;                  // rows of a tile
    constexpr int B_ROWS = GT_N / CG;             // B rows a CTA holds
    constexpr int STAGE = GT_HALF + B_ROWS * GT_KB;
    constexpr int STAGES = CG == 2 ? GT_STAGES : GT_STAGES * GT_STAGE / STAGE;
    constexpr int TN = EPI == EPI_GATE ? GT_N / 2 : GT_N;   // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
    uint8_t *bufs = smem + GT_STAGES * GT_STAGE;
    GtBars *bar = reinterpret_cast<GtBars *>(bufs + 4 * GT_NBUF * GT_BUF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar->acc_full[t], 1);
            mbar_init(&bar->acc_empty[t], 4 * CG);
        }
        mbar_init(&bar->mma_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc<CG>(&bar->tmem, 2 * GT_N);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;

    const int n_tiles = p.tiles_m * p.tiles_n;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const int ksteps = p.kblocks * p.segs;
    // tiles in bands of 8 row blocks, so that the tiles in flight share rows of both operands in L2
    auto tile_at = [&](int t, int &m0, int &n0) {
        const int band = t / (8 * p.tiles_n), in = t - band * 8 * p.tiles_n;
        const int rows = min(8, p.tiles_m - 8 * band);
        m0 = (8 * band + in % rows) * TM;
        n0 = (in / rows) * TN;
    };

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = first; t < n_tiles && ok; t += step) {
                int m0, n0;
                tile_at(t, m0, n0);
                m0 += rank * 128;
                for (int kb = 0; kb < ksteps && ok; ++kb, ++it) {
                    const int s = it % STAGES;
                    ok = mbar_wait(&bar->empty[s], ((it / STAGES) & 1) ^ 1);
                    if (!ok) break;
                    const int seg = kb >= p.kblocks, k0 = (kb - seg * p.kblocks) * BK;
                    uint8_t *sa = smem + s * STAGE, *sb = sa + GT_HALF;
                    if (rank == 0) mbar_expect_tx(&bar->full[s], CG * STAGE);
                    const uint32_t fb = CG == 2 ? map_rank(&bar->full[s], 0) : su32(&bar->full[s]);
                    const CUtensorMap *ma = &maps.a[seg];
                    if constexpr (A_MN) {
                        tma_load<CG>(sa, ma, m0, k0, fb);
                        tma_load<CG>(sa + GT_HALF / 2, ma, m0 + 64, k0, fb);
                    } else {
                        tma_load<CG>(sa, ma, k0, m0, fb);
                    }
#pragma unroll
                    for (int h = 0; h < B_ROWS / 128; ++h) {   // 128 rows of B each: which half of the tile
                        const int half = CG == 2 ? rank : h;
                        const CUtensorMap *mb = EPI == EPI_GATE ? &maps.b[half] : &maps.b[seg];
                        const int nb = EPI == EPI_GATE ? n0 : n0 + 128 * half;
                        uint8_t *dst = sb + h * GT_HALF;
                        if constexpr (B_MN) {
                            tma_load<CG>(dst, mb, nb, k0, fb);
                            tma_load<CG>(dst + GT_HALF / 2, mb, nb + 64, k0, fb);
                        } else {
                            tma_load<CG>(dst, mb, k0, nb, fb);
                        }
                    }
                }
            }
            // every copy has landed before the CTAs leave: the last fills that no MMA waited for
            if (!ok && rank == 0)
                for (int j = it - 1; j >= 0 && j >= it - STAGES; --j)
                    mbar_wait(&bar->full[j % STAGES], (j / STAGES) & 1, true);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = (S8 ? (2u << 4) | (1u << 7) | (1u << 10)
                                       : (1u << 4) | (p.fp16 ? 0u : (1u << 7) | (1u << 10))) |
                                   (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u) | ((uint32_t)(GT_N >> 3) << 17) |
                                   ((uint32_t)(TM >> 4) << 24);
            int it = 0, n = 0;
            bool ok = true;
            for (int t = first; t < n_tiles && ok; t += step, ++n) {
                ok = mbar_wait(&bar->acc_empty[n & 1], ((n >> 1) & 1) ^ 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + GT_N * (n & 1);
                for (int kb = 0; kb < ksteps; ++kb, ++it) {
                    const int s = it % STAGES;
                    ok = mbar_wait(&bar->full[s], (it / STAGES) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a0 = su32(smem + s * STAGE), b0 = a0 + GT_HALF;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // 32 bytes of k: within the 128-byte rows, or 16 of the 128-byte rows
                        const uint64_t ad = A_MN ? smem_desc(a0 + 2048 * j, GT_HALF / 2) : smem_desc(a0 + 32 * j, 16);
                        const uint64_t bd = B_MN ? smem_desc(b0 + 2048 * j, GT_HALF / 2) : smem_desc(b0 + 32 * j, 16);
                        umma<S8, CG>(acc, ad, bd, idesc, (kb | j) != 0);
                    }
                    umma_commit<CG>(&bar->empty[s]);
                }
                if (ok) umma_commit<CG>(&bar->acc_full[n & 1]);
            }
            umma_commit<CG>(&bar->mma_done);   // no MMA may still use shared memory or TMEM when the CTAs leave
            mbar_wait(&bar->mma_done, 0, true);
        }
        __syncwarp();
    } else if (warp >= GT_EPI_W0) {
        const int q = warp - GT_EPI_W0;
        StoreRing ring{bufs + q * GT_NBUF * GT_BUF, lane};
        const uint32_t empty0 = CG == 2 ? map_rank(&bar->acc_empty[0], 0) : su32(&bar->acc_empty[0]);
        int n = 0;
        bool ok = true;
        for (int t = first; t < n_tiles && ok; t += step, ++n) {
            int m0, n0;
            tile_at(t, m0, n0);
            m0 += rank * 128 + 32 * q;                    // this warp's 32 rows
            const long long m = m0 + lane;
            const bool live = m < p.M;
            float rs = 1.f;
            if constexpr (S8) rs = live ? p.row_scale[m] : 0.f;
            ok = mbar_wait(&bar->acc_full[n & 1], (n >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + GT_N * (n & 1);
            const bool rows_in = m0 < p.M;
            if constexpr (EPI == EPI_STORE) {
                if (p.out_dtype == MOE_FP32) {
#pragma unroll 1
                    for (int c = 0; c < GT_N; c += 32) {
                        float v[32];
                        load_acc<S8>(acc + c, v);
                        if constexpr (S8) apply_scale(v, rs, p.col_scale0, n0 + c, p.N);
                        if (S8 && p.bias)
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] += n0 + c + i < p.N ? __ldg(p.bias + n0 + c + i) : 0.f;
                        stage32(ring.acquire(), lane, v);
                        ring.release(&maps.out[0], n0 + c, m0, rows_in && n0 + c < p.N, p.add);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < GT_N; c += 64) {
                        uint8_t *buf = ring.acquire();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float v[32];
                            const int nc = n0 + c + 32 * h;
                            load_acc<S8>(acc + c + 32 * h, v);
                            if constexpr (S8) apply_scale(v, rs, p.col_scale0, nc, p.N);
                            if (S8 && p.bias)
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] += nc + i < p.N ? __ldg(p.bias + nc + i) : 0.f;
                            stage16(buf, lane, h, v, p.out_dtype == MOE_FP16);
                        }
                        ring.release(&maps.out[0], n0 + c, m0, rows_in && n0 + c < p.N);
                    }
                }
            } else if constexpr (EPI == EPI_GATE) {
                if constexpr (S8) {   // h in fp32, for the quantisation that follows
#pragma unroll 1
                    for (int c = 0; c < TN; c += 32) {
                        float g[32], u[32];
                        load_acc<S8>(acc + c, g);
                        load_acc<S8>(acc + TN + c, u);
                        apply_scale(g, rs, p.col_scale0, n0 + c, p.N);
                        apply_scale(u, rs, p.col_scale1, n0 + c, p.N);
#pragma unroll
                        for (int i = 0; i < 32; ++i) g[i] = act_fwd(p.act, g[i]) * u[i];
                        stage32(ring.acquire(), lane, g);
                        ring.release(&maps.out[0], n0 + c, m0, rows_in && n0 + c < p.N);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < TN; c += 64) {
                        const bool in = rows_in && n0 + c < p.N;
                        uint8_t *bg = ring.base, *bu = ring.base + GT_BUF, *bh = ring.base + 2 * GT_BUF;
                        if (lane == 0) tma_wait_read<0>();
                        __syncwarp();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float g[32], u[32];
                            load_acc<S8>(acc + c + 32 * h, g);
                            load_acc<S8>(acc + TN + c + 32 * h, u);
                            if (p.extra) {
                                stage16(bg, lane, h, g, p.fp16);
                                stage16(bu, lane, h, u, p.fp16);
                            }
#pragma unroll
                            for (int i = 0; i < 32; ++i) g[i] = act_fwd(p.act, g[i]) * u[i];
                            stage16(bh, lane, h, g, p.fp16);
                        }
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0 && in) {
                            tma_store(&maps.out[0], n0 + c, m0, bh);
                            if (p.extra) {
                                tma_store(&maps.out[1], n0 + c, m0, bg);
                                tma_store(&maps.out[2], n0 + c, m0, bu);
                            }
                            tma_commit();
                        }
                    }
                }
            } else {
                const uint16_t *gp = (const uint16_t *)p.in1 + m * p.N, *up = (const uint16_t *)p.in2 + m * p.N;
#pragma unroll 1
                for (int c = 0; c < TN; c += 64) {
                    const bool in = rows_in && n0 + c < p.N;
                    uint8_t *bg = ring.base, *bu = ring.base + GT_BUF, *bh = ring.base + 2 * GT_BUF;
                    if (lane == 0) tma_wait_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v[32], du[32], hh[32];
                        load_acc<S8>(acc + c + 32 * h, v);
                        const int nc = n0 + c + 32 * h;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint4 gw = make_uint4(0, 0, 0, 0), uw = gw;
                            if (live && nc + 8 * j < p.N) {   // N is a multiple of 8
                                gw = *reinterpret_cast<const uint4 *>(gp + nc + 8 * j);
                                uw = *reinterpret_cast<const uint4 *>(up + nc + 8 * j);
                            }
                            const uint32_t gs[4] = {gw.x, gw.y, gw.z, gw.w}, us[4] = {uw.x, uw.y, uw.z, uw.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 z = unpack16(gs[i], p.fp16), u = unpack16(us[i], p.fp16);
                                const int e = 8 * j + 2 * i;
                                float a0, d0, a1, d1;
                                act_bwd(p.act, z.x, a0, d0);
                                act_bwd(p.act, z.y, a1, d1);
                                du[e] = v[e] * a0, du[e + 1] = v[e + 1] * a1;
                                hh[e] = a0 * u.x, hh[e + 1] = a1 * u.y;
                                v[e] *= u.x * d0, v[e + 1] *= u.y * d1;
                            }
                        }
                        stage16(bg, lane, h, v, p.fp16);
                        stage16(bu, lane, h, du, p.fp16);
                        if (p.extra) stage16(bh, lane, h, hh, p.fp16);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0 && in) {
                        tma_store(&maps.out[0], n0 + c, m0, bg);
                        tma_store(&maps.out[1], n0 + c, m0, bu);
                        if (p.extra) tma_store(&maps.out[2], n0 + c, m0, bh);
                        tma_commit();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(empty0 + 8 * (n & 1));   // the accumulator may be overwritten
        }
        if (lane == 0) tma_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    if (warp == 2) tmem_dealloc<CG>(tmem, 2 * GT_N);
    if constexpr (CG == 2) cluster_sync();   // neither CTA leaves while the other still frees the pair's TMEM
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (the library does not link libcuda).
EncodeFn encoder() {
    static EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeFn)p;
    }();
    return fn;
}

// Tiles of box_inner x box_outer elements of a row-major [outer][inner] matrix, 128-byte swizzle.
int encode(CUtensorMap *m, int dtype, const void *p, long long inner, long long outer, long long ld, int box_inner, int box_outer) {
    EncodeFn fn = encoder();
    if (!fn) return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available in this driver");
    const int size = dtype == DT_S8 ? 1 : dtype == MOE_FP32 ? 4 : 2;
    const CUtensorMapDataType t = dtype == DT_S8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : dtype == MOE_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                      : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer}, strides[1] = {(cuuint64_t)ld * size};
    const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_outer}, es[2] = {1, 1};
    const CUresult r = fn(m, t, 2, const_cast<void *>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

template <bool S8, bool A_MN, bool B_MN, int EPI, int CG>
int launch_tc(const Maps &maps, const TileArgs &p, cudaStream_t st) {
    auto kern = k_gemm_tc<S8, A_MN, B_MN, EPI, CG>;
    constexpr int kMaxDevices = 64;
    static int units[kMaxDevices] = {};   // tiles in flight on a device: looked up once, racing threads store the same
    int dev = 0;
    QE_CHECK(cudaGetDevice(&dev));
    if (dev >= kMaxDevices) return set_error(MOE_ERR_UNSUPPORTED, "device index above 63");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.blockDim = dim3(GT_NT);
    cfg.dynamicSmemBytes = GT_SMEM;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {CG, 1, 1};
    int n = __atomic_load_n(&units[dev], __ATOMIC_RELAXED);
    if (n == 0) {
        int sms = 0;
        QE_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GT_SMEM));
        QE_CHECK(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
        cfg.gridDim = dim3(sms / CG * CG);
        QE_CHECK(cudaOccupancyMaxActiveClusters(&n, kern, &cfg));
        if (n < 1) return set_error(MOE_ERR_UNSUPPORTED, "the device cannot hold the product's kernel");
        __atomic_store_n(&units[dev], n, __ATOMIC_RELAXED);
    }
    cfg.gridDim = dim3(std::min(n, p.tiles_m * p.tiles_n) * CG);
    QE_CHECK(cudaLaunchKernelEx(&cfg, kern, maps, p));
    QE_CHECK_LAUNCH("k_gemm_tc");
    return MOE_OK;
}

template <int CG>
int dispatch(const GemmArgs &g, const Maps &m, const TileArgs &p, cudaStream_t st) {
    if (g.type == DT_S8)
        return g.epi == EPI_GATE ? launch_tc<true, false, false, EPI_GATE, CG>(m, p, st)
                                 : launch_tc<true, false, false, EPI_STORE, CG>(m, p, st);
    if (g.epi == EPI_GATE) return launch_tc<false, false, false, EPI_GATE, CG>(m, p, st);
    if (g.epi == EPI_GATE_BWD) return launch_tc<false, false, true, EPI_GATE_BWD, CG>(m, p, st);
    if (g.a_mn) return launch_tc<false, true, true, EPI_STORE, CG>(m, p, st);
    if (g.b_mn) return launch_tc<false, false, true, EPI_STORE, CG>(m, p, st);
    return launch_tc<false, false, false, EPI_STORE, CG>(m, p, st);
}

}  // namespace

int read_dense_error(int *code) {
    const int zero = 0;
    QE_CHECK(cudaMemcpyFromSymbol(code, g_error, sizeof(int)));
    if (*code) QE_CHECK(cudaMemcpyToSymbol(g_error, &zero, sizeof(int)));
    return MOE_OK;
}

int launch_gemm(const GemmArgs &g, Link link, cudaStream_t st) {
    if (g.M <= kFewRows && !g.a_mn && !g.b_mn && g.segs == 1) return launch_rows(g, link, st);
    const int bk = g.type == DT_S8 ? 128 : 64;
    const int cg = g.M > 128 ? 2 : 1;
    Maps m;
    TileArgs p = {};
    p.M = g.M, p.N = g.N, p.segs = g.segs;
    p.kblocks = (g.K + bk - 1) / bk;
    const int tm = 128 * cg, tn = g.epi == EPI_GATE ? GT_N / 2 : GT_N;
    p.tiles_m = (g.M + tm - 1) / tm;
    p.tiles_n = (g.N + tn - 1) / tn;
    p.act = g.act;
    p.fp16 = g.type == MOE_FP16;
    p.out_dtype = g.out_dtype;
    p.add = g.add;
    p.extra = g.out2 != nullptr;
    p.in1 = g.in1, p.in2 = g.in2;
    p.row_scale = g.row_scale, p.col_scale0 = g.col_scale[0], p.col_scale1 = g.col_scale[1], p.bias = g.bias;
    for (int s = 0; s < 2; ++s) {
        const void *a = g.a[s] ? g.a[s] : g.a[0], *b = g.b[s] ? g.b[s] : g.b[0];
        if (g.a_mn) QE_TRY(encode(&m.a[s], g.type, a, g.M, g.K, g.lda, 64, bk));
        else QE_TRY(encode(&m.a[s], g.type, a, g.K, g.M, g.lda, bk, 128));
        if (g.b_mn) QE_TRY(encode(&m.b[s], g.type, b, g.N, g.K, g.ldb, 64, bk));
        else QE_TRY(encode(&m.b[s], g.type, b, g.K, g.N, g.ldb, bk, 128));
    }
    void *outs[3] = {g.out, g.out1 ? g.out1 : g.out, g.out2 ? g.out2 : g.out};
    for (int i = 0; i < 3; ++i) {
        const bool main = outs[i] == g.out;
        const int t = main ? g.out_dtype : g.type;
        QE_TRY(encode(&m.out[i], t, outs[i], g.N, g.M, main ? g.ldo : g.N, t == MOE_FP32 ? 32 : 64, 32));
    }
    return cg == 2 ? dispatch<2>(g, m, p, st) : dispatch<1>(g, m, p, st);
}

}  // namespace qeffn
