// Matrix products of the dense feed-forward operators on the tensor cores.
//
// C [M][N] = A . B^T with fp32 (8-bit operands: int32) accumulators in TMEM.  One persistent kernel.  A tile is 256 rows
// by C columns on a CTA pair (two SMs; the pair's MMAs have M = 256, each CTA holds 128 rows of A and half of B's rows,
// so that an operand byte enters shared memory once per 256 rows of the other operand), or 128 rows on one CTA where
// there are no more rows than that.  A k step is 128 bytes of the reduction index (64 16-bit or 128 8-bit values),
// staged by TMA through a ring of shared-memory stages with the 128-byte swizzle.  Operands may be stored with either
// index contiguous (the gradients read weights and activations as they lie; the MMA's transpose bits do the rest), and
// rows, columns and reduction tails past the end read as zeros (TMA) and are clipped on the way out.
//
//   warp 0: TMA producer (one lane)         warp 1: MMA issuer (one lane of the pair's first CTA)
//   warp 2: TMEM allocation                 warps 4..11: epilogue (TMEM lane quarter = warp % 4, two warps a quarter)
//
// A tile's columns are one or two sub-tiles of W <= 256, an accumulator of W TMEM columns each.  With one sub-tile TMEM
// holds two tiles' accumulators and the epilogue of a tile runs while the next tile's MMAs do; two sub-tiles serve
// calls whose tiles then all fit on the device at once.  The gated forward product takes the first half of a sub-tile's
// B rows from the gate matrix and the second from the up matrix: column c and column W/2 + c of a row meet in one
// thread.  Calls with few tiles split the reduction index over the CTAs of a cluster: the partial accumulators go to
// shared memory, and every CTA sums (in split order) and finishes some of the columns.
//
// The tile shape comes from a model of the time (choose(), below), not from a table of sizes.
#include <algorithm>

#include "dense.cuh"
#include "dense_ptx.cuh"
#include "moe_internal.cuh"

namespace qeffn {

using namespace dense;

namespace {

constexpr int GT_NT = 384;
constexpr int GT_W = 256;                   // largest sub-tile width; TMEM columns between accumulators
constexpr int GT_KB = 128;                  // bytes of the reduction index per stage
constexpr int GT_A = 128 * GT_KB;           // bytes of A per stage: 128 rows of one k step
constexpr int GT_MAX_STAGES = 8;
constexpr int GT_RING = 161 * 1024;         // bytes of the stage ring
constexpr int GT_EPI_W0 = 4, GT_EPI_NW = 8;
constexpr int GT_UNIT = 32;                 // columns an epilogue warp handles at a time
constexpr int GT_SLOT = 8192;               // an epilogue warp's store tiles: two of 32 rows x 128 bytes, or three x 64
constexpr int GT_SMEM = 1024 + GT_RING + GT_EPI_NW * GT_SLOT + 256;

// A launch is one product, or a group of up to four that share the tile shape (the gradients).
template <int NG>
struct Maps {
    CUtensorMap a[NG][2], b[NG][2], out[NG > 3 ? NG : 3];   // out: of one product's up to three outputs, or of each product
};

struct Product {
    int M, N, kblocks, segs;    // kblocks: k steps of one segment
    int tiles_m, tiles_n, start;   // start: index of its first tile
    int a_mn;
    int a_rows;                 // rows of an A box: fewer than 128 where all rows fit in one
    int b_ready;                // B does not depend on kernels of the same call: it may be loaded before the wait
    int out_dtype, add;
};

template <int NG>
struct TileArgs {
    Product prod[NG];
    int products, tiles;        // tiles of all products
    int big, rounds;            // order of the tiles, see Order
    int W, subs;                // sub-tile width, sub-tiles per tile
    int splits, kper;           // reduction splits (CTAs or pairs of a cluster), k steps each
    int stages, stage_bytes, b_bytes;   // b_bytes: a sub-tile's B in one CTA
    long long tile_wait;        // limit of the epilogue's wait for a tile, see tile_wait_cycles()
    int act;
    int fp16;                   // 16-bit operands (and out1, out2): fp16 rather than bf16
    int one_out;                // one output a tile: two store tiles take turns
    int wide;                   // it is 16-bit and its store tiles have 64 columns
    int extra;                  // out1 and out2 wanted (EPI_GATE: both, EPI_GATE_BWD: out2)
    const void *in1, *in2;
    const float *row_scale, *col_scale0, *col_scale1, *bias;
};

struct GtBars {
    uint64_t full[GT_MAX_STAGES], empty[GT_MAX_STAGES], acc_full[2], acc_empty[2], mma_done;
    uint32_t tmem;
};

template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    if constexpr (FP16) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}
// 32 values of four 16-byte loads (the type's branch outside the loop, as with the activations below).
template <bool FP16>
__device__ __forceinline__ void unpack_as(const uint4 (&w)[4], float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t e[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = FP16 ? __half22float2(*reinterpret_cast<const __half2 *>(&e[i]))
                                  : make_float2(__uint_as_float(e[i] << 16), __uint_as_float(e[i] & 0xFFFF0000u));
            v[8 * j + 2 * i] = f.x, v[8 * j + 2 * i + 1] = f.y;
        }
    }
}
__device__ __forceinline__ void unpack16(const uint4 (&w)[4], float (&v)[32], int fp16) {
    if (fp16) unpack_as<true>(w, v);
    else unpack_as<false>(w, v);
}

// 32 values of this lane's row into a store tile of 32 rows: of 64 bytes (64-byte swizzle: 16-byte part c of row r at part
// c ^ (r / 2 % 4)), or half h of 128 bytes (128-byte swizzle: part c at c ^ (r % 8)).
template <bool FP16>
__device__ __forceinline__ void stage16_as(uint8_t *buf, int lane, const float (&v)[32], bool wide, int h) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 w = make_uint4(pack16<FP16>(v[8 * c], v[8 * c + 1]), pack16<FP16>(v[8 * c + 2], v[8 * c + 3]),
                                   pack16<FP16>(v[8 * c + 4], v[8 * c + 5]), pack16<FP16>(v[8 * c + 6], v[8 * c + 7]));
        const int at = wide ? lane * 128 + (((4 * h + c) ^ (lane & 7)) << 4) : lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4);
        *reinterpret_cast<uint4 *>(buf + at) = w;
    }
}
__device__ __forceinline__ void stage16(uint8_t *buf, int lane, const float (&v)[32], int fp16, bool wide = false, int h = 0) {
    if (fp16) stage16_as<true>(buf, lane, v, wide, h);
    else stage16_as<false>(buf, lane, v, wide, h);
}
// 32 fp32 values: the whole 128-byte row (128-byte swizzle).
__device__ __forceinline__ void stage32(uint8_t *buf, int lane, const float (&v)[32]) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<float4 *>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}

template <bool S8>
__device__ __forceinline__ float acc_value(uint32_t r) { return S8 ? (float)(int)r : __uint_as_float(r); }

// v[i] *= rs * cs[n + i]: the scales' product first, as the plain form has it.
__device__ __forceinline__ void apply_scale(float (&v)[32], float rs, const float *cs, int n, int N) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= rs * (n + i < N ? __ldg(cs + n + i) : 0.f);
}

// g = act(g) u for a unit; the choice of the activation stays outside the unrolled loops (inside, the code of all three
// for 32 elements did not fit the instruction cache: 4.6 us for one tile's epilogue).
template <int ACT>
__device__ __forceinline__ void gate_as(float (&g)[32], const float (&u)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) g[i] = act_fwd(ACT, g[i]) * u[i];
}
__device__ __forceinline__ void gate_all(int act, float (&g)[32], const float (&u)[32]) {
    if (act == MOE_ACT_SILU) gate_as<MOE_ACT_SILU>(g, u);
    else if (act == MOE_ACT_GELU_TANH) gate_as<MOE_ACT_GELU_TANH>(g, u);
    else gate_as<MOE_ACT_GELU>(g, u);
}
// In: v = dh, u = up, g = gate.  Out: v = dg, u = du, g = h.
template <int ACT>
__device__ __forceinline__ void gate_bwd_as(float (&v)[32], float (&u)[32], float (&g)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float a, d;
        act_bwd(ACT, g[i], a, d);
        const float dh = v[i], up = u[i];
        v[i] = dh * up * d;
        u[i] = dh * a;
        g[i] = a * up;
    }
}
__device__ __forceinline__ void gate_bwd_all(int act, float (&v)[32], float (&u)[32], float (&g)[32]) {
    if (act == MOE_ACT_SILU) gate_bwd_as<MOE_ACT_SILU>(v, u, g);
    else if (act == MOE_ACT_GELU_TANH) gate_bwd_as<MOE_ACT_GELU_TANH>(v, u, g);
    else gate_bwd_as<MOE_ACT_GELU>(v, u, g);
}

// A_MN: A's row index is contiguous (0, 1; 2: as each product of the group says).
template <bool S8, int A_MN, bool B_MN, int EPI, int CG, int NG>
__global__ void __launch_bounds__(GT_NT, 1) k_gemm_tc(const __grid_constant__ Maps<NG> maps, const __grid_constant__ TileArgs<NG> p) {
    constexpr int BK = S8 ? 128 : 64;             // reduction values per stage
    constexpr int TM = 128 * CG;                  // rows of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
    uint8_t *slots = smem + GT_RING;
    GtBars *bar = reinterpret_cast<GtBars *>(slots + GT_EPI_NW * GT_SLOT);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: uniform
    const uint32_t crank = cluster_rank();
    const uint32_t rank = CG == 2 ? crank & 1 : 0, even = crank - rank;   // rank in the pair, the pair's first CTA
    const int split = crank / CG;
    const int W = p.W, half = W / 2;
    const int tile_cols = (EPI == EPI_GATE ? half : W) * p.subs;          // output columns of a tile
    const bool two_acc = p.subs == 1;                                     // accumulators of two tiles in TMEM

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar->acc_full[t], 1);
            mbar_init(&bar->acc_empty[t], GT_EPI_NW * CG);
        }
        mbar_init(&bar->mma_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc<CG>(&bar->tmem, 2 * GT_W);
    if (warp == 3) {   // the copies' descriptors
        if (lane < 2 * p.products && (lane % 2 == 0 || p.prod[lane / 2].segs == 2)) prefetch_map(&maps.a[lane / 2][lane % 2]);
        if (lane < 2 * p.products && (lane % 2 == 0 || p.prod[lane / 2].segs == 2 || EPI == EPI_GATE))
            prefetch_map(&maps.b[lane / 2][lane % 2]);
        const int outs = EPI == EPI_STORE ? p.products : EPI == EPI_GATE ? (p.extra ? 3 : 1) : p.extra ? 3 : 2;
        if (lane < outs) prefetch_map(&maps.out[lane]);
    }
    tc_fence_before();
    __syncthreads();
    if (CG * p.splits > 1) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;
    const Order<(NG > 1)> order(p.tiles, p.big, p.rounds, blockIdx.x / (CG * p.splits), gridDim.x / (CG * p.splits));
    // tiles of a product in bands of 8 row blocks, so that the tiles in flight share rows of both operands in L2
    auto tile_at = [&](int t, int &m0, int &n0) {
        int g = 0;
        if constexpr (NG > 1)
            while (g + 1 < p.products && t >= p.prod[g + 1].start) ++g;
        const Product &pr = p.prod[g];
        t -= pr.start;
        const int band = t / (8 * pr.tiles_n), in = t - band * 8 * pr.tiles_n;
        const int rows = min(8, pr.tiles_m - 8 * band);
        m0 = (8 * band + in % rows) * TM;
        n0 = (in / rows) * tile_cols;
        return g;
    };
    const int k_begin = split * p.kper;
    auto k_end_of = [&](const Product &pr) { return min(pr.kblocks * pr.segs, k_begin + p.kper); };
    auto a_mn = [&](const Product &pr) { return A_MN == 2 ? pr.a_mn != 0 : A_MN == 1; };

    // programmatic launch: all of the above overlapped the kernel before; its results are touched from here on (the
    // producer of a product whose B is an input of the call first fills the ring with B)
    bool b_early = false;
    int t0 = 0;
    if (warp == 0) {
        t0 = order.at(0);
        int m0, n0;
        b_early = t0 >= 0 && p.prod[tile_at(t0, m0, n0)].b_ready;
    }
    if (!b_early) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;");
    }

    if (warp == 0) {
        int s = 0, filled = 0;
        uint32_t phase = 0;
        bool ok = true;
        // copies of k step kb of tile (m0, n0) into stage st: A's and B's (by the elected lane)
        auto load_a = [&](int st, int g, int kb, int m0) {
            const Product &pr = p.prod[g];
            const int seg = kb >= pr.kblocks, k0 = (kb - seg * pr.kblocks) * BK;
            uint8_t *sa = smem + st * p.stage_bytes;
            const uint32_t fb = CG == 2 ? map_rank(&bar->full[st], even) : su32(&bar->full[st]);
            if (a_mn(pr)) {
                tma_load<CG>(sa, &maps.a[g][seg], m0, k0, fb);
                tma_load<CG>(sa + GT_A / 2, &maps.a[g][seg], m0 + 64, k0, fb);
            } else {
                tma_load<CG>(sa, &maps.a[g][seg], k0, m0, fb);
            }
        };
        auto load_b = [&](int st, int g, int kb, int n0) {
            const Product &pr = p.prod[g];
            const int seg = kb >= pr.kblocks, k0 = (kb - seg * pr.kblocks) * BK;
            uint8_t *sb = smem + st * p.stage_bytes + GT_A;
            const uint32_t fb = CG == 2 ? map_rank(&bar->full[st], even) : su32(&bar->full[st]);
            const int a_bytes = a_mn(pr) ? GT_A : pr.a_rows * GT_KB;
            if (rank == 0) mbar_expect_tx(&bar->full[st], CG * (p.stage_bytes - GT_A + a_bytes));
            auto rows = [&](int sub, int h) {   // half h of a sub-tile's rows
                const CUtensorMap *mb = EPI == EPI_GATE ? &maps.b[g][h] : &maps.b[g][seg];
                const int nb = EPI == EPI_GATE ? n0 + sub * half : n0 + sub * W + h * half;
                if constexpr (B_MN) {   // chunks of 64 rows; the pair's last chunk may be half used
                    for (int c = 0; c < (CG == 2 ? half : W); c += 64, sb += 64 * 128) tma_load<CG>(sb, mb, nb + c, k0, fb);
                } else {
                    tma_load<CG>(sb, mb, k0, nb, fb);
                    sb += half * 128;
                }
            };
            if constexpr (CG == 2) {
                rows(0, rank);
                if (p.subs == 2) rows(1, rank);
            } else if constexpr (B_MN) {
                rows(0, 0);
                if (p.subs == 2) rows(1, 0);
            } else {
                rows(0, 0);
                rows(0, 1);
                if (p.subs == 2) rows(1, 0), rows(1, 1);
            }
        };
        int early = 0;   // stages whose B was requested before the wait
        if (b_early) {
            int m0, n0;
            const int g = tile_at(t0, m0, n0);
            early = min(p.stages, k_end_of(p.prod[g]) - k_begin);
            if (elect_one())
                for (int j = 0; j < early; ++j) load_b(j, g, k_begin + j, n0);
            __syncwarp();
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;");
        }
        for (int k = 0, t; ok && (t = order.at(k)) >= 0; ++k) {
            int m0, n0;
            const int g = tile_at(t, m0, n0);
            m0 += rank * 128;
            const int k_end = k_end_of(p.prod[g]);
            for (int kb = k_begin; kb < k_end; ++kb) {
                ok = mbar_wait(&bar->empty[s], phase ^ 1);
                if (!ok) break;
                if (elect_one()) {
                    if (filled >= early) load_b(s, g, kb, n0);
                    load_a(s, g, kb, m0);
                }
                __syncwarp();
                ++filled;
                if (++s == p.stages) s = 0, phase ^= 1;
            }
        }
        // after a failed wait every copy has to land before the CTAs leave: the last fills, which no MMA waited for, and
        // B requested ahead for fills that never came (their barriers stay open: the wait runs its full time)
        if (!ok && rank == 0) {
            for (int j = filled; j < early; ++j) mbar_wait(&bar->full[j], 0, true);
            for (int j = 0; j < p.stages && j < filled; ++j) {
                if (s == 0) s = p.stages, phase ^= 1;
                --s;
                mbar_wait(&bar->full[s], phase, true);
            }
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        const uint32_t idesc = (S8 ? (2u << 4) | (1u << 7) | (1u << 10)
                                   : (1u << 4) | (p.fp16 ? 0u : (1u << 7) | (1u << 10))) |
                               (B_MN ? 1u << 16 : 0u) | ((uint32_t)(W >> 3) << 17) |
                               ((uint32_t)(TM >> 4) << 24);
        int s = 0, n = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t; ok && (t = order.at(n)) >= 0; ++n) {
            const int slot = two_acc ? n & 1 : 0, use = two_acc ? n >> 1 : n;
            ok = mbar_wait(&bar->acc_empty[slot], (use & 1) ^ 1);
            if (!ok) break;
            tc_fence_after();
            int m0, n0;
            const Product &pr = p.prod[tile_at(t, m0, n0)];
            const int k_end = k_end_of(pr);
            const bool amn = a_mn(pr);
            const uint32_t id = idesc | (amn ? 1u << 15 : 0u), a_lead = amn ? 64 * 128 : 16, a_step = amn ? 128 : 2;
            for (int kb = k_begin; kb < k_end; ++kb) {
                ok = mbar_wait(&bar->full[s], phase);
                if (!ok) break;
                tc_fence_after();
                // 32 bytes of k at a time: within the 128-byte rows, or 16 of the 128-byte rows
                const uint32_t a0 = su32(smem + s * p.stage_bytes), acc = tmem + GT_W * slot;
                const uint64_t ad = smem_desc(a0, a_lead), bd = smem_desc(a0 + GT_A, B_MN ? 64 * 128 : 16);
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma<S8, CG>(acc, ad + a_step * j, bd + (B_MN ? 128 : 2) * j, id, kb > k_begin || j > 0);
                    if (p.subs == 2) {
                        const uint64_t b1 = bd + (p.b_bytes >> 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            umma<S8, CG>(acc + GT_W, ad + a_step * j, b1 + (B_MN ? 128 : 2) * j, id, kb > k_begin || j > 0);
                    }
                    umma_commit<CG>(&bar->empty[s], even);
                }
                __syncwarp();
                if (++s == p.stages) s = 0, phase ^= 1;
            }
            if (ok && elect_one()) umma_commit<CG>(&bar->acc_full[slot], even);
            __syncwarp();
        }
        if (elect_one()) umma_commit<CG>(&bar->mma_done, even);   // no MMA may still use shared memory or TMEM when the CTAs leave
        __syncwarp();
        mbar_wait(&bar->mma_done, 0, true);
    }

    const int q = warp & 3, team = (warp - GT_EPI_W0) >> 2;   // epilogue: lane quarter, which of its two warps
    uint8_t *slot_buf = slots + (warp - GT_EPI_W0) * GT_SLOT;
    // Splits: column of a partial tile in shared memory, the sub-tiles' columns following each other.
    auto part_col = [&](int col) { return col < GT_W ? col : col - GT_W + W; };
    // Columns [col, col + 32) of this lane's accumulator row: from TMEM, or summed over the splits of the cluster.
    auto get = [&](uint32_t acc, int col, float (&v)[32]) {
        uint32_t r[32];
        if (p.splits == 1) {
            tmem_ld32(acc + col, r);
            tmem_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = acc_value<S8>(r[i]);
        } else {
            int sum[32] = {};
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
            for (int j = 0; j < p.splits; ++j) {
                const uint32_t src = map_rank(smem + ((part_col(col) / 4) * 128 + 32 * q + lane) * 16, j * CG + rank);
                uint4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = ld_cluster(src + i * 2048);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t e[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (S8) sum[4 * i + k] += (int)e[k];
                        else v[4 * i + k] += __uint_as_float(e[k]);
                    }
                }
            }
            if constexpr (S8)
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = (float)sum[i];
        }
    };
    // Store tiles: two in turn where a tile has one output, else all at once.
    int turn = 0;
    auto acquire = [&]() {
        if (elect_one()) {
            if (p.one_out) tma_wait_read<1>();
            else tma_wait_read<0>();
        }
        __syncwarp();
        return slot_buf + 4096 * turn;
    };
    const bool wide = (EPI == EPI_STORE || (EPI == EPI_GATE && !S8)) && p.wide;
    const int unit_cols = wide ? 2 * GT_UNIT : GT_UNIT;
    // One unit of 32 (wide: 64) output columns: sub-tile `sub`, columns c.. of it.
    auto unit = [&](const Product &pr, const CUtensorMap *out, uint32_t acc, int sub, int c, int m0, int n0, float rs) {
        const int n = n0 + sub * (EPI == EPI_GATE ? half : W) + c;   // output column
        const long long m = m0 + lane;
        const bool in = m0 < pr.M && n < pr.N;
        const int col = sub * GT_W + c;
        float v[32];
        uint8_t *buf = nullptr;
        if constexpr (EPI == EPI_STORE) {
#pragma unroll 1
            for (int h = 0; h <= (int)wide; ++h) {
                const int nh = n + 32 * h;
                get(acc, col + 32 * h, v);
                if constexpr (S8) {
                    apply_scale(v, rs, p.col_scale0, nh, pr.N);
                    if (p.bias)
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] += nh + i < pr.N ? __ldg(p.bias + nh + i) : 0.f;
                }
                if (h == 0) buf = acquire();
                if (pr.out_dtype == MOE_FP32) stage32(buf, lane, v);
                else stage16(buf, lane, v, pr.out_dtype == MOE_FP16, wide, h);
            }
        } else if constexpr (EPI == EPI_GATE) {
#pragma unroll 1
            for (int h = 0; h <= (int)wide; ++h) {
                float u[32];
                get(acc, col + 32 * h, v);
                get(acc, col + half + 32 * h, u);
                if constexpr (S8) {
                    apply_scale(v, rs, p.col_scale0, n, pr.N);
                    apply_scale(u, rs, p.col_scale1, n, pr.N);
                }
                if (h == 0) buf = acquire();
                if constexpr (!S8)
                    if (p.extra) {
                        stage16(buf + 2048, lane, v, p.fp16);
                        stage16(buf + 4096, lane, u, p.fp16);
                    }
                gate_all(p.act, v, u);
                if constexpr (S8) stage32(buf, lane, v);   // h in fp32, for the quantisation that follows
                else stage16(buf, lane, v, p.fp16, wide, h);
            }
        } else {
            const uint4 *gp = reinterpret_cast<const uint4 *>((const uint16_t *)p.in1 + m * pr.N + n);
            const uint4 *up = reinterpret_cast<const uint4 *>((const uint16_t *)p.in2 + m * pr.N + n);
            uint4 gw[4], uw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                gw[j] = uw[j] = make_uint4(0, 0, 0, 0);
                if (m < pr.M && n + 8 * j < pr.N) gw[j] = gp[j], uw[j] = up[j];   // N is a multiple of 8
            }
            get(acc, col, v);
            buf = acquire();
            float du[32], hh[32];
            unpack16(gw, hh, p.fp16);
            unpack16(uw, du, p.fp16);
            gate_bwd_all(p.act, v, du, hh);
            stage16(buf, lane, v, p.fp16);
            stage16(buf + 2048, lane, du, p.fp16);
            if (p.extra) stage16(buf + 4096, lane, hh, p.fp16);
        }
        fence_async_smem();
        __syncwarp();
        if (in && elect_one()) {
            if (EPI == EPI_STORE && pr.add) tma_add(out, n, m0, buf);
            else tma_store(out, n, m0, buf);
            if (EPI == EPI_GATE_BWD || (EPI == EPI_GATE && !S8 && p.extra)) tma_store(out + 1, n, m0, buf + 2048);
            if (EPI != EPI_STORE && !S8 && p.extra) tma_store(out + 2, n, m0, buf + 4096);
            tma_commit();
        }
        if (p.one_out && in) turn ^= 1;
    };

    const int sub_cols = EPI == EPI_GATE ? half : W;   // output columns of a sub-tile
    if (p.splits == 1) {
        if (warp >= GT_EPI_W0) {
            const uint32_t empty0 = CG == 2 ? map_rank(&bar->acc_empty[0], even) : su32(&bar->acc_empty[0]);
            for (int n = 0, t; (t = order.at(n)) >= 0; ++n) {
                int m0, n0;
                const int g = tile_at(t, m0, n0);
                const Product &pr = p.prod[g];
                m0 += rank * 128 + 32 * q;                    // this warp's 32 rows
                float rs = 1.f;
                if constexpr (S8) rs = m0 + lane < pr.M ? p.row_scale[m0 + lane] : 0.f;
                const int slot = two_acc ? n & 1 : 0, use = two_acc ? n >> 1 : n;
                if constexpr (EPI == EPI_GATE_BWD)   // gate and up of this row: on their way to L2 while the MMAs run
                    if (m0 + lane < pr.M) {
                        const long long at = (long long)(m0 + lane) * pr.N;
                        for (int c = n0 + 64 * team; c < min(n0 + tile_cols, pr.N); c += 128) {
                            prefetch_l2((const uint16_t *)p.in1 + at + c);
                            prefetch_l2((const uint16_t *)p.in2 + at + c);
                        }
                    }
                if (!mbar_wait(&bar->acc_full[slot], use & 1, false, p.tile_wait)) break;
                tc_fence_after();
                const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + GT_W * slot;
                for (int sub = 0; sub < p.subs; ++sub)
#pragma unroll 1
                    for (int c = unit_cols * team; c < sub_cols; c += 2 * unit_cols)
                        unit(pr, &maps.out[g], acc, sub, c, m0, n0, rs);
                tc_fence_before();
                __syncwarp();
                if (elect_one()) mbar_arrive_cluster(empty0 + 8 * slot);   // the accumulators may be overwritten
            }
        }
    } else {
        // one tile per cluster: every split leaves its accumulators in shared memory (16 bytes, four columns, a row; the
        // ring is free once the last MMA has completed), and the splits share out the units
        int m0, n0;
        const int g = tile_at(order.at(0), m0, n0);
        const Product &pr = p.prod[g];
        m0 += rank * 128 + 32 * q;
        if (warp >= GT_EPI_W0 && mbar_wait(&bar->acc_full[0], 0, false, p.tile_wait)) {
            tc_fence_after();
            for (int c = 32 * team; c < W * p.subs; c += 64) {
                uint32_t r[32];
                tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (c < W ? c : c - W + GT_W), r);
                tmem_wait();
                uint4 *dst = reinterpret_cast<uint4 *>(smem) + (c / 4) * 128 + 32 * q + lane;
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i * 128] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
            }
            tc_fence_before();
        }
        cluster_sync();
        if (warp >= GT_EPI_W0) {
            float rs = 1.f;
            if constexpr (S8) rs = m0 + lane < pr.M ? p.row_scale[m0 + lane] : 0.f;
            for (int sub = 0; sub < p.subs; ++sub)
#pragma unroll 1
                for (int c = unit_cols * (split + p.splits * team); c < sub_cols; c += 2 * unit_cols * p.splits)
                    unit(pr, &maps.out[g], 0, sub, c, m0, n0, rs);
        }
    }
    if (warp >= GT_EPI_W0 && elect_one()) tma_wait_read<0>();   // the stores have read shared memory; the grid's end completes them
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (CG * p.splits > 1) cluster_sync();
    tc_fence_after();
    if (warp == 2) tmem_dealloc<CG>(tmem, 2 * GT_W);
    if (CG == 2) cluster_sync();   // neither CTA leaves while the other still frees the pair's TMEM
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

// Tiles of box_inner x box_outer elements of a row-major [outer][inner] matrix, swizzled over the tile row's 64 or 128
// bytes.
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
                          box_inner * size == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

constexpr int kMaxDevices = 64;

int current_device(int *dev) {
    QE_CHECK(cudaGetDevice(dev));
    return *dev < kMaxDevices ? MOE_OK : set_error(MOE_ERR_UNSUPPORTED, "device index above 63");
}

template <bool S8, int A_MN, bool B_MN, int EPI, int CG, int NG>
int launch_tc(const Maps<NG> &maps, const TileArgs<NG> &p, int clusters, cudaStream_t st) {
    auto kern = k_gemm_tc<S8, A_MN, B_MN, EPI, CG, NG>;
    static int ready[kMaxDevices] = {};   // this kernel's shared-memory limit is set on the device
    int dev = 0;
    QE_TRY(current_device(&dev));
    if (!__atomic_load_n(&ready[dev], __ATOMIC_RELAXED)) {
        QE_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GT_SMEM));
        __atomic_store_n(&ready[dev], 1, __ATOMIC_RELAXED);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    cfg.gridDim = dim3(clusters * CG * p.splits);
    cfg.blockDim = dim3(GT_NT);
    cfg.dynamicSmemBytes = GT_SMEM;
    cfg.stream = st;
    cfg.attrs = at;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)(CG * p.splits), 1, 1};
    cfg.numAttrs = 2;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    QE_CHECK(cudaLaunchKernelEx(&cfg, kern, maps, p));
    QE_CHECK_LAUNCH("k_gemm_tc");
    return MOE_OK;
}

// Clusters of `size` CTAs that the current device runs at once (looked up once per device and size; racing threads
// store the same number).
int active_clusters(int size, int *out) {
    static int known[kMaxDevices][9] = {};
    int dev = 0;
    QE_TRY(current_device(&dev));
    int n = __atomic_load_n(&known[dev][size], __ATOMIC_RELAXED);
    if (n == 0) {
        auto kern = k_gemm_tc<false, 0, false, EPI_STORE, 1, 1>;   // every variant has this kernel's needs
        QE_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GT_SMEM));
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at[1];
        cfg.gridDim = dim3(size * 1024);
        cfg.blockDim = dim3(GT_NT);
        cfg.dynamicSmemBytes = GT_SMEM;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim = {(unsigned)size, 1, 1};
        QE_CHECK(cudaOccupancyMaxActiveClusters(&n, kern, &cfg));
        if (n < 1) return set_error(MOE_ERR_UNSUPPORTED, "the device cannot hold the product's kernel");
        __atomic_store_n(&known[dev][size], n, __ATOMIC_RELAXED);
    }
    *out = n;
    return MOE_OK;
}

struct Shape {
    int cg, W, subs, splits;
};

// Rows of B that a CTA loads for a sub-tile: whole chunks of 64 where the row index is contiguous.
int b_rows(bool b_mn, int W, int cg) { return b_mn ? (W / cg + 63) / 64 * 64 : W / cg; }

// k steps of all segments.
int k_steps(const GemmArgs &g) {
    const int bk = g.type == DT_S8 ? 128 : 64;
    return (g.K + bk - 1) / bk * g.segs;
}

// The tile shape with the least modelled time, in SM cycles.  A k step takes the longer of its MMAs (2 cycles a column:
// 128 rows x 64 values x 1 column at 4096 multiply-adds a cycle) and its shared-memory traffic (the copies' writes and
// the MMAs' reads, 0.9 cycles a 128-byte row).  Narrow sub-tiles are counted 4 % slower in long launches, where their
// extra traffic costs clock (4096 x 4096 x 8192 over and over: W = 192 231 us, 256 222 us; one at a time 197 and 195).  A
// tile's epilogue takes 2820 cycles and 14 a column (the gate's gradient, with its loads, 56), hidden behind the next
// tile where there is one; a split adds the exchange, 2400 cycles, 32 a column and 266 a CTA of the cluster; a pair 1770
// to start.  Fitted to 6,700 timings of 118 products (24 to 2,200 rows) on B200: the chosen shape is on average 1.4 % and
// at most 15 % slower than the fastest one; outside that range it extrapolates.  It knows neither the kind of
// activation (the gate's epilogue takes longer for the erf form: 8-bit block, 8192 rows of 640 x 7680, 311 us against 215
// with SiLU) nor HBM.
int choose(const GemmArgs &g, Shape *best, long long *time) {
    const int ksteps = k_steps(g);
    long long least = -1;
    for (int cg = g.M > 128 ? 2 : 1; cg >= 1; --cg) {
        const int tiles_m = (g.M + 128 * cg - 1) / (128 * cg), a_rows = g.a_mn ? 128 : std::min(g.M, 128);
        for (int splits = 1; splits <= 8 / cg && splits <= ksteps; splits = splits < 4 ? splits + 1 : 2 * splits) {
            const int kper = (ksteps + splits - 1) / splits;
            if ((splits - 1) * kper >= ksteps) continue;   // no split without a k step
            int room = 0;
            QE_TRY(active_clusters(cg * splits, &room));
            for (int subs = 1; subs <= 2; ++subs) {
                // sub-tile widths: whole 32-column units of both halves (gate), 64 rows where B's row index is contiguous
                const int unit = g.b_mn || g.epi == EPI_GATE ? 64 : 32;
                for (int W = unit; W <= GT_W; W += unit) {
                    const int C = W * subs, out = g.epi == EPI_GATE ? C / 2 : C;
                    const int tiles_n = (g.N + out - 1) / out, waves = (int)(((long long)tiles_m * tiles_n + room - 1) / room);
                    if (splits > 1 && C * 512 > GT_RING) break;    // the partial tile has to fit
                    const int br = b_rows(g.b_mn, W, cg);
                    int step = std::max(2 * C, 9 * (a_rows * (subs + 1) + 2 * subs * br) / 10);
                    if (W < GT_W && waves >= 3) step += step / 25;
                    const long long main = (long long)kper * step, epi = 2820 + C * (g.epi == EPI_GATE_BWD ? 56 : g.epi == EPI_GATE ? 15 : 14);
                    long long t = cg == 2 ? 1770 : 0;
                    if (splits > 1) t += waves * (main + 2400 + 32 * C + 266 * cg * splits + epi / splits);
                    else if (subs == 2) t += waves * (main + epi);
                    else t += (waves - 1) * std::max(main, epi) + main + epi;
                    if (least < 0 || t < least) {
                        least = t;
                        *best = {cg, W, subs, splits};
                    }
                    if (tiles_n == 1) break;   // wider tiles only waste columns
                }
            }
        }
    }
    *time = least;
    return MOE_OK;
}

constexpr long long kLaunchCycles = 7600;   // a launch's own, in the models

// The same for products in one launch (16-bit, B's row index contiguous, stored plainly; pairs, one sub-tile), and the
// order of its tiles.  `big`: the first one's reduction is longer and its tiles go first.  Back to back, a k step takes
// 1.18 times the above and a tile 500 cycles more, or its share of HBM's write rate (1800 cycles and 5 a column).  The
// reduction is not split: narrow matrices with many rows leave most pairs without a tile (backward pass, 8192 rows of
// 256 x 256: 6 tiles of weight gradients, 51 us for a floor of 4).
int choose_group(const GemmArgs *g, int n, bool big, Shape *best, int *rounds, long long *time) {
    long long least = -1;
    int room = 0;
    QE_TRY(active_clusters(2, &room));
    for (int W = big ? 192 : 128; W <= GT_W; W += 64) {   // narrower tiles never measured faster
        const long long step = std::max(2 * W, 18 * (128 + b_rows(true, W, 2)) / 10), epi = 1800 + 5 * W;
        long long t_big = 0, t_small = 0, n_big = 0, n_small = 0;
        for (int i = 0; i < n; ++i) {
            const long long tiles = (long long)((g[i].M + 255) / 256) * ((g[i].N + W - 1) / W);
            const long long t = std::max(k_steps(g[i]) * step * 118 / 100 + 500, epi);
            if (big && i == 0) t_big = t, n_big = tiles;
            else t_small = t, n_small += tiles;
        }
        const long long over = n_big % room, rest = room - over;   // clusters with and without one more big tile
        for (long long r = 0; r <= (over ? n_small / rest : 0); ++r) {
            const long long after = (n_small - r * rest + room - 1) / room;
            const long long t = 1770 + epi + n_big / room * t_big + std::max((over ? t_big : 0) + after * t_small, (r + after) * t_small);
            if (least < 0 || t < least) {
                least = t;
                *best = {2, W, 1, 1};
                *rounds = (int)r;
            }
        }
    }
    *time = least;
    return MOE_OK;
}

template <int CG>
int dispatch(const GemmArgs &g, const Maps<1> &m, const TileArgs<1> &p, int clusters, cudaStream_t st) {
    if (g.type == DT_S8)
        return g.epi == EPI_GATE ? launch_tc<true, 0, false, EPI_GATE, CG, 1>(m, p, clusters, st)
                                 : launch_tc<true, 0, false, EPI_STORE, CG, 1>(m, p, clusters, st);
    if (g.epi == EPI_GATE) return launch_tc<false, 0, false, EPI_GATE, CG, 1>(m, p, clusters, st);
    if (g.epi == EPI_GATE_BWD) return launch_tc<false, 0, true, EPI_GATE_BWD, CG, 1>(m, p, clusters, st);
    if (g.b_mn) return launch_tc<false, 0, true, EPI_STORE, CG, 1>(m, p, clusters, st);
    return launch_tc<false, 0, false, EPI_STORE, CG, 1>(m, p, clusters, st);
}

// Product i of a launch: its sizes and descriptors.
template <int NG>
int set_product(const GemmArgs &g, int i, const Shape &sh, Maps<NG> &m, TileArgs<NG> &p) {
    const int bk = g.type == DT_S8 ? 128 : 64, half = sh.W / 2, tm = 128 * sh.cg;
    const int tn = (g.epi == EPI_GATE ? half : sh.W) * sh.subs;
    Product &pr = p.prod[i];
    pr.M = g.M, pr.N = g.N, pr.segs = g.segs;
    pr.kblocks = (g.K + bk - 1) / bk;
    pr.tiles_m = (g.M + tm - 1) / tm;
    pr.tiles_n = (g.N + tn - 1) / tn;
    pr.start = p.tiles;
    p.tiles += pr.tiles_m * pr.tiles_n;
    pr.a_mn = g.a_mn;
    pr.a_rows = sh.cg == 1 && pr.tiles_m == 1 ? (g.M + 7) / 8 * 8 : 128;   // whole 8-row swizzle groups
    pr.b_ready = g.b_ready;
    pr.out_dtype = g.out_dtype;
    pr.add = g.add;
    const int na = g.segs, nb = g.epi == EPI_GATE ? 2 : g.segs;
    for (int s = 0; s < na; ++s) {
        if (g.a_mn) QE_TRY(encode(&m.a[i][s], g.type, g.a[s], g.M, g.K, g.lda, 64, bk));
        else QE_TRY(encode(&m.a[i][s], g.type, g.a[s], g.K, g.M, g.lda, bk, pr.a_rows));
    }
    for (int s = 0; s < nb; ++s) {
        if (g.b_mn) QE_TRY(encode(&m.b[i][s], g.type, g.b[s], g.N, g.K, g.ldb, 64, bk));
        else QE_TRY(encode(&m.b[i][s], g.type, g.b[s], g.K, g.N, g.ldb, bk, half));
    }
    return encode(&m.out[i], g.out_dtype, g.out, g.N, g.M, g.ldo, g.out_dtype != MOE_FP32 && p.wide ? 2 * GT_UNIT : GT_UNIT, 32);
}

template <int NG>
void set_shape(const GemmArgs &g, const Shape &sh, int ksteps, TileArgs<NG> &p) {
    p.W = sh.W, p.subs = sh.subs, p.splits = sh.splits;
    p.kper = (ksteps + sh.splits - 1) / sh.splits;
    p.tile_wait = tile_wait_cycles(p.kper);
    p.b_bytes = b_rows(g.b_mn, sh.W, sh.cg) * GT_KB;
    p.stage_bytes = GT_A + sh.subs * p.b_bytes;
    p.stages = std::min(GT_MAX_STAGES, GT_RING / p.stage_bytes);
    p.fp16 = g.type == MOE_FP16;
}

}  // namespace

int read_dense_error(int *code) {
    const int zero = 0;
    QE_CHECK(cudaMemcpyFromSymbol(code, g_error, sizeof(int)));
    if (*code) QE_CHECK(cudaMemcpyToSymbol(g_error, &zero, sizeof(int)));
    return MOE_OK;
}

static int launch_shape(const GemmArgs &g, const Shape &sh, cudaStream_t st) {
    Maps<1> m;
    TileArgs<1> p = {};
    p.extra = g.out2 != nullptr;
    p.one_out = g.epi == EPI_STORE || (g.epi == EPI_GATE && !p.extra);
    p.wide = p.one_out && g.out_dtype != MOE_FP32 && (g.epi == EPI_GATE ? sh.W / 2 : sh.W) % (2 * GT_UNIT) == 0;
    QE_TRY(set_product(g, 0, sh, m, p));
    p.products = 1;
    set_shape(g, sh, k_steps(g), p);
    p.act = g.act;
    p.in1 = g.in1, p.in2 = g.in2;
    p.row_scale = g.row_scale, p.col_scale0 = g.col_scale[0], p.col_scale1 = g.col_scale[1], p.bias = g.bias;
    if (g.out1) QE_TRY(encode(&m.out[1], g.type, g.out1, g.N, g.M, g.N, GT_UNIT, 32));
    if (g.out2) QE_TRY(encode(&m.out[2], g.type, g.out2, g.N, g.M, g.N, GT_UNIT, 32));
    int clusters = p.tiles;
    if (p.splits == 1) {
        QE_TRY(active_clusters(sh.cg, &clusters));
        clusters = std::min(clusters, p.tiles);
    }
    return sh.cg == 2 ? dispatch<2>(g, m, p, clusters, st) : dispatch<1>(g, m, p, clusters, st);
}

int launch_gemm(const GemmArgs &g, cudaStream_t st) {
    if (rows_fit(g)) return launch_rows(g, st);
    Shape sh = {};
    long long time = 0;
    QE_TRY(choose(g, &sh, &time));
    return launch_shape(g, sh, st);
}

static int launch_group(const GemmArgs *g, int n, bool big, const Shape &sh, int rounds, cudaStream_t st) {
    Maps<kGroup> m;
    TileArgs<kGroup> p = {};
    int longest = 0;
    p.one_out = 1;
    p.wide = 1;
    for (int i = 0; i < n; ++i)
        if (g[i].out_dtype == MOE_FP32) p.wide = 0;
    for (int i = 0; i < n; ++i) {
        QE_TRY(set_product(g[i], i, sh, m, p));
        longest = std::max(longest, k_steps(g[i]));
        if (big && i == 0) p.big = p.tiles;
    }
    p.products = n;
    p.rounds = rounds;
    set_shape(g[0], sh, longest, p);
    int clusters = 0;
    QE_TRY(active_clusters(sh.cg, &clusters));
    return launch_tc<false, 2, true, EPI_STORE, 2, kGroup>(m, p, std::min(clusters, p.tiles), st);
}

int launch_gradients(const GemmArgs *dx, const GemmArgs *dw, int n_dw, cudaStream_t st) {
    GemmArgs all[kGroup];
    Shape sh = {}, sh_x = {}, sh_w = {};
    int rounds = 0, rounds_w = 0;
    long long t_all = 0, t_x = 0, t_w = 0;
    if (n_dw == 0) return dx ? launch_gemm(*dx, st) : MOE_OK;
    QE_TRY(choose_group(dw, n_dw, false, &sh_w, &rounds_w, &t_w));
    if (dx) {
        all[0] = *dx;
        for (int i = 0; i < n_dw; ++i) all[1 + i] = dw[i];
        QE_TRY(choose_group(all, 1 + n_dw, true, &sh, &rounds, &t_all));
        QE_TRY(choose(*dx, &sh_x, &t_x));
        // one launch where that is modelled at least 7 % faster: its clusters with a tile of dx less take more of the
        // others.  Measured on B200: 1001 rows of 2560 x 5120 102 us (two launches 113), 500 rows of 4000 x 2000 38 (47),
        // 1500 rows of 1024 x 1024 21.6 (24.5); but 600 rows of 1024 x 4096 47 (48), 150 rows of 2048 x 8192 84 (60),
        // where dx alone splits its reduction
        if (100 * (t_all + kLaunchCycles) <= 93 * (t_x + t_w + 2 * kLaunchCycles))
            return launch_group(all, 1 + n_dw, true, sh, rounds, st);
        QE_TRY(launch_shape(*dx, sh_x, st));
    }
    return launch_group(dw, n_dw, false, sh_w, rounds_w, st);
}

}  // namespace qeffn
