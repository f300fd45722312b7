// Entry points of the dense feed-forward operators (declared in include/moe.h): argument checks,
// workspace layout, and the products each call is made of.
#include <initializer_list>

#include "dense.cuh"
#include "moe_internal.cuh"

using namespace qeffn;

namespace {

constexpr int kMaxRows = 1 << 30;   // of either operand: the kernels' row and column indices, a tile past the end, are 32-bit
constexpr int kMaxDim = 65536;   // 127 * 127 * 65536 < 2^31: an 8-bit product's sum stays in int32

int bad(const char *what) { return set_error(MOE_ERR_INVALID_ARG, what); }
int unsupported(const char *what) { return set_error(MOE_ERR_UNSUPPORTED, what); }

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Row distance of a matrix of `cols` columns of `size` bytes (0: contiguous); < 0: not usable.
long long row_dist(long long ld, int cols, int size) {
    if (ld == 0) return cols;
    if (ld < cols || (ld * size) % 16 != 0) return -1;
    return ld;
}

// The device of the call's data becomes current for the call's duration.
struct DeviceScope {
    int before = -1;
    bool changed = false;
    int enter(const void *p) {
        cudaPointerAttributes at;
        QE_CHECK(cudaPointerGetAttributes(&at, p));
        if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
            return bad("the data pointers must be device memory");
        QE_CHECK(cudaGetDevice(&before));
        if (at.device != before) {
            QE_CHECK(cudaSetDevice(at.device));
            changed = true;
        }
        return MOE_OK;
    }
    ~DeviceScope() {
        if (changed) cudaSetDevice(before);
    }
};

// Consecutive 256-byte aligned parts of the workspace.
struct Carve {
    uint8_t *base;
    long long used = 0;
    explicit Carve(void *p) : base((uint8_t *)p) {}
    void *take(long long bytes) {
        void *p = base ? base + used : nullptr;
        used += (bytes + 255) / 256 * 256;
        return p;
    }
};

int check_workspace(const void *ws, long long have, long long need) {
    if (need == 0) return MOE_OK;
    if (!ws || have < need) return bad("workspace: smaller than the *_workspace call names");
    if (!aligned(ws, 256)) return bad("workspace: not 256-byte aligned");
    return MOE_OK;
}

int check_rows(int T) {
    if (T < 0) return bad("T is negative");
    return T <= kMaxRows ? MOE_OK : unsupported("T: at most 2^30");
}

int check_act(int act) {
    return act == MOE_ACT_SILU || act == MOE_ACT_GELU_TANH || act == MOE_ACT_GELU ? MOE_OK : bad("act: not a moe_act");
}

int check_dims(int d, int I, int unit) {
    if (d <= 0 || I <= 0) return bad("d_model and d_ff must be positive");
    if (d % unit != 0 || I % unit != 0 || d > kMaxDim || I > kMaxDim)
        return unsupported("d_model and d_ff must be multiples of 8 (8-bit weights: 16) up to 65536");
    return MOE_OK;
}

int check_ffn(const moe_ffn *f) {
    if (!f) return MOE_ERR_INVALID_ARG;
    if (f->dtype != MOE_BF16 && f->dtype != MOE_FP16) return bad("dtype: MOE_BF16 or MOE_FP16");
    QE_TRY(check_act(f->act));
    return check_dims(f->d_model, f->d_ff, 8);
}

int check_ffn_s8(const moe_ffn_s8 *f) {
    if (!f) return MOE_ERR_INVALID_ARG;
    if (f->dtype != MOE_BF16 && f->dtype != MOE_FP16) return bad("dtype: MOE_BF16 or MOE_FP16");
    QE_TRY(check_act(f->act));
    return check_dims(f->d_model, f->d_ff, 16);
}

struct FfnSpace {
    void *h = nullptr, *dg = nullptr, *du = nullptr;
    long long bytes = 0;
    FfnSpace(const moe_ffn *f, int T, bool backward, void *ws) {
        Carve c(ws);
        const long long n = 2LL * T * f->d_ff;
        h = c.take(n);
        if (backward) {
            dg = c.take(n);
            du = c.take(n);
        }
        bytes = c.used;
    }
};

struct S8Space {
    int8_t *xq, *hq;
    float *xs, *hs, *h;
    long long bytes;
    S8Space(const moe_ffn_s8 *f, int T, void *ws) {
        Carve c(ws);
        xq = (int8_t *)c.take((long long)T * f->d_model);
        xs = (float *)c.take(4LL * T);
        h = (float *)c.take(4LL * T * f->d_ff);
        hq = (int8_t *)c.take((long long)T * f->d_ff);
        hs = (float *)c.take(4LL * T);
        bytes = c.used;
    }
};

bool ptrs16(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p && !aligned(p, 16)) return false;
    return true;
}

}  // namespace

extern "C" {

int moe_ffn_workspace(const moe_ffn *f, int T, int backward, long long *bytes) {
    if (!f || !bytes || T < 0) return MOE_ERR_INVALID_ARG;
    QE_TRY(check_ffn(f));
    *bytes = FfnSpace(f, T, backward != 0, nullptr).bytes;
    return MOE_OK;
}

int moe_ffn_forward(const moe_ffn *f, const void *x, long long ld_x, int T, void *y, long long ld_y, void *gate,
                    void *up, void *workspace, long long workspace_bytes, void *stream) {
    QE_TRY(check_ffn(f));
    QE_TRY(check_rows(T));
    if (T == 0) return MOE_OK;
    if (!x || !y || !f->w_gate || !f->w_up || !f->w_down) return bad("NULL x, y or weights");
    if ((gate == nullptr) != (up == nullptr)) return bad("gate and up: both or neither");
    const int d = f->d_model, I = f->d_ff;
    const long long lx = row_dist(ld_x, d, 2), ly = row_dist(ld_y, d, 2);
    if (lx < 0 || ly < 0) return bad("ld_x, ld_y: at least d_model and a multiple of 16 bytes");
    if (!ptrs16({x, y, f->w_gate, f->w_up, f->w_down, gate, up})) return bad("matrix pointers must be 16-byte aligned");
    FfnSpace w(f, T, false, workspace);
    QE_TRY(check_workspace(workspace, workspace_bytes, w.bytes));
    DeviceScope dev;
    QE_TRY(dev.enter(x));
    cudaStream_t st = (cudaStream_t)stream;

    GemmArgs g;
    g.type = f->dtype;
    g.M = T, g.N = I, g.K = d;
    g.a[0] = x, g.lda = lx;
    g.b[0] = f->w_gate, g.b[1] = f->w_up, g.ldb = d;
    g.epi = EPI_GATE, g.act = f->act;
    g.out = w.h, g.out_dtype = f->dtype, g.ldo = I, g.out1 = gate, g.out2 = up;
    QE_TRY(launch_gemm(g, st));

    GemmArgs y2;
    y2.type = f->dtype;
    y2.M = T, y2.N = d, y2.K = I;
    y2.a[0] = w.h, y2.lda = I;
    y2.b[0] = f->w_down, y2.ldb = I;
    y2.out = y, y2.out_dtype = f->dtype, y2.ldo = ly;
    y2.b_ready = true;
    return launch_gemm(y2, st);
}

int moe_ffn_backward(const moe_ffn *f, const void *x, long long ld_x, const void *gate, const void *up, const void *dy,
                     long long ld_dy, int T, void *dx, long long ld_dx, void *dw_gate, void *dw_up, void *dw_down,
                     int flags, void *workspace, long long workspace_bytes, void *stream) {
    QE_TRY(check_ffn(f));
    QE_TRY(check_rows(T));
    if (flags & ~(MOE_FFN_GRAD_FP32 | MOE_FFN_GRAD_ADD)) return bad("flags: unknown bits");
    if ((flags & MOE_FFN_GRAD_ADD) && !(flags & MOE_FFN_GRAD_FP32)) return bad("MOE_FFN_GRAD_ADD needs MOE_FFN_GRAD_FP32");
    const bool dw = dw_gate || dw_up || dw_down;
    if (dw && (!dw_gate || !dw_up || !dw_down)) return bad("weight gradients: all three or none");
    const int d = f->d_model, I = f->d_ff;
    cudaStream_t st = (cudaStream_t)stream;
    const bool f32 = flags & MOE_FFN_GRAD_FP32, add = flags & MOE_FFN_GRAD_ADD;
    if (!ptrs16({x, gate, up, dy, dx, dw_gate, dw_up, dw_down, f->w_gate, f->w_up, f->w_down}))
        return bad("matrix pointers must be 16-byte aligned");
    if (T == 0) {   // sums over no rows
        if (!dw || add) return MOE_OK;
        DeviceScope dev;
        QE_TRY(dev.enter(dw_gate));
        const size_t bytes = (size_t)d * I * (f32 ? 4 : 2);
        for (void *p : {dw_gate, dw_up, dw_down}) QE_CHECK(cudaMemsetAsync(p, 0, bytes, st));
        return MOE_OK;
    }
    if (!gate || !up || !dy || !f->w_down) return bad("NULL gate, up, dy or w_down");
    if (dx && (!f->w_gate || !f->w_up)) return bad("dx needs w_gate and w_up");
    if (dw && !x) return bad("weight gradients need x");
    const long long lx = row_dist(ld_x, d, 2), ldy = row_dist(ld_dy, d, 2), ldx = row_dist(ld_dx, d, 2);
    if (lx < 0 || ldy < 0 || ldx < 0) return bad("ld_x, ld_dy, ld_dx: at least d_model and a multiple of 16 bytes");
    FfnSpace w(f, T, true, workspace);
    QE_TRY(check_workspace(workspace, workspace_bytes, w.bytes));
    if (!dx && !dw) return MOE_OK;
    DeviceScope dev;
    QE_TRY(dev.enter(dy));

    GemmArgs g;   // dh = dy Wd, and from it dg, du and h
    g.type = f->dtype;
    g.M = T, g.N = I, g.K = d;
    g.a[0] = dy, g.lda = ldy;
    g.b[0] = f->w_down, g.ldb = I, g.b_mn = true;
    g.epi = EPI_GATE_BWD, g.act = f->act;
    g.in1 = gate, g.in2 = up;
    g.out = w.dg, g.out_dtype = f->dtype, g.ldo = I, g.out1 = w.du, g.out2 = dw ? w.h : nullptr;
    QE_TRY(launch_gemm(g, st));

    GemmArgs px;
    px.type = f->dtype;
    px.M = T, px.N = d, px.K = I, px.segs = 2;
    px.a[0] = w.dg, px.a[1] = w.du, px.lda = I;
    px.b[0] = f->w_gate, px.b[1] = f->w_up, px.ldb = d, px.b_mn = true, px.b_ready = true;
    px.out = dx, px.out_dtype = f->dtype, px.ldo = ldx;
    GemmArgs pw[3];   // gate, up, down
    for (int i = 0; i < 3; ++i) {
        GemmArgs &p = pw[i];
        p.type = f->dtype;
        p.K = T;
        p.a_mn = p.b_mn = true;
        p.out_dtype = f32 ? (int)MOE_FP32 : f->dtype;
        p.add = add;
        if (i < 2) {
            p.M = I, p.N = d, p.lda = I, p.ldb = lx, p.ldo = d;
            p.a[0] = i == 0 ? w.dg : w.du, p.b[0] = x, p.b_ready = true;
            p.out = i == 0 ? dw_gate : dw_up;
        } else {
            p.M = d, p.N = I, p.lda = ldy, p.ldb = I, p.ldo = I;
            p.a[0] = dy, p.b[0] = w.h;
            p.out = dw_down;
        }
    }
    return launch_gradients(dx ? &px : nullptr, pw, dw ? 3 : 0, st);
}

int moe_quantize_s8(const void *x, int dtype, long long ld_x, int rows, int cols, int8_t *q, float *scale,
                    void *stream) {
    if (dtype != MOE_BF16 && dtype != MOE_FP16 && dtype != MOE_FP32) return bad("dtype: not a moe_dtype");
    QE_TRY(check_rows(rows));
    if (cols <= 0) return bad("cols must be positive");
    if (cols > kMaxDim) return unsupported("cols: at most 65536");
    if (rows == 0) return MOE_OK;
    if (!x || !q || !scale) return bad("NULL x, q or scale");
    const int size = dtype == MOE_FP32 ? 4 : 2;
    const long long lx = ld_x == 0 ? cols : ld_x;
    if (lx < cols || !aligned(x, size) || !aligned(scale, 4)) return bad("ld_x at least cols, pointers aligned to their type");
    DeviceScope dev;
    QE_TRY(dev.enter(x));
    return launch_quantize_s8(x, dtype, lx, rows, cols, q, scale, (cudaStream_t)stream);
}

int moe_matmul_s8_workspace(int T, int N, int K, long long *bytes) {
    if (!bytes || T < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    *bytes = 0;
    return MOE_OK;
}

int moe_matmul_s8(const int8_t *a, const float *a_scale, int T, const int8_t *w, const float *w_scale, int N, int K,
                  const float *bias, void *y, int y_dtype, long long ld_y, void *workspace, long long workspace_bytes,
                  void *stream) {
    if (y_dtype != MOE_BF16 && y_dtype != MOE_FP16 && y_dtype != MOE_FP32) return bad("y_dtype: not a moe_dtype");
    QE_TRY(check_rows(T));
    if (N <= 0 || K <= 0) return bad("N and K must be positive");
    if (K % 16 != 0 || K > kMaxDim || N % 8 != 0 || N > kMaxRows)
        return unsupported("K: a multiple of 16 up to 65536; N: a multiple of 8 up to 2^30");
    if (T == 0) return MOE_OK;
    if (!a || !a_scale || !w || !w_scale || !y) return bad("NULL a, w, scales or y");
    if (!ptrs16({a, w, y}) || !aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4))
        return bad("matrix pointers must be 16-byte aligned, scales and bias 4-byte");
    const long long ly = row_dist(ld_y, N, y_dtype == MOE_FP32 ? 4 : 2);
    if (ly < 0) return bad("ld_y: at least N and a multiple of 16 bytes");
    long long need = 0;
    QE_TRY(moe_matmul_s8_workspace(T, N, K, &need));
    QE_TRY(check_workspace(workspace, workspace_bytes, need));
    DeviceScope dev;
    QE_TRY(dev.enter(a));
    GemmArgs g;
    g.type = DT_S8;
    g.M = T, g.N = N, g.K = K;
    g.a[0] = a, g.lda = K, g.b[0] = w, g.ldb = K;
    g.row_scale = a_scale, g.col_scale[0] = w_scale, g.bias = bias;
    g.out = y, g.out_dtype = y_dtype, g.ldo = ly;
    return launch_gemm(g, (cudaStream_t)stream);
}

int moe_ffn_s8_workspace(const moe_ffn_s8 *f, int T, long long *bytes) {
    if (!f || !bytes || T < 0) return MOE_ERR_INVALID_ARG;
    QE_TRY(check_ffn_s8(f));
    *bytes = S8Space(f, T, nullptr).bytes;
    return MOE_OK;
}

int moe_ffn_s8_forward(const moe_ffn_s8 *f, const void *x, long long ld_x, int T, void *y, long long ld_y,
                       void *workspace, long long workspace_bytes, void *stream) {
    QE_TRY(check_ffn_s8(f));
    QE_TRY(check_rows(T));
    if (T == 0) return MOE_OK;
    if (!x || !y || !f->w_gate || !f->w_up || !f->w_down || !f->s_gate || !f->s_up || !f->s_down)
        return bad("NULL x, y, weights or scales");
    const int d = f->d_model, I = f->d_ff;
    const long long lx = row_dist(ld_x, d, 2), ly = row_dist(ld_y, d, 2);
    if (lx < 0 || ly < 0) return bad("ld_x, ld_y: at least d_model and a multiple of 16 bytes");
    if (!ptrs16({x, y, f->w_gate, f->w_up, f->w_down}) || !aligned(f->s_gate, 4) || !aligned(f->s_up, 4) ||
        !aligned(f->s_down, 4))
        return bad("matrix pointers must be 16-byte aligned, scales 4-byte");
    S8Space w(f, T, workspace);
    QE_TRY(check_workspace(workspace, workspace_bytes, w.bytes));
    DeviceScope dev;
    QE_TRY(dev.enter(x));
    cudaStream_t st = (cudaStream_t)stream;
    QE_TRY(launch_quantize_s8(x, f->dtype, lx, T, d, w.xq, w.xs, st));
    GemmArgs g;
    g.type = DT_S8;
    g.M = T, g.N = I, g.K = d;
    g.a[0] = w.xq, g.lda = d;
    g.b[0] = f->w_gate, g.b[1] = f->w_up, g.ldb = d;
    g.row_scale = w.xs, g.col_scale[0] = f->s_gate, g.col_scale[1] = f->s_up;
    g.epi = EPI_GATE, g.act = f->act;
    g.out = w.h, g.out_dtype = MOE_FP32, g.ldo = I;
    g.b_ready = true;
    QE_TRY(launch_gemm(g, st));
    QE_TRY(launch_quantize_s8(w.h, MOE_FP32, I, T, I, w.hq, w.hs, st));
    GemmArgs p;
    p.type = DT_S8;
    p.M = T, p.N = d, p.K = I;
    p.a[0] = w.hq, p.lda = I, p.b[0] = f->w_down, p.ldb = I;
    p.row_scale = w.hs, p.col_scale[0] = f->s_down;
    p.out = y, p.out_dtype = f->dtype, p.ldo = ly;
    p.b_ready = true;
    return launch_gemm(p, st);
}

int moe_ffn_get_device_error(int *code) {
    if (!code) return MOE_ERR_INVALID_ARG;
    QE_CHECK(cudaDeviceSynchronize());
    return read_dense_error(code);
}

}  // extern "C"
