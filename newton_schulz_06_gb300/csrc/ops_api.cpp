// C entry points of the operators of a block's training step (last section
// of include/muon.h): argument checks, then the launch.  Every check runs
// before any CUDA call.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "ops_internal.h"
#include "overlap.h"

using namespace muon;

namespace {

constexpr int64_t MAX_ROWS = (int64_t(1) << 31) - 1;
constexpr int64_t MAX_COLS = int64_t(1) << 20;

// One call's error: the code and its message, written to the caller's buffer
// (nothing here allocates, so nothing throws across the C boundary).
struct Err {
    char* buf;
    size_t len;
    Err(char* b, size_t n) : buf(b), len(n) {
        if (buf && len) buf[0] = '\0';
    }
    int fail(int code, const char* fmt, ...) const __attribute__((format(printf, 3, 4))) {
        if (buf && len) {
            va_list ap;
            va_start(ap, fmt);
            std::vsnprintf(buf, len, fmt, ap);
            va_end(ap);
        }
        return code;
    }
    int bad(const char* what) const { return fail(MUON_ERR_INVALID_ARG, "%s", what); }
    int bad(const char* name, const char* what) const {
        return fail(MUON_ERR_INVALID_ARG, "%s %s", name, what);
    }
    int done(cudaError_t e) const {
        return e == cudaSuccess ? MUON_OK : fail(MUON_ERR_CUDA, "%s", cudaGetErrorString(e));
    }
};

bool dtype_ok(int d) { return d == MUON_F32 || d == MUON_BF16; }
bool aligned(const void* p, int dtype) {
    return reinterpret_cast<uintptr_t>(p) % (dtype == MUON_F32 ? 4 : 2) == 0;
}

int check_shape(const Err& err, int64_t rows, int64_t cols) {
    if (rows < 0 || rows > MAX_ROWS) return err.bad("rows out of range");
    if (cols < 1 || cols > MAX_COLS) return err.bad("cols out of range");
    return MUON_OK;
}

// A tensor of rows x cols: its pointer (unless there are no rows), element
// alignment and leading dimension.
int check_tensor(const Err& err, const char* name, const void* p, int dtype, int64_t rows,
                 int64_t cols, int64_t ld, bool read_only) {
    if (rows == 0) return MUON_OK;
    if (!p) return err.bad(name, "is NULL");
    if (!aligned(p, dtype)) return err.bad(name, "is not aligned to its elements");
    if (rows > 1 && ld < cols && !(read_only && ld == 0))
        return err.bad(name, "has too small a leading dimension");
    return MUON_OK;
}

int check_vector(const Err& err, const char* name, const void* p, int dtype) {
    if (p && !aligned(p, dtype))
        return err.bad(name, "is not aligned to its elements");
    return MUON_OK;
}

int check_ckpt(const Err& err, const muon_ckpt8& s, int64_t rows, int64_t cols) {
    if (rows == 0) return MUON_OK;
    if (!s.q || !s.e) return err.bad("saved checkpoint: q or e is NULL");
    if (reinterpret_cast<uintptr_t>(s.q) % 16 != 0)
        return err.bad("saved checkpoint: q is not aligned to 16 bytes");
    if (rows > 1 && (s.ld_q % 32 != 0 || s.ld_q < ops::ceil_div(cols, 32) * 32))
        return err.bad("saved checkpoint: ld_q is no multiple of 32 or too small");
    if (rows > 1 && s.ld_e < ops::ceil_div(cols, 32))
        return err.bad("saved checkpoint: ld_e is too small");
    return MUON_OK;
}

int check_workspace(const Err& err, const void* ws, size_t bytes, size_t need) {
    if (need == 0) return MUON_OK;
    if (!ws || bytes < need)
        return err.fail(MUON_ERR_NO_WORKSPACE,
                        "workspace is NULL or smaller than the %zu bytes this call needs", need);
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
        return err.bad("workspace is not aligned to 256 bytes");
    return MUON_OK;
}

#define RETURN_IF(expr)        \
    do {                       \
        const int rc_ = (expr); \
        if (rc_) return rc_;   \
    } while (0)

int check_norm_grad(const Err& err, const muon_layer_norm_grad_args* a) {
    if (!a) return err.bad("args is NULL");
    RETURN_IF(check_shape(err, a->rows, a->cols));
    if (!dtype_ok(a->x_dtype) || !dtype_ok(a->w_dtype)) return err.bad("unknown element type");
    return MUON_OK;
}

int check_weight_grad(const Err& err, const muon_weight_grad_args* a) {
    if (!a) return err.bad("args is NULL");
    RETURN_IF(check_shape(err, a->rows, a->n));
    RETURN_IF(check_shape(err, a->rows, a->k));
    if (!dtype_ok(a->g_dtype) || !dtype_ok(a->w_dtype)) return err.bad("unknown element type");
    if (a->experts < 1 || a->experts > 65536) return err.bad("experts out of range");
    if (!a->offsets && a->experts != 1) return err.bad("experts without offsets");
    if (a->experts * ops::ceil_div(a->n, 256) * ops::ceil_div(a->k, 256) > (int64_t(1) << 30))
        return err.fail(MUON_ERR_UNSUPPORTED, "more than 2^30 tiles of 256 x 256");
    return MUON_OK;
}

int check_route(const Err& err, int64_t tokens, int64_t experts, int64_t k, int z_dtype) {
    if (!dtype_ok(z_dtype)) return err.bad("unknown element type");
    if (experts < 1 || experts > 1024) return err.bad("experts out of range (1 .. 1024)");
    if (k < 1 || k > 32 || k > experts) return err.bad("k out of range (1 .. min(experts, 32))");
    if (tokens < 0 || tokens > MAX_ROWS / k) return err.bad("tokens out of range");
    return MUON_OK;
}

// Rows, widths, experts and the number of tiles of a gated feed-forward block.
int check_ffn(const Err& err, int64_t rows, int64_t hidden, int64_t inner, int64_t experts,
              const int32_t* offsets, int activation) {
    constexpr int64_t WIDEST = 262144;
    if (rows < 0 || rows > MAX_ROWS - 256) return err.bad("rows out of range");
    if (hidden < 1 || hidden > WIDEST) return err.bad("hidden out of range");
    if (inner < 1 || inner > WIDEST) return err.bad("inner out of range");
    if (experts < 1 || experts > 1024) return err.bad("experts out of range (1 .. 1024)");
    if (!offsets && experts != 1) return err.bad("experts without offsets");
    if (activation < MUON_ACT_SILU || activation > MUON_ACT_GELU_TANH) return err.bad("unknown activation");
    // the kernels count tiles of 32 rows and 128 columns, and of 32 x 256, in 32 bits
    const int64_t wide = hidden > inner ? hidden : inner;
    if ((rows / 32 + experts) * ops::ceil_div(wide, 128) > (int64_t(1) << 30) ||
        experts * ops::ceil_div(wide, 256) * ops::ceil_div(wide, 32) > (int64_t(1) << 28))
        return err.fail(MUON_ERR_UNSUPPORTED, "too many tiles");
    return check_vector(err, "offsets", offsets, MUON_F32);
}

// A matrix an expert, or one for all (stride 0).
int check_weights(const Err& err, const char* name, const void* p, int64_t n, int64_t k, int64_t ld,
                  int64_t experts, int64_t stride) {
    RETURN_IF(check_tensor(err, name, p, MUON_BF16, n, k, ld, true));
    if (experts > 1 && stride < 0) return err.bad(name, "has a negative stride");
    return MUON_OK;
}
int check_grads(const Err& err, const char* name, const void* p, int dtype, int64_t n, int64_t k, int64_t ld,
                int64_t experts, int64_t stride) {
    if (!p) return MUON_OK;
    RETURN_IF(check_tensor(err, name, p, dtype, n, k, ld, false));
    if (experts > 1 && stride < (n > 1 ? (n - 1) * ld : 0) + k) return err.bad(name, "has too small a stride");
    return MUON_OK;
}

// Tensors of a call that may not share memory with what it still reads or with
// each other.
struct Named {
    const char* name;
    ops::Area area;
    Named(const char* what, const void* p, int dtype, int64_t rows, int64_t cols, int64_t ld, int64_t matrices = 1,
          int64_t stride = 0)
        : name(what), area(p, cols * (dtype == MUON_F32 ? 4 : 2)) {
        const int size = dtype == MUON_F32 ? 4 : 2;
        area.axis(rows, ld * size).axis(matrices, stride * size);
        end = area.p + area.span();
        there = p && rows > 0;
    }
    __int128 end;
    bool there;
};
int check_apart(const Err& err, const Named& a, const Named& b) {
    if (a.there && b.there && a.area.p < b.end && b.area.p < a.end && ops::share(a.area, b.area))
        return err.fail(MUON_ERR_INVALID_ARG, "%s and %s share memory", a.name, b.name);
    return MUON_OK;
}
// The same, but for tensors of one address and one layout.
int check_apart_or_same(const Err& err, const Named& a, const Named& b) {
    const bool same = a.area.p == b.area.p && a.area.axes == b.area.axes &&
                      (a.area.axes == 0 || a.area.stride[0] == b.area.stride[0]);
    return same ? MUON_OK : check_apart(err, a, b);
}

int check_forward(const Err& err, const muon_gated_ffn_args* a) {
    if (!a) return err.bad("args is NULL");
    return check_ffn(err, a->rows, a->hidden, a->inner, a->experts, a->offsets, a->activation);
}
int check_backward(const Err& err, const muon_gated_ffn_grad_args* a) {
    if (!a) return err.bad("args is NULL");
    RETURN_IF(check_ffn(err, a->rows, a->hidden, a->inner, a->experts, a->offsets, a->activation));
    if (!dtype_ok(a->g_dtype)) return err.bad("unknown element type");
    return MUON_OK;
}

int check_rotary_tensor(const Err& err, const char* name, const muon_rotary_tensor& t, int dtype,
                        int64_t batch, int64_t seq) {
    if (t.heads < 0 || t.heads > 65536) return err.bad(name, "has heads out of range");
    if (t.heads == 0 || batch == 0 || seq == 0) return MUON_OK;
    if (!t.x || !t.y) return err.bad(name, "is NULL");
    if (!aligned(t.x, dtype) || !aligned(t.y, dtype)) return err.bad(name, "is not aligned to its elements");
    if (t.x_batch < 0 || t.x_seq < 0 || t.x_head < 0 || t.y_batch < 0 || t.y_seq < 0 || t.y_head < 0)
        return err.bad(name, "has a negative stride");
    if ((batch > 1 && t.y_batch == 0) || (seq > 1 && t.y_seq == 0) || (t.heads > 1 && t.y_head == 0))
        return err.bad(name, "is written to places that share memory");
    if (t.x == t.y && ((batch > 1 && t.x_batch != t.y_batch) || (seq > 1 && t.x_seq != t.y_seq) ||
                       (t.heads > 1 && t.x_head != t.y_head)))
        return err.bad(name, "is written in place with other strides");
    return MUON_OK;
}

ops::Area rotary_area(const muon_rotary_args& a, const muon_rotary_tensor& t, bool written, int64_t values) {
    const int64_t size = a.x_dtype == MUON_F32 ? 4 : 2;
    ops::Area area(written ? t.y : t.x, values * size);
    area.axis(t.heads, (written ? t.y_head : t.x_head) * size);
    area.axis(a.seq, (written ? t.y_seq : t.x_seq) * size);
    area.axis(a.batch, (written ? t.y_batch : t.x_batch) * size);
    return area;
}
// Blocks read and write in any order: what one writes no other may read or
// write.
int check_rotary_areas(const Err& err, const muon_rotary_args& a) {
    const muon_rotary_tensor* const t[2] = {&a.q, &a.k};
    const char* const name[2] = {"q", "k"};
    // what follows a head's pairs is copied for both tensors or stays for both
    bool copy = false;
    for (const muon_rotary_tensor* x : t) copy = copy || (x->heads && x->x != x->y);
    const int64_t values = copy ? a.head : 2 * a.pairs;
    for (int i = 0; i < 2; ++i) {
        if (!t[i]->heads) continue;
        const ops::Area y = rotary_area(a, *t[i], true, values);
        if (y.folded()) return err.bad(name[i], "is written to places that share memory");
        if (t[i]->x != t[i]->y && ops::share(y, rotary_area(a, *t[i], false, values)))
            return err.bad(name[i], "is written to memory that it shares with its result");
        const muon_rotary_tensor& other = *t[1 - i];
        if (!other.heads) continue;
        if (ops::share(y, rotary_area(a, other, false, values)) ||
            (i == 0 && ops::share(y, rotary_area(a, other, true, values))))
            return err.bad(name[i], "is written to memory that it shares with the other tensor");
    }
    return MUON_OK;
}

}  // namespace

extern "C" {

MUON_API int muon_ckpt8_pack(const void* x, int x_dtype, int64_t rows, int64_t cols,
                             int64_t ld_x, const muon_ckpt8* saved, void* cuda_stream,
                             char* err_buf, size_t err_len) {
    const Err err{err_buf, err_len};
    if (!saved) return err.bad("saved is NULL");
    RETURN_IF(check_shape(err, rows, cols));
    if (!dtype_ok(x_dtype)) return err.bad("unknown element type");
    RETURN_IF(check_tensor(err, "x", x, x_dtype, rows, cols, ld_x, true));
    RETURN_IF(check_ckpt(err, *saved, rows, cols));
    if (rows == 0) return MUON_OK;
    return err.done(ops::launch_ckpt8_pack(x, x_dtype, rows, cols, ld_x, *saved,
                                           static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_ckpt8_unpack(const muon_ckpt8* saved, int64_t rows, int64_t cols, void* x,
                               int x_dtype, int64_t ld_x, void* cuda_stream, char* err_buf,
                               size_t err_len) {
    const Err err{err_buf, err_len};
    if (!saved) return err.bad("saved is NULL");
    RETURN_IF(check_shape(err, rows, cols));
    if (!dtype_ok(x_dtype)) return err.bad("unknown element type");
    RETURN_IF(check_tensor(err, "x", x, x_dtype, rows, cols, ld_x, false));
    RETURN_IF(check_ckpt(err, *saved, rows, cols));
    if (rows == 0) return MUON_OK;
    return err.done(ops::launch_ckpt8_unpack(*saved, rows, cols, x, x_dtype, ld_x,
                                             static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_layer_norm(const muon_layer_norm_args* a, void* cuda_stream, char* err_buf,
                             size_t err_len) {
    const Err err{err_buf, err_len};
    if (!a) return err.bad("args is NULL");
    RETURN_IF(check_shape(err, a->rows, a->cols));
    if (!dtype_ok(a->x_dtype) || !dtype_ok(a->w_dtype)) return err.bad("unknown element type");
    if (!(a->eps >= 0.f)) return err.bad("eps is negative or not a number");
    RETURN_IF(check_tensor(err, "x", a->x, a->x_dtype, a->rows, a->cols, a->ld_x, true));
    RETURN_IF(check_tensor(err, "y", a->y, a->x_dtype, a->rows, a->cols, a->ld_y, false));
    RETURN_IF(check_vector(err, "weight", a->weight, a->w_dtype));
    RETURN_IF(check_vector(err, "bias", a->bias, a->w_dtype));
    RETURN_IF(check_vector(err, "mean", a->mean, MUON_F32));
    RETURN_IF(check_vector(err, "rstd", a->rstd, MUON_F32));
    if (a->x == a->y && a->rows > 1 && a->ld_x != a->ld_y)
        return err.bad("y is x with another leading dimension");
    if (a->saved.q) RETURN_IF(check_ckpt(err, a->saved, a->rows, a->cols));
    if (a->rows == 0) return MUON_OK;
    return err.done(ops::launch_layer_norm(*a, static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_layer_norm_grad_workspace(const muon_layer_norm_grad_args* a, size_t* bytes) {
    const Err err{nullptr, 0};
    if (!bytes) return MUON_ERR_INVALID_ARG;
    RETURN_IF(check_norm_grad(err, a));
    *bytes = ops::layer_norm_grad_workspace(*a);
    return MUON_OK;
}

MUON_API int muon_layer_norm_grad(const muon_layer_norm_grad_args* a, void* ws, size_t bytes,
                                  void* cuda_stream, char* err_buf, size_t err_len) {
    const Err err{err_buf, err_len};
    RETURN_IF(check_norm_grad(err, a));
    RETURN_IF(check_tensor(err, "dy", a->dy, a->x_dtype, a->rows, a->cols, a->ld_dy, true));
    RETURN_IF(check_tensor(err, "dx", a->dx, a->x_dtype, a->rows, a->cols, a->ld_dx, false));
    RETURN_IF(check_vector(err, "weight", a->weight, a->w_dtype));
    RETURN_IF(check_vector(err, "dweight", a->dweight, a->w_dtype));
    RETURN_IF(check_vector(err, "dbias", a->dbias, a->w_dtype));
    RETURN_IF(check_tensor(err, "rstd", a->rstd, MUON_F32, a->rows, 1, 1, true));
    if (a->saved.q) {
        if (a->x) return err.bad("both x and saved are given");
        RETURN_IF(check_ckpt(err, a->saved, a->rows, a->cols));
    } else {
        RETURN_IF(check_tensor(err, "x", a->x, a->x_dtype, a->rows, a->cols, a->ld_x, true));
        RETURN_IF(check_tensor(err, "mean", a->mean, MUON_F32, a->rows, 1, 1, true));
        if (a->rows && a->x == a->dx) return err.bad("dx must not be x");
    }
    if (a->rows > 1 && a->dy == a->dx && a->ld_dy != a->ld_dx)
        return err.bad("dx is dy with another leading dimension");
    RETURN_IF(check_workspace(err, ws, bytes, ops::layer_norm_grad_workspace(*a)));
    if (a->rows == 0 && !a->dweight && !a->dbias) return MUON_OK;
    return err.done(ops::launch_layer_norm_grad(*a, ws, static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_weight_grad_workspace(const muon_weight_grad_args* a, size_t* bytes) {
    const Err err{nullptr, 0};
    if (!bytes) return MUON_ERR_INVALID_ARG;
    RETURN_IF(check_weight_grad(err, a));
    *bytes = ops::weight_grad_workspace(*a);
    return MUON_OK;
}

MUON_API int muon_weight_grad(const muon_weight_grad_args* a, void* ws, size_t bytes,
                              void* cuda_stream, char* err_buf, size_t err_len) {
    const Err err{err_buf, err_len};
    RETURN_IF(check_weight_grad(err, a));
    RETURN_IF(check_tensor(err, "dy", a->dy, MUON_BF16, a->rows, a->n, a->ld_dy, true));
    RETURN_IF(check_ckpt(err, a->saved, a->rows, a->k));
    RETURN_IF(check_vector(err, "weight", a->weight, a->w_dtype));
    RETURN_IF(check_vector(err, "bias", a->bias, a->w_dtype));
    RETURN_IF(check_vector(err, "offsets", a->offsets, MUON_F32));
    RETURN_IF(check_tensor(err, "g", a->g, a->g_dtype, a->n, a->k, a->ld_g, false));
    if (a->experts > 1) {
        const int64_t last = a->n > 1 ? (a->n - 1) * a->ld_g + a->k : a->k;
        if (a->stride_g < last) return err.bad("stride_g is too small");
    }
    if (a->c) {
        RETURN_IF(check_tensor(err, "c", a->c, a->g_dtype, a->n, a->k, a->ld_c, true));
        if (a->experts > 1 && a->stride_c < 0) return err.bad("stride_c is negative");
        if (a->c == a->g && ((a->n > 1 && a->ld_c != a->ld_g) ||
                             (a->experts > 1 && a->stride_c != a->stride_g)))
            return err.bad("c is g with other strides");
    }
    RETURN_IF(check_workspace(err, ws, bytes, ops::weight_grad_workspace(*a)));
    return err.done(ops::launch_weight_grad(*a, ws, static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_route_workspace(const muon_route_args* a, size_t* bytes) {
    const Err err{nullptr, 0};
    if (!a || !bytes) return MUON_ERR_INVALID_ARG;
    RETURN_IF(check_route(err, a->tokens, a->experts, a->k, a->z_dtype));
    *bytes = ops::route_workspace(*a);
    return MUON_OK;
}

MUON_API int muon_route(const muon_route_args* a, void* ws, size_t bytes, void* cuda_stream,
                        char* err_buf, size_t err_len) {
    const Err err{err_buf, err_len};
    if (!a) return err.bad("args is NULL");
    RETURN_IF(check_route(err, a->tokens, a->experts, a->k, a->z_dtype));
    RETURN_IF(check_tensor(err, "logits", a->logits, a->z_dtype, a->tokens, a->experts, a->ld_z,
                           true));
    RETURN_IF(check_tensor(err, "indices", a->indices, MUON_F32, a->tokens, a->k, a->k, false));
    RETURN_IF(check_tensor(err, "weights", a->weights, MUON_F32, a->tokens, a->k, a->k, false));
    RETURN_IF(check_tensor(err, "counts", a->counts, MUON_F32, 1, 1, 1, false));
    RETURN_IF(check_tensor(err, "offsets", a->offsets, MUON_F32, 1, 1, 1, false));
    RETURN_IF(check_tensor(err, "loss", a->loss, MUON_F32, 1, 1, 1, false));
    RETURN_IF(check_tensor(err, "kept", a->kept, MUON_F32, 1, 1, 1, false));
    RETURN_IF(check_workspace(err, ws, bytes, ops::route_workspace(*a)));
    return err.done(ops::launch_route(*a, ws, static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_route_grad(const muon_route_grad_args* a, void* cuda_stream, char* err_buf,
                             size_t err_len) {
    const Err err{err_buf, err_len};
    if (!a) return err.bad("args is NULL");
    RETURN_IF(check_route(err, a->tokens, a->experts, a->k, a->z_dtype));
    RETURN_IF(check_tensor(err, "logits", a->logits, a->z_dtype, a->tokens, a->experts, a->ld_z,
                           true));
    RETURN_IF(check_tensor(err, "dlogits", a->dlogits, a->z_dtype, a->tokens, a->experts,
                           a->ld_dz, false));
    RETURN_IF(check_tensor(err, "indices", a->indices, MUON_F32, a->tokens, a->k, a->k, true));
    RETURN_IF(check_tensor(err, "weights", a->weights, MUON_F32, a->tokens, a->k, a->k, true));
    RETURN_IF(check_tensor(err, "counts", a->counts, MUON_F32, 1, 1, 1, true));
    RETURN_IF(check_tensor(err, "kept", a->kept, MUON_F32, 1, 1, 1, true));
    RETURN_IF(check_vector(err, "dloss", a->dloss, MUON_F32));
    if (a->dweights)
        RETURN_IF(check_tensor(err, "dweights", a->dweights, MUON_F32, a->tokens, a->k, a->ld_dw,
                               true));
    if (a->tokens > 1 && a->logits == a->dlogits && a->ld_z != a->ld_dz)
        return err.bad("dlogits is logits with another leading dimension");
    if (a->tokens == 0) return MUON_OK;
    return err.done(ops::launch_route_grad(*a, static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_gated_ffn_workspace(const muon_gated_ffn_args* a, size_t* bytes) {
    const Err err{nullptr, 0};
    if (!bytes) return MUON_ERR_INVALID_ARG;
    RETURN_IF(check_forward(err, a));
    *bytes = ops::gated_ffn_workspace(*a);
    return MUON_OK;
}

MUON_API int muon_gated_ffn(const muon_gated_ffn_args* a, void* ws, size_t bytes, void* cuda_stream,
                            char* err_buf, size_t err_len) {
    const Err err{err_buf, err_len};
    RETURN_IF(check_forward(err, a));
    RETURN_IF(check_tensor(err, "x", a->x, MUON_BF16, a->rows, a->hidden, a->ld_x, true));
    RETURN_IF(check_weights(err, "w_gate", a->w_gate, a->inner, a->hidden, a->ld_gate, a->experts, a->stride_gate));
    RETURN_IF(check_weights(err, "w_up", a->w_up, a->inner, a->hidden, a->ld_up, a->experts, a->stride_up));
    RETURN_IF(check_weights(err, "w_down", a->w_down, a->hidden, a->inner, a->ld_down, a->experts, a->stride_down));
    RETURN_IF(check_tensor(err, "y", a->y, MUON_BF16, a->rows, a->hidden, a->ld_y, false));
    if (!a->gate != !a->up) return err.bad("one of gate and up without the other");
    if (a->gate) {
        RETURN_IF(check_tensor(err, "gate", a->gate, MUON_BF16, a->rows, a->inner, a->ld_kept, false));
        RETURN_IF(check_tensor(err, "up", a->up, MUON_BF16, a->rows, a->inner, a->ld_kept, false));
    }
    RETURN_IF(check_workspace(err, ws, bytes, ops::gated_ffn_workspace(*a)));
    const Named x("x", a->x, MUON_BF16, a->rows, a->hidden, a->ld_x);
    const Named y("y", a->y, MUON_BF16, a->rows, a->hidden, a->ld_y);
    const Named gate("gate", a->gate, MUON_BF16, a->rows, a->inner, a->ld_kept);
    const Named up("up", a->up, MUON_BF16, a->rows, a->inner, a->ld_kept);
    const Named weights[3] = {
        {"w_gate", a->w_gate, MUON_BF16, a->inner, a->hidden, a->ld_gate, a->experts, a->stride_gate},
        {"w_up", a->w_up, MUON_BF16, a->inner, a->hidden, a->ld_up, a->experts, a->stride_up},
        {"w_down", a->w_down, MUON_BF16, a->hidden, a->inner, a->ld_down, a->experts, a->stride_down}};
    for (const Named* out : {&y, &gate, &up})
        for (const Named& w : weights) RETURN_IF(check_apart(err, *out, w));
    RETURN_IF(check_apart(err, gate, up));
    for (const Named* kept : {&gate, &up}) {
        RETURN_IF(check_apart(err, *kept, x));
        RETURN_IF(check_apart(err, *kept, y));
    }
    return err.done(ops::launch_gated_ffn(*a, ws, static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_gated_ffn_grad_workspace(const muon_gated_ffn_grad_args* a, size_t* bytes) {
    const Err err{nullptr, 0};
    if (!bytes) return MUON_ERR_INVALID_ARG;
    RETURN_IF(check_backward(err, a));
    *bytes = ops::gated_ffn_grad_workspace(*a);
    return MUON_OK;
}

MUON_API int muon_gated_ffn_grad(const muon_gated_ffn_grad_args* a, void* ws, size_t bytes, void* cuda_stream,
                                 char* err_buf, size_t err_len) {
    const Err err{err_buf, err_len};
    RETURN_IF(check_backward(err, a));
    const bool x_grads = a->dw_gate || a->dw_up;
    RETURN_IF(check_tensor(err, "dy", a->dy, MUON_BF16, a->rows, a->hidden, a->ld_dy, true));
    if (x_grads) RETURN_IF(check_tensor(err, "x", a->x, MUON_BF16, a->rows, a->hidden, a->ld_x, true));
    RETURN_IF(check_tensor(err, "gate", a->gate, MUON_BF16, a->rows, a->inner, a->ld_kept, true));
    RETURN_IF(check_tensor(err, "up", a->up, MUON_BF16, a->rows, a->inner, a->ld_kept, true));
    if (a->dx) {
        RETURN_IF(check_weights(err, "w_gate", a->w_gate, a->inner, a->hidden, a->ld_gate, a->experts,
                                a->stride_gate));
        RETURN_IF(check_weights(err, "w_up", a->w_up, a->inner, a->hidden, a->ld_up, a->experts, a->stride_up));
        RETURN_IF(check_tensor(err, "dx", a->dx, MUON_BF16, a->rows, a->hidden, a->ld_dx, false));
    }
    RETURN_IF(check_weights(err, "w_down", a->w_down, a->hidden, a->inner, a->ld_down, a->experts, a->stride_down));
    RETURN_IF(check_grads(err, "dw_gate", a->dw_gate, a->g_dtype, a->inner, a->hidden, a->ld_dw_gate, a->experts,
                          a->stride_dw_gate));
    RETURN_IF(check_grads(err, "dw_up", a->dw_up, a->g_dtype, a->inner, a->hidden, a->ld_dw_up, a->experts,
                          a->stride_dw_up));
    RETURN_IF(check_grads(err, "dw_down", a->dw_down, a->g_dtype, a->hidden, a->inner, a->ld_dw_down, a->experts,
                          a->stride_dw_down));
    // dy and x are read after dx is written
    if (a->rows && a->dx && ((a->dw_down && a->dx == a->dy) || (x_grads && a->dx == a->x)))
        return err.bad("dx is dy or x, which a weight's gradient reads");
    void* const made[3] = {a->dgate, a->dup, a->h};
    for (const void* m : made)
        if (m) RETURN_IF(check_tensor(err, "dgate, dup or h", m, MUON_BF16, a->rows, a->inner, a->ld_d, false));
    RETURN_IF(check_workspace(err, ws, bytes, ops::gated_ffn_grad_workspace(*a)));
    const int g = a->g_dtype;
    const Named dy("dy", a->dy, MUON_BF16, a->rows, a->hidden, a->ld_dy);
    const Named x("x", x_grads ? a->x : nullptr, MUON_BF16, a->rows, a->hidden, a->ld_x);
    const Named dx("dx", a->dx, MUON_BF16, a->rows, a->hidden, a->ld_dx);
    const Named kept[2] = {{"gate", a->gate, MUON_BF16, a->rows, a->inner, a->ld_kept},
                           {"up", a->up, MUON_BF16, a->rows, a->inner, a->ld_kept}};
    const Named on_way[3] = {{"dgate", a->dgate, MUON_BF16, a->rows, a->inner, a->ld_d},
                             {"dup", a->dup, MUON_BF16, a->rows, a->inner, a->ld_d},
                             {"h", a->h, MUON_BF16, a->rows, a->inner, a->ld_d}};
    const Named weights[3] = {
        {"w_gate", a->dx ? a->w_gate : nullptr, MUON_BF16, a->inner, a->hidden, a->ld_gate, a->experts, a->stride_gate},
        {"w_up", a->dx ? a->w_up : nullptr, MUON_BF16, a->inner, a->hidden, a->ld_up, a->experts, a->stride_up},
        {"w_down", a->w_down, MUON_BF16, a->hidden, a->inner, a->ld_down, a->experts, a->stride_down}};
    const Named grads[3] = {
        {"dw_gate", a->dw_gate, g, a->inner, a->hidden, a->ld_dw_gate, a->experts, a->stride_dw_gate},
        {"dw_up", a->dw_up, g, a->inner, a->hidden, a->ld_dw_up, a->experts, a->stride_dw_up},
        {"dw_down", a->dw_down, g, a->hidden, a->inner, a->ld_dw_down, a->experts, a->stride_dw_down}};
    for (int i = 0; i < 3; ++i) {
        // what DHIDDEN writes, each value in the place of its g or u at most
        RETURN_IF(check_apart(err, on_way[i], dy));
        for (const Named& k : kept) RETURN_IF(check_apart_or_same(err, on_way[i], k));
        for (const Named& w : weights) RETURN_IF(check_apart(err, on_way[i], w));
        RETURN_IF(check_apart(err, on_way[i], x));
        RETURN_IF(check_apart(err, on_way[i], dx));
        for (int j = 0; j < 3; ++j) {
            if (j > i) RETURN_IF(check_apart(err, on_way[i], on_way[j]));
            RETURN_IF(check_apart(err, on_way[i], grads[j]));
        }
        // what the weights' gradients read
        if (a->dw_down) RETURN_IF(check_apart(err, grads[i], dy));
        RETURN_IF(check_apart(err, grads[i], x));
        RETURN_IF(check_apart(err, grads[i], dx));
        for (int j = i + 1; j < 3; ++j) RETURN_IF(check_apart(err, grads[i], grads[j]));
    }
    for (int i = 0; i < 2; ++i) RETURN_IF(check_apart(err, dx, weights[i]));
    if (a->dw_down) RETURN_IF(check_apart(err, dx, dy));
    RETURN_IF(check_apart(err, dx, x));
    return err.done(ops::launch_gated_ffn_grad(*a, ws, static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_rotary(const muon_rotary_args* a, void* cuda_stream, char* err_buf, size_t err_len) {
    const Err err{err_buf, err_len};
    if (!a) return err.bad("args is NULL");
    if (!dtype_ok(a->x_dtype)) return err.bad("unknown element type");
    if (a->layout != MUON_ROTARY_HALF && a->layout != MUON_ROTARY_INTERLEAVED) return err.bad("unknown layout");
    if (a->pairs < 1 || a->pairs > 256) return err.bad("pairs out of range (1 .. 256)");
    if (a->head < 2 * a->pairs || a->head > 65536) return err.bad("head out of range (2 * pairs .. 65536)");
    if (a->batch < 0 || a->seq < 0 || a->batch > MAX_ROWS || a->seq > MAX_ROWS ||
        a->batch * a->seq > MAX_ROWS)
        return err.bad("batch or seq out of range");
    if (!std::isfinite(a->scale)) return err.bad("scale is not finite");
    if (!a->turns) return err.bad("turns is NULL");
    RETURN_IF(check_rotary_tensor(err, "q", a->q, a->x_dtype, a->batch, a->seq));
    RETURN_IF(check_rotary_tensor(err, "k", a->k, a->x_dtype, a->batch, a->seq));
    if (a->positions) {
        if (a->stride_positions < 0) return err.bad("positions has a negative stride");
        if (reinterpret_cast<uintptr_t>(a->positions) % (a->positions_64 ? 8 : 4) != 0)
            return err.bad("positions is not aligned to its elements");
    }
    if ((a->q.heads + a->k.heads) * a->head > (int64_t(1) << 28)) return err.bad("heads out of range");
    if (a->batch * a->seq == 0 || a->q.heads + a->k.heads == 0) return MUON_OK;
    RETURN_IF(check_rotary_areas(err, *a));
    return err.done(ops::launch_rotary(*a, static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_rotary_frequencies(int64_t pairs, double base, int scaling, double factor, double original,
                                     double fast, double slow, uint64_t* turns, float* scale, char* err_buf,
                                     size_t err_len) {
    const Err err{err_buf, err_len};
    if (!turns || !scale) return err.bad("turns or scale is NULL");
    if (pairs < 1 || pairs > 256) return err.bad("pairs out of range (1 .. 256)");
    if (!(base > 1.0) || !std::isfinite(base)) return err.bad("base is not above 1");
    if (scaling < MUON_ROTARY_PLAIN || scaling > MUON_ROTARY_YARN) return err.bad("unknown scaling");
    if (!(factor >= 1.0) || !std::isfinite(factor)) return err.bad("factor is below 1");
    if (scaling == MUON_ROTARY_NTK) {
        if (pairs < 2) return err.bad("pairs must be 2 or more with this scaling");
        base *= std::pow(factor, double(pairs) / double(pairs - 1));
    }
    constexpr double TURN = 6.283185307179586476925;
    double low = 0.0, high = 0.0;
    if (scaling == MUON_ROTARY_YARN) {
        if (!(original >= 1.0) || !std::isfinite(original)) return err.bad("original is below 1");
        if (!(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)) return err.bad("need 0 < slow < fast");
        // the pair that turns so many times in the original positions
        const auto place = [&](double n) { return double(pairs) * std::log(original / (n * TURN)) / std::log(base); };
        low = std::fmax(std::floor(place(fast)), 0.0);
        high = std::fmin(std::ceil(place(slow)), double(2 * pairs - 1));
    }
    for (int64_t i = 0; i < pairs; ++i) {
        double f = std::pow(base, -double(i) / double(pairs));
        if (scaling == MUON_ROTARY_LINEAR) f /= factor;
        if (scaling == MUON_ROTARY_YARN) {
            const double r = std::fmin(std::fmax((double(i) - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            f = f / factor * r + f * (1.0 - r);
        }
        turns[i] = static_cast<uint64_t>(std::ldexp(f / TURN, 64));
    }
    *scale = scaling == MUON_ROTARY_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
    return MUON_OK;
}

MUON_API int muon_dropout(const muon_dropout_args* a, void* cuda_stream, char* err_buf, size_t err_len) {
    const Err err{err_buf, err_len};
    if (!a) return err.bad("args is NULL");
    RETURN_IF(check_shape(err, a->rows, a->cols));
    if (!dtype_ok(a->x_dtype)) return err.bad("unknown element type");
    if (!(a->p >= 0.0 && a->p <= 1.0)) return err.bad("p out of range (0 .. 1)");
    RETURN_IF(check_tensor(err, "x", a->x, a->x_dtype, a->rows, a->cols, a->ld_x, true));
    if (a->residual)
        RETURN_IF(check_tensor(err, "residual", a->residual, a->x_dtype, a->rows, a->cols, a->ld_r, true));
    RETURN_IF(check_tensor(err, "y", a->y, a->x_dtype, a->rows, a->cols, a->ld_y, false));
    if (reinterpret_cast<uintptr_t>(a->counter) % 8 != 0) return err.bad("counter is not aligned to its elements");
    if (a->rows > 1 && a->x == a->y && a->ld_x != a->ld_y) return err.bad("y is x with another leading dimension");
    if (a->rows > 1 && a->residual == a->y && a->ld_r != a->ld_y)
        return err.bad("y is residual with another leading dimension");
    if (a->rows == 0) return MUON_OK;
    const Named y("y", a->y, a->x_dtype, a->rows, a->cols, a->ld_y);
    RETURN_IF(check_apart_or_same(err, y, Named("x", a->x, a->x_dtype, a->rows, a->cols, a->ld_x)));
    RETURN_IF(check_apart_or_same(err, y, Named("residual", a->residual, a->x_dtype, a->rows, a->cols, a->ld_r)));
    return err.done(ops::launch_dropout(*a, static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_ops_sync(void* cuda_stream, char* err_buf, size_t err_len) {
    const Err err{err_buf, err_len};
    int code = 0;
    const cudaError_t e = ops::ops_status(static_cast<cudaStream_t>(cuda_stream), &code);
    if (e != cudaSuccess) return err.done(e);
    if (code)
        return err.fail(MUON_ERR_TIMEOUT, "a bounded wait of an operator ran out on the GPU");
    return MUON_OK;
}

MUON_API int muon_debug_ops_wait_timeout(int limit_ms, void* cuda_stream, char* err_buf,
                                         size_t err_len) {
    const Err err{err_buf, err_len};
    if (limit_ms < 1 || limit_ms > 10000) return err.bad("need 1 <= limit_ms <= 10000");
    return err.done(ops::launch_ring_timeout(static_cast<unsigned long long>(limit_ms) * 1000000ull,
                                             static_cast<cudaStream_t>(cuda_stream)));
}

MUON_API int muon_debug_ffn_wait_timeout(int limit_ms, void* cuda_stream, char* err_buf,
                                         size_t err_len) {
    const Err err{err_buf, err_len};
    if (limit_ms < 1 || limit_ms > 10000) return err.bad("need 1 <= limit_ms <= 10000");
    return err.done(ops::launch_ffn_timeout(static_cast<unsigned long long>(limit_ms) * 1000000ull,
                                            static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
