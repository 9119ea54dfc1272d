// C entry points of the operators of a block's training step (last section
// of include/muon.h): argument checks, then the launch.  Every check runs
// before any CUDA call.
#include <cstdarg>
#include <cstdio>

#include "ops_internal.h"

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

}  // extern "C"
