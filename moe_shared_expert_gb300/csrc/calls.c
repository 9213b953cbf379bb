/* Python entry of the routed-expert calls, the sorted rows and the 8-bit integer products: arguments by vectorcall into the
 * C ABI's functions (whose addresses the package hands over), a fifth of what ctypes takes for as many arguments.  Integers
 * and None (a null pointer) only; every check of the arguments is the library's. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "mse.h"

static __typeof__(&moe_route) f_route;
static __typeof__(&fp8_block_linear) f_linear;
static __typeof__(&fp8_block_matmul) f_matmul;
static __typeof__(&moe_experts_forward) f_experts;

static __typeof__(&moe_sort) f_sort;
static __typeof__(&moe_unsort) f_unsort;
static __typeof__(&moe_unsort_backward) f_unsort_backward;
static __typeof__(&int8_quantise) f_int8_quantise;
static __typeof__(&int8_matmul) f_int8_matmul;
static __typeof__(&int8_grouped_matmul) f_int8_grouped;
static __typeof__(&int8_linear) f_int8_linear;

static long long integer(PyObject *o) { return o == Py_None ? 0 : PyLong_AsLongLong(o); }
static int small(PyObject *o) {
    const long long v = integer(o);
    if (v != (int)v && !PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "number beyond an int");
    return (int)v;
}
static void *address(PyObject *o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }

static int take(Py_ssize_t n, Py_ssize_t want, const char *name) {
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, got %zd", name, want, n);
    return 0;
}

#define I(k) integer(a[k])
#define S(k) small(a[k])
#define P(k) address(a[k])
#define READY(f, name)                                              \
    if (!(f)) {                                                     \
        PyErr_SetString(PyExc_RuntimeError, name ": bind() first"); \
        return NULL;                                                \
    }

/* Arguments are converted before the call, so that a bad one calls nothing.  The interpreter's lock is let go over the
 * call, as ctypes does: a launch waits where the queue of launches is full, perhaps for a host function in Python. */
#define CALL(expression)                  \
    if (PyErr_Occurred()) return NULL;    \
    mse_status status;                    \
    Py_BEGIN_ALLOW_THREADS                \
    status = (expression);                \
    Py_END_ALLOW_THREADS                  \
    return PyLong_FromLong((long)status);

static PyObject *route(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_route, "moe_route")
    if (!take(n, 17, "moe_route")) return NULL;
    const void *logits = P(0);
    const int dtype = S(1);
    const long long T = I(2), E = I(3), ld = I(4);
    const float *bias = P(5);
    const int scoring = S(6), groups = S(7), kept = S(8), top = S(9), k = S(10), norm = S(11);
    const double scale = PyFloat_AsDouble(a[12]);
    int32_t *ids = P(13);
    float *weights = P(14);
    const long long cap = I(15);
    void *stream = P(16);
    CALL(f_route(logits, (mse_dtype)dtype, T, E, ld, bias, (mse_score)scoring, groups, kept, top, k, norm,
                 (float)scale, ids, weights, cap, stream))
}

static PyObject *matmul(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_matmul, "fp8_block_matmul")
    if (!take(n, 13, "fp8_block_matmul")) return NULL;
    const uint8_t *xq = P(0), *wq = P(3);
    const long long ldx = I(1), ldw = I(4), T = I(6), N = I(7), K = I(8), cap = I(11);
    const int dtype = S(10);
    const float *xs = P(2), *ws = P(5);
    void *out = P(9), *stream = P(12);
    CALL(f_matmul(xq, ldx, xs, wq, ldw, ws, T, N, K, out, (mse_dtype)dtype, cap, stream))
}

static PyObject *linear(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_linear, "fp8_block_linear")
    if (!take(n, 14, "fp8_block_linear")) return NULL;
    const mse_bf16 *x = P(0);
    const uint8_t *wq = P(2);
    const float *ws = P(4);
    const long long ldx = I(1), ldw = I(3), T = I(5), N = I(6), K = I(7), cap = I(10), bytes = I(12);
    const int dtype = S(9);
    void *y = P(8), *workspace = P(11), *stream = P(13);
    CALL(f_linear(x, ldx, wq, ldw, ws, T, N, K, y, (mse_dtype)dtype, cap, workspace, (size_t)bytes, stream))
}

static PyObject *experts(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_experts, "moe_experts_forward")
    if (!take(n, 21, "moe_experts_forward")) return NULL;
    const mse_bf16 *x = P(0), *shared = P(15);
    const int32_t *ids = P(3);
    const float *weights = P(4), *s_gate_up = P(8), *s_down = P(11);
    const uint8_t *w_gate_up = P(6), *w_down = P(9);
    mse_bf16 *y = P(16);
    void *workspace = P(18), *stream = P(20);
    const long long T = I(1), H = I(2), ld_gate_up = I(7), ld_down = I(10), E = I(12), inter = I(13),
                    first = I(14), cap = I(17), bytes = I(19);
    const int k = S(5);
    CALL(f_experts(x, T, H, ids, weights, k, w_gate_up, ld_gate_up, s_gate_up, w_down, ld_down, s_down, E,
                   inter, first, shared, y, cap, workspace, (size_t)bytes, stream))
}

static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (!take(n, 4, "bind")) return NULL;
    void *const p[4] = {P(0), P(1), P(2), P(3)};
    if (PyErr_Occurred()) return NULL;
    f_route = (__typeof__(&moe_route))p[0];
    f_linear = (__typeof__(&fp8_block_linear))p[1];
    f_matmul = (__typeof__(&fp8_block_matmul))p[2];
    f_experts = (__typeof__(&moe_experts_forward))p[3];
    Py_RETURN_NONE;
}

static PyObject *sort(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_sort, "moe_sort")
    if (!take(n, 19, "moe_sort")) return NULL;
    const void *x = P(0);
    const int bytes = S(1), k = S(6);
    const long long T = I(2), H = I(3), ldx = I(4), E = I(7), first = I(8), ldr = I(11), cap = I(12), space = I(17);
    const int32_t *ids = P(5);
    const float *scales = P(9);
    void *rows = P(10), *workspace = P(16), *stream = P(18);
    float *row_scales = P(13);
    int32_t *place = P(14), *offsets = P(15);
    CALL(f_sort(x, bytes, T, H, ldx, ids, k, E, first, scales, rows, ldr, cap, row_scales, place, offsets, workspace,
                (size_t)space, stream))
}

static PyObject *unsort(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_unsort, "moe_unsort")
    if (!take(n, 14, "moe_unsort")) return NULL;
    const void *rows = P(0), *base = P(9);
    const int rows_dtype = S(1), k = S(8), y_dtype = S(11);
    const long long n_rows = I(2), ldr = I(3), T = I(6), H = I(7), cap = I(12);
    const int32_t *place = P(4);
    const float *weights = P(5);
    void *y = P(10), *stream = P(13);
    CALL(f_unsort(rows, (mse_dtype)rows_dtype, n_rows, ldr, place, weights, T, H, k, base, y, (mse_dtype)y_dtype, cap,
                  stream))
}

static PyObject *unsort_backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_unsort_backward, "moe_unsort_backward")
    if (!take(n, 16, "moe_unsort_backward")) return NULL;
    const void *dy = P(0), *rows = P(4);
    const int dy_dtype = S(1), rows_dtype = S(5), k = S(10);
    const int32_t *place = P(2);
    const float *weights = P(3);
    const long long ldr = I(6), n_rows = I(7), T = I(8), H = I(9), ldd = I(12), cap = I(13);
    void *drows = P(11), *stream = P(15);
    float *dweights = P(14);
    CALL(f_unsort_backward(dy, (mse_dtype)dy_dtype, place, weights, rows, (mse_dtype)rows_dtype, ldr, n_rows, T, H, k,
                           drows, ldd, cap, dweights, stream))
}

static PyObject *quantise(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_int8_quantise, "int8_quantise")
    if (!take(n, 12, "int8_quantise")) return NULL;
    const void *x = P(0);
    const int dtype = S(1), swiglu = S(5);
    const long long rows = I(2), K = I(3), ldx = I(4), ldq = I(8), cap = I(9);
    const int32_t *last = P(6);
    int8_t *q = P(7);
    float *scales = P(10);
    void *stream = P(11);
    CALL(f_int8_quantise(x, (mse_dtype)dtype, rows, K, ldx, swiglu, last, q, ldq, cap, scales, stream))
}

static PyObject *matmul8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_int8_matmul, "int8_matmul")
    if (!take(n, 15, "int8_matmul")) return NULL;
    const int8_t *xq = P(0), *wq = P(3);
    const float *xs = P(2), *ws = P(5);
    const long long ldx = I(1), ldw = I(4), T = I(6), N = I(7), K = I(8), cap = I(11), bytes = I(13);
    const int dtype = S(10);
    void *out = P(9), *workspace = P(12), *stream = P(14);
    CALL(f_int8_matmul(xq, ldx, xs, wq, ldw, ws, T, N, K, out, (mse_dtype)dtype, cap, workspace, (size_t)bytes, stream))
}

static PyObject *grouped8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_int8_grouped, "int8_grouped_matmul")
    if (!take(n, 17, "int8_grouped_matmul")) return NULL;
    const int8_t *xq = P(0), *wq = P(5);
    const float *xs = P(2), *ws = P(7);
    const int32_t *offsets = P(3);
    const long long ldx = I(1), groups = I(4), ldw = I(6), T = I(8), N = I(9), K = I(10), cap = I(13), bytes = I(15);
    const int dtype = S(12);
    void *out = P(11), *workspace = P(14), *stream = P(16);
    CALL(f_int8_grouped(xq, ldx, xs, offsets, groups, wq, ldw, ws, T, N, K, out, (mse_dtype)dtype, cap, workspace,
                        (size_t)bytes, stream))
}

static PyObject *linear8(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    READY(f_int8_linear, "int8_linear")
    if (!take(n, 15, "int8_linear")) return NULL;
    const void *x = P(0);
    const int x_dtype = S(1), y_dtype = S(10);
    const int8_t *wq = P(3);
    const float *ws = P(5);
    const long long ldx = I(2), ldw = I(4), T = I(6), N = I(7), K = I(8), cap = I(11), bytes = I(13);
    void *y = P(9), *workspace = P(12), *stream = P(14);
    CALL(f_int8_linear(x, (mse_dtype)x_dtype, ldx, wq, ldw, ws, T, N, K, y, (mse_dtype)y_dtype, cap, workspace,
                       (size_t)bytes, stream))
}

static PyObject *bind_rows(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (!take(n, 7, "bind_rows")) return NULL;
    void *const p[7] = {P(0), P(1), P(2), P(3), P(4), P(5), P(6)};
    if (PyErr_Occurred()) return NULL;
    f_sort = (__typeof__(&moe_sort))p[0];
    f_unsort = (__typeof__(&moe_unsort))p[1];
    f_unsort_backward = (__typeof__(&moe_unsort_backward))p[2];
    f_int8_quantise = (__typeof__(&int8_quantise))p[3];
    f_int8_matmul = (__typeof__(&int8_matmul))p[4];
    f_int8_grouped = (__typeof__(&int8_grouped_matmul))p[5];
    f_int8_linear = (__typeof__(&int8_linear))p[6];
    Py_RETURN_NONE;
}

#define METHOD(name, f, doc) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, doc}
static PyMethodDef methods[] = {
    METHOD("bind", bind, "bind(moe_route, fp8_block_linear, fp8_block_matmul, moe_experts_forward): addresses"),
    METHOD("moe_route", route, "mse.h: moe_route"),
    METHOD("fp8_block_matmul", matmul, "mse.h: fp8_block_matmul"),
    METHOD("fp8_block_linear", linear, "mse.h: fp8_block_linear"),
    METHOD("moe_experts_forward", experts, "mse.h: moe_experts_forward"),
    METHOD("bind_rows", bind_rows,
           "bind_rows(moe_sort, moe_unsort, moe_unsort_backward, int8_quantise, int8_matmul, int8_grouped_matmul, "
           "int8_linear): addresses"),
    METHOD("moe_sort", sort, "mse.h: moe_sort"),
    METHOD("moe_unsort", unsort, "mse.h: moe_unsort"),
    METHOD("moe_unsort_backward", unsort_backward, "mse.h: moe_unsort_backward"),
    METHOD("int8_quantise", quantise, "mse.h: int8_quantise"),
    METHOD("int8_matmul", matmul8, "mse.h: int8_matmul"),
    METHOD("int8_grouped_matmul", grouped8, "mse.h: int8_grouped_matmul"),
    METHOD("int8_linear", linear8, "mse.h: int8_linear"),
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
