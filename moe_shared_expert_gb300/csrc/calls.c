/* Python entry of the routed-expert calls: arguments by vectorcall into the C ABI's functions (whose
 * addresses the package hands over), a fifth of what ctypes takes for as many arguments.  Integers and
 * None (a null pointer) only; every check of the arguments is the library's. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "mse.h"

static __typeof__(&moe_route) f_route;
static __typeof__(&fp8_block_linear) f_linear;
static __typeof__(&fp8_block_matmul) f_matmul;
static __typeof__(&moe_experts_forward) f_experts;

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

#define METHOD(name, f, doc) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, doc}
static PyMethodDef methods[] = {
    METHOD("bind", bind, "bind(moe_route, fp8_block_linear, fp8_block_matmul, moe_experts_forward): addresses"),
    METHOD("moe_route", route, "mse.h: moe_route"),
    METHOD("fp8_block_matmul", matmul, "mse.h: fp8_block_matmul"),
    METHOD("fp8_block_linear", linear, "mse.h: fp8_block_linear"),
    METHOD("moe_experts_forward", experts, "mse.h: moe_experts_forward"),
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
