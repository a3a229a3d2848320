/* calls.c -- the router's and the dense products' calls of the Python binding, as
 * a CPython extension: it looks a call's tensors over (type, shape, layout, device)
 * and makes the call of the C ABI. A small call's time is its host's: for a
 * router of one token 5.7 us through ctypes with the checks in Python, 3.8 us
 * through here, of which the kernel's launch is 1.9.
 *
 * Each function returns the library's status, or -1 where an argument is not what
 * the call takes; ep.py then looks at them one by one and says which. Plain C, for the
 * interpreter (3.9 or later) whose headers it was built with; no header of torch or CUDA.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "ep.h"

/* From ep.py's bind(): the library's entry points, torch's types, the calls that
 * give the current device and its stream. */
static struct {
    ep_status_t (*route)(const void*, int, int64_t, int, int, const float*, int, int, int, int, int,
                         float, int64_t*, float*, void*);
    ep_status_t (*route_grad)(const float*, const void*, int, const int64_t*, int64_t, int, int, int,
                              int, float, void*, int32_t*, void*);
    ep_status_t (*linear)(const uint16_t*, int64_t, int64_t, const uint16_t*, int64_t, const float*,
                          int, const void*, int, void*, uint16_t*, int32_t*, void*);
    ep_status_t (*act_grad)(const void*, int, const uint16_t*, int64_t, int64_t, int, uint16_t*,
                            int64_t, float*, void*);
    ep_status_t (*grad_input)(const uint16_t*, int64_t, int64_t, int64_t, const uint16_t*, int64_t,
                              uint16_t*, int32_t*, void*);
    ep_status_t (*grad_weight)(const uint16_t*, int64_t, int64_t, int64_t, const uint16_t*, int64_t,
                               int, void*, int, int32_t*, void*);
} g_lib;
static PyObject *g_bf16, *g_f32, *g_i32, *g_i64, *g_device, *g_stream;
static PyObject *s_dtype, *s_shape, *s_is_contiguous, *s_get_device, *s_data_ptr;

/* A call in the making: the device its tensors have to be on (the current one, asked
 * for with the first of them), and whether all has fitted so far. */
typedef struct {
    long device;
    int ok;
} Call;

static long as_long(PyObject* v) { /* steals v; -2 and no exception where it is no number */
    long r = -2;
    if (v != NULL) {
        r = PyLong_AsLong(v);
        Py_DECREF(v);
    }
    if (PyErr_Occurred()) {
        PyErr_Clear();
        r = -2;
    }
    return r;
}

/* The two sizes of a matrix. */
static void sizes(Call* c, PyObject* t, int64_t* rows, int64_t* cols) {
    *rows = *cols = -1;
    PyObject* shape = PyObject_GetAttr(t, s_shape);
    if (shape != NULL && PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 2) {
        *rows = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
        *cols = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
    } else {
        c->ok = 0;
    }
    Py_XDECREF(shape);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        c->ok = 0;
    }
}

/* The address of a contiguous tensor of this type and shape (cols < 0: of one
 * dimension; rows < 0 too: any) on the call's device; a null pointer for None. */
static void* address(Call* c, PyObject* t, PyObject* dtype, int64_t rows, int64_t cols) {
    if (t == Py_None || !c->ok) return NULL;
    void* p = NULL;
    int ok = 0;
    PyObject* type = PyObject_GetAttr(t, s_dtype);
    PyObject* shape = PyObject_GetAttr(t, s_shape);
    PyObject* flat = NULL;
    if (type == dtype && shape != NULL && PyTuple_Check(shape)) {
        const Py_ssize_t n = PyTuple_GET_SIZE(shape);
        ok = rows < 0 && cols < 0;
        ok = ok || (n == (cols < 0 ? 1 : 2) && PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0)) == rows &&
             (cols < 0 || PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1)) == cols));
    }
    if (ok) {
        flat = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        ok = flat == Py_True;
    }
    if (ok) {
        const long device = as_long(PyObject_CallMethodNoArgs(t, s_get_device));
        if (device >= 0 && c->device < 0) c->device = as_long(PyObject_CallNoArgs(g_device));
        ok = device >= 0 && device == c->device;
    }
    if (ok) {
        PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
        if (v != NULL) {
            p = PyLong_AsVoidPtr(v);
            Py_DECREF(v);
        } else {
            ok = 0;
        }
    }
    Py_XDECREF(type);
    Py_XDECREF(shape);
    Py_XDECREF(flat);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        ok = 0;
    }
    if (!ok) c->ok = 0;
    return p;
}

/* As address(), of a tensor that has to be there. */
static void* needed(Call* c, PyObject* t, PyObject* dtype, int64_t rows, int64_t cols) {
    if (t == Py_None) c->ok = 0;
    return address(c, t, dtype, rows, cols);
}

/* ep_type_t and torch's type of a tensor that may be bf16 or fp32. */
static PyObject* kind_of(Call* c, PyObject* t, int* kind) {
    PyObject* type = PyObject_GetAttr(t, s_dtype);
    *kind = type == g_bf16 ? EP_BF16 : EP_F32;
    if (type != g_bf16 && type != g_f32) c->ok = 0;
    if (type == NULL) PyErr_Clear();
    Py_XDECREF(type);
    return *kind == EP_BF16 ? g_bf16 : g_f32;
}

/* A number that fits an int. */
static int number(Call* c, PyObject* v) {
    const long n = PyLong_AsLong(v);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        c->ok = 0;
    }
    if (n < INT32_MIN || n > INT32_MAX) c->ok = 0;
    return (int)n;
}
static int truth(Call* c, PyObject* v) {
    const int b = PyObject_IsTrue(v);
    if (b < 0) {
        PyErr_Clear();
        c->ok = 0;
    }
    return b;
}
static float real(Call* c, PyObject* v) {
    const double n = PyFloat_AsDouble(v);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        c->ok = 0;
    }
    return (float)n;
}

/* The stream: a raw handle, or None for the device's current one. */
static void* stream_of(Call* c, PyObject* stream) {
    if (!c->ok) return NULL;
    PyObject* v = NULL;
    if (stream == Py_None) {
        PyObject* device = PyLong_FromLong(c->device);
        if (device != NULL) v = PyObject_CallOneArg(g_stream, device);
        Py_XDECREF(device);
    } else {
        v = stream;
        Py_INCREF(v);
    }
    void* p = v == NULL ? NULL : PyLong_AsVoidPtr(v);
    Py_XDECREF(v);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        c->ok = 0;
    }
    return p;
}

/* The call itself, other threads running meanwhile: it may wait where a kernel is
 * loaded for the first time. */
#define MAKE(call)                      \
    ep_status_t code = EP_OK;           \
    if (!c.ok) return PyLong_FromLong(-1); \
    Py_BEGIN_ALLOW_THREADS              \
    code = call;                        \
    Py_END_ALLOW_THREADS                \
    return PyLong_FromLong((long)code);

#define ARGS(count)                                                          \
    Call c = {-1, 1};                                                        \
    (void)self;                                                              \
    if (n != (count)) {                                                      \
        PyErr_SetString(PyExc_TypeError, "expected " #count " arguments");   \
        return NULL;                                                         \
    }

/* logits, topk_idx, topk_w, bias, score, groups, topk_groups, group_score,
 * renormalize, scale, stream */
static PyObject* route(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    ARGS(11)
    int64_t T, E, rows, K;
    int kind;
    sizes(&c, a[0], &T, &E);
    sizes(&c, a[1], &rows, &K);
    PyObject* type = kind_of(&c, a[0], &kind);
    void* logits = needed(&c, a[0], type, T, E);
    int64_t* idx = needed(&c, a[1], g_i64, T, K);
    float* w = needed(&c, a[2], g_f32, T, K);
    const float* bias = address(&c, a[3], g_f32, E, -1);
    const int score = number(&c, a[4]), groups = number(&c, a[5]), kept = number(&c, a[6]);
    const int worth = number(&c, a[7]), renormalize = truth(&c, a[8]);
    const float scale = real(&c, a[9]);
    void* s = stream_of(&c, a[10]);
    if (score < 0 || worth < 0 || E > INT32_MAX || K > INT32_MAX) c.ok = 0;
    MAKE(g_lib.route(logits, kind, T, (int)E, (int)K, bias, score, groups, kept, worth,
         renormalize, scale, idx, w, s))
}

/* d_topk_w, logits, topk_idx, d_logits, score, renormalize, scale, status, stream */
static PyObject* route_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    ARGS(9)
    int64_t T, E, rows, K;
    int kind;
    sizes(&c, a[1], &T, &E);
    sizes(&c, a[2], &rows, &K);
    PyObject* type = kind_of(&c, a[1], &kind);
    const float* dw = needed(&c, a[0], g_f32, T, K);
    const void* logits = needed(&c, a[1], type, T, E);
    const int64_t* idx = needed(&c, a[2], g_i64, T, K);
    void* d = needed(&c, a[3], type, T, E);
    const int score = number(&c, a[4]), renormalize = truth(&c, a[5]);
    const float scale = real(&c, a[6]);
    int32_t* status = address(&c, a[7], g_i32, -1, -1);
    void* s = stream_of(&c, a[8]);
    if (score < 0 || E > INT32_MAX || K > INT32_MAX) c.ok = 0;
    MAKE(g_lib.route_grad(dw, logits, kind, idx, T, (int)E, (int)K, score, renormalize,
         scale, d, status, s))
}

/* x, w, y, bias, activation, residual, z, status, stream */
static PyObject* linear(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    ARGS(9)
    int64_t M, K, wide, k2, m2, N;
    int kind;
    sizes(&c, a[0], &M, &K);
    sizes(&c, a[1], &wide, &k2);
    sizes(&c, a[2], &m2, &N);
    const int act = number(&c, a[4]);
    if (act < 0 || wide != (act == EP_ACT_SWIGLU ? 2 * N : N)) c.ok = 0;
    PyObject* type = kind_of(&c, a[2], &kind);
    const uint16_t* x = needed(&c, a[0], g_bf16, M, K);
    const uint16_t* w = needed(&c, a[1], g_bf16, wide, K);
    void* y = needed(&c, a[2], type, M, N);
    const float* bias = address(&c, a[3], g_f32, wide, -1);
    const void* residual = address(&c, a[5], type, M, N);
    uint16_t* z = address(&c, a[6], g_bf16, M, wide);
    int32_t* status = address(&c, a[7], g_i32, -1, -1);
    void* s = stream_of(&c, a[8]);
    MAKE(g_lib.linear(x, M, K, w, N, bias, act, residual, kind, y, z, status, s))
}

/* dy, z, dz, d_bias, activation, stream */
static PyObject* act_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    ARGS(6)
    int64_t M, N;
    int kind;
    sizes(&c, a[0], &M, &N);
    const int act = number(&c, a[4]);
    const int64_t wide = act == EP_ACT_SWIGLU ? 2 * N : N, pitch = (wide + 7) / 8 * 8;
    if (act < 0 || (act != EP_ACT_NONE && a[1] == Py_None)) c.ok = 0;
    PyObject* type = kind_of(&c, a[0], &kind);
    const void* dy = needed(&c, a[0], type, M, N);
    const uint16_t* z = address(&c, a[1], g_bf16, M, wide);
    uint16_t* dz = address(&c, a[2], g_bf16, M, pitch);
    float* d_bias = address(&c, a[3], g_f32, wide, -1);
    void* s = stream_of(&c, a[5]);
    MAKE(g_lib.act_grad(dy, kind, z, M, N, act, dz, pitch, d_bias, s))
}

/* dz, w, dx, status, stream */
static PyObject* grad_input(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    ARGS(5)
    int64_t M, pitch, N, K;
    sizes(&c, a[0], &M, &pitch);
    sizes(&c, a[1], &N, &K);
    const uint16_t* dz = needed(&c, a[0], g_bf16, M, (N + 7) / 8 * 8);
    const uint16_t* w = needed(&c, a[1], g_bf16, N, K);
    uint16_t* dx = needed(&c, a[2], g_bf16, M, K);
    int32_t* status = address(&c, a[3], g_i32, -1, -1);
    void* s = stream_of(&c, a[4]);
    MAKE(g_lib.grad_input(dz, pitch, M, N, w, K, dx, status, s))
}

/* dz, x, d_w, accumulate, status, stream */
static PyObject* grad_weight(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    ARGS(6)
    int64_t M, pitch, N, K;
    int kind;
    sizes(&c, a[0], &M, &pitch);
    sizes(&c, a[2], &N, &K);
    PyObject* type = kind_of(&c, a[2], &kind);
    const uint16_t* dz = needed(&c, a[0], g_bf16, M, (N + 7) / 8 * 8);
    const uint16_t* x = needed(&c, a[1], g_bf16, M, K);
    void* d_w = needed(&c, a[2], type, N, K);
    const int accumulate = truth(&c, a[3]);
    int32_t* status = address(&c, a[4], g_i32, -1, -1);
    void* s = stream_of(&c, a[5]);
    MAKE(g_lib.grad_weight(dz, pitch, M, N, x, K, kind, d_w, accumulate, status, s))
}

/* The six entry points' addresses, torch's bf16, fp32, int32 and int64, the calls
 * that give the current device and its stream. */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    ARGS(12)
    (void)c;
    void* p[6];
    for (int i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return NULL;
    }
    *(void**)&g_lib.route = p[0];
    *(void**)&g_lib.route_grad = p[1];
    *(void**)&g_lib.linear = p[2];
    *(void**)&g_lib.act_grad = p[3];
    *(void**)&g_lib.grad_input = p[4];
    *(void**)&g_lib.grad_weight = p[5];
    PyObject** const to[6] = {&g_bf16, &g_f32, &g_i32, &g_i64, &g_device, &g_stream};
    for (int i = 0; i < 6; ++i) {
        Py_INCREF(a[6 + i]);
        Py_XSETREF(*to[i], a[6 + i]);
    }
    Py_RETURN_NONE;
}

#define CALL(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {CALL(bind),       CALL(route),       CALL(route_grad), CALL(linear),
                                CALL(act_grad),   CALL(grad_input),  CALL(grad_weight), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (!s_dtype || !s_shape || !s_is_contiguous || !s_get_device || !s_data_ptr) return NULL;
    return PyModule_Create(&module);
}
