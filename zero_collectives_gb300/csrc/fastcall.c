/*
 * fastcall.c -- a CPython extension that makes one prepared dpred_flush_bucket
 * call with less host overhead than ctypes.
 *
 * A training loop flushes the same buckets every step with the same
 * arguments.  ctypes converts all seventeen arguments on every call (about
 * 1.3 us); here they are converted once, by prepare(), into a C struct kept in
 * a capsule, and flush() passes them on together with the per-call stream and
 * probe.  call() makes one unprepared call from plain integers, for the
 * binding's flush_bucket; linear(), linear_dgrad() and linear_wgrad() do the
 * same for the linear-layer products, embedding() and the others below them for the
 * rest of a training step.  The function called is the library's own dpred_flush_bucket, whose
 * address the Python binding hands over (the library is loaded once, by the
 * binding, so the plan cache and the error state are the ones every other
 * call uses).  This module adds no arithmetic: argument marshalling only.
 * It is optional: where it cannot be built (no Python headers), the binding
 * makes the same call through ctypes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include "dpred.h"

typedef int (*flush_fn)(int32_t, int32_t, void*, int64_t, const dpred_task*, int32_t, const int32_t*, int32_t,
                        int32_t, void* const*, int32_t, int32_t, int32_t, dpred_probe*, void*, size_t, void*);

typedef struct {
    flush_fn fn;
    int32_t world, in_dt, n_tasks, n_params, out_dt, pre_div, rto, flags;
    void* grads;
    int64_t ld;
    const dpred_task* tasks;
    const int32_t* owner;
    void* const* dst;
    void* workspace;
    size_t workspace_bytes;
} Prepared;

static const char* kCapsule = "dpred.prepared_flush";

static void release(PyObject* cap) { free(PyCapsule_GetPointer(cap, kCapsule)); }

/* prepare(fn, world, in_dt, grads, ld, tasks, n_tasks, owner, n_params, out_dt, dst, pre_div,
 *         reduce_to_owner, flags, workspace, workspace_bytes) -> capsule
 * Pointers are integer addresses (0 = NULL); the caller keeps the memory behind
 * them alive for as long as the capsule is used. */
static PyObject* prepare(PyObject* self, PyObject* args) {
    (void)self;
    unsigned long long fn, grads, tasks, owner, dst, ws, ws_bytes;
    long long ld;
    int world, in_dt, n_tasks, n_params, out_dt, pre_div, rto, flags;
    if (!PyArg_ParseTuple(args, "KiiKLKiKiiKiiiKK", &fn, &world, &in_dt, &grads, &ld, &tasks, &n_tasks, &owner,
                          &n_params, &out_dt, &dst, &pre_div, &rto, &flags, &ws, &ws_bytes))
        return NULL;
    if (!fn) {
        PyErr_SetString(PyExc_ValueError, "null function address");
        return NULL;
    }
    Prepared* p = (Prepared*)malloc(sizeof(Prepared));
    if (!p) return PyErr_NoMemory();
    p->fn = (flush_fn)(uintptr_t)fn;
    p->world = world;
    p->in_dt = in_dt;
    p->grads = (void*)(uintptr_t)grads;
    p->ld = (int64_t)ld;
    p->tasks = (const dpred_task*)(uintptr_t)tasks;
    p->n_tasks = n_tasks;
    p->owner = (const int32_t*)(uintptr_t)owner;
    p->n_params = n_params;
    p->out_dt = out_dt;
    p->dst = (void* const*)(uintptr_t)dst;
    p->pre_div = pre_div;
    p->rto = rto;
    p->flags = flags;
    p->workspace = (void*)(uintptr_t)ws;
    p->workspace_bytes = (size_t)ws_bytes;
    PyObject* cap = PyCapsule_New(p, kCapsule, release);
    if (!cap) free(p);
    return cap;
}

/* The interpreter lock is released around the library call, as ctypes does:
 * a plan that needs workspace copies it to the device, which can block. */
static int call(const Prepared* p, dpred_probe* probe, PyObject* stream_arg) {
    const unsigned long long stream = PyLong_AsUnsignedLongLong(stream_arg);
    if (stream == (unsigned long long)-1 && PyErr_Occurred()) return INT32_MIN;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = p->fn(p->world, p->in_dt, p->grads, p->ld, p->tasks, p->n_tasks, p->owner, p->n_params, p->out_dt, p->dst,
               p->pre_div, p->rto, p->flags, probe, p->workspace, p->workspace_bytes, (void*)(uintptr_t)stream);
    Py_END_ALLOW_THREADS
    return rc;
}

/* flush(capsule, stream) -> status code of dpred_flush_bucket */
static PyObject* flush(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 2) {
        PyErr_SetString(PyExc_TypeError, "flush(prepared, stream)");
        return NULL;
    }
    const Prepared* p = (const Prepared*)PyCapsule_GetPointer(args[0], kCapsule);
    if (!p) return NULL;
    const int rc = call(p, NULL, args[1]);
    return rc == INT32_MIN ? NULL : PyLong_FromLong(rc);
}

/* The probe counters of one call as (status, flush_index, tasks, reduced_elems,
 * owner_tasks, owner_elems, [kept_elems of each rank]). */
static PyObject* probe_tuple(int rc, const dpred_probe* probe, int world) {
    const int w = world < 0 ? 0 : (world > DPRED_MAX_WORLD ? DPRED_MAX_WORLD : world);
    PyObject* kept = PyList_New(w);
    if (!kept) return NULL;
    for (int r = 0; r < w; ++r) {
        PyObject* v = PyLong_FromLongLong(probe->kept_elems[r]);
        if (!v) {
            Py_DECREF(kept);
            return NULL;
        }
        PyList_SET_ITEM(kept, r, v);
    }
    return Py_BuildValue("(iLLLLLN)", rc, (long long)probe->flush_index, (long long)probe->tasks,
                         (long long)probe->reduced_elems, (long long)probe->owner_tasks, (long long)probe->owner_elems,
                         kept);
}

/* flush_probed(capsule, stream, flush_index)
 *   -> (status, flush_index, tasks, reduced_elems, owner_tasks, owner_elems, [kept_elems of each rank])
 * The counters live on this call's stack, so concurrent calls share nothing. */
static PyObject* flush_probed(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 3) {
        PyErr_SetString(PyExc_TypeError, "flush_probed(prepared, stream, flush_index)");
        return NULL;
    }
    const Prepared* p = (const Prepared*)PyCapsule_GetPointer(args[0], kCapsule);
    if (!p) return NULL;
    dpred_probe probe;
    memset(&probe, 0, sizeof probe);
    probe.flush_index = PyLong_AsLongLong(args[2]);
    if (probe.flush_index == -1 && PyErr_Occurred()) return NULL;
    const int rc = call(p, &probe, args[1]);
    if (rc == INT32_MIN) return NULL;
    return probe_tuple(rc, &probe, p->world);
}

/* call(fn, world, in_dt, grads, ld, tasks, n_tasks, owner, n_params, out_dt, dst, pre_div,
 *      reduce_to_owner, flags, workspace, workspace_bytes, stream, flush_index)
 * One unprepared dpred_flush_bucket call; addresses are integers (0 = NULL).
 * flush_index None: no probe, returns the status code; an integer: returns the
 * probe tuple of flush_probed. */
static PyObject* call_once(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 18) {
        PyErr_SetString(PyExc_TypeError, "call() takes 18 arguments");
        return NULL;
    }
    /* addresses and the workspace size are unsigned; the other arguments are
     * signed and reach the library as ctypes would pass them */
    static const int kUnsigned[16] = {1, 0, 0, 1, 0, 1, 0, 1, 0, 0, 1, 0, 0, 0, 1, 1};
    unsigned long long u[16];
    for (int i = 0; i < 16; ++i) {
        if (kUnsigned[i]) {
            u[i] = PyLong_AsUnsignedLongLong(args[i]);
        } else {
            const long long v = PyLong_AsLongLong(args[i]);
            u[i] = (unsigned long long)v;
        }
        if (u[i] == (unsigned long long)-1 && PyErr_Occurred()) return NULL;
    }
    if (!u[0]) {
        PyErr_SetString(PyExc_ValueError, "null function address");
        return NULL;
    }
    Prepared p;
    p.fn = (flush_fn)(uintptr_t)u[0];
    p.world = (int32_t)u[1];
    p.in_dt = (int32_t)u[2];
    p.grads = (void*)(uintptr_t)u[3];
    p.ld = (int64_t)u[4];
    p.tasks = (const dpred_task*)(uintptr_t)u[5];
    p.n_tasks = (int32_t)u[6];
    p.owner = (const int32_t*)(uintptr_t)u[7];
    p.n_params = (int32_t)u[8];
    p.out_dt = (int32_t)u[9];
    p.dst = (void* const*)(uintptr_t)u[10];
    p.pre_div = (int32_t)u[11];
    p.rto = (int32_t)u[12];
    p.flags = (int32_t)u[13];
    p.workspace = (void*)(uintptr_t)u[14];
    p.workspace_bytes = (size_t)u[15];
    if (args[17] == Py_None) {
        const int rc = call(&p, NULL, args[16]);
        return rc == INT32_MIN ? NULL : PyLong_FromLong(rc);
    }
    dpred_probe probe;
    memset(&probe, 0, sizeof probe);
    probe.flush_index = PyLong_AsLongLong(args[17]);
    if (probe.flush_index == -1 && PyErr_Occurred()) return NULL;
    const int rc = call(&p, &probe, args[16]);
    if (rc == INT32_MIN) return NULL;
    return probe_tuple(rc, &probe, p.world);
}

/* linear(fn, ...), linear_dgrad(fn, ...), linear_wgrad(fn, ...): one call of the
 * entry point at address fn with its arguments as integers (addresses too; 0 =
 * NULL), returning its status code. */
#define DPRED_MAX_INTS 20
static int integers(PyObject* const* args, Py_ssize_t nargs, Py_ssize_t want, long long* v) {
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, nargs);
        return -1;
    }
    for (Py_ssize_t i = 0; i < want; ++i) {
        v[i] = PyLong_AsLongLong(args[i]);
        if (v[i] == -1 && PyErr_Occurred()) return -1;
    }
    if (!v[0]) {
        PyErr_SetString(PyExc_ValueError, "null function address");
        return -1;
    }
    return 0;
}
#define DPRED_I32(i) ((int32_t)v[i])
#define DPRED_PTR(i) ((void*)(uintptr_t)v[i])

static PyObject* linear(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    long long v[DPRED_MAX_INTS + 1];
    if (integers(args, nargs, 21, v)) return NULL;
    int (*fn)(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t, int32_t, const void*, int32_t,
              const void*, int64_t, void*, int64_t, int32_t, void*, int64_t, void*, size_t, void*) = DPRED_PTR(0);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(v[1], v[2], v[3], DPRED_PTR(4), v[5], DPRED_PTR(6), v[7], DPRED_I32(8), DPRED_PTR(9), DPRED_I32(10),
            DPRED_PTR(11), v[12], DPRED_PTR(13), v[14], DPRED_I32(15), DPRED_PTR(16), v[17], DPRED_PTR(18),
            (size_t)v[19], DPRED_PTR(20));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* linear_dgrad(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    long long v[DPRED_MAX_INTS + 1];
    if (integers(args, nargs, 19, v)) return NULL;
    int (*fn)(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t, int32_t, const void*, int64_t,
              const void*, int64_t, int32_t, void*, int64_t, void*, size_t, void*) = DPRED_PTR(0);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(v[1], v[2], v[3], DPRED_PTR(4), v[5], DPRED_PTR(6), v[7], DPRED_I32(8), DPRED_PTR(9), v[10], DPRED_PTR(11),
            v[12], DPRED_I32(13), DPRED_PTR(14), v[15], DPRED_PTR(16), (size_t)v[17], DPRED_PTR(18));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* linear_wgrad(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    long long v[DPRED_MAX_INTS + 1];
    if (integers(args, nargs, 16, v)) return NULL;
    int (*fn)(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t, int32_t, int32_t, void*, int64_t,
              float*, void*, size_t, void*) = DPRED_PTR(0);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(v[1], v[2], v[3], DPRED_PTR(4), v[5], DPRED_PTR(6), v[7], DPRED_I32(8), DPRED_I32(9), DPRED_PTR(10), v[11],
            DPRED_PTR(12), DPRED_PTR(13), (size_t)v[14], DPRED_PTR(15));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* As integers(), for entry points with floating arguments: bit i of `reals` says
 * that argument i is one (it goes to r[i]). */
#define DPRED_MAX_ARGS 36
static int numbers(PyObject* const* args, Py_ssize_t nargs, Py_ssize_t want, unsigned long long reals, long long* v, double* r) {
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, nargs);
        return -1;
    }
    for (Py_ssize_t i = 0; i < want; ++i) {
        if (reals >> i & 1) {
            r[i] = PyFloat_AsDouble(args[i]);
            if (r[i] == -1.0 && PyErr_Occurred()) return -1;
        } else {
            v[i] = PyLong_AsLongLong(args[i]);
            if (v[i] == -1 && PyErr_Occurred()) return -1;
        }
    }
    if (!v[0]) {
        PyErr_SetString(PyExc_ValueError, "null function address");
        return -1;
    }
    return 0;
}
#define DPRED_REAL(i) ((float)r[i])

static PyObject* embedding(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    long long v[DPRED_MAX_ARGS];
    double r[DPRED_MAX_ARGS];
    if (numbers(args, nargs, 14, 1ull << 9, v, r)) return NULL;
    int (*fn)(int64_t, int64_t, int64_t, int32_t, const void*, int32_t, const void*, int64_t, float, int32_t, void*, int64_t,
              void*) = DPRED_PTR(0);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(v[1], v[2], v[3], DPRED_I32(4), DPRED_PTR(5), DPRED_I32(6), DPRED_PTR(7), v[8], DPRED_REAL(9), DPRED_I32(10),
            DPRED_PTR(11), v[12], DPRED_PTR(13));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* embedding_grad(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    long long v[DPRED_MAX_ARGS];
    double r[DPRED_MAX_ARGS];
    if (numbers(args, nargs, 18, 1ull << 10, v, r)) return NULL;
    int (*fn)(int64_t, int64_t, int64_t, int32_t, const void*, int64_t, int32_t, const void*, int64_t, float, int32_t, int32_t, void*,
              int64_t, void*, size_t, void*) = DPRED_PTR(0);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(v[1], v[2], v[3], DPRED_I32(4), DPRED_PTR(5), v[6], DPRED_I32(7), DPRED_PTR(8), v[9], DPRED_REAL(10), DPRED_I32(11),
            DPRED_I32(12), DPRED_PTR(13), v[14], DPRED_PTR(15), (size_t)v[16], DPRED_PTR(17));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* block_norm(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    long long v[DPRED_MAX_ARGS];
    double r[DPRED_MAX_ARGS];
    if (numbers(args, nargs, 22, 1ull << 13 | 1ull << 16, v, r)) return NULL;
    int (*fn)(int64_t, int64_t, int32_t, const void*, int64_t, const void*, int64_t, int32_t, const void*, int32_t, const void*, int64_t,
              float, int32_t, const void*, float, void*, int64_t, void*, int64_t, void*) = DPRED_PTR(0);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(v[1], v[2], DPRED_I32(3), DPRED_PTR(4), v[5], DPRED_PTR(6), v[7], DPRED_I32(8), DPRED_PTR(9), DPRED_I32(10), DPRED_PTR(11),
            v[12], DPRED_REAL(13), DPRED_I32(14), DPRED_PTR(15), DPRED_REAL(16), DPRED_PTR(17), v[18], DPRED_PTR(19), v[20], DPRED_PTR(21));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* block_norm_grad(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    long long v[DPRED_MAX_ARGS];
    double r[DPRED_MAX_ARGS];
    if (numbers(args, nargs, 33, 1ull << 17 | 1ull << 20, v, r)) return NULL;
    int (*fn)(int64_t, int64_t, int32_t, const void*, int64_t, const void*, int64_t, const void*, int64_t, const void*, int64_t, int32_t,
              const void*, int32_t, const void*, int64_t, float, int32_t, const void*, float, void*, int64_t, void*, int64_t, int32_t,
              void*, void*, void*, int32_t, void*, size_t, void*) = DPRED_PTR(0);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(v[1], v[2], DPRED_I32(3), DPRED_PTR(4), v[5], DPRED_PTR(6), v[7], DPRED_PTR(8), v[9], DPRED_PTR(10), v[11], DPRED_I32(12),
            DPRED_PTR(13), DPRED_I32(14), DPRED_PTR(15), v[16], DPRED_REAL(17), DPRED_I32(18), DPRED_PTR(19), DPRED_REAL(20), DPRED_PTR(21),
            v[22], DPRED_PTR(23), v[24], DPRED_I32(25), DPRED_PTR(26), DPRED_PTR(27), DPRED_PTR(28), DPRED_I32(29), DPRED_PTR(30),
            (size_t)v[31], DPRED_PTR(32));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* grad_norm(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    long long v[DPRED_MAX_ARGS];
    double r[DPRED_MAX_ARGS];
    if (numbers(args, nargs, 7, 0, v, r)) return NULL;
    int (*fn)(const dpred_grad_tensor*, int32_t, float*, void*, size_t, void*) = DPRED_PTR(0);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(DPRED_PTR(1), DPRED_I32(2), DPRED_PTR(3), DPRED_PTR(4), (size_t)v[5], DPRED_PTR(6));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyObject* clip_grads(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    long long v[DPRED_MAX_ARGS];
    double r[DPRED_MAX_ARGS];
    if (numbers(args, nargs, 9, 1ull << 3 | 1ull << 4, v, r)) return NULL;
    int (*fn)(const dpred_grad_tensor*, int32_t, float, float, float*, void*, size_t, void*) = DPRED_PTR(0);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(DPRED_PTR(1), DPRED_I32(2), DPRED_REAL(3), DPRED_REAL(4), DPRED_PTR(5), DPRED_PTR(6), (size_t)v[7], DPRED_PTR(8));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyMethodDef kMethods[] = {
    {"embedding", (PyCFunction)(void (*)(void))embedding, METH_FASTCALL, "One dpred_embedding call from numbers."},
    {"embedding_grad", (PyCFunction)(void (*)(void))embedding_grad, METH_FASTCALL, "One dpred_embedding_grad call from numbers."},
    {"block_norm", (PyCFunction)(void (*)(void))block_norm, METH_FASTCALL, "One dpred_block_norm call from numbers."},
    {"block_norm_grad", (PyCFunction)(void (*)(void))block_norm_grad, METH_FASTCALL, "One dpred_block_norm_grad call from numbers."},
    {"grad_norm", (PyCFunction)(void (*)(void))grad_norm, METH_FASTCALL, "One dpred_grad_norm call from numbers."},
    {"clip_grads", (PyCFunction)(void (*)(void))clip_grads, METH_FASTCALL, "One dpred_clip_grads call from numbers."},
    {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, "One dpred_linear call from integers."},
    {"linear_dgrad", (PyCFunction)(void (*)(void))linear_dgrad, METH_FASTCALL, "One dpred_linear_dgrad call from integers."},
    {"linear_wgrad", (PyCFunction)(void (*)(void))linear_wgrad, METH_FASTCALL, "One dpred_linear_wgrad call from integers."},
    {"prepare", prepare, METH_VARARGS, "Convert one dpred_flush_bucket call's arguments once."},
    {"flush", (PyCFunction)(void (*)(void))flush, METH_FASTCALL, "Make a prepared dpred_flush_bucket call."},
    {"flush_probed", (PyCFunction)(void (*)(void))flush_probed, METH_FASTCALL,
     "Make a prepared dpred_flush_bucket call and return its probe counters."},
    {"call", (PyCFunction)(void (*)(void))call_once, METH_FASTCALL, "Make one unprepared dpred_flush_bucket call."},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, kMethods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&kModule); }
