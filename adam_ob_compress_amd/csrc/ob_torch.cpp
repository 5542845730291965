// ob_torch.cpp -- the Python module _obtorch: the calls over lists of tensors with torch tensors as arguments.
// Each function checks its tensors (type, size, device, layout), takes their addresses and makes the call of the C ABI;
// no arithmetic here, and no torch type crosses that boundary.
//
// Why compiled: asked from Python, the five properties of a tensor cost 0.3 us, here 0.01 to 0.02.  A step's call with
// 16 tensors took 17.6 us all in Python, 6.3 to 6.6 with the addresses read here and the call made by ctypes, and takes
// 4.9 to 5.4 now (time until the call returns; every call is a fifth shorter in some processes); the others went from
// 5.4 to 5.9 (ctypes) to 4.5 to 5.1.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <memory>
#include <stdexcept>
#include <string>
#include <vector>

#include "ob_adam.h"

namespace {

// What a list expects of its tensors.
struct List {
    ob_tensors handle;
    long device;
    int64_t state_elems;
    std::vector<int64_t> numel;
    std::string g_types, p_types;   // c10 scalar types
};

constexpr const char* kListName = "adam_ob_compress_amd.list";

// An argument that is not as it should be: `where` among the call's (0 gradients, 1 parameters, from 2 on the flat
// buffers in their order), `index` in a list.  Returned to Python as a negative number, which explains it there.
struct Bad {
    int64_t where, index;
    PyObject* code() const { return PyLong_FromLongLong(-(1 + (where << 32) + index)); }
};

// The address of a dense GPU tensor of this kind; throws Bad otherwise, also for one whose storage does not hold it (released
// or shrunk: its address is NULL, which would mean that the tensor is left out, or its end is behind the memory).
void* address(PyObject* item, at::ScalarType type, int64_t numel, long device, Bad at)
{
    if (!THPVariable_Check(item)) throw at;
    const at::Tensor& t = THPVariable_Unpack(item);
    if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != device || t.is_neg() || t.scalar_type() != type ||
        t.numel() != numel || !t.is_contiguous() || !t.has_storage())
        throw at;
    if (numel == 0) return nullptr;
    void* p = nullptr;
    try {   // a tensor without memory of its own (a fake one) throws c10's error
        if (t.storage().nbytes() / t.itemsize() >= static_cast<size_t>(t.storage_offset() + numel)) p = t.data_ptr();
    } catch (...) {
    }
    if (!p) throw at;
    return p;
}

// The same for an optional flat buffer: None -> NULL.
void* flat(PyObject* item, at::ScalarType type, int64_t numel, long device, int64_t where)
{
    return item == Py_None ? nullptr : address(item, type, numel, device, Bad{where, 0});
}

// The addresses of a list or tuple of tensors or Nones; others: where it has a tensor, so must this one.
std::vector<void*> addresses(PyObject* tensors, PyObject* others, const List& l, const std::string& types, int64_t where)
{
    if (!PyList_Check(tensors) && !PyTuple_Check(tensors)) throw Bad{where, 0};
    const Py_ssize_t T = static_cast<Py_ssize_t>(l.numel.size());
    if (PySequence_Fast_GET_SIZE(tensors) != T) throw Bad{where, 0};
    PyObject** items = PySequence_Fast_ITEMS(tensors);
    PyObject** other = others ? PySequence_Fast_ITEMS(others) : nullptr;   // checked before, of the same length
    std::vector<void*> out(l.numel.size());
    for (Py_ssize_t j = 0; j < T; ++j) {
        if (items[j] == Py_None) {
            if (other && other[j] != Py_None) throw Bad{where, j};
            continue;
        }
        out[j] = address(items[j], static_cast<at::ScalarType>(types[j]), l.numel[j], l.device, Bad{where, j});
    }
    return out;
}

const List& list_of(PyObject* capsule)
{
    const void* l = PyCapsule_CheckExact(capsule) ? PyCapsule_GetPointer(capsule, kListName) : nullptr;
    if (!l) throw std::invalid_argument("the list of tensors is destroyed");
    return *static_cast<const List*>(l);
}

// f() with the mistakes of a call's arguments turned into what Python sees
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f)
{
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const Bad& b) {
        return PyErr_Occurred() ? nullptr : b.code();   // a number that was none comes first
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
}

// The library's call, without the interpreter's lock (a launch may wait for room in its queue).
template <class F>
PyObject* status_of(F&& call)
{
    if (PyErr_Occurred()) return nullptr;   // an address that was no number
    ob_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
}

hipStream_t stream_of(PyObject* s) { return static_cast<hipStream_t>(PyLong_AsVoidPtr(s)); }
const ob_adamw_hparams* hparams_of(PyObject* h)
{
    return h == Py_None ? nullptr : static_cast<const ob_adamw_hparams*>(PyLong_AsVoidPtr(h));
}
ob_control* control_of(PyObject* c, const List& l, int64_t where)
{
    return static_cast<ob_control*>(flat(c, at::kInt, OB_CONTROL_BYTES / 4, l.device, where));
}

// list(handle, numels, g_types, p_types, device, state_elems): a capsule for the calls below
PyObject* list(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject* {
        auto l = std::make_unique<List>();
        l->handle = static_cast<ob_tensors>(PyLong_AsVoidPtr(args[0]));
        if (!PyTuple_Check(args[1]) || !PyBytes_Check(args[2]) || !PyBytes_Check(args[3]) ||
            PyBytes_GET_SIZE(args[2]) != PyTuple_GET_SIZE(args[1]) || PyBytes_GET_SIZE(args[3]) != PyTuple_GET_SIZE(args[1]))
            throw std::invalid_argument("element counts and types of one length are needed");
        for (Py_ssize_t j = 0; j < PyTuple_GET_SIZE(args[1]); ++j)
            l->numel.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], j)));
        l->g_types.assign(PyBytes_AS_STRING(args[2]), l->numel.size());
        l->p_types.assign(PyBytes_AS_STRING(args[3]), l->numel.size());
        l->device = PyLong_AsLong(args[4]);
        l->state_elems = PyLong_AsLongLong(args[5]);
        if (PyErr_Occurred()) return nullptr;
        PyObject* c = PyCapsule_New(l.get(), kListName, [](PyObject* self) {
            delete static_cast<List*>(PyCapsule_GetPointer(self, kListName));
        });
        if (c) l.release();
        return c;
    });
}

// The norm that a step's call takes first, by a pair (g_mult, max_norm) or None.
struct Norm {
    bool on;
    float g_mult = 1.0f, max_norm = 0.0f;
    explicit Norm(PyObject* pair) : on(pair != Py_None)
    {
        if (!on) return;
        if (!PyTuple_Check(pair) || PyTuple_GET_SIZE(pair) != 2) throw std::invalid_argument("norm must be (g_mult, max_norm)");
        g_mult = static_cast<float>(PyFloat_AsDouble(PyTuple_GET_ITEM(pair, 0)));
        max_norm = static_cast<float>(PyFloat_AsDouble(PyTuple_GET_ITEM(pair, 1)));
    }
    // check, then the norm (which counts the step) and the step: what the step refuses is not counted
    template <class Check, class Step>
    ob_status with(const List& l, const std::vector<void*>& g, const ob_adamw_hparams* hp, ob_control* ctl, hipStream_t s,
                   Check&& check, Step&& step) const
    {
        if (on) {
            if (ob_status st = check()) return st;
            if (ob_status st = ob_grad_norm(l.handle, g.data(), g_mult, max_norm, hp, ctl, s)) return st;
        }
        return step();
    }
};

// grad_norm(list, grads, g_mult, max_norm, hparams' address or None, control, stream)
PyObject* grad_norm(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        const List& l = list_of(args[0]);
        const std::vector<void*> g = addresses(args[1], nullptr, l, l.g_types, 0);
        const float g_mult = static_cast<float>(PyFloat_AsDouble(args[2])), max_norm = static_cast<float>(PyFloat_AsDouble(args[3]));
        const ob_adamw_hparams* hp = hparams_of(args[4]);
        ob_control* ctl = control_of(args[5], l, 2);
        hipStream_t s = stream_of(args[6]);
        return status_of([&] { return ob_grad_norm(l.handle, g.data(), g_mult, max_norm, hp, ctl, s); });
    });
}

// adamw_step(list, grads, params, hparams' address, stream, master, m, v, control, norm)
PyObject* adamw_step(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 10, [&] {
        const List& l = list_of(args[0]);
        const std::vector<void*> g = addresses(args[1], nullptr, l, l.g_types, 0);
        const std::vector<void*> p = addresses(args[2], args[1], l, l.p_types, 1);
        const ob_adamw_hparams* hp = hparams_of(args[3]);
        hipStream_t s = stream_of(args[4]);
        float* f[3];
        for (int j = 0; j < 3; ++j) f[j] = static_cast<float*>(flat(args[5 + j], at::kFloat, l.state_elems, l.device, 2 + j));
        ob_control* ctl = control_of(args[8], l, 5);
        const Norm norm(args[9]);
        return status_of([&] {
            return norm.with(
                l, g, hp, ctl, s, [&] { return ob_adamw_check(l.handle, g.data(), p.data(), f[0], f[1], f[2], hp, ctl); },
                [&] { return ob_adamw_step(l.handle, g.data(), p.data(), f[0], f[1], f[2], hp, ctl, s); });
        });
    });
}

// adamw8_step(list, grads, params, hparams' address, stream, master, m_codes, m_scales, v_codes, v_scales, control, norm)
PyObject* adamw8_step(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 12, [&] {
        const List& l = list_of(args[0]);
        const std::vector<void*> g = addresses(args[1], nullptr, l, l.g_types, 0);
        const std::vector<void*> p = addresses(args[2], args[1], l, l.p_types, 1);
        const ob_adamw_hparams* hp = hparams_of(args[3]);
        hipStream_t s = stream_of(args[4]);
        const int64_t N = l.state_elems, B = N / OB_STATE_BLOCK;
        auto* master = static_cast<float*>(flat(args[5], at::kFloat, N, l.device, 2));
        auto* mc = static_cast<int8_t*>(flat(args[6], at::kChar, N, l.device, 3));
        auto* mq = static_cast<float*>(flat(args[7], at::kFloat, B, l.device, 4));
        auto* vc = static_cast<uint8_t*>(flat(args[8], at::kByte, N, l.device, 5));
        auto* vq = static_cast<float*>(flat(args[9], at::kFloat, B, l.device, 6));
        ob_control* ctl = control_of(args[10], l, 7);
        const Norm norm(args[11]);
        return status_of([&] {
            return norm.with(
                l, g, hp, ctl, s, [&] { return ob_adamw8_check(l.handle, g.data(), p.data(), master, mc, mq, vc, vq, hp, ctl); },
                [&] { return ob_adamw8_step(l.handle, g.data(), p.data(), master, mc, mq, vc, vq, hp, ctl, s); });
        });
    });
}

// state8(encode, n, device, stream, m, v, m_codes, m_scales, v_codes, v_scales): a conversion on the current device
PyObject* state8(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 10, [&] {
        const int64_t N = PyLong_AsLongLong(args[1]), B = (N + OB_STATE_BLOCK - 1) / OB_STATE_BLOCK;
        const long device = PyLong_AsLong(args[2]);
        hipStream_t s = stream_of(args[3]);
        auto* m = static_cast<float*>(flat(args[4], at::kFloat, N, device, 2));
        auto* v = static_cast<float*>(flat(args[5], at::kFloat, N, device, 3));
        auto* mc = static_cast<int8_t*>(flat(args[6], at::kChar, N, device, 4));
        auto* mq = static_cast<float*>(flat(args[7], at::kFloat, B, device, 5));
        auto* vc = static_cast<uint8_t*>(flat(args[8], at::kByte, N, device, 6));
        auto* vq = static_cast<float*>(flat(args[9], at::kFloat, B, device, 7));
        const bool encode = args[0] == Py_True;
        return status_of([&] {
            return encode ? ob_state8_encode(N, m, v, mc, mq, vc, vq, s) : ob_state8_decode(N, mc, mq, vc, vq, m, v, s);
        });
    });
}

// scalar_type(dtype): its code in the type strings of list()
PyObject* scalar_type(PyObject*, PyObject* dtype)
{
    if (!THPDtype_Check(dtype)) {
        PyErr_SetString(PyExc_TypeError, "expected a torch.dtype");
        return nullptr;
    }
    return PyLong_FromLong(static_cast<long>(reinterpret_cast<THPDtype*>(dtype)->scalar_type));
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef fast(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {fast<list>("list"),
                         fast<grad_norm>("grad_norm"),
                         fast<adamw_step>("adamw_step"),
                         fast<adamw8_step>("adamw8_step"),
                         fast<state8>("state8"),
                         {"scalar_type", scalar_type, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_obtorch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__obtorch(void) { return PyModule_Create(&module); }
