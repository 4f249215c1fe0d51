// binding.cpp -- the Python side of the operators around the state pool: torch tensors checked and
// handed to the C ABI (include/gdn2.h).
//
// The rest of the package binds the ABI over ctypes. These operators are called once per decode step,
// and for one sequence a step takes 3 to 7 us on the GPU: the same checks in Python and a ctypes
// call of up to 17 arguments took 9 to 15 us, these take about 4, launch included. Every function
// checks each tensor's type, device, shape and layout before the library is called, makes the tensors'
// device current, allocates missing outputs on the call's stream, and raises what the package's
// other functions raise. Nothing is kept between calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <optional>
#include <string>

#include "gdn2.h"

namespace {

// The library's functions, from the library that the package has loaded, and the class of its errors.
decltype(&gdn2_state_store) p_store;
decltype(&gdn2_state_load) p_load;
decltype(&gdn2_decode_multi_q8) p_decode;
decltype(&gdn2_decode_multi_q8_prologue) p_decode_prologue;
decltype(&gdn2_verify_drafts) p_verify;
decltype(&gdn2_state_commit) p_commit;
decltype(&gdn2_state_commit_q8) p_commit_q8;
decltype(&gdn2_last_error_string) p_error;
PyObject* error_class;

struct Raised {};  // a Python error is set
[[noreturn]] void raise(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Raised();
}

using Sizes = std::initializer_list<int64_t>;

template <class S>
std::string text(const S& sizes) {
    std::string s = "(";
    size_t n = 0;
    for (int64_t x : sizes) s += (n++ ? ", " : "") + std::to_string(x);
    return s + (n == 1 ? ",)" : ")");
}

const char* name_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kChar: return "torch.int8";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        default: return nullptr;
    }
}
std::string dtype_of(PyObject* o) {
    if (const char* n = name_of(THPVariable_Unpack(o).scalar_type())) return n;
    PyObject* d = PyObject_GetAttrString(o, "dtype");
    PyObject* s = d ? PyObject_Str(d) : nullptr;
    const char* c = s ? PyUnicode_AsUTF8(s) : nullptr;
    std::string r = c ? c : "?";
    Py_XDECREF(s);
    Py_XDECREF(d);
    PyErr_Clear();
    return r;
}
std::string device_name(at::Device d) { return "cuda:" + std::to_string((int)d.index()); }

const at::Tensor& cuda_tensor(const char* name, PyObject* o, const char* layout = "") {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor" + layout);
    return THPVariable_Unpack(o);
}

int to_int(const char* name, int64_t x) {
    if (x > INT_MAX) raise(PyExc_ValueError, std::string(name) + " = " + std::to_string(x) + " is above 2^31 - 1");
    return (int)x;
}

// The address of a tensor that the call needs at this shape, dense, of this type, on this device; null for None
// where that is allowed.
void* at_shape(const char* name, PyObject* o, Sizes sizes, at::ScalarType type, at::Device device, bool optional = false) {
    if (o == Py_None) {
        if (optional) return nullptr;
        raise(PyExc_ValueError, std::string(name) + " is required");
    }
    const at::Tensor& t = cuda_tensor(name, o);
    if (t.sizes() != at::IntArrayRef(sizes.begin(), sizes.size()))
        raise(PyExc_ValueError, std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(sizes));
    if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    if (t.scalar_type() != type) raise(PyExc_TypeError, std::string(name) + " is " + dtype_of(o) + ", expected " + name_of(type));
    if (t.device() != device) raise(PyExc_ValueError, std::string(name) + " is on " + device_name(t.device()) + ", expected " + device_name(device));
    return t.data_ptr();
}

int dtype_code(PyObject* o) {
    const at::ScalarType t = THPVariable_Unpack(o).scalar_type();
    if (t == at::kBFloat16) return GDN2_BF16;
    if (t == at::kFloat) return GDN2_F32;
    raise(PyExc_TypeError, "unsupported element type " + dtype_of(o) + "; use bfloat16 or float32");
}

// The call's device made current, and its stream: the one given, or the device's current one.
struct On {
    c10::cuda::CUDAGuard device;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    cudaStream_t stream;
    On(at::Device d, PyObject* given) : device(d) {
        if (given == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
            return;
        }
        PyObject* dev = PyObject_GetAttrString(given, "device");
        PyObject* index = dev ? PyObject_GetAttrString(dev, "index") : nullptr;
        const long i = index ? PyLong_AsLong(index) : -1;
        Py_XDECREF(index);
        Py_XDECREF(dev);
        if (PyErr_Occurred()) throw Raised();
        if (i != d.index()) raise(PyExc_ValueError, "stream is on cuda:" + std::to_string(i) + ", the tensors on " + device_name(d));
        PyObject* handle = PyObject_GetAttrString(given, "cuda_stream");
        stream = handle ? static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle)) : nullptr;
        Py_XDECREF(handle);
        if (PyErr_Occurred()) throw Raised();
        guard.emplace(c10::cuda::getStreamFromExternal(stream, d.index()));
    }
    gdn2_stream_t get() const { return reinterpret_cast<gdn2_stream_t>(stream); }
};

template <class F>
void call(F&& f) {
    gdn2_status st;
    std::string what;
    Py_BEGIN_ALLOW_THREADS;
    st = f();
    if (st != GDN2_OK) what = p_error();
    Py_END_ALLOW_THREADS;
    if (st == GDN2_OK) return;
    PyObject* e = PyObject_CallFunction(error_class, "is", (int)st, what.c_str());
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    throw Raised();
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, at::Device device) {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
}
PyObject* given_or(PyObject* o, at::Tensor& made) {
    if (o == Py_None && made.defined()) return THPVariable_Wrap(made);
    Py_INCREF(o);
    return o;
}

// Codes [n_slots, Hv, dk, dv] and scales [n_slots, Hv, dk] of an 8-bit pool.
struct Pool {
    at::ScalarType type;
    gdn2_q8_format format;
    int n_slots, h, dk, dv;
    at::Device device;
    void* codes;
    float* scales;
    Pool(PyObject* c, PyObject* s) : device(at::kCUDA) {
        const char* layout = " [n_slots, Hv, dk, dv]";
        const at::Tensor& t = cuda_tensor("codes", c, layout);
        if (t.dim() != 4) raise(PyExc_ValueError, std::string("codes must be a CUDA tensor") + layout);
        type = t.scalar_type();
        if (type != at::kChar && type != at::kFloat8_e4m3fn)
            raise(PyExc_TypeError, "codes is " + dtype_of(c) + ", expected torch.int8 or torch.float8_e4m3fn");
        format = type == at::kChar ? GDN2_Q8_INT8 : GDN2_Q8_E4M3;
        device = t.device();
        n_slots = to_int("n_slots", t.size(0));
        h = to_int("Hv", t.size(1));
        dk = to_int("dk", t.size(2));
        dv = to_int("dv", t.size(3));
        codes = at_shape("codes", c, {n_slots, h, dk, dv}, type, device);
        scales = static_cast<float*>(at_shape("scales", s, {n_slots, h, dk}, at::kFloat, device));
    }
};

int64_t size0(PyObject* o) {
    if (!THPVariable_Check(o)) return 0;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.dim() ? t.size(0) : 0;
}
int32_t* ints(const char* name, PyObject* o, Sizes sizes, at::Device d, bool optional) {
    return static_cast<int32_t*>(at_shape(name, o, sizes, at::kInt, d, optional));
}
float* floats(const char* name, PyObject* o, Sizes sizes, at::Device d, bool optional = false) {
    return static_cast<float*>(at_shape(name, o, sizes, at::kFloat, d, optional));
}

// ---------------------------------------------------------------- the functions
// (S, codes, scales, slots, stream)
PyObject* store(PyObject* const* a) {
    const Pool p(a[1], a[2]);
    const int n = to_int("N", size0(a[0]));
    const float* S = floats("S", a[0], {n, p.h, p.dk, p.dv}, p.device);
    const int32_t* slots = ints("slots", a[3], {n}, p.device, true);
    const On on(p.device, a[4]);
    call([&] { return p_store(n, p.h, p.dk, p.dv, p.format, S, slots, p.codes, p.scales, p.n_slots, on.get()); });
    return PyTuple_Pack(2, a[1], a[2]);
}

// (codes, scales, slots, n_seq, S, stream)
PyObject* load(PyObject* const* a) {
    const Pool p(a[0], a[1]);
    int64_t n = a[2] != Py_None ? size0(a[2]) : a[4] != Py_None ? size0(a[4]) : p.n_slots;
    if (a[3] != Py_None) {
        const long long m = PyLong_AsLongLong(a[3]);
        if (PyErr_Occurred()) throw Raised();
        if ((a[2] != Py_None || a[4] != Py_None) && m != n)
            raise(PyExc_ValueError, "n_seq = " + std::to_string(m) + ", but slots or S has " + std::to_string(n) + " sequences");
        n = m;
    }
    if (n < 0) raise(PyExc_ValueError, "n_seq = " + std::to_string(n) + " is negative");
    const int N = to_int("N", n);
    const int32_t* slots = ints("slots", a[2], {N}, p.device, true);
    float* S = floats("S", a[4], {N, p.h, p.dk, p.dv}, p.device, true);
    const On on(p.device, a[5]);
    at::Tensor made;
    if (!S) {
        made = empty({N, p.h, p.dk, p.dv}, at::kFloat, p.device);
        S = made.mutable_data_ptr<float>();
    }
    call([&] { return p_load(N, p.h, p.dk, p.dv, p.format, p.codes, p.scales, p.n_slots, slots, S, on.get()); });
    return given_or(a[4], made);
}

// (q, k, v, log_alpha, b, w, codes, scales, slots, slots_out, o, code_steps, scale_steps, want_steps, stream,
//  code of the output type, prologue)
PyObject* decode(PyObject* const* a) {
    const Pool p(a[6], a[7]);
    const at::Device d = p.device;
    for (int i : {0, 2}) {
        const char* name = i ? "v" : "q";
        const at::Tensor& t = cuda_tensor(name, a[i]);
        if (t.dim() != 4) raise(PyExc_ValueError, std::string(name) + " has shape " + text(t.sizes()) + ", expected (N, n_tok) + (heads, channels)");
    }
    const at::Tensor &q = THPVariable_Unpack(a[0]), &v = THPVariable_Unpack(a[2]);
    const int64_t N = v.size(0), n_tok = v.size(1), h = v.size(2), dv = v.size(3), hq = q.size(2), dk = q.size(3);
    const bool prologue = PyObject_IsTrue(a[16]), want = PyObject_IsTrue(a[13]);
    const long oc = PyLong_AsLong(a[15]);
    if (PyErr_Occurred()) throw Raised();
    const at::ScalarType t = q.scalar_type(), ot = oc == GDN2_BF16 ? at::kBFloat16 : at::kFloat;
    const int code = dtype_code(a[0]);
    const void *q_ = at_shape("q", a[0], {N, n_tok, hq, dk}, t, d), *k_ = at_shape("k", a[1], {N, n_tok, hq, dk}, t, d);
    const void *v_ = at_shape("v", a[2], {N, n_tok, h, dv}, t, d);
    const void* la = at_shape("log_alpha", a[3], {N, n_tok, h, dk}, prologue ? t : at::kFloat, d);
    const void *b_ = at_shape("b", a[4], {N, n_tok, h, dk}, t, d), *w_ = at_shape("w", a[5], {N, n_tok, h, dv}, t, d);
    at_shape("codes", a[6], {p.n_slots, h, dk, dv}, p.type, d);
    const int32_t *slots = ints("slots", a[8], {N}, d, true), *slots_out = ints("slots_out", a[9], {N}, d, true);
    void* o = at_shape("o", a[10], {N, n_tok, h, dv}, ot, d, true);
    void* cs = at_shape("code_steps", a[11], {N, n_tok, h, dk, dv}, p.type, d, true);
    float* ss = floats("scale_steps", a[12], {N, n_tok, h, dk}, d, true);
    if ((a[11] == Py_None) != (a[12] == Py_None)) raise(PyExc_ValueError, "code_steps and scale_steps are given together or not at all");
    const gdn2_shape sh{to_int("N", N), to_int("N * n_tok", N * n_tok), to_int("Hqk", hq), p.h, p.dk, p.dv, (gdn2_dtype)code, (gdn2_dtype)oc};
    const On on(d, a[14]);
    at::Tensor mo, mc, ms;
    if (a[10] == Py_None) {
        mo = empty({N, n_tok, h, dv}, ot, d);
        o = mo.mutable_data_ptr();
    }
    if (a[11] == Py_None && want) {
        mc = empty({N, n_tok, h, dk, dv}, p.type, d);
        ms = empty({N, n_tok, h, dk}, at::kFloat, d);
        cs = mc.mutable_data_ptr();
        ss = ms.mutable_data_ptr<float>();
    }
    call([&] {
        return prologue ? p_decode_prologue(&sh, p.format, (int)n_tok, slots, slots_out, q_, k_, v_, la, b_, w_, p.codes, p.scales, p.n_slots, o, cs, ss, on.get())
                        : p_decode(&sh, p.format, (int)n_tok, slots, slots_out, q_, k_, v_, static_cast<const float*>(la), b_, w_, p.codes, p.scales,
                                   p.n_slots, o, cs, ss, on.get());
    });
    PyObject *x = given_or(a[10], mo), *y = given_or(a[11], mc), *z = given_or(a[12], ms);
    return Py_BuildValue("NNN", x, y, z);
}

// (target_probs, draft_probs, draft_tokens, u_accept, u_sample, n_drafted, n_accepted, tokens, stream)
PyObject* verify(PyObject* const* a) {
    const char* layout = " [N, n_draft + 1, V]";
    const at::Tensor& t = cuda_tensor("target_probs", a[0], layout);
    if (t.dim() != 3) raise(PyExc_ValueError, std::string("target_probs must be a CUDA tensor") + layout);
    const at::Device d = t.device();
    const at::ScalarType type = t.scalar_type();
    const int code = dtype_code(a[0]);
    const int64_t N = t.size(0), n1 = t.size(1), V = t.size(2), n = n1 - 1;
    if (n < 0) raise(PyExc_ValueError, "target_probs has no place for a token: its second size is n_draft + 1");
    const void *p_ = at_shape("target_probs", a[0], {N, n1, V}, type, d), *q_ = at_shape("draft_probs", a[1], {N, n, V}, type, d, true);
    const int32_t* drafts = ints("draft_tokens", a[2], {N, n}, d, false);
    const float *u = floats("u_accept", a[3], {N, n}, d), *ul = floats("u_sample", a[4], {N}, d);
    const int32_t* lens = ints("n_drafted", a[5], {N}, d, true);
    int32_t *acc = ints("n_accepted", a[6], {N}, d, true), *tok = ints("tokens", a[7], {N, n1}, d, true);
    const int n_ = to_int("n_draft", n), N_ = to_int("N", N), V_ = to_int("V", V);
    const On on(d, a[8]);
    at::Tensor ma, mt;
    if (a[6] == Py_None) {
        ma = empty({N}, at::kInt, d);
        acc = ma.mutable_data_ptr<int32_t>();
    }
    if (a[7] == Py_None) {
        mt = empty({N, n1}, at::kInt, d);
        tok = mt.mutable_data_ptr<int32_t>();
    }
    call([&] { return p_verify(N_, n_, V_, (gdn2_dtype)code, p_, q_, drafts, lens, u, ul, acc, tok, on.get()); });
    PyObject *x = given_or(a[6], ma), *y = given_or(a[7], mt);
    return Py_BuildValue("NN", x, y);
}

// (S_steps, index, S_pool, slots, stream)
PyObject* commit(PyObject* const* a) {
    const char* layout = " [n_slots, Hv, dk, dv]";
    const at::Tensor& pool = cuda_tensor("S_pool", a[2], layout);
    if (pool.dim() != 4) raise(PyExc_ValueError, std::string("S_pool must be a CUDA tensor") + layout);
    const at::Device d = pool.device();
    const int64_t n_slots = pool.size(0), h = pool.size(1), dk = pool.size(2), dv = pool.size(3);
    const bool five = THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).dim() == 5;
    const int64_t N = five ? THPVariable_Unpack(a[0]).size(0) : 0, n_tok = five ? THPVariable_Unpack(a[0]).size(1) : 0;
    float* P = floats("S_pool", a[2], {n_slots, h, dk, dv}, d);
    const float* steps = floats("S_steps", a[0], {N, n_tok, h, dk, dv}, d);
    const int32_t *index = ints("index", a[1], {N}, d, false), *slots = ints("slots", a[3], {N}, d, true);
    const int n_[6] = {to_int("N", N), to_int("Hv", h), to_int("dk", dk), to_int("dv", dv), to_int("n_tok", n_tok), to_int("n_slots", n_slots)};
    const On on(d, a[4]);
    call([&] { return p_commit(n_[0], n_[1], n_[2], n_[3], n_[4], steps, index, slots, P, n_[5], on.get()); });
    Py_INCREF(a[2]);
    return a[2];
}

// (code_steps, scale_steps, index, codes, scales, slots, stream)
PyObject* commit_q8(PyObject* const* a) {
    const Pool p(a[3], a[4]);
    const bool five = THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).dim() == 5;
    const int64_t N = five ? THPVariable_Unpack(a[0]).size(0) : 0, n_tok = five ? THPVariable_Unpack(a[0]).size(1) : 0;
    const void* cs = at_shape("code_steps", a[0], {N, n_tok, p.h, p.dk, p.dv}, p.type, p.device);
    const float* ss = floats("scale_steps", a[1], {N, n_tok, p.h, p.dk}, p.device);
    const int32_t *index = ints("index", a[2], {N}, p.device, false), *slots = ints("slots", a[5], {N}, p.device, true);
    const int N_ = to_int("N", N), T_ = to_int("n_tok", n_tok);
    const On on(p.device, a[6]);
    call([&] { return p_commit_q8(N_, p.h, p.dk, p.dv, T_, cs, ss, index, slots, p.codes, p.scales, p.n_slots, on.get()); });
    return PyTuple_Pack(2, a[3], a[4]);
}

// (error class, addresses of the library's functions in the order below)
PyObject* init(PyObject* const* a) {
    void* f[8];
    for (int i = 0; i < 8; ++i) {
        f[i] = PyLong_AsVoidPtr(a[1 + i]);
        if (PyErr_Occurred()) throw Raised();
    }
    Py_INCREF(a[0]);
    Py_XSETREF(error_class, a[0]);
    p_store = reinterpret_cast<decltype(p_store)>(f[0]);
    p_load = reinterpret_cast<decltype(p_load)>(f[1]);
    p_decode = reinterpret_cast<decltype(p_decode)>(f[2]);
    p_decode_prologue = reinterpret_cast<decltype(p_decode_prologue)>(f[3]);
    p_verify = reinterpret_cast<decltype(p_verify)>(f[4]);
    p_commit = reinterpret_cast<decltype(p_commit)>(f[5]);
    p_commit_q8 = reinterpret_cast<decltype(p_commit_q8)>(f[6]);
    p_error = reinterpret_cast<decltype(p_error)>(f[7]);
    Py_RETURN_NONE;
}

// A function of exactly kArgs arguments as a Python function; no C++ exception leaves it.
template <PyObject* (*kFunction)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", kArgs, n);
        return nullptr;
    }
    try {
        return kFunction(args);
    } catch (const Raised&) {
    } catch (...) {  // torch's own, out of memory among them
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

template <PyObject* (*kFunction)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kFunction, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<init, 9>("init"),     method<store, 5>("store"),   method<load, 6>("load"),           method<decode, 17>("decode"),
    method<verify, 9>("verify"), method<commit, 5>("commit"), method<commit_q8, 7>("commit_q8"), {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding(void) { return PyModule_Create(&module); }
