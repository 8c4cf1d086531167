// Python entries of the calls of a decoding step: sptp_rope,
// sptp_rope_append_kv, sptp_paged_attn_decode (with and without a cap or slopes),
// sptp_paged_attn_prompt and sptp_lora.
//
// Those calls last 2 to 8 us on the device, and reading the shapes, types and
// addresses of their 4 to 12 tensors one attribute at a time from Python takes
// longer than that: rotation, append and attention cost 5.3, 7.5 and 9.4 us a
// call that way and 2.5, 2.7 and 4.4 us this way, of which 1.4, 1.4 and 2.9 are
// the launches; prompts' attention 10.1 and 4.6, adapters 10.9 and 3.7.
//
// The entries here take only calls that are right as they stand: tensors of the
// expected shapes and types, dense, on the current device.  Anything else, an
// error of the library included, returns NotImplemented, and the caller's own
// checks, which name what is wrong, then make the same call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "sptp.h"

namespace {

// of the library in use
int (*rope_call)(const sptp_rope_args*) = nullptr;
int (*append_call)(const sptp_rope_append_kv_args*) = nullptr;
int (*decode_call)(const sptp_paged_attn_decode_args*) = nullptr;
int (*decode_ex_call)(const sptp_paged_attn_decode_args*, float, const float*) = nullptr;
int (*prompt_call)(const sptp_paged_attn_prompt_args*) = nullptr;
decltype(&sptp_lora_ex) lora_call = nullptr;

struct Unfit {};  // thrown: not a call for these entries

void need(bool ok) {
    if (!ok) throw Unfit{};
}

const at::Tensor* tensor_or_none(PyObject* o) {
    if (o == Py_None) return nullptr;
    need(THPVariable_Check(o));
    return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o) {
    const at::Tensor* t = tensor_or_none(o);
    need(t != nullptr);
    return *t;
}

int integer(PyObject* o) {
    need(PyLong_Check(o));
    int overflow = 0;
    const long v = PyLong_AsLongAndOverflow(o, &overflow);
    need(overflow == 0 && v >= INT_MIN && v <= INT_MAX);
    return static_cast<int>(v);
}

float real(PyObject* o) {
    need(PyFloat_Check(o) || PyLong_Check(o));
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unfit{};
    }
    const float f = static_cast<float>(v);
    need(std::fabs(v) <= FLT_MAX && (f != 0.f) == (v != 0.0));
    return f;
}

int size(int64_t n) {
    need(n <= INT_MAX);
    return static_cast<int>(n);
}

void has_shape(const at::Tensor& t, std::initializer_list<int64_t> shape) {
    need(t.sizes() == at::IntArrayRef(shape));
}

int dtype_code(const at::Tensor& t) {
    const at::ScalarType d = t.scalar_type();
    need(d == at::kBFloat16 || d == at::kFloat);
    return d == at::kBFloat16 ? SPTP_BF16 : SPTP_FP32;
}

// Dense, on device `dev`; its address.
template <typename T = void>
T* data(const at::Tensor& t, int dev) {
    need(t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided && t.is_contiguous());
    return static_cast<T*>(t.data_ptr());
}

// The current device, which the tensors of a call have to be on.
int device_for(const at::Tensor& t) {
    need(t.is_cuda());
    return c10::cuda::current_device();
}

// An output: the caller's, or a new one.
struct Out {
    at::Tensor own;
    PyObject* given = nullptr;
    void* at;

    Out(PyObject* o, const at::Tensor& like, at::ScalarType dtype, std::initializer_list<int64_t> shape, int dev) {
        if (const at::Tensor* t = tensor_or_none(o)) {
            need(t->scalar_type() == dtype);
            has_shape(*t, shape);
            given = o;
            at = data(*t, dev);
        } else {
            own = at::empty(at::IntArrayRef(shape), like.options().dtype(dtype));
            at = own.data_ptr();
        }
    }
    PyObject* object() { return given ? Py_NewRef(given) : THPVariable_Wrap(own); }
};

// The page pool and its sizes.
struct Cache {
    void *k, *v, *k_scale = nullptr, *v_scale = nullptr;
    int num_pages, heads, page_size, D, kv_type;

    Cache(PyObject* o, int P, at::ScalarType dtype, int dev) {
        need(PyTuple_CheckExact(o) && PyTuple_GET_SIZE(o) == 4);
        const at::Tensor &tk = tensor(PyTuple_GET_ITEM(o, 0)), &tv = tensor(PyTuple_GET_ITEM(o, 1));
        const at::Tensor *ks = tensor_or_none(PyTuple_GET_ITEM(o, 2)), *vs = tensor_or_none(PyTuple_GET_ITEM(o, 3));
        const at::ScalarType kind = tk.scalar_type();
        need(tk.dim() == 5 && tk.size(0) == P && tv.sizes() == tk.sizes() && tv.scalar_type() == kind);
        if (kind == dtype) {
            need(ks == nullptr && vs == nullptr);
            kv_type = SPTP_KV_SAME;
        } else {
            need(kind == at::kByte && dtype == at::kBFloat16 && ks != nullptr && vs != nullptr);
            need(ks->scalar_type() == at::kFloat && vs->scalar_type() == at::kFloat);
            need(ks->sizes() == tk.sizes().slice(0, 4) && vs->sizes() == ks->sizes());
            k_scale = data(*ks, dev);
            v_scale = data(*vs, dev);
            kv_type = SPTP_KV_E4M3;
        }
        num_pages = size(tk.size(1));
        heads = size(tk.size(2));
        page_size = size(tk.size(3));
        D = size(tk.size(4));
        k = data(tk, dev);
        v = data(tv, dev);
    }
};

// Makes the call without the interpreter's lock: a full launch queue waits here.
template <typename F, typename... Args>
void make(F call, Args... args) {
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = call(args...);
    Py_END_ALLOW_THREADS;
    need(rc == SPTP_OK);
}

// The out and lse of an attention: (out, lse, write_lse) at o[0], o[1], o[2].
struct Outs {
    Out out;
    PyObject* lse = nullptr;
    float* lse_at = nullptr;

    Outs(PyObject* o_out, PyObject* o_lse, PyObject* write, const at::Tensor& q, int P, int rows, int Hq, int D, int dev)
        : out(o_out, q, q.scalar_type(), {P, rows, static_cast<int64_t>(Hq) * D}, dev) {
        if (o_lse == Py_None && write == Py_False) {
            lse = Py_NewRef(Py_None);
        } else {
            need(o_lse != Py_None || write == Py_True);
            Out l(o_lse, q, at::kFloat, {P, rows, Hq}, dev);
            lse_at = static_cast<float*>(l.at);
            lse = l.object();
        }
    }
    ~Outs() { Py_XDECREF(lse); }
    PyObject* object() {
        PyObject* l = lse;
        lse = nullptr;
        return Py_BuildValue("(NN)", out.object(), l);
    }
};

// fp32 slopes [P][Hq], or none
const float* slopes_of(PyObject* o, int P, int Hq, int dev) {
    const at::Tensor* t = tensor_or_none(o);
    if (t == nullptr) return nullptr;
    need(t->scalar_type() == at::kFloat);
    has_shape(*t, {P, Hq});
    return data<const float>(*t, dev);
}

// (x, positions, turns, Hr, interleaved, transpose, gain, out)
PyObject* rope(PyObject* const* o) {
    const at::Tensor &x = tensor(o[0]), &positions = tensor(o[1]), &turns = tensor(o[2]);
    const int dev = device_for(x);
    need(x.dim() == 4 && turns.dim() == 1 && turns.scalar_type() == at::kLong && positions.scalar_type() == at::kInt);
    has_shape(positions, {x.size(1)});
    sptp_rope_args a;
    a.P = size(x.size(0));
    a.M = size(x.size(1));
    a.H = size(x.size(2));
    a.D = size(x.size(3));
    a.Hr = o[3] == Py_None ? a.H : integer(o[3]);
    a.rot = size(2 * turns.size(0));
    a.interleaved = integer(o[4]);
    a.transpose = integer(o[5]);
    a.gain = real(o[6]);
    a.dtype = dtype_code(x);
    a.x = data(x, dev);
    a.positions = data(positions, dev);
    a.turns = data(turns, dev);
    Out out(o[7], x, x.scalar_type(), {a.P, a.M, a.H, a.D}, dev);
    a.out = out.at;
    a.cuda_stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    make(rope_call, &a);
    return out.object();
}

// (qkv, positions, seq_ids, page_table, turns, cache, Hq, interleaved, gain, q_out, workspace)
PyObject* append(PyObject* const* o) {
    const at::Tensor &qkv = tensor(o[0]), &positions = tensor(o[1]), &seq_ids = tensor(o[2]), &table = tensor(o[3]);
    const at::Tensor *turns = tensor_or_none(o[4]), &ws = tensor(o[10]);
    const int dev = device_for(qkv);
    need(qkv.dim() == 3 && table.dim() == 2 && positions.scalar_type() == at::kInt &&
         seq_ids.scalar_type() == at::kInt && table.scalar_type() == at::kInt);
    need(turns == nullptr || (turns->dim() == 1 && turns->scalar_type() == at::kLong));
    sptp_rope_append_kv_args a;
    a.P = size(qkv.size(0));
    a.M = size(qkv.size(1));
    has_shape(positions, {a.M});
    has_shape(seq_ids, {a.M});
    const Cache c(o[5], a.P, qkv.scalar_type(), dev);
    a.Hq = integer(o[6]);
    a.Hkv = c.heads;
    a.D = c.D;
    need(qkv.size(2) == (a.Hq + 2ll * a.Hkv) * a.D);
    a.rot = turns ? size(2 * turns->size(0)) : 0;
    a.interleaved = integer(o[7]);
    a.gain = real(o[8]);
    a.B = size(table.size(0));
    a.max_pages = size(table.size(1));
    a.num_pages = c.num_pages;
    a.page_size = c.page_size;
    a.dtype = dtype_code(qkv);
    a.kv_type = c.kv_type;
    a.qkv = data(qkv, dev);
    a.positions = data(positions, dev);
    a.seq_ids = data(seq_ids, dev);
    a.page_table = data(table, dev);
    a.turns = turns ? data(*turns, dev) : nullptr;
    a.k_cache = c.k;
    a.v_cache = c.v;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.workspace = data(ws, dev);
    a.ws_bytes = ws.nbytes();
    need(a.Hq >= 0);
    Out q(o[9], qkv, qkv.scalar_type(), {a.P, a.M, a.Hq, a.D}, dev);
    a.q_out = q.at;
    a.cuda_stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    make(append_call, &a);
    return q.object();
}

// (q, cache, page_table, seq_lens, scale, window, out, lse, workspace, write_lse), and with EX (.., cap, slopes)
template <bool EX>
PyObject* decode(PyObject* const* o) {
    const at::Tensor &q = tensor(o[0]), &table = tensor(o[2]), &lens = tensor(o[3]), &ws = tensor(o[8]);
    const int dev = device_for(q);
    need(q.dim() == 4 && table.dim() == 2 && table.scalar_type() == at::kInt && lens.scalar_type() == at::kInt);
    sptp_paged_attn_decode_args a;
    a.P = size(q.size(0));
    a.B = size(q.size(1));
    a.Hq = size(q.size(2));
    a.D = size(q.size(3));
    const Cache c(o[1], a.P, q.scalar_type(), dev);
    need(c.D == a.D && table.size(0) == a.B);
    has_shape(lens, {a.B});
    a.Hkv = c.heads;
    a.max_pages = size(table.size(1));
    a.num_pages = c.num_pages;
    a.page_size = c.page_size;
    a.scale = o[4] == Py_None ? static_cast<float>(std::pow(a.D, -0.5)) : real(o[4]);
    a.window = integer(o[5]);
    a.dtype = dtype_code(q);
    a.kv_type = c.kv_type;
    a.q = data(q, dev);
    a.k_cache = c.k;
    a.v_cache = c.v;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.page_table = data(table, dev);
    a.seq_lens = data(lens, dev);
    a.workspace = data(ws, dev);
    a.ws_bytes = ws.nbytes();
    const float cap = EX ? real(o[10]) : 0.f;
    const float* slopes = EX ? slopes_of(o[11], a.P, a.Hq, dev) : nullptr;
    Outs outs(o[6], o[7], o[9], q, a.P, a.B, a.Hq, a.D, dev);
    a.out = outs.out.at;
    a.lse = outs.lse_at;
    a.cuda_stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    if constexpr (EX) {
        need(decode_ex_call != nullptr);
        make(decode_ex_call, &a, cap, slopes);
    } else {
        make(decode_call, &a);
    }
    return outs.object();
}

// (q, cache, page_table, seq_lens, row_starts, scale, window, cap, slopes, prefix_lens, out, lse, workspace, write_lse)
PyObject* prompt(PyObject* const* o) {
    const at::Tensor &q = tensor(o[0]), &table = tensor(o[2]), &lens = tensor(o[3]), &starts = tensor(o[4]), &ws = tensor(o[12]);
    const at::Tensor* prefixes = tensor_or_none(o[9]);
    const int dev = device_for(q);
    need(q.dim() == 4 && table.dim() == 2 && table.scalar_type() == at::kInt && lens.scalar_type() == at::kInt &&
         starts.scalar_type() == at::kInt && prompt_call != nullptr);
    sptp_paged_attn_prompt_args a;
    a.P = size(q.size(0));
    a.M = size(q.size(1));
    a.Hq = size(q.size(2));
    a.D = size(q.size(3));
    a.B = size(table.size(0));
    const Cache c(o[1], a.P, q.scalar_type(), dev);
    need(c.D == a.D);
    has_shape(lens, {a.B});
    has_shape(starts, {a.B + 1ll});
    if (prefixes != nullptr) {
        need(prefixes->scalar_type() == at::kInt);
        has_shape(*prefixes, {a.B});
    }
    a.Hkv = c.heads;
    a.max_pages = size(table.size(1));
    a.num_pages = c.num_pages;
    a.page_size = c.page_size;
    a.scale = o[5] == Py_None ? static_cast<float>(std::pow(a.D, -0.5)) : real(o[5]);
    a.window = integer(o[6]);
    a.cap = real(o[7]);
    a.dtype = dtype_code(q);
    a.kv_type = c.kv_type;
    a.q = data(q, dev);
    a.k_cache = c.k;
    a.v_cache = c.v;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.page_table = data(table, dev);
    a.seq_lens = data(lens, dev);
    a.row_starts = data(starts, dev);
    a.prefix_lens = prefixes ? data(*prefixes, dev) : nullptr;
    a.slopes = slopes_of(o[8], a.P, a.Hq, dev);
    a.workspace = data(ws, dev);
    a.ws_bytes = ws.nbytes();
    Outs outs(o[10], o[11], o[13], q, a.P, a.M, a.Hq, a.D, dev);
    a.out = outs.out.at;
    a.lse = outs.lse_at;
    a.cuda_stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    make(prompt_call, &a);
    return outs.object();
}

// (x, A, B, ids, base, gains, out, workspace, status_workspace, check_only)
PyObject* lora(PyObject* const* o) {
    const at::Tensor &x = tensor(o[0]), &A = tensor(o[1]), &B = tensor(o[2]), &ids = tensor(o[3]), &base = tensor(o[4]),
                     &ws = tensor(o[7]);
    const at::Tensor *gains = tensor_or_none(o[5]), *status = tensor_or_none(o[8]);
    need(o[9] == Py_False || o[9] == Py_True);
    const int dev = device_for(x);
    const at::ScalarType type = x.scalar_type();
    need((x.dim() == 2 || x.dim() == 3) && A.dim() == 3 && B.dim() == 3 && base.dim() == 3 && lora_call != nullptr);
    need(A.scalar_type() == type && B.scalar_type() == type && base.scalar_type() == type && ids.scalar_type() == at::kInt);
    const bool rowwise = x.dim() == 3;
    const int adapters = size(A.size(0)), R = size(A.size(1)), K = size(A.size(2)), N = size(B.size(1));
    const int P = size(base.size(0)), M = size(x.size(x.dim() - 2));
    need(P >= 1 && (rowwise ? K : N) % P == 0);
    const int n = rowwise ? N : N / P;
    has_shape(B, {adapters, N, R});
    has_shape(ids, {M});
    has_shape(base, {P, M, n});
    if (rowwise)
        has_shape(x, {P, M, K / P});
    else
        has_shape(x, {M, K});
    if (gains != nullptr) {
        need(gains->scalar_type() == at::kFloat);
        has_shape(*gains, {adapters});
    }
    const sptp_dtype dtype = static_cast<sptp_dtype>(dtype_code(x));
    void *xp = data(x, dev), *Ap = data(A, dev), *Bp = data(B, dev), *bp = data(base, dev), *wp = data(ws, dev);
    const int* ip = data<const int>(ids, dev);
    const float* gp = gains ? data<const float>(*gains, dev) : nullptr;
    void* sp = status ? data(*status, dev) : nullptr;
    Out out(o[6], x, type, {P, M, n}, dev);
    make(lora_call, xp, Ap, Bp, ip, gp, P, M, K, N, R, adapters, rowwise ? 1 : 0, dtype, bp, out.at, wp, ws.nbytes(),
         static_cast<void*>(c10::cuda::getCurrentCUDAStream(dev).stream()), sp, o[9] == Py_True ? 1 : 0);
    return out.object();
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n == N && rope_call != nullptr) {
        try {
            return F(args);
        } catch (...) {
            PyErr_Clear();
        }
    }
    Py_RETURN_NOTIMPLEMENTED;
}

bool addresses(PyObject* const* args, Py_ssize_t n, void* (&p)[3]) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "three addresses expected");
        return false;
    }
    for (int i = 0; i < 3; ++i)
        if ((p[i] = PyLong_AsVoidPtr(args[i])) == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address of 0");
            return false;
        }
    return true;
}

// Addresses of the library's calls: (sptp_rope_packed, sptp_rope_append_kv_packed, sptp_paged_attn_decode_packed).
PyObject* use(PyObject*, PyObject* const* args, Py_ssize_t n) {
    void* p[3];
    if (!addresses(args, n, p)) return nullptr;
    rope_call = reinterpret_cast<decltype(rope_call)>(p[0]);
    append_call = reinterpret_cast<decltype(append_call)>(p[1]);
    decode_call = reinterpret_cast<decltype(decode_call)>(p[2]);
    Py_RETURN_NONE;
}

// And of (sptp_paged_attn_decode_ex, sptp_paged_attn_prompt, sptp_lora_ex).
PyObject* use_batch(PyObject*, PyObject* const* args, Py_ssize_t n) {
    void* p[3];
    if (!addresses(args, n, p)) return nullptr;
    decode_ex_call = reinterpret_cast<decltype(decode_ex_call)>(p[0]);
    prompt_call = reinterpret_cast<decltype(prompt_call)>(p[1]);
    lora_call = reinterpret_cast<decltype(lora_call)>(p[2]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__decode_binding() {
    static PyMethodDef methods[] = {
        {"use", method(use), METH_FASTCALL, nullptr},
        {"rope", method(entry<rope, 8>), METH_FASTCALL, nullptr},
        {"append", method(entry<append, 11>), METH_FASTCALL, nullptr},
        {"decode", method(entry<decode<false>, 10>), METH_FASTCALL, nullptr},
        {"use_batch", method(use_batch), METH_FASTCALL, nullptr},
        {"decode_ex", method(entry<decode<true>, 12>), METH_FASTCALL, nullptr},
        {"prompt", method(entry<prompt, 14>), METH_FASTCALL, nullptr},
        {"lora", method(entry<lora, 10>), METH_FASTCALL, nullptr},
        {nullptr, nullptr, 0, nullptr},
    };
    static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode_binding", nullptr, -1, methods};
    return PyModule_Create(&module);
}
