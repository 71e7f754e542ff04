// The binding of the operators whose calls a decoding step waits for: arguments are
// checked, outputs and workspaces allocated and the library called without a Python
// statement in between.  A call through ctypes costs the host some 16 us with three
// outputs (1.5 us of them an argument list of 17, 1.5 - 3 an allocation, 0.5 - 0.7 a
// tensor that is checked), a multiple of what the GPU needs for a few rows; here a
// layer norm of a few rows costs it 4.6 us, a linear layer 3.3 to 5.7, a beam step 6.9.
//
// Every function takes its arguments by place, as layers.py passes them on, the last
// being the raw handle of the stream (None: torch's current one).  On another stream
// than torch's the caller has ordered that one behind it; what is allocated here is
// marked as used there.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <cstdarg>
#include <limits>
#include <optional>
#include <string>
#include <vector>

#include "../../include/sgemm_layers.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr int64_t kMost = 2147483647;  // sizes and leading dimensions of the library are 32-bit

// An exception that Python has been told of.
using Told = python_error;

[[noreturn]] void refuse(PyObject *type, const char *format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    Told told;
    told.persist();
    throw told;
}

[[noreturn]] void told() {
    Told t;
    t.persist();
    throw t;
}

// ---------------------------------------------------------------- arguments

const char *type_name(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return "torch.float32";
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Half: return "torch.float16";
        case ScalarType::Byte: return "torch.uint8";
        case ScalarType::Int: return "torch.int32";
        default: return c10::toString(t);
    }
}

// The library's code of an element type, or -1.
int code_of(ScalarType t) {
    return t == ScalarType::Float ? SGEMM_F32 : t == ScalarType::BFloat16 ? SGEMM_BF16 : t == ScalarType::Half ? SGEMM_F16 : -1;
}

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a CUDA tensor, not %s", name, Py_TYPE(o)->tp_name);
    const Tensor &t = THPVariable_Unpack(o);
    // views whose numbers are not those in memory
    if (t.is_conj() || t.is_neg()) refuse(PyExc_ValueError, "%s is a conjugate or negated view: resolve_conj() and resolve_neg() make it plain", name);
    return t;
}

bool given(PyObject *o) { return o != Py_None; }

// A number that fits the library's 32 bits.
int whole(PyObject *o, const char *name) {
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    if (v == -1 && PyErr_Occurred()) told();
    if (over || v > kMost || v < -kMost) refuse(PyExc_ValueError, "%s is %S: it must fit 32 bits", name, o);
    return (int)v;
}

float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) told();
    return (float)v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) told();
    return v;
}

std::string shape_of(const Tensor &t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + (t.dim() == 1 ? ",)" : ")");
}

void same_device(const Tensor &t, const char *name, int index) {
    if (t.get_device() != index)
        refuse(PyExc_ValueError, "%s is on %s, not on cuda:%d", name, t.device().str().c_str(), index);
}

struct Matrix {
    void *p = nullptr;
    int ld = 1;
    int64_t rows = 0, cols = 0;
};

// A matrix with unit column stride.
Matrix rows_of(const Tensor &t, const char *name) {
    Matrix m{t.data_ptr(), 1, t.size(0), t.size(1)};
    if (m.rows > kMost || m.cols > kMost)
        refuse(PyExc_ValueError, "%s is (%lld, %lld): rows and columns must be below 2^31", name, (long long)m.rows, (long long)m.cols);
    int64_t ld = m.cols;
    if (!t.is_contiguous()) {
        if (m.cols > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "%s must have unit column stride", name);
        if (m.rows > 1) {
            ld = t.stride(0);
            if (ld < m.cols) refuse(PyExc_ValueError, "%s has rows that overlap", name);
            if (ld > kMost)
                refuse(PyExc_ValueError, "%s has rows %lld elements apart: they must be below 2^31", name, (long long)ld);
        }
    }
    m.ld = (int)std::max<int64_t>(ld, 1);
    return m;
}

// A call's first tensor: a 2-D CUDA one of a type that the operator takes.
int first_code(const Tensor &t, const char *name) {
    const int code = code_of(t.scalar_type());
    if (code < 0) refuse(PyExc_TypeError, "%s must be float32, bfloat16 or float16", name);
    if (!t.is_cuda() || t.dim() != 2) refuse(PyExc_TypeError, "%s must be a 2-D CUDA tensor", name);
    return code;
}

Matrix matrix(PyObject *o, const char *name, ScalarType type, int index, int64_t rows, int64_t cols) {
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || !t.is_cuda() || t.dim() != 2)
        refuse(PyExc_TypeError, "%s must be a 2-D %s CUDA tensor", name, type_name(type));
    same_device(t, name, index);
    if ((rows >= 0 && t.size(0) != rows) || t.size(1) != cols) {
        if (rows >= 0)
            refuse(PyExc_ValueError, "%s is %s, not (%lld, %lld)", name, shape_of(t).c_str(), (long long)rows, (long long)cols);
        refuse(PyExc_ValueError, "%s is %s, not ('any', %lld)", name, shape_of(t).c_str(), (long long)cols);
    }
    return rows_of(t, name);
}

// A dense vector of n elements of one of two types; null where it is not given.
void *vector(PyObject *o, const char *name, int64_t n, ScalarType type, ScalarType other, int index) {
    if (!given(o)) return nullptr;
    const Tensor &t = tensor(o, name);
    if ((t.scalar_type() != type && t.scalar_type() != other) || !t.is_cuda() || t.dim() != 1)
        refuse(PyExc_TypeError, "%s must be a 1-D CUDA tensor of %s or %s", name, type_name(type), type_name(other));
    if (t.size(0) != n) refuse(PyExc_ValueError, "%s has %lld elements, not %lld", name, (long long)t.size(0), (long long)n);
    same_device(t, name, index);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be dense", name);
    return t.data_ptr();
}
const float *floats(PyObject *o, const char *name, int64_t n, int index) {
    return static_cast<const float *>(vector(o, name, n, ScalarType::Float, ScalarType::Float, index));
}

// ---------------------------------------------------------------- calls

void check(int status, const char *where) {
    if (status == SGEMM_OK) return;
    PyObject *module = PyImport_ImportModule("dense_fp32_matrix_04_gb300");
    PyObject *type = module ? PyObject_GetAttrString(module, "SgemmError") : nullptr;
    PyObject *error = type ? PyObject_CallFunction(type, "is", status, where) : nullptr;
    if (error) PyErr_SetObject(type, error);
    Py_XDECREF(error);
    Py_XDECREF(type);
    Py_XDECREF(module);
    told();
}

// Other Python threads may run while this exists.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// The device and the stream that a call runs on, and what it allocates.
class Call {
   public:
    Call(const Tensor &first, PyObject *stream) : index_(first.get_device()) {
        if (index_ != c10::cuda::current_device()) guard_.emplace(static_cast<c10::DeviceIndex>(index_));
        const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index_));
        stream_ = current.stream();
        if (given(stream)) {
            const long long handle = PyLong_AsLongLong(stream);
            if (handle == -1 && PyErr_Occurred()) told();
            other_ = reinterpret_cast<cudaStream_t>(handle) != stream_;
            stream_ = reinterpret_cast<cudaStream_t>(handle);
        }
    }
    int index() const { return index_; }
    cudaStream_t stream() const { return stream_; }
    // Memory of the call's own: a workspace, given back to torch when the call returns.
    c10::DataPtr memory(int64_t bytes) {
        Unlocked other_threads;
        return allocate(bytes);
    }
    // A tensor of its own, with a storage of its own: what a call returns may be saved, resized or
    // given back one by one.
    struct Wanted {
        c10::DimVector sizes;
        ScalarType type;
        int64_t pitch = 0;  // elements from a row to the next; 0: dense
        bool wanted = true;
        int64_t bytes() const {
            return (pitch ? sizes[0] * pitch : c10::multiply_integers(sizes)) * (int64_t)c10::elementSize(type);
        }
    };
    template <size_t N>
    std::array<Tensor, N> empty(const std::array<Wanted, N> &all) {
        std::array<c10::DataPtr, N> at;
        {
            Unlocked other_threads;
            for (size_t i = 0; i < N; ++i)
                if (all[i].wanted) at[i] = allocate(all[i].bytes());
        }
        std::array<Tensor, N> made;
        for (size_t i = 0; i < N; ++i)
            if (all[i].wanted) made[i] = tensor_of(all[i], std::move(at[i]));
        return made;
    }
    Tensor empty(at::IntArrayRef sizes, ScalarType type) {
        return empty<1>({{{c10::DimVector(sizes.begin(), sizes.end()), type}}})[0];
    }
    // Calls the library.
    template <class F>
    void run(const char *where, F &&f) {
        int status;
        {
            Unlocked other_threads;
            status = f();
        }
        check(status, where);
    }
    // NaN in all of t, on the call's stream.
    void fill_nan(const Tensor &t) {
        const c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(stream_, static_cast<c10::DeviceIndex>(index_)));
        t.fill_(std::numeric_limits<double>::quiet_NaN());
    }

   private:
    c10::DataPtr allocate(int64_t bytes) const {
        c10::DataPtr p = c10::cuda::CUDACachingAllocator::get()->allocate((size_t)bytes);
        if (other_)
            c10::cuda::CUDACachingAllocator::recordStream(
                p, c10::cuda::getStreamFromExternal(stream_, static_cast<c10::DeviceIndex>(index_)));
        return p;
    }
    // (at::empty's own steps, which are a third of what at::empty costs)
    static Tensor tensor_of(const Wanted &w, c10::DataPtr p) {
        auto storage = c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), (size_t)w.bytes(), std::move(p),
                                                             c10::cuda::CUDACachingAllocator::get(), /*resizable=*/true);
        Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(std::move(storage)), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                            c10::scalarTypeToTypeMeta(w.type));
        const int64_t strides[2] = {w.pitch, 1};
        if (w.pitch) t.unsafeGetTensorImpl()->set_sizes_and_strides(w.sizes, strides);
        else t.unsafeGetTensorImpl()->set_sizes_contiguous(w.sizes);
        return t;
    }

    int index_;
    std::optional<c10::cuda::CUDAGuard> guard_;
    cudaStream_t stream_;
    bool other_ = false;
};

// A tuple of new tensors (one that is not defined: None).
PyObject *tuple(std::initializer_list<Tensor> made) {
    PyObject *out = PyTuple_New((Py_ssize_t)made.size());
    if (!out) told();
    Py_ssize_t i = 0;
    for (const Tensor &t : made) {
        PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(out);
            told();
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

void count_arguments(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse(PyExc_TypeError, "%zd arguments, not %zd", n, want);
}

// An output that is given, or a new one of type `code` of shape M x N; with `bytes` also a
// workspace of that size.
struct Output {
    Tensor made;
    c10::DataPtr space;
    Matrix m;
    int code;
    PyObject *given_object = nullptr;
    PyObject *result() const { return given_object ? Py_NewRef(given_object) : THPVariable_Wrap(made); }
};
Output product_output(Call &call, PyObject *out, PyObject *out_dtype, ScalarType otherwise, int64_t M, int64_t N, size_t bytes = 0) {
    Output o;
    ScalarType type = otherwise;
    if (bytes) o.space = call.memory((int64_t)bytes);
    if (given(out)) {
        type = tensor(out, "out").scalar_type();
        o.code = code_of(type);
        if (o.code < 0) refuse(PyExc_TypeError, "out must be float32, bfloat16 or float16");
        o.m = matrix(out, "out", type, call.index(), M, N);
        o.given_object = out;
        return o;
    }
    if (given(out_dtype)) {
        if (!THPDtype_Check(out_dtype)) refuse(PyExc_TypeError, "out_dtype must be float32, bfloat16 or float16");
        type = reinterpret_cast<THPDtype *>(out_dtype)->scalar_type;
    }
    o.code = code_of(type);
    if (o.code < 0) refuse(PyExc_TypeError, "out_dtype must be float32, bfloat16 or float16");
    o.made = call.empty<1>({{{{M, N}, type}}})[0];
    o.m = Matrix{o.made.data_ptr(), (int)std::max<int64_t>(N, 1), M, N};
    return o;
}

// ---------------------------------------------------------------- layer norm

// x, w, bias, add, eps, out, stream
PyObject *layer_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_arguments(n, 7);
    const Tensor &x = tensor(a[0], "x");
    const int code = first_code(x, "x"), dev = x.get_device();
    const Matrix X = rows_of(x, "x");
    const int64_t T = X.rows, D = X.cols;
    const ScalarType dt = x.scalar_type(), wt = tensor(a[1], "w").scalar_type();
    const void *w = vector(a[1], "w", D, ScalarType::Float, dt, dev), *b = vector(a[2], "bias", D, wt, wt, dev);
    const float eps = real(a[4]);
    const bool add = given(a[3]), out = given(a[5]);
    if (out && !add) refuse(PyExc_ValueError, "out is for the sum with add, which is not given");
    Matrix A, R;
    if (add) A = matrix(a[3], "add", dt, dev, T, D);
    if (out) R = matrix(a[5], "out", dt, dev, T, D);
    Call call(x, a[6]);
    Tensor r, normed, stats;
    if (add && !out) {
        const auto made = call.empty<3>({{{{T, D}, dt}, {{T, D}, dt}, {{2, T}, ScalarType::Float}}});
        r = made[0], normed = made[1], stats = made[2];
        R = Matrix{r.data_ptr(), D ? (int)D : 1, T, D};
    } else {
        const auto made = call.empty<2>({{{{T, D}, dt}, {{2, T}, ScalarType::Float}}});
        normed = made[0], stats = made[1];
    }
    call.run("sgemm_layer_norm", [&] {
        return sgemm_layer_norm((int)T, (int)D, code, X.p, X.ld, add ? A.p : nullptr, A.ld, w, b, code_of(wt), eps, add ? R.p : nullptr,
                           R.ld, normed.data_ptr(), D ? (int)D : 1, static_cast<float *>(stats.data_ptr()), call.stream());
    });
    if (!D && T) call.fill_nan(stats);  // the mean of nothing
    PyObject *got = tuple({r, normed, stats});
    if (!r.defined()) {
        Py_DECREF(PyTuple_GET_ITEM(got, 0));
        PyTuple_SET_ITEM(got, 0, Py_NewRef(out ? a[5] : a[0]));
    }
    return got;
    END_HANDLE_TH_ERRORS
}

// x, w, stats, dn, dr, bias, out, stream
PyObject *layer_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_arguments(n, 8);
    const Tensor &x = tensor(a[0], "x");
    const int code = first_code(x, "x"), dev = x.get_device();
    const Matrix X = rows_of(x, "x");
    const int64_t T = X.rows, D = X.cols;
    const ScalarType dt = x.scalar_type(), wt = tensor(a[1], "w").scalar_type();
    const Matrix DN = matrix(a[3], "dn", dt, dev, T, D);
    Matrix DR;
    if (given(a[4])) DR = matrix(a[4], "dr", dt, dev, T, D);
    const void *w = vector(a[1], "w", D, ScalarType::Float, dt, dev);
    const Tensor &stats = tensor(a[2], "stats");
    if (stats.scalar_type() != ScalarType::Float || stats.dim() != 2 || stats.size(0) != 2 || stats.size(1) != T ||
        !stats.is_contiguous() || stats.get_device() != dev)
        refuse(PyExc_ValueError, "stats must be the (2, T) float32 tensor that layer_norm returned");
    const bool bias = truth(a[5]), out = given(a[6]);
    Matrix DX;
    if (out) DX = matrix(a[6], "out", dt, dev, T, D);
    Call call(x, a[7]);
    const size_t need = sgemm_layer_norm_backward_workspace_size((int)T, (int)D);
    const c10::DataPtr ws = call.memory((int64_t)need);
    const auto made = call.empty<3>({{{{T, D}, dt, 0, !out}, {{D}, wt}, {{D}, wt, 0, bias}}});
    const Tensor &dx = out ? tensor(a[6], "out") : made[0], &dw = made[1], &db = made[2];
    if (!out) DX = Matrix{dx.data_ptr(), D ? (int)D : 1, T, D};
    call.run("sgemm_layer_norm_backward", [&] {
        return sgemm_layer_norm_backward((int)T, (int)D, code, X.p, X.ld, w, code_of(wt), static_cast<const float *>(stats.data_ptr()),
                                    DN.p, DN.ld, given(a[4]) ? DR.p : nullptr, DR.ld, DX.p, DX.ld,
                                    dw.data_ptr(), bias ? db.data_ptr() : nullptr, ws.get(), need, call.stream());
    });
    // (a tensor that is given comes back as the object that it is: THPVariable_Wrap finds it)
    return tuple({dx, dw, db});
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- 4-bit floating point

// Columns that share a scale of this type, or 0.
int block_of(ScalarType t) { return t == ScalarType::Float8_e4m3fn ? 16 : t == ScalarType::Float8_e8m0fnu ? 32 : 0; }
ScalarType scales_type(int block) { return block == 16 ? ScalarType::Float8_e4m3fn : ScalarType::Float8_e8m0fnu; }

// Shape of the tiles that hold the block scales of rows x K columns.
struct Tiles {
    int64_t rows, bytes;
    Tiles(int64_t M, int64_t K, int block) : rows((M + 127) / 128), bytes(((K + block - 1) / block + 3) / 4 * 512) {}
};

struct BlockScales {
    const unsigned char *p;
    int block;
};
BlockScales block_scales(PyObject *o, const char *name, int64_t rows, int64_t K, int index) {
    const Tensor &t = tensor(o, name);
    const int block = block_of(t.scalar_type());
    if (!block || !t.is_cuda() || t.dim() != 2)
        refuse(PyExc_TypeError, "%s must be a 2-D CUDA tensor of float8_e4m3fn (blocks of 16) or float8_e8m0fnu (of 32)", name);
    same_device(t, name, index);
    const Tiles want(rows, K, block);
    if (t.size(0) != want.rows || t.size(1) != want.bytes)
        refuse(PyExc_ValueError, "%s is %s, not the (%lld, %lld) of tiles for %lld rows of %lld", name, shape_of(t).c_str(),
               (long long)want.rows, (long long)want.bytes, (long long)rows, (long long)K);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be dense", name);
    return {static_cast<const unsigned char *>(t.data_ptr()), block};
}

// Packed codes of `cols` bytes a row (any number of rows where `rows` is negative).
Matrix codes(PyObject *o, const char *name, int index, int64_t rows, int64_t cols) {
    Matrix m = matrix(o, name, ScalarType::Byte, index, rows, cols);
    if (!m.cols) {
        m.ld = 16;
        return m;
    }
    if (m.rows > 1 && m.ld % 16)
        refuse(PyExc_ValueError, "%s has rows %d bytes apart: they must be a multiple of 16, as quantize_fp4 lays them out. Dense rows, as "
               "copies between devices have them, become such by torch.nn.functional.pad(q, (0, -q.shape[1] %% 16))[:, :q.shape[1]]", name, m.ld);
    if (reinterpret_cast<uintptr_t>(m.p) % 16) refuse(PyExc_ValueError, "%s must start on 16 bytes", name);
    if (m.rows <= 1) m.ld = (int)std::max<int64_t>((m.cols + 15) / 16 * 16, 16);
    return m;
}

// x, block, stream
PyObject *quantize_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_arguments(n, 3);
    const Tensor &x = tensor(a[0], "x");
    const int code = first_code(x, "x");
    const Matrix X = rows_of(x, "x");
    const int block = whole(a[1], "block");
    if (block != 16 && block != 32) refuse(PyExc_ValueError, "block is %d: it must be 16 or 32", block);
    Call call(x, a[2]);
    const int64_t pitch = std::max<int64_t>((X.cols + 31) / 32 * 16, 16);
    const Tiles shape(X.rows, X.cols, block);
    const auto made = call.empty<3>({{{{X.rows, (X.cols + 1) / 2}, ScalarType::Byte, pitch},
                                      {{shape.rows, shape.bytes}, scales_type(block)},
                                      {{X.rows}, ScalarType::Float, 0, block == 16}}});
    const Tensor &packed = made[0], &tiles = made[1], &scale = made[2];
    call.run("sgemm_quantize_fp4", [&] {
        return sgemm_quantize_fp4((int)X.rows, (int)X.cols, code, X.p, X.ld, block, static_cast<unsigned char *>(packed.data_ptr()),
                             (int)pitch, static_cast<unsigned char *>(tiles.data_ptr()),
                             block == 16 ? static_cast<float *>(scale.data_ptr()) : nullptr, call.stream());
    });
    return tuple({packed, tiles, scale});
    END_HANDLE_TH_ERRORS
}

// s, stream
PyObject *lay_out_fp4_scales(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_arguments(n, 2);
    const Tensor &s = tensor(a[0], "s");
    const int block = block_of(s.scalar_type());
    if (!block || !s.is_cuda() || s.dim() != 2)
        refuse(PyExc_TypeError, "s must be a 2-D CUDA tensor of float8_e4m3fn (blocks of 16) or float8_e8m0fnu (of 32)");
    const Matrix S = rows_of(s, "s");
    if (S.cols > (1 << 24) / block)
        refuse(PyExc_ValueError, "s has %lld blocks of %d: more than 2^24 columns", (long long)S.cols, block);
    const int64_t K = S.cols * block;
    Call call(s, a[1]);
    const Tiles shape(S.rows, K, block);
    const Tensor tiles = call.empty({shape.rows, shape.bytes}, s.scalar_type());
    call.run("sgemm_fp4_lay_out_scales", [&] {
        return sgemm_fp4_lay_out_scales((int)S.rows, (int)K, block, static_cast<const unsigned char *>(S.p), S.ld,
                                   static_cast<unsigned char *>(tiles.data_ptr()), call.stream());
    });
    return THPVariable_Wrap(tiles);
    END_HANDLE_TH_ERRORS
}

// a, a_block, a_scale, w, w_block, w_scale, bias, out_dtype, out, stream
PyObject *matmul_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_arguments(n, 10);
    const Tensor &first = tensor(a[0], "a");
    if (first.scalar_type() != ScalarType::Byte) refuse(PyExc_TypeError, "a must be torch.uint8");
    if (!first.is_cuda() || first.dim() != 2) refuse(PyExc_TypeError, "a must be a 2-D CUDA tensor");
    const int dev = first.get_device();
    const Matrix A = codes(a[0], "a", dev, -1, first.size(1)), W = codes(a[3], "w", dev, -1, A.cols);
    const int64_t M = A.rows, N = W.rows, K = 2 * A.cols;  // the half behind an odd number of columns is 0
    if (K > kMost) refuse(PyExc_ValueError, "a has %lld columns of codes: two for each must fit 32 bits", (long long)A.cols);
    const BlockScales as = block_scales(a[1], "a_block", M, K, dev), ws = block_scales(a[4], "w_block", N, K, dev);
    if (as.block != ws.block) refuse(PyExc_ValueError, "a has blocks of %d, w of %d", as.block, ws.block);
    const float *a_scale = floats(a[2], "a_scale", M, dev), *w_scale = floats(a[5], "w_scale", N, dev),
                *bias = floats(a[6], "bias", N, dev);
    Call call(first, a[9]);
    const Output out = product_output(call, a[8], a[7], ScalarType::Float, M, N);
    call.run("sgemm_fp4", [&] {
        return sgemm_fp4((int)M, (int)N, (int)K, as.block, static_cast<const unsigned char *>(A.p), A.ld, as.p, a_scale,
                    static_cast<const unsigned char *>(W.p), W.ld, ws.p, w_scale, bias, out.m.p, out.m.ld, out.code, call.stream());
    });
    return out.result();
    END_HANDLE_TH_ERRORS
}

// x, w, w_block, w_scale, bias, out_dtype, out, workspace, stream
PyObject *linear_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_arguments(n, 9);
    const Tensor &x = tensor(a[0], "x");
    const int code = first_code(x, "x"), dev = x.get_device();
    const Matrix X = rows_of(x, "x");
    const int64_t M = X.rows, K = X.cols;
    const Matrix W = codes(a[1], "w", dev, -1, (K + 1) / 2);
    const int64_t N = W.rows;
    const BlockScales ws = block_scales(a[2], "w_block", N, K, dev);
    const float *w_scale = floats(a[3], "w_scale", N, dev), *bias = floats(a[4], "bias", N, dev);
    void *space = nullptr;
    size_t size = 0;
    if (given(a[7])) {
        const Tensor &t = tensor(a[7], "workspace");
        if (!t.is_cuda()) refuse(PyExc_TypeError, "workspace must be a CUDA tensor");
        same_device(t, "workspace", dev);
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be dense");
        space = t.data_ptr();
        size = t.nbytes();
    }
    Call call(x, a[8]);
    const size_t need = given(a[7]) ? 0 : sgemm_linear_fp4_workspace_size((int)M, (int)K, ws.block);
    const Output out = product_output(call, a[6], a[5], x.scalar_type(), M, N, need);
    if (need) space = out.space.get(), size = need;
    call.run("sgemm_linear_fp4", [&] {
        return sgemm_linear_fp4((int)M, (int)N, (int)K, code, X.p, X.ld, ws.block, static_cast<const unsigned char *>(W.p), W.ld, ws.p,
                           w_scale, bias, out.m.p, out.m.ld, out.code, space, size, call.stream());
    });
    return out.result();
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- beams

// A dense 2-D tensor with an entry for each beam.
const Tensor &beams(PyObject *o, const char *name, ScalarType type, ScalarType other, int index) {
    const Tensor &t = tensor(o, name);
    if ((t.scalar_type() != type && t.scalar_type() != other) || !t.is_cuda() || t.dim() != 2)
        refuse(PyExc_TypeError, "%s must be a 2-D CUDA tensor of %s or %s", name, type_name(type), type_name(other));
    same_device(t, name, index);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be dense", name);
    return t;
}

// logits, score, top, scale, mask, finished, end, stream
PyObject *beam_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_arguments(n, 8);
    const Tensor &z = tensor(a[0], "logits");
    const int code = first_code(z, "logits"), dev = z.get_device();
    const Matrix Z = rows_of(z, "logits");
    const int64_t T = Z.rows, V = Z.cols;
    const Tensor &score = beams(a[1], "score", ScalarType::Float, ScalarType::Float, dev);
    const int64_t B = score.size(0), W = score.size(1);
    if (B * W != T) refuse(PyExc_ValueError, "score is (%lld, %lld), logits has %lld rows", (long long)B, (long long)W, (long long)T);
    const int64_t top = given(a[2]) ? whole(a[2], "top") : W;
    if (top < 1 || top > 32 || W < 1 || W > 32)
        refuse(PyExc_ValueError, "%lld beams and the best %lld: they must be 1 .. 32", (long long)W, (long long)top);
    const float scale = real(a[3]);
    const unsigned char *finished = nullptr;
    if (given(a[5])) {
        const Tensor &f = beams(a[5], "finished", ScalarType::Bool, ScalarType::Byte, dev);
        if (f.size(0) != B || f.size(1) != W)
            refuse(PyExc_ValueError, "finished is %s, not (%lld, %lld)", shape_of(f).c_str(), (long long)B, (long long)W);
        finished = static_cast<const unsigned char *>(f.data_ptr());
    }
    const int end = whole(a[6], "end");
    if (end < 0) refuse(PyExc_ValueError, "end is %d: it must be a column", end);
    Matrix mask;
    if (given(a[4])) {
        mask = matrix(a[4], "mask", ScalarType::Int, dev, -1, (V + 31) / 32);
        if (mask.rows != 1 && mask.rows != T)
            refuse(PyExc_ValueError, "mask has %lld rows, not 1 or %lld", (long long)mask.rows, (long long)T);
        if (!V) mask = Matrix{};  // no words, and no pointer to them
    }
    Call call(z, a[7]);
    const size_t size = sgemm_beam_step_workspace_size((int)B, (int)W, (int)top);
    const c10::DataPtr ws = call.memory((int64_t)size);
    const auto made = call.empty<3>({{{{B, top}, ScalarType::Float}, {{B, top}, ScalarType::Int}, {{B, top}, ScalarType::Int}}});
    const Tensor &best = made[0], &parent = made[1], &token = made[2];
    call.run("sgemm_beam_step", [&] {
        return sgemm_beam_step((int)B, (int)W, (int)V, code, Z.p, Z.ld, scale, static_cast<const int32_t *>(mask.p), mask.ld,
                          (int)mask.rows, static_cast<const float *>(score.data_ptr()), finished, end, (int)top,
                          static_cast<float *>(best.data_ptr()), static_cast<int32_t *>(parent.data_ptr()),
                          static_cast<int32_t *>(token.data_ptr()), ws.get(), size, call.stream());
    });
    return tuple({best, parent, token});
    END_HANDLE_TH_ERRORS
}

// Rows of two tensors of the same shape behind the first dimension: `outer` runs of
// `inner` elements, which are a distance apart in each.
struct Runs {
    int64_t outer = 1, inner = 1, a = 0, b = 0;
    Runs(const Tensor &x, const Tensor &y) {
        struct Dim {
            int64_t n, a, b;
        };
        std::vector<Dim> dims;  // outermost first, merged where they follow on in both
        for (int64_t d = 1; d < x.dim(); ++d) {
            Dim next{x.size(d), x.stride(d), y.stride(d)};
            if (next.n == 1) continue;
            if (!dims.empty() && dims.back().a == next.n * next.a && dims.back().b == next.n * next.b) {
                next.n *= dims.back().n;
                dims.pop_back();
            }
            dims.push_back(next);
        }
        if (!dims.empty() && dims.back().a == 1 && dims.back().b == 1) {
            inner = dims.back().n;
            dims.pop_back();
        }
        if (dims.size() > 1)
            refuse(PyExc_ValueError, "rows of states must be one dense run, or runs at one distance from each other");
        if (!dims.empty()) outer = dims.back().n, a = dims.back().a, b = dims.back().b;
    }
};

// state, parent, out, stream
PyObject *beam_reorder(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count_arguments(n, 4);
    const Tensor &state = tensor(a[0], "state");
    if (!state.is_cuda() || state.dim() < 1) refuse(PyExc_TypeError, "state must be a CUDA tensor with a row for each beam");
    const int dev = state.get_device();
    const Tensor &parent = beams(a[1], "parent", ScalarType::Int, ScalarType::Int, dev);
    const int64_t B = parent.size(0), top = parent.size(1), T = state.size(0);
    if (B ? T % B : T)
        refuse(PyExc_ValueError, "state has %lld rows, which are not %lld groups of as many beams", (long long)T, (long long)B);
    const int64_t W = B ? T / B : 1;
    if (B && (W < 1 || W > 32 || top < 1 || top > 32))
        refuse(PyExc_ValueError, "%lld beams and %lld parents: they must be 1 .. 32", (long long)W, (long long)top);
    if (B * W > kMost) refuse(PyExc_ValueError, "state has %lld rows: they must be below 2^31", (long long)T);
    c10::DimVector shape(state.sizes().begin(), state.sizes().end());
    shape[0] = B * top;
    Call call(state, a[3]);
    Tensor out;
    if (given(a[2])) {
        out = tensor(a[2], "out");
        if (out.scalar_type() != state.scalar_type() || !out.is_cuda() || out.get_device() != dev)
            refuse(PyExc_TypeError, "out must be a %s tensor on cuda:%d", type_name(state.scalar_type()), dev);
        if (out.sizes() != at::IntArrayRef(shape))
            refuse(PyExc_ValueError, "out is %s, which is not the shape of the state with %lld rows", shape_of(out).c_str(),
                   (long long)(B * top));
    } else {
        out = call.empty(shape, state.scalar_type());
    }
    if (B && out.numel()) {
        const Runs runs(state, out);
        const int64_t size = state.element_size();
        call.run("sgemm_beam_reorder", [&] {
        return sgemm_beam_reorder((int)B, (int)W, (int)top, runs.outer, runs.inner * size, state.data_ptr(), state.stride(0) * size,
                                 runs.a * size, static_cast<const int32_t *>(parent.data_ptr()), out.data_ptr(),
                                 out.stride(0) * size, runs.b * size, call.stream());
    });
    }
    return given(a[2]) ? Py_NewRef(a[2]) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

#define FUNCTION(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef functions[] = {FUNCTION(layer_norm),    FUNCTION(layer_norm_backward), FUNCTION(quantize_fp4),
                           FUNCTION(lay_out_fp4_scales), FUNCTION(matmul_fp4),     FUNCTION(linear_fp4),
                           FUNCTION(beam_step),     FUNCTION(beam_reorder),        {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, functions, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
