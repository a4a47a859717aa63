// bind.cpp — the Python binding of the calls over e4m3 pools with a scale per
// (block, kv head) and of those of caches that evict tokens, as a CPython module
// over PyTorch's C++ tensors.
//
// It does what the ctypes binding does for the other entry points, argument
// marshalling only: types, devices, contiguity and shapes are checked, outputs
// that were not given are allocated, and the C function of include/pa.h is
// called on the given or the current stream.  Done in Python, these checks were
// 10 to 15 of the 17 to 25 us that a small call took on the host, more than the
// kernels of such a call.
//
// A function returns its outputs, or the library's status as an int where that
// is not PA_OK (the caller raises PaError); TypeError and ValueError are raised
// here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pa.h"

namespace {

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Refused{};
}

std::string sizes_text(const at::Tensor& t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int int_of(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v != static_cast<int>(v)) refuse(PyExc_OverflowError, "a size does not fit 32 bits");
    return static_cast<int>(v);
}
int int_of(int64_t v) {
    if (v != static_cast<int>(v)) refuse(PyExc_OverflowError, "a size does not fit 32 bits");
    return static_cast<int>(v);
}
float float_of(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return static_cast<float>(v);
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

// The pools of a call and the device they are on.
struct Pools {
    const at::Tensor &k, &v, &ks, &vs;
    int blocks, block, heads, dim;

    Pools(PyObject* k_, PyObject* v_, PyObject* ks_, PyObject* vs_)
        : k(tensor(k_, "k_cache")), v(tensor(v_, "v_cache")), ks(tensor(ks_, "k_scales")), vs(tensor(vs_, "v_scales")) {
        if (k.scalar_type() != at::kByte || v.scalar_type() != at::kByte)
            refuse(PyExc_TypeError, "fp8 pools are uint8 tensors of e4m3 codes");
        if (k.dim() != 4) refuse(PyExc_ValueError, "k_cache must be [num_blocks, block_size, num_kv_heads, head_dim]");
        if (!k.sizes().equals(v.sizes())) refuse(PyExc_ValueError, "shapes of k_cache and v_cache differ");
        blocks = int_of(k.size(0));
        block = int_of(k.size(1));
        heads = int_of(k.size(2));
        dim = int_of(k.size(3));
        for (const at::Tensor* t : {&ks, &vs})
            if (t->dim() != 2 || t->size(0) != blocks || t->size(1) != heads)
                refuse(PyExc_ValueError, "k_scales and v_scales must be [num_blocks, num_kv_heads] = [" +
                                             std::to_string(blocks) + ", " + std::to_string(heads) + "], got " +
                                             sizes_text(ks) + " and " + sizes_text(vs));
    }

    // Pointer of a contiguous tensor of `type` on the pools' device (or, with host_ok, in pinned host memory).
    void* at(const at::Tensor& t, const char* name, at::ScalarType type, bool host_ok = false) const {
        if (t.scalar_type() != type)
            refuse(PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
        if (t.device() != k.device() && !(host_ok && t.is_cpu() && t.is_pinned()))
            refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on the pools' device" +
                                         (host_ok ? " or pinned host memory" : ""));
        if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
    void* at(PyObject* o, const char* name, at::ScalarType type) const {
        return o == Py_None ? nullptr : at(tensor(o, name), name, type);
    }
    void* kp() const { return at(k, "k_cache", at::kByte); }
    void* vp() const { return at(v, "v_cache", at::kByte); }
    float* ksp() const { return static_cast<float*>(at(ks, "k_scales", at::kFloat)); }
    float* vsp() const { return static_cast<float*>(at(vs, "v_scales", at::kFloat)); }
};

struct Workspace {
    void* ptr = nullptr;
    size_t bytes = 0;
    Workspace(const Pools& p, PyObject* o) {
        if (o == Py_None) return;
        const at::Tensor& t = tensor(o, "workspace");
        ptr = p.at(t, "workspace", t.scalar_type());
        bytes = t.nbytes();
    }
};

const int32_t* i32(void* p) { return static_cast<const int32_t*>(p); }

// Without the interpreter lock while it lives: a launch may wait for room in its queue, and other threads go on meanwhile.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// The handle of a stream given as an object with cuda_stream, or as a number.
cudaStream_t handle_of(PyObject* stream) {
    PyObject* raw = PyObject_HasAttrString(stream, "cuda_stream") ? PyObject_GetAttrString(stream, "cuda_stream")
                                                                 : (Py_INCREF(stream), stream);
    if (!raw) throw Refused{};
    void* s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw Refused{};
    return static_cast<cudaStream_t>(s);
}

// Memory for an output on the device of `like`.  Where the caller gives a stream it is that stream's, as if allocated with it
// current: memory that the current stream has freed may still be in use by its earlier work, which the given stream does
// not wait for.  The current stream, where the caller takes the output up, is noted as a user.
at::Tensor new_output(const at::Tensor& like, PyObject* stream, at::IntArrayRef shape, at::ScalarType type) {
    const auto options = like.options().dtype(type);
    if (stream == Py_None || !like.is_cuda()) return at::empty(shape, options);
    const c10::DeviceIndex device = like.device().index();
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(device);
    cudaStream_t handle = handle_of(stream);
    if (handle == cudaStreamLegacy) handle = nullptr;
    if (handle == current.stream()) return at::empty(shape, options);
    const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(handle, device));
    at::Tensor t = at::empty(shape, options);
    t.record_stream(current.unwrap());
    return t;
}

// Runs `call(stream)` with the tensor's device current, on the given stream (None: the device's current one).
template <typename F>
int on_device(const at::Tensor& like, PyObject* stream, F call, const char* what = "the pools") {
    if (!like.is_cuda()) refuse(PyExc_ValueError, std::string(what) + " must be CUDA tensors");
    const c10::cuda::CUDAGuard guard(like.device());
    void* s = stream == Py_None ? c10::cuda::getCurrentCUDAStream(like.device().index()).stream() : handle_of(stream);
    const Unlocked unlocked;
    return call(s);
}

template <typename F>
PyObject* guarded(F body) {
    try {
        return body();
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool counted(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

PyObject* status_or(int rc, PyObject* result) {
    if (rc == PA_OK) return Py_INCREF(result), result;
    return PyLong_FromLong(rc);
}

// k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables, seq_idx, pos, workspace, slot_mapping, error_count,
// stream -> slot_mapping
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 13)) return nullptr;
    return guarded([&] {
        const at::Tensor &kn = tensor(a[0], "k_new"), &vn = tensor(a[1], "v_new");
        const Pools p(a[2], a[3], a[4], a[5]);
        const at::Tensor &bt = tensor(a[6], "block_tables"), &seq = tensor(a[7], "seq_idx"), &pos = tensor(a[8], "pos");
        if (kn.dim() != 3 || kn.size(1) != p.heads || kn.size(2) != p.dim || !kn.sizes().equals(vn.sizes()))
            refuse(PyExc_ValueError, "shapes of k_new, v_new and the pools disagree");
        const int T = int_of(kn.size(0));
        if (seq.numel() != T || pos.numel() != T ||
            (a[10] != Py_None && tensor(a[10], "slot_mapping").numel() != T))
            refuse(PyExc_ValueError, "seq_idx, pos and slot_mapping must have one entry for each of the " +
                                         std::to_string(T) + " tokens");
        if (bt.dim() != 2) refuse(PyExc_ValueError, "block_tables must be [num_seqs, max_blocks_per_seq]");
        const Workspace ws(p, a[9]);
        void *knp = p.at(kn, "k_new", at::kBFloat16), *vnp = p.at(vn, "v_new", at::kBFloat16), *kp = p.kp(), *vp = p.vp();
        float *ks = p.ksp(), *vs = p.vsp();
        const int32_t *btp = i32(p.at(bt, "block_tables", at::kInt)), *sp = i32(p.at(seq, "seq_idx", at::kInt)),
                      *pp = i32(p.at(pos, "pos", at::kInt));
        int64_t* slots = static_cast<int64_t*>(p.at(a[10], "slot_mapping", at::kLong));
        int32_t* err = static_cast<int32_t*>(p.at(a[11], "error_count", at::kInt));
        const int S = int_of(bt.size(0)), W = int_of(bt.size(1));
        const int rc = on_device(p.k, a[12], [&](void* s) {
            return pa_write_kv_paged_fp8_block(knp, vnp, T, p.heads, p.dim, kp, vp, ks, vs, p.blocks, p.block, btp, S, W,
                                               sp, pp, slots, ws.ptr, ws.bytes, err, s);
        });
        return status_or(rc, a[10]);
    });
}

// k_cache, v_cache, k_scales, v_scales, block_tables, seq_idx, pos, k_out, v_out, float32, error_count, stream ->
// (k_out, v_out)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 12)) return nullptr;
    return guarded([&] {
        const Pools p(a[0], a[1], a[2], a[3]);
        const at::Tensor &bt = tensor(a[4], "block_tables"), &seq = tensor(a[5], "seq_idx"), &pos = tensor(a[6], "pos");
        if (pos.numel() != seq.numel()) refuse(PyExc_ValueError, "seq_idx and pos differ in length");
        if (bt.dim() != 2) refuse(PyExc_ValueError, "block_tables must be [num_seqs, max_blocks_per_seq]");
        const int T = int_of(seq.numel());
        at::ScalarType type = a[9] == Py_True ? at::kFloat : at::kBFloat16;
        if (a[7] != Py_None) type = tensor(a[7], "k_out").scalar_type();
        else if (a[8] != Py_None) type = tensor(a[8], "v_out").scalar_type();
        if (type != at::kFloat && type != at::kBFloat16)
            refuse(PyExc_TypeError, std::string("unsupported dtype ") + type_name(type) + " (float32 or bfloat16)");
        const int64_t shape[3] = {T, p.heads, p.dim};
        auto out = [&](PyObject* o, const char* name) {
            return o != Py_None ? tensor(o, name) : new_output(p.k, a[11], shape, type);
        };
        const at::Tensor ko = out(a[7], "k_out"), vo = out(a[8], "v_out");
        if (!ko.sizes().equals(shape) || !vo.sizes().equals(shape) || vo.scalar_type() != type)
            refuse(PyExc_ValueError, "k_out and v_out must be [" + std::to_string(T) + ", " + std::to_string(p.heads) +
                                         ", " + std::to_string(p.dim) + "] of one dtype");
        void *kop = p.at(ko, "k_out", type), *vop = p.at(vo, "v_out", type), *kp = p.kp(), *vp = p.vp();
        float *ks = p.ksp(), *vs = p.vsp();
        const int32_t *btp = i32(p.at(bt, "block_tables", at::kInt)), *sp = i32(p.at(seq, "seq_idx", at::kInt)),
                      *pp = i32(p.at(pos, "pos", at::kInt));
        int32_t* err = static_cast<int32_t*>(p.at(a[10], "error_count", at::kInt));
        const int S = int_of(bt.size(0)), W = int_of(bt.size(1));
        const int rc = on_device(p.k, a[11], [&](void* s) {
            return pa_read_kv_paged_fp8_block(kop, vop, T, p.heads, p.dim, type == at::kFloat ? PA_F32 : PA_BF16, kp, vp,
                                              ks, vs, p.blocks, p.block, btp, S, W, sp, pp, err, s);
        });
        if (rc != PA_OK) return PyLong_FromLong(rc);
        PyObject *k = THPVariable_Wrap(ko), *v = k ? THPVariable_Wrap(vo) : nullptr;
        PyObject* pair = v ? PyTuple_Pack(2, k, v) : nullptr;
        Py_XDECREF(k);
        Py_XDECREF(v);
        return pair;
    });
}

at::Tensor out_like(const Pools& p, PyObject* o, const at::Tensor& q, PyObject* stream) {
    if (!p.k.is_cuda()) refuse(PyExc_ValueError, "the pools must be CUDA tensors");
    (void)p.at(q, "q", at::kBFloat16);  // before anything is allocated like it
    return o == Py_None ? new_output(p.k, stream, q.sizes(), at::kBFloat16) : tensor(o, "out");
}

// q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, max_context_len, scale, workspace, out,
// error_count, stream -> out
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 13)) return nullptr;
    return guarded([&] {
        const at::Tensor& q = tensor(a[0], "q");
        const Pools p(a[1], a[2], a[3], a[4]);
        const at::Tensor &bt = tensor(a[5], "block_tables"), &ctx = tensor(a[6], "context_lens");
        if (q.dim() != 3 || q.size(2) != p.dim) refuse(PyExc_ValueError, "head_dim of q and k_cache differ");
        const int N = int_of(q.size(0));
        if (bt.dim() != 2 || bt.size(0) != N || ctx.numel() != N ||
            (a[10] != Py_None && !tensor(a[10], "out").sizes().equals(q.sizes())))
            refuse(PyExc_ValueError, "shapes of q, out, block_tables and context_lens disagree");
        const int max_ctx = int_of(a[7]);
        const float scale = float_of(a[8]);
        const Workspace ws(p, a[9]);
        const at::Tensor out = out_like(p, a[10], q, a[12]);
        void *op = p.at(out, "out", at::kBFloat16, true), *qp = p.at(q, "q", at::kBFloat16), *kp = p.kp(), *vp = p.vp();
        float *ks = p.ksp(), *vs = p.vsp();
        const int32_t *btp = i32(p.at(bt, "block_tables", at::kInt)), *cp = i32(p.at(ctx, "context_lens", at::kInt));
        int32_t* err = static_cast<int32_t*>(p.at(a[11], "error_count", at::kInt));
        const int Hq = int_of(q.size(1)), W = int_of(bt.size(1));
        const int rc = on_device(p.k, a[12], [&](void* s) {
            return pa_decode_fp8_block(op, qp, N, Hq, p.heads, p.dim, kp, vp, ks, vs, p.blocks, p.block, btp, W, cp,
                                       max_ctx, scale, ws.ptr, ws.bytes, err, s);
        });
        return rc != PA_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
    });
}

// q, cu_q_lens, q_start_pos, seq_of_chunk, max_q_len, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
// max_context_len, scale, workspace, out, error_count, stream -> out
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 17)) return nullptr;
    return guarded([&] {
        const at::Tensor &q = tensor(a[0], "q"), &cu = tensor(a[1], "cu_q_lens"), &start = tensor(a[2], "q_start_pos"),
                         &seq = tensor(a[3], "seq_of_chunk");
        const Pools p(a[5], a[6], a[7], a[8]);
        const at::Tensor &bt = tensor(a[9], "block_tables"), &ctx = tensor(a[10], "context_lens");
        if (q.dim() != 3 || q.size(2) != p.dim) refuse(PyExc_ValueError, "head_dim of q and k_cache differ");
        const int T = int_of(q.size(0)), C = int_of(start.numel());
        if (cu.numel() != C + 1 || seq.numel() != C ||
            (a[14] != Py_None && !tensor(a[14], "out").sizes().equals(q.sizes())))
            refuse(PyExc_ValueError, "shapes of q, out, cu_q_lens, q_start_pos and seq_of_chunk disagree");
        if (bt.dim() != 2 || bt.size(0) != ctx.numel())
            refuse(PyExc_ValueError, "shapes of block_tables and context_lens disagree");
        const int max_q = int_of(a[4]), max_ctx = int_of(a[11]);
        const float scale = float_of(a[12]);
        const Workspace ws(p, a[13]);
        const at::Tensor out = out_like(p, a[14], q, a[16]);
        void *op = p.at(out, "out", at::kBFloat16, true), *qp = p.at(q, "q", at::kBFloat16), *kp = p.kp(), *vp = p.vp();
        float *ks = p.ksp(), *vs = p.vsp();
        const int32_t *cup = i32(p.at(cu, "cu_q_lens", at::kInt)), *st = i32(p.at(start, "q_start_pos", at::kInt)),
                      *sq = i32(p.at(seq, "seq_of_chunk", at::kInt)), *btp = i32(p.at(bt, "block_tables", at::kInt)),
                      *cp = i32(p.at(ctx, "context_lens", at::kInt));
        int32_t* err = static_cast<int32_t*>(p.at(a[15], "error_count", at::kInt));
        const int Hq = int_of(q.size(1)), S = int_of(bt.size(0)), W = int_of(bt.size(1));
        const int rc = on_device(p.k, a[16], [&](void* s) {
            return pa_prefill_chunk_fp8_block(op, qp, cup, st, sq, C, T, max_q, S, Hq, p.heads, p.dim, kp, vp, ks, vs,
                                              p.blocks, p.block, btp, W, cp, max_ctx, scale, ws.ptr, ws.bytes, err, s);
        });
        return rc != PA_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
    });
}

// ---------------------------------------------------------------- caches that evict tokens
// Pointer of a contiguous tensor of `type` on the device of `like` (or, with host_ok, in pinned host memory).
void* data_of(const at::Tensor& like, const at::Tensor& t, const char* name, at::ScalarType type, bool host_ok = false) {
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
    if (t.device() != like.device() && !(host_ok && t.is_cpu() && t.is_pinned()))
        refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on the device of the other arguments" +
                                     (host_ok ? ", or pinned host memory" : ""));
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
}
void* data_or_null(const at::Tensor& like, PyObject* o, const char* name, at::ScalarType type) {
    return o == Py_None ? nullptr : data_of(like, tensor(o, name), name, type);
}

int float_code(at::ScalarType t) {
    if (t != at::kFloat && t != at::kBFloat16)
        refuse(PyExc_TypeError, std::string("unsupported dtype ") + type_name(t) + " (float32 or bfloat16)");
    return t == at::kFloat ? PA_F32 : PA_BF16;
}

bool true_of(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}

// The pools of a call, float32 or bfloat16.
struct Cache {
    const at::Tensor &k, &v;
    at::ScalarType type;
    int dtype, blocks, block, heads, dim;
    void *kp, *vp;

    Cache(PyObject* k_, PyObject* v_) : k(tensor(k_, "k_cache")), v(tensor(v_, "v_cache")), type(k.scalar_type()) {
        dtype = float_code(type);
        if (k.dim() != 4) refuse(PyExc_ValueError, "k_cache must be [num_blocks, block_size, num_kv_heads, head_dim]");
        if (!k.sizes().equals(v.sizes())) refuse(PyExc_ValueError, "shapes of k_cache and v_cache differ");
        blocks = int_of(k.size(0));
        block = int_of(k.size(1));
        heads = int_of(k.size(2));
        dim = int_of(k.size(3));
        kp = data_of(k, k, "k_cache", type);
        vp = data_of(k, v, "v_cache", type);
    }
    void* at(const at::Tensor& t, const char* name, at::ScalarType t_, bool host_ok = false) const {
        return data_of(k, t, name, t_, host_ok);
    }
};

struct Scratch {
    void* ptr = nullptr;
    size_t bytes = 0;
    Scratch(const at::Tensor& like, PyObject* o) {
        if (o == Py_None) return;
        const at::Tensor& t = tensor(o, "workspace");
        ptr = data_of(like, t, "workspace", t.scalar_type());
        bytes = t.nbytes();
    }
};

// One row for each sequence and kv head: [num_seqs, num_kv_heads, width].
int key_rows(const at::Tensor& t, const char* name, int seqs, int heads) {
    if (t.dim() != 3 || t.size(0) != seqs || t.size(1) != heads)
        refuse(PyExc_ValueError, std::string(name) + " must be [num_seqs, num_kv_heads, width] = [" + std::to_string(seqs) +
                                     ", " + std::to_string(heads) + ", ...], got " + sizes_text(t));
    return int_of(t.size(2));
}

// Rows [tokens, heads, head_dim] of which only the tokens may be apart.
struct Rows {
    const at::Tensor& t;
    int64_t stride;
    Rows(PyObject* o, const char* name) : t(tensor(o, name)) {
        if (t.dim() != 3) refuse(PyExc_ValueError, std::string(name) + " must be [num_tokens, heads, head_dim]");
        if ((t.size(2) > 1 && t.stride(2) != 1) || (t.size(1) > 1 && t.stride(1) != t.size(2)))
            refuse(PyExc_ValueError, std::string("the heads and elements of ") + name + " must be contiguous");
        stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
    }
    void* on(const at::Tensor& like, const char* name, at::ScalarType type) const {
        if (t.scalar_type() != type)
            refuse(PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
        if (t.device() != like.device())
            refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on the device of the other arguments");
        return t.data_ptr();
    }
};

// rope_pos [num_axes, T] or [T], inv_freq [rot_dim / 2], axis [rot_dim / 2] or None
struct Turns {
    const int32_t *pos, *axis;
    const float* inv_freq;
    int axes, rot;
    Turns(const at::Tensor& like, PyObject* pos_, PyObject* inv_freq_, PyObject* axis_, int tokens) {
        const at::Tensor &p = tensor(pos_, "rope_pos"), &f = tensor(inv_freq_, "inv_freq");
        if ((p.dim() != 1 && p.dim() != 2) || p.size(-1) != tokens)
            refuse(PyExc_ValueError, "rope_pos must be [num_axes, " + std::to_string(tokens) + "] or one axis, got " +
                                         sizes_text(p));
        axes = p.dim() == 2 ? int_of(p.size(0)) : 1;
        if (f.dim() != 1) refuse(PyExc_ValueError, "inv_freq must be [rot_dim / 2]");
        rot = int_of(2 * f.numel());
        pos = static_cast<const int32_t*>(data_of(like, p, "rope_pos", at::kInt));
        inv_freq = static_cast<const float*>(data_of(like, f, "inv_freq", at::kFloat));
        axis = static_cast<const int32_t*>(data_or_null(like, axis_, "axis", at::kInt));
        if (axis_ != Py_None && tensor(axis_, "axis").numel() != f.numel())
            refuse(PyExc_ValueError, "axis must have one entry for each of the " + std::to_string(f.numel()) + " pairs");
    }
};

// The output for q's shape: the given tensor, or new memory.
at::Tensor rows_out(const at::Tensor& like, PyObject* o, const char* name, PyObject* stream) {
    if (o == Py_None) return new_output(like, stream, like.sizes(), like.scalar_type());
    const at::Tensor& t = tensor(o, name);
    if (!t.sizes().equals(like.sizes())) refuse(PyExc_ValueError, std::string(name) + " must have its input's shape");
    return t;
}

// q, k, rope_pos, inv_freq, axis, interleaved, q_out, k_out, error_count, stream -> (q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 10)) return nullptr;
    return guarded([&] {
        const Rows q(a[0], "q"), k(a[1], "k");
        const at::ScalarType type = q.t.scalar_type();
        const int dtype = float_code(type), T = int_of(q.t.size(0)), D = int_of(q.t.size(2));
        if (k.t.size(0) != T || k.t.size(2) != D) refuse(PyExc_ValueError, "shapes of q and k disagree");
        if (!q.t.is_cuda()) refuse(PyExc_ValueError, "q must be a CUDA tensor");
        void *qp = q.on(q.t, "q", type), *kp = k.on(q.t, "k", type);
        const Turns turns(q.t, a[2], a[3], a[4], T);
        const bool inter = true_of(a[5]);
        const at::Tensor qo = rows_out(q.t, a[6], "q_out", a[9]), ko = rows_out(k.t, a[7], "k_out", a[9]);
        void *qop = data_of(q.t, qo, "q_out", type), *kop = data_of(q.t, ko, "k_out", type);
        int32_t* err = static_cast<int32_t*>(data_or_null(q.t, a[8], "error_count", at::kInt));
        const int Hq = int_of(q.t.size(1)), Hk = int_of(k.t.size(1));
        const int rc = on_device(q.t, a[9], [&](void* s) {
            return pa_rope(qop, kop, qp, kp, T, Hq, Hk, D, dtype, q.stride, k.stride, turns.pos, turns.axes,
                           turns.inv_freq, turns.axis, turns.rot, inter, err, s);
        }, "q and k");
        if (rc != PA_OK) return PyLong_FromLong(rc);
        PyObject *x = THPVariable_Wrap(qo), *y = x ? THPVariable_Wrap(ko) : nullptr;
        PyObject* pair = y ? PyTuple_Pack(2, x, y) : nullptr;
        Py_XDECREF(x);
        Py_XDECREF(y);
        return pair;
    });
}

// q, k_new, v_new, rope_pos, inv_freq, axis, interleaved, k_cache, v_cache, block_tables, seq_idx, pos, q_out, key_weights,
// key_pos, token_pos, slot_mapping, error_count, stream -> q_out
PyObject* rope_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 19)) return nullptr;
    return guarded([&] {
        const Rows q(a[0], "q"), k(a[1], "k_new"), v(a[2], "v_new");
        const Cache c(a[7], a[8]);
        const at::Tensor &bt = tensor(a[9], "block_tables"), &seq = tensor(a[10], "seq_idx"), &pos = tensor(a[11], "pos");
        const int T = int_of(k.t.size(0)), Hq = int_of(q.t.size(1));
        if (k.t.size(1) != c.heads || k.t.size(2) != c.dim || !k.t.sizes().equals(v.t.sizes()) || q.t.size(0) != T ||
            q.t.size(2) != c.dim)
            refuse(PyExc_ValueError, "shapes of q, k_new, v_new and the pools disagree");
        if (seq.numel() != T || pos.numel() != T || (a[15] != Py_None && tensor(a[15], "token_pos").numel() != T) ||
            (a[16] != Py_None && tensor(a[16], "slot_mapping").numel() != T))
            refuse(PyExc_ValueError, "seq_idx, pos, token_pos and slot_mapping must have one entry for each of the " +
                                         std::to_string(T) + " tokens");
        if (bt.dim() != 2) refuse(PyExc_ValueError, "block_tables must be [num_seqs, max_blocks_per_seq]");
        void *qp = q.on(c.k, "q", c.type), *kp = k.on(c.k, "k_new", c.type), *vp = v.on(c.k, "v_new", c.type);
        const Turns turns(c.k, a[3], a[4], a[5], T);
        const bool inter = true_of(a[6]);
        const int S = int_of(bt.size(0)), W = int_of(bt.size(1));
        float* weights = static_cast<float*>(data_or_null(c.k, a[13], "key_weights", at::kFloat));
        int32_t* places = static_cast<int32_t*>(data_or_null(c.k, a[14], "key_pos", at::kInt));
        if ((a[13] == Py_None) != (a[14] == Py_None))
            refuse(PyExc_ValueError, "key_weights and key_pos are given together");
        int width = 0;
        if (a[13] != Py_None) {
            width = key_rows(tensor(a[13], "key_weights"), "key_weights", S, c.heads);
            if (key_rows(tensor(a[14], "key_pos"), "key_pos", S, c.heads) != width)
                refuse(PyExc_ValueError, "shapes of key_weights and key_pos differ");
        }
        const at::Tensor qo = rows_out(q.t, a[12], "q_out", a[18]);
        void* qop = c.at(qo, "q_out", c.type);
        const int32_t *btp = i32(c.at(bt, "block_tables", at::kInt)), *sp = i32(c.at(seq, "seq_idx", at::kInt)),
                      *pp = i32(c.at(pos, "pos", at::kInt)),
                      *tp = i32(data_or_null(c.k, a[15], "token_pos", at::kInt));
        int64_t* slots = static_cast<int64_t*>(data_or_null(c.k, a[16], "slot_mapping", at::kLong));
        int32_t* err = static_cast<int32_t*>(data_or_null(c.k, a[17], "error_count", at::kInt));
        const int rc = on_device(c.k, a[18], [&](void* s) {
            return pa_rope_write_kv_paged(qop, qp, kp, vp, T, Hq, c.heads, c.dim, c.dtype, q.stride, k.stride, v.stride,
                                          turns.pos, turns.axes, turns.inv_freq, turns.axis, turns.rot, inter, c.kp, c.vp,
                                          c.blocks, c.block, btp, S, W, sp, pp, weights, places, width, tp, slots, err, s);
        });
        return rc != PA_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(qo);
    });
}

// q, k_cache, v_cache, block_tables, context_lens, max_context_len, scale, key_weights, workspace, out, error_count,
// stream -> out
PyObject* decode_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 12)) return nullptr;
    return guarded([&] {
        const at::Tensor& q = tensor(a[0], "q");
        const Cache c(a[1], a[2]);
        const at::Tensor &bt = tensor(a[3], "block_tables"), &ctx = tensor(a[4], "context_lens"),
                         &weights = tensor(a[7], "key_weights");
        if (q.dim() != 3 || q.size(2) != c.dim) refuse(PyExc_ValueError, "head_dim of q and k_cache differ");
        const int N = int_of(q.size(0)), Hq = int_of(q.size(1));
        if (bt.dim() != 2 || bt.size(0) != N || ctx.numel() != N ||
            (a[9] != Py_None && !tensor(a[9], "out").sizes().equals(q.sizes())))
            refuse(PyExc_ValueError, "shapes of q, out, block_tables and context_lens disagree");
        const int max_ctx = int_of(a[5]), width = key_rows(weights, "key_weights", N, c.heads), W = int_of(bt.size(1));
        const float scale = float_of(a[6]);
        void* qp = c.at(q, "q", c.type);
        const at::Tensor out = a[9] == Py_None ? new_output(c.k, a[11], q.sizes(), c.type) : tensor(a[9], "out");
        void* op = c.at(out, "out", c.type, true);
        float* wp = static_cast<float*>(c.at(weights, "key_weights", at::kFloat));
        const int32_t *btp = i32(c.at(bt, "block_tables", at::kInt)), *cp = i32(c.at(ctx, "context_lens", at::kInt));
        int32_t* err = static_cast<int32_t*>(data_or_null(c.k, a[10], "error_count", at::kInt));
        const Scratch ws(c.k, a[8]);
        const int rc = on_device(c.k, a[11], [&](void* s) {
            return pa_decode_weights(op, qp, N, Hq, c.heads, c.dim, c.dtype, c.kp, c.vp, c.blocks, c.block, btp, W, cp,
                                     max_ctx, scale, wp, width, ws.ptr, ws.bytes, err, s);
        });
        return rc != PA_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
    });
}

// q, cu_q_lens, q_start_pos, seq_of_chunk, max_q_len, k_cache, v_cache, block_tables, context_lens, max_context_len, scale,
// key_weights, workspace, out, error_count, stream -> out
PyObject* prefill_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 16)) return nullptr;
    return guarded([&] {
        const at::Tensor &q = tensor(a[0], "q"), &cu = tensor(a[1], "cu_q_lens"), &start = tensor(a[2], "q_start_pos"),
                         &seq = tensor(a[3], "seq_of_chunk");
        const Cache c(a[5], a[6]);
        const at::Tensor &bt = tensor(a[7], "block_tables"), &ctx = tensor(a[8], "context_lens"),
                         &weights = tensor(a[11], "key_weights");
        if (q.dim() != 3 || q.size(2) != c.dim) refuse(PyExc_ValueError, "head_dim of q and k_cache differ");
        const int T = int_of(q.size(0)), Hq = int_of(q.size(1)), C = int_of(start.numel());
        if (cu.numel() != C + 1 || seq.numel() != C ||
            (a[13] != Py_None && !tensor(a[13], "out").sizes().equals(q.sizes())))
            refuse(PyExc_ValueError, "shapes of q, out, cu_q_lens, q_start_pos and seq_of_chunk disagree");
        if (bt.dim() != 2 || bt.size(0) != ctx.numel())
            refuse(PyExc_ValueError, "shapes of block_tables and context_lens disagree");
        const int S = int_of(bt.size(0)), W = int_of(bt.size(1)), max_q = int_of(a[4]), max_ctx = int_of(a[9]);
        const int width = key_rows(weights, "key_weights", S, c.heads);
        const float scale = float_of(a[10]);
        void* qp = c.at(q, "q", c.type);
        const at::Tensor out = a[13] == Py_None ? new_output(c.k, a[15], q.sizes(), c.type) : tensor(a[13], "out");
        void* op = c.at(out, "out", c.type, true);
        float* wp = static_cast<float*>(c.at(weights, "key_weights", at::kFloat));
        const int32_t *cup = i32(c.at(cu, "cu_q_lens", at::kInt)), *st = i32(c.at(start, "q_start_pos", at::kInt)),
                      *sq = i32(c.at(seq, "seq_of_chunk", at::kInt)), *btp = i32(c.at(bt, "block_tables", at::kInt)),
                      *cp = i32(c.at(ctx, "context_lens", at::kInt));
        int32_t* err = static_cast<int32_t*>(data_or_null(c.k, a[14], "error_count", at::kInt));
        const Scratch ws(c.k, a[12]);
        const int rc = on_device(c.k, a[15], [&](void* s) {
            return pa_prefill_chunk_weights(op, qp, cup, st, sq, C, T, max_q, S, Hq, c.heads, c.dim, c.dtype, c.kp, c.vp,
                                            c.blocks, c.block, btp, W, cp, max_ctx, scale, wp, width, ws.ptr, ws.bytes,
                                            err, s);
        });
        return rc != PA_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
    });
}

// k_cache, v_cache, block_tables, context_lens, max_context_len, key_weights, key_pos, next_pos, budget, keep_first,
// keep_recent, workspace, new_lens, error_count, stream -> new_lens
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!counted(n, 15)) return nullptr;
    return guarded([&] {
        const Cache c(a[0], a[1]);
        const at::Tensor &bt = tensor(a[2], "block_tables"), &ctx = tensor(a[3], "context_lens"),
                         &weights = tensor(a[5], "key_weights"), &places = tensor(a[6], "key_pos"),
                         &next = tensor(a[7], "next_pos");
        if (bt.dim() != 2 || bt.size(0) != ctx.numel() || next.numel() != ctx.numel() ||
            (a[12] != Py_None && tensor(a[12], "new_lens").numel() != ctx.numel()))
            refuse(PyExc_ValueError, "shapes of block_tables, context_lens, next_pos and new_lens disagree");
        const int S = int_of(bt.size(0)), W = int_of(bt.size(1)), max_ctx = int_of(a[4]), budget = int_of(a[8]),
                  first = int_of(a[9]), recent = int_of(a[10]);
        const int width = key_rows(weights, "key_weights", S, c.heads);
        if (key_rows(places, "key_pos", S, c.heads) != width)
            refuse(PyExc_ValueError, "shapes of key_weights and key_pos differ");
        const int32_t *btp = i32(c.at(bt, "block_tables", at::kInt)), *cp = i32(c.at(ctx, "context_lens", at::kInt)),
                      *np = i32(c.at(next, "next_pos", at::kInt));
        float* wp = static_cast<float*>(c.at(weights, "key_weights", at::kFloat));
        int32_t* pp = static_cast<int32_t*>(c.at(places, "key_pos", at::kInt));
        const at::Tensor lens = a[12] == Py_None ? new_output(c.k, a[14], ctx.sizes(), at::kInt) : tensor(a[12], "new_lens");
        int32_t* lp = static_cast<int32_t*>(c.at(lens, "new_lens", at::kInt));
        int32_t* err = static_cast<int32_t*>(data_or_null(c.k, a[13], "error_count", at::kInt));
        const Scratch ws(c.k, a[11]);
        const int rc = on_device(c.k, a[14], [&](void* s) {
            return pa_evict_tokens(c.kp, c.vp, c.blocks, c.block, c.heads, c.dim, c.dtype, btp, S, W, cp, max_ctx, wp, pp,
                                   width, np, budget, first, recent, lp, ws.ptr, ws.bytes, err, s);
        });
        return rc != PA_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(lens);
    });
}

PyMethodDef methods[] = {
    {"write", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(write)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(read)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode)), METH_FASTCALL, nullptr},
    {"prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prefill)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope)), METH_FASTCALL, nullptr},
    {"rope_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope_write)), METH_FASTCALL, nullptr},
    {"decode_weights", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode_weights)), METH_FASTCALL, nullptr},
    {"prefill_weights", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prefill_weights)), METH_FASTCALL, nullptr},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(evict)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_bind(void) { return PyModule_Create(&module); }
