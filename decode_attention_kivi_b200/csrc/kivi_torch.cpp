// kivi_torch.cpp - the Python side of the paged-cache and packed-attention calls:
// checks of the torch tensors and the call of the C ABI.
//
// A step of a server makes several of these calls per layer on small tensors.
// The same checks and the marshalling of some twenty arguments in Python take 8
// to 15 us a call, longer than the kernels of a small step; here they take about
// one.  The C functions are called by the addresses that the loader passes, so
// that this module serves whatever build of the library was loaded.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/kivi.h"

namespace {

decltype(&kivi_paged_assign) f_assign;
decltype(&kivi_paged_append) f_append;
decltype(&kivi_packed_attention) f_packed;
decltype(&kivi_paged_attention) f_paged;

// A call's tensors; every check after a failed one is skipped.
struct Call {
  bool ok = true;
  int device = -2;
  int count = 0;
  const at::Tensor* used[16];  // of a call; some twice

  template <typename... A>
  void fail(const char* format, A... args) {
    if (ok) PyErr_Format(PyExc_ValueError, format, args...);
    ok = false;
  }
  void require(bool condition, const char* message) {
    if (ok && !condition) fail("%s", message);
  }
  // The tensor behind `o`, on the call's device (that of its first tensor).
  const at::Tensor* tensor(PyObject* o, const char* name) {
    if (!ok) return nullptr;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    const int dev = t.is_cuda() ? (int)t.get_device() : -1;
    if (device == -2) device = dev;
    if (dev < 0)
      fail("%s: tensors must be CUDA tensors", name);
    else if (dev != device)
      fail("tensors on cuda:%d and cuda:%d: one device is needed", device, dev);
    if (ok) used[count++] = &t;
    return &t;
  }
  // The call runs on the current device, whose stream it takes.
  void on_current_device() {
    if (!ok) return;
    const int current = (int)c10::cuda::current_device();
    if (device != current) fail("tensors on cuda:%d, but cuda:%d is current", device, current);
  }
  int32_t* ints(PyObject* o, std::initializer_list<int64_t> shape, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!ok) return nullptr;
    if (t->scalar_type() != at::kInt || !t->is_contiguous() ||
        t->sizes() != at::IntArrayRef(shape.begin(), shape.size())) {
      fail("%s must be a contiguous int32 tensor of the call's shape", name);
      return nullptr;
    }
    return static_cast<int32_t*>(t->data_ptr());
  }
  // Elements between the rows of t [rows][heads][channels]: a row is contiguous, rows may be apart
  // (a slice of a wider projection).
  int64_t row_stride(const at::Tensor* t, const char* name) {
    if (!ok) return 0;
    const int64_t heads = t->size(1), dim = t->size(2);
    if ((t->stride(2) != 1 && dim > 1) || (t->stride(1) != dim && heads > 1))
      fail("%s: heads and channels of a row must be contiguous", name);
    return t->size(0) < 2 ? heads * dim : t->stride(0);
  }
  // The call's stream, asked for last: the current one, a torch stream, or a handle.  Torch is told
  // that the tensors are used on a stream of its own other than the current one, so that the caller
  // may drop them right after the call.  A handle may be gone by the time a tensor is dropped, so the
  // caller keeps the tensors until that stream has run the call.
  void* stream(PyObject* o) {
    if (!ok) return nullptr;
    const auto current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device);
    if (o == Py_None) return current.stream();
    if (!THPStream_Check(o)) {
      void* s = PyLong_AsVoidPtr(o);
      if (PyErr_Occurred()) ok = false;
      return s;
    }
    const auto* t = reinterpret_cast<THPStream*>(o);
    const auto s = c10::cuda::CUDAStream::unpack3(
        t->stream_id, (c10::DeviceIndex)t->device_index, (c10::DeviceType)t->device_type);
    if (s.device_index() != device) {
      fail("stream on cuda:%d, but the tensors are on cuda:%d", (int)s.device_index(), device);
      return nullptr;
    }
    if (s != current)
      for (int i = 0; i < count; ++i)
        c10::cuda::CUDACachingAllocator::recordStream(used[i]->storage().data_ptr(), s);
    return s.stream();
  }
  int32_t int32(PyObject* o) {
    if (!ok) return 0;
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
      ok = false;
      return 0;
    }
    if (v < INT32_MIN || v > INT32_MAX) fail("an integer argument does not fit 32 bits");
    return (int32_t)v;
  }
};

bool rows_type(const at::Tensor& t) {
  return t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf;
}
int32_t type_of(const at::Tensor& t) { return t.scalar_type() == at::kHalf ? KIVI_FP16 : KIVI_BF16; }

// Sizes of the calls are int32 in the C ABI.
bool int32_sizes(const at::Tensor& t) {
  for (const int64_t n : t.sizes())
    if (n > INT32_MAX) return false;
  return true;
}

struct Pages {
  const at::Tensor *k, *v;
};
Pages pages_of(Call& c, PyObject* k, PyObject* v, const at::Tensor* like) {
  Pages p{c.tensor(k, "k_pages"), c.tensor(v, "v_pages")};
  if (!c.ok) return p;
  c.require(p.k->dim() == 4 && p.k->sizes() == p.v->sizes() && int32_sizes(*p.k),
            "pages: k and v [num_pages][Hkv][page_size][D]");
  c.require(rows_type(*p.k) && p.v->scalar_type() == p.k->scalar_type() &&
                p.k->scalar_type() == like->scalar_type(),
            "pages must be bf16 or fp16 like the rows");
  c.require(p.k->is_contiguous() && p.v->is_contiguous(), "pages must be contiguous");
  return p;
}

bool arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments needed, got %zd", want, got);
  return false;
}

// assign(lengths, new_tokens, block_table, free_pages, num_free, page_size, kv_lengths,
//        num_free_out, offsets, slots, positions, status, stream) -> status of the C call
PyObject* assign(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 13)) return nullptr;
  Call c;
  const at::Tensor* table = c.tensor(a[2], "block_table");
  const at::Tensor* free = c.tensor(a[3], "free_pages");
  const at::Tensor* slots = c.tensor(a[9], "slots");
  if (!c.ok) return nullptr;
  c.require(table->dim() == 2 && free->dim() == 1 && slots->dim() == 1 && int32_sizes(*table) &&
                int32_sizes(*free) && int32_sizes(*slots),
            "block_table [B][W], free_pages [num_pages], slots [rows]");
  if (!c.ok) return nullptr;
  const int64_t B = table->size(0), width = table->size(1), pages = free->size(0),
                rows = slots->size(0);
  const int32_t* lengths = c.ints(a[0], {B}, "lengths");
  const int32_t* new_tokens = c.ints(a[1], {B}, "new_tokens");
  int32_t* t = c.ints(a[2], {B, width}, "block_table");
  int32_t* f = c.ints(a[3], {pages}, "free_pages");
  const int32_t* num_free = c.ints(a[4], {1}, "num_free");
  const int32_t page_size = c.int32(a[5]);
  int32_t* kv = c.ints(a[6], {B}, "kv_lengths");
  int32_t* num_free_out = c.ints(a[7], {1}, "num_free_out");
  int32_t* offsets = c.ints(a[8], {B + 1}, "offsets");
  int32_t* s = c.ints(a[9], {rows}, "slots");
  int32_t* positions = c.ints(a[10], {rows}, "positions");
  int32_t* status = c.ints(a[11], {1}, "status");
  c.on_current_device();
  void* stream = c.stream(a[12]);
  if (!c.ok) return nullptr;
  kivi_status rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f_assign(lengths, new_tokens, (int32_t)B, t, (int32_t)width, f, num_free, (int32_t)pages,
                page_size, kv, num_free_out, offsets, s, positions, (int32_t)rows,
                reinterpret_cast<uint32_t*>(status), stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
  END_HANDLE_TH_ERRORS
}

// append(k_new, v_new, slots, k_pages, v_pages, status or None, stream) -> status of the C call
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 7)) return nullptr;
  Call c;
  const at::Tensor* k = c.tensor(a[0], "k_new");
  const at::Tensor* v = c.tensor(a[1], "v_new");
  if (!c.ok) return nullptr;
  const Pages p = pages_of(c, a[3], a[4], k);
  if (!c.ok) return nullptr;
  const int64_t hkv = p.k->size(1), dim = p.k->size(3);
  c.require(k->dim() == 3 && k->size(1) == hkv && k->size(2) == dim && v->sizes() == k->sizes() &&
                v->scalar_type() == k->scalar_type() && int32_sizes(*k),
            "k_new and v_new must be [rows][Hkv][D] of the pages' type");
  if (!c.ok) return nullptr;
  const int64_t rows = k->size(0);
  const int32_t* slots = c.ints(a[2], {rows}, "slots");
  int32_t* status = a[5] == Py_None ? nullptr : c.ints(a[5], {1}, "status");
  const int64_t ks = c.row_stride(k, "k_new"), vs = c.row_stride(v, "v_new");
  c.on_current_device();
  void* stream = c.stream(a[6]);
  if (!c.ok) return nullptr;
  kivi_status rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f_append(k->data_ptr(), ks, v->data_ptr(), vs, slots, (int32_t)rows, p.k->data_ptr(),
                p.v->data_ptr(), (int32_t)p.k->size(0), (int32_t)p.k->size(2), (int32_t)hkv,
                (int32_t)dim, reinterpret_cast<uint32_t*>(status), stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
  END_HANDLE_TH_ERRORS
}

// q and out of an attention call, its offsets and its workspace.
struct Rows {
  const at::Tensor *q, *out, *offsets, *workspace;
  at::Tensor fresh;  // the output, where the caller gave none
  int64_t q_stride, out_stride;
  const int32_t* off;
  int32_t B, rows, hq, dim;
};

void rows_of(Call& c, Rows& r, PyObject* q, PyObject* out, PyObject* offsets, PyObject* workspace) {
  r.q = c.tensor(q, "q");
  r.offsets = c.tensor(offsets, "offsets");
  r.workspace = c.tensor(workspace, "workspace");
  if (!c.ok) return;
  c.require(r.q->dim() == 3 && int32_sizes(*r.q), "q must be [rows][Hq][D]");
  c.require(rows_type(*r.q), "q, k and v must all be bf16 or all fp16");
  c.require(r.offsets->dim() == 1 && r.offsets->numel() >= 1 && int32_sizes(*r.offsets),
            "offsets must be [requests + 1]");
  c.require(r.workspace->is_contiguous(), "workspace must be contiguous");
  if (!c.ok) return;
  r.B = (int32_t)(r.offsets->numel() - 1);
  r.rows = (int32_t)r.q->size(0);
  r.hq = (int32_t)r.q->size(1);
  r.dim = (int32_t)r.q->size(2);
  r.off = c.ints(offsets, {r.B + 1}, "offsets");
  r.q_stride = c.row_stride(r.q, "q");
  c.on_current_device();
  if (!c.ok) return;
  if (out == Py_None) {
    r.fresh = at::empty(r.q->sizes(), r.q->options());
    r.out = &r.fresh;
  } else {
    r.out = c.tensor(out, "out");
    if (!c.ok) return;
    c.require(r.out->sizes() == r.q->sizes() && r.out->scalar_type() == r.q->scalar_type(),
              "out must have the shape and type of q");
  }
  r.out_stride = c.row_stride(r.out, "out");
}

// The output tensor, or the C call's status where it failed.
PyObject* result(kivi_status rc, const Rows& r, PyObject* out) {
  if (rc != KIVI_OK) return PyLong_FromLong(rc);
  if (out == Py_None) return THPVariable_Wrap(r.fresh);
  Py_INCREF(out);
  return out;
}

// packed(q, k, v, offsets, workspace, out or None, sm_scale, stream) -> out, or a status
PyObject* packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 8)) return nullptr;
  Call c;
  Rows r{};
  rows_of(c, r, a[0], a[5], a[3], a[4]);
  const at::Tensor* k = c.tensor(a[1], "k");
  const at::Tensor* v = c.tensor(a[2], "v");
  if (!c.ok) return nullptr;
  c.require(k->dim() == 3 && k->size(0) == r.rows && k->size(2) == r.dim && int32_sizes(*k) &&
                v->sizes() == k->sizes(),
            "shapes: q and out [rows][Hq][D], k and v [rows][Hkv][D]");
  c.require(k->scalar_type() == r.q->scalar_type() && v->scalar_type() == r.q->scalar_type(),
            "q, k and v must all be bf16 or all fp16");
  const int64_t ks = c.row_stride(k, "k"), vs = c.row_stride(v, "v");
  const double scale = c.ok ? PyFloat_AsDouble(a[6]) : 0.0;
  if (c.ok && PyErr_Occurred()) c.ok = false;
  void* stream = c.stream(a[7]);
  if (!c.ok) return nullptr;
  kivi_status rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f_packed(r.q->data_ptr(), r.q_stride, k->data_ptr(), ks, v->data_ptr(), vs,
                r.out->data_ptr(), r.out_stride, type_of(*r.q), r.off, r.B, r.rows,
                (int32_t)k->size(1), r.hq, r.dim, (float)scale, r.workspace->data_ptr(),
                r.workspace->nbytes(), stream);
  Py_END_ALLOW_THREADS
  return result(rc, r, a[5]);
  END_HANDLE_TH_ERRORS
}

// paged(q, k_pages, v_pages, block_table, kv_lengths, offsets, workspace, max_new or None,
//       out or None, sm_scale, stream) -> out, or a status
PyObject* paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 11)) return nullptr;
  Call c;
  Rows r{};
  rows_of(c, r, a[0], a[8], a[5], a[6]);
  if (!c.ok) return nullptr;
  const Pages p = pages_of(c, a[1], a[2], r.q);
  const at::Tensor* table = c.tensor(a[3], "block_table");
  if (!c.ok) return nullptr;
  c.require(p.k->size(3) == r.dim && table->dim() == 2 && int32_sizes(*table),
            "shapes: q and out [rows][Hq][D], pages [num_pages][Hkv][page_size][D], table [B][W]");
  if (!c.ok) return nullptr;
  const int32_t width = (int32_t)table->size(1);
  const int32_t* t = c.ints(a[3], {r.B, width}, "block_table");
  const int32_t* kv = c.ints(a[4], {r.B}, "kv_lengths");
  const int32_t max_new = a[7] == Py_None ? (r.rows > 1 ? r.rows : 1) : c.int32(a[7]);
  const double scale = c.ok ? PyFloat_AsDouble(a[9]) : 0.0;
  if (c.ok && PyErr_Occurred()) c.ok = false;
  void* stream = c.stream(a[10]);
  if (!c.ok) return nullptr;
  kivi_status rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f_paged(r.q->data_ptr(), r.q_stride, p.k->data_ptr(), p.v->data_ptr(), r.out->data_ptr(),
               r.out_stride, type_of(*r.q), t, width, kv, r.off, r.B, r.rows, max_new,
               (int32_t)p.k->size(0), (int32_t)p.k->size(2), (int32_t)p.k->size(1), r.hq, r.dim,
               (float)scale, r.workspace->data_ptr(), r.workspace->nbytes(), stream);
  Py_END_ALLOW_THREADS
  return result(rc, r, a[8]);
  END_HANDLE_TH_ERRORS
}

// library(assign, append, packed, paged): the addresses of the C functions
PyObject* library(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 4)) return nullptr;
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  f_assign = reinterpret_cast<decltype(f_assign)>(p[0]);
  f_append = reinterpret_cast<decltype(f_append)>(p[1]);
  f_packed = reinterpret_cast<decltype(f_packed)>(p[2]);
  f_paged = reinterpret_cast<decltype(f_paged)>(p[3]);
  Py_RETURN_NONE;
}

#define KIVI_METHOD(f) {#f, (PyCFunction)(void*)f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KIVI_METHOD(library), KIVI_METHOD(assign), KIVI_METHOD(append),
                         KIVI_METHOD(packed),  KIVI_METHOD(paged),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kivi_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kivi_torch() {
  PyObject* m = PyModule_Create(&module);
  // what the build compiled this for, for the loader's check
  if (m != nullptr && PyModule_AddStringConstant(m, "target", KIVI_BINDING_TARGET) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
