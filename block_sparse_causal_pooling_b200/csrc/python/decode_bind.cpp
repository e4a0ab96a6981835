// Native part of the decode binding (decode.py): argument checks, outputs and the calls into
// libstem.so, as one extension module.
//
// A generating program makes two such calls a layer. Marshalled in Python (checks, five tensors, an
// argument struct, the stream) they were bound by the host: 27 us for 16 new tokens whose kernel takes
// 8, 48 for a decode step of 16. Here a call takes about 1 us more than its kernels. Nothing is
// computed in this file.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <structmember.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "stem.h"

namespace {

PyObject* g_error = nullptr;  // StemError(code, where)

struct Failed {};  // a Python exception is set

[[noreturn]] void fail(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Failed{};
}

void check_rc(int rc, const char* where) {
  if (rc == STEM_OK) return;
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", rc, where) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Failed{};
}

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t n = 0; n < s.size(); ++n) t += (n ? ", " : "") + std::to_string(s[n]);
  return t + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

void need(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape,
          at::Device dev) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " +
                              c10::toString(t.scalar_type()));
  if (t.sizes() != shape)
    fail(PyExc_ValueError, std::string(name) + " must have shape " + text(shape) + ", got " +
                               text(t.sizes()));
  if (t.device() != dev)
    fail(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", the cache on " +
                               dev.str());
  if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + " must be contiguous");
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  return v;
}

int32_t narrow(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX)
    fail(PyExc_ValueError, std::string(name) + " is out of range");
  return static_cast<int32_t>(v);
}

// ------------------------------------------------------------------ the cache

struct Cache {
  PyObject_HEAD
  stem_cache_t c;
  PyObject* tensors[4];  // pages, kbar, vnorm, table: kept alive
  int device;
};

PyTypeObject* g_cache = nullptr;

const Cache& cache_of(PyObject* o) {
  if (!PyObject_TypeCheck(o, g_cache)) fail(PyExc_TypeError, "cache must be a PagedCache");
  const Cache& c = *reinterpret_cast<Cache*>(o);
  if (!c.tensors[0]) fail(PyExc_ValueError, "the PagedCache was not initialised");
  return c;
}

at::Device device_of(const Cache& c) {
  return at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(c.device));
}

// (pages, kbar, vnorm, table, block, format, vsum)
int cache_init(PyObject* self, PyObject* args, PyObject*) {
  Cache& c = *reinterpret_cast<Cache*>(self);
  PyObject* t[4];
  int block, format, vsum;
  if (!PyArg_ParseTuple(args, "OOOOiii", &t[0], &t[1], &t[2], &t[3], &block, &format, &vsum))
    return -1;
  try {
    const at::Tensor &pages = tensor(t[0], "pages"), &kbar = tensor(t[1], "kbar"),
                     &vnorm = tensor(t[2], "vnorm"), &table = tensor(t[3], "table");
    if (kbar.dim() != 3 || table.dim() != 2)
      fail(PyExc_ValueError, "kbar must be [num_pages, Hkv, D] and table [nseq, max_blocks]");
    const int64_t n = kbar.size(0), Hkv = kbar.size(1), D = kbar.size(2);
    const int64_t size = stem_cache_page_bytes(narrow(D, "D"), block, format);
    if (size == 0)
      fail(PyExc_ValueError, "D and block must be 64 or 128, got " + std::to_string(D) + " and " +
                                 std::to_string(block));
    const at::Device dev = pages.device();
    if (!dev.is_cuda())
      fail(PyExc_ValueError, "the cache must be on a CUDA device, got " + dev.str());
    need(pages, "pages", at::kByte, {n, Hkv, size}, dev);
    need(kbar, "kbar", at::kFloat, {n, Hkv, D}, dev);
    need(vnorm, "vnorm", at::kFloat, {n, Hkv}, dev);
    need(table, "table", at::kInt, table.sizes(), dev);
    stem_cache_t s;
    s.pages = pages.data_ptr();
    s.kbar = static_cast<float*>(kbar.data_ptr());
    s.vnorm = static_cast<float*>(vnorm.data_ptr());
    s.table = static_cast<const int32_t*>(table.data_ptr());
    s.num_pages = narrow(n, "num_pages");
    s.Hkv = narrow(Hkv, "Hkv");
    s.D = static_cast<int32_t>(D);
    s.block = block;
    s.format = format;
    s.nseq = narrow(table.size(0), "nseq");
    s.max_blocks = narrow(table.size(1), "max_blocks");
    s.vsum = vsum;
    c.c = s;
    c.device = dev.index();
    for (int i = 0; i < 4; ++i) {
      PyObject* old = c.tensors[i];
      c.tensors[i] = Py_NewRef(t[i]);
      Py_XDECREF(old);
    }
  } catch (const Failed&) {
    return -1;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return -1;
  }
  return 0;
}

void cache_dealloc(PyObject* self) {
  Cache& c = *reinterpret_cast<Cache*>(self);
  for (PyObject* t : c.tensors) Py_XDECREF(t);
  PyTypeObject* type = Py_TYPE(self);
  type->tp_free(self);
  Py_DECREF(type);
}

PyMemberDef cache_members[] = {
    {"pages", T_OBJECT_EX, offsetof(Cache, tensors[0]), READONLY, nullptr},
    {"kbar", T_OBJECT_EX, offsetof(Cache, tensors[1]), READONLY, nullptr},
    {"vnorm", T_OBJECT_EX, offsetof(Cache, tensors[2]), READONLY, nullptr},
    {"table", T_OBJECT_EX, offsetof(Cache, tensors[3]), READONLY, nullptr},
    {"Hkv", T_INT, offsetof(Cache, c.Hkv), READONLY, nullptr},
    {"D", T_INT, offsetof(Cache, c.D), READONLY, nullptr},
    {"block", T_INT, offsetof(Cache, c.block), READONLY, nullptr},
    {"format", T_INT, offsetof(Cache, c.format), READONLY, nullptr},
    {"nseq", T_INT, offsetof(Cache, c.nseq), READONLY, nullptr},
    {"max_blocks", T_INT, offsetof(Cache, c.max_blocks), READONLY, nullptr},
    {"vsum_code", T_INT, offsetof(Cache, c.vsum), READONLY, nullptr},
    {nullptr, 0, 0, 0, nullptr}};

PyType_Slot cache_slots[] = {{Py_tp_init, reinterpret_cast<void*>(cache_init)},
                             {Py_tp_new, reinterpret_cast<void*>(PyType_GenericNew)},
                             {Py_tp_dealloc, reinterpret_cast<void*>(cache_dealloc)},
                             {Py_tp_members, cache_members},
                             {0, nullptr}};
PyType_Spec cache_spec = {"block_sparse_causal_pooling_b200._decode.Cache", sizeof(Cache), 0,
                          Py_TPFLAGS_DEFAULT | Py_TPFLAGS_BASETYPE, cache_slots};

// ------------------------------------------------------------------ calls

const int32_t* ints(PyObject* o, const char* name, at::IntArrayRef shape, at::Device dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  need(t, name, at::kInt, shape, dev);
  return static_cast<const int32_t*>(t.data_ptr());
}

// None: torch's current stream of the device; else a cudaStream_t's address.
c10::cuda::CUDAStream stream_of(PyObject* o, int device) {
  const auto dev = static_cast<c10::DeviceIndex>(device);
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev);
  return c10::cuda::getStreamFromExternal(
      reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(integer(o))), dev);
}

bool count_is(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return false;
}

// (cache, k, v, pos, count, status, stream)
PyObject* rows(bool write, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 7)) return nullptr;
  try {
    const Cache& c = cache_of(a[0]);
    const at::Device dev = device_of(c);
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const stem_cache_t& s = c.c;
    if (k.dim() != 4 || k.size(0) != s.nseq || k.size(1) != s.Hkv || k.size(3) != s.D)
      fail(PyExc_ValueError, "k must be [" + std::to_string(s.nseq) + ", " +
                                 std::to_string(s.Hkv) + ", T, " + std::to_string(s.D) +
                                 "], got " + text(k.sizes()));
    bool alike = v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type();
    for (int64_t n = 0; alike && n < 4; ++n)  // (the stride of an axis of one row says nothing)
      alike = k.size(n) == 1 || v.stride(n) == k.stride(n);
    if (!alike) fail(PyExc_ValueError, "k and v must have the same shape, dtype and strides");
    if (k.device() != dev || v.device() != dev)
      fail(PyExc_ValueError, "k and v must be on the cache's device " + dev.str());
    if (k.stride(3) != 1)
      fail(PyExc_ValueError, "k and v must be contiguous in their last dimension");
    if (k.scalar_type() != at::kBFloat16 && k.scalar_type() != at::kFloat)
      fail(PyExc_TypeError, std::string("k and v must be bfloat16 or float32, got ") +
                                c10::toString(k.scalar_type()));
    const int dtype = k.scalar_type() == at::kBFloat16 ? STEM_BF16 : STEM_F32;
    const int32_t* pos = ints(a[3], "pos", {s.nseq}, dev);
    const int32_t* count = ints(a[4], "count", {s.nseq}, dev);
    auto* status = const_cast<int32_t*>(ints(a[5], "status", {1}, dev));
    void* st = stream_of(a[6], c.device).stream();
    const int64_t strides[3] = {k.stride(0), k.stride(1), k.stride(2)};
    const int T = narrow(k.size(2), "T");
    void *kp = k.data_ptr(), *vp = v.data_ptr();
    c10::cuda::CUDAGuard guard(dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = write ? stem_cache_append(&s, kp, vp, dtype, T, strides, pos, count, status, st)
               : stem_cache_read(&s, kp, vp, dtype, T, strides, pos, count, status, st);
    Py_END_ALLOW_THREADS
    check_rc(rc, write ? "stem_cache_append" : "stem_cache_read");
    Py_RETURN_NONE;
  } catch (const Failed&) {
    return nullptr;
  }
}

PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return rows(true, a, n);
  END_HANDLE_TH_ERRORS
}
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return rows(false, a, n);
  END_HANDLE_TH_ERRORS
}

// A given output, checked, or a new one.
at::Tensor output(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape,
                  at::Device dev) {
  if (o == Py_None) return at::detail::empty_cuda(shape, type, dev, c10::nullopt);
  const at::Tensor& t = tensor(o, name);
  need(t, name, type, shape, dev);
  return t;
}

enum { kSelect = 1, kAttend = 2 };

// (what, cache, q, lens, rows, budget, kcap, method address, sel_idx, sel_cnt, out, lse, workspace,
//  status, stream) -> (out, lse, sel_idx, sel_cnt), None where what does not ask for it
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 15)) return nullptr;
  try {
    const int64_t what = integer(a[0]);
    const char* name = what == kSelect   ? "stem_decode_select"
                       : what == kAttend ? "stem_decode_attn"
                                         : "stem_decode";
    const Cache& c = cache_of(a[1]);
    const stem_cache_t& s = c.c;
    const at::Device dev = device_of(c);
    const at::Tensor& q = tensor(a[2], "q");
    if (q.dim() != 3 || q.size(2) != s.D)
      fail(PyExc_ValueError, "q must be [R, Hq, " + std::to_string(s.D) + "], got " + text(q.sizes()));
    const int64_t R = q.size(0), Hq = q.size(1), kcap = integer(a[6]);
    need(q, "q", at::kBFloat16, q.sizes(), dev);
    if (kcap < 1) fail(PyExc_ValueError, "kcap must be at least 1");
    if (kcap > s.max_blocks) check_rc(STEM_ERR_ARG, name);  // (before lists of that size are made)
    stem_decode_args_t d = {};
    d.cache = &s;
    d.q = q.data_ptr();
    d.lens = ints(a[3], "lens", {R}, dev);
    d.rows = ints(a[4], "rows", {R}, dev);
    d.budget = ints(a[5], "budget", {s.max_blocks}, dev);
    d.R = narrow(R, "R");
    d.Hq = narrow(Hq, "Hq");
    d.kcap = narrow(kcap, "kcap");
    d.dtype = STEM_BF16;
    d.method = reinterpret_cast<const stem_method_t*>(static_cast<uintptr_t>(integer(a[7])));
    d.status = const_cast<int32_t*>(ints(a[13], "status", {1}, dev));
    // (what is made here is made for the call's stream: the allocator may hand out memory that work
    // on another stream still uses)
    const c10::cuda::CUDAStream stream = stream_of(a[14], c.device);
    c10::cuda::CUDAStreamGuard guard(stream);
    void* st = stream.stream();
    const at::Tensor idx = output(a[8], "sel_idx", at::kInt, {R, Hq, kcap}, dev);
    const at::Tensor cnt = output(a[9], "sel_cnt", at::kInt, {R, Hq}, dev);
    d.sel_idx = static_cast<int32_t*>(idx.data_ptr());
    d.sel_cnt = static_cast<int32_t*>(cnt.data_ptr());
    at::Tensor out, lse, workspace;
    if (what & kAttend) {
      out = output(a[10], "out", at::kBFloat16, q.sizes(), dev);
      lse = output(a[11], "lse", at::kFloat, {R, Hq}, dev);
      d.out = out.data_ptr();
      d.lse = static_cast<float*>(lse.data_ptr());
      if (a[12] == Py_None) {
        workspace = at::detail::empty_cuda(
            {static_cast<int64_t>(stem_decode_workspace_size(&s, d.R, d.Hq, d.kcap))}, at::kByte,
            dev, c10::nullopt);
      } else {
        workspace = tensor(a[12], "workspace");
        need(workspace, "workspace", at::kByte, workspace.sizes(), dev);
      }
      d.workspace = workspace.data_ptr();
      d.workspace_bytes = static_cast<size_t>(workspace.numel());
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = what == kSelect ? stem_decode_select(&d, st)
                         : what == kAttend ? stem_decode_attn(&d, st) : stem_decode(&d, st);
    Py_END_ALLOW_THREADS
    check_rc(rc, name);
    // given tensors go back as the objects they came as
    auto back = [](PyObject* given, const at::Tensor& t) {
      if (given != Py_None || !t.defined()) return Py_NewRef(given);
      return THPVariable_Wrap(t);
    };
    PyObject* r[4] = {back(a[10], out), back(a[11], lse), back(a[8], idx), back(a[9], cnt)};
    PyObject* all = r[0] && r[1] && r[2] && r[3] ? PyTuple_New(4) : nullptr;
    for (int i = 0; i < 4; ++i) {
      if (all)
        PyTuple_SET_ITEM(all, i, r[i]);
      else
        Py_XDECREF(r[i]);
    }
    return all;
  } catch (const Failed&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (cache, R, Hq, kcap)
PyObject* workspace_size(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 4)) return nullptr;
  try {
    const Cache& c = cache_of(a[0]);
    c10::cuda::CUDAGuard guard(device_of(c));
    return PyLong_FromSize_t(stem_decode_workspace_size(
        &c.c, narrow(integer(a[1]), "R"), narrow(integer(a[2]), "Hq"), narrow(integer(a[3]), "kcap")));
  } catch (const Failed&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  PyObject* old = g_error;
  g_error = Py_NewRef(type);
  Py_XDECREF(old);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(read)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode)), METH_FASTCALL, nullptr},
    {"workspace_size", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(workspace_size)),
     METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode() {
  PyObject* m = PyModule_Create(&module);
  if (!m) return nullptr;
  g_cache = reinterpret_cast<PyTypeObject*>(PyType_FromSpec(&cache_spec));
  if (!g_cache || PyModule_AddObjectRef(m, "Cache", reinterpret_cast<PyObject*>(g_cache)) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
