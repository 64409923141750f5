// torch_calls.cpp -- the cache-side calls (append, page keys, page-selected and
// shared-prefix decode) taken from Python objects straight to the C ABI.
//
// These calls launch one to three kernels of a few microseconds each, less than
// argument checks in Python and a foreign-function call take: appending one
// token to each of 64 sequences took 9.0 us a call through them and 3 us on the
// device.  The checks are those of the binding, made on the tensors' own fields.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <limits>
#include <stdexcept>
#include <string>

#include "../../include/mla.h"

namespace {

constexpr int64_t kD = 576, kNope = 512, kPage = 64;

// A refused argument: ValueError with this text.
struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};
// A Python error is already set.
struct PythonError {};
// A library error: MLAError(code, mla_last_error()).
struct LibraryError {
  int code;
};

void require(bool ok, const char* what) {
  if (!ok) throw BadArgument(what);
}
void require(bool ok, const char* name, const std::string& what, int index) {
  if (!ok)
    throw BadArgument(std::string(name) + " must be " + what + " on cuda:" + std::to_string(index));
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw BadArgument(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t whole(PyObject* o) {
  PyObject* i = PyNumber_Index(o);
  if (!i) throw PythonError{};
  const long long v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
// An int of the C ABI; what does not fit is refused there as out of range.
int whole32(PyObject* o) {
  const int64_t v = whole(o);
  if (v > std::numeric_limits<int>::max() || v < std::numeric_limits<int>::min())
    throw BadArgument("an integer argument does not fit in 32 bits");
  return static_cast<int>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}

// `t` as a contiguous int32 tensor on device `index`.  An int64 value past int32 becomes
// the nearest int32: out of the cache's or the table's range as it was (a cast would wrap
// it onto another index).
at::Tensor int32_on(const at::Tensor& t, const char* name, int index) {
  require(t.is_cuda() && t.get_device() == index, name, "a tensor", index);
  if (t.scalar_type() != at::kInt) {
    require(t.scalar_type() == at::kLong, name, "int32 (or int64)", index);
    return t.clamp(std::numeric_limits<int>::min(), std::numeric_limits<int>::max())
        .to(at::kInt)
        .contiguous();
  }
  return t.contiguous();
}

// Device index of a CUDA bf16 [b, s_q, h_q, 576] query.
int query(const at::Tensor& q) {
  require(q.is_cuda() && q.dim() == 4 && q.size(3) == kD && q.scalar_type() == at::kBFloat16,
          "q must be CUDA bf16 [b, s_q, h_q, 576]");
  require(q.size(0) <= std::numeric_limits<int>::max() &&
              q.size(1) <= std::numeric_limits<int>::max() &&
              q.size(2) <= std::numeric_limits<int>::max(),
          "q is too large");
  return q.get_device();
}

void bf16_cache(const at::Tensor& c, int index) {
  require(c.is_cuda() && c.get_device() == index && c.dim() == 4 && c.size(1) == kPage &&
              c.size(3) == kD && c.scalar_type() == at::kBFloat16 && c.is_contiguous() &&
              c.size(0) <= std::numeric_limits<int>::max() &&
              c.size(2) <= std::numeric_limits<int>::max(),
          "kcache must be contiguous CUDA bf16 [NB, 64, h_kv, 576] on the queries' device");
}

// An output given by the caller, or a new one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type,
                  at::Device device) {
  if (o == Py_None) return at::empty(shape, at::TensorOptions().dtype(type).device(device));
  const at::Tensor& t = tensor(o, name);
  if (t.sizes() != shape || t.scalar_type() != type || !t.is_contiguous() || t.device() != device) {
    std::string want = std::string("contiguous ") + c10::toString(type) + " [";
    for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
    require(false, name, want + "]", device.index());
  }
  return t;
}

at::Tensor workspace(PyObject* o, size_t bytes, at::Device device) {
  if (o == Py_None)
    return at::empty({static_cast<int64_t>(bytes < 256 ? 256 : bytes)},
                     at::TensorOptions().dtype(at::kByte).device(device));
  const at::Tensor& t = tensor(o, "workspace");
  require(t.device() == device && t.is_contiguous(), "workspace", "contiguous", device.index());
  require(t.nbytes() >= bytes, "workspace too small");
  return t;
}

// The GIL, free for the life of this object: an exception that leaves it takes it back.
struct FreeGil {
  PyThreadState* state = PyEval_SaveThread();
  ~FreeGil() { PyEval_RestoreThread(state); }
};

// call(stream) with device `index` current, on its current stream; the GIL is
// free meanwhile, as in a ctypes call.  (What torch does here throws on a CUDA error.)
template <class Call>
void launch(int index, Call call) {
  int rc;
  {
    FreeGil free_gil;
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    rc = call(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
  }
  if (rc != MLA_OK) throw LibraryError{rc};
}

void check(int rc) {
  if (rc != MLA_OK) throw LibraryError{rc};
}

// MLAError(code, text) of the binding; no library message is longer than its
// thread's buffer, which holds the text of the failed call.
void set_library_error(int code) {
  PyObject* m = PyImport_ImportModule("mla_paged_kv_03_b200.binding");
  if (!m) return;
  PyObject* type = PyObject_GetAttrString(m, "MLAError");
  Py_DECREF(m);
  if (!type) return;
  PyObject* e = PyObject_CallFunction(type, "is", code, mla_last_error());
  if (e) PyErr_SetObject(type, e);
  Py_XDECREF(e);
  Py_DECREF(type);
}

// body() with its C++ exceptions turned into Python errors.
template <class Body>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, Body body) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
    return nullptr;
  }
  try {
    return body();
  } catch (const PythonError&) {
  } catch (const LibraryError& e) {
    set_library_error(e.code);
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {  // torch's own (out of memory, ..) as torch raises them
    std::exception_ptr e = std::current_exception();
    torch::translate_exception_to_python(e);
  }
  return nullptr;
}

float softmax_scale(PyObject* o) {
  return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(kD)))
                      : static_cast<float>(number(o));
}

PyObject* pack(std::initializer_list<at::Tensor> outputs) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(outputs.size()));
  if (!r) throw PythonError{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : outputs) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// (kv, slots, kcache, positions, norm_gain, eps, rope_base, rows) -> rows
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 8, [&]() -> PyObject* {
    const at::Tensor& cache = tensor(a[2], "kcache");
    const int64_t width = cache.dim() ? cache.size(-1) : 0;
    int row_bytes = 0;
    if (cache.scalar_type() == at::kBFloat16 && width == kD)
      row_bytes = 2 * kD;
    else if (cache.scalar_type() == at::kByte && (width == 656 || width == 528 || width == 288))
      row_bytes = static_cast<int>(width);
    require(row_bytes != 0,
            "kcache must be bf16 [..., 576] or uint8 [..., 656], [..., 528] or [..., 288]");
    const int64_t d = row_bytes >= 656 ? kD : kNope;
    at::Tensor kv = tensor(a[0], "kv");
    if (!(kv.is_cuda() && kv.dim() == 2 && kv.size(1) == d && kv.scalar_type() == at::kBFloat16))
      throw BadArgument("kv must be CUDA bf16 [n, " + std::to_string(d) + "] for " +
                        std::to_string(row_bytes) + "-byte cache rows");
    const int index = kv.get_device();
    const int64_t n = kv.size(0);
    require(cache.is_cuda() && cache.get_device() == index && cache.is_contiguous(), "kcache",
            "contiguous and", index);
    require(n <= std::numeric_limits<int>::max(), "kv has too many rows");
    if (n == 0) return Py_NewRef(a[7]);
    int64_t stride = n > 1 ? kv.stride(0) : d;
    if (kv.stride(1) != 1 || stride % 8 || stride < d || stride >= int64_t{1} << 32 ||
        reinterpret_cast<uintptr_t>(kv.data_ptr()) % 16) {
      kv = kv.clone(at::MemoryFormat::Contiguous);
      stride = d;
    }
    const at::Tensor slots = int32_on(tensor(a[1], "slots"), "slots", index);
    require(slots.dim() == 1 && slots.size(0) == n, "slots must be [n]");
    at::Tensor positions, gain, rows;
    if (a[3] != Py_None) {
      positions = int32_on(tensor(a[3], "positions"), "positions", index);
      require(positions.dim() == 1 && positions.size(0) == n, "positions must be [n]");
    }
    if (a[4] != Py_None) {
      gain = tensor(a[4], "norm_gain");
      require(gain.is_cuda() && gain.get_device() == index && gain.dim() == 1 &&
                  gain.size(0) == kNope,
              "norm_gain", "[512]", index);
      gain = gain.to(at::kFloat).contiguous();
    }
    if (a[7] != Py_None)
      rows = output(a[7], "rows", {n, d}, at::kBFloat16, kv.device());
    const double eps = number(a[5]), base = number(a[6]);
    launch(index, [&](cudaStream_t stream) {
      return mla_cache_append(kv.data_ptr(), stride, static_cast<int>(d),
                              static_cast<const int32_t*>(slots.data_ptr()),
                              positions.defined()
                                  ? static_cast<const int32_t*>(positions.data_ptr())
                                  : nullptr,
                              gain.defined() ? static_cast<const float*>(gain.data_ptr()) : nullptr,
                              static_cast<float>(eps), static_cast<float>(base),
                              static_cast<int>(n), cache.data_ptr(), cache.numel() / width,
                              row_bytes, rows.defined() ? rows.data_ptr() : nullptr, stream);
    });
    return Py_NewRef(a[7]);
  });
}

struct PageArgs {
  int blocks, batch, max_pages;
  const at::Tensor& cache;
  const at::Tensor& keys;
  const at::Tensor& scales;
  at::Tensor table, lengths;
};

// kcache, page_keys, page_scales, block_table, cache_seqlens
PageArgs page_args(PyObject* kcache, PyObject* page_keys, PyObject* page_scales,
                   PyObject* block_table, PyObject* cache_seqlens, int index) {
  const at::Tensor& cache = tensor(kcache, "kcache");
  bf16_cache(cache, index);
  const at::Tensor& keys = tensor(page_keys, "page_keys");
  const at::Tensor& scales = tensor(page_scales, "page_scales");
  require(keys.is_cuda() && keys.get_device() == index && keys.dim() == 2 &&
              keys.size(0) == cache.size(0) && keys.size(1) == kD &&
              keys.scalar_type() == at::kChar && keys.is_contiguous(),
          "page_keys", "contiguous int8 [NB, 576]", index);
  require(scales.is_cuda() && scales.get_device() == index && scales.dim() == 1 &&
              scales.size(0) == cache.size(0) && scales.scalar_type() == at::kFloat &&
              scales.is_contiguous(),
          "page_scales", "contiguous fp32 [NB]", index);
  const at::Tensor& table = tensor(block_table, "block_table");
  require(table.dim() == 2 && table.numel() <= std::numeric_limits<int>::max(),
          "block_table must be [b, max_pages]");
  const at::Tensor& lengths = tensor(cache_seqlens, "cache_seqlens");
  require(lengths.dim() == 1 && lengths.size(0) == table.size(0), "cache_seqlens must be [b]");
  return {static_cast<int>(cache.size(0)), static_cast<int>(table.size(0)),
          static_cast<int>(table.size(1)), cache, keys, scales,
          int32_on(table, "block_table", index), int32_on(lengths, "cache_seqlens", index)};
}

// (kcache, block_table, cache_seqlens, page_keys, page_scales, tail_pages) -> None
PyObject* page_keys_update(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 6, [&]() -> PyObject* {
    const at::Tensor& cache = tensor(a[0], "kcache");
    const int index = cache.is_cuda() ? static_cast<int>(cache.get_device()) : -1;
    const PageArgs p = page_args(a[0], a[3], a[4], a[1], a[2], index);
    require(cache.size(2) == 1, "kcache must be [NB, 64, 1, 576]");
    const int tail = a[5] == Py_None ? p.max_pages : whole32(a[5]);
    if (p.batch == 0) Py_RETURN_NONE;  // (empty tensors have no address)
    launch(index, [&](cudaStream_t stream) {
      return mla_page_keys_update(cache.data_ptr(), p.blocks,
                                  static_cast<const int32_t*>(p.table.data_ptr()), p.max_pages,
                                  static_cast<const int32_t*>(p.lengths.data_ptr()), p.batch, tail,
                                  static_cast<int8_t*>(p.keys.data_ptr()),
                                  static_cast<float*>(p.scales.data_ptr()), stream);
    });
    Py_RETURN_NONE;
  });
}

// (q, kcache, page_keys, page_scales, block_table, cache_seqlens, topk_pages, causal,
//  softmax_scale, d_v, num_sm_parts, pages, out, lse, workspace) -> (out, lse, pages)
PyObject* page_sparse_decode(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 15, [&]() -> PyObject* {
    at::Tensor q = tensor(a[0], "q");
    const int index = query(q);
    const PageArgs p = page_args(a[1], a[2], a[3], a[4], a[5], index);
    require(p.table.size(0) == q.size(0), "block_table must be [b, max_pages]");
    q = q.contiguous();
    const int b = p.batch, s_q = static_cast<int>(q.size(1)), h_q = static_cast<int>(q.size(2));
    const int topk = whole32(a[6]), d_v = whole32(a[9]);
    int parts = 0;
    if (a[10] == Py_None)
      check(mla_num_sm_parts(index, h_q, 1, &parts));
    else
      parts = whole32(a[10]);
    size_t bytes = 0;
    check(mla_page_sparse_workspace_size(b, s_q, h_q, d_v, p.max_pages, topk, parts, &bytes));
    const at::Device dev = q.device();
    const at::Tensor out = output(a[12], "out", {b, s_q, h_q, d_v}, at::kBFloat16, dev);
    const at::Tensor lse = output(a[13], "lse", {b, s_q, h_q}, at::kFloat, dev);
    const at::Tensor pages = output(a[11], "pages", {b, s_q, topk}, at::kInt, dev);
    const at::Tensor ws = workspace(a[14], bytes, dev);
    if (b == 0) return pack({out, lse, pages});
    const float scale = softmax_scale(a[8]);
    const bool causal = truth(a[7]);
    launch(index, [&](cudaStream_t stream) {
      return mla_page_sparse_decode(
          q.data_ptr(), p.cache.data_ptr(), p.blocks, static_cast<const int8_t*>(p.keys.data_ptr()),
          static_cast<const float*>(p.scales.data_ptr()),
          static_cast<const int32_t*>(p.table.data_ptr()), p.max_pages,
          static_cast<const int32_t*>(p.lengths.data_ptr()), b, s_q, h_q,
          static_cast<int>(p.cache.size(2)), d_v, topk, scale, causal, parts, ws.data_ptr(),
          ws.nbytes(), static_cast<int32_t*>(pages.data_ptr()), out.data_ptr(),
          static_cast<float*>(lse.data_ptr()), stream);
    });
    return pack({out, lse, pages});
  });
}

// (q, kcache, prefix_table, prefix_len, block_table, cache_seqlens, metadata, num_splits,
//  num_sm_parts, causal, softmax_scale, out, lse, workspace) -> (out, lse)
PyObject* shared_prefix_decode(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 14, [&]() -> PyObject* {
    at::Tensor q = tensor(a[0], "q");
    const int index = query(q);
    const at::Tensor& cache = tensor(a[1], "kcache");
    bf16_cache(cache, index);
    const int prefix_len = whole32(a[3]);
    at::Tensor prefix;
    if (prefix_len > 0) {
      require(a[2] != Py_None, "prefix_table must be [>= ceil(prefix_len / 64)]");
      prefix = int32_on(tensor(a[2], "prefix_table"), "prefix_table", index);
      require(prefix.dim() == 1 && prefix.size(0) >= (int64_t{prefix_len} + kPage - 1) / kPage,
              "prefix_table must be [>= ceil(prefix_len / 64)]");
    }
    const at::Tensor& table_in = tensor(a[4], "block_table");
    require(table_in.dim() == 2 && table_in.size(0) == q.size(0) &&
                table_in.numel() <= std::numeric_limits<int>::max(),
            "block_table must be [b, max_pages]");
    const at::Tensor table = int32_on(table_in, "block_table", index);
    const at::Tensor lengths = int32_on(tensor(a[5], "cache_seqlens"), "cache_seqlens", index);
    require(lengths.dim() == 1 && lengths.size(0) == q.size(0), "cache_seqlens must be [b]");
    q = q.contiguous();
    const int b = static_cast<int>(q.size(0)), s_q = static_cast<int>(q.size(1)),
              h_q = static_cast<int>(q.size(2));
    const int parts = whole32(a[8]);
    at::Tensor metadata = tensor(a[6], "metadata");
    const at::Tensor& splits = tensor(a[7], "num_splits");
    require(metadata.is_cuda() && splits.is_cuda() && metadata.get_device() == index &&
                splits.get_device() == index && metadata.scalar_type() == at::kInt &&
                splits.scalar_type() == at::kInt && metadata.is_contiguous() &&
                splits.is_contiguous(),
            "metadata and num_splits", "the plan,", index);
    const int rows = static_cast<int>(
        std::min<int64_t>(int64_t{s_q} * h_q, std::numeric_limits<int>::max()));
    // (a plan of another call is recognised on the device by its metadata)
    size_t bytes = 0, metadata_bytes = 0, splits_bytes = 0;
    check(mla_shared_prefix_metadata_size(b, rows, prefix_len, parts, &metadata_bytes,
                                          &splits_bytes));
    require(metadata.nbytes() >= metadata_bytes, "metadata is too small for num_sm_parts");
    // num_splits too short for this call is another plan's, whatever the metadata says:
    // with metadata that names no plan the device refuses it without reading it
    if (splits.nbytes() < splits_bytes) metadata = at::zeros_like(metadata);
    check(mla_shared_prefix_workspace_size(b, rows, prefix_len, parts, &bytes));
    const at::Device dev = q.device();
    const at::Tensor out = output(a[11], "out", {b, s_q, h_q, kNope}, at::kBFloat16, dev);
    const at::Tensor lse = output(a[12], "lse", {b, s_q, h_q}, at::kFloat, dev);
    const at::Tensor ws = workspace(a[13], bytes, dev);
    if (b == 0) return pack({out, lse});
    const float scale = softmax_scale(a[10]);
    const bool causal = truth(a[9]);
    launch(index, [&](cudaStream_t stream) {
      return mla_shared_prefix_decode_fwd(
          q.data_ptr(), cache.data_ptr(), static_cast<int>(cache.size(0)),
          prefix.defined() ? static_cast<const int32_t*>(prefix.data_ptr()) : nullptr, prefix_len,
          static_cast<const int32_t*>(table.data_ptr()), static_cast<int>(table.size(1)),
          static_cast<const int32_t*>(lengths.data_ptr()), b, s_q, h_q,
          static_cast<int>(cache.size(2)), static_cast<int>(kNope), scale, causal,
          static_cast<const int32_t*>(metadata.data_ptr()),
          static_cast<const int32_t*>(splits.data_ptr()), parts, ws.data_ptr(), ws.nbytes(),
          out.data_ptr(), static_cast<float*>(lse.data_ptr()), stream);
    });
    return pack({out, lse});
  });
}

PyMethodDef kMethods[] = {
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_append)),
     METH_FASTCALL, nullptr},
    {"page_keys_update", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_keys_update)),
     METH_FASTCALL, nullptr},
    {"page_sparse_decode",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_sparse_decode)), METH_FASTCALL,
     nullptr},
    {"shared_prefix_decode",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(shared_prefix_decode)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods,
                       nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "BUILT_WITH", MLA_BUILT_WITH) < 0) Py_CLEAR(m);
  return m;
}
