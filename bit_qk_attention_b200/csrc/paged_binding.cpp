// The Python side of the paged cache's entry points: checks of tensors, allocation of results, the call.
//
// These calls are made many times per second on small tensors, where ctypes and checks in Python took two to
// three times as long as the library and the launch: host time of attention_paged for one token, with its two
// allocations, 13.7 us and now 5.6 (4.5 of it the library and the launch); of cache_write 7.6 and 3.3, of
// cache_read 9.9 and 5.5. Each function returns the C call's status where that is not BA_OK, for the caller to
// raise, else its result. The C functions are handed over by address, so that this module and ctypes use the
// one loaded library.
#include <ATen/ATen.h>
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <stdexcept>
#include <string>

#include "binattn.h"

namespace {

decltype(&ba_kv_block_bytes) f_block_bytes = nullptr;
decltype(&ba_cache_write) f_write = nullptr;
decltype(&ba_cache_read) f_read = nullptr;
decltype(&ba_paged_workspace_bytes) f_workspace = nullptr;
decltype(&ba_attention_paged) f_attend = nullptr;

PyObject* out_of_memory = nullptr;  // torch.OutOfMemoryError

struct Refused : std::runtime_error {
  PyObject* type;
  Refused(PyObject* t, const std::string& what) : std::runtime_error(what), type(t) {}
};

void want(bool ok, const char* what) {
  if (!ok) throw Refused(PyExc_ValueError, what);
}

const at::Tensor& tensor(PyObject* x, const char* name) {
  if (!THPVariable_Check(x)) throw Refused(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(x);
}

int64_t whole(PyObject* x) {
  const int64_t v = PyLong_AsLongLong(x);
  if (v == -1 && PyErr_Occurred()) throw Refused(nullptr, "");
  return v;
}

// Larger numbers than a C int holds mean the same as the largest.
int up_to_int(PyObject* x) {
  int over = 0;
  const int64_t v = PyLong_AsLongLongAndOverflow(x, &over);
  if (v == -1 && over == 0 && PyErr_Occurred()) throw Refused(nullptr, "");
  const int64_t most = 0x7fffffff;
  if (over > 0 || v > most) return static_cast<int>(most);
  return over < 0 || v < -most ? -static_cast<int>(most) : static_cast<int>(v);
}

ba_dtype dtype_of(at::ScalarType t, bool wide, const char* name) {
  if (t == at::kBFloat16) return BA_BF16;
  if (t == at::kHalf) return BA_F16;
  if (t == at::kFloat && wide) return BA_F32;
  throw Refused(wide ? PyExc_TypeError : PyExc_ValueError,
                std::string(name) + (wide ? " must be fp16, bf16 or fp32" : " must be fp16 or bf16"));
}

at::ScalarType scalar_type(PyObject* x) {
  if (!THPDtype_Check(x)) throw Refused(PyExc_TypeError, "dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(x)->scalar_type;
}

// data, page_size, d at args[0 .. 2].
ba_kv_cache cache_of(PyObject* const* args, int64_t* dev) {
  const at::Tensor& t = tensor(args[0], "cache data");
  want(t.scalar_type() == at::kByte && t.dim() == 3 && t.is_cuda() && t.is_contiguous(),
       "cache data must be a contiguous uint8 CUDA tensor [pages, heads, block bytes]");
  ba_kv_cache c{};
  c.data = t.data_ptr();
  c.num_pages = t.size(0);
  c.page_size = up_to_int(args[1]);
  c.n_kv_heads = static_cast<int>(std::min<int64_t>(t.size(1), 0x7fffffff));
  c.d = up_to_int(args[2]);
  const size_t bytes = f_block_bytes(c.page_size, c.d);
  want(bytes != 0 && static_cast<size_t>(t.size(2)) == bytes, "cache blocks must have kv_block_bytes(page_size, d) bytes");
  *dev = t.get_device();
  return c;
}

void check_index(const at::Tensor& t, const char* name, at::ScalarType type, int64_t dev, at::IntArrayRef shape) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || t.sizes() != shape || !t.is_contiguous()) {
    std::string s;
    for (int64_t n : shape) s += (s.empty() ? "" : ", ") + std::to_string(n);
    throw Refused(PyExc_ValueError, std::string(name) + " must be a contiguous " + at::toString(type) +
                                        " tensor of shape [" + s + "] on the cache's device");
  }
}

// Rows [tokens, heads, d] of 16-bit numbers.
ba_dtype check_rows(const at::Tensor& t, const char* name, int64_t dev, int64_t heads, int64_t d) {
  if (t.dim() != 3 || t.size(2) != d || (heads >= 0 && t.size(1) != heads))
    throw Refused(PyExc_ValueError,
                  std::string(name) + " must be [tokens, heads, " + std::to_string(d) + "] with the cache's heads");
  if (t.stride(2) != 1 && d > 1 && t.numel() > 0)
    throw Refused(PyExc_ValueError, std::string(name) + " must be contiguous in its last dimension");
  if (!t.is_cuda() || t.get_device() != dev)
    throw Refused(PyExc_ValueError, std::string(name) + " must be on the cache's device");
  return dtype_of(t.scalar_type(), false, name);
}

void* stream_of(PyObject* x) { return reinterpret_cast<void*>(static_cast<intptr_t>(whole(x))); }

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t wanted, F&& f) {
  try {
    if (n != wanted) throw Refused(PyExc_TypeError, "wrong number of arguments");
    return f();
  } catch (const Refused& e) {
    if (e.type != nullptr) PyErr_SetString(e.type, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(out_of_memory, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// bind(addresses of the five C functions, torch.OutOfMemoryError)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    auto at_ = [&](int i) { return reinterpret_cast<void*>(static_cast<intptr_t>(whole(args[i]))); };
    f_block_bytes = reinterpret_cast<decltype(f_block_bytes)>(at_(0));
    f_write = reinterpret_cast<decltype(f_write)>(at_(1));
    f_read = reinterpret_cast<decltype(f_read)>(at_(2));
    f_workspace = reinterpret_cast<decltype(f_workspace)>(at_(3));
    f_attend = reinterpret_cast<decltype(f_attend)>(at_(4));
    Py_INCREF(args[5]);
    out_of_memory = args[5];
    Py_RETURN_NONE;
  });
}

// write(data, page_size, d, k, v, slots, stream) -> status
PyObject* write(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    int64_t dev;
    const ba_kv_cache c = cache_of(args, &dev);
    const at::Tensor &k = tensor(args[3], "k"), &v = tensor(args[4], "v"), &slots = tensor(args[5], "slots");
    const ba_dtype dt = check_rows(k, "k", dev, c.n_kv_heads, c.d);
    want(check_rows(v, "v", dev, c.n_kv_heads, c.d) == dt && v.size(0) == k.size(0), "k and v must share dtype and shape");
    const int64_t T = k.size(0);
    check_index(slots, "slots", at::kLong, dev, {T});
    return PyLong_FromLong(f_write(k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), dt, T,
                                   slots.data_ptr<int64_t>(), &c, stream_of(args[6])));
  });
}

// read(data, page_size, d, slots, dtype, k_out, v_out, stream) -> (k, v) or a status
PyObject* read(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    int64_t dev;
    const ba_kv_cache c = cache_of(args, &dev);
    const at::Tensor& slots = tensor(args[3], "slots");
    const int64_t T = slots.numel();
    check_index(slots, "slots", at::kLong, dev, {T});
    std::optional<at::ScalarType> type;
    if (args[4] != Py_None) type = scalar_type(args[4]);
    at::Tensor out[2];
    for (int i = 0; i < 2; ++i) {
      if (args[5 + i] == Py_None) continue;
      const char* name = i == 0 ? "k_out" : "v_out";
      out[i] = tensor(args[5 + i], name);
      if (!type) type = out[i].scalar_type();
      check_index(out[i], name, *type, dev, {T, c.n_kv_heads, c.d});
    }
    const ba_dtype dt = dtype_of(type.value_or(at::kBFloat16), true, "dtype");
    for (auto& o : out)
      if (!o.defined()) o = at::empty({T, c.n_kv_heads, c.d}, slots.options().dtype(type.value_or(at::kBFloat16)));
    const ba_status st = f_read(&c, slots.data_ptr<int64_t>(), T, out[0].data_ptr(), out[1].data_ptr(), dt, stream_of(args[7]));
    if (st != BA_OK) return PyLong_FromLong(st);
    PyObject* pair = PyTuple_New(2);
    for (int i = 0; i < 2; ++i) {
      PyObject* o = args[5 + i];
      if (o == Py_None)
        o = THPVariable_Wrap(std::move(out[i]));
      else
        Py_INCREF(o);
      PyTuple_SET_ITEM(pair, i, o);
    }
    return pair;
  });
}

// attend(data, page_size, d, q, page_table, kv_lens, cu_seqlens_q, max_q_len, max_kv_len, causal, window, sinks,
//        softmax_scale, out, out_dtype, return_lse, workspace, stream) -> o, (o, lse) or a status
PyObject* attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 18, [&]() -> PyObject* {
    int64_t dev;
    const ba_kv_cache c = cache_of(args, &dev);
    const at::Tensor &q = tensor(args[3], "q"), &table = tensor(args[4], "page_table"), &kv = tensor(args[5], "kv_lens");
    const ba_dtype dt = check_rows(q, "q", dev, -1, c.d);
    const int64_t T = q.size(0), heads = q.size(1), B = kv.numel();
    want(heads <= 0x7fffffff && B <= 0x7fffffff, "too many heads or sequences");
    check_index(kv, "kv_lens", at::kInt, dev, {B});
    ba_paged_seqs s{};
    if (args[6] != Py_None) {
      const at::Tensor& cu = tensor(args[6], "cu_seqlens_q");
      check_index(cu, "cu_seqlens_q", at::kInt, dev, {B + 1});
      s.cu_seqlens_q = cu.data_ptr<int32_t>();
    }
    want(table.scalar_type() == at::kInt && table.dim() == 2 && table.size(0) == B && table.is_cuda() &&
             table.get_device() == dev && (table.stride(1) == 1 || table.size(1) <= 1),
         "page_table must be an int32 tensor [sequences, pages] on the cache's device, contiguous in its last dimension");
    want(table.size(1) <= 0x7fffffff, "page_table has too many pages");
    s.B = static_cast<int>(B);
    s.T = T;
    s.n_heads = static_cast<int>(heads);
    s.max_q_len = args[7] != Py_None ? up_to_int(args[7])
                                     : (args[6] == Py_None ? 1 : static_cast<int>(std::min<int64_t>(T, 0x7fffffff)));
    s.kv_lens = kv.data_ptr<int32_t>();
    s.page_table = table.data_ptr<int32_t>();
    s.table_stride = table.stride(0);
    s.max_pages = static_cast<int>(table.size(1));
    s.max_kv_len = table.size(1) * c.page_size;
    if (args[8] != Py_None) s.max_kv_len = std::min<int64_t>(s.max_kv_len, up_to_int(args[8]));
    const int causal = PyObject_IsTrue(args[9]);
    if (causal < 0) throw Refused(nullptr, "");
    s.causal = causal;
    s.window = up_to_int(args[10]);
    s.sinks = up_to_int(args[11]);
    const double scale = PyFloat_AsDouble(args[12]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refused(nullptr, "");
    at::Tensor out, lse, ws;
    ba_dtype odt = dt;
    const bool typed = args[14] != Py_None;
    const at::ScalarType type = typed ? scalar_type(args[14]) : q.scalar_type();
    if (args[13] != Py_None) {
      out = tensor(args[13], "out");
      check_index(out, "out", typed ? type : out.scalar_type(), dev, {T, heads, c.d});
      odt = dtype_of(out.scalar_type(), true, "out");
    } else {
      odt = dtype_of(type, true, "out_dtype");
      out = at::empty({T, heads, c.d}, q.options().dtype(type));
    }
    const int with_lse = PyObject_IsTrue(args[15]);
    if (with_lse < 0) throw Refused(nullptr, "");
    if (with_lse) lse = at::empty({T, heads}, q.options().dtype(at::kFloat));
    if (args[16] != Py_None) {
      ws = tensor(args[16], "workspace");
      want(ws.is_cuda() && ws.get_device() == dev && ws.is_contiguous(),
           "workspace must be a contiguous tensor on the cache's device");
    } else {
      // (size_t) -1 stands for arguments that the call below refuses.
      const size_t bytes = f_workspace(&c, &s);
      if (bytes != 0 && bytes != static_cast<size_t>(-1))
        ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
    }
    const ba_status st = f_attend(q.data_ptr(), q.stride(0), q.stride(1), dt, &c, &s, static_cast<float>(scale), out.data_ptr(),
                                  odt, with_lse ? lse.data_ptr<float>() : nullptr, ws.defined() ? ws.data_ptr() : nullptr,
                                  ws.defined() ? ws.nbytes() : 0, stream_of(args[17]));
    if (st != BA_OK) return PyLong_FromLong(st);
    PyObject* o = args[13];
    if (o == Py_None)
      o = THPVariable_Wrap(std::move(out));
    else
      Py_INCREF(o);
    if (!with_lse) return o;
    PyObject* pair = PyTuple_New(2);
    PyTuple_SET_ITEM(pair, 0, o);
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(lse)));
    return pair;
  });
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(write)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch whose tensors this module can take.
PyMODINIT_FUNC PyInit__paged() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", BA_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
