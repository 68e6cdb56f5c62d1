// binding.cpp -- the Python side of the paged-cache calls: checks torch tensors
// and packs them into the argument structs of include/sskip_attn.h.
//
// The calls of a decode step are a few microseconds long on the GPU; checking
// and packing fourteen tensors from Python takes longer than that (an append of
// 64 tokens 11.0 us a call, from here 4.7, of which the launch is 3.3).  Nothing is computed or
// kept here.  The C functions come as addresses, so that the release and the
// debug library share this file.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>

#include "../../include/sskip_attn.h"

namespace {

struct Raised {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised{};
}

using Tensor = at::Tensor;

// An argument that may be None.
const Tensor* optional(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
  return &THPVariable_Unpack(o);
}

const Tensor& required(PyObject* o, const char* name) {
  const Tensor* t = optional(o, name);
  if (!t) raise(PyExc_ValueError, "%s is missing", name);
  return *t;
}

void of_type(const Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, at::toString(type),
          at::toString(t.scalar_type()));
}

void contiguous(const Tensor& t, const char* name) {
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
}

void* address(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

int number(long long n, const char* name) {
  if (n < -0x7FFFFFFF || n > 0x7FFFFFFF) raise(PyExc_ValueError, "%s is out of range", name);
  return (int)n;
}

// Every tensor of a call is on the device that its stream belongs to.
void on_device(std::initializer_list<const Tensor*> tensors, int device) {
  if (device < 0) raise(PyExc_ValueError, "expected CUDA tensors");
  for (const Tensor* t : tensors)
    if (t && !(t->is_cuda() && t->get_device() == device))
      raise(PyExc_ValueError, "all tensors of a call must be on one CUDA device (%d)", device);
}

// A paged cache: bf16 [num_pages, Hkv, page_size, d] or uint8 [num_pages, Hkv,
// page_size / 16, 10 d] pages and an int32 [B, max_pages] block table.
sskip_paged_cache paged(const Tensor* k, const Tensor* v, const Tensor* table, long long d,
                        int* Hkv) {
  if (!k || !v || !table)
    raise(PyExc_ValueError, "a cache needs k_pages, v_pages and block_table");
  if (k->dim() != 4 || v->sizes() != k->sizes() || v->scalar_type() != k->scalar_type())
    raise(PyExc_ValueError, "k_pages and v_pages must be 4-D and of one shape and dtype");
  contiguous(*k, "k_pages");
  contiguous(*v, "v_pages");
  contiguous(*table, "block_table");
  of_type(*table, at::kInt, "block_table");
  if (table->dim() != 2) raise(PyExc_ValueError, "block_table must be 2-D");
  sskip_paged_cache c{};
  long long rows = k->size(2);
  const long long width = k->size(3);
  if (k->scalar_type() == at::kByte) {
    if (width != 10 * d)
      raise(PyExc_ValueError, "4-bit records of d = %lld hold %lld bytes, got %lld", d, 10 * d, width);
    c.kv_format = SSKIP_KV_INT4;
    rows *= 16;
  } else if (k->scalar_type() == at::kBFloat16) {
    if (width != d) raise(PyExc_ValueError, "pages hold rows of %lld, expected d = %lld", width, d);
    c.kv_format = SSKIP_KV_BF16;
  } else {
    raise(PyExc_TypeError, "pages must be bf16, or uint8 records, got %s",
          at::toString(k->scalar_type()));
  }
  c.k_pages = k->data_ptr();
  c.v_pages = v->data_ptr();
  c.block_table = static_cast<const int*>(table->data_ptr());
  c.num_pages = number(k->size(0), "num_pages");
  c.page_size = number(rows, "page_size");
  c.max_pages = number(table->size(1), "max_pages");
  c.B = number(table->size(0), "B");
  *Hkv = number(k->size(1), "Hkv");
  return c;
}

// [T, H, d] bf16, heads packed, any stride between tokens: that stride (a
// single token's means nothing).
long long token_stride(const Tensor& t, const char* name) {
  of_type(t, at::kBFloat16, name);
  if (t.dim() != 3) raise(PyExc_ValueError, "%s must be [T, H, d]", name);
  if (t.stride(2) != 1 || (t.stride(1) != t.size(2) && t.size(1) > 1))
    raise(PyExc_ValueError, "%s: the heads of a token must be packed", name);
  return t.size(0) <= 1 ? t.size(1) * t.size(2) : t.stride(0);
}

const int* tokens(const Tensor* t, long long T, const char* name) {
  if (!t) return nullptr;
  of_type(*t, at::kInt, name);
  contiguous(*t, name);
  if (t->numel() != T) raise(PyExc_ValueError, "%s needs %lld entries", name, T);
  return static_cast<const int*>(t->data_ptr());
}

// out_len of a [T / out_len, H, out_len, d] (or [T, H, d]) output.
long long rows_out(const Tensor& t, long long T, long long H, long long d, const char* name) {
  of_type(t, at::kBFloat16, name);
  contiguous(t, name);
  const long long out_len = t.dim() == 4 ? t.size(2) : 1;
  if ((t.dim() != 3 && t.dim() != 4) || t.size(0) * out_len != T || t.size(1) != H ||
      t.size(t.dim() - 1) != d)
    raise(PyExc_ValueError, "%s must be [T / out_len, %lld, out_len, %lld] with T = %lld", name, H, d, T);
  return out_len;
}

void* weight(const Tensor* t, long long d, const char* name) {
  if (!t) return nullptr;
  of_type(*t, at::kBFloat16, name);
  contiguous(*t, name);
  if (t->numel() != d) raise(PyExc_ValueError, "%s must hold %lld values", name, d);
  return t->data_ptr();
}

float real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)x;
}

long long integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x;
}

// Calls the library's function at an address; its status as a Python number.
template <typename Args>
PyObject* launch(PyObject* function, const Args& args, PyObject* stream) {
  auto fn = reinterpret_cast<int (*)(const Args*, void*)>(PyLong_AsVoidPtr(function));
  void* st = PyLong_AsVoidPtr(stream);
  if (PyErr_Occurred()) throw Raised{};
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = fn(&args, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

template <typename Body>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, Body body) {
  try {
    if (got != want) raise(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return body();
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// append(function, stream, device, q, k, v, seq_ids, positions, q_out, k_out,
//        v_out, k_pages, v_pages, block_table, turns, interleaved, attn_factor,
//        q_weight, k_weight, eps)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 20, [&] {
    const Tensor *q = optional(a[3], "q"), *k = optional(a[4], "k"), *v = optional(a[5], "v");
    const Tensor *seq = optional(a[6], "seq_ids"), *pos = optional(a[7], "positions");
    const Tensor *qo = optional(a[8], "q_out"), *ko = optional(a[9], "k_out");
    const Tensor *vo = optional(a[10], "v_out"), *kp = optional(a[11], "k_pages");
    const Tensor *vp = optional(a[12], "v_pages"), *table = optional(a[13], "block_table");
    const Tensor *turns = optional(a[14], "turns"), *qw = optional(a[17], "q_weight");
    const Tensor* kw = optional(a[18], "k_weight");
    if (!q && !k) raise(PyExc_ValueError, "q, or k and v, must be given");
    sskip_kv_append_args s{};
    if (q) s.q_stride = token_stride(*q, "q");
    if (k || v) {
      if (!k || !v) raise(PyExc_ValueError, "k and v come together");
      s.k_stride = token_stride(*k, "k");
      s.v_stride = token_stride(*v, "v");
      if (v->sizes() != k->sizes() || (q && (q->size(0) != k->size(0) || q->size(2) != k->size(2))))
        raise(PyExc_ValueError, "q, k and v must have one T and d, k and v one shape");
    }
    const Tensor& first = q ? *q : *k;
    const long long T = first.size(0), d = first.size(2);
    const long long Hq = q ? q->size(1) : 0, Hkv = k ? k->size(1) : 0;
    long long out_len = 0;
    auto output = [&](const Tensor* t, long long H, const char* name) {
      if (!t) return;
      const long long L = rows_out(*t, T, H, d, name);
      if (out_len && L != out_len)
        raise(PyExc_ValueError, "q_out, k_out and v_out must share one layout");
      out_len = L;
    };
    output(qo, Hq, "q_out");
    output(ko, Hkv, "k_out");
    output(vo, Hkv, "v_out");
    if (turns) {
      of_type(*turns, at::kLong, "turns");
      contiguous(*turns, "turns");
    }
    if (kp || vp) {
      int heads;
      s.cache = paged(kp, vp, table, d, &heads);
      if (heads != Hkv)
        raise(PyExc_ValueError, "the pages hold %d heads, k and v %lld", heads, Hkv);
    }
    s.q = address(q);
    s.k = address(k);
    s.v = address(v);
    s.seq_ids = tokens(seq, T, "seq_ids");
    s.positions = tokens(pos, T, "positions");
    s.q_weight = weight(qw, d, "q_weight");
    s.k_weight = weight(kw, d, "k_weight");
    s.turns = static_cast<const uint64_t*>(address(turns));
    s.q_out = address(qo);
    s.k_out = address(ko);
    s.v_out = address(vo);
    s.T = number(T, "T");
    s.Hq = number(Hq, "Hq");
    s.Hkv = number(Hkv, "Hkv");
    s.d = number(d, "d");
    s.rot_dim = turns ? number(2 * turns->numel(), "rot_dim") : 0;
    s.interleaved = PyObject_IsTrue(a[15]);
    if (s.interleaved < 0) throw Raised{};
    s.out_len = out_len ? number(out_len, "out_len") : 1;
    s.attn_factor = real(a[16]);
    s.eps = real(a[19]);
    on_device({q, k, v, seq, pos, qo, ko, vo, kp, vp, table, turns, qw, kw}, (int)integer(a[2]));
    return launch(a[0], s, a[1]);
  });
}

// gather(function, stream, device, k_pages, v_pages, block_table, seq_ids,
//        positions, k_out, v_out)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Tensor &kp = required(a[3], "k_pages"), &vp = required(a[4], "v_pages");
    const Tensor &table = required(a[5], "block_table"), &seq = required(a[6], "seq_ids");
    const Tensor &pos = required(a[7], "positions");
    const Tensor &ko = required(a[8], "k_out"), &vo = required(a[9], "v_out");
    if (ko.dim() < 1) raise(PyExc_ValueError, "k_out must be [T / out_len, Hkv, out_len, d]");
    const long long d = ko.size(ko.dim() - 1), T = seq.numel();
    sskip_kv_gather_args s{};
    s.cache = paged(&kp, &vp, &table, d, &s.Hkv);
    const long long out_len = rows_out(ko, T, s.Hkv, d, "k_out");
    if (rows_out(vo, T, s.Hkv, d, "v_out") != out_len)
      raise(PyExc_ValueError, "k_out and v_out must share one layout");
    s.seq_ids = tokens(&seq, T, "seq_ids");
    s.positions = tokens(&pos, T, "positions");
    s.k_out = address(&ko);
    s.v_out = address(&vo);
    s.T = number(T, "T");
    s.d = number(d, "d");
    s.out_len = number(out_len, "out_len");
    on_device({&kp, &vp, &table, &seq, &pos, &ko, &vo}, (int)integer(a[2]));
    return launch(a[0], s, a[1]);
  });
}

// decode(function, stream, device, q, k_pages, v_pages, block_table, seqlens, o,
//        lse, sm_scale, threshold_scale_factor, num_splits, workspace,
//        skip_count, tile_state)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    const Tensor& q = required(a[3], "q");
    const Tensor &kp = required(a[4], "k_pages"), &vp = required(a[5], "v_pages");
    const Tensor &table = required(a[6], "block_table"), &lens = required(a[7], "seqlens");
    const Tensor &o = required(a[8], "o"), &lse = required(a[9], "lse");
    const Tensor *ws = optional(a[13], "workspace"), *count = optional(a[14], "skip_count");
    const Tensor* state = optional(a[15], "tile_state");
    of_type(q, at::kBFloat16, "q");
    of_type(o, at::kBFloat16, "o");
    of_type(lse, at::kFloat, "lse");
    contiguous(q, "q");
    contiguous(o, "o");
    contiguous(lse, "lse");
    if (q.dim() != 3) raise(PyExc_ValueError, "q must be [B, Hq, d]");
    const long long B = q.size(0), Hq = q.size(1), d = q.size(2);
    sskip_decode_paged_args s{};
    s.cache = paged(&kp, &vp, &table, d, &s.Hkv);
    if (o.sizes() != q.sizes() || lse.numel() != B * Hq || s.cache.B != B)
      raise(PyExc_ValueError, "q, o, lse and block_table must belong to one batch");
    s.q = address(&q);
    s.seqlens = tokens(&lens, B, "seqlens");
    s.o = address(&o);
    s.lse = static_cast<float*>(address(&lse));
    if (ws) {
      contiguous(*ws, "workspace");
      s.workspace = address(ws);
      s.workspace_bytes = ws->nbytes();
    }
    if (count) {
      of_type(*count, at::kLong, "skip_count");
      contiguous(*count, "skip_count");
      if (count->numel() < 2) raise(PyExc_ValueError, "skip_count needs 2 entries");
      s.skip_count = static_cast<unsigned long long*>(address(count));
    }
    if (state) {
      of_type(*state, at::kByte, "tile_state");
      contiguous(*state, "tile_state");
      const long long tiles = ((long long)s.cache.max_pages * s.cache.page_size + 63) / 64;
      if (state->numel() != B * s.Hkv * tiles)
        raise(PyExc_ValueError, "tile_state must be [B, Hkv, ceil(max_pages * page_size / 64)]");
      s.tile_state = static_cast<uint8_t*>(address(state));
    }
    s.Hq = number(Hq, "Hq");
    s.d = number(d, "d");
    s.sm_scale = real(a[10]);
    s.threshold_scale_factor = real(a[11]);
    s.num_splits = number(integer(a[12]), "num_splits");
    on_device({&q, &kp, &vp, &table, &lens, &o, &lse, ws, count, state}, (int)integer(a[2]));
    return launch(a[0], s, a[1]);
  });
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, nullptr},
    {"gather", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(gather)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
