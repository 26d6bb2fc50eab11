// The Python binding's quick way: the argument checks, new outputs and the call of
// the rotary and 4-bit entry points in one C++ function each.  A small call is
// bound by the host (a decode step over 3060 positions takes the GPU 8.7 us, and
// the same checks in Python 15), most of it attribute look-ups.
//
// Each function takes its Python counterpart's arguments by position and returns
//   the result     the call is enqueued,
//   an int         the library's status, not 0,
//   NotImplemented  something is not as the quick way expects it (a wrong type, shape
//                  or device, a tensor subclass, a stream given): the Python
//                  function then does the call, or finds the error's words.
// The library is reached through the addresses that bind() is given, so the module
// serves whichever build the process has loaded.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>

#include "../../include/decode_attn.h"

namespace {

struct Library {
  decltype(&decode_rope) rope;
  decltype(&decode_kv_append_rope) append_rope;
  decltype(&decode_kv_append_fp4) append_fp4;
  decltype(&decode_kv_read_fp4) read_fp4;
  decltype(&decode_attn_fp4) attn_fp4;
  decltype(&decode_attn_fp4_workspace_size) attn_fp4_size;
} lib{};
// torch's current device and raw stream, and the binding's workspace cache
PyObject *get_device = nullptr, *get_stream = nullptr, *scratch = nullptr;

// Lets other threads run Python meanwhile: the allocator and a launch may wait for
// something that one of them holds (a full stream behind a Python host function).
class NoGil {
 public:
  NoGil() : state_(PyEval_SaveThread()) {}
  ~NoGil() { PyEval_RestoreThread(state_); }
  NoGil(const NoGil&) = delete;

 private:
  PyThreadState* state_;
};
at::Tensor new_tensor(at::IntArrayRef sizes, const at::TensorOptions& options) {
  NoGil free;
  return at::empty(sizes, options);
}
template <class F, class... Args>
int call(F f, Args... args) {
  NoGil free;
  return f(args...);
}

PyObject* other_way() { return Py_NewRef(Py_NotImplemented); }

// A plain tensor on CUDA device `index`; null for all else.
const at::Tensor* on_cuda(PyObject* o, int index) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.get_device() == index ? &t : nullptr;
}
const at::Tensor* dense(PyObject* o, int index, at::ScalarType type) {
  const at::Tensor* t = on_cuda(o, index);
  return t && t->scalar_type() == type && t->is_contiguous() ? t : nullptr;
}
const at::Tensor* dense(PyObject* o, int index, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor* t = dense(o, index, type);
  return t && t->sizes() == shape ? t : nullptr;
}
bool half_type(at::ScalarType t) { return t == at::kHalf || t == at::kBFloat16; }
int dtype_code(at::ScalarType t) {
  return t == at::kBFloat16 ? DECODE_ATTN_DTYPE_BF16 : DECODE_ATTN_DTYPE_FP16;
}

// The elements between the rows of [rows, heads, dim] whose heads lie together, -1
// for another layout.
int64_t row_stride(const at::Tensor& t) {
  const int64_t rows = t.size(0), h = t.size(1), d = t.size(2);
  if (t.numel() == 0 || t.is_contiguous()) return h * d;
  const int64_t s0 = t.stride(0);
  if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && h > 1)) return -1;
  if (rows == 1) return h * d;
  return s0 >= h * d && s0 % 8 == 0 ? s0 : -1;
}
// A tensor [rows, heads, dim] of a type, with its stride.
const at::Tensor* rows_of(PyObject* o, int index, at::ScalarType type, int64_t* stride) {
  const at::Tensor* t = on_cuda(o, index);
  if (!t || t->scalar_type() != type || t->dim() != 3) return nullptr;
  *stride = row_stride(*t);
  return *stride >= 0 ? t : nullptr;
}

// The current device's index where a tensor lies on it, else -1.
int current_index(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return -1;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) return -1;
  PyObject* r = PyObject_CallNoArgs(get_device);
  if (!r) return -1;
  const long now = PyLong_AsLong(r);
  Py_DECREF(r);
  return now == t.get_device() ? (int)now : -1;
}
bool current_stream(int index, void** stream) {
  PyObject* i = PyLong_FromLong(index);
  PyObject* r = i ? PyObject_CallOneArg(get_stream, i) : nullptr;
  Py_XDECREF(i);
  if (!r) return false;
  *stream = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}
// err_flag: None or an int32 tensor.
bool error_flag(PyObject* o, int index, int32_t** flag) {
  *flag = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = dense(o, index, at::kInt);
  if (t) *flag = static_cast<int32_t*>(t->data_ptr());
  return t != nullptr;
}
bool whole(PyObject* o, int64_t least, int64_t most, int64_t* v) {
  if (!PyLong_Check(o)) return false;
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return *v >= least && *v <= most;
}
bool truth(PyObject* o, bool* v) {
  *v = o == Py_True;
  return PyBool_Check(o);
}
bool fits(int64_t v) { return v >= 0 && v <= INT32_MAX; }

template <class T>
T* data(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// The page table and what goes with it.
bool table_and_lens(PyObject* table, PyObject* lens, int index, const at::Tensor** tb,
                    const at::Tensor** ln) {
  *tb = dense(table, index, at::kInt);
  if (!*tb || (*tb)->dim() != 2) return false;
  if (!lens) return true;
  *ln = dense(lens, index, at::kInt, {(*tb)->size(0)});
  return *ln != nullptr;
}

// Six tensors of a 4-bit cache: k_pages, v_pages, k_scales, v_scales, k_blocks, v_blocks.
bool fp4_cache(PyObject* const* o, int index, decode_kv_cache* c, int64_t (&shape)[4]) {
  const at::Tensor* k = on_cuda(o[0], index);
  if (!k || (k->scalar_type() != at::kByte && k->scalar_type() != at::kFloat4_e2m1fn_x2) ||
      !k->is_contiguous() || k->dim() != 4)
    return false;
  const at::Tensor* v = dense(o[1], index, k->scalar_type(), k->sizes());
  const int64_t P = k->size(0), PS = k->size(1), H = k->size(2), half = k->size(3);
  const at::Tensor* ks = dense(o[2], index, at::kFloat, {P, H, PS});
  const at::Tensor* vs = dense(o[3], index, at::kFloat, {P, H, PS});
  const at::Tensor* kb = dense(o[4], index, at::kFloat8_e4m3fn, {P, H, PS, half / 8});
  const at::Tensor* vb = dense(o[5], index, at::kFloat8_e4m3fn, {P, H, PS, half / 8});
  if (!v || !ks || !vs || !kb || !vb) return false;
  *c = decode_kv_cache{DECODE_ATTN_KV_E2M1, k->data_ptr(), v->data_ptr(), data<float>(ks),
                       data<float>(vs), data<uint8_t>(kb), data<uint8_t>(vb)};
  shape[0] = P, shape[1] = PS, shape[2] = H, shape[3] = 2 * half;
  return true;
}

bool params_of(decode_attn_params* p, int64_t batch, int64_t heads, const int64_t (&shape)[4],
               int64_t max_pages, at::ScalarType type) {
  if (!fits(batch) || !fits(heads) || !fits(shape[0]) || !fits(shape[1]) || !fits(shape[2]) ||
      !fits(shape[3]) || !fits(max_pages))
    return false;
  *p = decode_attn_params{};
  p->batch = (int32_t)batch;
  p->num_q_heads = (int32_t)heads;
  p->num_kv_heads = (int32_t)shape[2];
  p->head_dim = (int32_t)shape[3];
  p->page_size = (int32_t)shape[1];
  p->max_pages_per_seq = (int32_t)max_pages;
  p->num_pages = (int32_t)shape[0];
  p->scale = 1.0f;
  p->num_queries = 1;
  p->dtype = dtype_code(type);
  return true;
}

PyObject* finish(int status, PyObject* result) {
  if (status == 0) return result;
  Py_DECREF(result);
  return PyLong_FromLong(status);
}

#define QUICK_BEGIN try {
// (as torch's own calls raise: no memory, an argument, anything else)
#define QUICK_END                                                      \
  }                                                                    \
  catch (const std::exception&) {                                      \
    torch::translate_exception_to_python(std::current_exception());    \
    return nullptr;                                                    \
  }

// (x, positions, table, interleaved, backward, out, err_flag, stream)
PyObject* quick_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  QUICK_BEGIN
  if (n != 8 || a[7] != Py_None) return other_way();
  const int index = current_index(a[0]);
  if (index < 0) return PyErr_Occurred() ? nullptr : other_way();
  const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
  int64_t xs, os;
  const at::Tensor* x = half_type(type) ? rows_of(a[0], index, type, &xs) : nullptr;
  // (a gradient is the Python way's)
  if (!x || (x->requires_grad() && c10::GradMode::is_enabled())) return other_way();
  const at::Tensor* pos = dense(a[1], index, at::kInt, {x->size(0)});
  const at::Tensor* table = dense(a[2], index, at::kFloat);
  bool interleaved, backward;
  int32_t* err;
  if (!pos || !table || table->dim() != 2 || table->size(1) > x->size(2) ||
      !truth(a[3], &interleaved) || !truth(a[4], &backward) || !error_flag(a[6], index, &err) ||
      !fits(x->size(0)) || !fits(x->size(1)) || !fits(x->size(2)) || !fits(table->size(0)))
    return other_way();
  at::Tensor made;
  const at::Tensor* out;
  if (a[5] == Py_None) {
    made = new_tensor(x->sizes(), x->options());
    out = &made;
    os = x->size(1) * x->size(2);
  } else {
    out = rows_of(a[5], index, type, &os);
    if (!out || out->sizes() != x->sizes()) return other_way();
  }
  void* stream;
  if (!current_stream(index, &stream)) return nullptr;
  const decode_rope_params p{(int32_t)x->size(0), (int32_t)x->size(1), (int32_t)x->size(2),
                             (int32_t)table->size(1), (int32_t)table->size(0), interleaved,
                             backward, dtype_code(type)};
  const int st = call(lib.rope, &p, x->data_ptr(), xs, data<int32_t>(pos), data<float>(table),
                          out->data_ptr(), os, err, stream);
  return finish(st, a[5] == Py_None ? THPVariable_Wrap(made) : Py_NewRef(a[5]));
  QUICK_END
}

// (k_new, v_new, row_offsets, seq_lens, k_pages, v_pages, k_scales, v_scales, k_blocks,
//  v_blocks, page_table, table, q, q_out, interleaved, err_flag, stream); table None:
// decode_kv_append_fp4
PyObject* quick_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  QUICK_BEGIN
  if (n != 17 || a[16] != Py_None) return other_way();
  const int index = current_index(a[4]);
  if (index < 0) return PyErr_Occurred() ? nullptr : other_way();
  const at::Tensor& pool = THPVariable_Unpack(a[4]);
  const bool turn = a[11] != Py_None;
  decode_kv_cache c{};
  int64_t shape[4];
  if (a[8] != Py_None) {
    if (!fp4_cache(a + 4, index, &c, shape)) return other_way();
  } else {
    const bool quant = pool.scalar_type() == at::kFloat8_e4m3fn;
    if (!turn || a[9] != Py_None || (!quant && !half_type(pool.scalar_type())) ||
        !pool.is_contiguous() || pool.dim() != 4 ||
        (!quant && (a[6] != Py_None || a[7] != Py_None)))
      return other_way();
    const at::Tensor* v = dense(a[5], index, pool.scalar_type(), pool.sizes());
    for (int i = 0; i < 4; ++i) shape[i] = pool.size(i);
    const at::Tensor *ks = nullptr, *vs = nullptr;
    if (quant) {
      ks = dense(a[6], index, at::kFloat, {shape[0], shape[2], shape[1]});
      vs = dense(a[7], index, at::kFloat, {shape[0], shape[2], shape[1]});
    }
    if (!v || (quant && (!ks || !vs))) return other_way();
    c = decode_kv_cache{quant ? DECODE_ATTN_KV_E4M3 : DECODE_ATTN_KV_16BIT, pool.data_ptr(),
                        v->data_ptr(), data<float>(ks), data<float>(vs), nullptr, nullptr};
  }
  if (!THPVariable_CheckExact(a[0])) return other_way();
  const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
  if (!half_type(type) || (c.kv_format == DECODE_ATTN_KV_16BIT && type != pool.scalar_type()))
    return other_way();
  int64_t ks, vs, qs = 0, os = 0;
  const at::Tensor *k = rows_of(a[0], index, type, &ks), *v = rows_of(a[1], index, type, &vs);
  const at::Tensor *tb, *lens;
  int32_t* err;
  bool interleaved;
  if (!k || !v || k->sizes() != v->sizes() || k->size(1) != shape[2] || k->size(2) != shape[3] ||
      !table_and_lens(a[10], a[3], index, &tb, &lens) || !error_flag(a[15], index, &err) ||
      !truth(a[14], &interleaved) || !fits(k->size(0)))
    return other_way();
  const int64_t B = tb->size(0), total = k->size(0);
  const at::Tensor* off = dense(a[2], index, at::kInt, {B + 1});
  if (!off) return other_way();
  decode_rope_rows rope{};
  at::Tensor made;
  PyObject* given = a[13];
  int64_t heads = shape[2];
  if (turn) {
    const at::Tensor* table = dense(a[11], index, at::kFloat);
    if (!table || table->dim() != 2 || table->size(1) > shape[3] || !fits(table->size(0)))
      return other_way();
    rope.table = data<float>(table);
    rope.table_rows = (int32_t)table->size(0);
    rope.rot_dim = (int32_t)table->size(1);
    rope.interleaved = interleaved;
    if (a[12] != Py_None) {
      const at::Tensor* q = rows_of(a[12], index, type, &qs);
      if (!q || q->size(0) != total || q->size(2) != shape[3]) return other_way();
      heads = q->size(1);
      if (given == Py_None) {
        made = new_tensor(q->sizes(), q->options());
        os = heads * shape[3];
        rope.q_out = made.data_ptr();
      } else {
        const at::Tensor* o = rows_of(given, index, type, &os);
        if (!o || o->sizes() != q->sizes()) return other_way();
        rope.q_out = o->data_ptr();
      }
      rope.q = q->data_ptr();
      rope.q_stride = qs;
      rope.q_out_stride = os;
    } else if (given != Py_None) {
      return other_way();
    }
  } else if (a[12] != Py_None || given != Py_None) {
    return other_way();
  }
  decode_attn_params p;
  void* stream;
  if (!params_of(&p, B, heads, shape, tb->size(1), type)) return other_way();
  if (!current_stream(index, &stream)) return nullptr;
  const int32_t *o32 = data<int32_t>(off), *l32 = data<int32_t>(lens), *t32 = data<int32_t>(tb);
  const void *kp = k->data_ptr(), *vp = v->data_ptr();
  const int st = turn ? call(lib.append_rope, &p, &c, &rope, (int32_t)total, kp, ks, vp, vs, o32,
                             l32, t32, err, stream)
                      : call(lib.append_fp4, &p, &c, (int32_t)total, kp, ks, vp, vs, o32, l32, t32,
                             err, stream);
  return finish(st, made.defined() ? THPVariable_Wrap(made) : Py_NewRef(given));
  QUICK_END
}

// (k_pages, v_pages, k_scales, v_scales, k_blocks, v_blocks, page_table, row_offsets,
//  total_rows, starts, bfloat16, k_out, v_out, err_flag, stream)
PyObject* quick_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  QUICK_BEGIN
  if (n != 15 || a[14] != Py_None) return other_way();
  const int index = current_index(a[0]);
  if (index < 0) return PyErr_Occurred() ? nullptr : other_way();
  decode_kv_cache c;
  int64_t shape[4], total;
  const at::Tensor *tb, *starts = nullptr;
  int32_t* err;
  bool bf16;
  if (!fp4_cache(a, index, &c, shape) || !table_and_lens(a[6], nullptr, index, &tb, nullptr) ||
      !whole(a[8], 0, INT32_MAX, &total) || !truth(a[10], &bf16) ||
      !error_flag(a[13], index, &err))
    return other_way();
  const int64_t B = tb->size(0);
  const at::Tensor* off = dense(a[7], index, at::kInt, {B + 1});
  if (!off) return other_way();
  if (a[9] != Py_None && !(starts = dense(a[9], index, at::kInt, {B}))) return other_way();
  const at::ScalarType type = bf16 ? at::kBFloat16 : at::kHalf;
  at::Tensor made[2];
  void* out[2];
  for (int i = 0; i < 2; ++i) {
    if (a[11 + i] == Py_None) {
      made[i] = new_tensor({total, shape[2], shape[3]}, tb->options().dtype(type));
      out[i] = made[i].data_ptr();
    } else {
      const at::Tensor* t = dense(a[11 + i], index, type, {total, shape[2], shape[3]});
      if (!t) return other_way();
      out[i] = t->data_ptr();
    }
  }
  decode_attn_params p;
  void* stream;
  if (!params_of(&p, B, shape[2], shape, tb->size(1), type)) return other_way();
  if (!current_stream(index, &stream)) return nullptr;
  const int st =
      call(lib.read_fp4, &p, &c, (int32_t)total, data<int32_t>(tb), data<int32_t>(off),
                   data<int32_t>(starts), out[0], out[1], err, stream);
  if (st) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New(2);
  for (int i = 0; r && i < 2; ++i)
    PyTuple_SET_ITEM(r, i, made[i].defined() ? THPVariable_Wrap(made[i]) : Py_NewRef(a[11 + i]));
  return r;
  QUICK_END
}

// (q, k_pages, v_pages, k_scales, v_scales, k_blocks, v_blocks, page_table, seq_lens, scale,
//  window, out, max_seq_len, workspace, err_flag, split_min, force_chunk, stream, schedule)
PyObject* quick_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  QUICK_BEGIN
  if (n != 19 || a[17] != Py_None) return other_way();
  const int index = current_index(a[0]);
  if (index < 0) return PyErr_Occurred() ? nullptr : other_way();
  const at::Tensor& q = THPVariable_Unpack(a[0]);
  const at::ScalarType type = q.scalar_type();
  if (!half_type(type) || !q.is_contiguous() || (q.dim() != 3 && q.dim() != 4))
    return other_way();
  const int64_t T = q.dim() == 4 ? q.size(1) : 1;
  const int64_t Hq = q.size(-2), D = q.size(-1), B = q.size(0);
  decode_kv_cache c;
  int64_t shape[4], window, max_len = 0, split_min, force_chunk, schedule;
  const at::Tensor *tb, *lens;
  int32_t* err;
  if (!fp4_cache(a + 1, index, &c, shape) || shape[3] != D ||
      !table_and_lens(a[7], a[8], index, &tb, &lens) || tb->size(0) != B ||
      !error_flag(a[14], index, &err) || !PyFloat_Check(a[9]) ||
      !whole(a[10], INT32_MIN, INT32_MAX, &window) ||
      (a[12] != Py_None && !whole(a[12], INT32_MIN, INT32_MAX, &max_len)) ||
      !whole(a[15], INT32_MIN, INT32_MAX, &split_min) ||
      !whole(a[16], INT32_MIN, INT32_MAX, &force_chunk) ||
      !whole(a[18], INT32_MIN, INT32_MAX, &schedule) || !fits(T))
    return other_way();
  decode_attn_params p;
  if (!params_of(&p, B, Hq, shape, tb->size(1), type)) return other_way();
  p.max_seq_len = (int32_t)max_len;
  p.scale = (float)PyFloat_AS_DOUBLE(a[9]);
  p.window = (int32_t)window;
  p.split_min = (int32_t)split_min;
  p.force_chunk = (int32_t)force_chunk;
  p.num_queries = (int32_t)T;
  p.schedule = (int32_t)schedule;
  at::Tensor made;
  void* out;
  if (a[11] == Py_None) {
    made = new_tensor(q.sizes(), q.options());
    out = made.data_ptr();
  } else {
    const at::Tensor* t = dense(a[11], index, type, q.sizes());
    if (!t) return other_way();
    out = t->data_ptr();
  }
  void *stream, *ws = nullptr;
  size_t ws_bytes = 0;
  if (!current_stream(index, &stream)) return nullptr;
  PyObject* buffer = nullptr;  // held until the call is enqueued
  if (a[13] == Py_None) {
    const size_t need = lib.attn_fp4_size(&p, index);
    if (need) {
      PyObject* args[] = {PyLong_FromLong(index), PyLong_FromSize_t(need), Py_True, Py_None};
      buffer = args[0] && args[1] ? PyObject_Vectorcall(scratch, args, 4, nullptr) : nullptr;
      Py_XDECREF(args[0]);
      Py_XDECREF(args[1]);
      if (!buffer) return nullptr;
    }
  } else {
    buffer = Py_NewRef(a[13]);
  }
  if (buffer) {
    const at::Tensor* t = on_cuda(buffer, index);
    if (!t || !t->is_contiguous()) {
      Py_DECREF(buffer);
      return other_way();
    }
    ws = t->data_ptr();
    ws_bytes = (size_t)t->nbytes();
  }
  const int st = call(lib.attn_fp4, &p, &c, q.data_ptr(), data<int32_t>(tb), data<int32_t>(lens),
                      out, ws, ws_bytes, err, stream);
  Py_XDECREF(buffer);
  return finish(st, made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[11]));
  QUICK_END
}

// (addresses of the six library functions in Library's order, get_device, get_stream, scratch)
PyObject* quick_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses and three functions");
    return nullptr;
  }
  void* f[6];
  for (int i = 0; i < 6; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  lib.rope = reinterpret_cast<decltype(lib.rope)>(f[0]);
  lib.append_rope = reinterpret_cast<decltype(lib.append_rope)>(f[1]);
  lib.append_fp4 = reinterpret_cast<decltype(lib.append_fp4)>(f[2]);
  lib.read_fp4 = reinterpret_cast<decltype(lib.read_fp4)>(f[3]);
  lib.attn_fp4 = reinterpret_cast<decltype(lib.attn_fp4)>(f[4]);
  lib.attn_fp4_size = reinterpret_cast<decltype(lib.attn_fp4_size)>(f[5]);
  Py_XSETREF(get_device, Py_NewRef(a[6]));
  Py_XSETREF(get_stream, Py_NewRef(a[7]));
  Py_XSETREF(scratch, Py_NewRef(a[8]));
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FAST(quick_bind)},     {"rope", FAST(quick_rope)},
                         {"append", FAST(quick_append)}, {"read_fp4", FAST(quick_read)},
                         {"attn_fp4", FAST(quick_attn)}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
