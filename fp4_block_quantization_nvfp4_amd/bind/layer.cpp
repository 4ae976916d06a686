// Torch binding of the layer operators (layer.py, attention.py): checks the arguments,
// allocates the outputs and calls the C ABI.  Native, since single-token calls
// are bound by the host: the same steps in Python with ctypes take 12 to 16 us
// a call, more than their kernels.
//
// Refusals are ValueErrors; a status of the C ABI goes to _lib.check, which
// raises NVFP4Error.  Every function takes positional arguments only.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "nvfp4.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject *g_check, *g_stream, *g_device;  // _lib.check; torch's raw stream of a device; its current device

constexpr ScalarType F8 = ScalarType::Float8_e4m3fn, E8 = ScalarType::Float8_e8m0fnu;

#define REFUSE_IF(cond, ...) TORCH_CHECK_VALUE(!(cond), __VA_ARGS__)

// The current stream.  The kernels run on the current device, where another
// device's memory may not be mapped: `on`, whose device all tensors share, has
// to be there.
void* stream(const Tensor& on) {
  PyObject* dev = PyObject_CallNoArgs(g_device);
  if (!dev) throw python_error();
  const long current = PyLong_AsLong(dev);
  PyObject* s = current == on.get_device() ? PyObject_CallOneArg(g_stream, dev) : nullptr;
  Py_DECREF(dev);
  if (PyErr_Occurred()) throw python_error();
  REFUSE_IF(!s, "tensors on the current device, cuda:", current, ", are required: these are on cuda:", on.get_device());
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!p && PyErr_Occurred()) throw python_error();
  return p;
}

void check(nvfp4_status st, const char* what) {
  if (st == NVFP4_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", (int)st, what);
  Py_XDECREF(r);
  throw python_error();
}

void count(Py_ssize_t n, Py_ssize_t want, const char* what) {
  TORCH_CHECK_TYPE(n == want, what, ": ", want, " arguments expected");
}

const Tensor& tensor(PyObject* o, const char* what, bool anywhere = false) {
  const bool is = THPVariable_Check(o);
  REFUSE_IF(!is || (!anywhere && !THPVariable_Unpack(o).is_cuda()), what, ": a device tensor is required (no CPU path)");
  return THPVariable_Unpack(o);
}

bool row_dtype(ScalarType t) { return t == ScalarType::Float || t == ScalarType::BFloat16; }
nvfp4_dtype code(ScalarType t) { return t == ScalarType::Float ? NVFP4_F32 : NVFP4_BF16; }
int64_t groups(int64_t K) { return (K + 31) / 32; }
template <typename T>
T* ptr(const Tensor& t) { return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr; }
const uint8_t* bytes(const Tensor& t) { return ptr<uint8_t>(t); }

// A 2-D contiguous float32 or bfloat16 device tensor.
const Tensor& rows(PyObject* o, const char* what) {
  const Tensor& x = tensor(o, what);
  REFUSE_IF(x.dim() != 2, what, ": a 2-D [M, K] tensor is required");
  REFUSE_IF(!row_dtype(x.scalar_type()), what, ": float32 or bfloat16 input required");
  REFUSE_IF(!x.is_contiguous(), what, ": input must be contiguous");
  return x;
}

const Tensor& same(PyObject* o, const Tensor& like, const char* what) {
  const bool ok = THPVariable_Check(o);
  const Tensor& t = ok ? THPVariable_Unpack(o) : like;
  REFUSE_IF(!ok || t.sizes() != like.sizes() || t.scalar_type() != like.scalar_type() || t.device() != like.device() ||
                !t.is_contiguous(),
            what, " must be a contiguous ", like.scalar_type(), " ", like.sizes(), " tensor on the same device");
  return t;
}

const Tensor& array(PyObject* o, ScalarType dt, int64_t n, const Tensor& like, const char* what) {
  const bool ok = THPVariable_Check(o);
  const Tensor& t = ok ? THPVariable_Unpack(o) : like;
  REFUSE_IF(!ok || t.scalar_type() != dt || t.device() != like.device() || t.numel() != n || !t.is_contiguous(), what,
            " must be a contiguous ", dt, " tensor of ", n, " elements on the same device");
  return t;
}

const Tensor& codes(PyObject* o, const char* what) {
  const Tensor& t = tensor(o, what);
  REFUSE_IF(t.dim() != 2 || (t.scalar_type() != F8 && t.scalar_type() != ScalarType::Byte) || !t.is_contiguous(), what,
            " must be a contiguous 2-D float8_e4m3fn (or uint8) tensor");
  return t;
}

const Tensor& scale_bytes(PyObject* o, int64_t T, int64_t n, const Tensor& like, const char* what) {
  const bool ok = THPVariable_Check(o);
  const Tensor& t = ok ? THPVariable_Unpack(o) : like;
  REFUSE_IF(!ok || (t.scalar_type() != E8 && t.scalar_type() != ScalarType::Byte) || t.dim() != 2 || t.size(0) != T ||
                t.size(1) != n || t.device() != like.device() || !t.is_contiguous(),
            what, " must be a contiguous float8_e8m0fnu (or uint8) [", T, ", ", n, "] tensor on the same device");
  return t;
}

// What at::empty allocates, without its dispatch (half a microsecond each).
Tensor make(const Tensor& like, at::IntArrayRef sizes, ScalarType dt) {
  return Tensor(at::detail::empty_cuda(sizes, dt, like.device(), std::nullopt));
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

ScalarType out_type(PyObject* o) {
  REFUSE_IF(!THPDtype_Check(o) || !row_dtype(reinterpret_cast<THPDtype*>(o)->scalar_type), "out_dtype must be float32 or bfloat16");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// New reference, None for an undefined tensor.
PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

template <typename... Ts>
PyObject* pack(const Ts&... ts) {
  PyObject* r = PyTuple_New(sizeof...(ts));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  bool ok = true;
  ((ok = ok && PyTuple_SetItem(r, i++, wrap(ts)) == 0 && PyTuple_GET_ITEM(r, i - 1)), ...);
  if (!ok) {
    Py_DECREF(r);
    throw python_error();
  }
  return r;
}

// (x, weight, residual or None, eps)
PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 4, "add_rms_norm");
  const Tensor& x = rows(a[0], "add_rms_norm");
  const int64_t T = x.size(0), H = x.size(1);
  const Tensor& w = array(a[1], ScalarType::Float, H, x, "weight");
  const Tensor none;
  const Tensor& res = a[2] == Py_None ? none : same(a[2], x, "residual");
  const double eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) throw python_error();
  const Tensor c = make(x, {T, H}, F8), s = make(x, {T, groups(H)}, E8), rstd = make(x, {T}, ScalarType::Float);
  const Tensor hidden = res.defined() ? make(x, {T, H}, x.scalar_type()) : Tensor();
  check(nvfp4_add_rms_norm(x.data_ptr(), ptr<void>(res), code(x.scalar_type()), ptr<float>(w), T, H, (float)eps,
                           ptr<uint8_t>(c), ptr<uint8_t>(s), ptr<void>(hidden), ptr<float>(rstd), stream(x)),
        "nvfp4_add_rms_norm");
  return pack(c, s, hidden.defined() ? hidden : x, rstd);
  END_HANDLE_TH_ERRORS
}

// (dy, hidden, weight, rstd, dhidden or None)
PyObject* add_rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 5, "add_rms_norm_backward");
  const Tensor& dy = rows(a[0], "add_rms_norm_backward");
  const int64_t T = dy.size(0), H = dy.size(1);
  const Tensor& hidden = same(a[1], dy, "hidden");
  const Tensor none;
  const Tensor& dh = a[4] == Py_None ? none : same(a[4], dy, "dhidden");
  const Tensor& w = array(a[2], ScalarType::Float, H, dy, "weight");
  const Tensor& rstd = array(a[3], ScalarType::Float, T, dy, "rstd");
  const Tensor dx = make(dy, {T, H}, dy.scalar_type()), dw = make(dy, {H}, ScalarType::Float);
  const int64_t need = (int64_t)nvfp4_add_rms_norm_backward_workspace_bytes(T, H);
  const Tensor ws = make(dy, {need < 4 ? 4 : need}, ScalarType::Byte);
  check(nvfp4_add_rms_norm_backward(dy.data_ptr(), hidden.data_ptr(), ptr<void>(dh), code(dy.scalar_type()),
                                    ptr<float>(w), ptr<float>(rstd), T, H, dx.data_ptr(), ptr<float>(dw),
                                    ws.data_ptr(), (size_t)ws.numel(), stream(dy)),
        "nvfp4_add_rms_norm_backward");
  return pack(dx, dw);
  END_HANDLE_TH_ERRORS
}

// (gate_up, keep)
PyObject* swiglu_checkpoint(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 2, "swiglu_checkpoint");
  const Tensor& x = rows(a[0], "swiglu_checkpoint");
  REFUSE_IF(x.size(1) % 32 != 0, "swiglu_checkpoint: gate_up must be [T, 2F] with F % 16 == 0");
  const bool keep = truth(a[1]);
  const int64_t T = x.size(0), F = x.size(1) / 2;
  const Tensor c = make(x, {T, F}, F8), s = make(x, {T, groups(F)}, E8);
  const Tensor kept = keep ? make(x, {T, 2 * F}, F8) : Tensor(), ks = keep ? make(x, {T, 2 * groups(F)}, E8) : Tensor();
  check(nvfp4_swiglu(x.data_ptr(), code(x.scalar_type()), T, F, ptr<uint8_t>(c), ptr<uint8_t>(s), ptr<uint8_t>(kept),
                     ptr<uint8_t>(ks), stream(x)),
        "nvfp4_swiglu");
  return pack(c, s, kept, ks);
  END_HANDLE_TH_ERRORS
}

// (dout, kept, kept_scales)
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 3, "swiglu_backward");
  const Tensor& d = rows(a[0], "swiglu_backward");
  const int64_t T = d.size(0), F = d.size(1);
  const Tensor& kept = codes(a[1], "kept");
  REFUSE_IF(kept.size(0) != T || kept.size(1) != 2 * F || kept.device() != d.device(), "kept must be [T, 2F] on dout's device");
  const Tensor& ks = scale_bytes(a[2], T, 2 * groups(F), d, "kept_scales");
  const Tensor out = make(d, {T, 2 * F}, d.scalar_type());
  check(nvfp4_swiglu_backward(d.data_ptr(), code(d.scalar_type()), T, F, bytes(kept), bytes(ks), out.data_ptr(), stream(d)),
        "nvfp4_swiglu_backward");
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// Rows that are bfloat16, or mx8 with a scale; sets xs.
const Tensor& product_rows(PyObject* xo, PyObject* so, Tensor& xs, const char* what) {
  if (so == Py_None) {
    const Tensor& x = rows(xo, what);
    REFUSE_IF(x.scalar_type() != ScalarType::BFloat16, what, ": x must be bfloat16, or float8_e4m3fn with x_scale");
    return x;
  }
  const Tensor& x = codes(xo, what);
  xs = scale_bytes(so, x.size(0), groups(x.size(1)), x, "x_scale");
  return x;
}

// 4-bit weights as matvec (E = 0) and grouped_matmul take them.
struct Weights {
  Tensor packed, scale, amax;
  nvfp4_scale_mode mode = NVFP4_SCALE_NONE;
  int64_t N;
  float bound;

  // a: global_amax, row_scaled, bound
  Weights(PyObject* po, PyObject* so, const Tensor& x, int64_t E, int64_t K, nvfp4_block blocks, PyObject* const* a) {
    for (PyObject* o : {po, so}) {
      const bool ok = THPVariable_Check(o);
      REFUSE_IF(!ok || THPVariable_Unpack(o).scalar_type() != ScalarType::Byte || THPVariable_Unpack(o).device() != x.device(),
                o == po ? "packed" : "scale", " must be a uint8 tensor on x's device");
    }
    const Tensor &p = THPVariable_Unpack(po), &s = THPVariable_Unpack(so);
    const int64_t d = E ? 1 : 0;
    REFUSE_IF(p.dim() != d + 2 || (E && p.size(0) != E) || p.size(d + 1) * 2 != K, "packed must be ", E ? "[E, N, " : "[N, ", K / 2, "]");
    N = p.size(d);
    const int64_t r = blocks == NVFP4_BLOCK_1X16 ? N : blocks == NVFP4_BLOCK_16X16 ? N / 16 : K / 16;
    const int64_t c = blocks == NVFP4_BLOCK_16X16_T ? N / 16 : K / 16;
    REFUSE_IF(s.dim() != d + 2 || (E && s.size(0) != E) || s.size(d) != r || s.size(d + 1) != c, "scale must be ",
              E ? "[E, " : "[", r, ", ", c, "]");
    packed = p.is_contiguous() ? p : p.contiguous();
    scale = s.is_contiguous() ? s : s.contiguous();
    const bool by_row = truth(a[1]);
    bound = (float)PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) throw python_error();
    if (a[0] == Py_None) {
      REFUSE_IF(by_row, "row_scaled needs a global_amax for each row");
      return;
    }
    const int64_t experts = E ? E : 1;
    mode = by_row ? NVFP4_SCALE_ROW : NVFP4_SCALE_TENSOR;
    if (THPVariable_Check(a[0])) {
      amax = array(a[0], ScalarType::Float, by_row ? experts * N : experts, x, "global_amax");
    } else {
      REFUSE_IF(by_row, "row_scaled needs a global_amax for each row");
      const double v = PyFloat_AsDouble(a[0]);
      if (PyErr_Occurred()) throw python_error();
      amax = at::full({experts}, v, x.options().dtype(ScalarType::Float));
    }
  }
};

// (x, packed, scale, x_scale or None, tile16, global_amax, row_scaled, bound, out_dtype)
PyObject* matvec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9, "matvec");
  Tensor xs;
  const Tensor& x = product_rows(a[0], a[3], xs, "matvec");
  const nvfp4_block blocks = truth(a[4]) ? NVFP4_BLOCK_16X16 : NVFP4_BLOCK_1X16;
  const Weights w(a[1], a[2], x, 0, x.size(1), blocks, a + 5);
  const ScalarType dt = out_type(a[8]);
  const Tensor out = make(x, {x.size(0), w.N}, dt);
  check(nvfp4_matvec(x.data_ptr(), bytes(xs), x.size(0), w.N, x.size(1), bytes(w.packed), bytes(w.scale), blocks,
                     ptr<float>(w.amax), w.mode, w.bound, out.data_ptr(), code(dt), stream(x)),
        "nvfp4_matvec");
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// (x, ends, packed, scale, x_scale or None, tile16, transposed_tiles, global_amax, row_scaled, bound, out_dtype)
PyObject* grouped_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 11, "grouped_matmul");
  Tensor xs;
  const Tensor& x = product_rows(a[0], a[4], xs, "grouped_matmul");
  const bool tile = truth(a[5]), transposed = truth(a[6]);
  REFUSE_IF(transposed && !tile, "transposed_tiles goes with tile16");
  const nvfp4_block blocks = transposed ? NVFP4_BLOCK_16X16_T : tile ? NVFP4_BLOCK_16X16 : NVFP4_BLOCK_1X16;
  const int64_t E = THPVariable_Check(a[2]) && THPVariable_Unpack(a[2]).dim() == 3 ? THPVariable_Unpack(a[2]).size(0) : 0;
  REFUSE_IF(E < 1, "packed must be [E, N, K / 2] with at least one expert");
  const Weights w(a[2], a[3], x, E, x.size(1), blocks, a + 7);
  const Tensor& ends = array(a[1], ScalarType::Int, E, x, "ends");
  const ScalarType dt = out_type(a[10]);
  const Tensor out = make(x, {x.size(0), w.N}, dt);
  check(nvfp4_grouped_matmul(x.data_ptr(), bytes(xs), x.size(0), E, w.N, x.size(1), ptr<int32_t>(ends), bytes(w.packed),
                             bytes(w.scale), blocks, ptr<float>(w.amax), w.mode, w.bound, out.data_ptr(), code(dt), stream(x)),
        "nvfp4_grouped_matmul");
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// (dy, x, ends, x_scale or None, out_dtype)
PyObject* grouped_wgrad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 5, "grouped_wgrad");
  const Tensor& dy = rows(a[0], "grouped_wgrad");
  REFUSE_IF(dy.scalar_type() != ScalarType::BFloat16, "grouped_wgrad: dy must be bfloat16");
  Tensor xs;
  const Tensor& x = product_rows(a[1], a[3], xs, "grouped_wgrad");
  REFUSE_IF(x.size(0) != dy.size(0) || x.device() != dy.device(), "dy and x must have the same rows, on one device");
  const ScalarType dt = out_type(a[4]);
  const int64_t E = THPVariable_Check(a[2]) ? THPVariable_Unpack(a[2]).numel() : 0;
  REFUSE_IF(E < 1, "ends must hold at least one expert");
  const Tensor& ends = array(a[2], ScalarType::Int, E, dy, "ends");
  const int64_t N = dy.size(1), K = x.size(1);
  const Tensor dw = make(dy, {E, N, K}, dt);
  const int64_t need = (int64_t)nvfp4_grouped_wgrad_workspace_bytes(dy.size(0), E, N, K);
  const Tensor ws = need ? make(dy, {need}, ScalarType::Byte) : Tensor();
  check(nvfp4_grouped_wgrad_split(dy.data_ptr(), x.data_ptr(), bytes(xs), dy.size(0), E, N, K, ptr<int32_t>(ends),
                                  dw.data_ptr(), code(dt), ptr<void>(ws), (size_t)need, stream(dy)),
        "nvfp4_grouped_wgrad_split");
  return wrap(dw);
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------- attention on an NVFP4 cache

// Rows of heads [T, H, D]: the elements of a row lie side by side, tokens and heads as they like.
const Tensor& head_rows(PyObject* o, const char* what, nvfp4_heads& h) {
  const Tensor& x = tensor(o, what);
  REFUSE_IF(x.dim() != 3, what, ": a 3-D [T, heads, D] tensor is required");
  REFUSE_IF(!row_dtype(x.scalar_type()), what, ": float32 or bfloat16 input required");
  REFUSE_IF(x.numel() != 0 && x.stride(2) != 1 && x.size(2) != 1, what, ": the elements of a head must be contiguous");
  // a stride that is not walked along may be anything
  h = {x.data_ptr(), x.size(1), x.size(0) > 1 ? x.stride(0) : 0, x.size(1) > 1 ? x.stride(1) : 0};
  const int64_t unit = x.scalar_type() == ScalarType::Float ? 4 : 8;
  REFUSE_IF(x.numel() != 0 && (reinterpret_cast<uintptr_t>(h.at) % 16 != 0 || h.token % unit != 0 || h.head % unit != 0), what,
            ": rows must start at multiples of 16 bytes");
  return x;
}

const Tensor& like_rows(PyObject* o, const Tensor& like, int64_t H, const char* what, nvfp4_heads& h) {
  const Tensor& x = head_rows(o, what, h);
  REFUSE_IF(x.size(0) != like.size(0) || x.size(2) != like.size(2) || x.scalar_type() != like.scalar_type() || x.device() != like.device() ||
                (H >= 0 && x.size(1) != H),
            what, " must be a ", like.scalar_type(), " [", like.size(0), ", ", H >= 0 ? std::to_string(H) : std::string("heads"), ", ", like.size(2),
            "] tensor on the same device");
  return x;
}

// positions, freqs, q_weight, k_weight, interleaved, multiplier, eps
struct Rope {
  Tensor positions, freqs, qw, kw;
  nvfp4_rope r;
  Rope(PyObject* const* a, const Tensor& q) {
    const int64_t D = q.size(2);
    const bool ok = THPVariable_Check(a[1]) && THPVariable_Unpack(a[1]).dim() == 1;
    REFUSE_IF(!ok, "freqs must be a 1-D float64 tensor");
    const int64_t half = THPVariable_Unpack(a[1]).size(0);
    freqs = array(a[1], ScalarType::Double, half, q, "freqs");
    positions = array(a[0], ScalarType::Int, q.size(0), q, "positions");
    if (a[2] != Py_None) qw = array(a[2], ScalarType::Float, D, q, "q_weight");
    if (a[3] != Py_None) kw = array(a[3], ScalarType::Float, D, q, "k_weight");
    const int inter = truth(a[4]);
    const double mult = PyFloat_AsDouble(a[5]), eps = PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) throw python_error();
    r = {ptr<int32_t>(positions), ptr<double>(freqs), 2 * half, inter, mult, eps, ptr<float>(qw), ptr<float>(kw)};
  }
};

// k, k_scale, v, v_scale, k_amax, v_amax of a cache
struct Pages {
  Tensor t[4], ka, va;
  nvfp4_cache c;
  explicit Pages(PyObject* const* a) {
    static const char* const kNames[] = {"cache.k", "cache.k_scale", "cache.v", "cache.v_scale"};
    for (int i = 0; i < 4; ++i) {
      const Tensor& x = tensor(a[i], kNames[i]);
      REFUSE_IF(x.dim() != 4 || x.scalar_type() != ScalarType::Byte || !x.is_contiguous(), kNames[i], " must be a contiguous 4-D uint8 tensor");
      t[i] = x;
    }
    const int64_t P = t[0].size(0), H = t[0].size(1), S = t[0].size(2), half = t[0].size(3);
    REFUSE_IF(half % 8 != 0 || half == 0 || H == 0, "cache.k must be [pages, heads, page_size, dim / 2] with heads >= 1 and dim % 16 == 0");
    for (int i = 1; i < 4; ++i)
      REFUSE_IF(t[i].device() != t[0].device() || t[i].sizes() != at::IntArrayRef({P, H, S, i == 2 ? half : half / 8}), kNames[i],
                " must be ", at::IntArrayRef({P, H, S, i == 2 ? half : half / 8}), " on the same device");
    if (a[4] != Py_None) ka = array(a[4], ScalarType::Float, H, t[0], "k_amax");
    if (a[5] != Py_None) va = array(a[5], ScalarType::Float, H, t[0], "v_amax");
    c = {ptr<uint8_t>(t[0]), ptr<uint8_t>(t[1]), ptr<uint8_t>(t[2]), ptr<uint8_t>(t[3]), ptr<float>(ka), ptr<float>(va), P, S, H, 2 * half};
  }
};

// (q, k, positions, freqs, q_weight, k_weight, interleaved, multiplier, eps)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9, "norm_rope");
  nvfp4_heads hq, hk;
  const Tensor& q = head_rows(a[0], "q", hq);
  const Tensor& k = like_rows(a[1], q, -1, "k", hk);
  const Rope r(a + 2, q);
  const Tensor qo = make(q, q.sizes(), q.scalar_type()), ko = make(q, k.sizes(), q.scalar_type());
  check(nvfp4_norm_rope(&hq, &hk, code(q.scalar_type()), q.size(0), q.size(2), &r.r, qo.data_ptr(), ko.data_ptr(), stream(q)),
        "nvfp4_norm_rope");
  return pack(qo, ko);
  END_HANDLE_TH_ERRORS
}

// (dq, dk, q, k, positions, freqs, q_weight, k_weight, interleaved, multiplier, eps)
PyObject* norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 11, "norm_rope_backward");
  nvfp4_heads hdq, hdk, hq, hk;
  const Tensor& q = head_rows(a[2], "q", hq);
  const Tensor& k = like_rows(a[3], q, -1, "k", hk);
  const Tensor& dq = like_rows(a[0], q, q.size(1), "dq", hdq);
  const Tensor& dk = like_rows(a[1], q, k.size(1), "dk", hdk);
  const Rope r(a + 4, q);
  const int64_t T = q.size(0), D = q.size(2);
  const Tensor qo = make(q, dq.sizes(), q.scalar_type()), ko = make(q, dk.sizes(), q.scalar_type());
  const bool weights = r.qw.defined() || r.kw.defined();
  const int64_t need = weights ? (int64_t)nvfp4_norm_rope_backward_workspace_bytes(T, D) : 0;
  const Tensor dw = weights ? make(q, {2, D}, ScalarType::Float) : Tensor(), ws = need ? make(q, {need}, ScalarType::Byte) : Tensor();
  check(nvfp4_norm_rope_backward(&hdq, &hdk, &hq, &hk, code(q.scalar_type()), T, D, &r.r, qo.data_ptr(), ko.data_ptr(),
                                 ptr<float>(dw), ptr<void>(ws), (size_t)need, stream(q)),
        "nvfp4_norm_rope_backward");
  return pack(qo, ko, r.qw.defined() ? dw.select(0, 0) : Tensor(), r.kw.defined() ? dw.select(0, 1) : Tensor());
  END_HANDLE_TH_ERRORS
}

// (q, k, v, slots, k, k_scale, v, v_scale, k_amax, v_amax of the cache, positions, freqs, q_weight, k_weight,
// interleaved, multiplier, eps)
PyObject* norm_rope_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 17, "norm_rope_write");
  nvfp4_heads hq, hk, hv;
  const Tensor& q = head_rows(a[0], "q", hq);
  const Pages c(a + 4);
  const Tensor& k = like_rows(a[1], q, c.c.heads, "k", hk);
  like_rows(a[2], k, c.c.heads, "v", hv);
  REFUSE_IF(q.size(2) != c.c.dim || q.device() != c.t[0].device(), "q, k and v must have the cache's head size, on its device");
  const Tensor& slots = array(a[3], ScalarType::Int, q.size(0), q, "slots");
  const Rope r(a + 10, q);
  const Tensor qo = make(q, q.sizes(), q.scalar_type());
  check(nvfp4_norm_rope_write(&hq, &hk, &hv, code(q.scalar_type()), q.size(0), &r.r, &c.c, ptr<int32_t>(slots), qo.data_ptr(),
                              stream(q)),
        "nvfp4_norm_rope_write");
  return wrap(qo);
  END_HANDLE_TH_ERRORS
}

// (k, v, slots, k, k_scale, v, v_scale, k_amax, v_amax of the cache)
PyObject* write_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9, "write_cache");
  nvfp4_heads hk, hv;
  const Tensor& k = head_rows(a[0], "k", hk);
  const Pages c(a + 3);
  like_rows(a[1], k, c.c.heads, "v", hv);
  REFUSE_IF(k.size(1) != c.c.heads || k.size(2) != c.c.dim || k.device() != c.t[0].device(),
            "k and v must have the cache's heads and head size, on its device");
  const Tensor& slots = array(a[2], ScalarType::Int, k.size(0), k, "slots");
  check(nvfp4_write_cache(&hk, &hv, code(k.scalar_type()), k.size(0), &c.c, ptr<int32_t>(slots), stream(k)), "nvfp4_write_cache");
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (slots, k, k_scale, v, v_scale, k_amax, v_amax of the cache, out_dtype)
PyObject* read_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8, "read_cache");
  const Pages c(a + 1);
  const Tensor& s = tensor(a[0], "slots");
  const Tensor& slots = array(a[0], ScalarType::Int, s.numel(), c.t[0], "slots");
  const ScalarType dt = out_type(a[7]);
  const int64_t T = slots.numel();
  const Tensor k = make(slots, {T, c.c.heads, c.c.dim}, dt), v = make(slots, {T, c.c.heads, c.c.dim}, dt);
  check(nvfp4_read_cache(&c.c, ptr<int32_t>(slots), T, k.data_ptr(), v.data_ptr(), code(dt), stream(slots)), "nvfp4_read_cache");
  return pack(k, v);
  END_HANDLE_TH_ERRORS
}

// (q, k, k_scale, v, v_scale, k_amax, v_amax of the cache, table, lens, ends or None, scale or None, causal)
PyObject* cache_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12, "cache_attention");
  nvfp4_heads hq;
  const Tensor& q = head_rows(a[0], "q", hq);
  REFUSE_IF(q.scalar_type() != ScalarType::BFloat16, "q: bfloat16 is required");
  const Pages c(a + 1);
  REFUSE_IF(q.size(2) != c.c.dim || q.device() != c.t[0].device(), "q must have the cache's head size, on its device");
  REFUSE_IF(q.size(1) % c.c.heads != 0, "q must have a multiple of the cache's heads");
  const bool ok = THPVariable_Check(a[7]) && THPVariable_Unpack(a[7]).dim() == 2;
  REFUSE_IF(!ok, "table must be a 2-D int32 tensor");
  const int64_t B = THPVariable_Unpack(a[7]).size(0), width = THPVariable_Unpack(a[7]).size(1), T = q.size(0);
  const Tensor& table = array(a[7], ScalarType::Int, B * width, q, "table");
  const Tensor& lens = array(a[8], ScalarType::Int, B, q, "lens");
  const Tensor none;
  const Tensor& ends = a[9] == Py_None ? none : array(a[9], ScalarType::Int, B, q, "ends");
  REFUSE_IF(!ends.defined() && T != B, "without ends q must have one query for each of the table's ", B, " sequences");
  double scale = a[10] == Py_None ? 1.0 / std::sqrt((double)c.c.dim) : PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) throw python_error();
  const bool causal = truth(a[11]);
  const Tensor out = make(q, q.sizes(), ScalarType::BFloat16), lse = make(q, {T, q.size(1)}, ScalarType::Float);
  const int64_t need = (int64_t)nvfp4_cache_attention_workspace_bytes(T, q.size(1), &c.c, B, width);
  const Tensor ws = need ? make(q, {need}, ScalarType::Byte) : Tensor();
  check(nvfp4_cache_attention(&hq, T, &c.c, ptr<int32_t>(table), B, width, ptr<int32_t>(lens), ptr<int32_t>(ends), (float)scale, causal,
                              out.data_ptr(), ptr<float>(lse), ptr<void>(ws), (size_t)need, stream(q)),
        "nvfp4_cache_attention");
  return pack(out, lse);
  END_HANDLE_TH_ERRORS
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {ENTRY(add_rms_norm), ENTRY(add_rms_norm_backward), ENTRY(swiglu_checkpoint), ENTRY(swiglu_backward),
                          ENTRY(matvec),       ENTRY(grouped_matmul),        ENTRY(grouped_wgrad),     ENTRY(norm_rope),
                          ENTRY(norm_rope_backward), ENTRY(norm_rope_write),  ENTRY(write_cache),     ENTRY(read_cache),
                          ENTRY(cache_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_layer", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

PyObject* attribute(const char* module, const char* name) {
  PyObject* m = PyImport_ImportModule(module);
  PyObject* f = m ? PyObject_GetAttrString(m, name) : nullptr;
  Py_XDECREF(m);
  return f;
}

}  // namespace

PyMODINIT_FUNC PyInit__layer() {
  g_check = attribute("fp4_block_quantization_nvfp4_amd._lib", "check");
  g_stream = attribute("torch._C", "_cuda_getCurrentRawStream");
  g_device = attribute("torch._C", "_cuda_getDevice");
  if (!g_check || !g_stream || !g_device) return nullptr;
  return PyModule_Create(&kModule);
}
