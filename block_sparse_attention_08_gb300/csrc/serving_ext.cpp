// serving_ext.cpp -- the Python side of the chunked-serving calls: checks of the
// tensors, outputs that the caller does not pass, and the call into libmsa.
//
// These calls take 3 to 20 us on the device; checked and marshalled in Python
// they took 20 to 24 us of the host's time each, so that a decode step waited
// for them.  Here a call costs its output allocations (about 1 us each) and its
// launches.  The functions take positional arguments only (the package's
// functions of the same names, which have the defaults and the documentation,
// pass them) and return the outputs, or a whole number: the status of a call
// that libmsa refused.
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <stdexcept>
#include <sstream>
#include <string>

#include "../../include/msa.h"

namespace {

constexpr int64_t kH = 64, kG = 4, kD = 128;

// A Python exception on its way out.
struct Raise {
  PyObject* type;
  std::string text;
};
struct Raised {};  // one that Python has set already
struct Refused : std::runtime_error {  // a call that libmsa refused
  explicit Refused(msa_status st) : std::runtime_error(std::string("libmsa: ") + msa_status_string(st)), status(st) {}
  msa_status status;
};

using Sizes = std::initializer_list<int64_t>;

template <class T>
std::string shape_text(const T& sizes) {
  std::ostringstream s;
  s << '(';
  size_t n = 0;
  for (int64_t v : sizes) s << (n++ ? ", " : "") << v;
  s << (n == 1 ? ",)" : ")");
  return s.str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Raise{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}
const at::Tensor& tensor_of(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims)
    throw Raise{PyExc_ValueError, std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " +
                                      std::to_string(dims) + " dimensions"};
  return t;
}

// The device that the call's first tensor fixes.
c10::DeviceIndex device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) throw Raise{PyExc_ValueError, std::string(name) + " must be a CUDA tensor"};
  return t.get_device();
}
void on_device(const at::Tensor& t, const char* name, c10::DeviceIndex index) {
  if (!t.is_cuda()) throw Raise{PyExc_ValueError, std::string(name) + " must be a CUDA tensor"};
  if (t.get_device() != index)
    throw Raise{PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                      ", expected cuda:" + std::to_string(index)};
}
// t must be a dense tensor of that type and shape on that device.
void fit(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::DeviceIndex index) {
  on_device(t, name, index);
  if (t.scalar_type() != type)
    throw Raise{PyExc_ValueError, std::string(name) + " must have dtype " + c10::toString(type) + ", got " +
                                      c10::toString(t.scalar_type())};
  if (t.sizes() != shape)
    throw Raise{PyExc_ValueError,
                std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape)};
  if (!t.is_contiguous()) throw Raise{PyExc_ValueError, std::string(name) + " must be contiguous"};
}
// The output that the caller passes, or a new one.
at::Tensor output(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::DeviceIndex index) {
  if (o == Py_None) return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, index)));
  const at::Tensor& t = tensor(o, name);
  fit(t, name, type, shape, index);
  return t;
}

// Tells autograd that a call wrote tensors that the caller had before (undefined ones are skipped): a graph that saved one,
// as the rotation saves its positions, then refuses its backward instead of reading the new values.
void changed(std::initializer_list<at::Tensor> written) {
  for (const at::Tensor& t : written)
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// New outputs of one call as parts of one allocation (four of them took 3 us more): next(type, shape) gives the next.
class Parts {
 public:
  Parts(c10::DeviceIndex index, int64_t bytes)
      : buf_(at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(c10::Device(c10::kCUDA, index)))) {}
  static int64_t room(int64_t bytes) { return (bytes + 255) / 256 * 256; }
  at::Tensor next(at::ScalarType type, int64_t n) { return next(type, at::IntArrayRef{n}); }
  at::Tensor next(at::ScalarType type, at::IntArrayRef shape) {
    const int64_t size = static_cast<int64_t>(c10::elementSize(type));
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf_.storage()),
                                                            c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset((buf_.storage_offset() + at_) / size);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    at_ += room(t.numel() * size);
    return t;
  }

 private:
  at::Tensor buf_;
  int64_t at_ = 0;
};

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// Address and size of a call's workspace: the given buffer, or, for a call that only needs the error word, one word per
// device that nothing reads (so it needs no initial value, and calls may share it).
struct Space {
  void* at;
  size_t bytes;
  at::Tensor keep;
};
Space error_word(PyObject* o, c10::DeviceIndex index) {
  if (o != Py_None) {
    const at::Tensor& t = tensor(o, "workspace");
    on_device(t, "workspace", index);
    return {t.data_ptr(), static_cast<size_t>(t.nbytes()), t};
  }
  constexpr int64_t kBytes = 256;
  static std::atomic<void*> words[64];
  const bool kept = index < 64;
  if (kept)
    if (void* p = words[index].load(std::memory_order_acquire)) return {p, kBytes, {}};
  at::Tensor t =
      at::empty({kBytes}, at::TensorOptions().dtype(at::kByte).device(c10::Device(c10::kCUDA, index)));
  // (during a capture it belongs to the graph)
  if (kept && c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) {
    void* none = nullptr;
    if (words[index].compare_exchange_strong(none, t.data_ptr())) new at::Tensor(t);  // kept for the process
  }
  return {t.data_ptr(), kBytes, t};
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

// Runs `call` (a call into libmsa on the device's current stream, without the interpreter's lock); its status.
template <class F>
msa_status run(c10::DeviceIndex index, F call) {
  const c10::cuda::CUDAGuard guard(index);
  void* stream = c10::cuda::getCurrentCUDAStream(index).stream();
  msa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = call(stream);
  Py_END_ALLOW_THREADS
  return st;
}

// An entry: `n` positional arguments; exceptions become Python's.
template <class F>
PyObject* entry(const char* name, Py_ssize_t have, Py_ssize_t want, F body) {
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, have);
    return nullptr;
  }
  try {
    return body();
  } catch (const Raise& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (const Raised&) {
  } catch (const Refused& e) {
    return PyLong_FromLong(e.status);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// (outputs...) as a tuple, None for one that is not there.
PyObject* pack(std::initializer_list<at::Tensor> outputs) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(outputs.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : outputs) {
    PyObject* o = t.defined() ? wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// seq_lens, new_lens, page_table, free_pages, num_free, num_slots, capacity, cu_seqlens_q, slots, positions, num_free_out,
// workspace
PyObject* map_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("map_slots", n, 12, [&]() -> PyObject* {
    const at::Tensor& lens = tensor_of(a[0], "seq_lens", 1);
    const int64_t batch = lens.size(0), num_slots = whole(a[5]), capacity = whole(a[6]);
    const c10::DeviceIndex d = device_of(lens, "seq_lens");
    const at::Tensor &news = tensor(a[1], "new_lens"), &table = tensor_of(a[2], "page_table", 2),
                     &pages = tensor_of(a[3], "free_pages", 1), &num = tensor(a[4], "num_free");
    fit(lens, "seq_lens", at::kInt, {batch}, d);
    fit(news, "new_lens", at::kInt, {batch}, d);
    fit(table, "page_table", at::kInt, {batch, table.size(1)}, d);
    fit(pages, "free_pages", at::kInt, {pages.size(0)}, d);
    fit(num, "num_free", at::kInt, {1}, d);
    if (batch < 1 || batch > INT32_MAX || table.size(1) < 1 || table.size(1) > INT32_MAX || capacity < 1)
      return PyLong_FromLong(MSA_ERR_SHAPE);
    if (capacity >= (1LL << 31)) return PyLong_FromLong(MSA_ERR_SHAPE);
    at::Tensor cu, slots, positions, left;
    if (a[7] == Py_None && a[8] == Py_None && a[9] == Py_None && a[10] == Py_None) {
      Parts parts(d, Parts::room(4 * (batch + 1)) + Parts::room(8 * capacity) + Parts::room(4 * capacity) + Parts::room(4));
      cu = parts.next(at::kInt, batch + 1);
      slots = parts.next(at::kLong, capacity);
      positions = parts.next(at::kInt, capacity);
      left = parts.next(at::kInt, 1);
    } else {
      cu = output(a[7], "cu_seqlens_q", at::kInt, {batch + 1}, d);
      slots = output(a[8], "slots", at::kLong, {capacity}, d);
      positions = output(a[9], "positions", at::kInt, {capacity}, d);
      left = output(a[10], "num_free_out", at::kInt, {1}, d);
    }
    const Space ws = error_word(a[11], d);
    const msa_status st = run(d, [&](void* stream) {
      return msa_map_slots(lens.const_data_ptr<int32_t>(), news.const_data_ptr<int32_t>(), static_cast<int>(batch),
                           table.data_ptr<int32_t>(), static_cast<int>(table.size(1)),
                           pages.size(0) ? pages.const_data_ptr<int32_t>() : nullptr, pages.size(0),
                           num.const_data_ptr<int32_t>(), num_slots, capacity, cu.data_ptr<int32_t>(),
                           slots.data_ptr<int64_t>(), positions.data_ptr<int32_t>(), left.data_ptr<int32_t>(), ws.at,
                           ws.bytes, stream);
    });
    if (st != MSA_OK) return PyLong_FromLong(st);
    changed({table, cu, slots, positions, left});
    return pack({cu, slots, positions, left});
  });
}

// The rotation's form, from positions, inv_freq, axes (None or a sequence of whole numbers) and interleaved.
msa_rotary_config rotary_form(const at::Tensor& positions, const at::Tensor& inv_freq, PyObject* axes,
                              PyObject* interleaved) {
  const int64_t pairs = inv_freq.size(0), rows = positions.dim() == 2 ? positions.size(0) : 1;
  msa_rotary_config rot{static_cast<int>(2 * pairs), truth(interleaved), static_cast<int>(rows), {}};
  if (pairs > 64)
    throw Raise{PyExc_ValueError, "inv_freq has " + std::to_string(pairs) + " entries, at most 64 pairs of a head can turn"};
  if (axes == Py_None) return rot;
  PyObject* list = PySequence_Fast(axes, "axes must be a sequence");
  if (!list) throw Raised{};
  const Py_ssize_t have = PySequence_Fast_GET_SIZE(list);
  std::string wrong;
  if (have != pairs)
    wrong = "axes has " + std::to_string(have) + " entries, inv_freq has " + std::to_string(pairs);
  bool raised = false;
  for (Py_ssize_t j = 0; j < have && wrong.empty() && !raised; ++j) {
    const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(list, j));
    if (v == -1 && PyErr_Occurred()) raised = true;
    else if (v < 0 || v >= rows) wrong = "axes must lie in [0, " + std::to_string(rows) + "), the rows of positions";
    else rot.axis[j] = static_cast<uint8_t>(v);
  }
  Py_DECREF(list);
  if (raised) throw Raised{};
  if (!wrong.empty()) throw Raise{PyExc_ValueError, wrong};
  return rot;
}
void fit_angles(const at::Tensor& positions, const at::Tensor& inv_freq, int64_t tokens, c10::DeviceIndex d) {
  if (positions.dim() == 2) fit(positions, "positions", at::kInt, {positions.size(0), tokens}, d);
  else fit(positions, "positions", at::kInt, {tokens}, d);
  fit(inv_freq, "inv_freq", at::kFloat, {inv_freq.size(0)}, d);
}

// Stride between the tokens of a bf16 [tokens, heads, 128] tensor whose heads are dense (heads < 0: any number).
int64_t token_stride(const at::Tensor& t, const char* name, int64_t tokens, int64_t heads, c10::DeviceIndex d) {
  on_device(t, name, d);
  if (t.scalar_type() != at::kBFloat16)
    throw Raise{PyExc_ValueError, std::string(name) + " must have dtype BFloat16, got " + c10::toString(t.scalar_type())};
  if (heads < 0) heads = t.size(1);
  if (t.size(0) != tokens || t.size(1) != heads || t.size(2) != kD)
    throw Raise{PyExc_ValueError, std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " +
                                      shape_text(Sizes{tokens, heads, kD})};
  if (t.stride(2) != 1 || (t.stride(1) != kD && heads > 1))
    throw Raise{PyExc_ValueError, std::string(name) + " must have dense heads, got strides " + shape_text(t.strides())};
  if (tokens == 1) return heads * kD;  // a single token's stride says nothing
  if (t.stride(0) < heads * kD || t.stride(0) % 8)
    throw Raise{PyExc_ValueError, std::string(name) + " must have tokens a multiple of 8 elements apart that do not overlap, "
                                                      "got " + std::to_string(t.stride(0))};
  return t.stride(0);
}

// q, k, positions, inv_freq, axes, interleaved, inverse, q_out, k_out
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("rotary", n, 9, [&]() -> PyObject* {
    const at::Tensor& q = tensor_of(a[0], "q", 3);
    const at::Tensor &positions = tensor(a[2], "positions"), &inv_freq = tensor_of(a[3], "inv_freq", 1);
    const msa_rotary_config rot = rotary_form(positions, inv_freq, a[4], a[5]);
    const bool inverse = truth(a[6]);
    const c10::DeviceIndex d = device_of(q, "q");
    const int64_t tokens = q.size(0), heads = q.size(1), qs = token_stride(q, "q", tokens, -1, d);
    fit_angles(positions, inv_freq, tokens, d);
    at::Tensor k, ko;
    int64_t ks = 0;
    if (a[1] != Py_None) {
      k = tensor_of(a[1], "k", 3);
      ks = token_stride(k, "k", tokens, -1, d);
    } else if (a[8] != Py_None) {
      throw Raise{PyExc_ValueError, "k_out without k"};
    }
    if (tokens < 1) return PyLong_FromLong(MSA_ERR_SHAPE);
    const at::Tensor qo = output(a[7], "q_out", at::kBFloat16, q.sizes(), d);
    if (k.defined()) ko = output(a[8], "k_out", at::kBFloat16, k.sizes(), d);
    const msa_status st = run(d, [&](void* stream) {
      return msa_rotary(&rot, q.const_data_ptr(), qs, static_cast<int>(heads), k.defined() ? k.const_data_ptr() : nullptr,
                        ks, k.defined() ? static_cast<int>(k.size(1)) : 0, positions.const_data_ptr<int32_t>(),
                        inv_freq.const_data_ptr<float>(), tokens, inverse, qo.data_ptr(),
                        ko.defined() ? ko.data_ptr() : nullptr, stream);
    });
    if (st != MSA_OK) return PyLong_FromLong(st);
    changed({qo, ko});
    return pack({qo, ko});
  });
}

// The rotation as an autograd function: its gradient is the rotation back (so it can be differentiated again).
struct Rotary : torch::autograd::Function<Rotary> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx, const at::Tensor& q,
                                                const at::Tensor& k, const at::Tensor& positions,
                                                const at::Tensor& inv_freq, const msa_rotary_config& rot, bool inverse) {
    ctx->save_for_backward({positions, inv_freq});
    ctx->saved_data["rot"] = std::string(reinterpret_cast<const char*>(&rot), sizeof(rot));
    ctx->saved_data["inverse"] = inverse;
    return turn(q, k, positions, inv_freq, rot, inverse);
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const auto saved = ctx->get_saved_variables();
    msa_rotary_config rot;
    std::memcpy(&rot, ctx->saved_data["rot"].toStringRef().data(), sizeof(rot));
    const bool inverse = !ctx->saved_data["inverse"].toBool();
    // (a gradient may come in any layout, and begin anywhere)
    auto dense = [](const at::Tensor& t) {
      const at::Tensor c = t.contiguous();
      return reinterpret_cast<uintptr_t>(c.const_data_ptr()) % 16 ? c.clone() : c;
    };
    const at::Tensor gq = dense(grads[0]), gk = dense(grads[1]);
    torch::autograd::variable_list out = c10::GradMode::is_enabled() ? apply(gq, gk, saved[0], saved[1], rot, inverse)
                                      : turn(gq, gk, saved[0], saved[1], rot, inverse);
    out.resize(6);  // none for the other arguments
    return out;
  }
  static torch::autograd::variable_list turn(const at::Tensor& q, const at::Tensor& k, const at::Tensor& positions,
                                             const at::Tensor& inv_freq, const msa_rotary_config& rot, bool inverse) {
    const c10::cuda::CUDAGuard guard(q.get_device());
    const at::Tensor qo = at::empty(q.sizes(), q.options()), ko = at::empty(k.sizes(), k.options());
    const int64_t tokens = q.size(0);
    auto stride = [&](const at::Tensor& t) { return tokens == 1 ? t.size(1) * kD : t.stride(0); };
    const msa_status st =
        msa_rotary(&rot, q.const_data_ptr(), stride(q), static_cast<int>(q.size(1)), k.const_data_ptr(), stride(k),
                   static_cast<int>(k.size(1)), positions.const_data_ptr<int32_t>(), inv_freq.const_data_ptr<float>(),
                   tokens, inverse, qo.data_ptr(), ko.data_ptr(), c10::cuda::getCurrentCUDAStream(q.get_device()).stream());
    if (st != MSA_OK) throw Refused(st);
    return {qo, ko};
  }
};

// q, k, positions, inv_freq, axes, interleaved
PyObject* rotary_autograd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("rotary_autograd", n, 6, [&]() -> PyObject* {
    const at::Tensor &q = tensor_of(a[0], "q", 3), &k = tensor_of(a[1], "k", 3);
    const at::Tensor &positions = tensor(a[2], "positions"), &inv_freq = tensor_of(a[3], "inv_freq", 1);
    const msa_rotary_config rot = rotary_form(positions, inv_freq, a[4], a[5]);
    const c10::DeviceIndex d = device_of(q, "q");
    const int64_t tokens = q.size(0);
    token_stride(q, "q", tokens, -1, d);
    token_stride(k, "k", tokens, -1, d);
    fit_angles(positions, inv_freq, tokens, d);
    if (tokens < 1) return PyLong_FromLong(MSA_ERR_SHAPE);
    const auto out = Rotary::apply(q, k, positions, inv_freq, rot, false);
    return pack({out[0], out[1]});
  });
}

// A pair of caches [slots, 4, 128]: whether they hold E4M3 bytes.
bool fit_caches(const at::Tensor& k, const at::Tensor& v, c10::DeviceIndex d) {
  const at::ScalarType type = k.scalar_type();
  const bool fp8 = type == at::kFloat8_e4m3fn || type == at::kByte;
  if (!fp8 && type != at::kBFloat16)
    throw Raise{PyExc_ValueError, std::string("k_cache must be bf16, float8_e4m3fn or uint8, got ") + c10::toString(type)};
  fit(k, "k_cache", type, {k.size(0), kG, kD}, d);
  fit(v, "v_cache", type, {k.size(0), kG, kD}, d);
  return fp8;
}

// q, k, v, positions, inv_freq, slots, k_cache, v_cache, axes, interleaved, k_scale, v_scale, q_out, k_out, workspace
PyObject* rotary_insert(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("rotary_insert", n, 15, [&]() -> PyObject* {
    const at::Tensor& q = tensor_of(a[0], "q", 3);
    const at::Tensor &positions = tensor(a[3], "positions"), &inv_freq = tensor_of(a[4], "inv_freq", 1);
    const msa_rotary_config rot = rotary_form(positions, inv_freq, a[8], a[9]);
    const float k_scale = static_cast<float>(number(a[10])), v_scale = static_cast<float>(number(a[11]));
    const c10::DeviceIndex d = device_of(q, "q");
    const at::Tensor &k = tensor_of(a[1], "k", 3), &v = tensor_of(a[2], "v", 3), &slots = tensor(a[5], "slots"),
                     &k_cache = tensor_of(a[6], "k_cache", 3), &v_cache = tensor(a[7], "v_cache");
    const int64_t tokens = q.size(0), qs = token_stride(q, "q", tokens, kH, d), ks = token_stride(k, "k", tokens, kG, d),
                  vs = token_stride(v, "v", tokens, kG, d);
    fit_angles(positions, inv_freq, tokens, d);
    fit(slots, "slots", at::kLong, {tokens}, d);
    const bool fp8 = fit_caches(k_cache, v_cache, d);
    if (tokens < 1) return PyLong_FromLong(MSA_ERR_SHAPE);
    const at::Tensor qo = output(a[12], "q_out", at::kBFloat16, q.sizes(), d);
    at::Tensor ko;
    if (a[13] != Py_None) ko = output(a[13], "k_out", at::kBFloat16, {tokens, kG, kD}, d);
    const Space ws = error_word(a[14], d);
    const msa_status st = run(d, [&](void* stream) {
      return msa_rotary_insert(&rot, q.const_data_ptr(), qs, k.const_data_ptr(), ks, v.const_data_ptr(), vs,
                               positions.const_data_ptr<int32_t>(), inv_freq.const_data_ptr<float>(),
                               slots.const_data_ptr<int64_t>(), tokens, qo.data_ptr(),
                               ko.defined() ? ko.data_ptr() : nullptr, k_cache.data_ptr(), v_cache.data_ptr(), fp8, k_scale,
                               v_scale, k_cache.size(0), ws.at, ws.bytes, stream);
    });
    if (st != MSA_OK) return PyLong_FromLong(st);
    changed({qo, ko, k_cache, v_cache});
    return wrap(qo);
  });
}

// An int8 cache: its caches [slots, 4, 128], and its scales by page, KV head and slot.
void fit_int8(const at::Tensor& k, const at::Tensor& v, const at::Tensor& ks, const at::Tensor& vs, c10::DeviceIndex d) {
  const int64_t slots = k.size(0);
  fit(k, "k_cache", at::kChar, {slots, kG, kD}, d);
  fit(v, "v_cache", at::kChar, {slots, kG, kD}, d);
  if (slots % kD)
    throw Raise{PyExc_ValueError, "k_cache has " + std::to_string(slots) + " slots, expected a multiple of 128"};
  fit(ks, "k_scales", at::kBFloat16, {slots / kD, kG, kD}, d);
  fit(vs, "v_scales", at::kBFloat16, {slots / kD, kG, kD}, d);
}

// kind, q, k_cache, v_cache, k_scale, v_scale, seq_lens, page_table, cu_seqlens_q, group_offsets, shared_lens, scale, out, lse,
// workspace.  kind: 0 bf16, 1 E4M3 (one number each for k_scale and v_scale), 2 int8 (the rows' scales); group_offsets and
// shared_lens None: msa_attend_chunk
PyObject* attend_chunk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("attend_chunk", n, 15, [&]() -> PyObject* {
    const int64_t kind = whole(a[0]);
    const bool shared = a[9] != Py_None || a[10] != Py_None;
    const at::Tensor& q = tensor_of(a[1], "q", 3);
    const c10::DeviceIndex d = device_of(q, "q");
    const at::Tensor &k = tensor_of(a[2], "k_cache", 3), &v = tensor(a[3], "v_cache"), &lens = tensor(a[6], "seq_lens"),
                     &table = tensor_of(a[7], "page_table", 2), &cu = tensor(a[8], "cu_seqlens_q");
    const float scale = a[11] == Py_None ? 0.088388347648318447f : static_cast<float>(number(a[11]));  // 1 / sqrt(128)
    const int64_t tokens = q.size(0), batch = table.size(0), width = table.size(1);
    fit(q, "q", at::kBFloat16, {tokens, kH, kD}, d);
    float k_scale = 1.f, v_scale = 1.f;
    at::Tensor k_scales, v_scales, offsets, lengths;
    if (kind == 2) {
      k_scales = tensor(a[4], "k_scales");
      v_scales = tensor(a[5], "v_scales");
      fit_int8(k, v, k_scales, v_scales, d);
    } else {
      k_scale = static_cast<float>(number(a[4]));
      v_scale = static_cast<float>(number(a[5]));
      if (fit_caches(k, v, d) != (kind == 1))
        throw Raise{PyExc_ValueError, std::string(shared ? "msa_attend_shared" : "msa_attend_chunk") +
                                          (kind == 1 ? "_fp8kv takes float8_e4m3fn or uint8 caches, got "
                                                     : " takes bf16 caches, got ") +
                                          c10::toString(k.scalar_type())};
    }
    fit(table, "page_table", at::kInt, {batch, width}, d);
    fit(lens, "seq_lens", at::kInt, {batch}, d);
    fit(cu, "cu_seqlens_q", at::kInt, {batch + 1}, d);
    int groups = 0;
    if (shared) {
      lengths = tensor_of(a[10], "shared_lens", 1);
      offsets = tensor(a[9], "group_offsets");
      const int64_t g = lengths.size(0);
      fit(lengths, "shared_lens", at::kInt, {g}, d);
      fit(offsets, "group_offsets", at::kInt, {g + 1}, d);
      if (g > batch)
        throw Raise{PyExc_ValueError, "shared_lens has " + std::to_string(g) + " groups, the batch " + std::to_string(batch) +
                                          " requests"};
      groups = static_cast<int>(g);
    }
    if (tokens < 1 || batch < 1 || batch > INT32_MAX || width < 1 || width > INT32_MAX)
      return PyLong_FromLong(MSA_ERR_SHAPE);
    const at::Tensor out = output(a[12], "out", at::kBFloat16, q.sizes(), d);
    at::Tensor lse;
    if (a[13] != Py_None) lse = output(a[13], "lse", at::kFloat, {tokens, kH}, d);
    msa_config cfg;
    msa_config_default(&cfg);
    Space ws;
    if (a[14] == Py_None) {
      size_t bytes = 0;
      const msa_status st = msa_workspace_size(&cfg, groups ? MSA_MODE_SHARED : MSA_MODE_CHUNK, tokens, static_cast<int>(width),
                                               &bytes);
      if (st != MSA_OK) return PyLong_FromLong(st);
      ws.keep = at::empty({static_cast<int64_t>(bytes)},
                          at::TensorOptions().dtype(at::kByte).device(c10::Device(c10::kCUDA, d)));
      ws.at = ws.keep.data_ptr();
      ws.bytes = bytes;
    } else {
      ws = error_word(a[14], d);
    }
    const msa_status st = run(d, [&](void* stream) {
      const void *qp = q.const_data_ptr(), *kp = k.const_data_ptr(), *vp = v.const_data_ptr();
      const int32_t *lp = lens.const_data_ptr<int32_t>(), *tp = table.const_data_ptr<int32_t>(),
                    *cp = cu.const_data_ptr<int32_t>(), *gp = groups ? offsets.const_data_ptr<int32_t>() : nullptr,
                    *sl = groups ? lengths.const_data_ptr<int32_t>() : nullptr;
      const void *ks = kind == 2 ? k_scales.const_data_ptr() : nullptr, *vs = kind == 2 ? v_scales.const_data_ptr() : nullptr;
      float* sp = lse.defined() ? lse.data_ptr<float>() : nullptr;
      const int b = static_cast<int>(batch), w = static_cast<int>(width);
      void* op = out.data_ptr();
      if (kind == 2)
        return msa_attend_shared_int8kv(&cfg, qp, kp, vp, ks, vs, lp, tp, cp, b, w, gp, sl, groups, tokens, k.size(0), scale, op,
                                        sp, ws.at, ws.bytes, stream);
      if (kind == 1)
        return msa_attend_shared_fp8kv(&cfg, qp, kp, vp, k_scale, v_scale, lp, tp, cp, b, w, gp, sl, groups, tokens, k.size(0),
                                       scale, op, sp, ws.at, ws.bytes, stream);
      return msa_attend_shared(&cfg, qp, kp, vp, lp, tp, cp, b, w, gp, sl, groups, tokens, k.size(0), scale, op, sp, ws.at,
                               ws.bytes, stream);
    });
    if (st != MSA_OK) return PyLong_FromLong(st);
    changed({out, lse});
    return wrap(out);
  });
}

// k, v, slots, k_cache, v_cache, k_scales, v_scales, workspace
PyObject* quantize_insert(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("quantize_insert", n, 8, [&]() -> PyObject* {
    const at::Tensor &k = tensor_of(a[0], "k", 3), &v = tensor_of(a[1], "v", 3);
    const c10::DeviceIndex d = device_of(k, "k");
    const at::Tensor &slots = tensor(a[2], "slots"), &kc = tensor_of(a[3], "k_cache", 3), &vc = tensor(a[4], "v_cache"),
                     &ks = tensor(a[5], "k_scales"), &vs = tensor(a[6], "v_scales");
    const int64_t tokens = k.size(0), k_stride = token_stride(k, "k", tokens, kG, d),
                  v_stride = token_stride(v, "v", tokens, kG, d);
    fit(slots, "slots", at::kLong, {tokens}, d);
    fit_int8(kc, vc, ks, vs, d);
    if (tokens < 1) return PyLong_FromLong(MSA_ERR_SHAPE);
    const Space ws = error_word(a[7], d);
    const msa_status st = run(d, [&](void* stream) {
      return msa_quantize_insert(k.const_data_ptr(), k_stride, v.const_data_ptr(), v_stride, slots.const_data_ptr<int64_t>(),
                                 tokens, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), kc.size(0), ws.at,
                                 ws.bytes, stream);
    });
    if (st != MSA_OK) return PyLong_FromLong(st);
    changed({kc, vc, ks, vs});
    Py_RETURN_NONE;
  });
}

// k_cache, v_cache, k_scales, v_scales, page_table, cu_seqlens, total_tokens, starts, k_out, v_out, workspace
PyObject* dequantize_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("dequantize_gather", n, 11, [&]() -> PyObject* {
    const at::Tensor& kc = tensor_of(a[0], "k_cache", 3);
    const c10::DeviceIndex d = device_of(kc, "k_cache");
    const at::Tensor &vc = tensor(a[1], "v_cache"), &ks = tensor(a[2], "k_scales"), &vs = tensor(a[3], "v_scales"),
                     &table = tensor_of(a[4], "page_table", 2), &cu = tensor(a[5], "cu_seqlens");
    const int64_t tokens = whole(a[6]), batch = table.size(0), width = table.size(1);
    fit_int8(kc, vc, ks, vs, d);
    fit(table, "page_table", at::kInt, {batch, width}, d);
    fit(cu, "cu_seqlens", at::kInt, {batch + 1}, d);
    at::Tensor starts;
    if (a[7] != Py_None) {
      starts = tensor(a[7], "starts");
      fit(starts, "starts", at::kInt, {batch}, d);
    }
    if (tokens < 1 || tokens > INT32_MAX || batch < 1 || batch > INT32_MAX || width < 1 || width > INT32_MAX)
      return PyLong_FromLong(MSA_ERR_SHAPE);
    at::Tensor ko, vo;
    // (one allocation for both of a short read, which waits for the host; long ones may be freed by themselves)
    if (a[8] == Py_None && a[9] == Py_None && tokens <= 4096) {
      const Sizes shape{tokens, kG, kD};
      Parts parts(d, 2 * Parts::room(tokens * kG * kD * 2));
      ko = parts.next(at::kBFloat16, shape);
      vo = parts.next(at::kBFloat16, shape);
    } else {
      ko = output(a[8], "k_out", at::kBFloat16, {tokens, kG, kD}, d);
      vo = output(a[9], "v_out", at::kBFloat16, {tokens, kG, kD}, d);
    }
    const Space ws = error_word(a[10], d);
    const msa_status st = run(d, [&](void* stream) {
      return msa_dequantize_gather(kc.const_data_ptr(), vc.const_data_ptr(), ks.const_data_ptr(), vs.const_data_ptr(),
                                   kc.size(0), table.const_data_ptr<int32_t>(),
                                   starts.defined() ? starts.const_data_ptr<int32_t>() : nullptr,
                                   cu.const_data_ptr<int32_t>(), static_cast<int>(batch), static_cast<int>(width), tokens,
                                   ko.data_ptr(), vo.data_ptr(), ws.at, ws.bytes, stream);
    });
    if (st != MSA_OK) return PyLong_FromLong(st);
    changed({ko, vo});
    return pack({ko, vo});
  });
}

// q, k_cache, v_cache, k_scales, v_scales, q2k, seq_lens, page_table, scale, out, workspace
PyObject* sparse_attend_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("sparse_attend_int8", n, 11, [&]() -> PyObject* {
    const at::Tensor& q = tensor_of(a[0], "q", 3);
    const c10::DeviceIndex d = device_of(q, "q");
    const at::Tensor &kc = tensor_of(a[1], "k_cache", 3), &vc = tensor(a[2], "v_cache"), &ks = tensor(a[3], "k_scales"),
                     &vs = tensor(a[4], "v_scales"), &q2k = tensor_of(a[5], "q2k", 3), &lens = tensor(a[6], "seq_lens"),
                     &table = tensor_of(a[7], "page_table", 2);
    const float scale = a[8] == Py_None ? 0.088388347648318447f : static_cast<float>(number(a[8]));  // 1 / sqrt(128)
    const int64_t batch = q.size(0), width = table.size(1), topk = q2k.size(2);
    fit(q, "q", at::kBFloat16, {batch, kH, kD}, d);
    fit_int8(kc, vc, ks, vs, d);
    fit(q2k, "q2k", at::kInt, {kG, batch, topk}, d);
    fit(lens, "seq_lens", at::kInt, {batch}, d);
    fit(table, "page_table", at::kInt, {batch, width}, d);
    if (batch < 1 || batch > INT32_MAX || width < 1 || width > INT32_MAX || topk < 1 || topk > 16)
      return PyLong_FromLong(MSA_ERR_SHAPE);
    const at::Tensor out = output(a[9], "out", at::kBFloat16, q.sizes(), d);
    msa_config cfg;
    msa_config_default(&cfg);
    cfg.topk = static_cast<int>(topk);
    cfg.local_blocks = 0;
    const Space ws = error_word(a[10], d);
    const msa_status st = run(d, [&](void* stream) {
      return msa_sparse_attend_decode_int8kv(&cfg, q.const_data_ptr(), kc.const_data_ptr(), vc.const_data_ptr(),
                                             ks.const_data_ptr(), vs.const_data_ptr(), q2k.const_data_ptr<int32_t>(),
                                             lens.const_data_ptr<int32_t>(), table.const_data_ptr<int32_t>(),
                                             static_cast<int>(batch), static_cast<int>(width), kc.size(0), scale,
                                             out.data_ptr(), ws.at, ws.bytes, stream);
    });
    if (st != MSA_OK) return PyLong_FromLong(st);
    changed({out});
    return wrap(out);
  });
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef kMethods[] = {method("map_slots", map_slots), method("rotary", rotary), method("rotary_autograd", rotary_autograd),
                          method("rotary_insert", rotary_insert), method("attend_chunk", attend_chunk),
                          method("quantize_insert", quantize_insert), method("dequantize_gather", dequantize_gather),
                          method("sparse_attend_int8", sparse_attend_int8),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "msa_serving", nullptr, -1, kMethods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_msa_serving() { return PyModule_Create(&kModule); }
