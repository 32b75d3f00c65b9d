// binding.cpp -- the native half of the Python binding for entry points whose calls are short.
//
// A serving step calls kernels of 5 to 10 us; checking and marshalling their arguments in Python
// cost 10 to 15 us per call (attribute reads, ctypes conversions, torch.empty). Here an entry point
// is described once by a line of text, and `invoke` checks the tensors, allocates the outputs and
// calls the C function from that description:
//
//   arguments            q:bf16[B,Hq,D]      contiguous tensor; a size name binds where it first
//                                            appears and must agree afterwards; "X/2" and "X+1" too
//                        q:io<T,Hq,D>        the heads of a token contiguous, any token stride (q.s);
//                                            io: bf16 or fp32, the same for all of a call
//                        k:any[N,...]        any dtype (the same for all), further sizes alike (N.size:
//                                            bytes of one entry of the first size)
//                        x:..?               may be None (a null pointer; its sizes stay 0)
//                        >out:bf16[B,D]      an output: checked if given, else allocated; ">o:..?k": only
//                                            where k is given
//                        #n  !flag           an integer, a truth value
//                        %sections           a sequence of ints: pointer, %.n entries, %.sum
//                        @ws(B,S,..)         a workspace, two Python arguments: the address of the C
//                                            function that gives its bytes for these sizes, and a tensor
//                                            or None (allocated); ws is its pointer, ws.n its bytes
//   "->" C arguments     names of tensors (data pointers), sizes, scalars, io (dtype code), %, %.n
//   "=>" results         one tensor, or a tuple
//
// The last Python argument is the stream (None: the device's current one; a torch stream; a raw
// handle), the last C argument its handle. What a call allocates comes from the memory pool of the
// stream that it runs on: a block of the current stream's pool may still be in use by work queued
// there, which the given stream does not wait for. Outputs are recorded on the current stream, where
// the caller will read them. Calls run on the tensors' device. Errors: TypeError for dtypes,
// ValueError for shapes, devices and layouts; a status other than 0 goes to the callable given to
// `on_error`.

#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <array>
#include <string>
#include <vector>

namespace {

constexpr int kMaxSyms = 32, kMaxTensors = 16, kMaxArgs = 40, kMaxSeq = 8;

enum class Kind { kTensor, kOut, kInt, kFlag, kSeq, kSizeFn, kWork };
enum class Layout { kContiguous, kHeads, kAlike };
enum class Type { kBf16, kF32, kI32, kIo, kAny };

struct Dim {
  int sym = -1;  // -1: the constant `add`
  int div = 1;
  int add = 0;
};

struct Item {
  Kind kind = Kind::kTensor;
  std::string name;
  Type type = Type::kBf16;
  Layout layout = Layout::kContiguous;
  std::vector<Dim> dims;
  bool optional = false;
  int only_with = -1;  // an output that exists only where this item is given
  int tensor = -1;     // index among the tensors
  int sym = -1;        // the symbol of a scalar, of a sequence's length, or of a layout's stride or size
  int sum = -1;        // the symbol of a sequence's sum
  std::vector<int> sizes;  // the symbols that a workspace's size function takes
};

struct CArg {
  enum { kTensorPtr, kSym, kIoCode, kSeqPtr } kind;
  int index;
};

struct Entry {
  std::string name;
  std::vector<Item> items;
  std::vector<CArg> cargs;
  std::vector<int> results;  // tensor indices
  std::vector<std::string> syms;
  int n_tensors = 0;
};

std::vector<Entry>& entries() {
  static std::vector<Entry> e;
  return e;
}
PyObject* g_on_error = nullptr;

int sym_of(Entry& e, const std::string& s, bool add) {
  for (size_t i = 0; i < e.syms.size(); ++i)
    if (e.syms[i] == s) return static_cast<int>(i);
  TORCH_CHECK(add && e.syms.size() < kMaxSyms, "binding: unknown name ", s, " in ", e.name);
  e.syms.push_back(s);
  return static_cast<int>(e.syms.size()) - 1;
}

Dim parse_dim(Entry& e, const std::string& s) {
  Dim d;
  if (isdigit(static_cast<unsigned char>(s[0]))) {
    d.add = std::stoi(s);
    return d;
  }
  const size_t op = s.find_first_of("/+");
  d.sym = sym_of(e, s.substr(0, op), true);
  if (op != std::string::npos) (s[op] == '/' ? d.div : d.add) = std::stoi(s.substr(op + 1));
  return d;
}

Entry parse(const std::string& name, const std::string& spec) {
  Entry e;
  e.name = name;
  std::vector<std::string> words;
  for (size_t i = 0; i < spec.size();) {
    const size_t j = spec.find_first_of(" \n", i);
    if (j != i) words.push_back(spec.substr(i, j == std::string::npos ? j : j - i));
    if (j == std::string::npos) break;
    i = j + 1;
  }
  int part = 0;
  for (const std::string& w : words) {
    if (w == "->" || w == "=>") {
      ++part;
      continue;
    }
    if (part == 0) {
      Item it;
      if (w[0] == '#' || w[0] == '!' || w[0] == '%') {
        it.kind = w[0] == '#' ? Kind::kInt : w[0] == '!' ? Kind::kFlag : Kind::kSeq;
        it.name = w.substr(1);
        if (it.kind != Kind::kSeq) {
          it.sym = sym_of(e, it.name, true);
        } else {
          it.sym = sym_of(e, "%.n", true);
          it.sum = sym_of(e, "%.sum", true);
        }
        e.items.push_back(it);
        continue;
      }
      if (w[0] == '@') {
        const size_t open = w.find('('), close = w.find(')');
        Item fn;
        fn.kind = Kind::kSizeFn;
        fn.name = w.substr(1, open - 1) + " size function";
        e.items.push_back(fn);
        it.kind = Kind::kWork;
        it.name = w.substr(1, open - 1);
        it.tensor = e.n_tensors++;
        it.sym = sym_of(e, it.name + ".n", true);
        std::string dims = w.substr(open + 1, close - open - 1);
        for (size_t i = 0; i < dims.size();) {
          size_t j = dims.find(',', i);
          if (j == std::string::npos) j = dims.size();
          it.sizes.push_back(sym_of(e, dims.substr(i, j - i), false));
          i = j + 1;
        }
        TORCH_CHECK(e.n_tensors <= kMaxTensors && it.sizes.size() <= 8, "binding: malformed workspace in ", name);
        e.items.push_back(it);
        continue;
      }
      const bool out = w[0] == '>';
      it.kind = out ? Kind::kOut : Kind::kTensor;
      const size_t colon = w.find(':'), open = w.find_first_of("[<", colon), close = w.find_last_of("]>");
      it.name = w.substr(out ? 1 : 0, colon - (out ? 1 : 0));
      const std::string type = w.substr(colon + 1, open - colon - 1);
      it.type = type == "bf16" ? Type::kBf16 : type == "f32" ? Type::kF32 : type == "i32" ? Type::kI32
                : type == "io" ? Type::kIo : Type::kAny;
      it.layout = w[open] == '<' ? Layout::kHeads : Layout::kContiguous;
      std::string dims = w.substr(open + 1, close - open - 1);
      for (size_t i = 0; i <= dims.size();) {
        size_t j = dims.find(',', i);
        if (j == std::string::npos) j = dims.size();
        const std::string one = dims.substr(i, j - i);
        if (one == "...") it.layout = Layout::kAlike;
        else it.dims.push_back(parse_dim(e, one));
        i = j + 1;
      }
      if (close + 1 < w.size()) {  // '?' and, for an output, the name that it goes with
        it.optional = true;
        for (size_t k = 0; k < e.items.size(); ++k)
          if (out && e.items[k].name == w.substr(close + 2)) it.only_with = static_cast<int>(k);
      }
      it.tensor = e.n_tensors++;
      TORCH_CHECK(e.n_tensors <= kMaxTensors, "binding: too many tensors in ", name);
      if (it.layout == Layout::kHeads) it.sym = sym_of(e, it.name + ".s", true);
      if (it.layout == Layout::kAlike) it.sym = sym_of(e, it.name + ".size", true);
      e.items.push_back(it);
    } else {
      int tensor = -1;
      for (const Item& it : e.items)
        if (it.tensor >= 0 && it.name == w) tensor = it.tensor;
      if (part == 2) {
        TORCH_CHECK(tensor >= 0, "binding: unknown result ", w, " in ", name);
        e.results.push_back(tensor);
      } else if (tensor >= 0) {
        e.cargs.push_back({CArg::kTensorPtr, tensor});
      } else if (w == "io") {
        e.cargs.push_back({CArg::kIoCode, 0});
      } else if (w == "%") {
        e.cargs.push_back({CArg::kSeqPtr, 0});
      } else {
        e.cargs.push_back({CArg::kSym, sym_of(e, w, false)});
      }
    }
  }
  TORCH_CHECK(part == 2 && e.cargs.size() < kMaxArgs, "binding: malformed description of ", name);
  return e;
}

const char* type_name(at::ScalarType t) { return c10::toString(t); }

// The state of one call.
struct Call {
  const Entry& e;
  std::array<int64_t, kMaxSyms> val{};
  std::array<bool, kMaxSyms> bound{};
  std::array<at::Tensor, kMaxTensors> t;
  std::array<PyObject*, kMaxTensors> given{};
  std::array<int, kMaxSeq> seq{};
  at::Device device{at::kCUDA, 0};
  bool has_device = false;
  at::ScalarType io = at::kBFloat16, any = at::kBFloat16;
  bool has_io = false, has_any = false;
  at::IntArrayRef alike;

  explicit Call(const Entry& entry) : e(entry) {}

  int64_t want(const Dim& d) const { return d.sym < 0 ? d.add : val[d.sym] / d.div + d.add; }

  // false with a Python error set
  bool shape_error(const Item& it, const at::Tensor& t) const {
    std::string s;
    for (const Dim& d : it.dims) {
      if (!s.empty()) s += ", ";
      s += d.sym < 0 || bound[d.sym] ? std::to_string(want(d)) : e.syms[d.sym];
    }
    std::string got;
    for (int64_t n : t.sizes()) got += (got.empty() ? "" : ", ") + std::to_string(n);
    PyErr_Format(PyExc_ValueError, "%s: expected shape [%s%s], got [%s]", it.name.c_str(), s.c_str(),
                 it.layout == Layout::kAlike ? ", ..." : "", got.c_str());
    return false;
  }

  at::ScalarType type_of(const Item& it) const {
    switch (it.type) {
      case Type::kBf16: return at::kBFloat16;
      case Type::kF32: return at::kFloat;
      case Type::kI32: return at::kInt;
      case Type::kIo: return io;
      default: return any;
    }
  }

  bool take(const Item& it, PyObject* o) {
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s: expected a tensor", it.name.c_str());
      return false;
    }
    t[it.tensor] = THPVariable_Unpack(o);
    given[it.tensor] = o;
    return check(it, t[it.tensor]);
  }

  bool check(const Item& it, const at::Tensor& t) {
    const at::ScalarType st = t.scalar_type();
    if (it.type == Type::kIo && !has_io) {
      if (st != at::kBFloat16 && st != at::kFloat) {
        PyErr_Format(PyExc_TypeError, "%s: expected BFloat16 or Float, got %s", it.name.c_str(), type_name(st));
        return false;
      }
      io = st;
      has_io = true;
    } else if (it.type == Type::kAny && !has_any) {
      any = st;
      has_any = true;
    }
    if (st != type_of(it)) {
      PyErr_Format(PyExc_TypeError, "%s: expected %s, got %s", it.name.c_str(), type_name(type_of(it)), type_name(st));
      return false;
    }
    if (!has_device) {
      if (!t.is_cuda()) {
        PyErr_Format(PyExc_ValueError, "%s: must be a CUDA tensor", it.name.c_str());
        return false;
      }
      device = t.device();
      has_device = true;
    } else if (t.device() != device) {
      PyErr_Format(PyExc_ValueError, "%s: expected a tensor on %s, got one on %s", it.name.c_str(), device.str().c_str(),
                   t.device().str().c_str());
      return false;
    }
    const at::IntArrayRef sizes = t.sizes();
    const size_t nd = it.dims.size();
    if (it.layout == Layout::kAlike ? sizes.size() < nd + 1 : sizes.size() != nd) return shape_error(it, t);
    for (size_t i = 0; i < nd; ++i) {
      const Dim& d = it.dims[i];
      if (d.sym >= 0 && !bound[d.sym]) {
        if (d.div != 1 || sizes[i] < d.add) return shape_error(it, t);
        if (sizes[i] > INT32_MAX) {
          PyErr_Format(PyExc_ValueError, "%s: a size of %lld does not fit 32 bits", it.name.c_str(),
                       static_cast<long long>(sizes[i]));
          return false;
        }
        val[d.sym] = sizes[i] - d.add;
        bound[d.sym] = true;
      } else if (sizes[i] != want(d)) {
        return shape_error(it, t);
      }
    }
    if (it.layout == Layout::kHeads) {
      const at::IntArrayRef st3 = t.strides();
      const int64_t T = sizes[0], H = sizes[1], D = sizes[2];
      if (st3[2] != 1 || (st3[1] != D && H > 1) || (st3[0] < H * D && T > 1)) {
        PyErr_Format(PyExc_ValueError, "%s: the heads of a token must be contiguous", it.name.c_str());
        return false;
      }
      val[it.sym] = T > 1 ? st3[0] : H * D;
      return true;
    }
    if (it.layout == Layout::kAlike) {
      if (alike.empty()) alike = sizes;
      if (sizes != alike) return shape_error(it, t);
      int64_t n = static_cast<int64_t>(t.element_size());
      for (size_t i = nd; i < sizes.size(); ++i) n *= sizes[i];
      val[it.sym] = n;
    }
    if (!t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s: must be contiguous", it.name.c_str());
      return false;
    }
    return true;
  }
};

using Fn = int (*)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                   int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                   int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                   int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t);

// All arguments of the C entry points are integers or pointers. In the calling conventions of the
// platforms that B200 comes with (x86-64 SysV, AArch64 AAPCS) each has a register or an 8-byte stack
// slot of its own, whose low half an int parameter reads, and the caller removes surplus ones: one
// signature of 40 words serves every entry point.
int call_words(void* fn, const std::array<int64_t, kMaxArgs>& a) {
  return reinterpret_cast<Fn>(fn)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12], a[13],
                                  a[14], a[15], a[16], a[17], a[18], a[19], a[20], a[21], a[22], a[23], a[24], a[25],
                                  a[26], a[27], a[28], a[29], a[30], a[31], a[32], a[33], a[34], a[35], a[36], a[37],
                                  a[38], a[39]);
}

PyObject* define(PyObject*, PyObject* args) {
  HANDLE_TH_ERRORS
  const char *name = nullptr, *spec = nullptr;
  if (!PyArg_ParseTuple(args, "ss", &name, &spec)) return nullptr;
  entries().push_back(parse(name, spec));
  return PyLong_FromSsize_t(static_cast<Py_ssize_t>(entries().size()) - 1);
  END_HANDLE_TH_ERRORS
}

PyObject* on_error(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_on_error, f);
  Py_RETURN_NONE;
}

// invoke(entry, address, *arguments, stream)
PyObject* invoke(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args < 3) {
    PyErr_SetString(PyExc_TypeError, "invoke(entry, address, *arguments, stream)");
    return nullptr;
  }
  const Py_ssize_t id = PyLong_AsSsize_t(args[0]);
  void* fn = PyLong_AsVoidPtr(args[1]);
  if (PyErr_Occurred()) return nullptr;
  if (id < 0 || id >= static_cast<Py_ssize_t>(entries().size()) || !fn) {
    PyErr_SetString(PyExc_ValueError, "no such entry");
    return nullptr;
  }
  const Entry& e = entries()[static_cast<size_t>(id)];
  if (n_args != static_cast<Py_ssize_t>(e.items.size()) + 3) {
    PyErr_Format(PyExc_TypeError, "%s: wrong number of arguments", e.name.c_str());
    return nullptr;
  }
  Call c(e);
  PyObject* const* a = args + 2;
  // scalars, inputs, then the outputs (whose sizes the others fix)
  for (size_t i = 0; i < e.items.size(); ++i) {
    const Item& it = e.items[i];
    if (it.kind == Kind::kInt) {
      PyObject* n = PyNumber_Index(a[i]);
      if (!n) return nullptr;
      const long v = PyLong_AsLong(n);
      Py_DECREF(n);
      if (v == -1 && PyErr_Occurred()) return nullptr;
      if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%s: %ld does not fit 32 bits", it.name.c_str(), v);
        return nullptr;
      }
      c.val[it.sym] = v;
      c.bound[it.sym] = true;
    } else if (it.kind == Kind::kFlag) {
      const int v = PyObject_IsTrue(a[i]);
      if (v < 0) return nullptr;
      c.val[it.sym] = v;
    } else if (it.kind == Kind::kSeq) {
      PyObject* s = PySequence_Fast(a[i], "expected a sequence of ints");
      if (!s) return nullptr;
      const Py_ssize_t n = PySequence_Fast_GET_SIZE(s);
      int64_t sum = 0;
      for (Py_ssize_t k = 0; k < n && k < kMaxSeq; ++k) {
        const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(s, k));
        if (v == -1 && PyErr_Occurred()) break;
        c.seq[static_cast<size_t>(k)] = static_cast<int>(std::max(-1L, std::min(v, 1L << 30)));
        sum += c.seq[static_cast<size_t>(k)];
      }
      Py_DECREF(s);
      if (PyErr_Occurred()) return nullptr;
      if (n > kMaxSeq) {
        PyErr_Format(PyExc_ValueError, "%s: at most %d entries", it.name.c_str(), kMaxSeq);
        return nullptr;
      }
      c.val[it.sym] = n;
      c.val[it.sum] = sum;
      c.bound[it.sym] = c.bound[it.sum] = true;
    }
  }
  for (size_t i = 0; i < e.items.size(); ++i) {
    const Item& it = e.items[i];
    if (it.kind != Kind::kTensor || (a[i] == Py_None && it.optional)) continue;
    if (!c.take(it, a[i])) return nullptr;
  }
  // the stream
  PyObject* so = a[e.items.size()];
  const c10::DeviceIndex dev = c.device.index();
  cudaStream_t stream = nullptr;
  if (so == Py_None) {
    stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  } else {
    PyObject* raw = PyLong_Check(so) ? Py_NewRef(so) : PyObject_GetAttrString(so, "cuda_stream");
    if (!raw) return nullptr;
    stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
    Py_DECREF(raw);
    if (PyErr_Occurred()) return nullptr;
  }
  // from here on the call's stream is the current one, whose pool the allocator takes from
  const c10::cuda::CUDAStream caller = c10::cuda::getCurrentCUDAStream(dev);
  const bool elsewhere = stream != caller.stream();
  c10::cuda::OptionalCUDAStreamGuard on_stream;
  if (elsewhere)
    on_stream.reset_stream(stream ? c10::cuda::getStreamFromExternal(stream, dev) : c10::cuda::getDefaultCUDAStream(dev));
  for (size_t i = 0; i < e.items.size(); ++i) {
    const Item& it = e.items[i];
    if (it.kind != Kind::kOut) continue;
    if (it.only_with >= 0 && a[it.only_with] == Py_None) {
      if (a[i] == Py_None) continue;
      PyErr_Format(PyExc_ValueError, "%s: there is no %s", it.name.c_str(), e.items[it.only_with].name.c_str());
      return nullptr;
    }
    if (a[i] != Py_None) {
      if (!c.take(it, a[i])) return nullptr;
      continue;
    }
    std::array<int64_t, 8> sizes{};
    for (size_t k = 0; k < it.dims.size(); ++k) sizes[k] = c.want(it.dims[k]);
    c.t[it.tensor] =
        at::detail::empty_cuda(at::IntArrayRef(sizes.data(), it.dims.size()), c.type_of(it), c.device, std::nullopt);
    if (it.layout == Layout::kHeads) c.val[it.sym] = sizes[1] * sizes[2];
    if (elsewhere) c10::cuda::CUDACachingAllocator::recordStream(c.t[it.tensor].storage().data_ptr(), caller);
  }
  for (size_t i = 0; i < e.items.size(); ++i) {
    const Item& it = e.items[i];
    if (it.kind != Kind::kWork) continue;
    std::array<int64_t, 8> a8{};
    for (size_t k = 0; k < it.sizes.size(); ++k) a8[k] = c.val[it.sizes[k]];
    void* size_fn = PyLong_AsVoidPtr(a[i - 1]);
    if (PyErr_Occurred()) return nullptr;
    const int64_t need = reinterpret_cast<int64_t (*)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                                                      int64_t)>(size_fn)(a8[0], a8[1], a8[2], a8[3], a8[4], a8[5],
                                                                         a8[6], a8[7]);
    if (a[i] == Py_None) {
      const int64_t bytes = std::max<int64_t>(need, 16);
      c.t[it.tensor] = at::detail::empty_cuda(at::IntArrayRef(&bytes, 1), at::kByte, c.device, std::nullopt);
    } else {
      if (!THPVariable_Check(a[i])) {
        PyErr_Format(PyExc_TypeError, "%s: expected a tensor", it.name.c_str());
        return nullptr;
      }
      c.t[it.tensor] = THPVariable_Unpack(a[i]);
      if (c.t[it.tensor].device() != c.device || !c.t[it.tensor].is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s: expected a contiguous tensor on %s", it.name.c_str(), c.device.str().c_str());
        return nullptr;
      }
    }
    c.val[it.sym] = static_cast<int64_t>(c.t[it.tensor].nbytes());
  }
  std::array<int64_t, kMaxArgs> words{};
  size_t n = 0;
  for (const CArg& x : e.cargs)
    words[n++] = x.kind == CArg::kTensorPtr
                     ? (c.t[x.index].defined() ? reinterpret_cast<int64_t>(c.t[x.index].data_ptr()) : 0)
                 : x.kind == CArg::kSym    ? c.val[x.index]
                 : x.kind == CArg::kIoCode ? (c.io == at::kFloat ? 1 : 0)
                                           : reinterpret_cast<int64_t>(c.seq.data());
  words[n++] = reinterpret_cast<int64_t>(stream);
  int status = 0;
  {
    const c10::cuda::CUDAGuard guard(dev);
    Py_BEGIN_ALLOW_THREADS;
    status = call_words(fn, words);
    Py_END_ALLOW_THREADS;
  }
  if (status != 0) {
    PyObject* r = g_on_error ? PyObject_CallFunction(g_on_error, "is", status, e.name.c_str()) : nullptr;
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", e.name.c_str(), status);
    return nullptr;
  }
  auto wrap = [&](int t) -> PyObject* {
    if (c.given[t]) return Py_NewRef(c.given[t]);
    if (!c.t[t].defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(c.t[t]);
  };
  if (e.results.empty()) Py_RETURN_NONE;
  if (e.results.size() == 1) return wrap(e.results[0]);
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(e.results.size()));
  for (size_t i = 0; out && i < e.results.size(); ++i) PyTuple_SET_ITEM(out, static_cast<Py_ssize_t>(i), wrap(e.results[i]));
  return out;
  END_HANDLE_TH_ERRORS
}

PyMethodDef g_methods[] = {
    {"define", define, METH_VARARGS, "define(name, description) -> entry"},
    {"on_error", on_error, METH_O, "on_error(callable(status, name))"},
    {"invoke", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(invoke)), METH_FASTCALL,
     "invoke(entry, address, *arguments, stream)"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", "Checks and marshals the arguments of short calls.", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
