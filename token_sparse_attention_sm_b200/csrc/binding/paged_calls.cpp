// paged_calls.cpp -- the plain form of the paged calls without Python between
// the checks: a decode step's kernels take a few microseconds, and checking a
// dozen tensors and allocating the results from Python took ten more.
//
// Each function takes the caller's tensors, the stream's workspace (its buffer
// is read here, and no other thread can replace it before the launches: the
// global lock is held throughout) and the stream, and returns the results when
// every argument is as the C entry point wants it; otherwise it returns None,
// having done nothing, and paged.py goes through the arguments itself and says
// what is wrong.  The C entry points
// are handed over by address (bind), so this module links against nothing of
// the library's; a status other than OK comes back as an int.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/extension.h>

#include "sparse_decode.h"

namespace {

using Plan = decltype(&sparse_paged_plan);
using Append = decltype(&sparse_paged_append);
using Attn = decltype(&sparse_paged_attn);
using Size = decltype(&sparse_paged_workspace_size);
Plan g_plan;
Append g_append;
Attn g_attn;
Size g_size;

py::object none() { return py::none(); }

// the buffer a paged.py workspace has now
at::Tensor buffer(const py::object &ws) {
  static PyObject *name = PyUnicode_InternFromString("buf");
  const auto buf = py::reinterpret_steal<py::object>(PyObject_GetAttr(ws.ptr(), name));
  if (!buf) throw py::error_already_set();
  return py::cast<at::Tensor>(buf);
}

// a dense int32 tensor of this device
bool ints(const at::Tensor &t, const at::Device &dev, int64_t dims) {
  return t.device() == dev && t.scalar_type() == at::kInt && t.dim() == dims && t.is_contiguous();
}

int dtype_code(const at::Tensor &t) {
  return t.scalar_type() == at::kFloat ? 0 : t.scalar_type() == at::kBFloat16 ? 1 : -1;
}

bool fits(int64_t x) { return x >= 0 && x <= INT32_MAX; }

// elements between the token rows of t [T, heads, d], -1 if it is not plain
int64_t row_stride(const at::Tensor &t, const at::Device &dev, int64_t heads, int64_t d) {
  if (t.device() != dev || t.dim() != 3 || t.size(1) != heads || t.size(2) != d ||
      t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
    return -1;
  if (t.size(0) < 2) return heads * d;
  const int64_t s = t.stride(0);
  return s >= heads * d && s * t.element_size() % 16 == 0 ? s : -1;
}

bool caches(const at::Tensor &K, const at::Tensor &V) {
  return K.is_cuda() && K.dim() == 4 && V.device() == K.device() && V.sizes() == K.sizes() &&
         V.scalar_type() == K.scalar_type() && K.is_contiguous() && V.is_contiguous() &&
         dtype_code(K) >= 0 && fits(K.size(0)) && fits(K.size(1)) && fits(K.size(2)) &&
         fits(K.size(3));
}


py::object attn(const py::object &ws, int64_t stream, const at::Tensor &q, const at::Tensor &K,
                const at::Tensor &V, const at::Tensor &table, const at::Tensor &q_start,
                const at::Tensor &kv_lens, int64_t window, int64_t sinks, int64_t max_new,
                bool want_lse, const c10::optional<at::Tensor> &out_given,
                const c10::optional<at::Tensor> &lse_given) {
  if (!caches(K, V) || q.scalar_type() != K.scalar_type() || q.dim() != 3) return none();
  const at::Device dev = K.device();
  const at::Tensor buf = buffer(ws);
  const int64_t T = q.size(0), Hq = q.size(1), d = K.size(3);
  const int64_t qs = row_stride(q, dev, Hq, d);
  if (qs < 0 || T < 1 || !fits(T) || !fits(Hq) || !ints(table, dev, 2) || !ints(q_start, dev, 1) ||
      !ints(kv_lens, dev, 1) || !fits(window) || !fits(sinks) || !fits(max_new) ||
      !fits(table.size(1)))
    return none();
  const int64_t B = table.size(0);
  if (q_start.size(0) != B + 1 || kv_lens.size(0) != B || !fits(B)) return none();
  const sparse_paged_shape_t sh = {(int32_t)B,         (int32_t)T,         (int32_t)Hq,
                                   (int32_t)K.size(1), (int32_t)d,         dtype_code(K),
                                   (int32_t)K.size(2), (int32_t)K.size(0), (int32_t)table.size(1),
                                   (int32_t)max_new};
  size_t need = 0;
  if (g_size(&sh, &need) != SPARSE_OK || buf.device() != dev || need > (size_t)buf.numel())
    return none();
  if (out_given && (out_given->device() != dev || out_given->scalar_type() != q.scalar_type() ||
                    out_given->sizes() != q.sizes() || !out_given->is_contiguous()))
    return none();
  if (lse_given && (lse_given->device() != dev || lse_given->scalar_type() != at::kFloat ||
                    lse_given->sizes() != q.sizes().slice(0, 2) || !lse_given->is_contiguous()))
    return none();
  want_lse = want_lse || lse_given;
  const at::Tensor out = out_given ? *out_given : at::empty({T, Hq, d}, q.options());
  at::Tensor lse;
  if (want_lse) lse = lse_given ? *lse_given : at::empty({T, Hq}, q.options().dtype(at::kFloat));
  const sparse_status_t rc =
      g_attn(&sh, q.data_ptr(), qs, K.data_ptr(), V.data_ptr(), table.data_ptr<int32_t>(),
             q_start.data_ptr<int32_t>(), kv_lens.data_ptr<int32_t>(), (int32_t)window,
             (int32_t)sinks, out.data_ptr(), want_lse ? lse.data_ptr<float>() : nullptr,
             buf.data_ptr(), (size_t)buf.numel(), reinterpret_cast<void *>(stream));
  if (rc != SPARSE_OK) return py::int_((int)rc);
  return py::make_tuple(out, want_lse ? py::cast(lse) : none());
}

py::object append(const py::object &ws, int64_t stream, const at::Tensor &K, const at::Tensor &V,
                  const at::Tensor &k_new, const at::Tensor &v_new, const at::Tensor &slots) {
  if (!caches(K, V) || k_new.scalar_type() != K.scalar_type() ||
      v_new.scalar_type() != K.scalar_type())
    return none();
  const at::Device dev = K.device();
  const at::Tensor buf = buffer(ws);
  const int64_t T = k_new.dim() == 3 ? k_new.size(0) : 0, Hkv = K.size(1), d = K.size(3);
  const int64_t ks = row_stride(k_new, dev, Hkv, d), vs = row_stride(v_new, dev, Hkv, d);
  if (ks < 0 || vs < 0 || T < 1 || !fits(T) || v_new.size(0) != T || !ints(slots, dev, 1) ||
      slots.size(0) != T || buf.device() != dev)
    return none();
  const sparse_paged_shape_t sh = {1,
                                   (int32_t)T,
                                   (int32_t)Hkv,
                                   (int32_t)Hkv,
                                   (int32_t)d,
                                   dtype_code(K),
                                   (int32_t)K.size(2),
                                   (int32_t)K.size(0),
                                   1,
                                   0};
  return py::int_((int)g_append(&sh, K.data_ptr(), V.data_ptr(), k_new.data_ptr(), ks,
                                v_new.data_ptr(), vs, slots.data_ptr<int32_t>(), buf.data_ptr(),
                                (size_t)buf.numel(), reinterpret_cast<void *>(stream)));
}

// (kv_lens, q_start, positions, slots, free_left): the given ones or new ones
py::object plan(const py::object &ws, int64_t stream, const at::Tensor &new_lens,
                const at::Tensor &lens, const at::Tensor &table, const at::Tensor &free_pages,
                const at::Tensor &free_count, int64_t page, int64_t T, int64_t pages,
                const c10::optional<at::Tensor> &kv_given,
                const c10::optional<at::Tensor> &left_given) {
  const at::Device dev = new_lens.device();
  const at::Tensor buf = buffer(ws);
  if (!dev.is_cuda() || !ints(new_lens, dev, 1) || !ints(lens, dev, 1) || !ints(table, dev, 2) ||
      !ints(free_pages, dev, 1) || !ints(free_count, dev, 1) || !fits(page) || !fits(T) ||
      !fits(pages) || buf.device() != dev)
    return none();
  const int64_t B = new_lens.size(0), F = free_pages.size(0);
  if (B < 1 || !fits(B) || !fits(F) || lens.size(0) != B || table.size(0) != B ||
      free_count.size(0) != 1 || !fits(table.size(1)))
    return none();
  if (kv_given && (!ints(*kv_given, dev, 1) || kv_given->size(0) != B)) return none();
  if (left_given && (!ints(*left_given, dev, 1) || left_given->size(0) != 1)) return none();
  const sparse_paged_shape_t sh = {(int32_t)B,    (int32_t)T,     1, 1, 64, 0, (int32_t)page,
                                   (int32_t)pages, (int32_t)table.size(1), 0};
  size_t need = 0;
  if (g_size(&sh, &need) != SPARSE_OK) return none();  // nothing is allocated for it
  // one allocation: positions, slots, q_start, then what was not given; the
  // results are tensors of their own on its storage (a view op costs 0.6 us)
  const int64_t n_kv = kv_given ? 0 : B, n_left = left_given ? 0 : 1;
  const at::Tensor all = at::empty({2 * T + B + 1 + n_kv + n_left}, new_lens.options());
  int64_t at_ = 0;
  auto take = [&](int64_t n) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                     all.dtype());
    impl->set_storage_offset(at_);
    impl->set_sizes_contiguous({n});
    at_ += n;
    return at::Tensor(std::move(impl));
  };
  const at::Tensor positions = take(T), slots = take(T), q_start = take(B + 1);
  const at::Tensor kv = kv_given ? *kv_given : take(B);
  const at::Tensor left = left_given ? *left_given : take(1);
  const sparse_status_t rc = g_plan(
      &sh, new_lens.data_ptr<int32_t>(), lens.data_ptr<int32_t>(), table.data_ptr<int32_t>(),
      free_pages.data_ptr<int32_t>(), (int32_t)F, free_count.data_ptr<int32_t>(),
      kv.data_ptr<int32_t>(), q_start.data_ptr<int32_t>(), positions.data_ptr<int32_t>(),
      slots.data_ptr<int32_t>(), left.data_ptr<int32_t>(), buf.data_ptr(), (size_t)buf.numel(),
      reinterpret_cast<void *>(stream));
  if (rc != SPARSE_OK) return py::int_((int)rc);
  return py::make_tuple(kv, q_start, positions, slots, left);
}

void bind(int64_t size, int64_t plan_fn, int64_t append_fn, int64_t attn_fn) {
  g_size = reinterpret_cast<Size>(size);
  g_plan = reinterpret_cast<Plan>(plan_fn);
  g_append = reinterpret_cast<Append>(append_fn);
  g_attn = reinterpret_cast<Attn>(attn_fn);
}

}  // namespace

PYBIND11_MODULE(_paged_calls, m) {
  m.attr("built_for") = PAGED_CALLS_TAG;  // read from the file before it is loaded
  m.def("bind", &bind);
  m.def("plan", &plan);
  m.def("append", &append);
  m.def("attn", &attn);
}
