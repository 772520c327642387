// Python binding of the decoder operators (include/q4_decoder.h, and
// include/q4_search.h in search_binding.h): checks of the tensors, their
// outputs and workspace from torch's allocator, the current stream, and the
// call.
//
// It is native because these operators are short: a decode step's norm runs
// for 2.5 us, and the same checks written in Python with a ctypes call take 13 us
// (this: 4.5 us, launch included).  Nothing is computed here.

#include "binding_helpers.h"
#include "search_binding.h"

namespace {

// kv_append(q, k, v, cache x 4, batch x 5, rope, interleaved, out)
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    want(n, 15);
    const at::Tensor &q = required(a[0], "q"), &k = required(a[1], "k"), &v = required(a[2], "v");
    const c10::Device dev = device_of(q, "q");
    const int dtype = type_code(q.scalar_type(), "q");
    TORCH_CHECK_VALUE(k.scalar_type() == q.scalar_type() && v.scalar_type() == q.scalar_type() && k.device() == dev &&
                          v.device() == dev,
                      "q, k and v must share a type and a device");
    TORCH_CHECK_VALUE(q.dim() == 2 && k.dim() == 2 && v.dim() == 2 && k.size(0) == q.size(0) && v.size(0) == q.size(0),
                      "q, k and v must be [rows, heads * head_dim] with the same rows");
    const int64_t rows = q.size(0), width = q.size(1);
    const q4_kv_cache c = cache_of(a + 3, dev);
    const q4_kv_batch b = batch_of(a + 7, rows, dev);
    const int64_t kv_width = static_cast<int64_t>(c.kv_heads) * c.head_dim;
    TORCH_CHECK_VALUE(width % c.head_dim == 0 && k.size(1) == kv_width && v.size(1) == kv_width, "need whole heads of ",
                      c.head_dim, ", and k and v [rows, ", kv_width, "]");
    // a row is contiguous; rows may lie apart (the stride of a single row says nothing)
    const auto stride = [&](const at::Tensor &t, const char *name) {
        TORCH_CHECK_VALUE(rows == 0 || t.size(1) <= 1 || t.stride(1) == 1, name, " must have contiguous rows");
        return rows <= 1 ? t.size(1) : t.stride(0);
    };
    const int64_t qs = stride(q, "q"), ks = stride(k, "k"), vs = stride(v, "v");
    const at::Tensor *rope = optional(a[12], "rope");
    const float *table = address<float>(rope, "rope", at::kFloat, dev);
    TORCH_CHECK_VALUE(!rope || (rope->dim() == 3 && rope->size(2) == 2), "rope must be [positions, rot / 2, 2]");
    const int64_t positions = rope ? rope->size(0) : 0, rot = rope ? 2 * rope->size(1) : 0;
    const int interleaved = PyObject_IsTrue(a[13]);
    at::Tensor out = output(a[14], "out", {rows, width}, at::kBFloat16, dev);
    const c10::hip::HIPGuard guard(dev.index());
    check(q4_kv_append(&c, &b, q.data_ptr(), qs, width / c.head_dim, k.data_ptr(), ks, v.data_ptr(), vs, dtype, table,
                       positions, rot, interleaved, out.data_ptr(),
                       c10::hip::getCurrentHIPStream(dev.index()).stream()),
          "q4_kv_append");
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// kv_attention(q, cache x 4, batch x 5, scale or None, window, out, dtype, workspace)
PyObject *kv_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    want(n, 15);
    const at::Tensor &q = required(a[0], "q");
    const c10::Device dev = device_of(q, "q");
    const void *src = address(&q, "q", at::kBFloat16, dev);
    const q4_kv_cache c = cache_of(a + 1, dev);
    TORCH_CHECK_VALUE(q.dim() == 2 && q.size(1) % c.head_dim == 0, "q must be [rows, heads * ", c.head_dim, "]");
    const q4_kv_batch b = batch_of(a + 5, q.size(0), dev);
    const int64_t heads = q.size(1) / c.head_dim;
    const float scale = a[10] == Py_None ? 1.0f / std::sqrt(static_cast<float>(c.head_dim)) : static_cast<float>(number(a[10]));
    const int64_t window = integer(a[11]);
    const at::ScalarType type = dtype_of(a[13]);
    const int out_code = type_code(type, "dtype");
    at::Tensor out = output(a[12], "out", q.sizes(), type, dev);
    const int64_t need = static_cast<int64_t>(q4_kv_attention_workspace(&c, &b, heads));
    const c10::hip::HIPGuard guard(dev.index());
    c10::DataPtr own;   // goes back to the allocator, for work on this stream after the call's
    void *ws = nullptr;
    int64_t ws_bytes = need;
    if (const at::Tensor *given = optional(a[14], "workspace")) {
        ws = address(given, "workspace", at::kByte, dev);
        ws_bytes = given->numel();
        TORCH_CHECK_VALUE(ws_bytes >= need, "workspace must hold ", need, " bytes");
    } else if (need) {
        own = c10::GetAllocator(dev.type())->allocate(need);
        ws = own.get();
    }
    check(q4_kv_attention(&c, &b, src, heads, scale, window, out.data_ptr(), out_code, ws, static_cast<size_t>(ws_bytes),
                          c10::hip::getCurrentHIPStream(dev.index()).stream()),
          "q4_kv_attention");
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// (address, rows) of a gate or modulation: [C], or [rows, C] with rows dividing M.
const float *shared_rows(const at::Tensor *t, const char *name, int64_t m, int64_t c, c10::Device dev, int64_t &rows) {
    rows = 0;
    if (!t) return nullptr;
    const float *p = address<float>(t, name, at::kFloat, dev);
    TORCH_CHECK_VALUE((t->dim() == 1 || t->dim() == 2) && t->size(-1) == c, name, " must be [", c, "] or [rows, ", c, "]");
    rows = t->dim() == 2 ? t->size(0) : 1;
    TORCH_CHECK_VALUE(rows >= 1 && m % rows == 0, "the rows of ", name, " must divide the ", m, " rows of the residual");
    return p;
}

// add_rmsnorm(residual, weight, y, post_weight, gate, scale, modulation, eps, dtype, residual_out, out)
PyObject *add_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    want(n, 11);
    const at::Tensor &res = required(a[0], "residual");
    const c10::Device dev = device_of(res, "residual");
    const at::ScalarType res_type = res.scalar_type();
    const int res_code = type_code(res_type, "residual");
    const void *src = address(&res, "residual", res_type, dev);
    TORCH_CHECK_VALUE(res.dim() == 2, "residual must be [M, C]");
    const int64_t m = res.size(0), c = res.size(1);
    const at::Tensor &w = required(a[1], "weight");
    const float *weight = address<float>(&w, "weight", at::kFloat, dev);
    has_shape(&w, "weight", {c});
    const at::Tensor *y = optional(a[2], "y"), *pw = optional(a[3], "post_weight"), *gate = optional(a[4], "gate"),
                     *mod = optional(a[6], "modulation");
    const float *post = address<float>(pw, "post_weight", at::kFloat, dev);
    has_shape(pw, "post_weight", {c});
    int64_t gate_rows, mod_rows;
    const float *at_gate = shared_rows(gate, "gate", m, c, dev, gate_rows);
    const float *at_mod = shared_rows(mod, "modulation", m, c, dev, mod_rows);
    const float scale = static_cast<float>(number(a[5])), eps = static_cast<float>(number(a[7]));
    const at::ScalarType type = dtype_of(a[8]);
    const int x_code = type_code(type, "dtype");
    const void *at_y = nullptr;
    int y_code = Q4_F32;
    at::Tensor r;
    if (y) {
        y_code = type_code(y->scalar_type(), "y");
        at_y = address(y, "y", y->scalar_type(), dev);
        has_shape(y, "y", {m, c});
        r = output(a[9], "residual_out", {m, c}, res_type, dev);
    } else {
        TORCH_CHECK_VALUE(!pw && !gate && a[9] == Py_None, "post_weight, gate and residual_out need y");
    }
    at::Tensor x = output(a[10], "out", {m, c}, type, dev);
    const c10::hip::HIPGuard guard(dev.index());
    check(q4_add_rmsnorm(src, res_code, at_y, y_code, m, c, weight, post, at_gate, gate_rows, scale, at_mod, mod_rows, eps,
                         r.defined() ? r.data_ptr() : nullptr, x.data_ptr(), x_code,
                         c10::hip::getCurrentHIPStream(dev.index()).stream()),
          "q4_add_rmsnorm");
    PyObject *first;
    if (y) {
        first = THPVariable_Wrap(std::move(r));
    } else {
        first = a[0];
        Py_INCREF(first);
    }
    PyObject *second = THPVariable_Wrap(std::move(x));
    PyObject *both = PyTuple_Pack(2, first, second);
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
    END_HANDLE_TH_ERRORS
}

// logits_adjust(logits, history, cu_history, prompt_lengths, repetition, frequency, presence, bias_ids, bias, cu_bias,
//               mask, out)
PyObject *logits_adjust(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    want(n, 12);
    const at::Tensor &z = required(a[0], "logits");
    const c10::Device dev = device_of(z, "logits");
    const float *src = address<float>(&z, "logits", at::kFloat, dev);
    TORCH_CHECK_VALUE(z.dim() == 2, "logits must be [M, V]");
    const int64_t m = z.size(0), v = z.size(1);
    const at::Tensor *history = optional(a[1], "history"), *cu_history = optional(a[2], "cu_history"),
                     *ids = optional(a[7], "bias_ids"), *bias = optional(a[8], "bias"), *cu_bias = optional(a[9], "cu_bias"),
                     *mask = optional(a[10], "mask");
    TORCH_CHECK_VALUE(!history == !cu_history, "history and cu_history go together");
    TORCH_CHECK_VALUE(!ids == !bias && !ids == !cu_bias, "bias, bias_ids and cu_bias go together");
    const auto list = [&](const at::Tensor *t, const char *name, at::ScalarType type, int64_t size) {
        void *p = address(t, name, type, dev);
        TORCH_CHECK_VALUE(!t || t->dim() == 1, name, " must be one-dimensional");
        if (size >= 0) has_shape(t, name, {size});
        return p;
    };
    const auto *at_history = static_cast<const int32_t *>(list(history, "history", at::kInt, -1));
    const auto *at_cu = static_cast<const int32_t *>(list(cu_history, "cu_history", at::kInt, m + 1));
    const auto *prompt = static_cast<const int32_t *>(list(optional(a[3], "prompt_lengths"), "prompt_lengths", at::kInt, m));
    const auto *rho = static_cast<const float *>(list(optional(a[4], "repetition"), "repetition", at::kFloat, m));
    const auto *frequency = static_cast<const float *>(list(optional(a[5], "frequency"), "frequency", at::kFloat, m));
    const auto *presence = static_cast<const float *>(list(optional(a[6], "presence"), "presence", at::kFloat, m));
    const auto *at_ids = static_cast<const int32_t *>(list(ids, "bias_ids", at::kInt, -1));
    const auto *at_bias = static_cast<const float *>(list(bias, "bias", at::kFloat, ids ? ids->numel() : -1));
    const auto *at_cub = static_cast<const int32_t *>(list(cu_bias, "cu_bias", at::kInt, m + 1));
    const auto *at_mask = address<const uint32_t>(mask, "mask", at::kInt, dev);
    has_shape(mask, "mask", {m, (v + 31) / 32});
    at::Tensor out = output(a[11], "out", {m, v}, at::kFloat, dev);
    const c10::hip::HIPGuard guard(dev.index());
    check(q4_logits_adjust(src, m, v, at_history, at_cu, history ? history->numel() : 0, prompt, rho, frequency, presence,
                           at_ids, at_bias, at_cub, ids ? ids->numel() : 0, at_mask, static_cast<float *>(out.data_ptr()),
                           c10::hip::getCurrentHIPStream(dev.index()).stream()),
          "q4_logits_adjust");
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *f) {
    Py_INCREF(f);
    Py_XDECREF(g_error);
    g_error = f;
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"kv_append", fast(kv_append), METH_FASTCALL, nullptr},
                         {"kv_attention", fast(kv_attention), METH_FASTCALL, nullptr},
                         {"add_rmsnorm", fast(add_rmsnorm), METH_FASTCALL, nullptr},
                         {"logits_adjust", fast(logits_adjust), METH_FASTCALL, nullptr},
                         {"beam_select", fast(beam_select), METH_FASTCALL, nullptr},
                         {"beam_advance", fast(beam_advance), METH_FASTCALL, nullptr},
                         {"kv_fork", fast(kv_fork), METH_FASTCALL, nullptr},
                         {"kv_compact", fast(kv_compact), METH_FASTCALL, nullptr},
                         {"kv_copy_blocks", fast(kv_copy_blocks), METH_FASTCALL, nullptr},
                         {"kv_summarize", fast(kv_summarize), METH_FASTCALL, nullptr},
                         {"kv_select", fast(kv_select), METH_FASTCALL, nullptr},
                         {"kv_attention_blocks", fast(kv_attention_blocks), METH_FASTCALL, nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q4decoder", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__q4decoder() { return PyModule_Create(&module); }
