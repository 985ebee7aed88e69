// row_binding.cpp -- regular calls of the row and vocabulary operators without
// Python between them and the C ABI.
//
// A call of a small size is paced by the host: the binding's checks, tensors
// and, under autograd, Functions in Python took 10 us of a 14 us distillation
// step and as long again in its backward.  The functions here make the same
// checks, allocate the same tensors and make the same C calls; they take calls
// whose outputs and workspaces are theirs to allocate and whose arguments are
// all in order.  To any other they return None, and the Python code takes the
// call, or says what is wrong with it.
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <optional>
#include <string>
#include <tuple>

#include "../../include/lsd_radix_sort.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// The C entry points of the library that Python has loaded.
struct Library {
    decltype(&segmented_row_topk_workspace_size) topk_size = nullptr;
    decltype(&segmented_row_topk) topk = nullptr;
    decltype(&topk_distill_workspace_size) distill_size = nullptr;
    decltype(&topk_distill_forward) distill_forward = nullptr;
    decltype(&topk_distill_backward) distill_backward = nullptr;
    decltype(&topk_distill_step) distill_step = nullptr;
    decltype(&expert_balance_step_workspace_size) balance_size = nullptr;
    decltype(&expert_balance_step) balance_step = nullptr;
    decltype(&expert_balance) balance = nullptr;
    decltype(&embedding_forward) embed_forward = nullptr;
    decltype(&embedding_backward_workspace_size) embed_size = nullptr;
    decltype(&embedding_backward) embed_backward = nullptr;
    decltype(&token_logprobs_workspace_size) logprobs_size = nullptr;
    decltype(&token_logprobs_forward) logprobs_forward = nullptr;
    decltype(&token_logprobs_topk) logprobs_topk = nullptr;
    decltype(&token_logprobs_backward) logprobs_backward = nullptr;
    decltype(&token_logprobs_step) logprobs_step = nullptr;
} lib;

template <typename F> void set(F &f, const py::dict &d, const char *name) {
    f = reinterpret_cast<F>(py::cast<uintptr_t>(d[name]));
}
void bind(const py::dict &d) {
    set(lib.topk_size, d, "segmented_row_topk_workspace_size");
    set(lib.topk, d, "segmented_row_topk");
    set(lib.distill_size, d, "topk_distill_workspace_size");
    set(lib.distill_forward, d, "topk_distill_forward");
    set(lib.distill_backward, d, "topk_distill_backward");
    set(lib.distill_step, d, "topk_distill_step");
    set(lib.balance_size, d, "expert_balance_step_workspace_size");
    set(lib.balance_step, d, "expert_balance_step");
    set(lib.balance, d, "expert_balance");
    set(lib.embed_forward, d, "embedding_forward");
    set(lib.embed_size, d, "embedding_backward_workspace_size");
    set(lib.embed_backward, d, "embedding_backward");
    set(lib.logprobs_size, d, "token_logprobs_workspace_size");
    set(lib.logprobs_forward, d, "token_logprobs_forward");
    set(lib.logprobs_topk, d, "token_logprobs_topk");
    set(lib.logprobs_backward, d, "token_logprobs_backward");
    set(lib.logprobs_step, d, "token_logprobs_step");
}

int type_code(at::ScalarType t) {
    switch (t) {
    case at::kHalf: return LRS_DTYPE_FP16;
    case at::kBFloat16: return LRS_DTYPE_BF16;
    case at::kFloat: return LRS_DTYPE_FP32;
    default: return -1;
    }
}
bool rows_contiguous(const Tensor &t) { return t.dim() == 2 && (t.stride(1) == 1 || t.size(1) <= 1); }
bool matrix(const Tensor &t, int &code) {
    code = t.defined() && t.is_cuda() ? type_code(t.scalar_type()) : -1;
    return code >= 0 && rows_contiguous(t);
}
bool ids(const Tensor &t, const Tensor &like, int &bytes) {
    if (!t.defined() || t.device() != like.device() || !rows_contiguous(t) || t.size(0) != like.size(0)) return false;
    bytes = t.scalar_type() == at::kLong ? 8 : t.scalar_type() == at::kInt ? 4 : 0;
    return bytes != 0;
}
bool by_row(const Tensor &t, const Tensor &like) {  // or none
    return !t.defined() || (t.device() == like.device() && t.scalar_type() == at::kFloat && t.dim() == 1 &&
                            t.size(0) == like.size(0) && t.is_contiguous());
}
bool mask_ok(const Tensor &t, const Tensor &like) {
    return !t.defined() || (t.device() == like.device() && (t.scalar_type() == at::kBool || t.scalar_type() == at::kByte) &&
                            t.dim() == 1 && t.size(0) == like.size(0) && t.is_contiguous());
}
// A Python argument as a tensor: false if it is none; None gives no tensor where it may.
bool take(py::handle h, Tensor &t, bool optional = false) {
    if (optional && h.is_none()) return true;
    if (!THPVariable_Check(h.ptr())) return false;
    t = THPVariable_Unpack(h.ptr());
    return true;
}
template <typename T = void> T *pointer(const Tensor &t) {
    return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr;
}
void *stream_of(const Tensor &t) { return c10::hip::getCurrentHIPStream(t.get_device()).stream(); }
Tensor make(const Tensor &like, at::IntArrayRef shape, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type));
}
Tensor like_rows(const Tensor &t) { return at::empty(t.sizes(), t.options()); }

// Optional tensors as autograd's Functions take them.
using Maybe = std::optional<Tensor>;
Maybe maybe(const Tensor &t) { return t.defined() ? Maybe(t) : Maybe(); }
Tensor given(const Maybe &t) { return t.has_value() ? *t : Tensor(); }

// ------------------------------------------------------------------- top k

py::object topk(py::handle matrix_in, int64_t k, bool descending) {
    Tensor x;
    int code;
    if (!take(matrix_in, x) || !matrix(x, code) || k < 0 || k > x.size(1)) return py::none();
    const int64_t rows = x.size(0), n = x.size(1);
    const Tensor values = make(x, {rows, k}, x.scalar_type()), indices = make(x, {rows, k}, at::kLong);
    const size_t need = lib.topk_size(rows, n, k, code, nullptr);
    const Tensor workspace = need ? make(x, {static_cast<int64_t>(need)}, at::kByte) : Tensor();
    if (lib.topk(pointer(x), x.stride(0), pointer(values), pointer<int64_t>(indices), rows, n, k, code, descending,
                 pointer(workspace), need, stream_of(x), nullptr) != LRS_OK)
        return py::none();
    return py::make_tuple(values, indices);
}

// -------------------------------------------- distillation from top logits

struct Distill {
    Tensor logits, values, indices, lse, weights;
    lrs_distill d{};
    bool take_all(py::handle s, py::handle v, py::handle i, py::handle l, py::handle w) {
        return take(s, logits) && take(v, values) && take(i, indices) && take(l, lse, true) && take(w, weights, true);
    }
    // False if an argument is not as it should be.
    bool fill(double temperature) {
        int code, teacher, bytes;
        if (!matrix(logits, code) || !matrix(values, teacher) || values.device() != logits.device() ||
            !ids(indices, logits, bytes) || values.size(0) != logits.size(0) || values.size(1) != indices.size(1) ||
            !by_row(lse, logits) || !by_row(weights, logits))
            return false;
        d = lrs_distill{pointer(logits), logits.stride(0), pointer(values), values.stride(0), pointer(indices),
                        indices.stride(0), pointer<float>(lse), pointer<float>(weights), logits.size(0), logits.size(1),
                        values.size(1), code, teacher, bytes, temperature};
        return true;
    }
    Tensor workspace() const {
        const size_t need = lib.distill_size(d.rows, d.n, d.k, d.dtype, nullptr);
        return make(values, {std::max<int64_t>(1, static_cast<int64_t>(need))}, at::kByte);
    }
    int forward(Tensor &loss, const Tensor &row_loss, Tensor &stats) const {
        const Tensor ws = workspace();
        loss = make(values, {}, at::kFloat);
        stats = make(values, {d.rows, d.k + 3}, at::kFloat);
        return lib.distill_forward(&d, pointer<float>(loss), pointer<float>(row_loss), pointer<float>(stats), pointer(ws),
                                   ws.numel(), stream_of(logits), nullptr);
    }
};

py::object distill_step(py::handle logits, py::handle values, py::handle indices, double temperature, py::handle lse,
                        py::handle weights) {
    Distill c;
    if (!c.take_all(logits, values, indices, lse, weights) || !c.fill(temperature)) return py::none();
    const Tensor ws = c.workspace(), loss = make(c.values, {}, at::kFloat), row_loss = make(c.values, {c.d.rows}, at::kFloat);
    const Tensor grad = like_rows(c.logits);
    if (lib.distill_step(&c.d, pointer<float>(loss), pointer<float>(row_loss), pointer(grad), grad.stride(0), pointer(ws),
                         ws.numel(), stream_of(grad), nullptr) != LRS_OK)
        return py::none();
    return py::make_tuple(loss, row_loss, grad);
}

py::object distill_forward(py::handle logits, py::handle values, py::handle indices, double temperature, py::handle lse,
                           py::handle weights) {
    Distill c;
    if (!c.take_all(logits, values, indices, lse, weights) || !c.fill(temperature)) return py::none();
    const Tensor row_loss = make(c.values, {c.d.rows}, at::kFloat);
    Tensor loss, stats;
    if (c.forward(loss, row_loss, stats) != LRS_OK) return py::none();
    return py::make_tuple(loss, row_loss, stats);
}

// The gradient of a loss that is not to be differentiated again.
Tensor final_gradient(const Tensor &grad, const char *name) {
    if (!at::GradMode::is_enabled()) return grad;
    auto error = std::make_shared<torch::autograd::DelayedError>(std::string(name) + " cannot be differentiated twice", 1);
    return (*error)({grad.detach().requires_grad_(true)})[0];
}
[[noreturn]] void failed(const char *name, int status) {
    throw std::runtime_error(std::string(name) + ": " + std::to_string(status));
}

struct DistillLoss : torch::autograd::Function<DistillLoss> {
    static Tensor forward(AutogradContext *ctx, const Tensor &logits, const Tensor &values, const Tensor &indices,
                          double temperature, const Maybe &lse, const Maybe &weights) {
        Distill c{logits, values, indices, given(lse), given(weights)};
        Tensor loss, stats;
        c.fill(temperature);
        const int status = c.forward(loss, Tensor(), stats);
        if (status != LRS_OK) failed("topk_distill_forward", status);
        ctx->save_for_backward({logits, values, indices, stats, c.lse, c.weights});
        ctx->saved_data["temperature"] = temperature;
        return loss;
    }
    static variable_list backward(AutogradContext *ctx, const variable_list &up) {
        const auto saved = ctx->get_saved_variables();
        Distill c{saved[0].detach(), saved[1], saved[2], saved[4], saved[5]};
        const Tensor scale = up[0].detach();
        if (!c.fill(ctx->saved_data["temperature"].toDouble()) || scale.scalar_type() != at::kFloat ||
            scale.numel() != 1)
            failed("topk_distill_backward", LRS_ERR_SIZE);
        const Tensor grad = like_rows(c.logits);
        const int status = lib.distill_backward(&c.d, pointer<float>(saved[3]), pointer<float>(scale), pointer(grad),
                                                grad.stride(0), stream_of(grad), nullptr);
        if (status != LRS_OK) failed("topk_distill_backward", status);
        return {final_gradient(grad, "topk_distill_loss"), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

py::object distill_loss(py::handle logits, py::handle values, py::handle indices, double temperature, py::handle lse,
                        py::handle weights) {
    Distill c;
    if (!c.take_all(logits, values, indices, lse, weights) || !c.fill(temperature) || c.d.k < 1 || c.d.k > LRS_MAX_TOPK ||
        !(temperature > 0) || !std::isfinite(temperature) || !std::isfinite(static_cast<float>(1.44269504088896340736 / temperature)) ||
        c.d.n > LRS_MAX_ROW_LEN || c.d.rows >= (int64_t(1) << 40) / std::max<int64_t>(1, c.d.n))
        return py::none();
    return py::cast(DistillLoss::apply(c.logits, c.values, c.indices, temperature, maybe(c.lse), maybe(c.weights)));
}

// ------------------------------------------ expert counts and balance loss

struct Balance {
    Tensor logits, indices, mask;
    int code = 0, bytes = 0;
    bool take_all(py::handle x, py::handle i, py::handle m) {
        return take(x, logits) && take(i, indices) && take(m, mask, true);
    }
    bool fill() { return matrix(logits, code) && ids(indices, logits, bytes) && mask_ok(mask, logits); }
    int step(double balance, double z, int score, Tensor &loss, Tensor &counts, const Tensor &kept, const Tensor &grad) const {
        const int64_t rows = logits.size(0), experts = logits.size(1), k = indices.size(1);
        const size_t need = lib.balance_size(rows, k, experts, nullptr);
        const Tensor ws = make(indices, {std::max<int64_t>(1, static_cast<int64_t>(need))}, at::kByte);
        loss = make(indices, {}, at::kFloat);
        counts = make(indices, {experts}, at::kInt);
        return lib.balance_step(pointer(logits), logits.stride(0), pointer(indices), indices.stride(0), bytes,
                                pointer<uint8_t>(mask), rows, k, experts, code, score, static_cast<float>(balance),
                                static_cast<float>(z), pointer<int32_t>(counts), pointer<int32_t>(kept), pointer<float>(loss),
                                pointer(grad), grad.defined() ? grad.stride(0) : 0, pointer(ws), need, stream_of(logits),
                                nullptr);
    }
};

py::object balance_step(py::handle logits, py::handle indices, double balance, double z, int score, py::handle mask,
                        bool want_kept, bool want_grad) {
    Balance c;
    if (!c.take_all(logits, indices, mask) || !c.fill()) return py::none();
    const Tensor kept = want_kept ? make(c.indices, {1}, at::kInt) : Tensor();
    const Tensor grad = want_grad ? like_rows(c.logits) : Tensor();
    Tensor loss, counts;
    if (c.step(balance, z, score, loss, counts, kept, grad) != LRS_OK) return py::none();
    return py::make_tuple(loss, counts, kept.defined() ? py::cast(kept) : py::none(),
                          grad.defined() ? py::cast(grad) : py::none());
}

struct BalanceLoss : torch::autograd::Function<BalanceLoss> {
    static variable_list forward(AutogradContext *ctx, const Tensor &logits, const Tensor &indices, double balance, double z,
                                 int64_t score, const Maybe &mask) {
        Balance c{logits, indices, given(mask)};
        c.fill();
        const Tensor kept = make(indices, {1}, at::kInt);
        Tensor loss, counts;
        const int status = c.step(balance, z, static_cast<int>(score), loss, counts, kept, Tensor());
        if (status != LRS_OK) failed("expert_balance_step", status);
        ctx->save_for_backward({logits, counts, kept, c.mask});
        ctx->saved_data["balance"] = balance;
        ctx->saved_data["z"] = z;
        ctx->saved_data["score"] = score;
        ctx->mark_non_differentiable({counts});
        return {loss, counts};
    }
    static variable_list backward(AutogradContext *ctx, const variable_list &up) {
        const auto saved = ctx->get_saved_variables();
        const Tensor logits = saved[0].detach(), counts = saved[1], kept = saved[2], mask = saved[3];
        const Tensor scale = up[0].detach();
        int code;
        if (!matrix(logits, code) || scale.scalar_type() != at::kFloat || scale.numel() != 1)
            failed("expert_balance", LRS_ERR_SIZE);
        const Tensor grad = like_rows(logits);
        const int status = lib.balance(pointer(logits), logits.stride(0), pointer<int32_t>(counts), pointer<int32_t>(kept),
                                       pointer<uint8_t>(mask), logits.size(0), logits.size(1), code,
                                       static_cast<int>(ctx->saved_data["score"].toInt()),
                                       static_cast<float>(ctx->saved_data["balance"].toDouble()),
                                       static_cast<float>(ctx->saved_data["z"].toDouble()), nullptr, pointer<float>(scale),
                                       pointer(grad), grad.stride(0), nullptr, 0, stream_of(grad), nullptr);
        if (status != LRS_OK) failed("expert_balance", status);
        return {final_gradient(grad, "expert_balance_loss"), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

py::object balance_loss(py::handle logits, py::handle indices, double balance, double z, int score, py::handle mask) {
    Balance c;
    const float a = static_cast<float>(balance), b = static_cast<float>(z);
    if (!c.take_all(logits, indices, mask) || !c.fill() || c.logits.size(1) < 1 || c.logits.size(1) > LRS_MAX_EXPERTS || !std::isfinite(a) || !std::isfinite(b) ||
        (score == LRS_SCORE_SIGMOID && b != 0.f) || c.logits.size(0) > INT32_MAX / std::max<int64_t>(1, c.indices.size(1)))
        return py::none();
    const auto out = BalanceLoss::apply(c.logits, c.indices, balance, z, static_cast<int64_t>(score), maybe(c.mask));
    return py::make_tuple(out[0], out[1]);
}

// ---------------------------------------------------------------- embedding

// None, or one of the row types; false for anything else.
bool take_type(py::handle h, at::ScalarType none, at::ScalarType &type) {
    type = none;
    if (h.is_none()) return true;
    if (!THPDtype_Check(h.ptr())) return false;
    type = reinterpret_cast<THPDtype *>(h.ptr())->scalar_type;
    return type_code(type) >= 0;
}
bool token_ids(const Tensor &t, const Tensor &like, lrs_token_ids &ids) {
    if (!t.defined() || t.device() != like.device()) return false;
    ids.id_bytes = t.scalar_type() == at::kLong ? 8 : t.scalar_type() == at::kInt ? 4 : 0;
    if (ids.id_bytes == 0) return false;
    ids.ids = pointer(t);
    if (t.is_contiguous()) {
        ids.lines = 1, ids.length = t.numel(), ids.stride = 0;
    } else if (t.dim() == 1) {
        ids.lines = t.size(0), ids.length = 1, ids.stride = t.stride(0);
    } else if (t.dim() == 2 && (t.stride(1) == 1 || t.size(1) <= 1)) {
        ids.lines = t.size(0), ids.length = t.size(1), ids.stride = t.stride(0);
    } else {
        return false;
    }
    return true;
}
// A row for every token: the stride, or -1 where the rows do not lie evenly apart.
int64_t token_rows(const Tensor &t, const Tensor &tokens) {
    const int64_t width = t.size(-1);
    const bool flat = t.dim() == 2 && t.size(0) == tokens.numel();
    if (!flat && !(t.dim() == tokens.dim() + 1 && t.sizes().slice(0, tokens.dim()) == tokens.sizes())) return -1;
    if (t.is_contiguous()) return width;
    return t.dim() == 2 && (t.stride(1) == 1 || width <= 1) ? t.stride(0) : -1;
}
bool finite(double v) { return std::isfinite(static_cast<float>(v)); }

struct Embed {
    Tensor weight, tokens;  // the gradient in the table's place for the backward
    lrs_token_ids ids{};
    int code = -1;
    int forward(Tensor &out, double scale, at::ScalarType type) const {
        std::vector<int64_t> shape(tokens.sizes().begin(), tokens.sizes().end());
        shape.push_back(weight.size(1));
        out = make(weight, shape, type);
        return lib.embed_forward(pointer(weight), weight.stride(0), &ids, pointer(out), weight.size(1), weight.size(0),
                                 weight.size(1), code, type_code(type), static_cast<float>(scale), stream_of(weight), nullptr);
    }
    bool fill_forward() { return matrix(weight, code) && token_ids(tokens, weight, ids); }
};

// The table's gradient of `grad`, into `out` if that is defined.
int embed_gradient(const Tensor &grad, int64_t stride, const lrs_token_ids &ids, int64_t vocab, double scale, int64_t padding,
                   at::ScalarType type, Tensor &out, bool add) {
    const int64_t width = grad.size(-1), tokens = ids.lines * ids.length;
    if (!out.defined()) out = make(grad, {vocab, width}, type);
    const size_t need = lib.embed_size(tokens, vocab, width, nullptr);
    const Tensor ws = make(grad, {std::max<int64_t>(1, static_cast<int64_t>(need))}, at::kByte);
    return lib.embed_backward(pointer(grad), stride, &ids, pointer(out), out.stride(0), vocab, width,
                              type_code(grad.scalar_type()), type_code(type), static_cast<float>(scale), padding, add,
                              pointer(ws), need, stream_of(grad), nullptr);
}

py::object embed_forward(py::handle weight, py::handle tokens, double scale, py::handle dtype) {
    Embed e;
    at::ScalarType type;
    if (!take(weight, e.weight) || !take(tokens, e.tokens) || !e.fill_forward() || !finite(scale) ||
        !take_type(dtype, e.weight.scalar_type(), type))
        return py::none();
    const c10::DeviceGuard guard(e.weight.device());
    Tensor out;
    return e.forward(out, scale, type) == LRS_OK ? py::cast(out) : py::object(py::none());
}

// None: no padding; -2: not one.
int64_t take_padding(py::handle h, int64_t vocab) {
    if (h.is_none()) return -1;
    if (!PyLong_Check(h.ptr())) return -2;
    const int64_t p = PyLong_AsLongLong(h.ptr());
    if (p == -1 && PyErr_Occurred()) PyErr_Clear();
    return p >= 0 && p < vocab ? p : -2;
}

py::object embed_backward(py::handle grad_in, py::handle tokens_in, int64_t vocab, double scale, py::handle padding_in,
                          py::handle dtype, py::handle out_in, bool add) {
    Tensor grad, tokens, out;
    lrs_token_ids ids{};
    if (!take(grad_in, grad) || !take(tokens_in, tokens) || !take(out_in, out, true) || !grad.is_cuda() || grad.dim() < 1 ||
        type_code(grad.scalar_type()) < 0 || !token_ids(tokens, grad, ids) || vocab < 0 || !finite(scale))
        return py::none();
    at::ScalarType type;
    const int64_t stride = token_rows(grad, tokens), padding = take_padding(padding_in, vocab);
    if (stride < 0 || padding < -1 || !take_type(dtype, out.defined() ? out.scalar_type() : grad.scalar_type(), type)) return py::none();
    if (out.defined()) {
        int code;
        if (!matrix(out, code) || out.device() != grad.device() || out.size(0) != vocab || out.size(1) != grad.size(-1) ||
            out.scalar_type() != type)
            return py::none();
    } else if (add) {
        return py::none();
    }
    const c10::DeviceGuard guard(grad.device());
    if (embed_gradient(grad, stride, ids, vocab, scale, padding, type, out, add) != LRS_OK) return py::none();
    return out_in.is_none() ? py::cast(out) : py::reinterpret_borrow<py::object>(out_in);
}

struct EmbedLookup : torch::autograd::Function<EmbedLookup> {
    static Tensor forward(AutogradContext *ctx, const Tensor &weight, const Tensor &tokens, double scale, int64_t padding,
                          int64_t type) {
        Embed e{weight, tokens};
        e.fill_forward();
        Tensor out;
        const int status = e.forward(out, scale, static_cast<at::ScalarType>(type));
        if (status != LRS_OK) failed("embedding_forward", status);
        ctx->save_for_backward({tokens});
        ctx->saved_data["vocab"] = weight.size(0);
        ctx->saved_data["type"] = static_cast<int64_t>(weight.scalar_type());
        ctx->saved_data["scale"] = scale;
        ctx->saved_data["padding"] = padding;
        return out;
    }
    static variable_list backward(AutogradContext *ctx, const variable_list &up) {
        const Tensor tokens = ctx->get_saved_variables()[0];
        Tensor grad = up[0].detach();
        const c10::DeviceGuard guard(grad.device());
        int64_t stride = token_rows(grad, tokens);
        if (stride < 0) {  // such as one number for all
            grad = grad.contiguous();
            stride = grad.size(-1);
        }
        lrs_token_ids ids{};
        Tensor out;
        int status = LRS_ERR_SIZE;
        if (token_ids(tokens, grad, ids))
            status = embed_gradient(grad, stride, ids, ctx->saved_data["vocab"].toInt(), ctx->saved_data["scale"].toDouble(),
                                    ctx->saved_data["padding"].toInt(),
                                    static_cast<at::ScalarType>(ctx->saved_data["type"].toInt()), out, false);
        if (status != LRS_OK) failed("embedding_backward", status);
        return {final_gradient(out, "embedding_lookup"), Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

py::object embed_lookup(py::handle weight, py::handle tokens, double scale, py::handle padding_in, py::handle dtype) {
    Embed e;
    at::ScalarType type;
    if (!take(weight, e.weight) || !take(tokens, e.tokens) || !e.fill_forward() || !finite(scale) ||
        !take_type(dtype, e.weight.scalar_type(), type))
        return py::none();
    const int64_t padding = take_padding(padding_in, e.weight.size(0));
    // what the library refuses is left to the Python code, which says so
    const int64_t rows = std::max<int64_t>(e.tokens.numel(), e.weight.size(0));
    if (padding < -1 || e.tokens.numel() > INT32_MAX || e.weight.size(0) >= INT32_MAX ||
        e.weight.size(1) > static_cast<int64_t>(LRS_MAX_ROW_LEN) ||
        rows >= (int64_t(1) << 40) / std::max<int64_t>(1, e.weight.size(1)))
        return py::none();
    const c10::DeviceGuard guard(e.weight.device());
    return py::cast(EmbedLookup::apply(e.weight, e.tokens, scale, padding, static_cast<int64_t>(type)));
}

// --------------------------------------- log probabilities of given tokens

struct Logprobs {
    Tensor logits, tokens, mask;
    lrs_logprobs d{};
    bool take_all(py::handle x, py::handle t, py::handle m) { return take(x, logits) && take(t, tokens) && take(m, mask, true); }
    bool fill(double temperature) {
        int code;
        if (!matrix(logits, code) || !tokens.defined() || tokens.device() != logits.device() || tokens.dim() != 1 ||
            tokens.size(0) != logits.size(0) || !mask_ok(mask, logits))
            return false;
        const int bytes = tokens.scalar_type() == at::kLong ? 8 : tokens.scalar_type() == at::kInt ? 4 : 0;
        d = lrs_logprobs{pointer(logits), logits.stride(0), pointer(tokens), tokens.stride(0), bytes, code,
                         pointer<uint8_t>(mask), logits.size(0), logits.size(1), temperature};
        return bytes != 0;
    }
    Tensor workspace(int64_t k) const {
        const size_t need = lib.logprobs_size(d.rows, d.n, k, d.dtype, nullptr);
        return make(tokens, {std::max<int64_t>(1, static_cast<int64_t>(need))}, at::kByte);
    }
    Tensor numbers() const { return make(tokens, {d.rows}, at::kFloat); }
    int forward(Tensor &logprobs, Tensor &entropy, Tensor &stats) const {
        const Tensor ws = workspace(0);
        logprobs = numbers();
        entropy = numbers();
        stats = make(tokens, {d.rows, 3}, at::kFloat);
        return lib.logprobs_forward(&d, pointer<float>(logprobs), pointer<float>(entropy), pointer<float>(stats), pointer(ws),
                                    ws.numel(), stream_of(logits), nullptr);
    }
};

py::object logprobs_forward(py::handle logits, py::handle tokens, double temperature, py::handle mask) {
    Logprobs c;
    if (!c.take_all(logits, tokens, mask) || !c.fill(temperature)) return py::none();
    const c10::DeviceGuard guard(c.logits.device());
    Tensor logprobs, entropy, stats;
    if (c.forward(logprobs, entropy, stats) != LRS_OK) return py::none();
    return py::make_tuple(logprobs, entropy, stats);
}

py::object logprobs_topk(py::handle logits, py::handle tokens, int64_t k, double temperature) {
    Logprobs c;
    if (!c.take_all(logits, tokens, py::none()) || !c.fill(temperature) || k < 0 || k > c.d.n) return py::none();
    const c10::DeviceGuard guard(c.logits.device());
    const Tensor ws = c.workspace(k), logprobs = c.numbers(), entropy = c.numbers(), ranks = make(c.tokens, {c.d.rows}, at::kInt);
    const Tensor top = make(c.tokens, {c.d.rows, k}, at::kFloat), indices = make(c.tokens, {c.d.rows, k}, at::kLong);
    if (lib.logprobs_topk(&c.d, k, pointer<float>(logprobs), pointer<float>(entropy), pointer<int32_t>(ranks), pointer<float>(top),
                          pointer<int64_t>(indices), pointer(ws), ws.numel(), stream_of(c.logits), nullptr) != LRS_OK)
        return py::none();
    return py::make_tuple(logprobs, entropy, ranks, top, indices);
}

py::object logprobs_step(py::handle logits, py::handle tokens, py::handle up, py::handle down, double temperature, py::handle mask) {
    Logprobs c;
    Tensor a, b;
    if (!c.take_all(logits, tokens, mask) || !c.fill(temperature) || !take(up, a, true) || !take(down, b, true) ||
        !by_row(a, c.logits) || !by_row(b, c.logits))
        return py::none();
    const c10::DeviceGuard guard(c.logits.device());
    const Tensor ws = c.workspace(0), logprobs = c.numbers(), entropy = c.numbers(), grad = like_rows(c.logits);
    if (lib.logprobs_step(&c.d, pointer<float>(a), pointer<float>(b), pointer<float>(logprobs), pointer<float>(entropy),
                          pointer(grad), grad.stride(0), pointer(ws), ws.numel(), stream_of(c.logits), nullptr) != LRS_OK)
        return py::none();
    return py::make_tuple(logprobs, entropy, grad);
}

py::object logprobs_backward(py::handle logits, py::handle tokens, py::handle stats_in, py::handle up, py::handle down,
                             double temperature, py::handle mask) {
    Logprobs c;
    Tensor a, b, stats;
    if (!c.take_all(logits, tokens, mask) || !c.fill(temperature) || !take(stats_in, stats) || !take(up, a, true) ||
        !take(down, b, true) || !by_row(a, c.logits) || !by_row(b, c.logits) || stats.device() != c.logits.device() ||
        stats.scalar_type() != at::kFloat || !stats.is_contiguous() || stats.dim() != 2 || stats.size(0) != c.d.rows || stats.size(1) != 3)
        return py::none();
    const c10::DeviceGuard guard(c.logits.device());
    const Tensor grad = like_rows(c.logits);
    if (lib.logprobs_backward(&c.d, pointer<float>(stats), pointer<float>(a), pointer<float>(b), pointer(grad), grad.stride(0),
                              stream_of(grad), nullptr) != LRS_OK)
        return py::none();
    return py::cast(grad);
}

struct TokenLogprobs : torch::autograd::Function<TokenLogprobs> {
    static variable_list forward(AutogradContext *ctx, const Tensor &logits, const Tensor &tokens, double temperature,
                                 const Maybe &mask) {
        Logprobs c{logits, tokens, given(mask)};
        c.fill(temperature);
        Tensor logprobs, entropy, stats;
        const int status = c.forward(logprobs, entropy, stats);
        if (status != LRS_OK) failed("token_logprobs_forward", status);
        ctx->save_for_backward({logits, tokens, stats, c.mask});
        ctx->saved_data["temperature"] = temperature;
        ctx->set_materialize_grads(false);
        return {logprobs, entropy};
    }
    static variable_list backward(AutogradContext *ctx, const variable_list &up) {
        const auto saved = ctx->get_saved_variables();
        Logprobs c{saved[0].detach(), saved[1], saved[3]};
        Tensor a, b, grad;
        if (up[0].defined()) a = up[0].detach().contiguous();
        if (up[1].defined()) b = up[1].detach().contiguous();
        if (!a.defined() && !b.defined()) return {Tensor(), Tensor(), Tensor(), Tensor()};
        const c10::DeviceGuard guard(c.logits.device());
        if (!c.fill(ctx->saved_data["temperature"].toDouble()) || !by_row(a, c.logits) || !by_row(b, c.logits))
            failed("token_logprobs_backward", LRS_ERR_SIZE);
        grad = like_rows(c.logits);
        const int status = lib.logprobs_backward(&c.d, pointer<float>(saved[2]), pointer<float>(a), pointer<float>(b),
                                                 pointer(grad), grad.stride(0), stream_of(grad), nullptr);
        if (status != LRS_OK) failed("token_logprobs_backward", status);
        return {final_gradient(grad, "token_logprobs"), Tensor(), Tensor(), Tensor()};
    }
};

py::object logprobs_autograd(py::handle logits, py::handle tokens, double temperature, py::handle mask) {
    Logprobs c;
    if (!c.take_all(logits, tokens, mask) || !c.fill(temperature) || !(temperature > 0) || !std::isfinite(temperature) ||
        !std::isfinite(static_cast<float>(1.44269504088896340736 / temperature)) || c.d.n > static_cast<int64_t>(LRS_MAX_ROW_LEN) ||
        c.d.rows >= (int64_t(1) << 40) / std::max<int64_t>(1, c.d.n))
        return py::none();
    const c10::DeviceGuard guard(c.logits.device());
    const auto out = TokenLogprobs::apply(c.logits, c.tokens, temperature, maybe(c.mask));
    return py::make_tuple(out[0], out[1]);
}

}  // namespace

PYBIND11_MODULE(_row_binding, m) {
    m.def("bind", &bind);
    m.def("topk", &topk);
    m.def("distill_step", &distill_step);
    m.def("distill_forward", &distill_forward);
    m.def("distill_loss", &distill_loss);
    m.def("balance_step", &balance_step);
    m.def("balance_loss", &balance_loss);
    m.def("embedding_forward", &embed_forward);
    m.def("embedding_backward", &embed_backward);
    m.def("embedding_lookup", &embed_lookup);
    m.def("logprobs_forward", &logprobs_forward);
    m.def("logprobs_topk", &logprobs_topk);
    m.def("logprobs_step", &logprobs_step);
    m.def("logprobs_backward", &logprobs_backward);
    m.def("logprobs_autograd", &logprobs_autograd);
}
