// Autograd nodes of balance_loss and swiglu_checkpoint, and the calls of the combine
// that keeps its rows.
//
// The nodes are a few microseconds of GPU work for a small batch, where the host bounds a
// step: a forward and backward through nodes written in Python took 110 us (balance
// loss, 256 tokens) and 95 us (SwiGLU, 8 rows), through these 55 and 49, on a host
// where torch's own x * 2 takes 44.  The nodes call the C entries themselves; the
// arguments' checks and errors are the Python binding's.  The combine's two calls have
// 15 tensors each to look at: a step of 64 tokens 20 us with them in Python, 13 here.
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/extension.h>

#include <unordered_set>

#include "balance.hpp"
#include "moe.h"

namespace py = pybind11;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused(s.str());
}

void check(moe_status st) {
  if (st != MOE_OK) refuse("libmoe status ", st, ": ", moe_status_str(st));
}

const char* dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    default: return at::toString(t);
  }
}

void on_gpu(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(name, " must be a GPU tensor");
}

// An argument that goes with a tensor on device `dev`: same device, contiguous.
void goes_with(const Tensor& t, c10::Device dev, const char* name) {
  on_gpu(t, name);
  if (t.device() != dev) refuse(name, " is on ", t.device(), ", expected device ", (int)dev.index());
  if (!t.is_contiguous()) refuse(name, " must be contiguous");
}

void typed(const Tensor& t, at::ScalarType want, const char* name) {
  if (t.scalar_type() != want) refuse(name, " must be ", dtype_name(want), ", got ", dtype_name(t.scalar_type()));
}

void* stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.get_device()).stream(); }

template <typename T>
T* at_or_null(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

// A leaf whose gradient accumulator belongs to another stream's graph that still lives:
// the engine would make that stream wait inside a capture, which ends the process.
void refuse_foreign_leaf(const Tensor& t, const char* name) {
  if (!at::GradMode::is_enabled() || !t.requires_grad() || !t.is_leaf()) return;
  const auto accumulator = torch::autograd::impl::try_get_grad_accumulator(t);
  if (!accumulator) return;
  const auto home = accumulator->stream();
  const auto here = c10::hip::getCurrentHIPStream(t.get_device());
  if (home && home->id() != here.id())
    refuse(name, " is a leaf of a graph that another stream built and that still lives: a captured backward needs leaves "
           "of its own (detach() them in the capture, or free that graph)");
}

bool capturing() { return c10::hip::currentStreamCaptureStatusMayInitCtx() != c10::hip::CaptureStatus::None; }

void refuse_foreign_leaves(const std::vector<std::optional<Tensor>>& tensors) {
  if (!capturing()) return;
  for (const auto& t : tensors)
    if (t && t->is_cuda()) refuse_foreign_leaf(*t, "an input");
}

// In a captured backward: a node that it will still come to and that an eager forward on the
// default stream made (a leaf's accumulator that a living graph holds, or a part of that graph
// itself).  The engine would make the default stream wait inside the capture, which ends the
// process.  Only nodes that this backward executes count, and any other stream may take part.
void refuse_default_stream_ahead() {
  if (!capturing()) return;
  const auto here = torch::autograd::get_current_node();
  if (!here) return;
  const auto* executed = torch::autograd::get_current_graph_task_exec_info();
  std::unordered_set<torch::autograd::Node*> seen;
  std::vector<torch::autograd::Node*> open{here.get()};
  while (!open.empty()) {
    const auto* node = open.back();
    open.pop_back();
    for (const auto& edge : node->next_edges()) {
      auto* next = edge.function.get();
      if (!next || !seen.insert(next).second) continue;
      if (executed && !executed->empty()) {
        const auto it = executed->find(next);
        if (it == executed->end() || !it->second.should_execute()) continue;
      }
      const auto home = next->stream();
      if (home && home->id() == c10::hip::getDefaultHIPStream(home->device_index()).id())
        refuse("a captured backward would reach ", next->name(), " of the default stream, of a graph that an eager "
               "forward built and that still lives: free that graph, or capture with leaves of its own");
      open.push_back(next);
    }
  }
}

// Gradients that cannot be differentiated again: a second derivative raises.
variable_list once(variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  variable_list in;
  for (auto& g : grads) {
    if (g.defined()) g = g.detach().requires_grad_();
    in.push_back(g);
  }
  auto error = std::make_shared<torch::autograd::DelayedError>(
      "the gradient of balance_loss and of swiglu_checkpoint is differentiable once", (int64_t)in.size());
  return (*error)(std::move(in));
}

// ----------------------------------------------------------------------------- balance loss

struct Choices {
  Tensor idx, mask, off;  // mask and off may be undefined
};

struct BalanceSizes {
  int64_t T, n, S;
  int32_t K, mask_ndim, dtype;
  bool keep;  // a backward may come
};

// The node's own integers: the tokens of each sequence and their sum, then on a 16-byte
// boundary the counts.  (The counts that it returns are the caller's, who may change them
// before the backward: a sum over ranks in place is not seen by autograd.)
int64_t counts_at(int64_t rows) { return (rows + 4) / 4 * 4; }
int32_t* kept_counts(const Tensor& tokens, int64_t rows) { return tokens.data_ptr<int32_t>() + counts_at(rows); }

struct BalanceNode : torch::autograd::Function<BalanceNode> {
  static variable_list forward(AutogradContext* ctx, const Tensor& given, const Choices& c, const BalanceSizes& z) {
    const Tensor logits = given.contiguous();
    const auto i32 = logits.options().dtype(at::kInt), f32 = logits.options().dtype(at::kFloat);
    const int64_t rows = z.S ? z.S : 1;
    size_t bytes = 0;
    check(moe_balance_workspace_size(z.T, z.n, z.S, &bytes));
    Tensor loss = at::empty({}, f32), z_loss = at::empty({}, f32);
    Tensor counts = z.S ? at::empty({z.S, z.n}, i32) : at::empty({z.n}, i32);
    Tensor tokens = at::empty({z.keep ? counts_at(rows) + rows * z.n : rows + 1}, i32);
    Tensor workspace = at::empty({(int64_t)bytes}, i32.dtype(at::kByte));
    check(moe::balance_forward(z.T, z.n, z.K, z.S, z.mask_ndim, z.dtype, logits.data_ptr(), c.idx.data_ptr<int32_t>(),
                               at_or_null<const uint8_t>(c.mask), at_or_null<const int32_t>(c.off),
                               loss.data_ptr<float>(), z_loss.data_ptr<float>(), counts.data_ptr<int32_t>(),
                               z.keep ? kept_counts(tokens, rows) : nullptr, tokens.data_ptr<int32_t>(),
                               workspace.data_ptr(), bytes, stream_of(logits)));
    ctx->save_for_backward({logits, c.mask, c.off, tokens});
    ctx->saved_data["K"] = (int64_t)z.K;
    ctx->mark_non_differentiable({counts});
    ctx->set_materialize_grads(false);
    return {loss, z_loss, counts};
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    if (!grads[0].defined() && !grads[1].defined()) return {Tensor(), Tensor(), Tensor()};
    refuse_default_stream_ahead();
    const auto saved = ctx->get_saved_variables();
    const Tensor &logits = saved[0], &mask = saved[1], &off = saved[2], &tokens = saved[3];
    const int64_t seqs = off.defined() ? off.numel() - 1 : 0;
    Tensor grad;
    {
      at::NoGradGuard no_grad;
      const c10::DeviceGuard guard(logits.device());
      grad = at::empty_like(logits);
      check(moe_balance_bwd(logits.size(0), logits.size(1), (int32_t)ctx->saved_data["K"].toInt(),
                            seqs, mask.defined() ? (int32_t)mask.dim() : 0,
                            logits.scalar_type() == at::kFloat ? MOE_DTYPE_FP32 : MOE_DTYPE_BF16, logits.data_ptr(),
                            at_or_null<const uint8_t>(mask), at_or_null<const int32_t>(off),
                            kept_counts(tokens, seqs ? seqs : 1), tokens.data_ptr<int32_t>(),
                            at_or_null<const float>(grads[0]), at_or_null<const float>(grads[1]), grad.data_ptr(),
                            stream_of(logits)));
    }
    return once({grad, Tensor(), Tensor()});
  }
};

std::tuple<Tensor, Tensor, Tensor> balance_loss(const Tensor& logits, const Tensor& idx,
                                                const std::optional<Tensor>& mask, const std::optional<Tensor>& off) {
  on_gpu(logits, "logits");
  if (logits.dim() != 2) refuse("logits must be a tensor of shape (T, n_ids), got ", logits.sizes());
  if (logits.scalar_type() != at::kFloat && logits.scalar_type() != at::kBFloat16)
    refuse("logits must be float32 or bfloat16, got ", dtype_name(logits.scalar_type()));
  if (idx.dim() != 2 || idx.size(0) != logits.size(0))
    refuse("topk_idx must be a tensor of shape (", logits.size(0), ", K), got ", idx.sizes());
  goes_with(idx, logits.device(), "topk_idx");
  typed(idx, at::kInt, "topk_idx");
  BalanceSizes z{logits.size(0), logits.size(1), 0, (int32_t)std::min<int64_t>(idx.size(1), 1 << 20), 0,
                 logits.scalar_type() == at::kFloat ? MOE_DTYPE_FP32 : MOE_DTYPE_BF16,
                 at::GradMode::is_enabled() && logits.requires_grad()};
  Choices c{idx, {}, {}};
  if (mask) {
    const Tensor& m = *mask;
    const bool by_slot = m.dim() == 2 && m.sizes() == idx.sizes();
    if (!by_slot && !(m.dim() == 1 && m.size(0) == z.T))
      refuse("x_active_mask must be a tensor of shape (", z.T, ",) or ", idx.sizes(), ", got ", m.sizes());
    goes_with(m, logits.device(), "x_active_mask");
    if (m.scalar_type() != at::kBool && m.scalar_type() != at::kByte)
      refuse("x_active_mask must be torch.uint8 or torch.bool, got ", dtype_name(m.scalar_type()));
    c.mask = m;
    z.mask_ndim = by_slot ? 2 : 1;
  }
  if (off) {
    if (off->dim() != 1 || off->numel() < 2)
      refuse("seq_offsets must hold the num_seqs + 1 ends of at least one sequence, got ", off->sizes());
    goes_with(*off, logits.device(), "seq_offsets");
    typed(*off, at::kInt, "seq_offsets");
    c.off = *off;
    z.S = off->numel() - 1;
  }
  const c10::DeviceGuard guard(logits.device());
  if (capturing()) refuse_foreign_leaf(logits, "logits");
  const variable_list r = BalanceNode::apply(logits, c, z);
  return {r[0], r[1], r[2]};
}

// ----------------------------------------------------------------------------- SwiGLU kept in 8 bits

struct SwigluNode : torch::autograd::Function<SwigluNode> {
  static Tensor forward(AutogradContext* ctx, const Tensor& given) {
    const Tensor gate_up = given.contiguous();
    auto sizes = gate_up.sizes().vec();
    const int64_t F = sizes.back() / 2, R = gate_up.numel() / (2 * F), nb = (F + 31) / 32;
    sizes.back() = F;
    const auto o = gate_up.options();
    Tensor h = at::empty(sizes, o), codes = at::empty({R, 2 * F}, o.dtype(at::kChar)), scales = at::empty({R, 2 * nb}, o);
    check(moe_swiglu_checkpoint_fwd(R, F, gate_up.data_ptr(), nullptr, h.data_ptr(), codes.data_ptr<int8_t>(),
                                    scales.data_ptr(), stream_of(gate_up)));
    ctx->save_for_backward({codes, scales});
    sizes.back() = 2 * F;
    ctx->saved_data["sizes"] = sizes;
    return h;
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    refuse_default_stream_ahead();
    const auto saved = ctx->get_saved_variables();
    const Tensor &codes = saved[0], &scales = saved[1];
    Tensor grad;
    {
      at::NoGradGuard no_grad;
      const c10::DeviceGuard guard(codes.device());
      const Tensor grad_h = grads[0].contiguous();
      grad = at::empty(ctx->saved_data["sizes"].toIntVector(), grad_h.options());
      check(moe_swiglu_checkpoint_bwd(codes.size(0), codes.size(1) / 2, codes.data_ptr<int8_t>(), scales.data_ptr(),
                                      nullptr, grad_h.data_ptr(), grad.data_ptr(), stream_of(codes)));
    }
    return once({grad});
  }
};

Tensor swiglu_checkpoint(const Tensor& gate_up) {
  on_gpu(gate_up, "gate_up");
  typed(gate_up, at::kBFloat16, "gate_up");
  if (!gate_up.dim() || gate_up.size(-1) % 2 || !gate_up.size(-1))
    refuse("gate_up must be a tensor of shape (..., 2F), got ", gate_up.sizes());
  const c10::DeviceGuard guard(gate_up.device());
  if (capturing()) refuse_foreign_leaf(gate_up, "gate_up");
  return SwigluNode::apply(gate_up);
}

// ----------------------------------------------------------------------------- combine

using Arg = const std::optional<Tensor>&;

// The entries' tensor arguments: contiguous, on one device, of their type and size.
struct Args {
  c10::Device dev;
  template <typename T = void>
  T* at(Arg t, at::ScalarType type, int64_t n, const char* name) const {
    if (!t) return nullptr;
    goes_with(*t, dev, name);
    typed(*t, type, name);
    if (t->numel() < n) refuse(name, " holds ", t->numel(), " elements, needs at least ", n);
    return static_cast<T*>(t->data_ptr());
  }
  const uint8_t* mask(Arg t, int64_t n) const {
    if (!t) return nullptr;
    return at<const uint8_t>(t, t->scalar_type() == at::kBool ? at::kBool : at::kByte, n, "x_active_mask");
  }
};

int64_t slots(const moe_shape& s) { return s.T * s.K; }
int64_t masked(const moe_shape& s) { return s.mask_ndim == 0 ? 0 : (s.mask_ndim == 1 ? s.T : slots(s)); }
int64_t blocks(const moe_shape& s) { return s.capacity * ((s.H + 31) / 32); }

// `stream`: a hipStream_t, or -1 for the current one of the tensors' device.
void* stream_or_current(int64_t stream, c10::Device dev) {
  return stream == -1 ? c10::hip::getCurrentHIPStream(dev.index()).stream() : reinterpret_cast<void*>(stream);
}

void combine_checkpoint(int64_t shape, int64_t stream, Arg y, Arg idx, Arg w, Arg assist, Arg counts, Arg mask,
                        Arg shared, Arg ori, Arg a1, Arg a2, Arg v, Arg out, Arg codes, Arg scales) {
  const moe_shape& s = *reinterpret_cast<const moe_shape*>(shape);
  if (!y) refuse("y must be a GPU tensor");
  on_gpu(*y, "y");
  const Args a{y->device()};
  const c10::DeviceGuard guard(a.dev);
  const int64_t q = s.const_expert_num * s.H;
  check(moe_combine_checkpoint(
      &s, a.at(y, at::kBFloat16, s.capacity * s.H, "y"), a.at<int32_t>(idx, at::kInt, slots(s), "topk_idx"),
      a.at<float>(w, at::kFloat, slots(s), "topk_weights"),
      a.at<int32_t>(assist, at::kInt, slots(s) + s.capacity, "assist_info_for_combine"),
      a.at<int32_t>(counts, at::kInt, s.num_experts, "ep_send_counts"), a.mask(mask, masked(s)),
      a.at(shared, at::kBFloat16, s.T * s.H, "shared_expert_x"), a.at(ori, at::kBFloat16, s.T * s.H, "ori_x"),
      a.at(a1, at::kBFloat16, q, "const_alpha_1"), a.at(a2, at::kBFloat16, q, "const_alpha_2"),
      a.at(v, at::kBFloat16, q, "const_v"), a.at(out, at::kBFloat16, s.T * s.H, "out"),
      a.at<int8_t>(codes, at::kChar, s.capacity * s.H, "y_codes"), a.at(scales, at::kBFloat16, blocks(s), "y_scales"),
      stream_or_current(stream, a.dev)));
}

void combine_bwd_weights_checkpoint(int64_t shape, int64_t stream, Arg grad_out, Arg codes, Arg scales, Arg idx, Arg w,
                                    Arg assist, Arg counts, Arg mask, Arg ori, Arg a1, Arg a2, Arg v, Arg grad_w,
                                    Arg row_w) {
  const moe_shape& s = *reinterpret_cast<const moe_shape*>(shape);
  if (!grad_out) refuse("grad_out must be a GPU tensor");
  on_gpu(*grad_out, "grad_out");
  const Args a{grad_out->device()};
  const c10::DeviceGuard guard(a.dev);
  const int64_t q = s.const_expert_num * s.H;
  check(moe_combine_bwd_weights_checkpoint(
      &s, a.at(grad_out, at::kBFloat16, s.T * s.H, "grad_out"),
      a.at<int8_t>(codes, at::kChar, s.capacity * s.H, "y_codes"), a.at(scales, at::kBFloat16, blocks(s), "y_scales"),
      a.at<int32_t>(idx, at::kInt, slots(s), "topk_idx"), a.at<float>(w, at::kFloat, slots(s), "topk_weights"),
      a.at<int32_t>(assist, at::kInt, slots(s) + s.capacity, "assist_info_for_combine"),
      a.at<int32_t>(counts, at::kInt, s.num_experts, "ep_send_counts"), a.mask(mask, masked(s)),
      a.at(ori, at::kBFloat16, s.T * s.H, "ori_x"), a.at(a1, at::kBFloat16, q, "const_alpha_1"),
      a.at(a2, at::kBFloat16, q, "const_alpha_2"), a.at(v, at::kBFloat16, q, "const_v"),
      a.at<float>(grad_w, at::kFloat, slots(s), "grad_topk_weights"),
      a.at<float>(row_w, at::kFloat, s.capacity, "row_weights"), stream_or_current(stream, a.dev)));
}

py::handle g_error;

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.def("raise_as", [](py::object cls) { g_error = cls.release(); });
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const Refused& e) {
      PyErr_SetString(g_error ? g_error.ptr() : PyExc_RuntimeError, e.what());
    }
  });
  m.def("balance_loss", &balance_loss);
  m.def("swiglu_checkpoint", &swiglu_checkpoint);
  m.def("combine_checkpoint", &combine_checkpoint);
  m.def("combine_bwd_weights_checkpoint", &combine_bwd_weights_checkpoint);
  m.def("refuse_foreign_leaves", &refuse_foreign_leaves);
  m.def("refuse_default_stream_ahead", &refuse_default_stream_ahead);
}
