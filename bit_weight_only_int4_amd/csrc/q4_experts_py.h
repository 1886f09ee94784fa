// q4_experts_py.h -- the native half of the Python binding of q4experts.h, part
// of q4_serve_py.cpp: checks, outputs and workspaces of the functions in
// mixture.py, which pass their arguments on by position.
#pragma once

namespace {

// [rows, n] of a type, unit stride along its rows; the pitch
int64_t matrix(const at::Tensor& t, const char* name, const char* what, int64_t rows, int64_t n,
               at::ScalarType type, const at::Device& dev) {
  if (t.dim() != 2 || t.scalar_type() != type || (rows >= 0 && t.size(0) != rows) ||
      (n >= 0 && t.size(1) != n) || (t.size(1) > 1 && t.stride(1) != 1))
    refuse("%s must be %s %s with unit stride along its rows, got %s %s", name, type_name(type), what,
           shape(t).c_str(), type_name(t.scalar_type()));
  same_device(t, name, dev);
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

void* dense(const at::Tensor& t, const char* name, at::IntArrayRef want, at::ScalarType type,
            const at::Device& dev) {
  if (t.scalar_type() != type || t.sizes() != want || !t.is_contiguous()) {
    std::string s;
    for (int64_t v : want) s += (s.empty() ? "" : ", ") + std::to_string(v);
    refuse("%s must be contiguous %s [%s], got %s %s", name, type_name(type), s.c_str(),
           shape(t).c_str(), type_name(t.scalar_type()));
  }
  same_device(t, name, dev);
  return t.data_ptr();
}

int32_t truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyFailed{};
  return v;
}

int64_t groups_of(int64_t K, int64_t gs) {
  if (gs < 0) refuse("group_size must not be negative, got %lld", (long long)gs);
  return gs == 0 ? 1 : (K + gs - 1) / gs;
}

// logits, top_k, score, bias, groups, top_groups, renormalize, scale, stream -> ids, weights
PyObject* route(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  const at::Device dev = x.device();
  const int32_t dtype = dtype_of(x, "logits");
  const int64_t ld = matrix(x, "logits", "[T, experts]", -1, -1, x.scalar_type(), dev);
  const int64_t T = x.size(0), E = x.size(1), k = integer(a[1]), groups = integer(a[4]), top = integer(a[5]);
  if (E < 1 || E > 1024) refuse("logits must have 1 .. 1024 experts, got %s", shape(x).c_str());
  if (groups < 1 || E % groups || top < 1 || top > groups)
    refuse("groups must divide %lld experts and top_groups be 1 .. groups, got %lld and %lld",
           (long long)E, (long long)groups, (long long)top);
  const int64_t most = std::min<int64_t>(32, E / groups * top);
  if (k < 1 || k > most) refuse("top_k must be 1 .. %lld, got %lld", (long long)most, (long long)k);
  const float* bias = given(a[3]) ? (const float*)vector(tensor(a[3], "bias"), "bias", E, at::kFloat, dev) : nullptr;
  const double scale = number(a[7]);
  const int32_t renorm = truth(a[6]);
  on_gpu(dev, "logits");
  const c10::DeviceGuard guard(dev);
  const at::Tensor ids = at::empty({T, k}, x.options().dtype(at::kInt));
  const at::Tensor weights = at::empty({T, k}, x.options().dtype(at::kFloat));
  check(q4_route(x.data_ptr(), ld, dtype, T, E, k, (int32_t)integer(a[2]), bias, groups, top, renorm,
                 (float)scale, (int32_t*)ids.data_ptr(), (float*)weights.data_ptr(), stream_of(a[8])),
        "q4_route");
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyFailed{};
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(ids));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(weights));
  return r;
}

// logits, ids, g_weights, score, renormalize, scale, dlogits, stream
PyObject* route_backward(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  const at::Device dev = x.device();
  const int32_t dtype = dtype_of(x, "logits");
  const int64_t ld = matrix(x, "logits", "[T, experts]", -1, -1, x.scalar_type(), dev);
  const int64_t T = x.size(0), E = x.size(1);
  const at::Tensor& ids_t = tensor(a[1], "ids");
  if (ids_t.dim() != 2) refuse("ids must be int32 [%lld, top_k], got %s", (long long)T, shape(ids_t).c_str());
  const int64_t k = ids_t.size(1);
  const int32_t* ids = (const int32_t*)dense(ids_t, "ids", {T, k}, at::kInt, dev);
  const float* g = (const float*)dense(tensor(a[2], "g_weights"), "g_weights", {T, k}, at::kFloat, dev);
  at::Tensor dx;
  int64_t ldd = E;
  if (given(a[6])) {
    dx = tensor(a[6], "dlogits");
    ldd = matrix(dx, "dlogits", "[T, experts]", T, E, x.scalar_type(), dev);
  }
  const int32_t renorm = truth(a[4]);
  const double scale = number(a[5]);
  on_gpu(dev, "logits");
  const c10::DeviceGuard guard(dev);
  if (!dx.defined()) dx = at::empty({T, E}, x.options());
  check(q4_route_backward(x.data_ptr(), ld, dtype, T, E, k, ids, (int32_t)integer(a[3]), renorm,
                          (float)scale, g, dx.data_ptr(), ldd, stream_of(a[7])),
        "q4_route_backward");
  return THPVariable_Wrap(dx);
}

struct ExpertWeights {
  int64_t E, H, W;
  const uint8_t *gate_up, *down;
  const float *gate_up_scales, *down_scales;
};

// gate_up, gate_up_scales, down, down_scales of a hidden size
ExpertWeights experts_of(PyObject* const* a, int64_t H, int64_t gs, const at::Device& dev) {
  const at::Tensor &gu = tensor(a[0], "gate_up"), &dn = tensor(a[2], "down");
  if (gu.dim() != 3 || gu.size(1) % 2) refuse("gate_up must be uint8 [experts, 2 * width, hidden / 2], got %s", shape(gu).c_str());
  ExpertWeights w;
  w.E = gu.size(0);
  w.H = H;
  w.W = gu.size(1) / 2;
  if (H % 8 || w.W % 8 || H < 8 || w.W < 8)
    refuse("hidden and width must be multiples of 8, got %lld and %lld", (long long)H, (long long)w.W);
  w.gate_up = (const uint8_t*)dense(gu, "gate_up", {w.E, 2 * w.W, H / 2}, at::kByte, dev);
  w.down = (const uint8_t*)dense(dn, "down", {w.E, H, w.W / 2}, at::kByte, dev);
  const at::Tensor &gus = tensor(a[1], "gate_up_scales"), &dns = tensor(a[3], "down_scales");
  const int64_t gh = groups_of(H, gs), gw = groups_of(w.W, gs);
  if (gs == 0) {
    w.gate_up_scales = (const float*)dense(gus, "gate_up_scales", {w.E, 2 * w.W}, at::kFloat, dev);
    w.down_scales = (const float*)dense(dns, "down_scales", {w.E, H}, at::kFloat, dev);
  } else {
    w.gate_up_scales = (const float*)dense(gus, "gate_up_scales", {w.E, gh, 2 * w.W}, at::kFloat, dev);
    w.down_scales = (const float*)dense(dns, "down_scales", {w.E, gw, H}, at::kFloat, dev);
  }
  return w;
}

// x, ids, weights, gate_up, gate_up_scales, down, down_scales, group_size, order, keep, out, workspace, stream
PyObject* experts(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const at::Device dev = x.device();
  const int32_t dtype = dtype_of(x, "x");
  const int64_t ldx = matrix(x, "x", "[T, hidden]", -1, -1, x.scalar_type(), dev);
  const int64_t T = x.size(0), H = x.size(1), gs = integer(a[7]);
  const at::Tensor& ids_t = tensor(a[1], "ids");
  if (ids_t.dim() != 2) refuse("ids must be int32 [%lld, top_k], got %s", (long long)T, shape(ids_t).c_str());
  const int64_t k = ids_t.size(1);
  const int32_t* ids = (const int32_t*)dense(ids_t, "ids", {T, k}, at::kInt, dev);
  const float* weights = (const float*)dense(tensor(a[2], "weights"), "weights", {T, k}, at::kFloat, dev);
  const ExpertWeights w = experts_of(a + 3, H, gs, dev);
  const bool keep = truth(a[9]);
  at::Tensor out;
  int64_t ldo = H;
  if (given(a[10])) {
    out = tensor(a[10], "out");
    ldo = matrix(out, "out", "[T, hidden]", T, H, x.scalar_type(), dev);
  }
  on_gpu(dev, "x");
  const c10::DeviceGuard guard(dev);
  if (!out.defined()) out = at::empty({T, H}, x.options());
  const at::Tensor pre = keep ? at::empty({T, k, 2 * w.W}, x.options().dtype(at::kFloat)) : at::Tensor();
  const Workspace ws(a[11], given(a[11]) ? 0 : q4_experts_workspace_bytes(dtype, T, H, w.W, w.E, k, gs), x.options());
  check(q4_experts(x.data_ptr(), ldx, dtype, T, H, w.W, w.E, k, ids, weights, w.gate_up, w.gate_up_scales,
                   w.down, w.down_scales, gs, (int32_t)integer(a[8]), out.data_ptr(), ldo,
                   keep ? (float*)pre.data_ptr() : nullptr, ws.p, ws.n, stream_of(a[12])),
        "q4_experts");
  if (!keep) return THPVariable_Wrap(out);
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyFailed{};
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(pre));
  return r;
}

// dout, ids, weights, pre, gate_up, gate_up_scales, down, down_scales, group_size, order, dx, workspace, stream
PyObject* experts_backward(PyObject* const* a) {
  const at::Tensor& d = tensor(a[0], "dout");
  const at::Device dev = d.device();
  const int32_t dtype = dtype_of(d, "dout");
  const int64_t ldd = matrix(d, "dout", "[T, hidden]", -1, -1, d.scalar_type(), dev);
  const int64_t T = d.size(0), H = d.size(1), gs = integer(a[8]);
  const at::Tensor& ids_t = tensor(a[1], "ids");
  if (ids_t.dim() != 2) refuse("ids must be int32 [%lld, top_k], got %s", (long long)T, shape(ids_t).c_str());
  const int64_t k = ids_t.size(1);
  const int32_t* ids = (const int32_t*)dense(ids_t, "ids", {T, k}, at::kInt, dev);
  const float* weights = (const float*)dense(tensor(a[2], "weights"), "weights", {T, k}, at::kFloat, dev);
  const ExpertWeights w = experts_of(a + 4, H, gs, dev);
  const float* pre = (const float*)dense(tensor(a[3], "pre"), "pre", {T, k, 2 * w.W}, at::kFloat, dev);
  at::Tensor dx;
  int64_t lddx = H;
  if (given(a[10])) {
    dx = tensor(a[10], "dx");
    lddx = matrix(dx, "dx", "[T, hidden]", T, H, d.scalar_type(), dev);
  }
  on_gpu(dev, "dout");
  const c10::DeviceGuard guard(dev);
  if (!dx.defined()) dx = at::empty({T, H}, d.options());
  const at::Tensor dw = at::empty({T, k}, d.options().dtype(at::kFloat));
  const Workspace ws(a[11], given(a[11]) ? 0 : q4_experts_backward_workspace_bytes(dtype, T, H, w.W, w.E, k, gs), d.options());
  check(q4_experts_backward(d.data_ptr(), ldd, dtype, T, H, w.W, w.E, k, ids, weights, pre, w.gate_up,
                            w.gate_up_scales, w.down, w.down_scales, gs, (int32_t)integer(a[9]), dx.data_ptr(),
                            lddx, (float*)dw.data_ptr(), ws.p, ws.n, stream_of(a[12])),
        "q4_experts_backward");
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyFailed{};
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(dx));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(dw));
  return r;
}

struct Head {
  int64_t M, V, K, ldx, gs;
  int32_t dtype;
  const uint8_t* qw;
  const float* scales;
  const int64_t* targets;
};

// x, qw, scales, targets, group_size
Head head_of(PyObject* const* a, const at::Tensor& x) {
  const at::Device dev = x.device();
  Head h;
  h.dtype = dtype_of(x, "x");
  h.ldx = matrix(x, "x", "[M, K]", -1, -1, x.scalar_type(), dev);
  h.M = x.size(0);
  h.K = x.size(1);
  h.gs = integer(a[4]);
  if (h.K % 8 || h.K < 8) refuse("K must be a multiple of 8, got %lld", (long long)h.K);
  const at::Tensor& q = tensor(a[1], "qw");
  if (q.dim() != 2) refuse("qw must be uint8 [vocab, %lld], got %s", (long long)(h.K / 2), shape(q).c_str());
  h.V = q.size(0);
  h.qw = (const uint8_t*)dense(q, "qw", {h.V, h.K / 2}, at::kByte, dev);
  const at::Tensor& s = tensor(a[2], "scales");
  const int64_t G = groups_of(h.K, h.gs);
  h.scales = h.gs == 0 ? (const float*)dense(s, "scales", {h.V}, at::kFloat, dev)
                       : (const float*)dense(s, "scales", {G, h.V}, at::kFloat, dev);
  h.targets = (const int64_t*)vector(tensor(a[3], "targets"), "targets", h.M, at::kLong, dev);
  return h;
}

// x, qw, scales, targets, group_size, order, workspace, stream -> loss, lse
PyObject* head_cross_entropy(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const Head h = head_of(a, x);
  on_gpu(x.device(), "x");
  const c10::DeviceGuard guard(x.device());
  const at::Tensor loss = at::empty({h.M}, x.options().dtype(at::kFloat));
  const at::Tensor lse = at::empty({h.M}, x.options().dtype(at::kFloat));
  const Workspace ws(a[6], given(a[6]) ? 0 : q4_head_cross_entropy_workspace_bytes(h.dtype, h.M, h.V, h.K, h.gs), x.options());
  check(q4_head_cross_entropy(x.data_ptr(), h.ldx, h.dtype, h.M, h.V, h.K, h.qw, h.scales, h.gs,
                              (int32_t)integer(a[5]), h.targets, (float*)loss.data_ptr(),
                              (float*)lse.data_ptr(), ws.p, ws.n, stream_of(a[7])),
        "q4_head_cross_entropy");
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyFailed{};
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(loss));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(lse));
  return r;
}

// x, qw, scales, targets, group_size, order, lse, g_loss, dx, workspace, stream
PyObject* head_cross_entropy_backward(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const at::Device dev = x.device();
  const Head h = head_of(a, x);
  const float* lse = (const float*)vector(tensor(a[6], "lse"), "lse", h.M, at::kFloat, dev);
  const float* g = (const float*)vector(tensor(a[7], "g_loss"), "g_loss", h.M, at::kFloat, dev);
  at::Tensor dx;
  int64_t lddx = h.K;
  if (given(a[8])) {
    dx = tensor(a[8], "dx");
    lddx = matrix(dx, "dx", "[M, K]", h.M, h.K, x.scalar_type(), dev);
  }
  on_gpu(dev, "x");
  const c10::DeviceGuard guard(dev);
  if (!dx.defined()) dx = at::empty({h.M, h.K}, x.options());
  const Workspace ws(a[9], given(a[9]) ? 0 : q4_head_cross_entropy_backward_workspace_bytes(h.dtype, h.M, h.V, h.K, h.gs), x.options());
  check(q4_head_cross_entropy_backward(x.data_ptr(), h.ldx, h.dtype, h.M, h.V, h.K, h.qw, h.scales, h.gs,
                                       (int32_t)integer(a[5]), h.targets, lse, g, dx.data_ptr(), lddx, ws.p,
                                       ws.n, stream_of(a[10])),
        "q4_head_cross_entropy_backward");
  return THPVariable_Wrap(dx);
}

}  // namespace
