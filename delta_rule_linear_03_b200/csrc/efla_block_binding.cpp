// efla_block_binding.cpp - the Python binding of the operators around the
// mixer: checks of types, shapes, devices and strides, outputs and scratch
// from PyTorch's allocator, and the C-ABI call on the current stream.
//
// Compiled, where the mixer's binding is ctypes, because a one-token step
// takes the GPU 2 us and the same checks and conversions in Python take 8 to
// 13.  Each function returns the call's status first; block.py turns it into
// an exception.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <climits>
#include <optional>
#include <tuple>
#include <vector>

#include "../../include/efla.h"

namespace {

using at::IntArrayRef;
using at::Tensor;
using Opt = std::optional<Tensor>;
using Dims = c10::SmallVector<int64_t, 5>;

// A size as the C ABI takes it.
int extent(const Tensor &t, int64_t i) {
    const int64_t n = t.size(i);
    TORCH_CHECK_VALUE(n <= INT_MAX, "sizes end at 2^31 - 1, got ", n);
    return (int)n;
}

std::string text(IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

void held(const Tensor &t, IntArrayRef shape, at::ScalarType type, int dev, const char *name) {
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape, name, " must be ", type, " ", text(shape), ", got ",
                      t.scalar_type(), " ", text(t.sizes()));
    TORCH_CHECK_VALUE(t.get_device() == dev, name, " must be on cuda:", dev, ", as the first argument is");
}

// A contiguous tensor of this shape, type and device.
void want(const Tensor &t, IntArrayRef shape, at::ScalarType type, int dev, const char *name) {
    held(t, shape, type, dev, name);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}
void want(const Opt &t, IntArrayRef shape, at::ScalarType type, int dev, const char *name) {
    if (t) want(*t, shape, type, dev, name);
}

// Device index of the activation that the others are held to.
int first(const Tensor &t, const char *name) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16, name,
                     " must be float32 or bfloat16, got ", t.scalar_type());
    return t.get_device();
}

efla_dtype_t code(at::ScalarType t) { return t == at::kFloat ? EFLA_F32 : EFLA_BF16; }
efla_dtype_t code(const Tensor &t) { return code(t.scalar_type()); }

// Elements from one token to the next of a tensor whose first `lead`
// dimensions count tokens: each token's values are contiguous, and the tokens
// evenly spaced.
long long rows(const Tensor &t, IntArrayRef shape, int lead, at::ScalarType type, int dev, const char *name) {
    held(t, shape, type, dev, name);
    const int n = (int)shape.size();
    long long width = 1;
    for (int i = lead; i < n; ++i) width *= shape[i];
    if (t.is_contiguous()) return width;
    const IntArrayRef stride = t.strides();
    long long step = 1, ld = -1;
    for (int i = n - 1; i >= lead; --i) {  // inside a token
        TORCH_CHECK_VALUE(shape[i] == 1 || stride[i] == step, "the values of one token of ", name, " must be contiguous");
        step *= shape[i];
    }
    for (int i = lead - 1; i >= 0; --i) {  // from token to token
        if (shape[i] == 1) continue;
        if (ld < 0) {
            ld = stride[i];
            step = ld * shape[i];
            TORCH_CHECK_VALUE(ld >= width, "the tokens of ", name, " must not overlap");
        } else {
            TORCH_CHECK_VALUE(stride[i] == step, "the tokens of ", name, " must be evenly spaced over the batch");
            step *= shape[i];
        }
    }
    return ld < 0 ? width : ld;
}

const void *ptr(const Tensor &t) { return t.const_data_ptr(); }
const void *ptr(const Opt &t) { return t ? t->const_data_ptr() : nullptr; }
const float *f32(const Tensor &t) { return t.const_data_ptr<float>(); }
const float *f32(const Opt &t) { return t ? t->const_data_ptr<float>() : nullptr; }
const int *i32(const Opt &t) { return t ? t->const_data_ptr<int>() : nullptr; }
void *out(const Tensor &t) { return t.mutable_data_ptr(); }
void *out(const Opt &t) { return t ? t->mutable_data_ptr() : nullptr; }
float *fout(const Tensor &t) { return t.mutable_data_ptr<float>(); }
float *fout(const Opt &t) { return t ? t->mutable_data_ptr<float>() : nullptr; }

// Straight from the allocator: the dispatcher's way there takes as long again.
Tensor fresh(const Tensor &like, IntArrayRef shape, at::ScalarType type) {
    return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}
Tensor fresh(const Tensor &like, IntArrayRef shape) { return fresh(like, shape, like.scalar_type()); }

// A caller's output, checked, or a new one.
Tensor output(const Opt &given, const Tensor &like, IntArrayRef shape, at::ScalarType type, int dev, const char *name) {
    if (!given) return fresh(like, shape, type);
    want(*given, shape, type, dev, name);
    return *given;
}

// The current stream of the tensors' device, which is made current for the call.
struct Call {
    c10::cuda::OptionalCUDAGuard guard;
    efla_stream_t stream;
    explicit Call(int dev) {
        if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
        stream = reinterpret_cast<efla_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
    }
};

// The caller's scratch where it is large enough, else a new one.
struct Scratch {
    Tensor t;
    void *p = nullptr;
    size_t n = 0;
    Scratch(size_t need, const Opt &given, const Tensor &like) {
        if (!need) return;
        if (given && given->nbytes() >= need) {
            TORCH_CHECK_VALUE(given->device() == like.device() && given->is_contiguous(), "workspace must be contiguous and on ",
                              like.device());
            t = *given;
        } else {
            t = fresh(like, {(int64_t)need}, at::kByte);
        }
        p = t.mutable_data_ptr();
        n = t.nbytes();
    }
};

// ------------------------------------------------------------------------------------------------- norm

std::tuple<int, Tensor, Opt, Opt> norm_fwd(const Tensor &x, const Tensor &weight, const Opt &residual, double eps, bool out8,
                                           int64_t group, const Opt &y_, const Opt &scale_, const Opt &res_out_) {
    const int dev = first(x, "x");
    const auto T = x.scalar_type();
    TORCH_CHECK_VALUE(x.dim() > 0, "x must have a last dimension to norm over");
    const IntArrayRef shape = x.sizes();
    const int C = extent(x, -1);
    const int64_t rows = C ? x.numel() / C : 0;
    want(x, shape, T, dev, "x");
    want(weight, {C}, at::kFloat, dev, "weight");
    Opt res_out, scale;
    if (residual) {
        const auto RT = residual->scalar_type();
        TORCH_CHECK_TYPE(RT == T || RT == at::kFloat, "residual must be float32 or ", T, ", got ", RT);
        want(*residual, shape, RT, dev, "residual");
        res_out = output(res_out_, x, shape, RT, dev, "res_out");
    } else {
        TORCH_CHECK_VALUE(!res_out_, "res_out needs a residual");
    }
    TORCH_CHECK_VALUE(group == 0 || group == 128, "group must be 128 or 0");
    const Tensor y = output(y_, x, shape, out8 ? at::kFloat8_e4m3fn : T, dev, "y");
    if (out8) {
        Dims groups(shape.begin(), shape.end());
        groups.back() = group ? (C + 127) / 128 : 1;
        scale = output(scale_, x, groups, at::kFloat, dev, "scale");
    } else {
        TORCH_CHECK_VALUE(!scale_, "scale is written with out8 only");
    }
    const Call call(dev);
    const int s = efla_norm_fwd(ptr(x), code(T), ptr(residual), residual ? code(*residual) : code(T), f32(weight), (float)eps,
                                out8 ? nullptr : out(y), out8 ? out(y) : nullptr, fout(scale), (int)group, out(res_out), rows, C,
                                call.stream);
    return {s, y, scale, res_out};
}

std::tuple<int, Tensor, Tensor, Tensor> norm_bwd(const Tensor &dy, const Tensor &h, const Tensor &weight, const Opt &dres_out,
                                                 double eps, const Opt &workspace) {
    const int dev = first(dy, "dy");
    const auto T = dy.scalar_type(), HT = h.scalar_type();
    TORCH_CHECK_VALUE(dy.dim() > 0, "dy must have a last dimension");
    const IntArrayRef shape = dy.sizes();
    const int C = extent(dy, -1);
    const int64_t rows = C ? dy.numel() / C : 0;
    TORCH_CHECK_TYPE(HT == T || HT == at::kFloat, "h must be float32 or ", T, ", got ", HT);
    want(dy, shape, T, dev, "dy");
    want(h, shape, HT, dev, "h");
    want(dres_out, shape, HT, dev, "dres_out");
    want(weight, {C}, at::kFloat, dev, "weight");
    const Tensor dx = fresh(dy, shape), dres = HT == T ? dx : fresh(h, shape), dw = fresh(dy, {C}, at::kFloat);
    const Call call(dev);
    const Scratch ws(efla_norm_bwd_workspace_size(rows, C), workspace, dy);
    const int s = efla_norm_bwd(ptr(dy), code(T), ptr(h), code(HT), f32(weight), (float)eps, ptr(dres_out), out(dx),
                                HT == T ? nullptr : out(dres), fout(dw), rows, C, ws.p, ws.n, call.stream);
    return {s, dx, dres, dw};
}

// ------------------------------------------------------------------------------------------------- conv

struct Conv {
    int dev, B, L, C, K;
    at::ScalarType T;
    long long ldx;
    Dims shape;  // of y
    Conv(const Tensor &x, const Tensor &weight, const Opt &bias, const Opt &state, const Opt &lengths, int64_t heads)
        : dev(first(x, "x")), T(x.scalar_type()) {
        TORCH_CHECK_VALUE(x.dim() == 3 && weight.dim() == 2, "x must be [B,L,C] and weight [C,K]");
        B = extent(x, 0), L = extent(x, 1), C = extent(x, 2), K = extent(weight, 1);
        ldx = rows(x, x.sizes(), 2, T, dev, "x");
        want(weight, {C, K}, at::kFloat, dev, "weight");
        want(bias, {C}, at::kFloat, dev, "bias");
        want(state, {B, K - 1, C}, T, dev, "state");
        want(lengths, {B}, at::kInt, dev, "lengths");
        TORCH_CHECK_VALUE(heads >= 0 && heads <= INT_MAX && (!heads || C % heads == 0), "heads must divide the channels");
        if (heads) shape = {B, heads, L, C / heads};
        else shape = {B, L, C};
    }
};

std::tuple<int, Tensor, Opt> conv_fwd(const Tensor &x, const Tensor &weight, const Opt &bias, const Opt &state,
                                      const Opt &lengths, bool silu, int64_t heads, bool want_state, const Opt &y_,
                                      const Opt &state_out_) {
    const Conv c(x, weight, bias, state, lengths, heads);
    const Tensor y = output(y_, x, c.shape, c.T, c.dev, "y");
    Opt so;
    if (state_out_ || want_state) so = output(state_out_, x, {c.B, c.K - 1, c.C}, c.T, c.dev, "state_out");
    const Call call(c.dev);
    const int s = efla_conv_fwd(ptr(x), c.ldx, code(c.T), f32(weight), f32(bias), ptr(state), i32(lengths), silu, out(y),
                                (int)heads, out(so), c.B, c.L, c.C, c.K, call.stream);
    return {s, y, so};
}

std::tuple<int, Tensor, Tensor, Opt, Opt> conv_bwd(const Tensor &dy, const Tensor &x, const Tensor &weight, const Opt &bias,
                                                   const Opt &state, const Opt &lengths, bool silu, int64_t heads,
                                                   const Opt &dstate_out, const Opt &workspace) {
    const Conv c(x, weight, bias, state, lengths, heads);
    want(dy, c.shape, c.T, c.dev, "dy");
    want(dstate_out, {c.B, c.K - 1, c.C}, c.T, c.dev, "dstate_out");
    const Tensor dx = fresh(x, {c.B, c.L, c.C}), dw = fresh(x, {c.C, c.K}, at::kFloat);
    Opt db, ds;
    if (bias) db = fresh(x, {c.C}, at::kFloat);
    if (state) ds = fresh(x, {c.B, c.K - 1, c.C});
    const Call call(c.dev);
    const Scratch ws(efla_conv_bwd_workspace_size(c.B, c.L, c.C, c.K), workspace, x);
    const int s = efla_conv_bwd(ptr(dy), ptr(x), c.ldx, code(c.T), f32(weight), f32(bias), ptr(state), i32(lengths), silu,
                                (int)heads, ptr(dstate_out), out(dx), fout(dw), fout(db), out(ds), c.B, c.L, c.C, c.K, ws.p,
                                ws.n, call.stream);
    return {s, dx, dw, db, ds};
}

std::tuple<int, Tensor> conv_step(const Tensor &x, const Opt &state, const Tensor &weight, const Opt &bias, bool silu,
                                  const Opt &y_) {
    const int dev = first(x, "x");
    const auto T = x.scalar_type();
    TORCH_CHECK_VALUE(x.dim() == 2 && weight.dim() == 2, "x must be [B,C] and weight [C,K]");
    const int B = extent(x, 0), C = extent(x, 1), K = extent(weight, 1);
    const long long ldx = rows(x, x.sizes(), 1, T, dev, "x");
    want(weight, {C, K}, at::kFloat, dev, "weight");
    want(bias, {C}, at::kFloat, dev, "bias");
    TORCH_CHECK_VALUE(state, "state must be given");
    want(*state, {B, K - 1, C}, T, dev, "state");
    const Tensor y = output(y_, x, {B, C}, T, dev, "y");
    const Call call(dev);
    const int s = efla_conv_step(ptr(x), ldx, code(T), out(state), f32(weight), f32(bias), silu, out(y), B, C, K,
                                 call.stream);
    return {s, y};
}

// ------------------------------------------------------------------------------------------------- scan

struct Scan {
    int dev, B, L, C, G, N;
    at::ScalarType T;
    Dims shape, bc;  // of x; of Bm
    long long ldx, lddt, ldb, ldc, ldz;
    Scan(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm, const Tensor &Cm, const Opt &D, const Opt &z,
         const Opt &bias, const Opt &lengths, int lead)
        : dev(first(x, "x")), T(x.scalar_type()) {
        TORCH_CHECK_VALUE(x.dim() == lead + 1 && A.dim() == 2 && Bm.dim() == lead + 2,
                          lead == 2 ? "x must be [B,L,C], A [C,N] and Bm [B,L,G,N]" : "x must be [B,C], A [C,N] and Bm [B,G,N]");
        shape.assign(x.sizes().begin(), x.sizes().end());
        B = extent(x, 0), L = lead == 2 ? extent(x, 1) : 1, C = extent(x, lead);
        N = extent(A, 1), G = extent(Bm, lead);
        bc.assign(shape.begin(), shape.begin() + lead);
        bc.push_back(G);
        bc.push_back(N);
        ldx = rows(x, shape, lead, T, dev, "x");
        lddt = rows(dt, shape, lead, T, dev, "dt");
        ldb = rows(Bm, bc, lead, T, dev, "Bm");
        ldc = rows(Cm, bc, lead, T, dev, "Cm");
        ldz = z ? rows(*z, shape, lead, T, dev, "z") : C;
        want(A, {C, N}, at::kFloat, dev, "A");
        want(D, {C}, at::kFloat, dev, "D");
        want(bias, {C}, at::kFloat, dev, "dt_bias");
        want(lengths, {B}, at::kInt, dev, "lengths");
        TORCH_CHECK_VALUE(G > 0 && C % G == 0, "the groups of Bm and Cm must divide the channels");
    }
};

std::tuple<int, Tensor, Opt> scan_fwd(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm, const Tensor &Cm,
                                      const Opt &D, const Opt &z, const Opt &bias, const Opt &h0, const Opt &lengths,
                                      bool softplus, bool want_state, const Opt &y_, const Opt &h_L_, const Opt &workspace) {
    const Scan c(x, dt, A, Bm, Cm, D, z, bias, lengths, 2);
    want(h0, {c.B, c.C, c.N}, at::kFloat, c.dev, "h0");
    const Tensor y = output(y_, x, c.shape, c.T, c.dev, "y");
    Opt hL;
    if (h_L_ || want_state) hL = output(h_L_, x, {c.B, c.C, c.N}, at::kFloat, c.dev, "h_L");
    const Call call(c.dev);
    const Scratch ws(efla_scan_fwd_workspace_size(c.B, c.L, c.C, c.G, c.N), workspace, x);
    const int s = efla_scan_fwd(ptr(x), c.ldx, ptr(dt), c.lddt, f32(A), ptr(Bm), c.ldb, ptr(Cm), c.ldc, f32(D), ptr(z), c.ldz,
                                f32(bias), f32(h0), i32(lengths), code(c.T), softplus, out(y), fout(hL), c.B, c.L, c.C, c.G,
                                c.N, ws.p, ws.n, call.stream);
    return {s, y, hL};
}

std::tuple<int, Tensor, Tensor, Tensor, Tensor, Tensor, Opt, Opt, Opt, Tensor> scan_bwd(
    const Tensor &dy, const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm, const Tensor &Cm, const Opt &D,
    const Opt &z, const Opt &bias, const Opt &h0, const Opt &lengths, bool softplus, const Opt &dh_L, const Opt &workspace) {
    const Scan c(x, dt, A, Bm, Cm, D, z, bias, lengths, 2);
    const Dims state{c.B, c.C, c.N};
    want(h0, state, at::kFloat, c.dev, "h0");
    want(dh_L, state, at::kFloat, c.dev, "dh_L");
    want(dy, c.shape, c.T, c.dev, "dy");
    const Tensor dx = fresh(x, c.shape), ddt = fresh(x, c.shape), dA = fresh(x, {c.C, c.N}, at::kFloat);
    const Tensor dB = fresh(x, c.bc), dC = fresh(x, c.bc), dh0 = fresh(x, state, at::kFloat);
    Opt dD, dz, db;
    if (D) dD = fresh(x, {c.C}, at::kFloat);
    if (z) dz = fresh(x, c.shape);
    if (bias) db = fresh(x, {c.C}, at::kFloat);
    const Call call(c.dev);
    const Scratch ws(efla_scan_bwd_workspace_size(c.B, c.L, c.C, c.G, c.N), workspace, x);
    const int s = efla_scan_bwd(ptr(dy), ptr(x), c.ldx, ptr(dt), c.lddt, f32(A), ptr(Bm), c.ldb, ptr(Cm), c.ldc, f32(D), ptr(z),
                                c.ldz, f32(bias), f32(h0), i32(lengths), f32(dh_L), code(c.T), softplus, out(dx), out(ddt),
                                fout(dA), out(dB), out(dC), fout(dD), out(dz), fout(db), fout(dh0), c.B, c.L, c.C, c.G, c.N,
                                ws.p, ws.n, call.stream);
    return {s, dx, ddt, dA, dB, dC, dD, dz, db, dh0};
}

std::tuple<int, Tensor> scan_step(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm, const Tensor &Cm,
                                  const Opt &h, const Opt &D, const Opt &z, const Opt &bias, bool softplus, const Opt &y_) {
    const Scan c(x, dt, A, Bm, Cm, D, z, bias, Opt(), 1);
    TORCH_CHECK_VALUE(h, "h must be given");
    want(*h, {c.B, c.C, c.N}, at::kFloat, c.dev, "h");
    const Tensor y = output(y_, x, c.shape, c.T, c.dev, "y");
    const Call call(c.dev);
    const int s = efla_scan_step(ptr(x), c.ldx, ptr(dt), c.lddt, f32(A), ptr(Bm), c.ldb, ptr(Cm), c.ldc, f32(D), ptr(z), c.ldz,
                                 f32(bias), code(c.T), softplus, fout(h), out(y), c.B, c.C, c.G, c.N, call.stream);
    return {s, y};
}

}  // namespace

PYBIND11_MODULE(_efla_block, m) {
    m.attr("torch_version") = EFLA_TORCH_VERSION;  // that of the headers and libraries this is built against
    m.def("norm_fwd", &norm_fwd);
    m.def("norm_bwd", &norm_bwd);
    m.def("conv_fwd", &conv_fwd);
    m.def("conv_bwd", &conv_bwd);
    m.def("conv_step", &conv_step);
    m.def("scan_fwd", &scan_fwd);
    m.def("scan_bwd", &scan_bwd);
    m.def("scan_step", &scan_step);
    m.def("token_stride", [](const Tensor &t, int lead) { return rows(t, t.sizes(), lead, t.scalar_type(), t.get_device(), "t"); });
}
