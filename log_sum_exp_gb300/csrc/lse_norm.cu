// lse_norm.cu -- the C entry points of the end of a block.  Kernels: lse_norm.cuh.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "lse_internal.h"
#include "lse_norm_common.cuh"

namespace lse {
namespace {

int64_t slots_of(int D, int EB, bool vec, bool aligned) {
    const int64_t s = (static_cast<int64_t>(D) * EB + 15) / 16;
    return s + (vec && !aligned ? 1 : 0);
}

BackwardPlan plan_norm_backward(int64_t T, int64_t slots, bool f32, int sms) {
    BackwardPlan p;
    p.v = 1;
    if (slots <= 8) p.tx = 8;
    else if (slots <= 32) p.tx = 32;
    else if (slots <= 64) p.tx = 64;
    else if (slots <= 128) p.tx = 128;
    else if (slots <= 256) p.tx = 256;
    else if (slots <= 512) p.tx = 512;
    else p.tx = 1024, p.v = slots <= 1024 ? 1 : slots <= 2048 ? 2 : 5;
    const int threads = p.tx < 128 ? 128 : p.tx;
    p.rows = threads / p.tx;
    const int64_t resident = static_cast<int64_t>(sms) * backward_ctas(threads, f32) / 8 * 8;
    int64_t grid = (T + p.rows - 1) / p.rows;
    if (grid > resident) grid = resident;
    p.grid = static_cast<int>((grid + 7) / 8 * 8);
    return p;
}

// Rows of one array: pointer, distance and alignment.  Checked here so that every array of
// a call is refused for the same reasons.
struct Rows {
    const void* p;
    int64_t stride;
    bool wanted;
};

// All rows start at the same offset from a 16-byte boundary, row by row.
bool same_offsets(const Rows* rows, int n, int EB) {
    for (int i = 1; i < n; ++i) {
        if (!rows[i].p) continue;
        if ((reinterpret_cast<uintptr_t>(rows[i].p) - reinterpret_cast<uintptr_t>(rows[0].p)) % 16 != 0) return false;
        if ((rows[i].stride - rows[0].stride) * EB % 16 != 0) return false;
    }
    return true;
}

lse_status check_norm(int dtype, int64_t T, int64_t D, const Rows* rows, int n, int gate_kind, const void* gate,
                      const void* weight, const void* post, int weight_dtype, float scale, float eps) {
    if (!valid_dtype(dtype) || !valid_dtype(weight_dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    if (weight_dtype != dtype && weight_dtype != LSE_F32) return LSE_ERR_UNSUPPORTED_DTYPE;
    if (T < 0 || D < 0 || D > kNormMaxColumns || T > INT32_MAX) return LSE_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !(fabsf(scale) <= 3.4e38f)) return LSE_ERR_INVALID_ARG;
    if (gate_kind != kNoGate && gate_kind != kChannelGate && gate_kind != kElementGate) return LSE_ERR_INVALID_ARG;
    const int eb = dtype == LSE_F32 ? 4 : 2, wb = weight_dtype == LSE_F32 ? 4 : 2;
    for (int i = 0; i < n; ++i) {
        if (!rows[i].p) {
            if (rows[i].wanted && T > 0 && D > 0) return LSE_ERR_INVALID_ARG;
            continue;
        }
        int64_t extent = 0;
        if (rows[i].stride < D || misaligned(rows[i].p, eb) || __builtin_mul_overflow(T, rows[i].stride, &extent) ||
            __builtin_mul_overflow(extent, static_cast<int64_t>(eb), &extent))
            return LSE_ERR_INVALID_ARG;
    }
    if (misaligned(weight, wb) || misaligned(post, wb) || (gate_kind == kChannelGate && misaligned(gate, wb))) return LSE_ERR_INVALID_ARG;
    if (T > 0 && D > 0 && (!weight || (gate_kind != kNoGate && !gate))) return LSE_ERR_INVALID_ARG;
    return LSE_OK;
}

void set_common(NormArgs* a, int dtype, int64_t T, int64_t D, const void* x, int64_t x_stride, const void* y,
                int64_t y_stride, int gate_kind, const void* gate, int64_t gate_stride, const void* post,
                const void* weight, int weight_dtype, float scale) {
    const int64_t eb = dtype == LSE_F32 ? 4 : 2;
    a->T = T;
    a->D = static_cast<int>(D);
    a->x = static_cast<const char*>(x);
    a->y = static_cast<const char*>(y);
    a->x_bytes = x_stride * eb;
    a->y_bytes = y_stride * eb;
    a->gate_kind = gate_kind;
    a->gate = static_cast<const char*>(gate);
    a->gate_bytes = gate_stride * eb;
    a->post = static_cast<const char*>(post);
    a->weight = static_cast<const char*>(weight);
    a->weights_f32 = weight_dtype == LSE_F32;
    a->weights_vec = !misaligned(weight, 16) && !misaligned(post, 16) && (gate_kind != kChannelGate || !misaligned(gate, 16));
    a->scale = scale;
    a->inv_d = static_cast<float>(1.0 / static_cast<double>(D));
}

bool on_boundaries(const Rows& r, int eb) { return !misaligned(r.p, 16) && r.stride * eb % 16 == 0; }

int mode_of(const Rows* rows, int n, int eb, const NormArgs& a) {
    if (!same_offsets(rows, n, eb)) return kSingle;
    return on_boundaries(rows[0], eb) && a.D * eb % 16 == 0 && a.weights_vec ? kWhole : kCover;
}

}  // namespace
}  // namespace lse

using namespace lse;

extern "C" {

lse_status lse_residual_norm(const void* x, lse_dtype dtype, int64_t T, int64_t D, int64_t x_stride, const void* y,
                             int64_t y_stride, const void* gate, lse_gate gate_kind, int64_t gate_stride,
                             const void* post_weight, const void* weight, lse_dtype weight_dtype, float scale,
                             float eps, void* h, int64_t h_stride, void* out, int64_t out_stride, float* rstd,
                             float* post_rstd, lse_stream_t stream) {
    if (!y && T > 0 && D > 0) {  // nothing to add: h is x
        if (gate_kind != LSE_GATE_NONE || post_weight || h || post_rstd) return LSE_ERR_INVALID_ARG;
    }
    const Rows rows[] = {{x, x_stride, true}, {y, y_stride, false}, {h, h_stride, false}, {out, out_stride, true},
                         {gate_kind == LSE_GATE_ELEMENT ? gate : nullptr, gate_stride, false}};
    const lse_status st = check_norm(dtype, T, D, rows, 5, gate_kind, gate, weight, post_weight, weight_dtype, scale, eps);
    if (st != LSE_OK) return st;
    if (misaligned(rstd, 4) || misaligned(post_rstd, 4)) return LSE_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return LSE_OK;
    const int eb = dtype == LSE_F32 ? 4 : 2;
    NormArgs a = {};
    set_common(&a, dtype, T, D, x, x_stride, y, y_stride, gate_kind, gate, gate_stride, post_weight, weight, weight_dtype, scale);
    a.eps = eps;
    a.h = static_cast<char*>(h);
    a.h_bytes = h_stride * eb;
    a.out = static_cast<char*>(out);
    a.out_bytes = out_stride * eb;
    a.rstd = rstd;
    a.post_rstd = post_rstd;
    const int mode = mode_of(rows, 5, eb, a);
    const int64_t slots = slots_of(a.D, eb, mode != kSingle, on_boundaries(rows[0], eb));
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int sms = 0;
    lse_status found = device_sms(&sms);
    if (found != LSE_OK) return found;
    const bool few = T <= 4 * sms;
    return cuda_status(dtype == LSE_F32 ? launch_norm_f32(a, mode, slots, few, s)
                       : dtype == LSE_BF16 ? launch_norm_bf16(a, mode, slots, few, s) : launch_norm_f16(a, mode, slots, few, s));
}

lse_status lse_residual_norm_backward(const void* grad_out, int64_t grad_out_stride, const void* grad_h,
                                      int64_t grad_h_stride, const void* x, lse_dtype dtype, int64_t T, int64_t D,
                                      int64_t x_stride, const void* y, int64_t y_stride, const void* gate,
                                      lse_gate gate_kind, int64_t gate_stride, const void* post_weight,
                                      const void* weight, lse_dtype weight_dtype, float scale, const float* rstd,
                                      const float* post_rstd, void* dx, int64_t dx_stride, void* dy, int64_t dy_stride,
                                      void* dgate, int64_t dgate_stride, void* dpost_weight, void* dweight,
                                      lse_stream_t stream) {
    if (!y && T > 0 && D > 0 && (gate_kind != LSE_GATE_NONE || post_weight || dy)) return LSE_ERR_INVALID_ARG;
    if ((dgate && gate_kind == LSE_GATE_NONE) || (dpost_weight && !post_weight)) return LSE_ERR_INVALID_ARG;
    const bool by_element = gate_kind == LSE_GATE_ELEMENT;
    const Rows rows[] = {{x, x_stride, true}, {y, y_stride, false}, {grad_out, grad_out_stride, true},
                         {grad_h, grad_h_stride, false}, {by_element ? gate : nullptr, gate_stride, false},
                         {dx, dx_stride, false}, {dy, dy_stride, false}, {by_element ? dgate : nullptr, dgate_stride, false}};
    lse_status st = check_norm(dtype, T, D, rows, 8, gate_kind, gate, weight, post_weight, weight_dtype, scale, 0.0f);
    if (st != LSE_OK) return st;
    const uintptr_t wb = weight_dtype == LSE_F32 ? 4 : 2;
    if (misaligned(rstd, 4) || misaligned(post_rstd, 4) || misaligned(dweight, wb) || misaligned(dpost_weight, wb) ||
        (!by_element && misaligned(dgate, wb)))
        return LSE_ERR_INVALID_ARG;
    if (D == 0) return LSE_OK;
    if (T > 0 && (!rstd || (post_weight && !post_rstd))) return LSE_ERR_INVALID_ARG;
    const int eb = dtype == LSE_F32 ? 4 : 2;
    NormArgs a = {};
    set_common(&a, dtype, T, D, x, x_stride, y, y_stride, gate_kind, gate, gate_stride, post_weight, weight, weight_dtype, scale);
    a.dout = static_cast<const char*>(grad_out);
    a.dout_bytes = grad_out_stride * eb;
    a.dh = static_cast<const char*>(grad_h);
    a.dh_bytes = grad_h_stride * eb;
    a.rstd_in = rstd;
    a.post_rstd_in = post_rstd;
    a.dx = static_cast<char*>(dx);
    a.dx_bytes = dx_stride * eb;
    a.dy = static_cast<char*>(dy);
    a.dy_bytes = dy_stride * eb;
    a.dgate = by_element ? static_cast<char*>(dgate) : nullptr;
    a.dgate_bytes = dgate_stride * eb;
    void* const dgate_columns = by_element ? nullptr : dgate;
    const bool sums = dweight || dpost_weight || dgate_columns;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    void* scratch = nullptr;
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        int sms = 0;
        if ((st = device_sms(&sms)) != LSE_OK) return st;
        const int mode = mode_of(rows, 8, eb, a);
        const BackwardPlan p = plan_norm_backward(T, slots_of(a.D, eb, mode != kSingle, on_boundaries(rows[0], eb)), dtype == LSE_F32, sms);
        if (sums) {
            st = take_scratch(&scratch, static_cast<size_t>(p.grid) * a.D * 2 * sizeof(float), s);
            if (st != LSE_OK) return st;
            a.part = static_cast<float*>(scratch);
            a.parts = p.grid;
        }
        e = dtype == LSE_F32 ? launch_norm_backward_f32(a, mode, p, s)
            : dtype == LSE_BF16 ? launch_norm_backward_bf16(a, mode, p, s) : launch_norm_backward_f16(a, mode, p, s);
    }
    if (sums && e == cudaSuccess) {
        NormFinishArgs f;
        f.part = a.part;
        f.parts = a.parts;
        f.D = a.D;
        f.post = post_weight;
        f.gate = gate_kind == LSE_GATE_CHANNEL ? gate : nullptr;
        f.weights_f32 = a.weights_f32;
        f.scale = scale;
        f.dweight = dweight;
        f.dpost = dpost_weight;
        f.dgate = dgate_columns;
        e = dtype == LSE_F32 ? launch_norm_finish_f32(f, s) : dtype == LSE_BF16 ? launch_norm_finish_bf16(f, s) : launch_norm_finish_f16(f, s);
    }
    if (scratch) {
        const cudaError_t freed = cudaFreeAsync(scratch, s);
        if (e == cudaSuccess) e = freed;
    }
    return cuda_status(e);
}

}  // extern "C"
