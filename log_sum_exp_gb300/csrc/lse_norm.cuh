// lse_norm.cuh -- the end of a block: norm of its output, gate, residual scale, the sum with
// the residual stream and the norm of the sum, and their gradient (sm_103a).
//
//     r1 = (mean y^2 + eps)^-1/2     a = y r1 w1     (w1 absent: a = y)
//     h  = x + s g a                 r2 = (mean h^2 + eps)^-1/2     out = h r2 w
//
// Bound by memory: x and y are read once, h and out written once, and a row stays in
// registers between its two sums, which depend on each other.  The sums are taken apart
// although sum h^2 could be written in sums that do not need r1: where x and s g a cancel,
// those lose all their digits.
//
// Gradient, with G what arrives at h from both sides and the normalised rows u = h r2, v = y r1:
//
//     n = w dout     G = dh + r2 n - u r2/D sum(n u)       dx = G
//     e = s g w1 G   dy = r1 (e - v/D sum(e v))            dgate = s w1 v G  (w1 absent: s y G)
//     dw = sum over rows of dout u                         dw1 = the same of s g v G
//
// sum(e v) needs G, which needs sum(n u); with q = s g w1 v it is sum q (dh + r2 n) -
// r2/D sum(n u) sum(q u), so one reduction per row carries all three sums.  The normalised rows
// are of magnitude 1 whatever the rows are; powers of r1 and r2 would leave the f32 range long
// before any result does (r2^3 / D is 0 for rows of an rms of 1e14).
// CTAs walk over rows and keep the sums over rows for the columns of each thread in
// registers; a second kernel adds the CTAs' parts in their order, so a repeated call gives
// equal bits.  For a gate of one value per column, dw1 = g S and dgate = w1 S share the sum
// S = sum s G v.
//
// Measured: 16384 x 4096 bf16 with post norm and a gate per column 86 us (6.2 TB/s), gradient 159
// us (5.1 TB/s); 5000 x 1001 f32 with a gate per element 18 us (5.6 TB/s) and 33 us (4.8 TB/s).  The
// gradient holds 8 columns' sums, factors and terms of 16-bit rows in 116 to 128 registers, so an SM
// has 512 threads of it: loading the next row during a row's sums took it from 313 to 272 us, the
// columns' factors in registers to 204, rows without edge checks to 159.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_elem.cuh"
#include "lse_internal.h"
#include "lse_norm_common.cuh"

namespace lse {
namespace {


// ---------------------------------------------------------------------------
// A thread's share of a row: V slots of 16 bytes.  kWhole: rows and weights on 16-byte
// boundaries and of whole vectors, so that nothing is checked but the row's end; kCover: the
// aligned vectors that cover the row, which lies `off` bytes behind a boundary in every array;
// kSingle: single elements, the lanes of a group next to each other.  Elements outside the row
// are zeros.
// ---------------------------------------------------------------------------

template <int DT> struct Slot {
    static constexpr int EB = DType<DT>::bytes, E = 16 / EB;
    uint32_t w[4];
};

template <int DT> __device__ __forceinline__ void slot_floats(const Slot<DT>& s, float (&f)[Slot<DT>::E]) {
    if constexpr (DT == kF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(s.w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = word_lo<DT>(s.w[i]);
            f[2 * i + 1] = word_hi<DT>(s.w[i]);
        }
    }
}

template <int DT> __device__ __forceinline__ Slot<DT> slot_of(const float (&f)[Slot<DT>::E]) {
    Slot<DT> s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == kF32) s.w[i] = __float_as_uint(f[i]);
        else s.w[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
    }
    return s;
}

// Columns of slot j of thread t: element i is column c + i * step.
template <int DT, int TX, int MODE> struct Columns {
    static constexpr bool kAlways = MODE == kWhole;
    int c, step;
    bool whole;  // no element lies outside the row
    bool any;
    __device__ __forceinline__ Columns(int j, int t, int off_e, int D) {
        constexpr int E = Slot<DT>::E;
        if constexpr (MODE == kWhole) {
            c = (j * TX + t) * E;
            step = 1;
            whole = any = c < D;
        } else if constexpr (MODE == kCover) {
            c = (j * TX + t) * E - off_e;
            step = 1;
            whole = c >= 0 && c + E <= D;
            any = c < D;
        } else {
            c = j * E * TX + t;
            step = TX;
            whole = false;
            any = c < D;
        }
    }
};

template <int DT, class C> __device__ __forceinline__ Slot<DT> load_slot(const char* row, const C& at, int D) {
    constexpr int E = Slot<DT>::E, EB = Slot<DT>::EB;
    Slot<DT> s;
    if (at.whole) {
        const uint4 v = ld_stream16(row + static_cast<int64_t>(at.c) * EB);
        s.w[0] = v.x, s.w[1] = v.y, s.w[2] = v.z, s.w[3] = v.w;
        return s;
    }
    s.w[0] = s.w[1] = s.w[2] = s.w[3] = 0;
    if constexpr (C::kAlways) return s;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = at.c + i * at.step;
        if (c < 0 || c >= D) continue;
        if constexpr (DT == kF32) s.w[i] = reinterpret_cast<const uint32_t*>(row)[c];
        else s.w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(row)[c]) << (i % 2 * 16);
    }
    return s;
}

template <int DT, class C> __device__ __forceinline__ void store_slot(char* row, const C& at, int D, const Slot<DT>& s) {
    constexpr int E = Slot<DT>::E, EB = Slot<DT>::EB;
    if (at.whole) {
        *reinterpret_cast<uint4*>(row + static_cast<int64_t>(at.c) * EB) = make_uint4(s.w[0], s.w[1], s.w[2], s.w[3]);
        return;
    }
    if constexpr (C::kAlways) return;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = at.c + i * at.step;
        if (c < 0 || c >= D) continue;
        if constexpr (DT == kF32) reinterpret_cast<uint32_t*>(row)[c] = s.w[i];
        else reinterpret_cast<unsigned short*>(row)[c] = static_cast<unsigned short>(s.w[i / 2] >> (i % 2 * 16));
    }
}

// The same columns of a vector of weights (1 outside the row: it meets zeros only).
template <int DT, class C>
__device__ __forceinline__ void load_weights(const char* p, const C& at, int D, const NormArgs& a,
                                             float (&f)[Slot<DT>::E]) {
    constexpr int E = Slot<DT>::E;
    if (C::kAlways || (at.whole && a.weights_vec)) {
        if (DT == kF32 || a.weights_f32) {
            const char* q = p + static_cast<int64_t>(at.c) * 4;
            if (C::kAlways || (at.c & 3) == 0) {
#pragma unroll
                for (int i = 0; i < E; i += 4) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(q + i * 4));
                    f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
                }
                return;
            }
        } else if (C::kAlways || (at.c & 7) == 0) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + static_cast<int64_t>(at.c) * 2));
            Slot<DT> s;
            s.w[0] = v.x, s.w[1] = v.y, s.w[2] = v.z, s.w[3] = v.w;
            slot_floats<DT>(s, f);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = at.c + i * at.step;
        f[i] = 1.0f;
        if (c < 0 || c >= D) continue;
        f[i] = (DT == kF32 || a.weights_f32) ? __ldg(reinterpret_cast<const float*>(p) + c) : load_elem<DT>(p, c);
    }
}

// Sums of N values over the TX threads of a row, in every one of them.  `buf` holds one
// value per warp; two calls in turn take different ones, so one barrier each suffices.
template <int TX, int N> __device__ __forceinline__ void row_sums(float (&v)[N], float (*buf)[32]) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int o = (TX < 32 ? TX : 32) / 2; o > 0; o >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    }
    if constexpr (TX > 32) {
        constexpr int W = TX / 32;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = warp / W * W;
        if (lane == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) buf[n][warp] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = lane < W ? buf[n][first + lane] : 0.0f;
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            v[n] = __shfl_sync(0xffffffffu, s, 0);
        }
    }
}

template <int TX> __host__ __device__ constexpr int norm_threads() { return TX < 128 ? 128 : TX; }

// s * gate * (post weight) of a slot: what y (times r1) is multiplied by.
template <int DT, class C>
__device__ __forceinline__ void block_factors(const NormArgs& a, const C& at, const char* gate_row, float (&f)[Slot<DT>::E]) {
    constexpr int E = Slot<DT>::E;
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = a.scale;
    if (a.post) {
        float w[E];
        load_weights<DT>(a.post, at, a.D, a, w);
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] *= w[i];
    }
    if (a.gate_kind != kNoGate) {
        float g[E];
        if (a.gate_kind == kChannelGate) load_weights<DT>(a.gate, at, a.D, a, g);
        else slot_floats<DT>(load_slot<DT>(gate_row, at, a.D), g);
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] *= g[i];
    }
}

// TX threads per row, V slots per thread.
template <int DT, int TX, int V, int MODE>
__global__ void __launch_bounds__(norm_threads<TX>()) norm_kernel(NormArgs a) {
    constexpr int E = Slot<DT>::E, EB = Slot<DT>::EB;
    __shared__ float buf[2][1][32];
    pdl_trigger();
    pdl_wait();
    const int t = threadIdx.x % TX;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (norm_threads<TX>() / TX) + threadIdx.x / TX;
    const bool live = row < a.T;
    const int D = live ? a.D : 0;
    const char* xr = a.x + row * a.x_bytes;
    const char* yr = a.y ? a.y + row * a.y_bytes : nullptr;
    const char* gr = a.gate_kind == kElementGate ? a.gate + row * a.gate_bytes : nullptr;
    const int off_e = MODE == kCover ? static_cast<int>(reinterpret_cast<uintptr_t>(xr) & 15) / EB : 0;

    Slot<DT> x[V], y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const Columns<DT, TX, MODE> at(j, t, off_e, D);
        x[j].w[0] = x[j].w[1] = x[j].w[2] = x[j].w[3] = 0;
        y[j] = x[j];
        if (!at.any) continue;
        x[j] = load_slot<DT>(xr, at, D);
        if (yr) y[j] = load_slot<DT>(yr, at, D);
    }
    float r1 = 1.0f;
    if (a.post) {
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float f[E];
            slot_floats<DT>(y[j], f);
#pragma unroll
            for (int i = 0; i < E; ++i) s[0] = fmaf(f[i], f[i], s[0]);
        }
        row_sums<TX, 1>(s, buf[0]);
        r1 = 1.0f / sqrtf(fmaf(s[0], a.inv_d, a.eps));
        if (a.post_rstd && live && t == 0) a.post_rstd[row] = r1;
    }
    float h[V][E];
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const Columns<DT, TX, MODE> at(j, t, off_e, D);
        slot_floats<DT>(x[j], h[j]);
        if (yr && at.any) {
            float f[E], q[E];
            slot_floats<DT>(y[j], f);
            block_factors<DT>(a, at, gr, q);
#pragma unroll
            for (int i = 0; i < E; ++i) h[j][i] = fmaf(f[i] * r1, q[i], h[j][i]);
        }
        if (a.h && at.any) store_slot<DT>(a.h + row * a.h_bytes, at, D, slot_of<DT>(h[j]));
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] = fmaf(h[j][i], h[j][i], s[0]);
    }
    row_sums<TX, 1>(s, buf[1]);
    const float r2 = 1.0f / sqrtf(fmaf(s[0], a.inv_d, a.eps));
    if (a.rstd && live && t == 0) a.rstd[row] = r2;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const Columns<DT, TX, MODE> at(j, t, off_e, D);
        if (!at.any) continue;
        float w[E];
        load_weights<DT>(a.weight, at, D, a, w);
#pragma unroll
        for (int i = 0; i < E; ++i) h[j][i] = h[j][i] * r2 * w[i];
        store_slot<DT>(a.out + row * a.out_bytes, at, D, slot_of<DT>(h[j]));
    }
}

// ---------------------------------------------------------------------------
// Gradient.  The grid is a multiple of 8, so all rows of a group lie at the same offset
// from a 16-byte boundary and a thread's slots are the same columns in each.
// ---------------------------------------------------------------------------
// What a slot adds to a row's sums: u = h r2, the gradient that arrives at h before the norm's
// sum is taken off, and q = s g w1 v.
template <int DT> struct GradSlot {
    float u[Slot<DT>::E], gh[Slot<DT>::E], q[Slot<DT>::E];
    Slot<DT> y, gate;
};
struct GradRow {
    const char *x, *y, *gate, *dout, *dh;
    float r1, r2;
};

// The arrays' words of a slot.
template <int DT> struct GradWords {
    Slot<DT> x, y, dn, dh, gate;
};
// What columns are multiplied by, row after row: weight, and scale times post weight times a gate
// of one value per column.
template <int DT> struct GradColumns {
    float w[Slot<DT>::E], c[Slot<DT>::E];
};
template <int DT, class C>
__device__ __forceinline__ void load_columns(const NormArgs& a, const C& at, int D, GradColumns<DT>& k) {
    constexpr int E = Slot<DT>::E;
    float f[E];
#pragma unroll
    for (int i = 0; i < E; ++i) k.w[i] = 0.0f, k.c[i] = a.scale;
    if (!at.any) return;
    load_weights<DT>(a.weight, at, D, a, k.w);
    if (a.post) {
        load_weights<DT>(a.post, at, D, a, f);
#pragma unroll
        for (int i = 0; i < E; ++i) k.c[i] *= f[i];
    }
    if (a.gate_kind == kChannelGate) {
        load_weights<DT>(a.gate, at, D, a, f);
#pragma unroll
        for (int i = 0; i < E; ++i) k.c[i] *= f[i];
    }
}
template <int DT, class C>
__device__ __forceinline__ void load_words(const GradRow& r, const C& at, int D, GradWords<DT>& w) {
    w.x.w[0] = w.x.w[1] = w.x.w[2] = w.x.w[3] = 0;
    w.y = w.dn = w.dh = w.gate = w.x;
    if (!at.any) return;
    w.x = load_slot<DT>(r.x, at, D);
    if (r.y) w.y = load_slot<DT>(r.y, at, D);
    w.dn = load_slot<DT>(r.dout, at, D);
    if (r.dh) w.dh = load_slot<DT>(r.dh, at, D);
    if (r.gate) w.gate = load_slot<DT>(r.gate, at, D);
}

template <int DT>
__device__ __forceinline__ void grad_slot(const GradRow& r, const GradWords<DT>& words, const GradColumns<DT>& k, GradSlot<DT>& g,
                                          float (&n)[Slot<DT>::E], float (*sw)[Slot<DT>::E]) {
    constexpr int E = Slot<DT>::E;
    float f[E];
    g.y = words.y;
    g.gate = words.gate;
    slot_floats<DT>(words.x, g.u);
    slot_floats<DT>(words.dn, n);
    slot_floats<DT>(words.dh, g.gh);
    slot_floats<DT>(words.y, f);
    if (r.gate) {
        slot_floats<DT>(words.gate, g.q);
#pragma unroll
        for (int i = 0; i < E; ++i) g.q[i] *= k.c[i];
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) g.q[i] = k.c[i];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        g.q[i] *= f[i] * r.r1;
        g.u[i] = (g.u[i] + g.q[i]) * r.r2;
        if (sw) (*sw)[i] = fmaf(n[i], g.u[i], (*sw)[i]);
        n[i] *= k.w[i];
        g.gh[i] = fmaf(n[i], r.r2, g.gh[i]);
    }
}

// One slot per thread stays in registers between the row's sums and its gradients; more
// (rows of more than 16 KB) are loaded again, from L2: with the sums over rows they would
// take more registers than an SM has.
template <int DT, int TX, int V, int MODE>
__global__ void __launch_bounds__(norm_threads<TX>(), backward_ctas(norm_threads<TX>(), DT == kF32)) norm_backward_kernel(NormArgs a) {
    constexpr int E = Slot<DT>::E, EB = Slot<DT>::EB, G = norm_threads<TX>() / TX;
    constexpr bool kAhead = V == 1 && TX < 1024;  // (1024 threads have 64 registers each)
    constexpr int kShared = G > 1 ? TX * V * E : 1;
    __shared__ float buf[2][3][32];
    __shared__ float sums[2][kShared];
    pdl_trigger();
    pdl_wait();
    const int t = threadIdx.x % TX, group = threadIdx.x / TX;
    float sw[V][E], sp[V][E];  // sums over rows: of dw, and of dw1 or what it shares with dgate
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) sw[j][i] = sp[j][i] = 0.0f;
    int off_e = 0;
    int turn = 0;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * G + group;
    if (MODE == kCover && first < a.T)
        off_e = static_cast<int>(reinterpret_cast<uintptr_t>(a.x + first * a.x_bytes) & 15) / EB;
    const auto row_at = [&](int64_t row, GradRow* r) {
        const bool live = row < a.T;
        r->x = a.x + row * a.x_bytes;
        r->y = a.y ? a.y + row * a.y_bytes : nullptr;
        r->gate = a.gate_kind == kElementGate ? a.gate + row * a.gate_bytes : nullptr;
        r->dout = a.dout + row * a.dout_bytes;
        r->dh = a.dh ? a.dh + row * a.dh_bytes : nullptr;
        r->r1 = live && a.post ? a.post_rstd_in[row] : 1.0f;
        r->r2 = live ? a.rstd_in[row] : 0.0f;
        return live ? a.D : 0;
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    // With one slot per thread (of 512 at most) the next row is loaded while this one's sums are put together.
    GradRow r;
    GradWords<DT> words;
    GradColumns<DT> columns;
    int D = 0;
    if constexpr (kAhead) {
        load_columns<DT>(a, Columns<DT, TX, MODE>(0, t, off_e, a.D), a.D, columns);
        D = row_at(first, &r);
        load_words<DT>(r, Columns<DT, TX, MODE>(0, t, off_e, D), D, words);
    }
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * G; base < a.T; base += step, turn ^= 1) {
        const int64_t row = base + group;
        if constexpr (!kAhead) D = row_at(row, &r);
        GradSlot<DT> g;
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const Columns<DT, TX, MODE> at(j, t, off_e, D);
            float n[E];
            if constexpr (!kAhead) {
                load_words<DT>(r, at, D, words);
                load_columns<DT>(a, at, D, columns);
            }
            grad_slot<DT>(r, words, columns, g, n, &sw[j]);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                s[0] = fmaf(n[i], g.u[i], s[0]);
                s[1] = fmaf(g.q[i], g.gh[i], s[1]);
                s[2] = fmaf(g.q[i], g.u[i], s[2]);
            }
        }
        GradRow next;
        int next_D = 0;
        if constexpr (kAhead) {
            next_D = row_at(row + step, &next);
            if (row + step - group < a.T) load_words<DT>(next, Columns<DT, TX, MODE>(0, t, off_e, next_D), next_D, words);
        }
        row_sums<TX, 3>(s, buf[turn]);
        const float k2 = s[0] * a.inv_d * r.r2;
        const float k1 = a.post ? (s[1] - k2 * s[2]) * a.inv_d : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const Columns<DT, TX, MODE> at(j, t, off_e, D);
            if (!at.any) continue;
            float f[E], e[E], o[E];
            if constexpr (V > 1) {
                load_words<DT>(r, at, D, words);
                load_columns<DT>(a, at, D, columns);
                grad_slot<DT>(r, words, columns, g, f, nullptr);
            } else if constexpr (!kAhead) {
                load_columns<DT>(a, at, D, columns);
            }
            slot_floats<DT>(g.y, f);
#pragma unroll
            for (int i = 0; i < E; ++i) g.gh[i] = fmaf(-g.u[i], k2, g.gh[i]);  // G
            if (a.dx) store_slot<DT>(a.dx + row * a.dx_bytes, at, D, slot_of<DT>(g.gh));
            if (!r.y) continue;
            if (r.gate) slot_floats<DT>(g.gate, e);
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] *= r.r1;  // v
            if (a.dy) {
#pragma unroll
                for (int i = 0; i < E; ++i) o[i] = fmaf(r.gate ? columns.c[i] * e[i] : columns.c[i], g.gh[i], -f[i] * k1) * r.r1;
                store_slot<DT>(a.dy + row * a.dy_bytes, at, D, slot_of<DT>(o));
            }
            // v G: the sum that dw1 and the gate of a column share, but for the scale
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] *= g.gh[i];
            if (r.gate) {
                if (a.dgate) {
#pragma unroll
                    for (int i = 0; i < E; ++i) o[i] = f[i] * columns.c[i];
                    store_slot<DT>(a.dgate + row * a.dgate_bytes, at, D, slot_of<DT>(o));
                }
#pragma unroll
                for (int i = 0; i < E; ++i) f[i] *= e[i];
            }
#pragma unroll
            for (int i = 0; i < E; ++i) sp[j][i] += f[i];
        }
        if constexpr (kAhead) {
            r = next;
            D = next_D;
        }
    }
    if (!a.part) return;
    // The CTA's part: the groups' sums one after the other.
    const int64_t stride = static_cast<int64_t>(a.parts) * a.D;
    float* pw = a.part + static_cast<int64_t>(blockIdx.x) * a.D;
    if constexpr (G > 1) {
        for (int i = threadIdx.x; i < kShared; i += norm_threads<TX>()) sums[0][i] = sums[1][i] = 0.0f;
        for (int g = 0; g < G; ++g) {
            __syncthreads();
            if (g != group) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const Columns<DT, TX, MODE> at(j, t, off_e, a.D);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int c = at.c + i * at.step;
                    if (c < 0 || c >= a.D) continue;
                    sums[0][c] += sw[j][i];
                    sums[1][c] += sp[j][i];
                }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += norm_threads<TX>()) {
            pw[c] = sums[0][c];
            pw[stride + c] = sums[1][c];
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const Columns<DT, TX, MODE> at(j, t, off_e, a.D);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = at.c + i * at.step;
                if (c < 0 || c >= a.D) continue;
                pw[c] = sw[j][i];
                pw[stride + c] = sp[j][i];
            }
        }
    }
}

// Sums the parts of 32 columns: the warps take the parts in turn, then their sums in order.
constexpr int kFinishWarps = 32;
template <int DT> __device__ __forceinline__ float weight_at(const void* p, bool f32, int c) {
    return f32 ? __ldg(static_cast<const float*>(p) + c) : load_elem<DT>(p, c);
}
template <int DT> __device__ __forceinline__ void put_weight(void* p, bool f32, int c, float v) {
    if (DT == kF32 || f32) static_cast<float*>(p)[c] = v;
    else static_cast<unsigned short*>(p)[c] = static_cast<unsigned short>(pack2<DT == kF32 ? kBF16 : DT>(v, 0.0f));
}

template <int DT>
__global__ void __launch_bounds__(32 * kFinishWarps) norm_finish_kernel(NormFinishArgs a) {
    __shared__ float sums[2][kFinishWarps][32];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s0 = 0.0f, s1 = 0.0f;
    if (c < a.D) {
        const float* p = a.part + c;
        const int64_t stride = static_cast<int64_t>(a.parts) * a.D;
#pragma unroll 10
        for (int i = warp; i < a.parts; i += kFinishWarps) {
            s0 += p[static_cast<int64_t>(i) * a.D];
            s1 += p[static_cast<int64_t>(i) * a.D + stride];
        }
    }
    sums[0][warp][lane] = s0;
    sums[1][warp][lane] = s1;
    __syncthreads();
    if (warp != 0 || c >= a.D) return;
    s0 = s1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kFinishWarps; ++w) {
        s0 += sums[0][w][lane];
        s1 += sums[1][w][lane];
    }
    s1 *= a.scale;
    const bool f32 = DT == kF32 || a.weights_f32;
    if (a.dweight) put_weight<DT>(a.dweight, f32, c, s0);
    if (a.dpost) put_weight<DT>(a.dpost, f32, c, a.gate ? s1 * weight_at<DT>(a.gate, f32, c) : s1);
    if (a.dgate) put_weight<DT>(a.dgate, f32, c, a.post ? s1 * weight_at<DT>(a.post, f32, c) : s1);
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <int DT, int MODE>
cudaError_t launch_norm(const NormArgs& a, int64_t slots, bool few, cudaStream_t s) {
    const auto go = [&](auto kernel, int tx) {
        const int threads = tx < 128 ? 128 : tx;
        const int64_t grid = (a.T + threads / tx - 1) / (threads / tx);
        return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads), s, a);
    };
    if (slots <= 16) return go(norm_kernel<DT, 8, 2, MODE>, 8);
    if (slots <= 64) return go(norm_kernel<DT, 32, 2, MODE>, 32);
    if (slots <= 128) return go(norm_kernel<DT, 32, 4, MODE>, 32);
    if (slots <= 256) return go(norm_kernel<DT, 128, 2, MODE>, 128);
    // Rows by the thousand: four slots per thread wait less at the rows' sums (16384 x 4096 bf16 82 us,
    // one slot 139; 8192 x 8192 86, two slots 104).  A few: fewer slots answer sooner (300 x 4096 3.1
    // us, four slots 4.7; 300 x 8192 4.3 and 5.5).
    if (slots <= 512) return few ? go(norm_kernel<DT, 512, 1, MODE>, 512) : go(norm_kernel<DT, 128, 4, MODE>, 128);
    if (slots <= 1024) return few ? go(norm_kernel<DT, 512, 2, MODE>, 512) : go(norm_kernel<DT, 256, 4, MODE>, 256);
    if (slots <= 2048) return go(norm_kernel<DT, 1024, 2, MODE>, 1024);
    if constexpr (DT != kF32) {
        return go(norm_kernel<DT, 1024, 3, MODE>, 1024);
    } else {
        if (slots <= 4096) return go(norm_kernel<DT, 1024, 4, MODE>, 1024);
        return go(norm_kernel<DT, 1024, 5, MODE>, 1024);
    }
}

template <int DT, int MODE>
cudaError_t launch_norm_backward(const NormArgs& a, const BackwardPlan& p, cudaStream_t s) {
    const auto go = [&](auto kernel, int threads) {
        return launch_pdl(kernel, dim3(static_cast<unsigned>(p.grid)), dim3(threads), s, a);
    };
    switch (p.tx) {
    case 8: return go(norm_backward_kernel<DT, 8, 1, MODE>, 128);
    case 32: return go(norm_backward_kernel<DT, 32, 1, MODE>, 128);
    case 64: return go(norm_backward_kernel<DT, 64, 1, MODE>, 128);
    case 128: return go(norm_backward_kernel<DT, 128, 1, MODE>, 128);
    case 256: return go(norm_backward_kernel<DT, 256, 1, MODE>, 256);
    case 512: return go(norm_backward_kernel<DT, 512, 1, MODE>, 512);
    default:
        return p.v == 1 ? go(norm_backward_kernel<DT, 1024, 1, MODE>, 1024)
               : p.v == 2 ? go(norm_backward_kernel<DT, 1024, 2, MODE>, 1024)
                          : go(norm_backward_kernel<DT, 1024, 5, MODE>, 1024);
    }
}

template <int DT> cudaError_t launch_norm_mode(const NormArgs& a, int mode, int64_t slots, bool few, cudaStream_t s) {
    return mode == kWhole ? launch_norm<DT, kWhole>(a, slots, few, s)
           : mode == kCover ? launch_norm<DT, kCover>(a, slots, few, s) : launch_norm<DT, kSingle>(a, slots, few, s);
}
template <int DT> cudaError_t launch_norm_backward_mode(const NormArgs& a, int mode, const BackwardPlan& p, cudaStream_t s) {
    return mode == kWhole ? launch_norm_backward<DT, kWhole>(a, p, s)
           : mode == kCover ? launch_norm_backward<DT, kCover>(a, p, s) : launch_norm_backward<DT, kSingle>(a, p, s);
}

}  // namespace
}  // namespace lse

// The launches of one element type.
#define LSE_DEFINE_NORM(DT, SUFFIX)                                                                                    \
    namespace lse {                                                                                                    \
    cudaError_t launch_norm_##SUFFIX(const NormArgs& a, int mode, int64_t slots, bool few, cudaStream_t s) {            \
        return launch_norm_mode<DT>(a, mode, slots, few, s);                                                           \
    }                                                                                                                  \
    cudaError_t launch_norm_backward_##SUFFIX(const NormArgs& a, int mode, const BackwardPlan& p, cudaStream_t s) {     \
        return launch_norm_backward_mode<DT>(a, mode, p, s);                                                           \
    }                                                                                                                  \
    cudaError_t launch_norm_finish_##SUFFIX(const NormFinishArgs& a, cudaStream_t s) {                                  \
        return launch_pdl(norm_finish_kernel<DT>, dim3((a.D + 31) / 32), dim3(32 * kFinishWarps), s, a);                \
    }                                                                                                                  \
    }
